"""The references of the gated delta rule and of rotary positions against their definitions and differences (CPU)."""
import numpy as np
import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_fwd_amd as ssd


def inputs(T, H, dk, dv, seed):
    r = np.random.default_rng(seed)
    q, k = r.standard_normal((2, T, H, dk))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    return dict(q=q, k=k, v=r.standard_normal((T, H, dv)), g=-r.random((T, H)), beta=r.random((T, H)),
                init=r.standard_normal((H, dv, dk))), r


def test_state_answers_its_key():
    """With beta = 1 a key just written is answered by its value, whatever the state held."""
    d, _ = inputs(9, 2, 8, 6, 1)
    o, S = ref.forward(d["k"], d["k"], d["v"], d["g"], np.ones((9, 2)), 1.0, d["init"])
    assert np.allclose(o, d["v"])


def test_gradients_against_differences():
    d, r = inputs(7, 2, 5, 4, 2)
    do, dfinal = r.standard_normal(d["v"].shape), r.standard_normal(d["init"].shape)

    def loss(x):
        o, S = ref.forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, x["init"])
        return (o * do).sum() + (S * dfinal).sum()

    g = ref.backward(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.7, do, d["init"], dfinal)
    for name, out in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dlog_decay"), ("beta", "dbeta"), ("init", "dinit")):
        for _ in range(5):
            way = r.standard_normal(d[name].shape)
            h = 1e-5
            plus, minus = (loss(dict(d, **{name: d[name] + s * way})) for s in (h, -h))
            assert abs((plus - minus) / (2 * h) - (g[out] * way).sum()) < 1e-6 * (1 + abs((g[out] * way).sum())), name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_reference(layout):
    """Lengths stay, positions add up, and what is turned back is what it was."""
    r = np.random.default_rng(3)
    x, freq = r.standard_normal((4, 3, 16)), 100.0 ** -np.arange(0, 1, 0.2)
    y = ref.rotate(x, np.array([3, 7, 0, 100000]), freq, layout, 1.0)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.array_equal(y[..., 10:], x[..., 10:]) and np.allclose(y[2], x[2])
    assert np.allclose(ref.rotate(y, np.array([3, 7, 0, 100000]), freq, layout, 1.0, inverse=True), x)
    assert np.allclose(ref.rotate(ref.rotate(x, np.full(4, 5), freq, layout, 1.0), np.full(4, 6), freq, layout, 1.0),
                       ref.rotate(x, np.full(4, 11), freq, layout, 1.0))


def test_rotary_frequencies():
    plain, one = ssd.rotary_frequencies(64)
    want = torch.tensor([10000.0 ** (-2 * i / 64) for i in range(32)])
    assert one == 1.0 and plain.dtype == torch.float32 and torch.allclose(plain, want)
    assert torch.allclose(ssd.rotary_frequencies(64, scaling="linear", factor=4.0)[0], want / 4)
    ntk = ssd.rotary_frequencies(64, scaling="ntk", factor=4.0)[0]
    assert ntk[0] == 1.0 and torch.allclose(ntk[-1], want[-1] / 4)
    parts, scale = ssd.rotary_frequencies(64, scaling="by_parts", factor=4.0, original_length=4096)
    turns = 4096 * want / (2 * np.pi)
    assert torch.allclose(parts[turns > 32], want[turns > 32]) and torch.allclose(parts[turns < 1], want[turns < 1] / 4)
    assert ((parts <= want * 1.000001) & (parts >= want / 4.000001)).all() and abs(scale - 1 - 0.1 * np.log(4)) < 1e-12
    for bad in (dict(rot=3), dict(rot=0), dict(rot=8, scaling="other"), dict(rot=8, base=-1.0), dict(rot=8, scaling="linear", factor=0.0),
                dict(rot=8, scaling="by_parts", factor=2.0), dict(rot=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            ssd.rotary_frequencies(**bad)

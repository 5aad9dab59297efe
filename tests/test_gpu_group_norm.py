"""GPU: group norm over channels-last rows against its definition in 64 bits.

Bounds. xh is u - mean over the deviation: the mean's and the deviation's sums
have M terms joined in trees and runs of at most M / 256 + 300 terms, so each is
off by at most c = (M / 256 + 300) 2^-24 of its terms' absolute sum; u itself is
exact, or a product with a silu of a few 2^-24. With |mean| up to a few
deviations that is at most 4 c on xh's scale max(1, |xh|) (|mean| rstd enters
once). The activation and the gate add a few 2^-23 relative. So fp32:
|err| <= 8 c (1 + |mean| rstd) (1 + |t|) |w| (1 + |gate|) scale; bf16 adds one
rounding of the output, 2^-8 |ref|.
"""
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
import ssd_chunked_scan_fwd_amd as ssd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


# samples, positions, channels, groups
SHAPES = [(1, 1, 1, 1), (5, 1, 64, 4), (33, 1, 2048, 16), (7, 1, 5120, 1), (3, 1, 8192, 1), (2, 1, 10240, 1), (9, 1, 70, 10),
          (2, 1, 3001, 1), (1, 2, 8, 1), (2, 37, 320, 32), (3, 1000, 40, 4), (1, 4097, 16, 2), (2, 65, 1032, 3), (5, 3, 21, 3),
          (2, 300, 7, 7), (700, 1, 256, 8), (1500, 1, 24, 3)]
FORMS = [("none", "", True), ("silu", "", True), ("none", "after", True), ("silu", "after", False), ("none", "before", False),
         ("silu", "before", True)]


def inputs(shape, dtype, gate, seed, offset=0.5):
    n, s, C, G = shape
    g = torch.Generator().manual_seed(seed)
    dims = (n, C) if s == 1 else (n, s, C)
    r = lambda *d: torch.randn(*d, generator=g)
    return dict(x=(r(*dims) * 2 + offset).to(dtype).cuda(), z=r(*dims).to(dtype).cuda() if gate else None,
                dy=r(*dims).to(dtype).cuda(), w=(1 + 0.2 * r(C)).cuda(), b=(0.2 * r(C)).cuda())


def want(d, shape, act, gate, center, eps, dy=True):
    n, s, C, G = shape
    v = lambda t: None if t is None else n64(t).reshape(n, s, C)
    return ref.norm(v(d["x"]), G, n64(d["w"]), n64(d["b"]), v(d["z"]), eps, act, gate, center, v(d["dy"]) if dy else None)


def hold(got, w, scale, dtype, c, what):
    got = n64(got).reshape(w.shape)
    assert np.all(np.isfinite(got)), what
    allow = c * scale + (2.0 ** -8 * abs(w) if dtype == BF else 0) + 1e-30
    worst = float(np.max(abs(got - w) / allow))
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_norm(shape, form, dtype):
    n, s, C, G = shape
    act, gate, center = form
    print(f"[norm] {shape} {form} {dtype}", flush=True)
    sys.stdout.flush()
    d = inputs(shape, dtype, gate, seed=C + s)
    eps = 1e-5
    y, stats = ssd.group_norm(d["x"], G, d["w"], d["b"], d["z"], eps, act, gate or "after", center)
    # the gradients are taken at the stats the forward call left
    g = ssd.group_norm_bwd(d["x"], G, stats, d["dy"], d["w"], d["b"], d["z"], act, gate or "after", center)
    torch.cuda.synchronize()
    w = want(d, shape, act, gate, center, eps)
    M = s * C // G
    c = (M / 256 + 300) * 2.0 ** -24
    up = lambda t: np.repeat(t, C // G, 1)[:, None, :]
    ratio = 1 + abs(up(w["mean"] * w["rstd"]))
    zz = 1.0 if d["z"] is None else 1 + abs(n64(d["z"]).reshape(n, s, C))
    scale = 8 * ratio * (1 + abs(w["t"])) * (1 + abs(n64(d["w"]))) * (zz if gate == "after" else 1.0)
    hold(y, w["y"], scale, dtype, c, "y")
    hold(stats[..., 0], w["mean"], 1 / w["rstd"] + abs(w["mean"]) * 2, F32, c, "mean")
    hold(stats[..., 1], w["rstd"], 4 * w["rstd"] * ratio.reshape(n, G, -1)[:, :, 0] if s == 1 else 4 * w["rstd"] * (1 + abs(w["mean"] * w["rstd"])),
         F32, c, "rstd")
    # xh's own error enters every gradient, at most 16 times (slopes of silu up to 1.1, both means)
    big = 16 * ratio * (1 + abs(w["t"])) * (1 + abs(w["xh"]))
    hold(g["dx"], w["dx"], big * (w["dx_abs"] + abs(w["dx"])), dtype, c, "dx")
    if gate:
        ref_scale = w["dz_abs"] if gate == "before" else zz * abs(n64(d["dy"]).reshape(n, s, C)) * (1 + abs(w["t"])) * (1 + abs(n64(d["w"])))
        hold(g["dz"], w["dz"], big * (ref_scale + abs(w["dz"])), dtype, c, "dz")
    cw = c + (n * s / 8 + 64) * 2.0 ** -24
    hold(g["dweight"], w["dweight"], float(big.max()) * (w["dweight_abs"] + w["dbias_abs"]), F32, cw, "dweight")
    hold(g["dbias"], w["dbias"], float(big.max()) * (w["dbias_abs"] + w["dweight_abs"]), F32, cw, "dbias")


@pytest.mark.parametrize("shape", [(40, 1, 64, 4), (2, 50, 64, 4)])
def test_optional_parameters(shape):
    """Without weight, bias and stats: those of ones and zeros."""
    n, s, C, G = shape
    d = inputs(shape, F32, "", 3)
    one, zero = torch.ones(C, device="cuda"), torch.zeros(C, device="cuda")
    a, none = ssd.group_norm(d["x"], G, want_stats=False)
    b, stats = ssd.group_norm(d["x"], G, one, zero)
    assert none is None and torch.equal(a, b)
    ga = ssd.group_norm_bwd(d["x"], G, stats, d["dy"])
    gb = ssd.group_norm_bwd(d["x"], G, stats, d["dy"], one, zero)
    assert torch.equal(ga["dx"], gb["dx"]) and ga["dweight"] is None and ga["dbias"] is None and ga["dz"] is None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(64, 1, 256, 4), (3, 40, 64, 4), (64, 1, 35, 5)])
def test_rows_in_wider_rows(shape, dtype):
    n, s, C, G = shape
    d = inputs(shape, dtype, "after", 9)
    wide = lambda t: torch.cat([torch.full_like(t[..., :8], float("nan")), t, t], -1)[..., 8:8 + C]
    x, z = wide(d["x"]), wide(d["z"])
    a, sa = ssd.group_norm(x, G, d["w"], d["b"], z)
    b, sb = ssd.group_norm(d["x"], G, d["w"], d["b"], d["z"])
    assert torch.equal(a, b) and torch.equal(sa, sb)
    ga = ssd.group_norm_bwd(x, G, sa, d["dy"], d["w"], d["b"], z)
    gb = ssd.group_norm_bwd(d["x"], G, sb, d["dy"], d["w"], d["b"], d["z"])
    for k in gb:
        assert torch.equal(ga[k], gb[k]), k


@pytest.mark.parametrize("shape", [(4, 1, 512, 2), (2, 600, 16, 2)])
def test_far_mean(shape):
    """A mean of 1000 deviations: nothing is lost to a difference of large sums."""
    n, s, C, G = shape
    d = inputs(shape, F32, "", 5, offset=2000.0)
    y, stats = ssd.group_norm(d["x"], G, d["w"], d["b"])
    w = want(d, shape, "none", "", True, 1e-5, dy=False)
    # the mean is held to 2^-24 of 2000 in a few roundings: 1e-3 of a deviation at most
    assert np.max(abs(n64(y).reshape(w["y"].shape) - w["y"])) <= 3e-3
    assert np.max(abs(n64(stats[..., 1]) / w["rstd"] - 1)) <= 1e-4


def test_constant_rows():
    """No deviation at all: the norm is 0, not NaN."""
    for shape in ((6, 64), (2, 30, 64)):
        x = torch.full(shape, 3.5, device="cuda")
        y, stats = ssd.group_norm(x, 4)
        assert torch.all(y == 0) and torch.all(torch.isfinite(stats))
        g = ssd.group_norm_bwd(x, 4, stats, torch.ones_like(x))
        assert torch.all(torch.isfinite(g["dx"]))


def test_gate_of_large_values():
    """silu(z) at the far ends: z on one side, 0 on the other."""
    x = torch.randn(8, 64, generator=torch.Generator().manual_seed(1)).cuda()
    z = torch.full((8, 64), 80.0, device="cuda")
    z[:, ::2] = -200.0
    y, _ = ssd.group_norm(x, 2, z=z)
    p, _ = ssd.group_norm(x, 2)
    assert torch.all(y[:, ::2] == 0)
    assert torch.allclose(y[:, 1::2], 80 * p[:, 1::2], rtol=1e-6, atol=0)


def test_gradient_against_differences():
    shape = (3, 11, 24, 3)
    n, s, C, G = shape
    d = inputs(shape, F32, "before", 21)
    act, gate, center, eps = "silu", "before", True, 1e-3
    y, stats = ssd.group_norm(d["x"], G, d["w"], d["b"], d["z"], eps, act, gate, center)
    g = ssd.group_norm_bwd(d["x"], G, stats, d["dy"], d["w"], d["b"], d["z"], act, gate, center)
    base = {k: n64(d[k]) for k in ("x", "z", "w", "b")}

    def loss(v):
        r = ref.norm(v["x"], G, v["w"], v["b"], v["z"], eps, act, gate, center)
        return (r["y"] * n64(d["dy"])).sum()

    rng = np.random.default_rng(2)
    for k, gk in (("x", "dx"), ("z", "dz"), ("w", "dweight"), ("b", "dbias")):
        u = rng.standard_normal(base[k].shape)
        h = 1e-5
        up, down = dict(base), dict(base)
        up[k], down[k] = base[k] + h * u, base[k] - h * u
        diff = (loss(up) - loss(down)) / (2 * h)
        got = (n64(g[gk]) * u).sum()
        assert abs(diff - got) <= 2e-5 * np.abs(n64(g[gk]) * u).sum(), (k, diff, got)


@pytest.mark.parametrize("C,G", [(8192, 64), (9000, 1)])
def test_offsets_beyond_32_bits(C, G):
    """More than 2^31 elements: the last rows as in a call on them alone."""
    n = 2 ** 31 // C + 300
    x = torch.empty(n, C, dtype=BF, device="cuda").normal_()
    y, stats = ssd.group_norm(x, G)
    y1, s1 = ssd.group_norm(x[-100:], G)
    assert torch.equal(y[-100:], y1) and torch.equal(stats[-100:], s1)
    g = ssd.group_norm_bwd(x, G, stats, y)["dx"]
    assert torch.equal(g[-100:], ssd.group_norm_bwd(x[-100:], G, s1, y1)["dx"])

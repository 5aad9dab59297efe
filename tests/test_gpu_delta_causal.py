"""GPU: what is not finite in a prompt of the gated delta rule reaches what the recurrence brings it to and nothing else:
no earlier token, no other value column than its own (of v and of a state), no other head, no other sequence."""
import numpy as np
import pytest
import torch

import delta_ref as ref
from test_gpu_delta import BF, F32, arrays, cu_of, make, n64, run_fwd, say

import ssd_chunked_scan_fwd_amd as ssd

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def clone(d):
    return {n: None if x is None else x.clone() for n, x in d.items()}


def finite_but(x, bad):
    """x is finite exactly where bad is not."""
    fin = torch.isfinite(x.float())
    assert bool((fin == ~bad).all()), (int((fin & bad).sum()), int((~fin & ~bad).sum()))


def check_rest(o, want, bad, d, name):
    """Where it is not bad, o is the rule's."""
    got, w = n64(o), want.copy()
    at = bad.cpu().numpy()
    got[at] = w[at] = 0.0
    ref.check(got, w, ref.rel_forward(d["q"].shape[1], d["q"].shape[3]), d["q"].dtype == BF, name)


# Walks of one value block, of two (bf16), keys of 256, and one cut into segments.
SHAPES = [(1, 200, 4, 2, 64, 32), (3, 130, 12, 6, 128, 128), (1, 140, 2, 1, 256, 40), (1, 2600, 2, 1, 32, 24), (1, 70, 2, 2, 16, 8)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_tokens_before_are_as_they_were(shape, dtype):
    say(f"[delta causal] {shape} {dtype}")
    b, T, H, Hk, dk, dv = shape
    d = make(*shape, dtype, seed=60 + T)
    rep = H // Hk
    clean, _ = run_fwd(d)
    want = ref.batch_forward(*arrays(d), 0.5, n64(d["init"]))["o"]
    tok = torch.arange(T, device="cuda")[None, :, None, None]
    head = torch.arange(H, device="cuda")[None, None, :, None]
    col = torch.arange(dv, device="cuda")[None, None, None, :]
    row = torch.arange(b, device="cuda")[:, None, None, None]
    r = b - 1
    for i, t in enumerate(sorted({0, 1, 15, 16, 37, 63, 64, T // 2 + 3, T - 2, T - 1})):
        for name, bad in (("v", NAN), ("v", INF), ("k", NAN), ("k", -INF), ("q", NAN), ("beta", NAN), ("beta", INF), ("g", NAN)):
            if (i + len(name)) % 2 and t not in (37, 63):
                continue   # every second pair
            e = clone(d)
            key, h, j = Hk - 1, H - 1, dv - 1
            if name in ("q", "k"):
                e[name][r, t, key, (5 * t) % dk] = bad
                reach = (row == r) & (head // rep == key) & (tok >= t if name == "k" else tok == t)
            elif name == "v":
                e[name][r, t, h, j] = bad
                reach = (row == r) & (head == h) & (col == j) & (tok >= t)
            else:
                e[name][r, t, h] = bad
                reach = (row == r) & (head == h) & (tok >= t)
            reach = reach.expand(b, T, H, dv)
            o, fin = run_fwd(e)
            finite_but(o, reach)
            check_rest(o, want, reach, d, f"{name} {bad} at {t}")
            first = t // 64 * 64   # chunks before and other heads and rows do not change at all
            assert torch.equal(o[:, :first], clean[:, :first]) and torch.equal(o[:r], clean[:r])
            if name != "q":
                finite_but(fin, reach[:, -1, :, :, None].expand(b, H, dv, dk))
            else:
                assert torch.isfinite(fin).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_state_that_is_not_finite(dtype):
    say(f"[delta causal] state {dtype}")
    d = make(2, 100, 4, 2, 64, 40, dtype, seed=70)
    clean, _ = run_fwd(d)
    for bad in (NAN, INF):
        e = clone(d)
        e["init"][1, 2, 17, 5] = bad
        o, fin = run_fwd(e)
        reach = torch.zeros(2, 100, 4, 40, dtype=torch.bool, device="cuda")
        reach[1, :, 2, 17] = True
        finite_but(o, reach)
        assert torch.equal(o[~reach], clean[~reach])
        finite_but(fin, reach[:, -1, :, :, None].expand(2, 4, 40, 64))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fill", [NAN, INF])
def test_padded_batch(fill, dtype):
    """Rows of different lengths in one batch: whatever stands behind a row's end, its tokens are answered."""
    say(f"[delta causal] padded {fill} {dtype}")
    lens, d = [1, 40, 64, 90, 129], make(5, 130, 4, 2, 64, 64, dtype, seed=71)
    want = ref.batch_forward(*arrays(d), 0.5, n64(d["init"]))["o"]
    for r, n in enumerate(lens):
        for x in ("q", "k", "v", "beta", "g"):
            d[x][r, n:] = fill
    o, _ = run_fwd(d)
    for r, n in enumerate(lens):
        ref.check(n64(o[r, :n]), want[r, :n], ref.rel_forward(130, 64), dtype == BF, str(n))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_packed(dtype):
    say(f"[delta causal] packed {dtype}")
    cu = [0, 100, 100, 300, 350]
    d = make(1, 350, 2, 1, 32, 32, dtype, 37, nseq=4)
    want = ref.batch_forward(*arrays(d), 0.5, n64(d["init"]), cu)["o"]
    for name in ("v", "k", "g", "beta"):
        e = clone(d)
        e[name][0, 240] = NAN
        o, fin = run_fwd(e, cu=cu)
        reach = torch.zeros(1, 350, 2, 32, dtype=torch.bool, device="cuda")
        reach[0, 240:300] = True
        finite_but(o, reach)
        check_rest(o, want, reach, d, name)
        assert not torch.isfinite(fin[2]).any() and torch.isfinite(fin[[0, 1, 3]]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_columns_side_by_side(dtype):
    """A state's column that is not finite from the start, and tokens of the columns beside it, one after the other."""
    say(f"[delta causal] columns {dtype}")
    b, T, H, dv = 1, 150, 2, 32
    d = make(b, T, H, 1, 64, dv, dtype, seed=72)
    want = ref.batch_forward(*arrays(d), 0.5, n64(d["init"]))["o"]
    reach = torch.zeros(b, T, H, dv, dtype=torch.bool, device="cuda")
    d["init"][0, 1, 9] = NAN
    reach[0, :, 1, 9] = True
    for t, j in ((40, 8), (41, 11), (70, 10), (149, 12)):
        d["v"][0, t, 1, j] = INF
        reach[0, t:, 1, j] = True
    o, fin = run_fwd(d)
    finite_but(o, reach)
    check_rest(o, want, reach, d, "columns")
    finite_but(fin, reach[:, -1, :, :, None].expand(b, H, dv, 64))

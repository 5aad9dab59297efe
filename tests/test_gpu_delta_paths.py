"""GPU: the gated delta rule on the sizes at which a call takes another path (value blocks a workgroup, value heads of a
key head in one workgroup), and the bits of its results on ordinary inputs."""
import numpy as np
import pytest
import torch

import delta_ref as ref
from test_delta_terms import REL24, RELBF, off
from test_gpu_delta import BF, F32, arrays, check_bwd, check_fwd, make, n64, run_bwd, run_fwd, say

import ssd_chunked_scan_fwd_amd as ssd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def starts(lens):
    return [0, *np.cumsum(lens).tolist()]


# Workgroups of one block of 16 value columns enough (256) that bf16 walks take two, keys of 24 to 128, value columns that
# fill the last pair of blocks, half of it or less. Packed sequences, some of no and of one token, take one, however many.
RAGGED = [65, 0, 1, 130, 64, 2, 33, 0, 128, 70]
WIDE = [(3, 130, 12, 6, 128, 128, None), (6, 100, 16, 8, 128, 40, None), (5, 70, 20, 10, 72, 40, None), (9, 67, 16, 4, 64, 32, None),
        (5, 129, 14, 7, 64, 128, None), (4, 200, 16, 16, 24, 96, None), (7, 65, 42, 21, 24, 8, None), (4, 128, 12, 12, 40, 200, None),
        (1, 0, 20, 10, 64, 64, RAGGED), (1, 0, 27, 9, 128, 40, RAGGED), (1, 0, 26, 26, 24, 128, RAGGED)]


@pytest.mark.parametrize("shape", WIDE)
def test_two_value_blocks(shape):
    say(f"[delta paths] two value blocks {shape}")
    b, T, H, Hk, dk, dv, lens = shape
    cu = None if lens is None else starts(lens)
    units = (len(lens or []) or b) * H * -(-dv // 16)
    assert units > (256 if cu is None else 768)
    d = make(b, T or cu[-1], H, Hk, dk, dv, BF, seed=units, nseq=len(lens) if lens else None)
    check_fwd(d, cu=cu, name=str(shape))
    check_bwd(d, cu=cu, name=str(shape))
    d["init"] = d["dfinal"] = None
    check_fwd(d, 1.0, cu=cu, name=str(shape))


# Chunks times key heads of 1024 and more, in chunks of 64 (bf16) as of 32: one workgroup takes the gradients of all value
# heads of a key head, over one to four steps of 32 value columns.
MANY = [65, 130, 0, 1, 64, 63] + [2, 1, 3] * 42
SHARED = [(130, 3, 16, 8, 128, 128, None), (172, 5, 18, 6, 64, 40, None), (33, 66, 32, 16, 16, 72, None), (1, 0, 24, 8, 128, 96, MANY),
          (1, 0, 16, 8, 64, 128, MANY), (1, 0, 36, 9, 40, 40, MANY)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHARED)
def test_gradients_of_shared_heads(shape, dtype):
    say(f"[delta paths] shared heads {shape} {dtype}")
    b, T, H, Hk, dk, dv, lens = shape
    cu = None if lens is None else starts(lens)
    T = T or cu[-1]
    assert (b * -(-T // 64) if lens is None else T // 64 + len(lens)) * Hk >= 1024
    d = make(b, T, H, Hk, dk, dv, dtype, seed=T + H, nseq=len(lens) if lens else None)
    check_bwd(d, cu=cu, name=str(shape))


BITS = [(1, 300, 8, 4, 64, 64), (2, 257, 6, 6, 128, 128), (1, 520, 4, 2, 32, 96), (5, 300, 16, 8, 128, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", BITS)
def test_bits_of_ordinary_results(shape, dtype):
    """24 bits of what is computed, within the bounds that terms of 16 bits do not keep to (test_delta_terms.py)."""
    say(f"[delta paths] bits {shape} {dtype}")
    d = make(*shape, dtype, seed=3)
    o, fin = run_fwd(d)
    g = run_bwd(d)
    q, k, v, ld, beta = arrays(d)
    want = ref.batch_forward(q, k, v, ld, beta, 0.5, n64(d["init"]))
    back = ref.batch_backward(q, k, v, ld, beta, 0.5, n64(d["do"]), n64(d["init"]), n64(d["dfinal"]))
    got = dict(final=off(n64(fin), want["final"]), dinit=off(n64(g["dinit"]), back["dinit"]), dbeta=off(n64(g["dbeta"]), back["dbeta"]))
    for n, x, w in (("o", o, want["o"]), *((n, g[n], back[n]) for n in ("dq", "dk", "dv"))):
        got[n] = off(n64(x), n64(torch.tensor(w).to(dtype)) if dtype == BF else w)
    print({n: f"{x:.2e}" for n, x in got.items()}, flush=True)
    for n, x in got.items():
        back_twice = 2 if n[0] == "d" else 1   # the gradients' walk begins with what the forward one left
        assert x <= back_twice * (RELBF if dtype == BF and n in ("o", "dq", "dk", "dv") else REL24), (n, x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("equal", [False, True])
def test_beta_up_to_two(equal, dtype):
    """What a state answers is taken out up to twice (eigenvalues down to -1): I - beta k k^T has norm at most 1 still, on
    which the bounds rest. Equal keys with beta = 2 and no decay turn the state's answer over at every token."""
    say(f"[delta paths] beta up to two {equal} {dtype}")
    d = make(2, 200, 4, 2, 64, 48, dtype, 12)
    d["beta"] *= 2
    if equal:
        d["k"][:] = 0.125
        d["beta"][:] = 2.0
        d["g"][:] = 0.0
    check_fwd(d)
    check_bwd(d)
    pool, o = d["init"].clone(), []
    for t in range(3):
        o.append(ssd.gated_delta_step(pool, *(d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), scale=0.5))
    short = {n: d[n][:, :3].contiguous() for n in ("q", "k", "v", "g", "beta")}
    want = ref.batch_forward(*arrays(short), 0.5, n64(d["init"]))
    ref.check(n64(torch.stack(o, 1)), want["o"], ref.rel_forward(3, 64), dtype == BF, "o of steps")
    ref.check(n64(pool), want["final"], ref.rel_forward(3, 64), False, "state after steps")

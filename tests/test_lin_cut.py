"""Packed batches whose sequences are cut into blocks: ragged last blocks, blocks that hold nothing, sequences
shorter than a block and empty ones between cut ones, rows before the first and behind the last, both directions."""
import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd
from test_gpu_lin_attn import check_bwd, check_fwd, decays, make

BF, F32 = torch.bfloat16, torch.float32

# starts, tokens of the batch
CUS = [([0, 701, 701, 702, 2035, 2099, 3000], 3000), ([5, 5, 640, 641, 2000], 2010), ([0, 1000, 1001, 1002], 1002)]
# H, Hk, dk, dv; the last two take the scans for heads above 128, the one before blocks of several chunks
DIMS = [(4, 2, 64, 64), (2, 2, 128, 128), (2, 1, 40, 96), (2, 2, 96, 40), (24, 8, 16, 16), (1, 1, 256, 72), (2, 1, 24, 200)]


def states_kept(shape, bwd):
    """Bytes of block states: none where no sequence is cut."""
    n = ssd.lin_attn_bwd_workspace_bytes(shape) if bwd else ssd.lin_attn_workspace_bytes(shape)
    sums = shape.seqlen * shape.nheads * (shape.dk + shape.dv) * 4 if bwd and shape.nheads != shape.nkv_heads else 0
    return n - sums


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cu,T", CUS)
def test_plans_are_cut(cu, T, dims):
    """What the tests below run: should the rule come to leave these whole, they need other sizes."""
    H, Hk, dk, dv = dims
    for dtype in (BF, F32):
        t = lambda h, d: torch.empty(1, T, h, d, dtype=dtype, device="meta")
        sh = ssd.lin_attn_shape(t(H, dk), t(Hk, dk), t(Hk, dv), torch.empty(len(cu), dtype=torch.int32, device="meta"))
        block = H * dk * dv * 4
        assert states_kept(sh, False) >= (len(cu) + 3) * block
        assert states_kept(sh, True) >= 2 * (len(cu) + 3) * block


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("cu,T", CUS)
def test_packed_and_cut(cu, T, dims, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"[lin cut] {cu} {dims} {dtype}", flush=True)
    H = dims[0]
    d = make(1, T, *dims, dtype, T + dims[2], nseq=len(cu) - 1)
    for n in ("q", "k", "v", "do"):   # what lies outside the sequences is not used
        d[n][:, :cu[0]] = float("nan")
        d[n][:, cu[-1]:] = float("nan")
    keep = {n: torch.nan_to_num(t) for n, t in d.items()}
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, fin = check_fwd(keep, decays(H), 0.125, cu)
    g = check_bwd(keep, decays(H), 0.125, cu)
    o1, fin1 = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], decays(H).cuda(), cu_seqlens=cut, scale=0.125, initial_state=d["init"])
    g1 = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], decays(H).cuda(), d["do"], cu_seqlens=cut, scale=0.125, initial_state=d["init"],
                          dfinal_state=d["dfinal"], want_dinit=True)
    inside = slice(cu[0], cu[-1])
    assert torch.equal(o[:, inside], o1[:, inside]) and torch.equal(fin, fin1) and torch.equal(g["dinit"], g1["dinit"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(g[n][:, inside], g1[n][:, inside])

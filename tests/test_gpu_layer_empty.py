"""GPU: batches without tokens, entries or samples run nothing and give what the formulas do: empty results, states
as they were handed in, sums of nothing. Their other arguments are checked as ever."""
import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b,T,cu", [(1, 0, None), (3, 0, None), (0, 5, None), (1, 0, [0, 0, 0])])
def test_prompts(b, T, cu, dtype):
    H, Hk, dk, dv = 4, 2, 16, 24
    q, k, v, do = z(b, T, H, dk, dtype=dtype), z(b, T, Hk, dk, dtype=dtype), z(b, T, Hk, dv, dtype=dtype), z(b, T, H, dv, dtype=dtype)
    n = b if cu is None else len(cu) - 1
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    ld, init, dfin = z(H) - 0.1, torch.randn(n, H, dv, dk, device="cuda"), torch.randn(n, H, dv, dk, device="cuda")
    o, fin = ssd.lin_attn_fwd(q, k, v, ld, cu_seqlens=cut, initial_state=init)
    assert o.shape == (b, T, H, dv) and o.dtype == dtype and torch.equal(fin, init) and (n == 0 or fin.data_ptr() != init.data_ptr())
    o, fin = ssd.lin_attn_fwd(q, k, v, ld, cu_seqlens=cut)
    assert fin.shape == (n, H, dv, dk) and torch.all(fin == 0)
    kept = torch.full_like(init, 3.0)
    o, fin = ssd.lin_attn_fwd(q, k, v, ld, cu_seqlens=cut, initial_state=init, final_state=kept)
    assert fin is kept and torch.equal(kept, init)
    assert ssd.lin_attn_fwd(q, k, v, ld, cu_seqlens=cut, want_final=False)[1] is None
    g = ssd.lin_attn_bwd(q, k, v, ld, do, cu_seqlens=cut, dfinal_state=dfin, want_dinit=True)
    assert g["dq"].shape == q.shape and g["dk"].shape == k.shape and g["dv"].shape == v.shape and torch.equal(g["dinit"], dfin)
    assert torch.all(ssd.lin_attn_bwd(q, k, v, ld, do, cu_seqlens=cut, want_dinit=True)["dinit"] == 0)
    for bad in (dict(log_decay=z(H + 1)), dict(scale=0.0), dict(initial_state=z(n + 1, H, dv, dk)), dict(o=z(b, T, H, dv + 8, dtype=dtype)),
                dict(q=z(b, T, H, 12, dtype=dtype), k=z(b, T, Hk, 12, dtype=dtype))):
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.lin_attn_fwd(**{**dict(q=q, k=k, v=v, log_decay=ld, cu_seqlens=cut), **bad})


@pytest.mark.parametrize("slots", [True, False])
def test_step(slots):
    pool = torch.randn(5, 4, 24, 16, device="cuda")
    before = pool.clone()
    sl = torch.zeros(0, dtype=torch.int32, device="cuda") if slots else None
    o = ssd.lin_attn_step(pool, z(0, 4, 16), z(0, 2, 16), z(0, 2, 24), z(4) - 0.1, slots=sl)
    assert o.shape == (0, 4, 24) and torch.equal(pool, before)
    for bad in (dict(log_decay=z(5)), dict(scale=float("nan")), dict(state=z(5, 4, 24, 8))):
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.lin_attn_step(**{**dict(state=pool, q=z(0, 4, 16), k=z(0, 2, 16), v=z(0, 2, 24), log_decay=z(4), slots=sl), **bad})


@pytest.mark.parametrize("shape", [(0, 64), (0, 9, 64)])
def test_norm(shape):
    x = z(*shape, dtype=BF)
    w, b = z(64) + 1, z(64)
    y, stats = ssd.group_norm(x, 4, w, b, x)
    assert y.shape == shape and y.dtype == BF and stats.shape == (0, 4, 2)
    g = ssd.group_norm_bwd(x, 4, stats, y, w, b, x)
    assert g["dx"].shape == shape and g["dz"].shape == shape and torch.all(g["dweight"] == 0) and torch.all(g["dbias"] == 0)
    assert ssd.group_norm(x, 4, want_stats=False)[1] is None
    for bad in (dict(groups=5), dict(weight=z(32)), dict(eps=0.0), dict(stats=z(1, 4, 2))):
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.group_norm(**{**dict(x=x, groups=4), **bad})

"""GPU: batches of the gated delta rule and of rotary positions without tokens run nothing; their sizes and other
arguments are checked as those of any batch."""
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
    x = dict(q=z(b, T, Hk, dk, dtype=dtype), k=z(b, T, Hk, dk, dtype=dtype), v=z(b, T, H, dv, dtype=dtype), log_decay=z(b, T, H),
             beta=z(b, T, H))
    n = b if cu is None else len(cu) - 1
    x["cu_seqlens"] = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    do, init = z(b, T, H, dv, dtype=dtype), torch.randn(n, H, dv, dk, device="cuda")
    o, fin = ssd.gated_delta_fwd(**x, initial_state=init)
    assert o.shape == (b, T, H, dv) and o.dtype == dtype and torch.equal(fin, init)
    assert torch.all(ssd.gated_delta_fwd(**x)[1] == 0) and ssd.gated_delta_fwd(**x, want_final=False)[1] is None
    g = ssd.gated_delta_bwd(**x, do=do, dfinal_state=init, want_dinit=True)
    assert g["dq"].shape == x["q"].shape and g["dbeta"].shape == (b, T, H) and torch.equal(g["dinit"], init)
    narrow = dict(q=z(b, T, Hk, 12, dtype=dtype), k=z(b, T, Hk, 12, dtype=dtype))
    wide = dict(v=z(b, T, H, 264, dtype=dtype))
    for bad in (narrow, wide, dict(scale=0.0), dict(beta=z(b, T, H + 1)), dict(initial_state=z(n + 1, H, dv, dk))):
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.gated_delta_fwd(**{**x, **bad})
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.gated_delta_bwd(**{**x, "do": z(b, T, H, 264, dtype=dtype) if bad is wide else do, **bad})


@pytest.mark.parametrize("lead", [(0,), (2, 0), (0, 5)])
def test_rotary(lead):
    positions = z(*lead, dtype=torch.int32)
    q, k = ssd.rotary(z(*lead, 4, 16), z(*lead, 2, 16), z(8), positions=positions)
    assert q.shape == (*lead, 4, 16) and k.shape == (*lead, 2, 16)
    for bad in (dict(scale=0.0), dict(q=z(*lead, 4, 1032), k=z(*lead, 2, 1032)), dict(freq=z(9)), dict(layout="both")):
        with pytest.raises((ValueError, ssd.SSDError)):
            ssd.rotary(**{**dict(q=z(*lead, 4, 16), k=z(*lead, 2, 16), freq=z(8), positions=positions), **bad})

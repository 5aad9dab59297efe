"""GPU: group norm with its results over its inputs: bit for bit as into other tensors."""
import ctypes

import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd
from ssd_chunked_scan_fwd_amd import binding

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


# samples, positions, channels, groups: rows in registers, a workgroup a row, single channels, too wide for registers, slabs
SHAPES = [(300, 1, 256, 8), (40, 1, 5120, 1), (50, 1, 70, 10), (3, 1, 10240, 1), (3, 700, 320, 32), (2, 301, 21, 3), (2, 33, 64, 4)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["after", "before"])
@pytest.mark.parametrize("shape", SHAPES)
def test_in_place(shape, gate, dtype):
    n, s, C, G = shape
    print(f"[norm in place] {shape} {gate} {dtype}", flush=True)
    g = torch.Generator().manual_seed(C)
    dims = (n, C) if s == 1 else (n, s, C)
    x, z, dy = (torch.randn(*dims, generator=g).to(dtype).cuda() for _ in range(3))
    w, b = (1 + 0.1 * torch.randn(C, generator=g)).cuda(), torch.randn(C, generator=g).cuda()
    y, stats = ssd.group_norm(x, G, w, b, z, gate=gate)
    for over in ("x", "z"):
        t = dict(x=x.clone(), z=z.clone())
        y1, s1 = ssd.group_norm(t["x"], G, w, b, t["z"], gate=gate, y=t[over])
        assert y1 is t[over] and torch.equal(y, y1) and torch.equal(stats, s1), over

    want = ssd.group_norm_bwd(x, G, stats, dy, w, b, z, gate=gate)
    shape_ = binding._norm_shape(x, G, z, "none", gate, True)
    ws, have = binding._norm_workspace(shape_, 1, None, x.device)
    at = lambda t: ctypes.c_void_p(None if t is None else t.data_ptr())
    for dx, dz in (("x", "z"), ("dy", "x"), ("z", "dy")):
        t = dict(x=x.clone(), z=z.clone(), dy=dy.clone())
        dw, db = torch.empty_like(w), torch.empty_like(b)
        st = ssd.lib().ssd_group_norm_bwd(at(t["x"]), at(t["z"]), at(w), at(b), at(stats), at(t["dy"]), at(t[dx]), at(t[dz]), at(dw),
                                          at(db), ctypes.byref(shape_), at(ws), have, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for got, name in ((t[dx], "dx"), (t[dz], "dz"), (dw, "dweight"), (db, "dbias")):
            assert torch.equal(got, want[name]), (dx, dz, name)

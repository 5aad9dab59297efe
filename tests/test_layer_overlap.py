"""CPU: outputs of the layer operators that share memory with inputs are refused, as blocks read the one
while others write the other; addresses are never dereferenced, as every call that would launch ends at its
check of `eps`, of the workspace or of the overlap."""
import ctypes

import pytest

import ssd_chunked_scan_fwd_amd as ssd
from test_layer_abi import INVALID, lin, lin_bytes, norm

MB = 1 << 20


def ptr(n):
    return ctypes.c_void_p(n)


# q, k, v, log_decay, cu, scale, init, o, final, shape, ws, bytes, stream
FWD = dict(q=0, k=1, v=2, init=6, o=7, final=8, ws=10)
BWD = dict(q=0, k=1, v=2, init=6, do=7, dfinal=8, dq=9, dk=10, dv=11, dinit=12, ws=14)


def fwd_args(sh, need, **at):
    a = [ptr(64 * MB * (i + 1)) for i in range(13)]
    a[4], a[5], a[9], a[11], a[12] = None, 1.0, ctypes.byref(sh), need, None
    for k, v in at.items():
        a[FWD[k]] = v
    return a


def bwd_args(sh, need, **at):
    a = [ptr(64 * MB * (i + 1)) for i in range(17)]
    a[4], a[5], a[13], a[15], a[16] = None, 1.0, ctypes.byref(sh), need, None
    for k, v in at.items():
        a[BWD[k]] = v
    return a


def states(sh):
    return max(sh.num_seqs, sh.batch) * sh.nheads * sh.dk * sh.dv * 4


@pytest.mark.parametrize("shift", [0, 16, 2 * 64 * 64 * 4, -16])
def test_states(shift):
    """A final state that begins, or ends, inside the initial one, as neighbouring slots of a pool do."""
    sh = lin(batch=2, nheads=2, nkv_heads=2)
    _, need = lin_bytes(sh)
    at = 1 << 40
    assert ssd.lib().ssd_lin_attn_fwd(*fwd_args(sh, need, init=ptr(at), final=ptr(at + shift))) == INVALID
    _, need = lin_bytes(sh, True)
    for other in ("init", "dfinal"):
        assert ssd.lib().ssd_lin_attn_bwd(*bwd_args(sh, need, dinit=ptr(at + shift), **{other: ptr(at)})) == INVALID


def test_outputs_over_inputs():
    sh = lin(batch=1, nheads=2, nkv_heads=2, q_row=3 * 128, k_row=3 * 128, v_row=3 * 128)
    _, need = lin_bytes(sh)
    base = 1 << 40
    rows = dict(q=ptr(base), k=ptr(base + 256), v=ptr(base + 512))     # one projection's rows of 768 bytes
    for o in (base, base + 512, base + 4095 * 768, base - 16, 64 * MB * 4):   # the last: over log_decay
        assert ssd.lib().ssd_lin_attn_fwd(*fwd_args(sh, need, o=ptr(o), **rows)) == INVALID
    for ws in (base + 768, 64 * MB * 8):
        assert ssd.lib().ssd_lin_attn_fwd(*fwd_args(sh, need, ws=ptr(ws), **rows)) == INVALID
    _, need = lin_bytes(sh, True)
    for out in ("dq", "dk", "dv"):
        assert ssd.lib().ssd_lin_attn_bwd(*bwd_args(sh, need, **{out: ptr(base)}, **rows)) == INVALID
        assert ssd.lib().ssd_lin_attn_bwd(*bwd_args(sh, need, **{out: ptr(64 * MB * 8 + 1024)}, **rows)) == INVALID   # do
    assert ssd.lib().ssd_lin_attn_bwd(*bwd_args(sh, need, dq=ptr(base + MB * 1024), dk=ptr(base + MB * 1024), **rows)) == INVALID


def test_step():
    sh = lin(batch=4)
    # state, q, k, v, ld, slots, num_slots, scale, o, shape, stream
    far = [ptr(64 * MB * (i + 1)) for i in range(9)]
    for i in (0, 1, 2, 3, 4, 5):
        a = far[:6] + [4, 1.0, far[i], ctypes.byref(sh), None]
        assert ssd.lib().ssd_lin_attn_step(*a) == INVALID, i
    a = far[:6] + [4, 1.0, ptr(64 * MB + 4 * 8 * 64 * 64 * 4 - 16), ctypes.byref(sh), None]   # inside the last slot
    assert ssd.lib().ssd_lin_attn_step(*a) == INVALID


def test_norm():
    L, n = ssd.lib(), ctypes.c_size_t(0)
    base = 1 << 40
    sh = norm(gate=1)
    size = 4 * 9 * 64 * 2
    L.ssd_group_norm_workspace_bytes(ctypes.byref(sh), 0, ctypes.byref(n))
    ws = ptr(1 << 41)
    for x, z, y in ((0, 2 * size, 16), (0, 2 * size, size - 16), (16, 2 * size, 0), (0, 2 * size, 2 * size - 16)):
        assert L.ssd_group_norm(ptr(base + x), ptr(base + z), None, None, 1e-5, ptr(base + y), None, ctypes.byref(sh), ws,
                                n.value, None) == INVALID
    wide = norm(x_row=128)   # y over rows that lie further apart than its own
    assert L.ssd_group_norm(ptr(base), None, None, None, 1e-5, ptr(base), None, ctypes.byref(wide), ws, n.value, None) == INVALID
    L.ssd_group_norm_workspace_bytes(ctypes.byref(sh), 1, ctypes.byref(n))
    far = [ptr(base + 64 * MB * i) for i in range(8)]
    for dx, dz in ((ptr(base + 16), far[6]), (far[5], ptr(base + 64 * MB + 16)), (ptr(base + 128 * MB - 16), far[6]), (far[5], far[5])):
        assert L.ssd_group_norm_bwd(far[0], far[1], None, None, far[3], far[2], dx, dz, None, None, ctypes.byref(sh), ws, n.value,
                                    None) == INVALID

"""CPU: refusals of the gated delta rule and of rotary positions, in the C ABI and in the binding; each case fails
validation, so nothing is launched and no address is dereferenced."""
import ctypes

import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd
from ssd_chunked_scan_fwd_amd import binding
from test_layer_abi import FAKE, INVALID, ODD, OK, UNSUPPORTED, WS_SMALL, _refused

MB = 1 << 20


def ptr(n):
    return ctypes.c_void_p(n)


def delta(**kw):
    base = dict(batch=2, seqlen=500, nheads=8, nqk_heads=2, dk=64, dv=64, num_seqs=0, dtype=1, q_row=0, k_row=0, v_row=0)
    base.update(kw)
    return binding.DeltaShape(*[base[f] for f, _ in binding.DeltaShape._fields_])


def delta_bytes(sh, bwd=False):
    n = ctypes.c_size_t(0)
    fn = "ssd_gated_delta_bwd_workspace_bytes" if bwd else "ssd_gated_delta_workspace_bytes"
    return getattr(ssd.lib(), fn)(ctypes.byref(sh), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(dk=8, dv=256), OK), (dict(dk=12), UNSUPPORTED), (dict(dv=264), UNSUPPORTED), (dict(dk=0), INVALID),
    (dict(nqk_heads=3), INVALID), (dict(nheads=0), INVALID), (dict(seqlen=0), INVALID), (dict(batch=0), INVALID),
    (dict(num_seqs=2), INVALID), (dict(batch=1, num_seqs=2), OK), (dict(num_seqs=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(q_row=2 * 64 - 8), INVALID), (dict(v_row=8 * 64 - 8), INVALID), (dict(q_row=2 * 64 + 4), UNSUPPORTED),
    (dict(k_row=1 << 40), UNSUPPORTED), (dict(batch=65536), UNSUPPORTED), (dict(batch=60000, seqlen=1 << 20), UNSUPPORTED)])
def test_shapes(kw, code):
    assert delta_bytes(delta(**kw))[0] == code
    assert delta_bytes(delta(**kw), True)[0] == code
    assert ssd.lib().ssd_gated_delta_workspace_bytes(None, ctypes.byref(ctypes.c_size_t(0))) == INVALID
    assert ssd.lib().ssd_gated_delta_workspace_bytes(ctypes.byref(delta()), None) == INVALID


def test_launch_limit():
    """More one-token sequences and heads than a grid has threads for (2^32) are refused, not half launched."""
    many = dict(batch=1, seqlen=65535, num_seqs=65535, dk=8, dv=8)
    assert delta_bytes(delta(nheads=120, nqk_heads=120, **many))[0] == OK
    assert delta_bytes(delta(nheads=260, nqk_heads=260, **many))[0] == UNSUPPORTED
    assert delta_bytes(delta(nheads=260, nqk_heads=260, **many), True)[0] == UNSUPPORTED


@pytest.mark.parametrize("sizes", [dict(batch=1, seqlen=1 << 20, nheads=1, nqk_heads=1), dict(batch=3, seqlen=40000, nheads=2, nqk_heads=1),
                                   dict(batch=1, seqlen=300000, nheads=2, nqk_heads=2, num_seqs=5), dict(batch=1, seqlen=1, nheads=64),
                                   dict(batch=64, seqlen=4096, nheads=32, nqk_heads=32)])
def test_workspace_holds_every_chunk(sizes):
    """Gates and matrices of every chunk of every sequence, whatever their lengths."""
    for dtype, C in ((1, 64), (0, 32)):
        sh = delta(dtype=dtype, **sizes)
        _, need = delta_bytes(sh)
        chunks = sh.batch * -(-sh.seqlen // C) if not sh.num_seqs else sh.seqlen // C + sh.num_seqs
        assert need >= chunks * sh.nheads * (6 * C * 4 + C * C * 4 + C * C * 4)


def test_fwd_validates():
    L, sh = ssd.lib(), delta(batch=1, nheads=2)
    st, need = delta_bytes(sh)
    assert st == OK and need > 0
    # q, k, v, log_decay, beta, cu, scale, init, o, final, shape, ws, bytes, stream
    far = [ptr(256 * MB * (i + 1)) for i in range(14)]
    args = far[:5] + [None, 1.0] + far[7:10] + [ctypes.byref(sh), far[11], need, None]
    for i in (0, 1, 2, 4, 8, 10, 11):
        a = list(args)
        a[i] = None
        assert L.ssd_gated_delta_fwd(*a) == INVALID, i
    for i in (0, 1, 2, 3, 4, 7, 8, 9, 11):
        a = list(args)
        a[i] = ODD
        assert L.ssd_gated_delta_fwd(*a) == INVALID, i
    for scale in (0.0, 1e-42, float("nan"), float("inf")):
        a = list(args)
        a[6] = scale
        assert L.ssd_gated_delta_fwd(*a) == INVALID
    a = list(args)
    a[12] = need - 1
    assert L.ssd_gated_delta_fwd(*a) == WS_SMALL
    a = list(args)
    a[5] = FAKE   # cu_seqlens without num_seqs
    assert L.ssd_gated_delta_fwd(*a) == INVALID
    for out, other in ((8, 0), (8, 2), (8, 3), (8, 4), (9, 7), (9, 8), (11, 0), (11, 8), (11, 9)):   # outputs over others
        a = list(args)
        a[out] = ptr(a[other].value + 256)
        assert L.ssd_gated_delta_fwd(*a) == INVALID, (out, other)


def test_bwd_validates():
    L, sh = ssd.lib(), delta()
    _, need = delta_bytes(sh, True)
    # q, k, v, ld, beta, cu, scale, init, do, dfinal, dq, dk, dv, dld, dbeta, dinit, shape, ws, bytes, stream
    far = [ptr(256 * MB * (i + 1)) for i in range(20)]
    args = far[:5] + [None, 1.0] + far[7:16] + [ctypes.byref(sh), far[17], need, None]
    for i in (0, 1, 2, 4, 8, 10, 11, 12, 14, 16, 17):
        a = list(args)
        a[i] = None
        assert L.ssd_gated_delta_bwd(*a) == INVALID, i
    for i in (0, 3, 4, 7, 8, 9, 10, 11, 12, 13, 14, 15, 17):
        a = list(args)
        a[i] = ODD
        assert L.ssd_gated_delta_bwd(*a) == INVALID, i
    a = list(args)
    a[18] = need - 1
    assert L.ssd_gated_delta_bwd(*a) == WS_SMALL
    for out, other in ((10, 0), (11, 1), (12, 2), (12, 8), (13, 3), (14, 4), (15, 9), (15, 7), (10, 11), (13, 14), (17, 2)):
        a = list(args)
        a[out] = ptr(a[other].value + 16)
        assert L.ssd_gated_delta_bwd(*a) == INVALID, (out, other)


def test_step_validates():
    L, sh = ssd.lib(), delta(batch=4)
    # state, q, k, v, ld, beta, slots, num_slots, scale, o, shape, stream
    far = [ptr(256 * MB * (i + 1)) for i in range(10)]
    args = far[:7] + [4, 1.0, far[9], ctypes.byref(sh), None]
    for i in (0, 1, 2, 3, 5, 9, 10):
        a = list(args)
        a[i] = None
        assert L.ssd_gated_delta_step(*a) == INVALID, i
    for i in (0, 1, 2, 3, 4, 5, 6, 9):
        a = list(args)
        a[i] = ODD
        assert L.ssd_gated_delta_step(*a) == INVALID, i
    for i in range(7):
        a = list(args)
        a[9] = a[i]
        assert L.ssd_gated_delta_step(*a) == INVALID, i
    a = list(args)
    a[6], a[7] = None, 3   # no slots: one state an entry
    assert L.ssd_gated_delta_step(*a) == INVALID
    a = list(args)
    a[7] = 0
    assert L.ssd_gated_delta_step(*a) == INVALID
    bad = delta(dk=20)
    a = list(args)
    a[10] = ctypes.byref(bad)
    assert L.ssd_gated_delta_step(*a) == UNSUPPORTED


def rot(**kw):
    base = dict(batch=2, seqlen=10, q_heads=4, k_heads=2, dim=64, rot=32, num_seqs=0, dtype=1, layout=0, inverse=0, q_row=0, k_row=0,
                q_out_row=0, k_out_row=0)
    base.update(kw)
    return binding.RotaryShape(*[base[f] for f, _ in binding.RotaryShape._fields_])


def rot_args(sh, **at):
    # q, k, freq, positions, cu, offsets, scale, q_out, k_out, shape, stream
    far = [ptr(64 * MB * (i + 1)) for i in range(9)]
    a = [far[0], far[1], far[2], None, None, None, 1.0, far[7], far[8], ctypes.byref(sh), None]
    for k, v in at.items():
        a[dict(q=0, k=1, freq=2, positions=3, cu=4, offsets=5, scale=6, q_out=7, k_out=8, shape=9)[k]] = v
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(batch=0), INVALID), (dict(seqlen=0), INVALID), (dict(q_heads=0), INVALID), (dict(k_heads=-1), INVALID), (dict(rot=0), INVALID),
    (dict(rot=31), INVALID), (dict(rot=66), INVALID), (dict(num_seqs=2), INVALID), (dict(inverse=2), INVALID), (dict(dtype=3), UNSUPPORTED),
    (dict(layout=2), UNSUPPORTED), (dict(dim=1032, rot=8), UNSUPPORTED), (dict(q_row=255), INVALID), (dict(k_out_row=127), INVALID),
    (dict(batch=65536), UNSUPPORTED), (dict(batch=60000, seqlen=1 << 20), UNSUPPORTED), (dict(k_heads=0), INVALID)])
def test_rotary_shapes(kw, code):
    assert ssd.lib().ssd_rotary(*rot_args(rot(**kw))) == code


def test_rotary_validates():
    L, sh = ssd.lib(), rot()
    for at in (dict(q=None), dict(k=None), dict(freq=None), dict(q_out=None), dict(k_out=None), dict(shape=None), dict(q=ODD), dict(k_out=ODD),
               dict(freq=ODD), dict(positions=ODD), dict(offsets=ODD), dict(cu=FAKE), dict(scale=0.0), dict(scale=float("nan")),
               dict(positions=FAKE, offsets=FAKE)):
        assert L.ssd_rotary(*rot_args(sh, **at)) == INVALID, at


def test_rotary_overlap():
    """In place, or apart; rows of one projection may lie between one another."""
    L, base = ssd.lib(), 1 << 40
    sh = rot()
    for at in (dict(q=ptr(base), q_out=ptr(base + 16)), dict(q=ptr(base), k_out=ptr(base)), dict(q_out=ptr(base), k_out=ptr(base + 128)),
               dict(q_out=ptr(base), freq=ptr(base + 64)), dict(q_out=ptr(base), positions=ptr(base)), dict(k=ptr(base), q_out=ptr(base))):
        assert L.ssd_rotary(*rot_args(sh, **at)) == INVALID, at
    wide = rot(q_row=1024, k_row=1024, q_out_row=1024, k_out_row=1024)
    for q_out, k_out in ((base + 512, base + 512 + 128), (base, base + 384), (base + 2048 - 128, base + 512)):
        assert L.ssd_rotary(*rot_args(wide, q=ptr(base), k=ptr(base + 512), q_out=ptr(q_out), k_out=ptr(k_out))) == INVALID, (q_out, k_out)


# ---------------------------------------------------------------- the binding

def _args(dtype=torch.bfloat16):
    z = torch.zeros
    return dict(q=z(1, 32, 2, 16, dtype=dtype), k=z(1, 32, 2, 16, dtype=dtype), v=z(1, 32, 4, 24, dtype=dtype), log_decay=z(1, 32, 4),
                beta=z(1, 32, 4))


BF = torch.bfloat16


@pytest.mark.parametrize("kw,what", [
    (dict(q=torch.zeros(1, 32, 16)), "q must"), (dict(q=torch.zeros(1, 32, 2, 16, dtype=torch.float16)), "dtype"),
    (dict(k=torch.zeros(1, 31, 2, 16, dtype=BF)), "k must"), (dict(k=torch.zeros(1, 32, 2, 16)), "k has dtype"),
    (dict(k=torch.zeros(1, 32, 1, 16, dtype=BF)), "k must"), (dict(v=torch.zeros(1, 32, 3, 24, dtype=BF)), "nheads"),
    (dict(v=torch.zeros(1, 32, 24, dtype=BF)), "v must"), (dict(log_decay=torch.zeros(4)), "log_decay"),
    (dict(log_decay=torch.zeros(1, 32, 4, dtype=BF)), "log_decay"), (dict(beta=None), "beta"), (dict(beta=torch.zeros(1, 32, 2)), "beta"),
    (dict(beta=torch.zeros(1, 4, 32).transpose(1, 2)), "beta"), (dict(initial_state=torch.zeros(1, 4, 16, 24)), "initial_state"),
    (dict(o=torch.zeros(1, 32, 4, 16, dtype=BF)), "o "), (dict(final_state=torch.zeros(2, 4, 24, 16)), "final_state"),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)), "cu_seqlens"), (dict(cu_seqlens=torch.zeros(1, dtype=torch.int32)), "cu_seqlens"),
    (dict(q=torch.zeros(1, 32, 2, 32, dtype=BF)[..., ::2]), "q must"), (dict(), "device tensor")])
def test_binding(kw, what):
    a = _args()
    a.update(kw)
    _refused(what, ssd.gated_delta_fwd, **a)
    for n in ("o", "final_state"):
        a.pop(n, None)
    if not set(kw) & {"o", "final_state"}:
        _refused(what, ssd.gated_delta_bwd, do=torch.zeros(1, 32, 4, 24, dtype=BF), **a)


@pytest.mark.parametrize("kw,what", [
    (dict(q=torch.zeros(3, 2)), "q must"), (dict(k=torch.zeros(2, 2, 16)), "k must"), (dict(v=torch.zeros(3, 3, 24)), "nheads"),
    (dict(k=torch.zeros(3, 2, 16, dtype=BF)), "k has dtype"), (dict(state=torch.zeros(5, 4, 16, 24)), "state"),
    (dict(state=torch.zeros(2, 4, 24, 16)), "slots"), (dict(slots=torch.zeros(2, dtype=torch.int32)), "slots"),
    (dict(slots=torch.zeros(3, dtype=torch.int64)), "slots"), (dict(o=torch.zeros(3, 4, 16)), "o "), (dict(beta=None), "beta"),
    (dict(log_decay=torch.zeros(4)), "log_decay"), (dict(), "device tensor")])
def test_step_binding(kw, what):
    a = dict(state=torch.zeros(5, 4, 24, 16), q=torch.zeros(3, 2, 16), k=torch.zeros(3, 2, 16), v=torch.zeros(3, 4, 24),
             log_decay=torch.zeros(3, 4), beta=torch.zeros(3, 4))
    a.update(kw)
    _refused(what, ssd.gated_delta_step, **a)


@pytest.mark.parametrize("kw,what", [
    (dict(q=torch.zeros(8, 16)), "q must"), (dict(q=torch.zeros(2, 5, 4, 16, dtype=torch.float16)), "dtype"), (dict(q=[1.0]), "q must"),
    (dict(k=torch.zeros(2, 5, 2, 8)), "k must"), (dict(k=torch.zeros(2, 4, 2, 16)), "k must"), (dict(freq=torch.zeros(2, 4)), "1-d"),
    (dict(freq=torch.zeros(9)), "freq"), (dict(freq=torch.zeros(0)), "freq"), (dict(layout="both"), "layout"),
    (dict(positions=torch.zeros(2, 5, dtype=torch.int32), offsets=torch.zeros(2, dtype=torch.int32)), "exclude"),
    (dict(cu_seqlens=torch.zeros(3, dtype=torch.int32)), "cu_seqlens"), (dict(q_out=torch.zeros(2, 5, 4, 8)), "q_out"),
    (dict(k=None, k_out=torch.zeros(2, 5, 2, 16)), "k_out"), (dict(q=torch.zeros(2, 5, 16, 4).transpose(2, 3)), "q must"),
    (dict(q=torch.zeros(2, 7, 4, 16)[:, :5]), "one distance"), (dict(q=torch.zeros(2, 4, 16), k=None), "positions"), (dict(), "device tensor")])
def test_rotary_binding(kw, what):
    a = dict(q=torch.zeros(2, 5, 4, 16), k=torch.zeros(2, 5, 2, 16), freq=torch.zeros(4))
    a.update(kw)
    _refused(what, ssd.rotary, **a)
    _refused(what, ssd.rotary_bwd, dq=a.pop("q"), dk=a.pop("k"), **a)

"""CPU: refusals of the layer operators (linear attention, group norm, pages), in
the C ABI and in the binding; each case fails validation, so nothing is launched.
"""
import ctypes

import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd
from ssd_chunked_scan_fwd_amd import binding

OK, INVALID, UNSUPPORTED, WS_SMALL = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1001)


def lin(**kw):
    base = dict(batch=2, seqlen=4096, nheads=8, nkv_heads=2, dk=64, dv=64, num_seqs=0, dtype=1, q_row=0, k_row=0, v_row=0)
    base.update(kw)
    return binding.LinShape(*[base[f] for f, _ in binding.LinShape._fields_])


def lin_bytes(sh, bwd=False):
    n = ctypes.c_size_t(0)
    fn = "ssd_lin_attn_bwd_workspace_bytes" if bwd else "ssd_lin_attn_workspace_bytes"
    return getattr(ssd.lib(), fn)(ctypes.byref(sh), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(dk=8, dv=256), OK), (dict(dk=12), UNSUPPORTED), (dict(dv=264), UNSUPPORTED), (dict(dk=0), INVALID),
    (dict(nkv_heads=3), INVALID), (dict(nheads=0), INVALID), (dict(seqlen=0), INVALID), (dict(batch=0), INVALID),
    (dict(num_seqs=2), INVALID), (dict(batch=1, num_seqs=2), OK), (dict(num_seqs=-1), INVALID), (dict(dtype=2), UNSUPPORTED),
    (dict(q_row=8 * 64 - 8), INVALID), (dict(q_row=8 * 64 + 4), UNSUPPORTED), (dict(k_row=1 << 40), UNSUPPORTED),
    (dict(batch=65536), UNSUPPORTED), (dict(batch=60000, seqlen=1 << 20), UNSUPPORTED)])
def test_lin_shapes(kw, code):
    assert lin_bytes(lin(**kw))[0] == code
    assert lin_bytes(lin(**kw), True)[0] == code


@pytest.mark.parametrize("kw,heads", [(dict(dk=8, dv=8), 255), (dict(dk=8, dv=256), 63), (dict(dk=8, dv=64, dtype=0), 63)])
def test_lin_launch_limit(kw, heads):
    """More one-token sequences and heads than a grid has threads for (2^32) are refused, not half launched."""
    many = dict(batch=1, seqlen=65535, num_seqs=65535, **kw)
    assert lin_bytes(lin(nheads=heads, nkv_heads=heads, **many))[0] == OK
    assert lin_bytes(lin(nheads=heads + 2, nkv_heads=heads + 2, **many))[0] == UNSUPPORTED
    assert lin_bytes(lin(nheads=heads + 2, nkv_heads=heads + 2, **many), True)[0] == UNSUPPORTED


def test_lin_fwd_validates():
    L, sh = ssd.lib(), lin(batch=1, nheads=2)
    st, need = lin_bytes(sh)
    assert st == OK and need > 0
    # q, k, v, log_decay, cu, scale, init, o, final, shape, ws, bytes, stream
    args = [FAKE, FAKE, FAKE, FAKE, None, 1.0, None, FAKE, None, ctypes.byref(sh), FAKE, need, None]
    for i in (0, 1, 2, 3, 7, 9, 10):
        a = list(args)
        a[i] = None
        assert L.ssd_lin_attn_fwd(*a) == INVALID, i
    for i in (0, 1, 2, 6, 7, 8, 10):
        a = list(args)
        a[i] = ODD
        assert L.ssd_lin_attn_fwd(*a) == INVALID, i
    for scale in (0.0, 1e-42, float("nan"), float("inf")):
        a = list(args)
        a[5] = scale
        assert L.ssd_lin_attn_fwd(*a) == INVALID
    a = list(args)
    a[11] = need - 1
    assert L.ssd_lin_attn_fwd(*a) == WS_SMALL
    a = list(args)
    a[4] = FAKE   # cu_seqlens without num_seqs
    assert L.ssd_lin_attn_fwd(*a) == INVALID


def test_lin_bwd_validates():
    L, sh = ssd.lib(), lin()
    _, need = lin_bytes(sh, True)
    # q, k, v, ld, cu, scale, init, do, dfinal, dq, dk, dv, dinit, shape, ws, bytes, stream
    args = [FAKE] * 4 + [None, 1.0, None, FAKE, None, FAKE, FAKE, FAKE, None, ctypes.byref(sh), FAKE, need, None]
    for i in (0, 1, 2, 3, 7, 9, 10, 11, 13, 14):
        a = list(args)
        a[i] = None
        assert L.ssd_lin_attn_bwd(*a) == INVALID, i
    for i in (7, 8, 12):
        a = list(args)
        a[i] = ODD
        assert L.ssd_lin_attn_bwd(*a) == INVALID, i
    a = list(args)
    a[15] = need - 1
    assert L.ssd_lin_attn_bwd(*a) == WS_SMALL


def test_lin_step_validates():
    L, sh = ssd.lib(), lin(batch=4)
    # state, q, k, v, ld, slots, num_slots, scale, o, shape, stream
    args = [FAKE] * 5 + [FAKE, 4, 1.0, FAKE, ctypes.byref(sh), None]
    for i in (0, 1, 2, 3, 4, 8, 9):
        a = list(args)
        a[i] = None
        assert L.ssd_lin_attn_step(*a) == INVALID, i
    a = list(args)
    a[5], a[6] = None, 3   # no slots: one state an entry
    assert L.ssd_lin_attn_step(*a) == INVALID
    a = list(args)
    a[0] = ODD
    assert L.ssd_lin_attn_step(*a) == INVALID
    bad = lin(dk=20)
    a = list(args)
    a[9] = ctypes.byref(bad)
    assert L.ssd_lin_attn_step(*a) == UNSUPPORTED


def norm(**kw):
    base = dict(samples=4, positions=9, channels=64, groups=4, x_row=0, z_row=0, dtype=1, act=0, gate=0, center=1)
    base.update(kw)
    return binding.NormShape(*[base[f] for f, _ in binding.NormShape._fields_])


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(samples=0), INVALID), (dict(positions=0), INVALID), (dict(groups=3), INVALID), (dict(groups=0), INVALID),
    (dict(x_row=63), INVALID), (dict(z_row=63), INVALID), (dict(dtype=5), UNSUPPORTED), (dict(act=2), UNSUPPORTED),
    (dict(gate=3), UNSUPPORTED), (dict(center=2), INVALID), (dict(samples=1 << 20, positions=1 << 20), UNSUPPORTED)])
def test_norm_shapes(kw, code):
    n = ctypes.c_size_t(0)
    for back in (0, 1):
        assert ssd.lib().ssd_group_norm_workspace_bytes(ctypes.byref(norm(**kw)), back, ctypes.byref(n)) == code


def test_norm_validates():
    L, sh = ssd.lib(), norm()
    n = ctypes.c_size_t(0)
    L.ssd_group_norm_workspace_bytes(ctypes.byref(sh), 0, ctypes.byref(n))
    # x, z, w, b, eps, y, stats, shape, ws, bytes, stream
    args = [FAKE, None, None, None, 1e-5, FAKE, None, ctypes.byref(sh), FAKE, n.value, None]
    for i, bad in ((0, None), (5, None), (7, None), (8, None), (1, FAKE), (0, ODD), (5, ODD), (2, ODD), (6, ODD), (4, 0.0),
                   (4, float("nan")), (4, -1.0)):
        a = list(args)
        a[i] = bad
        assert L.ssd_group_norm(*a) == INVALID, (i, bad)
    a = list(args)
    a[9] = n.value - 1
    assert L.ssd_group_norm(*a) == WS_SMALL
    L.ssd_group_norm_workspace_bytes(ctypes.byref(sh), 1, ctypes.byref(n))
    # x, z, w, b, stats, dy, dx, dz, dw, db, shape, ws, bytes, stream
    args = [FAKE, None, None, None, FAKE, FAKE, FAKE, None, None, None, ctypes.byref(sh), FAKE, n.value, None]
    for i, bad in ((0, None), (4, None), (5, None), (6, None), (7, FAKE), (1, FAKE), (4, ODD), (6, ODD), (8, ODD)):
        a = list(args)
        a[i] = bad
        assert L.ssd_group_norm_bwd(*a) == INVALID, (i, bad)


@pytest.mark.parametrize("kw", [
    dict(samples=1 << 21, positions=1, channels=4100, groups=1),     # single channels, in slabs
    dict(samples=1 << 22, positions=1, channels=2046, groups=1),     # single channels, a row a workgroup
    dict(samples=1 << 24, positions=1, channels=2048, groups=8),     # a group in half a wave
    dict(samples=1 << 25, positions=2, channels=8, groups=1)])       # a workgroup a sample
def test_norm_launch_limit(kw):
    """More rows and channels than a grid has threads for (2^32) are refused."""
    L, sh = ssd.lib(), norm(**kw)
    huge = 1 << 62
    assert L.ssd_group_norm(FAKE, None, None, None, 1e-5, FAKE, None, ctypes.byref(sh), FAKE, huge, None) == UNSUPPORTED
    assert L.ssd_group_norm_bwd(FAKE, None, None, None, FAKE, FAKE, FAKE, None, None, None, ctypes.byref(sh), FAKE, huge,
                                None) == UNSUPPORTED


def pages(**kw):
    base = dict(layers=2, slots=8, page_bytes=256)
    base.update(kw)
    return binding.PagesShape(*[base[f] for f, _ in binding.PagesShape._fields_])


def test_pages_validate():
    L = ssd.lib()
    for kw, code in ((dict(layers=0), INVALID), (dict(slots=0), INVALID), (dict(page_bytes=0), INVALID),
                     (dict(layers=70000), UNSUPPORTED), (dict(slots=(1 << 24) + 1), UNSUPPORTED)):
        sh = pages(**kw)
        assert L.ssd_pages_copy(FAKE, FAKE, FAKE, 1, ctypes.byref(sh), None) == code
        assert L.ssd_pages_clear(FAKE, FAKE, 1, ctypes.byref(sh), None) == code
        n = ctypes.c_size_t(0)
        assert L.ssd_pages_compact_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == code
    sh = pages()
    assert L.ssd_pages_copy(None, FAKE, FAKE, 1, ctypes.byref(sh), None) == INVALID
    assert L.ssd_pages_copy(FAKE, FAKE, FAKE, 0, ctypes.byref(sh), None) == INVALID
    assert L.ssd_pages_copy(FAKE, FAKE, FAKE, ssd.PAGES_MAX_PAIRS + 1, ctypes.byref(sh), None) == UNSUPPORTED
    assert L.ssd_pages_clear(FAKE, None, 1, ctypes.byref(sh), None) == INVALID
    n = ctypes.c_size_t(0)
    assert L.ssd_pages_compact_workspace_bytes(ctypes.byref(sh), ctypes.byref(n)) == OK
    assert L.ssd_pages_compact(FAKE, FAKE, FAKE, FAKE, ctypes.byref(sh), FAKE, n.value - 1, None) == WS_SMALL
    assert L.ssd_pages_compact(FAKE, FAKE, None, FAKE, ctypes.byref(sh), FAKE, n.value, None) == INVALID


# ---------------------------------------------------------------- the binding

def _refused(what, fn, *a, **kw):
    with pytest.raises((ValueError, TypeError)) as e:
        fn(*a, **kw)
    assert what in str(e.value), str(e.value)


def _lin_args(dtype=torch.bfloat16):
    z = torch.zeros
    return dict(q=z(1, 32, 4, 16, dtype=dtype), k=z(1, 32, 2, 16, dtype=dtype), v=z(1, 32, 2, 24, dtype=dtype), log_decay=z(4))


@pytest.mark.parametrize("kw,what", [
    (dict(q=torch.zeros(1, 32, 16)), "q must"), (dict(q=torch.zeros(1, 32, 4, 16, dtype=torch.float16)), "dtype"),
    (dict(k=torch.zeros(1, 31, 2, 16, dtype=torch.bfloat16)), "k must"), (dict(k=torch.zeros(1, 32, 2, 16)), "k has dtype"),
    (dict(k=torch.zeros(1, 32, 3, 16, dtype=torch.bfloat16), v=torch.zeros(1, 32, 3, 24, dtype=torch.bfloat16)), "nheads"),
    (dict(v=torch.zeros(1, 32, 4, 24, dtype=torch.bfloat16)), "v must"), (dict(log_decay=torch.zeros(2)), "log_decay"),
    (dict(log_decay=torch.zeros(4, dtype=torch.float64)), "log_decay"), (dict(log_decay=None), "log_decay"),
    (dict(initial_state=torch.zeros(1, 4, 16, 24)), "initial_state"), (dict(o=torch.zeros(1, 32, 4, 16, dtype=torch.bfloat16)), "o "),
    (dict(final_state=torch.zeros(2, 4, 24, 16)), "final_state"), (dict(cu_seqlens=torch.zeros(3, dtype=torch.int64)), "cu_seqlens"),
    (dict(cu_seqlens=torch.zeros(1, dtype=torch.int32)), "cu_seqlens"), (dict(q=torch.zeros(1, 32, 4, 32, dtype=torch.bfloat16)[..., ::2]), "q must"),
    (dict(q=torch.zeros(1, 32, 16, 4, dtype=torch.bfloat16).transpose(2, 3)), "q must"), (dict(), "device tensor")])
def test_lin_binding(kw, what):
    a = _lin_args()
    a.update(kw)
    _refused(what, ssd.lin_attn_fwd, **a)
    for n in ("o", "final_state"):
        a.pop(n, None)
    if kw and not set(kw) & {"o", "final_state"}:
        _refused(what, ssd.lin_attn_bwd, do=torch.zeros(1, 32, 4, 24, dtype=torch.bfloat16), **a)


def test_lin_binding_batch_strides():
    w = torch.zeros(2, 40, 4, 16, dtype=torch.bfloat16)[:, :32]   # rows of the batch do not follow on
    _refused("one distance", ssd.lin_attn_fwd, w, torch.zeros(2, 32, 2, 16, dtype=torch.bfloat16),
             torch.zeros(2, 32, 2, 24, dtype=torch.bfloat16), torch.zeros(4))


@pytest.mark.parametrize("kw,what", [
    (dict(q=torch.zeros(3, 4)), "q must"), (dict(k=torch.zeros(2, 2, 16)), "k must"), (dict(v=torch.zeros(3, 4, 24)), "v must"),
    (dict(k=torch.zeros(3, 2, 16, dtype=torch.bfloat16)), "k has dtype"), (dict(state=torch.zeros(5, 4, 16, 24)), "state"),
    (dict(state=torch.zeros(2, 4, 24, 16)), "slots"), (dict(slots=torch.zeros(2, dtype=torch.int32)), "slots"),
    (dict(slots=torch.zeros(3, dtype=torch.int64)), "slots"), (dict(o=torch.zeros(3, 4, 16)), "o "), (dict(log_decay=None), "log_decay"),
    (dict(state=torch.zeros(5, 4, 24, 16, dtype=torch.bfloat16)), "state"), (dict(), "device tensor")])
def test_step_binding(kw, what):
    a = dict(state=torch.zeros(5, 4, 24, 16), q=torch.zeros(3, 4, 16), k=torch.zeros(3, 2, 16), v=torch.zeros(3, 2, 24),
             log_decay=torch.zeros(4))
    a.update(kw)
    _refused(what, ssd.lin_attn_step, **a)


@pytest.mark.parametrize("kw,what", [
    (dict(x=torch.zeros(8)), "x must"), (dict(x=torch.zeros(3, 8, dtype=torch.float16)), "dtype"), (dict(groups=3), "groups"),
    (dict(groups=0), "groups"), (dict(weight=torch.zeros(4)), "weight"), (dict(bias=torch.zeros(8, dtype=torch.bfloat16)), "bias"),
    (dict(z=torch.zeros(3, 4)), "z must"), (dict(z=torch.zeros(3, 8, dtype=torch.bfloat16)), "z has"), (dict(act="relu"), "act"),
    (dict(gate="never"), "gate"), (dict(x=torch.zeros(8, 3).t()), "x must"), (dict(x=torch.zeros(4, 3, 8)[::2, 1:]), "x must"),
    (dict(), "device tensor")])
def test_norm_binding(kw, what):
    a = dict(x=torch.zeros(3, 8), groups=2)
    a.update(kw)
    _refused(what, ssd.group_norm, **a)
    x = a.pop("x")
    _refused(what, ssd.group_norm_bwd, x=x, stats=torch.zeros(x.shape[0], 2, 2), dy=torch.zeros(x.shape, dtype=x.dtype), **a)


def test_pages_binding():
    p, i = torch.zeros(1, 4, 8), torch.zeros(2, dtype=torch.int32)
    _refused("pool", ssd.pages_copy, torch.zeros(4, 8), i, i)
    _refused("contiguous", ssd.pages_copy, torch.zeros(2, 4, 8).transpose(0, 1), i, i)
    _refused("empty", ssd.pages_copy, torch.zeros(1, 4, 0), i, i)
    _refused("src", ssd.pages_copy, p, i.long(), i)
    _refused("dst", ssd.pages_copy, p, i, i[:1])
    _refused("device tensor", ssd.pages_copy, p, i, i)
    _refused("slots", ssd.pages_clear, p, i.float())
    _refused("live", ssd.pages_compact, p, torch.zeros(5, dtype=torch.uint8))
    _refused("live", ssd.pages_compact, p, torch.zeros(4, dtype=torch.int32))
    _refused("device tensor", ssd.pages_compact, p, torch.zeros(4, dtype=torch.bool))


def test_sizes_beyond_32_bits():
    """Sizes that the C structs would cut off to 32 bits are refused (shapes only: nothing is allocated)."""
    big = 1 << 32
    t = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")
    ld = t(1, dtype=torch.float32)
    idx = t(4, dtype=torch.int32)
    for call in (lambda: ssd.lin_attn_fwd(t(1, big + 8, 1, 8), t(1, big + 8, 1, 8), t(1, big + 8, 1, 8), ld),
                 lambda: ssd.lin_attn_fwd(t(1, 8, 1, big + 8), t(1, 8, 1, big + 8), t(1, 8, 1, 8), ld),
                 lambda: ssd.lin_attn_step(t(big + 8, 1, 8, 8, dtype=torch.float32), t(4, 1, 8), t(4, 1, 8), t(4, 1, 8), ld),
                 lambda: ssd.group_norm(t(big + 8, 64), 8),
                 lambda: ssd.group_norm(t(2, big // 2, 2, 64), 8),
                 lambda: ssd.pages_copy(t(1, big + 8, 4), idx, idx),
                 lambda: ssd.pages_copy(t(1, 8, 4), t(big + 1, dtype=torch.int32), t(big + 1, dtype=torch.int32)),
                 lambda: ssd.pages_clear(t(1, 8, 4), t(big + 1, dtype=torch.int32))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_shapes_handed_out_are_the_callers_own():
    q = torch.empty(1, 128, 2, 64, dtype=torch.bfloat16, device="meta")
    one = ssd.lin_attn_shape(q, q, q)
    one.dk = 8
    assert ssd.lin_attn_shape(q, q, q).dk == 64


def test_lin_states_not_in_place():
    """A prompt's final state over its initial one would be raced by the blocks; refused."""
    L, sh, other = ssd.lib(), lin(batch=1, nheads=2), ctypes.c_void_p(0x2000)
    _, need = lin_bytes(sh)
    args = [FAKE, FAKE, FAKE, FAKE, None, 1.0, other, FAKE, other, ctypes.byref(sh), FAKE, need, None]
    assert L.ssd_lin_attn_fwd(*args) == INVALID
    _, need = lin_bytes(sh, True)
    for init, dfinal in ((other, None), (None, other)):
        args = [FAKE] * 4 + [None, 1.0, init, FAKE, dfinal, FAKE, FAKE, FAKE, other, ctypes.byref(sh), FAKE, need, None]
        assert L.ssd_lin_attn_bwd(*args) == INVALID

"""GPU: the gated delta rule (prompts, gradients, the one-token step) against the
rule in 64 bits; the bounds are those of delta_ref.py."""
import sys

import numpy as np
import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_fwd_amd as ssd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def make(b, T, H, Hk, dk, dv, dtype, seed, nseq=None, states=True, lead=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    lead = lead or (b, T)
    unit = lambda *s: torch.nn.functional.normalize(r(*s), dim=-1)
    d = dict(q=unit(*lead, Hk, dk).to(dtype).cuda(), k=unit(*lead, Hk, dk).to(dtype).cuda(), v=r(*lead, H, dv).to(dtype).cuda(),
             g=(-torch.rand(*lead, H, generator=g) * 0.3).cuda(), beta=torch.rand(*lead, H, generator=g).cuda(),
             do=r(*lead, H, dv).to(dtype).cuda())
    st = (nseq or b, H, dv, dk)
    d["init"], d["dfinal"] = (r(*st).cuda() if states else None for _ in range(2))
    return d


def cu_of(cu):
    return None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")


def run_fwd(d, scale=0.5, cu=None, **kw):
    return ssd.gated_delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu_seqlens=cu_of(cu), scale=scale,
                               initial_state=d["init"], **kw)


def run_bwd(d, scale=0.5, cu=None, **kw):
    return ssd.gated_delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], d["do"], cu_seqlens=cu_of(cu), scale=scale,
                               initial_state=d["init"], dfinal_state=d["dfinal"], want_dinit=True, **kw)


def arrays(d, names=("q", "k", "v", "g", "beta")):
    out = [n64(d[n]) for n in names]
    if "g" in names and d["g"] is None:
        out[names.index("g")] = np.zeros(d["beta"].shape)
    return out


def check_fwd(d, scale=0.5, cu=None, name=""):
    o, fin = run_fwd(d, scale, cu)
    torch.cuda.synchronize()
    want = ref.batch_forward(*arrays(d), scale, n64(d["init"]), cu)
    rel = ref.rel_forward(d["q"].shape[1], d["q"].shape[3])
    got = n64(o)
    if cu is not None:
        got, want["o"] = got[:, cu[0]:cu[-1]], want["o"][:, cu[0]:cu[-1]]
    ref.check(got, want["o"], rel, d["q"].dtype == BF, name + " o")
    ref.check(n64(fin), want["final"], rel, False, name + " final")
    return o, fin


def check_bwd(d, scale=0.5, cu=None, name=""):
    r = run_bwd(d, scale, cu)
    torch.cuda.synchronize()
    q, k, v, g, beta = arrays(d)
    want = ref.batch_backward(q, k, v, g, beta, scale, n64(d["do"]), n64(d["init"]), n64(d["dfinal"]), cu)
    rel = ref.rel_backward(d["q"].shape[1], d["q"].shape[3], d["v"].shape[3])
    bf = d["q"].dtype == BF
    assert (r["dlog_decay"] is None) == (d["g"] is None)
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta", "dinit"):
        if r[n] is None:
            continue
        a, w = n64(r[n]), want[n]
        if cu is not None and n != "dinit":
            a, w = a[:, cu[0]:cu[-1]], w[:, cu[0]:cu[-1]]
        more = np.sqrt(ref.C) * np.linalg.norm(want["parts"]) if n == "dlog_decay" else 0.0
        ref.check(a, w, rel, bf and n in ("dq", "dk", "dv"), f"{name} {n}", more)
    return r


# b, T, H, Hk, dk, dv
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 2, 1, 16, 24), (1, 17, 1, 1, 32, 16), (1, 32, 2, 2, 64, 64), (1, 33, 2, 1, 64, 8),
          (1, 63, 3, 3, 64, 64), (1, 64, 2, 2, 128, 128), (2, 65, 4, 2, 40, 96), (1, 130, 4, 1, 128, 64), (1, 257, 2, 2, 64, 200),
          (1, 300, 6, 2, 96, 32), (1, 190, 1, 1, 256, 256), (3, 129, 2, 2, 32, 128), (1, 700, 4, 4, 16, 16), (1, 100, 2, 1, 200, 40)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    say(f"[delta fwd] {shape} {dtype}")
    check_fwd(make(*shape, dtype, seed=shape[1]), name=str(shape))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    say(f"[delta bwd] {shape} {dtype}")
    check_bwd(make(*shape, dtype, seed=100 + shape[1]), name=str(shape))


# Chunks and key heads enough that one workgroup takes the gradients of all value heads of a key head.
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(58, 67, 18, 9, 16, 24, None), (58, 70, 27, 9, 72, 8, None), (1, 900, 76, 38, 8, 32, [2, 2, 451, 460, 897])])
def test_backward_of_many_shared_heads(shape, dtype):
    *sizes, cu = shape
    say(f"[delta bwd shared] {shape} {dtype}")
    check_bwd(make(*sizes, dtype, seed=sizes[1], nseq=None if cu is None else len(cu) - 1), cu=cu, name=str(shape))


# Long sequences of few heads: cut into segments that are walked at once.
LONG = [(1, 4000, 1, 1, 64, 40, None), (2, 3001, 2, 1, 128, 128, None), (1, 2600, 1, 1, 256, 24, None), (1, 3500, 2, 2, 16, 256, None),
        (1, 4200, 1, 1, 32, 64, [0, 1500, 1500, 1501, 4200]), (1, 3900, 1, 1, 64, 64, [3, 20, 3900])]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", LONG)
def test_long_sequences(shape, dtype):
    say(f"[delta long] {shape} {dtype}")
    *sizes, cu = shape
    d = make(*sizes, dtype, seed=sizes[1], nseq=None if cu is None else len(cu) - 1)
    d["g"] *= 0.1   # a memory of some 70 tokens
    check_fwd(d, cu=cu, name=str(shape))
    check_bwd(d, cu=cu, name=str(shape))
    d["init"] = d["dfinal"] = None
    check_fwd(d, cu=cu, name=str(shape))
    check_bwd(d, cu=cu, name=str(shape))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_states_no_decay(dtype):
    say(f"[delta] no states, no decay {dtype}")
    d = make(2, 150, 4, 2, 64, 64, dtype, 7, states=False)
    check_fwd(d, -0.3)
    check_bwd(d, -0.3)
    d["g"] = None
    check_fwd(d)
    check_bwd(d)
    o, fin = run_fwd(d, want_final=False)
    assert fin is None


@pytest.mark.parametrize("dtype", [BF, F32])
def test_edge_gates(dtype):
    """Decays of 0 (log -inf, -250) and 1, beta of 0 and 1."""
    say(f"[delta] edge gates {dtype}")
    d = make(1, 200, 4, 2, 32, 64, dtype, 11)
    d["g"][:, ::7] = -float("inf")
    d["g"][:, 3::11] = -250.0
    d["g"][:, :, 1] = 0.0
    d["beta"][:, ::3] = 0.0
    d["beta"][:, 1::3] = 1.0
    d["beta"][:, :, 2] = 0.0
    with np.errstate(invalid="ignore"):
        check_fwd(d)
        check_bwd(d)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_equal_keys(dtype):
    """The same key at every token with beta = 1: the inverse is that of a full triangle of ones."""
    say(f"[delta] equal keys {dtype}")
    d = make(1, 160, 2, 1, 64, 32, dtype, 12)
    d["k"][:] = 0.125
    d["beta"][:] = 1.0
    d["g"][:] = 0.0
    o, fin = check_fwd(d)
    check_bwd(d)


CUS = [[0, 64, 64, 65, 192, 300], [0, 0, 0, 37], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10], [0, 129], [0, 200, 200], [5, 70, 133, 190]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cu", CUS)
def test_packed(cu, dtype):
    say(f"[delta] packed {cu} {dtype}")
    T = cu[-1] + (9 if cu[0] else 0)
    d = make(1, T, 4, 2, 64, 48, dtype, 13, nseq=len(cu) - 1)
    check_fwd(d, cu=cu)
    check_bwd(d, cu=cu)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_outside_sequences(dtype):
    """They may hold anything, and their outputs are left as they were."""
    say(f"[delta] rows outside {dtype}")
    cu, T = [5, 70, 133, 190], 260
    d = make(1, T, 2, 1, 32, 40, dtype, 14, nseq=3)
    for n in ("q", "k", "v", "do", "g", "beta"):
        d[n][:, :5] = float("nan")
        d[n][:, 190:] = float("inf")
    o = torch.full_like(d["v"], 7.0)
    fin = torch.empty_like(d["init"])
    run_fwd(d, cu=cu, o=o, final_state=fin)
    assert (o[:, :5] == 7).all() and (o[:, 190:] == 7).all()
    e = {n: (x[:, 5:190].contiguous() if n in ("q", "k", "v", "do", "g", "beta") else x) for n, x in d.items()}
    cu2 = [c - 5 for c in cu]
    o2, fin2 = run_fwd(e, cu=cu2)
    assert torch.equal(o[:, 5:190], o2) and torch.equal(fin, fin2)
    a, c = run_bwd(d, cu=cu), run_bwd(e, cu=cu2)
    for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
        assert torch.equal(a[n][:, 5:190], c[n]), n
    assert torch.equal(a["dinit"], c["dinit"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_a_projection(dtype):
    say(f"[delta] rows of a projection {dtype}")
    b, T, H, Hk, dk, dv = 2, 150, 4, 2, 64, 40
    d = make(b, T, H, Hk, dk, dv, dtype, 15)
    wide = torch.full((b, T, 2 * Hk * dk + H * dv + 24), float("nan"), dtype=dtype, device="cuda")
    at = [0, Hk * dk, 2 * Hk * dk + 8, 2 * Hk * dk + 8 + H * dv]
    e = dict(d, q=wide[..., at[0]:at[1]].unflatten(-1, (Hk, dk)), k=wide[..., at[1]:at[1] + Hk * dk].unflatten(-1, (Hk, dk)),
             v=wide[..., at[2]:at[3]].unflatten(-1, (H, dv)))
    for n in ("q", "k", "v"):
        e[n].copy_(d[n])
    for x, y in zip(run_fwd(d), run_fwd(e)):
        assert torch.equal(x, y)
    x, y = run_bwd(d), run_bwd(e)
    assert all(torch.equal(x[n], y[n]) for n in x)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("b,H,Hk,dk,dv", [(1, 1, 1, 8, 8), (3, 4, 2, 64, 40), (5, 6, 3, 128, 128), (2, 2, 1, 256, 256), (70, 2, 2, 16, 24),
                                         (2, 3, 3, 200, 96)])
def test_step(b, H, Hk, dk, dv, dtype):
    say(f"[delta step] {b} {H} {Hk} {dk} {dv} {dtype}")
    d = make(b, 1, H, Hk, dk, dv, dtype, 20 + b, lead=(b,))
    n = b + 3
    g = torch.Generator().manual_seed(5)
    pool = torch.randn(n, H, dv, dk, generator=g).cuda()
    slots = torch.randperm(n, generator=g)[:b].to(torch.int32)
    before = n64(pool)
    o = ssd.gated_delta_step(pool, d["q"], d["k"], d["v"], d["g"], d["beta"], slots=slots.cuda(), scale=0.5)
    q, k, v, ld, beta = arrays(d)
    want = before.copy()
    out = np.zeros(v.shape)
    for i, s in enumerate(slots.tolist()):
        w, f = ref.forward(*(ref.expand(x[i:i + 1], H) for x in (q, k)), v[i:i + 1], ld[i:i + 1], beta[i:i + 1], 0.5, before[s])
        out[i], want[s] = w[0], f
    ref.check(n64(o), out, ref.rel_forward(1, dk), dtype == BF, "o")
    ref.check(n64(pool), want, ref.rel_forward(1, dk), False, "state")


def test_step_padding_and_repeated_slots():
    """Entries outside the pool are padding; entries of one slot are its tokens in the order of the batch."""
    say("[delta step] padding, repeated slots")
    d = make(6, 1, 2, 1, 64, 32, BF, 31, lead=(6,))
    pool = torch.randn(3, 2, 32, 64, generator=torch.Generator().manual_seed(1)).cuda()
    slots = torch.tensor([2, -1, 0, 2, 3, 2], dtype=torch.int32, device="cuda")
    want = pool.clone()
    outs = []
    for i in range(6):
        s = int(slots[i])
        row = [d[n][i:i + 1].contiguous() for n in ("q", "k", "v", "g", "beta")]
        outs.append(ssd.gated_delta_step(want, *row, slots=slots[i:i + 1], scale=0.5) if 0 <= s < 3 else torch.zeros_like(row[2]))
    o = ssd.gated_delta_step(pool, d["q"], d["k"], d["v"], d["g"], d["beta"], slots=slots, scale=0.5)
    assert torch.equal(o, torch.cat(outs)) and torch.equal(pool, want)
    no = ssd.gated_delta_step(pool.clone(), d["q"][:3], d["k"][:3], d["v"][:3], None, d["beta"][:3], scale=0.5)
    zero = ssd.gated_delta_step(pool.clone(), d["q"][:3], d["k"][:3], d["v"][:3], torch.zeros_like(d["g"][:3]), d["beta"][:3], scale=0.5)
    assert torch.equal(no, zero)


def test_empty_calls():
    say("[delta] no tokens")
    d = make(2, 5, 2, 1, 16, 8, BF, 32)
    e = {n: (x[:, :0] if n in ("q", "k", "v", "do", "g", "beta") else x) for n, x in d.items()}
    o, fin = run_fwd(e)
    assert o.shape == (2, 0, 2, 8) and torch.equal(fin, d["init"])
    assert torch.equal(run_bwd(e)["dinit"], d["dfinal"])
    pool = torch.randn(2, 2, 8, 16, device="cuda")
    assert ssd.gated_delta_step(pool, *(d[n][:0, 0].contiguous() for n in ("q", "k", "v", "g", "beta"))).shape == (0, 2, 8)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_in_parts_and_steps(dtype):
    """A prompt continued from its state, then token by token, is the whole prompt."""
    say(f"[delta] parts and steps {dtype}")
    d = make(1, 180, 4, 2, 64, 64, dtype, 33)
    o, fin = run_fwd(d)
    part = lambda a, b: dict(d, **{n: d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")})
    o1, s1 = run_fwd(part(0, 77))
    o2, s2 = run_fwd(dict(part(77, 170), init=s1))
    pool, outs = s2.clone(), []
    for t in range(170, 180):
        outs.append(ssd.gated_delta_step(pool, *(d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), scale=0.5))
    got = torch.cat([o1, o2, torch.stack(outs, 1)], 1)
    rel = 2 * ref.rel_forward(180, 64)   # both sides are off the rule
    ref.check(n64(got), n64(o), rel + (ref.UBF if dtype == BF else 0), dtype == BF, "o")
    ref.check(n64(pool), n64(fin), rel, False, "state")


def test_other_stream_and_repeats():
    say("[delta] stream, bit for bit")
    d = make(1, 400, 8, 4, 128, 128, BF, 34)
    want, grads = run_fwd(d), run_bwd(d)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again, g2 = run_fwd(d), run_bwd(d)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    assert all(torch.equal(grads[n], g2[n]) for n in grads)


def test_captured():
    """Forward, backward and steps in one graph, replayed on new contents; eager work between the replays."""
    say("[delta] captured")
    d = make(1, 130, 4, 2, 64, 64, BF, 35)
    pool = torch.randn(4, 4, 64, 64, device="cuda")
    slots = torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    tok = {n: d[n][0, :2].contiguous() for n in ("q", "k", "v", "g", "beta")}
    steps = lambda p: ssd.gated_delta_step(p, *tok.values(), slots=slots, scale=0.5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_fwd(d), run_bwd(d), steps(pool.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    kept = pool.clone()
    with torch.cuda.graph(graph):
        o, fin = run_fwd(d)
        grads = run_bwd(d)
        y = steps(pool)
    pool.copy_(kept)
    for r in range(3):
        e = make(1, 130, 4, 2, 64, 64, BF, 40 + r)
        for n in d:
            d[n].copy_(e[n])
        for n in tok:
            tok[n].copy_(d[n][0, :2])
        eager = pool.clone()
        graph.replay()
        torch.cuda.synchronize()
        o2, fin2 = run_fwd(d)
        g2 = run_bwd(d)
        y2 = steps(eager)
        assert torch.equal(o, o2) and torch.equal(fin, fin2) and torch.equal(y, y2) and torch.equal(pool, eager)
        assert all(torch.equal(grads[n], g2[n]) for n in grads)


def test_one_workspace_for_many_calls():
    """A caller's workspace serves calls of one stream one after the other, whatever it holds."""
    say("[delta] workspace")
    d = make(2, 100, 4, 2, 64, 64, BF, 36)
    shape = ssd.gated_delta_shape(d["q"], d["k"], d["v"])
    size = max(ssd.gated_delta_workspace_bytes(shape), ssd.gated_delta_bwd_workspace_bytes(shape))
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    want, grads = run_fwd(d), run_bwd(d)
    for _ in range(2):
        got, g2 = run_fwd(d, workspace=ws), run_bwd(d, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(want, got)) and all(torch.equal(grads[n], g2[n]) for n in grads)
    assert (ws[size:] == 255).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_finite(dtype):
    """They stay in their sequence, and in a prompt in the chunks from theirs on."""
    say(f"[delta] not finite {dtype}")
    cu = [0, 100, 300, 350]
    d = make(1, 350, 2, 1, 32, 32, dtype, 37, nseq=3)
    want, gw = run_fwd(d, cu=cu), run_bwd(d, cu=cu)
    for name, bad in (("v", float("nan")), ("k", float("inf")), ("q", float("nan")), ("g", float("nan")), ("beta", float("inf"))):
        e = {n: (None if x is None else x.clone()) for n, x in d.items()}
        e[name][0, 240] = bad
        got, gg = run_fwd(e, cu=cu), run_bwd(e, cu=cu)
        keep = list(range(0, 228)) + list(range(300, 350))   # the chunk of token 240 begins at 100 + 128
        assert torch.equal(got[0][:, keep], want[0][:, keep]), name
        assert torch.equal(got[1][[0, 2]], want[1][[0, 2]])
        assert not torch.isfinite(got[0][:, 240].float()).all()
        if name != "q":
            assert not torch.isfinite(got[1][1]).any() or name == "beta"
        out = list(range(0, 100)) + list(range(300, 350))
        for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
            assert torch.equal(gg[n][:, out], gw[n][:, out]), (name, n)
        assert torch.equal(gg["dinit"][[0, 2]], gw["dinit"][[0, 2]])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_that_are_not_finite_in_segments(dtype):
    """The same where a walk is cut: a segment's map and own state carry them forwards only."""
    say(f"[delta] not finite, segments {dtype}")
    cu = [0, 1500, 3100]
    d = make(1, 3100, 1, 1, 32, 32, dtype, 38, nseq=2)
    want, gw = run_fwd(d, cu=cu), run_bwd(d, cu=cu)
    for name, at, bad in (("v", 700, float("nan")), ("k", 700, float("inf")), ("g", 2000, float("nan")), ("v", 1499, float("inf"))):
        e = {n: x.clone() for n, x in d.items()}
        e[name][0, at] = bad
        got, gg = run_fwd(e, cu=cu), run_bwd(e, cu=cu)
        s = int(at >= cu[1])
        first = cu[s] + (at - cu[s]) // 64 * 64   # where its chunk begins, at the earliest
        keep = [t for t in range(3100) if t < first or not cu[s] <= t < cu[s + 1]]
        out = [t for t in range(3100) if not cu[s] <= t < cu[s + 1]]
        assert torch.equal(got[0][:, keep], want[0][:, keep]), name
        assert torch.equal(got[1][1 - s], want[1][1 - s]), name
        assert not torch.isfinite(got[0][:, at].float()).all() and not torch.isfinite(got[1][s]).all()
        for n in ("dq", "dk", "dv", "dlog_decay", "dbeta"):
            assert torch.equal(gg[n][:, out], gw[n][:, out]), (name, n)
        assert torch.equal(gg["dinit"][1 - s], gw["dinit"][1 - s])


# A walk in segments, value heads summed in one workgroup, and added up by a launch of their own.
PATHS = [(1, 2600, 2, 1, 64, 64), (58, 67, 18, 9, 16, 24), (1, 150, 4, 2, 32, 48)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", PATHS)
def test_workspace_of_any_contents(shape, dtype):
    """Nothing is read from the workspace that the call has not written, and nothing written behind it."""
    say(f"[delta] workspace of NaN {shape} {dtype}")
    d = make(*shape, dtype, 50)
    size = ssd.gated_delta_bwd_workspace_bytes(ssd.gated_delta_shape(d["q"], d["k"], d["v"]))
    want, grads = run_fwd(d), run_bwd(d)
    assert all(torch.isfinite(x.float()).all() for x in [*want, *grads.values()])
    ws = torch.full((size + 256,), 255, dtype=torch.uint8, device="cuda")
    g2 = run_bwd(d, workspace=ws)
    ws[:size].fill_(255)
    got = run_fwd(d, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(want, got)) and all(torch.equal(grads[n], g2[n]) for n in grads)
    assert (ws[size:] == 255).all()


def test_graphs_that_share_a_workspace():
    """Two graphs on one workspace, replayed in turn, with eager calls on another workspace between."""
    say("[delta] graphs on one workspace")
    ds = [make(*PATHS[0], BF, 51), make(*PATHS[2], BF, 52)]
    size = max(ssd.gated_delta_bwd_workspace_bytes(ssd.gated_delta_shape(d["q"], d["k"], d["v"])) for d in ds)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = [(run_fwd(d), run_bwd(d)) for d in ds]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for d in ds:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((run_fwd(d, workspace=ws), run_bwd(d, workspace=ws)))
        graphs.append(g)
    for r in range(3):
        for i in (0, 1, 0):
            for x in [*outs[i][0], *outs[i][1].values()]:
                x.zero_()
            graphs[i].replay()
            other = run_fwd(ds[1 - i])
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want[1 - i][0], other))
            assert all(torch.equal(x, y) for x, y in zip(want[i][0], outs[i][0]))
            assert all(torch.equal(want[i][1][n], outs[i][1][n]) for n in want[i][1])


def test_two_streams_at_once():
    say("[delta] two streams")
    ds = [make(*PATHS[0], BF, 53), make(1, 700, 8, 4, 128, 128, BF, 54)]
    want = [(run_fwd(d), run_bwd(d)) for d in ds]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(4):
        for s, d in zip(streams, ds):
            with torch.cuda.stream(s):
                got.append((run_fwd(d), run_bwd(d)))
    torch.cuda.synchronize()
    for i, (fwd, grads) in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(want[i % 2][0], fwd))
        assert all(torch.equal(want[i % 2][1][n], grads[n]) for n in grads)

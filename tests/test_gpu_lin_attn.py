"""GPU: linear attention with one decay a head (prompts, gradients, the one-token
step) against the recurrence in 64 bits; the bounds are those of layer_ref.py.
"""
import sys

import numpy as np
import pytest
import torch

import layer_ref as ref
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


def decays(H, kind="mixed"):
    x = np.linspace(1.0, 10.0, H) if H > 1 else np.array([4.0])
    ld = np.log1p(-(2.0 ** -x))
    if kind == "edge":   # no memory at all, none forgotten, nearly none kept
        ld[0] = -np.inf
        if H > 1:
            ld[1] = 0.0
        if H > 2:
            ld[2] = -50.0
    return torch.tensor(ld, dtype=F32)


def make(b, T, H, Hk, dk, dv, dtype, seed, nseq=None, states=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(dtype).cuda()
    st = (nseq or b, H, dv, dk)
    d = dict(q=r(b, T, H, dk), k=r(b, T, Hk, dk), v=r(b, T, Hk, dv), do=r(b, T, H, dv))
    f = lambda: (4 * torch.randn(*st, generator=g)).cuda() if states else None
    d.update(init=f(), dfinal=f())
    return d


def memory(ld, T):
    """Steps over which a term matters: the rounding of later steps acts on what is left of it."""
    return T


def check_fwd(d, ld, scale, cu=None, name="", **kw):
    q, k, v = d["q"], d["k"], d["v"]
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, fin = ssd.lin_attn_fwd(q, k, v, ld.cuda(), cu_seqlens=cut, scale=scale, initial_state=d["init"], **kw)
    torch.cuda.synchronize()
    want, E = ref.attention(n64(q), n64(k), n64(v), n64(ld), scale, n64(d["init"]), cu)
    T, dk = q.shape[1], q.shape[3]
    kind = "bf16" if q.dtype == BF else "fp32"
    got = n64(o)
    if cu is not None:
        got = got[:, cu[0]:cu[-1]]
        want["o"], E["o"] = want["o"][:, cu[0]:cu[-1]], E["o"][:, cu[0]:cu[-1]]
    ref.check(got, want["o"], E["o"], kind, T, dk, name + " o")
    ref.check(n64(fin), want["final"], E["final"], "state" if q.dtype == BF else "fp32", T, dk, name + " final")
    return o, fin


def check_bwd(d, ld, scale, cu=None, name=""):
    q, k, v = d["q"], d["k"], d["v"]
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = ssd.lin_attn_bwd(q, k, v, ld.cuda(), d["do"], cu_seqlens=cut, scale=scale, initial_state=d["init"],
                         dfinal_state=d["dfinal"], want_dinit=True)
    torch.cuda.synchronize()
    want, E = ref.attention_bwd(n64(q), n64(k), n64(v), n64(ld), scale, n64(d["do"]), n64(d["init"]), n64(d["dfinal"]), cu)
    T, n = q.shape[1], max(q.shape[3], v.shape[3]) * (q.shape[2] // k.shape[2])
    kind = "bf16" if q.dtype == BF else "fp32"
    for name_, knd in (("dq", kind), ("dk", kind), ("dv", kind), ("dinit", "state" if q.dtype == BF else "fp32")):
        a, w, e = n64(g[name_]), want[name_], E[name_]
        if cu is not None and name_ != "dinit":
            a, w, e = a[:, cu[0]:cu[-1]], w[:, cu[0]:cu[-1]], e[:, cu[0]:cu[-1]]
        ref.check(a, w, e, knd, T, n, f"{name} {name_}")
    return g


# b, T, H, Hk, dk, dv
SHAPES = [(1, 1, 1, 1, 8, 8), (2, 2, 2, 1, 16, 24), (1, 63, 3, 3, 64, 64), (1, 64, 2, 2, 128, 128), (2, 65, 4, 2, 40, 96),
          (1, 130, 2, 1, 128, 64), (1, 257, 2, 2, 64, 200), (1, 300, 6, 2, 96, 32), (1, 190, 1, 1, 256, 256),
          (3, 129, 2, 2, 32, 128), (1, 700, 4, 4, 16, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    say(f"[lin fwd] {shape} {dtype}")
    b, T, H, Hk, dk, dv = shape
    check_fwd(make(*shape, dtype, seed=T), decays(H), dk ** -0.5, name=str(shape))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    say(f"[lin bwd] {shape} {dtype}")
    b, T, H, Hk, dk, dv = shape
    check_bwd(make(*shape, dtype, seed=100 + T), decays(H), dk ** -0.5, name=str(shape))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_no_states(dtype):
    say(f"[lin] no states {dtype}")
    d = make(2, 150, 4, 4, 64, 64, dtype, 7, states=False)
    check_fwd(d, decays(4), 0.3)
    check_bwd(d, decays(4), 0.3)
    o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], decays(4).cuda(), want_final=False)
    assert fin is None


@pytest.mark.parametrize("dtype", [BF, F32])
def test_edge_decays(dtype):
    """lam = 0 (each token alone), 1 (a plain sum) and almost 0."""
    say(f"[lin] edge decays {dtype}")
    d = make(1, 200, 4, 2, 32, 64, dtype, 11)
    check_fwd(d, decays(4, "edge"), -0.7)
    check_bwd(d, decays(4, "edge"), -0.7)


CUS = [[0, 64, 64, 65, 192, 300], [0, 0, 0, 37], [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10], [0, 129], [0, 500, 500]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cu", CUS)
def test_packed(cu, dtype):
    """Empty sequences, single tokens, ends inside and on a chunk; their states."""
    say(f"[lin] packed {cu} {dtype}")
    d = make(1, cu[-1], 4, 2, 64, 40, dtype, 13 + cu[-1], nseq=len(cu) - 1)
    check_fwd(d, decays(4), 0.125, cu)
    check_bwd(d, decays(4), 0.125, cu)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(dtype):
    rng = np.random.default_rng(3)
    cu = [0] + np.cumsum(rng.integers(0, 7, 150)).tolist()
    say(f"[lin] {len(cu) - 1} sequences {dtype}")
    d = make(1, cu[-1], 2, 2, 32, 32, dtype, 17, nseq=len(cu) - 1)
    check_fwd(d, decays(2), 0.2, cu)
    check_bwd(d, decays(2), 0.2, cu)


@pytest.mark.parametrize("S", [64, 65, 700])
def test_sequence_of_every_slot(S):
    """As many sequences as a wave has lanes, one more, and far more, some empty: each alone gives the same."""
    rng = np.random.default_rng(S)
    cu = [0] + np.cumsum(rng.integers(0, 4, S)).tolist()
    say(f"[lin] {S} sequences, {cu[-1]} tokens")
    d = make(1, cu[-1], 2, 1, 16, 16, F32, 61, nseq=S)
    check_fwd(d, decays(2), 0.3, cu)


@pytest.mark.parametrize("dims", [(64, 128), (128, 64), (16, 256)])
@pytest.mark.parametrize("T", [1, 2, 7, 32])
def test_short_sequences_keep_their_scores(T, dims):
    """From no state, the first 32 tokens are as exact as their type: their scores enter as the sum of two bf16
    values, which leaves 2^-16 of each (2^-8 of 2^-8), so that what remains is the result's own rounding:
    |err| <= 2^-8 |ref| + 2^-16 E + the bound of 32-bit sums; once rounded, a score would add 2^-8 E."""
    dk, dv = dims
    say(f"[lin short] {T} {dims}")
    d = make(2, T, 4, 4, dk, dv, BF, 60 + T)
    ld = decays(4)
    q, k, v, do = (n64(d[n]) for n in ("q", "k", "v", "do"))
    o, _ = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], ld.cuda(), scale=0.25)
    g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld.cuda(), d["do"], scale=0.25)
    want, E = ref.attention(q, k, v, n64(ld), 0.25)
    gw, gE = ref.attention_bwd(q, k, v, n64(ld), 0.25, do)
    for name, got, w, e in [("o", o, want["o"], E["o"])] + [(n, g[n], gw[n], gE[n]) for n in ("dq", "dk", "dv")]:
        left = (2.0 ** -16 + (2 * T + max(dk, dv) + 16) * 2.0 ** -24) * e
        over = abs(n64(got) - w) - (2.0 ** -8 * (abs(w) + left) + left)
        assert over.max() <= 0, (name, over.max())


def test_decay_not_a_number_shows():
    d = make(1, 80, 2, 2, 32, 32, BF, 63)
    ld = torch.tensor([float("nan"), -0.1], device="cuda")
    o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], ld, initial_state=d["init"])
    assert torch.all(torch.isnan(fin[:, 0])) and torch.all(torch.isfinite(fin[:, 1])) and torch.all(torch.isfinite(o[:, :, 1]))


def test_offsets_beyond_32_bits():
    """Rows so wide, and a batch so long, that offsets pass 2^31 elements: the last head and the last
    tokens against a call on them alone (the same kernels on the same 64-token chunks; blocks may
    be cut elsewhere, so each side is within its bound of the same values)."""
    H, D, T = 272, 128, 65600
    ld = decays(H).cuda()
    n = T * H * D
    assert n > 2 ** 31
    q = torch.empty(1, T, H, D, dtype=BF, device="cuda").normal_()
    k = torch.empty(1, T, 1, D, dtype=BF, device="cuda").normal_()
    v = torch.empty(1, T, 1, D, dtype=BF, device="cuda").normal_()
    o, fin = ssd.lin_attn_fwd(q, k, v, ld, scale=0.1)
    head = q[:, :, H - 1:]
    assert head.stride(1) == H * D
    o1, f1 = ssd.lin_attn_fwd(head, k, v, ld[H - 1:], scale=0.1)
    a, b = o[:, -4096:, H - 1].double(), o1[:, -4096:, 0].double()
    assert torch.linalg.norm(a - b) <= 2 * 7e-3 * torch.linalg.norm(b)
    assert torch.linalg.norm(fin[:, H - 1].double() - f1[:, 0].double()) <= 1e-5 * torch.linalg.norm(f1.double())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_outside_sequences_left_alone(dtype):
    say(f"[lin] rows before and behind the sequences {dtype}")
    cu = [5, 90, 90, 260]
    d = make(1, 300, 4, 2, 64, 64, dtype, 19, nseq=3)
    for t in "qkv":   # what lies outside the sequences is not used
        d[t][:, :5] = float("nan")
        d[t][:, 260:] = float("nan")
    o = torch.full((1, 300, 4, 64), 7.0, dtype=dtype, device="cuda")
    q, k, v = (torch.nan_to_num(d[t]) for t in "qkv")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], decays(4).cuda(), cu_seqlens=cut, initial_state=d["init"], o=o)
    assert torch.all(o[:, :5] == 7) and torch.all(o[:, 260:] == 7)
    want, wf = ssd.lin_attn_fwd(q, k, v, decays(4).cuda(), cu_seqlens=cut, initial_state=d["init"])
    assert torch.equal(got[:, 5:260], want[:, 5:260]) and torch.equal(fin, wf)
    assert torch.equal(fin[1], d["init"][1])


def test_cu_outside_the_batch_is_brought_in():
    """Entries past the batch: the sequences end with it (nothing is read or written beyond)."""
    d = make(1, 100, 2, 2, 32, 32, BF, 23, nseq=2)
    cu = torch.tensor([-3, 60, 1000], dtype=torch.int32, device="cuda")
    ok = torch.tensor([0, 60, 100], dtype=torch.int32, device="cuda")
    a = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], decays(2).cuda(), cu_seqlens=cu, initial_state=d["init"])
    b = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], decays(2).cuda(), cu_seqlens=ok, initial_state=d["init"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_wider_rows(dtype):
    """q, k and v as slices of one projection's rows."""
    say(f"[lin] wider rows {dtype}")
    b, T, H, Hk, dk, dv = 2, 100, 4, 2, 64, 32
    w = torch.randn(b, T, H * dk + Hk * dk + Hk * dv, generator=torch.Generator().manual_seed(5)).to(dtype).cuda()
    q, k, v = w.split([H * dk, Hk * dk, Hk * dv], -1)
    q, k, v = q.unflatten(-1, (H, dk)), k.unflatten(-1, (Hk, dk)), v.unflatten(-1, (Hk, dv))
    assert not q.is_contiguous()
    do = torch.randn(b, T, H, dv, device="cuda").to(dtype)
    ld = decays(H).cuda()
    a, b_ = ssd.lin_attn_fwd(q, k, v, ld), ssd.lin_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), ld)
    assert torch.equal(a[0], b_[0]) and torch.equal(a[1], b_[1])
    ga, gb = ssd.lin_attn_bwd(q, k, v, ld, do), ssd.lin_attn_bwd(q.contiguous(), k.contiguous(), v.contiguous(), ld, do)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(ga[n], gb[n])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_in_pieces(dtype):
    """A prompt in pieces, each from the state the last one left, then one token at a time."""
    say(f"[lin] in pieces {dtype}")
    H, dk, dv, T = 2, 64, 64, 333
    d = make(1, T, H, H, dk, dv, dtype, 29)
    ld = decays(H)
    want, E = ref.attention(n64(d["q"]), n64(d["k"]), n64(d["v"]), n64(ld), 0.2, n64(d["init"]))
    state, at, outs = d["init"], 0, []
    for n in (1, 64, 100, 163):
        o, state = ssd.lin_attn_fwd(d["q"][:, at:at + n].contiguous(), d["k"][:, at:at + n].contiguous(),
                                    d["v"][:, at:at + n].contiguous(), ld.cuda(), scale=0.2, initial_state=state)
        outs.append(o)
        at += n
    for t in range(at, T):
        outs.append(ssd.lin_attn_step(state, d["q"][:, t], d["k"][:, t].contiguous(), d["v"][:, t].contiguous(), ld.cuda(),
                                      scale=0.2)[:, None])
    kind = "bf16" if dtype == BF else "fp32"
    ref.check(n64(torch.cat(outs, 1)), want["o"], E["o"], kind, T, dk, "o")
    # five pieces leave five times the splitting's remainder in the state at most
    ref.check(n64(state), want["final"], 5 * E["final"], "state" if dtype == BF else "fp32", T, dk, "state")


def test_gradient_against_differences():
    """<grad, direction> against central differences of the 64-bit loss (which is
    of second order in each direction taken alone, so the difference is exact)."""
    b, T, H, Hk, dk, dv = 1, 90, 4, 2, 16, 24
    d = make(b, T, H, Hk, dk, dv, F32, 31)
    ld, scale = decays(H), 0.4
    g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld.cuda(), d["do"], scale=scale, initial_state=d["init"],
                         dfinal_state=d["dfinal"], want_dinit=True)
    x = {n: n64(d[n]) for n in ("q", "k", "v", "init")}

    def loss(y):
        r, _ = ref.attention(y["q"], y["k"], y["v"], n64(ld), scale, y["init"])
        return (r["o"] * n64(d["do"])).sum() + (r["final"] * n64(d["dfinal"])).sum()

    rng = np.random.default_rng(1)
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("init", "dinit")):
        u = rng.standard_normal(x[n].shape)
        up, down = dict(x), dict(x)
        up[n], down[n] = x[n] + 0.5 * u, x[n] - 0.5 * u
        diff = loss(up) - loss(down)
        got = (n64(g[gn]) * u).sum()
        size = np.abs(n64(g[gn]) * u).sum()
        assert abs(diff - got) <= 1e-5 * size, (n, diff, got)


# ---------------------------------------------------------------- the step

STEPS = [(1, 1, 1, 8, 8), (3, 2, 1, 64, 64), (5, 6, 3, 40, 96), (2, 4, 4, 128, 128), (4, 2, 2, 256, 200), (33, 8, 2, 16, 256)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", STEPS)
def test_step(shape, dtype):
    say(f"[lin step] {shape} {dtype}")
    b, H, Hk, dk, dv = shape
    d = make(b, 1, H, Hk, dk, dv, dtype, 41)
    pool = torch.randn(b + 3, H, dv, dk, generator=torch.Generator().manual_seed(2)).cuda() * 3
    slots = torch.randperm(b + 3, generator=torch.Generator().manual_seed(4))[:b].to(torch.int32)
    before = n64(pool)
    ld = decays(H)
    o = ssd.lin_attn_step(pool, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], ld.cuda(), slots=slots.cuda(), scale=0.3)
    want, E = ref.attention(n64(d["q"]), n64(d["k"]), n64(d["v"]), n64(ld), 0.3, before[slots.numpy()])
    ref.check(n64(o), want["o"][:, 0], E["o"][:, 0], "bf16" if dtype == BF else "fp32", 1, dk, "o")
    after = before.copy()
    after[slots.numpy()] = want["final"]
    Ea = abs(before)
    Ea[slots.numpy()] = E["final"]
    ref.check(n64(pool), after, Ea, "fp32", 1, 1, "pool")
    rest = [i for i in range(b + 3) if i not in slots.tolist()]
    assert np.array_equal(n64(pool)[rest], before[rest])


def test_step_padding_and_repeated_slots():
    """Slots outside the pool are padding; entries of one slot are its tokens in order."""
    H, dk, dv = 2, 64, 48
    order = [2, -1, 0, 2, 7, 2, 0, 3, 900]
    d = make(len(order), 1, H, H, dk, dv, F32, 43)
    pool = torch.randn(4, H, dv, dk, generator=torch.Generator().manual_seed(6)).cuda()
    one = pool.clone()
    ld = decays(H).cuda()
    sl = torch.tensor(order, dtype=torch.int32, device="cuda")
    o = ssd.lin_attn_step(pool, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], ld, slots=sl, scale=0.5)
    for i, s in enumerate(order):
        if not 0 <= s < 4:
            assert torch.all(o[i] == 0)
            continue
        w = ssd.lin_attn_step(one, d["q"][i], d["k"][i], d["v"][i], ld, slots=sl[i:i + 1], scale=0.5)
        assert torch.equal(o[i:i + 1], w)
    assert torch.equal(pool, one)


def test_step_many_repeats():
    """One slot many times in one call, more entries than a workgroup has threads."""
    b, H = 600, 1
    d = make(b, 1, H, H, 16, 16, F32, 47)
    pool = torch.zeros(2, H, 16, 16, device="cuda")
    sl = torch.ones(b, dtype=torch.int32, device="cuda")
    o = ssd.lin_attn_step(pool, d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], decays(H).cuda(), slots=sl)
    seq = lambda t: t[:, 0][None]
    want, E = ref.attention(n64(seq(d["q"])), n64(seq(d["k"])), n64(seq(d["v"])), n64(decays(H)), 1.0)
    ref.check(n64(o)[None], want["o"], E["o"], "fp32", b, 16, "o")
    assert torch.all(pool[0] == 0)


def test_step_decay_does_not_drift():
    """65536 steps that only decay a state: the decay's own rounding to 32 bits must not enter with every step.

    Of the log decays near -1e-5 the one whose decay is furthest from an fp32 value is taken: rounded once to 32
    bits it would be off by 65536 times that, 1.9e-3 of the state.

    What is left is the rounding of the state, and it has a sign. With c = 1 - lam, a state of n units in the last
    place loses d = c n units a step, rounded to a whole m; d itself falls by delta = c m a step. While m stands,
    d runs from m + 1/2 to m - 1/2 and the errors m - d cancel but for half a unit; a run cut short, at either end
    or where n passes a power of two, leaves at most 1 / (8 delta) units. Here c >= 1e-5 and n >= 2^23, so m >= 83
    and 1 / (8 delta) <= 151 units of at most 2^-23 of the state: 1.8e-5. A state of 0.5 to 1.5 that falls by
    half passes at most two powers of two: six runs cut short, 1.1e-4, and 100 whole ones a power of two, three
    times 50 units of 2^-23, 1.8e-5.
    """
    cand = torch.arange(200, dtype=torch.float32) * -1e-8 - 1e-5
    lam = torch.exp(cand.double())
    off = (lam.float().double() - lam).abs()
    ld = cand[off.argmax()]
    assert off.max() * 65536 > 1e-3
    b, dk, dv = 2048, 32, 256
    pool = torch.rand(1, 1, dv, dk, generator=torch.Generator().manual_seed(8)).cuda() + 0.5
    first = pool.double()
    zero = torch.zeros(b, 1, dk, device="cuda")
    v = torch.ones(b, 1, dv, device="cuda")
    sl = torch.zeros(b, dtype=torch.int32, device="cuda")
    for _ in range(32):
        ssd.lin_attn_step(pool, zero, zero, v, ld.cuda()[None], slots=sl)
    left = torch.exp(ld.double() * 65536).item()
    drift = (pool.double() / (first * left) - 1).abs().max().item()
    say(f"[lin step] drift {drift:.2e}")
    assert drift < 1.3e-4


def test_other_stream_and_two_calls_at_once():
    d = make(1, 500, 4, 4, 64, 64, BF, 51)
    e = make(1, 700, 4, 4, 64, 64, BF, 52)
    ld = decays(4).cuda()
    want = [ssd.lin_attn_fwd(x["q"], x["k"], x["v"], ld, initial_state=x["init"]) for x in (d, e)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for x, s in zip((d, e), streams):
        with torch.cuda.stream(s):
            got.append(ssd.lin_attn_fwd(x["q"], x["k"], x["v"], ld, initial_state=x["init"]))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_repeats_bitwise():
    d = make(2, 1000, 8, 2, 64, 64, BF, 53)
    ld = decays(8).cuda()
    one = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld, d["do"], initial_state=d["init"], dfinal_state=d["dfinal"], want_dinit=True)
    for _ in range(3):
        two = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld, d["do"], initial_state=d["init"], dfinal_state=d["dfinal"],
                               want_dinit=True)
        for n in one:
            assert torch.equal(one[n], two[n]), n

"""GPU: the layer operators run together as a model runs them: prompts, their
states into a pool, forks, steps, norms, compaction; a training step's chain of
gradients; captured in a graph.
"""
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


def n64(t):
    return t.detach().cpu().double().numpy()


def decays(H):
    return torch.tensor(np.log1p(-(2.0 ** -np.linspace(3, 9, H))), dtype=F32)


def test_serving_run():
    """Three prompts prefilled together; one forked in two; four streams decoded; one ends and the
    pool is made dense; decoding goes on. Every output against each stream's recurrence in 64 bits."""
    H, Hk, dk, dv, scale = 4, 2, 64, 64, 0.125
    lens = [70, 1, 200]
    ld = decays(H)
    g = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g)
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    prompt = [r(1, sum(lens), h, d).cuda() for h, d in ((H, dk), (Hk, dk), (Hk, dv))]
    o, fin = ssd.lin_attn_fwd(*prompt, ld.cuda(), cu_seqlens=cu, scale=scale)
    pool = torch.full((1, 6, H, dv, dk), 9.0, device="cuda")
    at = [5, 0, 3]                                   # slots of the three streams
    pool[0, at] = fin
    ssd.pages_clear(pool, torch.tensor([2], dtype=torch.int32, device="cuda"))   # a stream without a prompt
    ssd.pages_copy(pool, torch.tensor([3], dtype=torch.int32, device="cuda"), torch.tensor([1], dtype=torch.int32, device="cuda"))
    hist = [[n64(t[0, a:e]) for t in prompt] for a, e in zip(cu[:-1].tolist(), cu[1:].tolist())]
    streams = {5: hist[0], 0: hist[1], 3: hist[2], 1: [x.copy() for x in hist[2]],
               2: [np.zeros((0, h, d)) for h, d in ((H, dk), (Hk, dk), (Hk, dv))]}
    w, z_all = (1 + 0.1 * r(H * dv)).cuda(), []

    def decode(slots, steps):
        for _ in range(steps):
            q, k, v, z = (r(len(slots), *s) for s in ((H, dk), (Hk, dk), (Hk, dv), (H * dv,)))
            sl = torch.tensor(slots, dtype=torch.int32, device="cuda")
            o = ssd.lin_attn_step(pool[0], q.cuda(), k.cuda(), v.cuda(), ld.cuda(), slots=sl, scale=scale)
            y, _ = ssd.group_norm(o.view(len(slots), -1), H, w, z=z.cuda(), want_stats=False)
            for i, s in enumerate(slots):
                streams[s] = [np.concatenate([a, n64(t)[None]]) for a, t in zip(streams[s], (q[i], k[i], v[i]))]
                sq, sk, sv = streams[s]
                want, E = ref.attention(sq[None], sk[None], sv[None], n64(ld), scale)
                T = sq.shape[0]
                ref.check(n64(o[i]), want["o"][0, -1], E["o"][0, -1], "fp32", T, dk, f"slot {s}")
                # the norm of what the step left, in 64 bits: a few 2^-24 of (1 + |t|) (1 + |z|)
                ny = ref.norm(n64(o[i]).reshape(1, 1, -1), H, n64(w), None, n64(z[i]).reshape(1, 1, -1), 1e-5, "none", "after", True)
                assert np.max(abs(n64(y[i]) - ny["y"].ravel()) / ((1 + abs(ny["t"].ravel())) * (1 + abs(n64(z[i]))))) <= 64 * 2.0 ** -24

    decode([5, 0, 3, 1, 2], 3)
    live = torch.tensor([1, 1, 1, 0, 0, 1], dtype=torch.bool, device="cuda")   # slot 3 has ended, 4 was never used
    where, count = ssd.pages_compact(pool, live)
    where = where.tolist()
    assert count.item() == 4 and sorted(x for x in where if x >= 0) == [0, 1, 2, 3]
    streams = {where[s]: h for s, h in streams.items() if where[s] >= 0}
    decode([3, 2, 1, 0], 2)


def test_beams_reordered():
    """Beams take their parents' states, some twice, in one call, and go on as if run alone."""
    H, d = 2, 32
    ld = decays(H).cuda()
    g = torch.Generator().manual_seed(4)
    pool = torch.randn(2, 5, H, d, d, generator=g).cuda()
    alone = pool.clone()
    parent = [2, 2, 0, 4, 3]
    ssd.pages_copy(pool, torch.tensor(parent, dtype=torch.int32, device="cuda"), torch.arange(5, dtype=torch.int32, device="cuda"))
    x = [torch.randn(5, H, d, generator=g).cuda() for _ in range(3)]
    for layer in range(2):
        o = ssd.lin_attn_step(pool[layer], *x, ld)
        for i, p in enumerate(parent):
            s = alone[layer, p:p + 1].clone()
            assert torch.equal(o[i:i + 1], ssd.lin_attn_step(s, *[t[i:i + 1] for t in x], ld))
            assert torch.equal(pool[layer, i], s[0])


def chain(q, k, v, z, w, ld, scale, dy, ws=None):
    b, T, H, dv = z.shape
    o, _ = ssd.lin_attn_fwd(q, k, v, ld, scale=scale, want_final=False, workspace=ws and ws[0])
    rows = lambda t: t.view(b * T, H * dv)
    y, stats = ssd.group_norm(rows(o), H, w, z=rows(z))
    gn = ssd.group_norm_bwd(rows(o), H, stats, rows(dy), w, z=rows(z))
    ga = ssd.lin_attn_bwd(q, k, v, ld, gn["dx"].view(o.shape), scale=scale, workspace=ws and ws[1])
    return dict(y=y, dq=ga["dq"], dk=ga["dk"], dv=ga["dv"], dz=gn["dz"], dw=gn["dweight"])


def test_training_chain_against_differences():
    """Attention, then the norm of its heads and the gate: the gradients of the whole against
    differences of its 64-bit form (central, of relative error h^2 and 2^-53 / h with h = 1e-5)."""
    b, T, H, Hk, dk, dv, scale = 1, 70, 4, 2, 16, 32, 0.25
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g).cuda()
    q, k, v, z, dy = r(b, T, H, dk), r(b, T, Hk, dk), r(b, T, Hk, dv), r(b, T, H, dv), r(b, T, H, dv)
    w, ld = 1 + 0.1 * r(H * dv), decays(H).cuda()
    out = chain(q, k, v, z, w, ld, scale, dy)
    base = dict(q=n64(q), k=n64(k), v=n64(v), z=n64(z), w=n64(w))

    def loss(x):
        o, _ = ref.attention(x["q"], x["k"], x["v"], n64(ld), scale)
        flat = lambda t: t.reshape(b * T, 1, H * dv)
        y = ref.norm(flat(o["o"]), H, x["w"], None, flat(x["z"]), 1e-5, "none", "after", True)["y"]
        return (y * flat(n64(dy))).sum()

    rng, h = np.random.default_rng(0), 1e-5
    for n, gn in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("z", "dz"), ("w", "dw")):
        u = rng.standard_normal(base[n].shape)
        up, down = dict(base), dict(base)
        up[n], down[n] = base[n] + h * u, base[n] - h * u
        diff, got = (loss(up) - loss(down)) / (2 * h), (n64(out[gn]).reshape(u.shape) * u).sum()
        assert abs(diff - got) <= 1e-4 * np.abs(n64(out[gn]).reshape(u.shape) * u).sum(), (n, diff, got)


def capture(fn):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fn()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        out = fn()
    torch.cuda.synchronize()
    return g, out


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graphs_sharing_a_workspace(dtype):
    """Two captured training chains that use one workspace, replayed in turn with eager work
    between them: each replay gives what the eager call gave."""
    b, T, H, Hk, d = 1, 900, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    ld = decays(H).cuda()
    w = torch.ones(H * d, device="cuda")

    def data():
        r = lambda h: torch.randn(b, T, h, d, generator=g).to(dtype).cuda()
        return [r(H), r(Hk), r(Hk), r(H), w, ld, 0.1, r(H)]

    x, y = data(), data()
    sh = ssd.lin_attn_shape(x[0], x[1], x[2])
    n = max(256, ssd.lin_attn_workspace_bytes(sh)), max(256, ssd.lin_attn_bwd_workspace_bytes(sh))
    ws = [torch.empty(i, dtype=torch.uint8, device="cuda") for i in n]
    want = [{k: t.clone() for k, t in chain(*i).items()} for i in (x, y)]
    runs = [capture(lambda i=i: chain(*i, ws=ws)) for i in (x, y)]
    for i in range(3):
        for (graph, out), ref_ in zip(runs, want):
            for t in out.values():
                t.fill_(float("nan"))
            chain(*data())
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            for k in out:
                assert torch.equal(out[k], ref_[k]), (i, k)


def test_decode_graph():
    """A step, its norm and a reordering of the pool, captured: replays advance the streams."""
    H, d, b = 4, 64, 6
    ld = decays(H).cuda()
    g = torch.Generator().manual_seed(9)
    x = [torch.randn(b, H, d, generator=g).to(BF).cuda() for _ in range(4)]
    sl = torch.tensor([3, 1, -1, 0, 3, 7], dtype=torch.int32, device="cuda")
    src, dst = (torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([1, 0, 3], [0, 1, 5]))
    live = torch.tensor([1, 1, 0, 1, 0, 1, 1, 1], dtype=torch.uint8, device="cuda")
    pool0 = torch.randn(1, 8, H, d, d, generator=g).cuda()
    pool = pool0.clone()

    def run(pool):
        o = ssd.lin_attn_step(pool[0], x[0], x[1], x[2], ld, slots=sl, scale=0.2)
        y, _ = ssd.group_norm(o.view(b, -1), H, z=x[3].view(b, -1), want_stats=False)
        ssd.pages_copy(pool, src, dst)
        where, count = ssd.pages_compact(pool, live)
        ssd.pages_clear(pool, torch_slots)
        return [y, where, count]

    torch_slots = torch.tensor([6], dtype=torch.int32, device="cuda")
    graph, out = capture(lambda: run(pool))
    pool.copy_(pool0)
    eager = pool0.clone()
    for i in range(3):
        want = [t.clone() for t in run(eager)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, e in zip(out, want):
            assert torch.equal(a, e), i
        assert torch.equal(pool, eager), i

"""GPU: rotary positions against their definition in 64 bits; the bounds are those of delta_ref.py."""
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
    return t.detach().cpu().double().numpy()


def rnd(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


# b, T, H, Hk, dim, rot
SHAPES = [(1, 1, 1, 1, 2, 2), (2, 3, 2, 1, 8, 8), (1, 65, 4, 2, 64, 64), (2, 130, 8, 8, 128, 128), (1, 33, 3, 1, 80, 48),
          (1, 20, 2, 2, 96, 30), (3, 7, 5, 1, 33, 14), (1, 700, 40, 8, 128, 64), (1, 5, 1, 0, 256, 256), (1, 2, 1, 1, 1024, 1024),
          (1, 3000, 2, 2, 16, 16)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_against_definition(shape, dtype, layout):
    say(f"[rotary] {shape} {dtype} {layout}")
    b, T, H, Hk, dim, rot = shape
    q = rnd(b, T, H, dim, dtype=dtype, seed=1)
    k = rnd(b, T, Hk, dim, dtype=dtype, seed=2) if Hk else None
    freq, _ = ssd.rotary_frequencies(rot, device="cuda")
    off = torch.arange(b, dtype=torch.int32, device="cuda") * 1000
    pos = np.arange(T)[None] + 1000 * np.arange(b)[:, None]
    for inverse, fn in ((False, ssd.rotary), (True, ssd.rotary_bwd)):
        yq, yk = fn(q, k, freq, offsets=off, layout=layout, scale=1.25)
        for x, y, n in ((q, yq, "q"), (k, yk, "k")):
            if x is not None:
                ref.check_rotary(n64(y), n64(x), pos, n64(freq), layout, 1.25, dtype == BF, f"{n} {inverse}", inverse)
        assert (yk is None) == (k is None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_positions(dtype):
    """Positions up to 2^31 - 1 and below 0, with angles of 64 bits; far angles are off by what 64 bits leave of them."""
    say(f"[rotary] far positions {dtype}")
    pos = torch.tensor([[0, 1, -1, 999999, 10 ** 8, 2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    q = rnd(1, 7, 2, 64, dtype=dtype, seed=3)
    freq, _ = ssd.rotary_frequencies(64, device="cuda")
    y, none = ssd.rotary(q, None, freq, positions=pos)
    assert none is None
    ref.check_rotary(n64(y), n64(q), n64(pos), n64(freq), "half", 1.0, dtype == BF, "far")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cu", [[0, 64, 64, 65, 192, 300], [0, 0, 0, 37], [5, 70, 133, 190], [0, 40, 40], [0, 0]])
def test_packed(cu, dtype):
    say(f"[rotary] packed {cu} {dtype}")
    T, n = cu[-1] + 11, len(cu) - 1
    q, k = rnd(1, T, 4, 64, dtype=dtype, seed=4), rnd(1, T, 2, 64, dtype=dtype, seed=5)
    off = torch.tensor([100 * i + 7 for i in range(n)], dtype=torch.int32, device="cuda")
    freq, _ = ssd.rotary_frequencies(64, device="cuda")
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    oq, ok = torch.full_like(q, 9.0), torch.full_like(k, 9.0)
    ssd.rotary(q, k, freq, cu_seqlens=cut, offsets=off, q_out=oq, k_out=ok)
    pos = np.concatenate([np.arange(cu[i + 1] - cu[i]) + 100 * i + 7 for i in range(n)]) if cu[-1] > cu[0] else np.zeros(0)
    for x, y in ((q, oq), (k, ok)):
        ref.check_rotary(n64(y)[0, cu[0]:cu[-1]], n64(x)[0, cu[0]:cu[-1]], pos, n64(freq), "half", 1.0, dtype == BF, str(cu))
        assert (y[:, :cu[0]] == 9).all() and (y[:, cu[-1]:] == 9).all()
    given = torch.zeros(1, T, dtype=torch.int32, device="cuda")
    given[0, cu[0]:cu[-1]] = torch.as_tensor(pos, dtype=torch.int32)
    assert torch.equal(ssd.rotary(q, k, freq, positions=given)[0][:, cu[0]:cu[-1]], oq[:, cu[0]:cu[-1]])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim,rot,layout", [(64, 64, "half"), (80, 48, "interleaved"), (20, 6, "half"), (12, 12, "interleaved")])
def test_rows_of_a_projection_in_place(dim, rot, layout, dtype):
    say(f"[rotary] in place {dim} {rot} {layout} {dtype}")
    b, T, H, Hk = 2, 37, 4, 2
    wide = rnd(b, T, (H + 2 * Hk) * dim, dtype=dtype, seed=6)
    q, k = wide[..., :H * dim].unflatten(-1, (H, dim)), wide[..., H * dim:(H + Hk) * dim].unflatten(-1, (Hk, dim))
    freq, _ = ssd.rotary_frequencies(rot, device="cuda")
    want = ssd.rotary(q.contiguous(), k.contiguous(), freq, layout=layout)
    values = wide[..., (H + Hk) * dim:].clone()
    got = ssd.rotary(q, k, freq, layout=layout, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(wide[..., (H + Hk) * dim:], values)


def test_unaligned_rows():
    """Rows that do not begin on 16 bytes are taken element by element, to the same bits."""
    say("[rotary] unaligned")
    raw = rnd(1 * 9 * 2 * 64 + 1, dtype=BF, seed=7)
    freq, _ = ssd.rotary_frequencies(64, device="cuda")
    x = raw[1:].view(1, 9, 2, 64)
    assert torch.equal(ssd.rotary(x, None, freq)[0], ssd.rotary(x.clone(), None, freq)[0])


def test_single_tokens_and_gradient():
    """A token an entry is the prompt's token at its place; a gradient is the transpose of the map."""
    say("[rotary] tokens, gradient")
    q, k = rnd(2, 40, 4, 64, dtype=F32, seed=8), rnd(2, 40, 2, 64, dtype=F32, seed=9)
    freq, scale = ssd.rotary_frequencies(32, scaling="by_parts", factor=8.0, original_length=64, device="cuda")
    yq, yk = ssd.rotary(q, k, freq, scale=scale)
    at = torch.tensor([17, 3], dtype=torch.int32, device="cuda")
    rows = torch.arange(2, device="cuda")
    one = ssd.rotary(q[rows, at.long()].contiguous(), k[rows, at.long()].contiguous(), freq, positions=at, scale=scale)
    assert torch.equal(one[0], yq[rows, at.long()]) and torch.equal(one[1], yk[rows, at.long()])
    dy = rnd(2, 40, 4, 64, dtype=F32, seed=10)
    dx, _ = ssd.rotary_bwd(dy, None, freq, scale=scale)
    lhs, rhs = (n64(yq) * n64(dy)).sum(), (n64(q) * n64(dx)).sum()
    assert abs(lhs - rhs) <= 20 * ref.U32 * scale * (np.abs(n64(q)).sum(-1) * np.abs(n64(dy)).sum(-1)).sum()


def test_empty_stream_and_graph():
    say("[rotary] empty, stream, graph")
    freq, _ = ssd.rotary_frequencies(64, device="cuda")
    e, _ = ssd.rotary(torch.empty(2, 0, 4, 64, dtype=BF, device="cuda"), None, freq)
    assert e.shape == (2, 0, 4, 64)
    q, k = rnd(1, 50, 4, 64, dtype=BF, seed=11), rnd(1, 50, 4, 64, dtype=BF, seed=12)
    pos = torch.arange(50, dtype=torch.int32, device="cuda").view(1, 50)
    want = ssd.rotary(q, k, freq, positions=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ssd.rotary(q, k, freq, positions=pos)
    s.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ssd.rotary(q, k, freq, positions=pos)
    for r in range(3):
        pos += 1000
        q.copy_(rnd(1, 50, 4, 64, dtype=BF, seed=20 + r))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[0], ssd.rotary(q, k, freq, positions=pos)[0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_layer(dtype):
    """Queries and keys of one projection turned in place, the delta rule and linear attention on them, the norm behind:
    a prompt in one call, and in two with a step behind them, from the same pool of states."""
    say(f"[layer] {dtype}")
    b, T, H, d = 2, 97, 4, 64
    wide = rnd(b, T, 3 * H * d, dtype=dtype, seed=13)
    q, k, v = (wide[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    k.copy_(torch.nn.functional.normalize(k.float(), dim=-1))
    gen = torch.Generator().manual_seed(14)
    g, beta = (-torch.rand(b, T, H, generator=gen) * 0.2).cuda(), torch.rand(b, T, H, generator=gen).cuda()
    freq, _ = ssd.rotary_frequencies(d, device="cuda")
    raw = wide.clone()
    ssd.rotary(q, k, freq, q_out=q, k_out=k)
    o, fin = ssd.gated_delta_fwd(q, k, v, g, beta, scale=d ** -0.5)
    y, _ = ssd.group_norm(o.view(b * T, H * d), H)
    n = T - 1
    parts = raw[:, :n].contiguous()
    q1, k1, v1 = (parts[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    ssd.rotary(q1, k1, freq, q_out=q1, k_out=k1)
    o1, pool = ssd.gated_delta_fwd(q1, k1, v1, g[:, :n].contiguous(), beta[:, :n].contiguous(), scale=d ** -0.5)
    last = raw[:, n].contiguous()
    q2, k2, v2 = (last[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)) for i in range(3))
    pos = torch.full((b,), n, dtype=torch.int32, device="cuda")
    q2, k2 = ssd.rotary(q2, k2, freq, positions=pos)
    o2 = ssd.gated_delta_step(pool, q2, k2, v2.contiguous(), g[:, n].contiguous(), beta[:, n].contiguous(), scale=d ** -0.5)
    rel = 2 * ref.rel_forward(T, d)
    half = ref.UBF if dtype == BF else 0.0
    ref.check(n64(pool), n64(fin), rel, False, "state")
    ref.check(n64(o2), n64(o[:, n]), rel + half, dtype == BF, "last token")
    y2, _ = ssd.group_norm(torch.cat([o1, o2[:, None]], 1).view(b * T, H * d), H)
    # the norm divides by a group's deviation, which is that of its values: the same relative error, and its own rounding
    ref.check(n64(y2), n64(y), 4 * (rel + half), dtype == BF, "norm")
    w, _ = ssd.lin_attn_fwd(q, k, v, torch.full((H,), -0.1, device="cuda"), scale=d ** -0.5)
    assert w.shape == o.shape and torch.isfinite(w.float()).all()

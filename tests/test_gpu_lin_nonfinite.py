"""GPU: linear attention of bf16 operands with values that are not finite. A
result that such a value enters by the recurrence is not finite; every other one
is as without it: the places are compared with the recurrence in 64 bits, the
finite values held to the bounds of layer_ref.py, and infinite states are those
of the recurrence. fp32 operands are held to the same.
"""
import pytest
import torch

import layer_ref as ref
import ssd_chunked_scan_fwd_amd as ssd
from test_gpu_lin_infinite import _need_gpu, decays, hold, make, n64  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]
BF, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")

# T, H, Hk, dk, dv, packed sequences
SHAPES = [(200, 2, 1, 64, 64, None), (300, 2, 2, 128, 128, None), (130, 2, 1, 40, 96, None), (130, 2, 2, 96, 40, None),
          (130, 3, 3, 8, 8, None), (130, 2, 1, 8, 136, None), (150, 1, 1, 256, 200, None), (200, 2, 2, 16, 24, [0, 100, 100, 170, 200])]
# Tensors, and tokens with such a value in one channel: in a sequence's first (and, backwards, last) 32 tokens, in
# the middle of a chunk, on its last and first place.
PLACES = [("v", (20, 100)), ("v", (63,)), ("k", (20, 100)), ("k", (129,)), ("q", (64,)), ("q", (37, 100)), ("do", (20, 100))]


def inputs(shape, value, dtype, name, tokens):
    T, H, Hk, dk, dv, cu = shape
    print(f"[lin non-finite] {shape} {value} {dtype} {name} {tokens}", flush=True)
    d = make(T, H, Hk, dk, dv, dtype, T + dk, nseq=1 if cu is None else len(cu) - 1)
    for i, t in enumerate(tokens):
        d[name][0, t, 0, 5 + 2 * i] = value
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    return d, {n: n64(t) for n, t in d.items()}, decays(H), cut


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("shape", SHAPES)
def test_forwards(shape, value, dtype):
    """o, the final state, and dq, which is carried forwards too."""
    T, H, Hk, dk, dv, cu = shape
    kind, state = ("bf16", "state") if dtype == BF else ("fp32", "fp32")
    for name, tokens in PLACES:
        d, x, ld, cut = inputs(shape, value, dtype, name, tokens)
        o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], ld.cuda(), cu_seqlens=cut, scale=0.25, initial_state=d["init"])
        g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld.cuda(), d["do"], cu_seqlens=cut, scale=0.25, initial_state=d["init"])
        want, E = ref.attention(x["q"], x["k"], x["v"], n64(ld), 0.25, x["init"], cu)
        gw, gE = ref.attention_bwd(x["q"], x["k"], x["v"], n64(ld), 0.25, x["do"], x["init"], None, cu)
        hold(o, want["o"], E["o"], kind, T, dk, f"{name} o")
        hold(fin, want["final"], E["final"], state, T, dk, f"{name} final", infinite=True)
        hold(g["dq"], gw["dq"], gE["dq"], kind, T, max(dk, dv), f"{name} dq")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
@pytest.mark.parametrize("shape", SHAPES)
def test_backwards(shape, value, dtype):
    """dk, dv and the initial state's gradient, carried from the last token to the first."""
    T, H, Hk, dk, dv, cu = shape
    kind, state = ("bf16", "state") if dtype == BF else ("fp32", "fp32")
    n = max(dk, dv) * (H // Hk)
    for name, tokens in PLACES:
        d, x, ld, cut = inputs(shape, value, dtype, name, tokens)
        g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld.cuda(), d["do"], cu_seqlens=cut, scale=0.25, initial_state=d["init"],
                             dfinal_state=d["dfinal"], want_dinit=True)
        want, E = ref.attention_bwd(x["q"], x["k"], x["v"], n64(ld), 0.25, x["do"], x["init"], x["dfinal"], cu)
        for out in ("dk", "dv"):
            hold(g[out], want[out], E[out], kind, T, n, f"{name} {out}")
        hold(g["dinit"], want["dinit"], E["dinit"], state, T, n, f"{name} dinit", infinite=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_without_tokens(dtype):
    """What is not finite in their states stays, and reaches no neighbour."""
    cu = [0, 0, 70, 70, 130, 130]
    d = make(130, 2, 2, 64, 64, dtype, 21, nseq=5)
    d["init"][0, :, 3, 5], d["init"][2, :, 6, 1], d["init"][4, :, 2, 2] = INF, NAN, -INF
    cut = torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], decays(2).cuda(), cu_seqlens=cut, initial_state=d["init"])
    for s in (0, 2, 4):
        assert torch.equal(fin[s].view(torch.int32), d["init"][s].view(torch.int32))
    assert torch.all(torch.isfinite(o)) and torch.all(torch.isfinite(fin[[1, 3]]))
    g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], decays(2).cuda(), d["do"], cu_seqlens=cut, initial_state=d["init"],
                         dfinal_state=d["init"], want_dinit=True)
    for s in (0, 2, 4):
        assert torch.equal(g["dinit"][s].isfinite(), d["init"][s].isfinite())
    assert all(torch.all(torch.isfinite(g[n])) for n in ("dq", "dk", "dv")) and torch.all(torch.isfinite(g["dinit"][[1, 3]]))


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (136, 40)])
def test_captured_and_in_wider_rows(dims):
    """Rows of one projection with such values, forwards and backwards in a graph: every replay gives what the eager
    call on contiguous rows gave, with eager work between the replays."""
    dk, dv = dims
    T, H, Hk = 700, 4, 2
    g = torch.Generator().manual_seed(17)
    w = torch.randn(1, T, H * dk + Hk * (dk + dv), generator=g).to(BF).cuda()
    w[0, 300, 3], w[0, 500, H * dk + 9], w[0, 40, (H + Hk) * dk + 2] = NAN, INF, -INF
    q, k, v = (t.unflatten(-1, (-1, d)) for t, d in zip(w.split([H * dk, Hk * dk, Hk * dv], -1), (dk, dk, dv)))
    do = torch.randn(1, T, H, dv, generator=g).to(BF).cuda()
    ld = decays(H).cuda()

    def run(q, k, v):
        o, fin = ssd.lin_attn_fwd(q, k, v, ld, scale=0.2)
        return [o, fin] + [ssd.lin_attn_bwd(q, k, v, ld, do, scale=0.2)[n] for n in ("dq", "dk", "dv")]

    want = run(q.contiguous(), k.contiguous(), v.contiguous())
    assert not all(torch.all(torch.isfinite(t)) for t in want) and all(torch.any(torch.isfinite(t)) for t in want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(q, k, v)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        out = run(q, k, v)
    for i in range(3):
        for t in out:
            t.zero_()
        run(q.contiguous(), k.contiguous(), v.contiguous())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) and torch.equal(a.isnan(), b.isnan()), i

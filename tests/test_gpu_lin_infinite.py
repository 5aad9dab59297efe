"""GPU: infinities in the states of linear attention stay what they are: a decay
of an infinity is that infinity, as in the recurrence in 64 bits. Finite values
are held to the bounds of layer_ref.py.
"""
import numpy as np
import pytest
import torch

import layer_ref as ref
import ssd_chunked_scan_fwd_amd as ssd

pytestmark = [pytest.mark.gpu, pytest.mark.filterwarnings("ignore::RuntimeWarning")]
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ssd.lib()


def n64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def decays(H):
    """From half to one in a thousand forgotten with a token; the second head forgets nothing."""
    ld = np.log1p(-(2.0 ** -np.linspace(1.0, 10.0, H)))
    if H > 1:
        ld[1] = 0.0
    return torch.tensor(ld, dtype=F32)


def make(T, H, Hk, dk, dv, dtype, seed, nseq=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, d: torch.randn(1, T, h, d, generator=g).to(dtype).cuda()
    f = lambda: (4 * torch.randn(nseq, H, dv, dk, generator=g)).cuda()
    return dict(q=r(H, dk), k=r(Hk, dk), v=r(Hk, dv), do=r(H, dv), init=f(), dfinal=f())


def hold(got, want, E, kind, n, d, what, infinite=False):
    """Not finite exactly where the recurrence is not; finite values within their bound; where asked,
    infinite, of the recurrence's sign, where that is."""
    got = n64(got)
    fin = np.isfinite(want)
    wrong = np.argwhere(np.isfinite(got) != fin)
    assert len(wrong) == 0, f"{what}: {len(wrong)} places, first {wrong[0]}: {got[tuple(wrong[0])]}, {want[tuple(wrong[0])]}"
    worst = float(np.max(np.abs(got - want)[fin] / ref.bound(kind, want, E, n, d)[fin])) if fin.any() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"
    if infinite:
        lost = int((np.isinf(want) & (got != want)).sum())
        assert lost == 0, f"{what}: {lost} of {int(np.isinf(want).sum())} infinities lost"


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dims", [(64, 64), (32, 200)])
def test_in_states_handed_in(dims, dtype):
    """Forwards from an initial state, backwards from a final one."""
    dk, dv = dims
    T, H = 60, 16
    ld = decays(H)
    d = make(T, H, H, dk, dv, dtype, 3)
    d["init"][:, :, 3, 7] = INF
    d["dfinal"][:, :, 4, 6] = -INF
    o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], ld.cuda(), scale=0.25, initial_state=d["init"])
    g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld.cuda(), d["do"], scale=0.25, initial_state=d["init"],
                         dfinal_state=d["dfinal"], want_dinit=True)
    x = {n: n64(t) for n, t in d.items()}
    want, E = ref.attention(x["q"], x["k"], x["v"], n64(ld), 0.25, x["init"])
    gw, gE = ref.attention_bwd(x["q"], x["k"], x["v"], n64(ld), 0.25, x["do"], x["init"], x["dfinal"])
    kind, state = ("bf16", "state") if dtype == BF else ("fp32", "fp32")
    hold(o, want["o"], E["o"], kind, T, dk, "o")
    hold(fin, want["final"], E["final"], state, T, dk, "final", infinite=True)
    for n in ("dq", "dk", "dv"):
        hold(g[n], gw[n], gE[n], kind, T, max(dims), n)
    hold(g["dinit"], gw["dinit"], gE["dinit"], state, T, max(dims), "dinit", infinite=True)


@pytest.mark.parametrize("name", ["v", "k"])
def test_from_a_value(name):
    """One infinite channel of one token of an fp32 prompt: what it leaves in the state is kept."""
    T, H, dk, dv = 200, 8, 64, 48
    ld = decays(H)
    d = make(T, H, H, dk, dv, F32, 5)
    d[name][0, 90, :, 5] = INF
    o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], ld.cuda(), scale=0.25, initial_state=d["init"])
    want, E = ref.attention(*[n64(d[n]) for n in "qkv"], n64(ld), 0.25, n64(d["init"]))
    hold(o, want["o"], E["o"], "fp32", T, dk, "o")
    hold(fin, want["final"], E["final"], "fp32", T, dk, "final", infinite=True)


def test_in_a_step():
    H, dk, dv = 32, 64, 48
    ld = decays(H)
    d = make(5, H, H, dk, dv, F32, 9)
    d["init"][:, :, 3, 7] = INF
    d["init"][:, :, 4, 6] = -INF
    want, E = ref.attention(*[n64(d[n]) for n in "qkv"], n64(ld), 1.0, n64(d["init"]))
    state = d["init"].clone()
    for t in range(5):
        o = ssd.lin_attn_step(state, d["q"][:, t], d["k"][:, t], d["v"][:, t], ld.cuda())
        hold(o, want["o"][:, t], E["o"][:, t], "fp32", 5, dk, f"o {t}")
    hold(state, want["final"], E["final"], "fp32", 5, dk, "state", infinite=True)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_over_blocks(dtype):
    """A prompt cut into blocks, whose whole decay is below what fp32 holds: what is infinite at its start, or its end,
    is so at the other. The last head remembers nothing: its infinity times 0 is no number."""
    T, H, dk, dv = 900, 4, 32, 48
    ld = torch.tensor([-0.5, -2.0, -30.0, -INF], dtype=F32)
    d = make(T, H, H, dk, dv, dtype, 11)
    sh = ssd.lin_attn_shape(d["q"], d["k"], d["v"])
    assert ssd.lin_attn_workspace_bytes(sh) >= 4 * H * dk * dv * 4
    d["init"][:, :, 3, 7] = INF
    d["dfinal"][:, :, 4, 6] = -INF
    o, fin = ssd.lin_attn_fwd(d["q"], d["k"], d["v"], ld.cuda(), scale=0.25, initial_state=d["init"])
    g = ssd.lin_attn_bwd(d["q"], d["k"], d["v"], ld.cuda(), d["do"], scale=0.25, initial_state=d["init"],
                         dfinal_state=d["dfinal"], want_dinit=True)
    x = {n: n64(t) for n, t in d.items()}
    want, E = ref.attention(x["q"], x["k"], x["v"], n64(ld), 0.25, x["init"])
    gw, gE = ref.attention_bwd(x["q"], x["k"], x["v"], n64(ld), 0.25, x["do"], x["init"], x["dfinal"])
    state = "state" if dtype == BF else "fp32"
    hold(fin, want["final"], E["final"], state, T, dk, "final", infinite=True)
    hold(g["dinit"], gw["dinit"], gE["dinit"], state, T, dv, "dinit", infinite=True)

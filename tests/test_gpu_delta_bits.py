"""GPU: the bits that the gated delta rule keeps of what it computes, on inputs whose results are what is left when
large terms cancel. There a result rounds to its type far below the terms' own 16th bit, and shows every bit that an
operand lost on the way. Each bound is derived where it is used and none is of the terms' size times 2^-17 or more, which
operands of 16 bits would leave."""
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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,dk,dv", [(1, 8, 16), (1, 64, 40), (1, 128, 16), (70, 64, 128), (3, 256, 24)])
def test_state_under_a_query(T, dk, dv, dtype):
    """o = S q where S q is 2^-20 of S: rows of S in [1, 2), their odd columns the even ones and up to 15 steps of 2^-23,
    queries of 1 and -1 in turn. beta is 0 and nothing decays, so S stays.
    Split into terms of 8 bits, the first sum exactly (multiples of 2^-7, sums below 2^9), and so do the others, in any
    order. Joined, three sums are rounded twice, by at most 2^-24 of what is joined, which is below dk 2^-7 once the first
    have cancelled: first terms of a pair differ by one step of 2^-7 at most. o is rounded once to its type. With two
    terms, up to 2^-17 is left of each entry, some 2^-18 sqrt(dk) of a sum and all of o."""
    say(f"[delta bits] state under a query {T} {dk} {dv} {dtype}")
    r = np.random.default_rng(T + dk)
    n = 2 if T == 70 else 1
    S = np.empty((1, n, dv, dk))
    S[..., 0::2] = 1 + r.integers(0, (1 << 23) - 16, S[..., 0::2].shape) / 2 ** 23
    S[..., 1::2] = S[..., 0::2] + r.integers(1, 16, S[..., 0::2].shape) / 2 ** 23
    assert np.array_equal(S.astype(np.float32), S)
    sign = np.where(np.arange(dk) % 2, 1.0, -1.0) * np.where(r.random((T, n, dk // 2)) < 0.5, 1.0, -1.0).repeat(2, -1)
    q = torch.tensor(sign, dtype=dtype).cuda()[None]
    k = torch.nn.functional.normalize(torch.tensor(r.standard_normal((1, T, n, dk))), dim=-1).to(dtype).cuda()
    v = torch.tensor(r.standard_normal((1, T, n, dv))).to(dtype).cuda()
    zero = torch.zeros(1, T, n, device="cuda")
    init = torch.tensor(S, dtype=F32).cuda()
    want = np.einsum("hvk,thk->thv", S[0], sign)
    o, fin = ssd.gated_delta_fwd(q, k, v, zero, zero, initial_state=init)
    assert torch.equal(fin, init)
    room = (ref.UBF if dtype == BF else ref.U32) * np.abs(want) + 2 * ref.U32 * dk * 2.0 ** -7
    bad = np.abs(o[0].cpu().double().numpy() - want) / room
    assert bad.max() <= 1, bad.max()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_and_updates(dtype):
    """o = e^(g2) beta1 - beta2 with beta2 = e^(g2) beta1 rounded to 32 bits: two tokens of keys e1 and e2, values 1 and
    -1, a query of both. What is left of terms below 1 is below 2^-24, so o is what the terms lose on the way.
    In units of 2^-24: e^(g2) is off by 2 (1 of the hardware's 2^y, half a rounding, 0.2 of log2(e) itself); beta1 and its
    product with the inverse, a unit matrix, are exact; products of terms left out are 0.5; the sums of three groups of
    products are rounded by at most 1 each: 12 is more than twice all of it. Terms of 16 bits leave up to 2^-18 (64
    units) of a score, of each update and of their product, spread evenly: hardly one of 512 heads would keep to 12."""
    say(f"[delta bits] scores and updates {dtype}")
    H, r = 512, np.random.default_rng(5)
    g = np.zeros((2, H), np.float32)
    g[1] = -r.uniform(0.01, 0.7, H)
    beta = np.ones((2, H), np.float32)
    beta[0] = r.uniform(0.5, 1.0, H)
    beta[1] = (np.exp(g[1].astype(np.float64)) * beta[0]).astype(np.float32)
    k = torch.zeros(1, 2, 1, 8, dtype=dtype, device="cuda")
    k[0, 0, 0, 0] = k[0, 1, 0, 1] = 1
    q = torch.zeros_like(k)
    q[0, :, 0, :2] = 1
    v = torch.ones(1, 2, H, 8, dtype=dtype, device="cuda")
    v[0, 1] = -1
    o, _ = ssd.gated_delta_fwd(q, k, v, torch.tensor(g)[None].cuda(), torch.tensor(beta)[None].cuda())
    o = o[0].cpu().double().numpy()
    want = np.exp(g[1].astype(np.float64)) * beta[0] - beta[1]
    assert np.all(np.abs(o[0] - beta[0][:, None]) <= (ref.UBF if dtype == BF else ref.U32) * beta[0][:, None])
    worst = np.abs(o[1] - want[:, None]).max() / ref.U32
    assert worst <= 12, worst


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 3])
def test_decay_of_a_state(T, dtype):
    """A state of ones that only decays, down to e^-86: e^G in fp32. One token, in units of 2^-24 of the result: 2 of the
    hardware's 2^y (its last place), 1 of what puts y's rounding back; 4 are allowed. The log decays of more tokens add
    up in 64 bits, and what their sum has below 32 bits is a factor: 1 for it, 1 for the product, 6 allowed."""
    say(f"[delta bits] decay of a state {T} {dtype}")
    H, r = 4096, np.random.default_rng(T)
    total = -np.exp(np.linspace(np.log(1e-3), np.log(86.0), H))
    g = np.ascontiguousarray(total * r.dirichlet(np.ones(T), H).T, np.float32)
    q, k, v = (torch.randn(1, T, n, 8, generator=torch.Generator().manual_seed(n)).to(dtype).cuda() for n in (1, 1, H))
    init = torch.ones(1, H, 8, 8, device="cuda")
    _, fin = ssd.gated_delta_fwd(q, k, v, torch.tensor(g)[None].cuda(), torch.zeros(1, T, H, device="cuda"), initial_state=init)
    want = np.exp(g.astype(np.float64).sum(0))[:, None, None]
    worst = (np.abs(fin[0].cpu().double().numpy() - want) / want).max() / ref.U32
    assert worst <= (4 if T == 1 else 6), worst

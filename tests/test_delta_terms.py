"""CPU: what the bounds on the bits of the gated delta rule's results tell apart: the rule with every computed operand of a
product held in three terms of 8 bits keeps to them, with two it does not."""
import numpy as np
import pytest
import torch

import delta_ref as ref

# The products of a result, one after the other: keys and state, inverse, updates and keys, queries and state with
# scores and updates. Each sums in some 12 steps (pieces of 32 times pairs of terms), the inverse in twice as many, each
# rounded by at most 2^-24 of sums that the result's own size bounds: 60 in all, which add up as their roots do, to 8
# 2^-24; over the two or three chunks that these decays let a state remember, 13. Twice that is allowed, and a little less.
REL24 = 25 * ref.U32
# A result in bf16 differs from the 64-bit one rounded likewise where the two lie on different sides of a border: of
# values whose borders are 2^-7 of a power of two apart, a part 2 e / 2^-7 for an error e, each by 2^-7 of it. In the norm
# that is sqrt(2 e 2^-8), as the values of a normal distribution are twice their power of two in the mean.
RELBF = np.sqrt(2 * 13 * ref.U32 * 2.0 ** -8)


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def bf16(x):
    return torch.tensor(x).bfloat16().double().numpy()


def held(x, terms):
    """x as the sum of so many values of bf16."""
    rest, out = torch.tensor(x).float(), np.zeros(x.shape)
    for _ in range(terms):
        t = rest.bfloat16().float()
        out, rest = out + t.double().numpy(), rest - t
    return out


@pytest.mark.parametrize("terms,keeps", [(3, True), (2, False)])
def test_terms(terms, keeps):
    T, H, d, r = 300, 8, 64, np.random.default_rng(1)
    q, k = r.standard_normal((2, T, H, d))
    q, k = (bf16(x / np.linalg.norm(x, axis=-1, keepdims=True)) for x in (q, k))
    v, g, beta, S = bf16(r.standard_normal((T, H, d))), -0.3 * r.random((T, H)), r.random((T, H)), r.standard_normal((H, d, d))
    want, last = ref.forward(q, k, v, g, beta, 0.5, S)
    o = np.zeros_like(v)
    for t in range(T):
        D = np.exp(g[t])[:, None, None] * held(S, terms)
        u = held(beta[t][:, None] * (v[t] - np.matmul(D, k[t][:, :, None])[:, :, 0]), terms)
        S = D + u[:, :, None] * k[t][:, None, :]
        o[t] = 0.5 * np.matmul(held(S, terms), q[t][:, :, None])[:, :, 0]
    assert (off(S, last) <= REL24) == keeps and (off(o, want) <= REL24) == keeps
    assert (off(bf16(o), bf16(want)) <= RELBF) == keeps

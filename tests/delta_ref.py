"""Plain 64-bit forms of the gated delta rule and of rotary positions, and the
bounds that the GPU tests hold them to.

The rule, one sequence, [T, H, *]: u = beta (v - a S k), S' = a S + u k^T, o = scale
S' q. With |k| = 1, 0 <= beta <= 1 and a <= 1 the map of S is a contraction
(I - beta k k^T has norm at most 1), so an error made at one token is not enlarged
by the later ones: errors of different tokens only add up, and as their roundings
are independent, the norm of the sum grows with the square root of their number.
At a token an fp32 sum of n terms has n roundings of at most 2^-24 of the partial
sums, which the norms of the factors bound; independent ones add up to sqrt(n) 2^-24
of it. The sums of a token run over dk (state times key and query), over the chunk
of C <= 64 tokens (inverse, its product, scores, state update) and, backwards,
over dv. So, forwards,
    rel = sqrt(T) (sqrt(dk) + 4 sqrt(C)) 2^-24,
and backwards, whose walk begins with the states of the forward one,
    rel = sqrt(T) (2 sqrt(dk) + 2 sqrt(dv) + 8 sqrt(C)) 2^-24,
of the norm of what is summed. Single values are held to 8 such deviations (of
10^6 normal ones the largest is 5). A result in bf16 is rounded once more: 2^-8 of
the value.
What is summed: for o, each row of S times q, at most |S_r| |q|; as q has no
direction in particular, o's own norm stands for it unless S or q is 0, so the norm
over a whole tensor is that of the 64-bit result. The gradient of the log decays is
a sum over a chunk of q.dq + k.(read part of dk) - k.(write part): the norm of these,
times sqrt(C), is added to its own (`parts`).
"""
from __future__ import annotations

import numpy as np

U32, UBF, C = 2.0 ** -24, 2.0 ** -8, 64


def expand(x, H):
    return np.repeat(x, H // x.shape[-2], axis=-2)


def forward(q, k, v, g, beta, scale, init=None, keep=False):
    """One sequence, [T, H, *] in 64 bits: (o, last state[, states before each token, u])."""
    T, H, dk = k.shape
    S = np.zeros((H, v.shape[2], dk)) if init is None else init.copy()
    o, before, us = np.zeros((T, H, v.shape[2])), [], []
    for t in range(T):
        D = np.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - np.matmul(D, k[t][:, :, None])[:, :, 0])
        if keep:
            before.append(S)
            us.append(u)
        S = D + u[:, :, None] * k[t][:, None, :]
        o[t] = scale * np.matmul(S, q[t][:, :, None])[:, :, 0]
    return (o, S, before, us) if keep else (o, S)


def backward(q, k, v, g, beta, scale, do, init=None, dfinal=None):
    """dict(dq, dk, dv, dlog_decay, dbeta, dinit, parts) of one sequence, dq and dk per value head."""
    T, H, dk = k.shape
    _, S, before, us = forward(q, k, v, g, beta, scale, init, keep=True)
    L = np.zeros_like(S) if dfinal is None else dfinal.copy()
    out = dict(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v), dlog_decay=np.zeros((T, H)),
               dbeta=np.zeros((T, H)), parts=np.zeros((T, H)))
    mv = lambda M, x: np.matmul(M, x[:, :, None])[:, :, 0]
    vm = lambda x, M: np.matmul(x[:, None, :], M)[:, 0]
    after = S
    for t in range(T - 1, -1, -1):
        D, u = np.exp(g[t])[:, None, None] * before[t], us[t]
        out["dq"][t] = scale * vm(do[t], after)
        L = L + scale * do[t][:, :, None] * q[t][:, None, :]
        gu = mv(L, k[t])
        ge = beta[t][:, None] * gu
        out["dbeta"][t] = (gu * (v[t] - mv(D, k[t]))).sum(-1)
        out["dv"][t] = ge
        write, read = vm(u, L), -vm(ge, D)
        out["dk"][t] = write + read
        L = L - ge[:, :, None] * k[t][:, None, :]
        out["dlog_decay"][t] = (L * D).sum((1, 2))
        out["parts"][t] = (np.abs((q[t] * out["dq"][t]).sum(-1)) + np.abs((k[t] * read).sum(-1)) +
                           np.abs((k[t] * write).sum(-1)) + np.abs(out["dlog_decay"][t]))
        L = np.exp(g[t])[:, None, None] * L
        after = before[t]
    out["dinit"] = L
    return out


def sequences(b, T, cu):
    """(row, first token, end, index) of every sequence."""
    if cu is None:
        return [(r, 0, T, r) for r in range(b)]
    return [(0, int(cu[s]), int(cu[s + 1]), s) for s in range(len(cu) - 1)]


def batch_forward(q, k, v, g, beta, scale, init=None, cu=None):
    b, T, H, dv = v.shape
    q, k = expand(q, H), expand(k, H)
    o, fin = np.zeros((b, T, H, dv)), []
    for r, a, e, s in sequences(b, T, cu):
        o[r, a:e], f = forward(q[r, a:e], k[r, a:e], v[r, a:e], g[r, a:e], beta[r, a:e], scale, None if init is None else init[s])
        fin.append(f)
    return dict(o=o, final=np.stack(fin))


def batch_backward(q, k, v, g, beta, scale, do, init=None, dfinal=None, cu=None):
    b, T, H, dv = v.shape
    Hk = k.shape[2]
    q, k = expand(q, H), expand(k, H)
    shapes = dict(dq=q.shape, dk=k.shape, dv=v.shape, dlog_decay=g.shape, dbeta=g.shape, parts=g.shape)
    out = {n: np.zeros(s) for n, s in shapes.items()}
    out["dinit"] = []
    for r, a, e, s in sequences(b, T, cu):
        w = backward(q[r, a:e], k[r, a:e], v[r, a:e], g[r, a:e], beta[r, a:e], scale, do[r, a:e],
                     None if init is None else init[s], None if dfinal is None else dfinal[s])
        for n in shapes:
            out[n][r, a:e] = w[n]
        out["dinit"].append(w["dinit"])
    out["dinit"] = np.stack(out["dinit"])
    for n in ("dq", "dk"):
        out[n] = out[n].reshape(b, T, Hk, H // Hk, -1).sum(3)
    return out


def rel_forward(T, dk):
    return np.sqrt(max(T, 1)) * (np.sqrt(dk) + 4 * np.sqrt(C)) * U32


def rel_backward(T, dk, dv):
    return np.sqrt(max(T, 1)) * (2 * np.sqrt(dk) + 2 * np.sqrt(dv) + 8 * np.sqrt(C)) * U32


def check(got, ref, rel, bf16, what, more=0.0):
    """Norm and single values of `got` against the 64-bit `ref`; `more`: norm of what is summed besides."""
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, f"{what}: {got.shape} {ref.shape}"
    assert np.all(np.isfinite(got)), f"{what}: values that are not finite"
    if not got.size:
        return
    err, norm = got - ref, np.linalg.norm(ref) + more
    half = UBF if bf16 else 0.0
    assert np.linalg.norm(err) <= (half + rel) * norm + 1e-300, f"{what}: norm {np.linalg.norm(err) / max(norm, 1e-300):.3g}, allowed {half + rel:.3g}"
    single = half * np.abs(ref) + 8 * rel * np.maximum(norm / np.sqrt(got.size), np.abs(ref)) + 1e-300
    worst = float(np.max(np.abs(err) / single))
    assert worst <= 1.0, f"{what}: a value has {worst:.3g} of its allowance"


# ---------------------------------------------------------------- rotary positions

def rotate(x, pos, freq, layout, scale, inverse=False):
    """x [..., heads, d], pos [...] in 64 bits."""
    rot = 2 * len(freq)
    t = np.asarray(pos, np.float64)[..., None, None] * freq
    c, s = scale * np.cos(t), scale * (-np.sin(t) if inverse else np.sin(t))
    y = x.copy()
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    u, w = a * c - b * s, b * c + a * s
    if layout == "half":
        y[..., :rot // 2], y[..., rot // 2:rot] = u, w
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, w
    return y


def check_rotary(got, x, pos, freq, layout, scale, bf16, what, inverse=False):
    """A turned value is x c - y s, with c and s in fp32: the angle, in turns, is rounded once from at most half a
    turn (2^-25 of a turn, 2 pi 2^-25 < 2^-22 of a radian), sine and cosine by 2 units of 2^-24 and their product with
    scale by one, the two products and the sum by one each: 10 2^-24 (|x| + |y|) scale; turns are a product of 64 bits with
    1 / (2 pi) in 64 bits: 2^-52 of the angle. Copied values are as they were."""
    want = rotate(x, pos, freq, layout, scale, inverse)
    rot = 2 * len(freq)
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    angle = np.abs(np.asarray(pos, np.float64))[..., None, None] * freq
    size = (np.abs(a) + np.abs(b)) * abs(scale) * (10 * U32 + 2.0 ** -52 * angle)
    room = np.zeros_like(x)
    if layout == "half":
        room[..., :rot // 2] = room[..., rot // 2:rot] = size
    else:
        room[..., 0:rot:2] = room[..., 1:rot:2] = size
    if bf16:
        room[..., :rot] += UBF * np.abs(want[..., :rot])
    assert got.shape == want.shape
    bad = np.abs(got - want) > room
    assert not bad.any(), f"{what}: {int(bad.sum())} values, worst {np.max(np.abs(got - want) - room):.3g}"

"""Plain 64-bit forms of the layer operators (linear attention with one decay a
head, group norm, pages), and the bounds that the GPU tests hold them to.

Bounds of linear attention. Every output is a sum of products a b c (for o:
lam^(i-j) (q.k) v). With E the same sum over absolute values:
  fp32  each product passes through at most n steps of the recurrence (one
        rounding of the product, one of the sum, a step) and a sum of d terms:
        |err| <= (2 n + d + 16) 2^-24 E.
  bf16  two operands of the matrix products are rounded once (the masked
        scores, or the state, by 2^-8 relative each way of a term) and the output
        once: |err| <= 2^-8 (1 + 2^-6) E + 2^-8 |ref| + the fp32 bound, elementwise;
        as the roundings of different terms are independent, the error's norm is
        at most that of three roundings: rel-L2 <= sqrt(3) 2^-8 < 7e-3.
  states of bf16 inputs: the weighted operand is carried as two bf16 values,
        which leaves 2^-16 of it: |err| <= 2^-16 E + the fp32 bound.
The accumulated E of shared heads is the sum of theirs.
"""
from __future__ import annotations

import numpy as np

U32, UBF = 2.0 ** -24, 2.0 ** -8


def expand(x, H):
    """[.., Hk, d] -> [.., H, d]."""
    return np.repeat(x, H // x.shape[-2], axis=-2)


def scan(q, k, v, ld, scale, init=None):
    """One sequence, [T, H, *] in 64 bits: (o, last state [H, dv, dk])."""
    T, H, dk = q.shape
    lam = np.exp(ld)[:, None, None]
    D = np.zeros((H, v.shape[2], dk)) if init is None else init.copy()
    o = np.zeros((T, H, v.shape[2]))
    for t in range(T):
        D = lam * D + v[t][:, :, None] * k[t][:, None, :]
        o[t] = scale * (D @ q[t][:, :, None])[:, :, 0]
    return o, D


def scan_bwd(q, k, v, ld, scale, do, init=None, dfinal=None):
    """(dq, dk, dv, dinit) of one sequence, dk and dv per query head."""
    T, H, dk = q.shape
    lam = np.exp(ld)[:, None, None]
    D = np.zeros((H, v.shape[2], dk)) if init is None else init.copy()
    gq, gk, gv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for t in range(T):
        D = lam * D + v[t][:, :, None] * k[t][:, None, :]
        gq[t] = scale * (do[t][:, None, :] @ D)[:, 0]
    L = np.zeros((H, v.shape[2], dk)) if dfinal is None else dfinal.copy()
    for t in range(T - 1, -1, -1):
        L = L + scale * do[t][:, :, None] * q[t][:, None, :]
        gk[t] = (v[t][:, None, :] @ L)[:, 0]
        gv[t] = (L @ k[t][:, :, None])[:, :, 0]
        L = lam * L
    return gq, gk, gv, L


def sequences(b, T, cu):
    """(row, first token, end, index) of every sequence."""
    if cu is None:
        return [(r, 0, T, r) for r in range(b)]
    return [(0, int(cu[s]), int(cu[s + 1]), s) for s in range(len(cu) - 1)]


def attention(q, k, v, ld, scale, init=None, cu=None):
    """The whole batch; returns o, final, and both sums over absolute values."""
    b, T, H, dk = q.shape
    k, v = expand(k, H), expand(v, H)
    seqs = sequences(b, T, cu)
    o, E = np.zeros((b, T, H, v.shape[3])), np.zeros((b, T, H, v.shape[3]))
    fin, Ef = [], []
    for r, a, e, s in seqs:
        i = None if init is None else init[s]
        o[r, a:e], f = scan(q[r, a:e], k[r, a:e], v[r, a:e], ld, scale, i)
        E[r, a:e], ef = scan(abs(q[r, a:e]), abs(k[r, a:e]), abs(v[r, a:e]), ld, abs(scale), None if i is None else abs(i))
        fin.append(f)
        Ef.append(ef)
    return dict(o=o, final=np.stack(fin)), dict(o=E, final=np.stack(Ef))


def attention_bwd(q, k, v, ld, scale, do, init=None, dfinal=None, cu=None):
    b, T, H, dk = q.shape
    Hk = k.shape[2]
    k, v = expand(k, H), expand(v, H)

    def run(q, k, v, scale, do, init, dfinal):
        out = [np.zeros_like(q), np.zeros_like(k), np.zeros_like(v), []]
        for r, a, e, s in sequences(b, T, cu):
            g = scan_bwd(q[r, a:e], k[r, a:e], v[r, a:e], ld, scale, do[r, a:e], None if init is None else init[s],
                         None if dfinal is None else dfinal[s])
            for i in range(3):
                out[i][r, a:e] = g[i]
            out[3].append(g[3])
        share = lambda x: x.reshape(b, T, Hk, H // Hk, x.shape[3]).sum(3)
        return dict(dq=out[0], dk=share(out[1]), dv=share(out[2]), dinit=np.stack(out[3]))

    absn = lambda x: None if x is None else abs(x)
    return run(q, k, v, scale, do, init, dfinal), run(abs(q), abs(k), abs(v), abs(scale), abs(do), absn(init), absn(dfinal))


def bound(kind, ref, E, n, d):
    """Elementwise allowance: kind "fp32", "bf16" or "state" (fp32 states of bf16 inputs)."""
    b = (2 * n + d + 16) * U32 * E
    if kind == "bf16":
        b = b + UBF * (1 + 2.0 ** -6) * E + UBF * abs(ref)
    if kind == "state":
        b = b + 2.0 ** -16 * E
    return b + 1e-300


def check(got, ref, E, kind, n, d, what):
    got = np.asarray(got, np.float64)
    assert got.shape == ref.shape, f"{what}: {got.shape} {ref.shape}"
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    worst = float(np.max(np.abs(got - ref) / bound(kind, ref, E, n, d))) if got.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the allowance"
    if kind == "bf16" and got.size >= 4096:
        rel = float(np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300))
        assert rel <= 7e-3, f"{what}: rel-L2 {rel:.3g}"


# ---------------------------------------------------------------- group norm

def sig(v):
    return 1.0 / (1.0 + np.exp(-v))


def norm(x, G, w, bias, z, eps, act, gate, center, dy=None):
    """x [n, s, C] in 64 bits: dict(y, mean, rstd) and, with dy, the gradients."""
    n, s, C = x.shape
    Cg = C // G
    w = np.ones(C) if w is None else w
    bias = np.zeros(C) if bias is None else bias
    gate = gate if z is not None else ""
    sz = z * sig(z) if z is not None else None
    u = x * sz if gate == "before" else x
    ug = u.reshape(n, s, G, Cg)
    mean = ug.mean((1, 3)) if center else np.zeros((n, G))
    var = ((ug - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1.0 / np.sqrt(var + eps)
    up = lambda t: np.repeat(t, Cg, 1)[:, None, :]
    xh = (u - up(mean)) * up(rstd)
    t = xh * w + bias
    a = t * sig(t) if act == "silu" else t
    out = dict(y=a * sz if gate == "after" else a, mean=mean, rstd=rstd, t=t, xh=xh)
    if dy is None:
        return out
    slope = lambda v: sig(v) * (1 + v * (1 - sig(v)))
    # silu' = sig(v) (1 + v (1 - sig(v))) crosses zero at v = -1.28 as a difference of
    # numbers near 1: its error there is up to 4 2^-24 sig(v) (1 + |v|) < 6 2^-24, of no
    # relation to its value. So the sums over absolute values take |silu'| + 1 for it.
    wide = lambda v: abs(slope(v)) + 1
    g, ga = dy, abs(dy)
    if gate == "after":
        out["dz"] = dy * a * slope(z)
        g, ga = dy * sz, ga * abs(sz)
    if act == "silu":
        g, ga = g * slope(t), ga * wide(t)
    out["dweight"], out["dbias"] = (g * xh).sum((0, 1)), g.sum((0, 1))
    out["dweight_abs"], out["dbias_abs"] = (ga * abs(xh)).sum((0, 1)), ga.sum((0, 1))
    gx, gxa = g * w, ga * abs(w)
    mg = lambda q: up(q.reshape(n, s, G, Cg).mean((1, 3)))
    du = gx - xh * mg(gx * xh)
    if center:
        du = du - mg(gx)
    scale = gxa + abs(xh) * mg(gxa * abs(xh)) + mg(gxa)
    du, scale = du * up(rstd), scale * up(rstd)
    if gate == "before":
        out["dz"], out["dz_abs"] = du * x * slope(z), scale * abs(x) * wide(z)
        du, scale = du * sz, scale * abs(sz)
    out["dx"], out["dx_abs"] = du, scale
    return out

"""Gradients of the norm's weight and bias: sums over every row, each channel with an allowance of its own.

The definition is taken at the fp32 stats that the backward call is given, in 64 bits. With u = 2^-24, what a
row's term g xh is off by at most, to first order:
  sig   sigmoid(v) by exp2 and reciprocal: the exponent -v log2(e) is off by 1.5 |v| log2(e) u, so e^-v by
        (1.5 |v| + 2) u of itself, of which 1 - sig reaches the sum 1 + e^-v; that sum and the reciprocal add 3 u:
        e(v) = (1.5 |v| (1 - sig) + 5) u, relative.
  xh    (u_ - mean) rstd with u_ = x, or x z sig(z) to (e(z) + 2 u): rstd |u_| (e(z) + 2 u) + 2 u |xh|.
  t     xh w + b: |w| dxh + u (|xh w| + |t|).
  silu' s (1 + t (1 - s)), whose own derivative is at most 1/2:
        dt / 2 + s (|t| (s e + u) + 2 u (1 + |t| (1 - s))) + |silu'| (e + u), e = e(t).
  g     dy, times z sig(z) to e(z) + u, times silu': those errors, and 2 u |g|.
  g xh  |g| dxh + |xh| dg + u |g xh|.
Their sum passes no more than 320 + rows / 64 additions (of a thread's rows, of a workgroup's, of 8 accumulators
and 16 lanes of parts), each of which rounds a partial sum of at most the sum of |g xh|.
As roundings of different rows are independent, the error's norm over all channels stays near u times a few tens
of the result's: the per-term 16 u and sqrt(320) u of the additions are 34 u = 2e-6 of it; 1e-5 is held.
"""
import numpy as np
import pytest
import torch

import ssd_chunked_scan_fwd_amd as ssd

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24

# samples, positions, channels, groups
SHAPES = [(3, 1000, 40, 4), (1, 4097, 16, 2), (2, 65, 1032, 3), (2, 300, 7, 7), (700, 1, 256, 8), (1500, 1, 24, 3), (2500, 1, 70, 10),
          (400, 1, 5120, 1), (37, 1, 10240, 1), (9, 257, 64, 1), (1, 3000, 520, 8)]
FORMS = [("none", "", True), ("silu", "", True), ("none", "after", True), ("silu", "after", False), ("none", "before", False),
         ("silu", "before", True)]


def inputs(shape, dtype, gate, seed):
    n, s, C, G = shape
    g = torch.Generator().manual_seed(seed)
    dims = (n, C) if s == 1 else (n, s, C)
    r = lambda *d: torch.randn(*d, generator=g)
    return dict(x=(r(*dims) * 2 + 0.5).to(dtype), z=r(*dims).to(dtype) if gate else None, dy=r(*dims).to(dtype),
                w=1 + 0.2 * r(C), b=0.2 * r(C))


def sig(v):
    return 1.0 / (1.0 + np.exp(-v))


def terms(d, shape, act, gate, stats):
    """Every row's g xh and g, [n * s, C] in 64 bits, and what each is off by at most."""
    n, s, C, G = shape
    v = lambda t: None if t is None else t.cpu().double().numpy().reshape(n, s, C)
    x, z, dy, w, b = v(d["x"]), v(d["z"]), v(d["dy"]), d["w"].cpu().double().numpy(), d["b"].cpu().double().numpy()
    up = lambda t: np.repeat(t, C // G, 1)[:, None, :]
    mean, rstd = up(stats[..., 0]), up(stats[..., 1])
    e = lambda t: (1.5 * abs(t) * (1 - sig(t)) + 5) * U
    u_, du = x, 0.0
    if gate == "before":
        u_ = x * z * sig(z)
        du = abs(u_) * (e(z) + 2 * U)
    xh = (u_ - mean) * rstd
    dxh = rstd * du + 2 * U * abs(xh)
    t = xh * w + b
    dt = abs(w) * dxh + U * (abs(xh * w) + abs(t))
    g, dg = dy, 0.0
    if gate == "after":
        q = z * sig(z)
        g, dg = g * q, abs(g * q) * (e(z) + U)
    if act == "silu":
        st = sig(t)
        slope = st * (1 + t * (1 - st))
        dslope = dt / 2 + st * (abs(t) * (st * e(t) + U) + 2 * U * (1 + abs(t) * (1 - st))) + abs(slope) * (e(t) + U)
        g, dg = g * slope, abs(g) * dslope + dg * abs(slope)
    dg = dg + 2 * U * abs(g)
    flat = lambda t: np.broadcast_to(t, (n, s, C)).reshape(n * s, C)
    return flat(g * xh), flat(abs(g) * dxh + abs(xh) * dg + U * abs(g * xh)), flat(g), flat(dg)


def sums(d, shape, act, gate, stats):
    """[(result, allowance, rows' terms)] of dweight and dbias."""
    gx, dgx, g, dg = terms(d, shape, act, gate, stats)
    depth = 320 + gx.shape[0] / 64
    return [(t.sum(0), off.sum(0) + depth * U * abs(t).sum(0), t) for t, off in ((gx, dgx), (g, dg))]


def over(got, want, allow):
    """The share of the channels that are off by more than is allowed."""
    return float(np.mean(abs(got - want) > allow))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_what_the_allowance_catches(shape, form):
    """Zeros, a lost row and a row counted twice exceed it in most channels, so a lost slab or part does."""
    n, s, C, G = shape
    act, gate, center = form
    d = inputs(shape, F32, gate, C + s)
    x = d["x"].double().numpy().reshape(n, s, G, C // G)
    if gate == "before":
        z = d["z"].double().numpy().reshape(x.shape)
        x = x * z * sig(z)
    mean = x.mean((1, 3)) if center else np.zeros((n, G))
    stats = np.stack([mean, 1 / np.sqrt(((x - mean[:, None, :, None]) ** 2).mean((1, 3)) + 1e-5)], -1)
    for want, allow, rows in sums(d, shape, act, gate, stats):
        assert over(want, want, allow) == 0
        assert over(0 * want, want, allow) >= 0.9
        for r in (0, rows.shape[0] // 2, rows.shape[0] - 1):
            assert over(want - rows[r], want, allow) >= 0.5
            assert over(want + rows[r], want, allow) >= 0.5


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("shape", SHAPES)
def test_sums(shape, form, dtype):
    n, s, C, G = shape
    act, gate, center = form
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"[norm sums] {shape} {form} {dtype}", flush=True)
    d = {k: None if t is None else t.cuda() for k, t in inputs(shape, dtype, gate, C + s).items()}
    y, stats = ssd.group_norm(d["x"], G, d["w"], d["b"], d["z"], 1e-5, act, gate or "after", center)
    g = ssd.group_norm_bwd(d["x"], G, stats, d["dy"], d["w"], d["b"], d["z"], act, gate or "after", center)
    torch.cuda.synchronize()
    for name, (want, allow, _) in zip(("dweight", "dbias"), sums(d, shape, act, gate, stats.cpu().double().numpy())):
        got = g[name].cpu().double().numpy()
        worst = float(np.max(abs(got - want) / allow))
        rel = float(np.linalg.norm(got - want) / np.linalg.norm(want))
        assert worst <= 1 and rel <= 1e-5, f"{name}: {worst:.3g} of the allowance, rel-L2 {rel:.2g}"

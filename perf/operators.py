"""Workloads of the linear-attention layer's operators, for timing and checking.

Three families, as a layer of linear attention with one decay a head uses them:
the attention itself (a chunked form over prompts, its gradient, and the step
over one token a stream against a pool of states), the group norm with its
activation or gate that follows it (and its gradient), and the pages of the
state pool (copied or forked, and compacted).

Each case names one pass through one operator. `run` computes it in plain torch
operations, or, where `own` is true, with the library's calls.

Formulas (one head; lam = exp(log_decay), D the head's state, [Dv, Dk]):
  D_t = lam D_{t-1} + v_t k_t^T,   o_t = scale D_t q_t
  adjoint: L_t = scale do_t q_t^T + lam L_{t+1}  (L of the last token also has dfinal)
  dq_t = scale D_t^T do_t, dk_t = L_t^T v_t, dv_t = L_t k_t, dinit = lam L_first
Norm over the group of channels c and every position of a sample:
  u = x or x silu(z);  xh = (u - mean) rstd;  t = xh w + b;  y = act(t) or act(t) silu(z)
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the longest prompt of the repository's workloads, 32 heads of the usual width: prefill of one long document
        dict(name="fwd_prompt_16k", op="fwd", b=1, T=16384, H=32, Hk=32, dk=128, dv=128, lens="", init=False, dtype="bf16"),
        # a serving batch of ragged prompts packed together, continued from kept states, keys shared by 4 query heads;
        # one stream has no token in this batch, one has a single one
        dict(name="fwd_packed_ragged", op="fwd", b=1, T=5087, H=16, Hk=4, dk=64, dv=64,
             lens="701,0,1,1333,64,2047,130,811", init=True, dtype="bf16"),
        # a short fp32 run, as a user checking numerics makes it: launch latency
        dict(name="fwd_tiny_fp32", op="fwd", b=1, T=256, H=2, Hk=2, dk=16, dv=16, lens="", init=False, dtype="fp32"),
        # a training step's backward on long rows, 32 heads
        dict(name="bwd_train_8k", op="bwd", b=1, T=8192, H=32, Hk=32, dk=128, dv=128, lens="", init=False, dtype="bf16"),
        # backward of a smaller layer with shared keys, odd length, from a carried state and with its gradient
        dict(name="bwd_shared_odd", op="bwd", b=2, T=2047, H=24, Hk=8, dk=64, dv=64, lens="", init=True, dtype="bf16"),
        # one decode step of a full serving batch: 64 streams scattered over a pool of 80 states
        dict(name="step_b64", op="step", b=64, slots=80, H=32, Hk=32, dk=128, dv=128, dtype="bf16"),
        # one decode step of a single stream, fp32: the smallest call
        dict(name="step_b1_fp32", op="step", b=1, slots=4, H=24, Hk=24, dk=64, dv=64, dtype="fp32"),
        # the layer's own norm: each token's 32 heads normalised apart and gated, over the longest prompt
        dict(name="norm_token_gated", op="norm", n=16384, s=1, C=4096, G=32, act="none", gate="after", center=True, dtype="bf16"),
        # samples of a grid of positions (48 x 47, odd on purpose), channels last, silu after: groups of 10 channels
        dict(name="norm_grid_silu", op="norm", n=8, s=2256, C=320, G=32, act="silu", gate="", center=True, dtype="bf16"),
        # training through the gate-first root-mean-square norm of a block of 80 heads of 64
        dict(name="norm_bwd_rms_gated", op="norm_bwd", n=8192, s=1, C=5120, G=1, act="none", gate="before", center=False, dtype="bf16"),
        # four sequences forked to 28 new ones over two layers' pools (beam or best-of-n start)
        dict(name="pages_fork", op="copy", layers=2, slots=64, H=32, dk=128, dv=64, src=4, n=28),
        # a pool of 96 pages, about 60 % live after a wave of sequences ended, made dense again
        dict(name="pages_compact", op="compact", layers=1, slots=96, H=24, dk=64, dv=64, live=60),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["fwd", "fwd", "bwd", "bwd", "step", "norm", "norm", "norm_bwd", "copy", "compact"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    dims = [16, 32, 40, 64, 64, 96, 128, 128, 200, 256]
    if op in ("fwd", "bwd"):
        dk, dv = rng.choice(dims), rng.choice(dims)
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
        H = Hk * rng.choice([1, 1, 1, 2, 3, 4])
        if rng.random() < 0.4:
            lens = [rng.choice([0, 1, _logint(rng, 2, 4096), _logint(rng, 2, 4096)]) for _ in range(rng.randint(1, 9))]
            lens.append(_logint(rng, 1, 4096))
            return dict(op=op, b=1, T=sum(lens), H=H, Hk=Hk, dk=dk, dv=dv, lens=",".join(map(str, lens)),
                        init=rng.random() < 0.5, dtype=dtype)
        return dict(op=op, b=rng.choice([1, 1, 2, 3, 8]), T=_logint(rng, 1, 16384), H=H, Hk=Hk, dk=dk, dv=dv, lens="",
                    init=rng.random() < 0.5, dtype=dtype)
    if op == "step":
        b = _logint(rng, 1, 256)
        Hk = rng.choice([1, 2, 4, 8, 16, 24, 32])
        return dict(op=op, b=b, slots=b + rng.randint(0, 16), H=Hk * rng.choice([1, 1, 2, 4]), Hk=Hk,
                    dk=rng.choice(dims), dv=rng.choice(dims), dtype=dtype)
    if op in ("norm", "norm_bwd"):
        G = rng.choice([1, 1, 2, 8, 16, 32])
        C = G * rng.choice([7, 8, 10, 16, 40, 64, 128, 200])
        if rng.random() < 0.5:
            n, s = _logint(rng, 1, 16384), 1
        else:
            n, s = _logint(rng, 1, 16), _logint(rng, 2, 9216)
        gate = rng.choice(["", "after", "before"])
        return dict(op=op, n=n, s=s, C=C, G=G, act=rng.choice(["none", "silu"]), gate=gate,
                    center=rng.random() < 0.6, dtype=dtype)
    H, dk, dv = rng.choice([1, 8, 24, 32]), rng.choice([16, 64, 128]), rng.choice([16, 64, 128])
    slots, layers = _logint(rng, 4, 256), rng.randint(1, 3)
    if op == "copy":
        src = rng.randint(1, slots // 2)
        return dict(op=op, layers=layers, slots=slots, H=H, dk=dk, dv=dv, src=src, n=rng.randint(1, slots - src))
    return dict(op=op, layers=layers, slots=slots, H=H, dk=dk, dv=dv, live=rng.randint(0, slots))


def draw(rng):
    cap = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= cap[0] and w["flops"] <= cap[1]:
            return c


def work(case):
    e = 2 if case.get("dtype") == "bf16" else 4
    if case["op"] in ("fwd", "bwd"):
        tok = case["b"] * case["T"]
        H, Hk, dk, dv = case["H"], case["Hk"], case["dk"], case["dv"]
        nseq = len(_lens(case)) or case["b"]
        st = nseq * H * dk * dv * 4
        io = tok * (H * dk + Hk * dk + Hk * dv + H * dv) * e
        if case["op"] == "fwd":
            return dict(bytes=io + st * (2 if case["init"] else 1), flops=4 * tok * H * dk * dv)
        return dict(bytes=io + tok * (H * dk + Hk * dk + Hk * dv) * e + (3 * st if case["init"] else 0),
                    flops=10 * tok * H * dk * dv)
    if case["op"] == "step":
        b, H, Hk, dk, dv = (case[k] for k in ("b", "H", "Hk", "dk", "dv"))
        return dict(bytes=b * (2 * H * dk * dv * 4 + (H * dk + Hk * dk + Hk * dv + H * dv) * e), flops=6 * b * H * dk * dv)
    if case["op"] in ("norm", "norm_bwd"):
        el = case["n"] * case["s"] * case["C"]
        gate = 1 if case["gate"] else 0
        arrays = 2 + gate if case["op"] == "norm" else 3 + 2 * gate
        return dict(bytes=el * arrays * e + 4 * case["C"] * 4, flops=el * (10 if case["op"] == "norm" else 24))
    page = case["layers"] * case["H"] * case["dk"] * case["dv"] * 4
    if case["op"] == "copy":
        return dict(bytes=page * (min(case["src"], case["n"]) + case["n"]), flops=0)
    # pages that have to move: live ones above the live count (as many as holes below it), with live pages spread evenly
    return dict(bytes=int(2 * page * case["live"] * (1 - case["live"] / case["slots"])) + 8 * case["slots"], flops=0)


def _lens(case):
    return [int(v) for v in case["lens"].split(",")] if case.get("lens") else []


# ---------------------------------------------------------------- inputs

def _decays(H):
    # per-head decays as such layers fix them: 1 - 2^-x, x from 3 (fast) to 10 (slow) over the heads
    x = torch.linspace(3.0, 10.0, H, dtype=torch.float64) if H > 1 else torch.tensor([6.0], dtype=torch.float64)
    return torch.log1p(-torch.exp2(-x)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT.get(case.get("dtype", "fp32"))

    def rnd(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    st = {"case": case}
    if case["op"] in ("fwd", "bwd"):
        b, T, H, Hk, dk, dv = (case[k] for k in ("b", "T", "H", "Hk", "dk", "dv"))
        lens = _lens(case)
        nseq = len(lens) or b
        st.update(q=rnd(b, T, H, dk), k=rnd(b, T, Hk, dk), v=rnd(b, T, Hk, dv), ld=_decays(H).to(dev),
                  scale=dk ** -0.5, lens=lens, cu=None, init=None)
        if lens:
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        if case["init"]:  # states as a prefix leaves them: sums of about 1 / (1 - lam^2) outer products
            size = torch.rsqrt(1 - torch.exp(2 * st["ld"].double())).float()
            st["init"] = rnd(nseq, H, dv, dk, dtype=torch.float32) * size[None, :, None, None]
        if case["op"] == "bwd":
            st["do"] = rnd(b, T, H, dv)
            st["dfinal"] = rnd(nseq, H, dv, dk, dtype=torch.float32) if case["init"] else None
    elif case["op"] == "step":
        b, H, Hk, dk, dv = (case[k] for k in ("b", "H", "Hk", "dk", "dv"))
        ld = _decays(H).to(dev)
        size = torch.rsqrt(1 - torch.exp(2 * ld.double())).float()
        st.update(q=rnd(b, H, dk), k=rnd(b, Hk, dk), v=rnd(b, Hk, dv), ld=ld, scale=dk ** -0.5,
                  state=rnd(case["slots"], H, dv, dk, dtype=torch.float32) * size[None, :, None, None],
                  slots=torch.randperm(case["slots"], generator=g, device=dev)[:b].to(torch.int32))
    elif case["op"] in ("norm", "norm_bwd"):
        n, s, C, G = (case[k] for k in ("n", "s", "C", "G"))
        shape = (n, C) if s == 1 else (n, s, C)
        st.update(x=rnd(*shape) * 2 + 0.5, z=rnd(*shape) if case["gate"] else None,
                  w=1 + rnd(C, std=0.1, dtype=torch.float32), bias=rnd(C, std=0.1, dtype=torch.float32) if case["center"] else None,
                  eps=1e-5)
        if case["op"] == "norm_bwd":
            st["dy"] = rnd(*shape)
            u = st["x"].float() if case["gate"] != "before" else st["x"].float() * _silu(st["z"].float())
            u = u.view(n, s, G, C // G)
            mean = u.mean((1, 3)) if case["center"] else torch.zeros(n, G, device=dev)
            var = ((u - mean[:, None, :, None]) ** 2).mean((1, 3))
            st["stats"] = torch.stack([mean, torch.rsqrt(var + st["eps"])], -1).contiguous()  # as the forward pass keeps them
    else:
        L, slots = case["layers"], case["slots"]
        st["pool"] = rnd(L, slots, case["H"], case["dv"], case["dk"], dtype=torch.float32)
        perm = torch.randperm(slots, generator=g, device=dev).to(torch.int32)
        if case["op"] == "copy":
            st["src"] = perm[:case["src"]].repeat(-(-case["n"] // case["src"]))[:case["n"]].contiguous()
            st["dst"] = perm[case["src"]:case["src"] + case["n"]].contiguous()
        else:
            live = torch.zeros(slots, dtype=torch.uint8, device=dev)
            live[perm[:case["live"]].long()] = 1
            st["live"] = live
    return st


# ---------------------------------------------------------------- plain forms (32 bits)

def _silu(v):
    return v / (1 + torch.exp(-v))


def _scan_plain(q, k, v, ld, scale, init, first_pow=1, chunk=128):
    """o_i = scale sum_{j<=i} lam^(i-j) (q_i . k_j) v_j plus the carried state's term, over [B, T, H, *] in 32 bits,
    by chunks; the state entering token i is init times lam^(i + first_pow). Returns o and the last state [B, H, dq, dv]."""
    B, T, H, dq = q.shape
    dv = v.shape[-1]
    K = max(1, -(-T // chunk))
    pad = K * chunk - T

    def lay(t):  # [B * H, K, chunk, d]
        t = torch.cat([t, t.new_zeros(B, pad, H, t.shape[-1])], 1) if pad else t
        return t.transpose(1, 2).reshape(B * H, K, chunk, t.shape[-1]).contiguous()

    q, k, v = lay(q.float()), lay(k.float()), lay(v.float())
    g = ld.float().repeat(B)  # [B * H]
    i = torch.arange(chunk, device=q.device, dtype=torch.float32)
    diff = i[:, None] - i[None, :]
    D = torch.where(diff >= 0, torch.exp(g[:, None, None] * diff.clamp_min(0)), torch.zeros((), device=q.device))
    kt = k.transpose(2, 3).contiguous()
    o = torch.matmul(torch.matmul(q, kt) * D[:, None], v)
    last = torch.full((K,), float(chunk), device=q.device)  # tokens of each chunk
    last[K - 1] = chunk - pad
    wk = torch.exp(g[:, None, None] * (last[None, :, None] - 1 - i[None, None, :]).clamp_min(0))
    local = torch.matmul(kt, v * wk[..., None])  # [B * H, K, dq, dv]
    m = torch.arange(K, device=q.device, dtype=torch.float32)
    dm = m[:, None] - 1 - m[None, :]
    W = torch.where(dm >= 0, torch.exp(g[:, None, None] * (dm * chunk).clamp_min(0)), torch.zeros((), device=q.device))
    start = torch.matmul(W, local.reshape(B * H, K, dq * dv)).reshape(B * H, K, dq, dv)
    if init is not None:
        init = init.float().reshape(B * H, 1, dq, dv)
        p0 = torch.exp(g[:, None] * (m * chunk + first_pow - 1)[None, :])
        start = start + init * p0[:, :, None, None]
    wi = torch.exp(g[:, None] * (i + 1)[None, :])  # [B * H, chunk]
    o = o + torch.matmul(q, start) * wi[:, None, :, None]
    fin = start[:, K - 1] * torch.exp(g * last[K - 1])[:, None, None] + local[:, K - 1]
    o = o.reshape(B, H, K * chunk, dv)[:, :, :T].transpose(1, 2) * scale
    return o, fin.reshape(B, H, dq, dv)


def _pieces(st):
    """Rows or packed sequences as (row, first token, end) lists."""
    if st["cu"] is None:
        return None
    out, t = [], 0
    for n in st["lens"]:
        out.append((t, t + n))
        t += n
    return out


def _over_sequences(st, fn, names, inits):
    """fn over the whole batch, or sequence by sequence where packed; `fn` gets tensors and per-sequence states."""
    pieces = _pieces(st)
    if pieces is None:
        return fn(*[st[n] for n in names], *inits)
    outs = []
    for s, (a, b) in enumerate(pieces):
        outs.append(fn(*[st[n][:, a:b] for n in names], *[None if x is None else x[s:s + 1] for x in inits]))
    return [None if outs[0][i] is None else torch.cat([o[i] for o in outs], kind) for i, kind in enumerate(fn.cat)]


def _fwd_plain(st):
    rep = st["q"].shape[2] // st["k"].shape[2]

    def fn(q, k, v, init):
        k, v = k.float().repeat_interleave(rep, 2), v.float().repeat_interleave(rep, 2)
        if q.shape[1] == 0:
            z = q.new_zeros(1, 0, q.shape[2], v.shape[3], dtype=torch.float32)
            e = torch.zeros(1, q.shape[2], v.shape[3], q.shape[3], device=q.device)
            return z, e if init is None else init
        o, fin = _scan_plain(q, k, v, st["ld"], st["scale"], None if init is None else init.transpose(2, 3))
        return o, fin.transpose(2, 3)

    fn.cat = (1, 0)
    o, fin = _over_sequences(st, fn, ("q", "k", "v"), (st["init"],))
    return {"o": o.to(st["q"].dtype), "final": fin.contiguous()}


def _bwd_plain(st):
    H, Hk = st["q"].shape[2], st["k"].shape[2]
    scale, ld = st["scale"], st["ld"]

    def fn(q, k, v, do, init, dfinal):
        B, T = q.shape[:2]
        if T == 0:
            z = lambda t: t.float()
            dinit = dfinal if init is not None else None
            return z(q), z(k), z(v), dinit
        k, v = k.float().repeat_interleave(H // Hk, 2), v.float().repeat_interleave(H // Hk, 2)
        q, do = q.float(), do.float()
        dq, _ = _scan_plain(do, v, k, ld, scale, init)
        f = lambda t: t.flip(1)
        dfin = None if dfinal is None else dfinal / scale
        dv, rev = _scan_plain(f(k), f(q), f(do), ld, scale, None if dfin is None else dfin.transpose(2, 3), 0)
        dk, _ = _scan_plain(f(v), f(do), f(q), ld, scale, dfin, 0)
        share = lambda t: f(t).reshape(B, T, Hk, H // Hk, t.shape[3]).sum(3)
        dinit = None if init is None else rev.transpose(2, 3) * scale * torch.exp(ld)[None, :, None, None]
        return dq, share(dk), share(dv), dinit

    fn.cat = (1, 1, 1, 0)
    dq, dk, dv, dinit = _over_sequences(st, fn, ("q", "k", "v", "do"), (st["init"], st["dfinal"]))
    t = st["q"].dtype
    out = {"dq": dq.to(t), "dk": dk.to(t), "dv": dv.to(t)}
    if dinit is not None:
        out["dinit"] = dinit.contiguous()
    return out


def _step_plain(st):
    rep = st["q"].shape[1] // st["k"].shape[1]
    k, v = st["k"].float().repeat_interleave(rep, 1), st["v"].float().repeat_interleave(rep, 1)
    at = st["slots"].long()
    s = st["state"][at] * torch.exp(st["ld"])[None, :, None, None] + v[..., :, None] * k[..., None, :]
    st["state"][at] = s
    o = (s * st["q"].float()[..., None, :]).sum(-1) * st["scale"]
    return {"o": o.to(st["q"].dtype), "state": st["state"]}


def _norm_parts(st):
    c = st["case"]
    n, s, C, G = (c[k] for k in ("n", "s", "C", "G"))
    x = st["x"].float().view(n, s, G, C // G)
    z = st["z"].float().view(n, s, G, C // G) if c["gate"] else None
    w, b = st["w"].view(G, C // G), None if st["bias"] is None else st["bias"].view(G, C // G)
    return c, x, z, w, b


def _norm_plain(st):
    c, x, z, w, b = _norm_parts(st)
    u = x * _silu(z) if c["gate"] == "before" else x
    mean = u.mean((1, 3), keepdim=True) if c["center"] else torch.zeros_like(u[:, :1, :, :1])
    rstd = torch.rsqrt(((u - mean) ** 2).mean((1, 3), keepdim=True) + st["eps"])
    y = (u - mean) * rstd * w
    if b is not None:
        y = y + b
    if c["act"] == "silu":
        y = _silu(y)
    if c["gate"] == "after":
        y = y * _silu(z)
    stats = torch.stack([mean.view(c["n"], c["G"]), rstd.view(c["n"], c["G"])], -1)
    return {"y": y.view(st["x"].shape).to(st["x"].dtype), "stats": stats}


def _norm_bwd_plain(st):
    c, x, z, w, b = _norm_parts(st)
    dy = st["dy"].float().view(x.shape)
    mean, rstd = st["stats"][:, None, :, None, 0], st["stats"][:, None, :, None, 1]
    sz = _silu(z) if z is not None else None
    dsilu = lambda v: (lambda e: e * (1 + v * (1 - e)))(1 / (1 + torch.exp(-v)))
    u = x * sz if c["gate"] == "before" else x
    xh = (u - mean) * rstd
    t = xh * w if b is None else xh * w + b
    dz = None
    if c["gate"] == "after":
        a = _silu(t) if c["act"] == "silu" else t
        dz = dy * a * dsilu(z)
        dy = dy * sz
    if c["act"] == "silu":
        dy = dy * dsilu(t)
    out = {"dweight": (dy * xh).sum((0, 1)).view(-1)}
    if b is not None:
        out["dbias"] = dy.sum((0, 1)).view(-1)
    gx = dy * w
    du = gx - xh * (gx * xh).mean((1, 3), keepdim=True)
    if c["center"]:
        du = du - gx.mean((1, 3), keepdim=True)
    du = du * rstd
    if c["gate"] == "before":
        dz = du * x * dsilu(z)
        du = du * sz
    dt = st["x"].dtype
    out["dx"] = du.view(st["x"].shape).to(dt)
    if dz is not None:
        out["dz"] = dz.view(st["x"].shape).to(dt)
    return out


def _copy_plain(st):
    st["pool"][:, st["dst"].long()] = st["pool"][:, st["src"].long()]
    return {"pool": st["pool"]}


def _compact_plain(st):
    live = st["live"].bool()
    slots = live.numel()
    count = live.sum()
    at = torch.arange(slots, device=live.device)
    where = torch.where(live, at, torch.full_like(at, -1))
    hole = at[~live & (at < count)]
    high = at[live & (at >= count)]
    where[high] = hole
    st["pool"][:, hole] = st["pool"][:, high]
    return {"pool": st["pool"], "where": where.to(torch.int32), "count": count.to(torch.int32).view(1)}


# ---------------------------------------------------------------- the library's calls

def _own(st):
    import ssd_chunked_scan_fwd_amd as ssd
    c = st["case"]
    op = c["op"]
    if op == "fwd":
        o, fin = ssd.lin_attn_fwd(st["q"], st["k"], st["v"], st["ld"], cu_seqlens=st["cu"], scale=st["scale"],
                                  initial_state=st["init"])
        return {"o": o, "final": fin}
    if op == "bwd":
        r = ssd.lin_attn_bwd(st["q"], st["k"], st["v"], st["ld"], st["do"], cu_seqlens=st["cu"], scale=st["scale"],
                             initial_state=st["init"], dfinal_state=st["dfinal"], want_dinit=st["init"] is not None)
        return {k: r[k] for k in ("dq", "dk", "dv", "dinit") if r[k] is not None}
    if op == "step":
        o = ssd.lin_attn_step(st["state"], st["q"], st["k"], st["v"], st["ld"], slots=st["slots"], scale=st["scale"])
        return {"o": o, "state": st["state"]}
    if op == "norm":
        y, stats = ssd.group_norm(st["x"], c["G"], weight=st["w"], bias=st["bias"], z=st["z"], eps=st["eps"], act=c["act"],
                                  gate=c["gate"] or "after", center=c["center"])
        return {"y": y, "stats": stats}
    if op == "norm_bwd":
        r = ssd.group_norm_bwd(st["x"], c["G"], st["stats"], st["dy"], weight=st["w"], bias=st["bias"], z=st["z"],
                               act=c["act"], gate=c["gate"] or "after", center=c["center"])
        return {k: r[k] for k in ("dweight", "dbias", "dx", "dz") if r[k] is not None}
    if op == "copy":
        ssd.pages_copy(st["pool"], st["src"], st["dst"])
        return {"pool": st["pool"]}
    where, count = ssd.pages_compact(st["pool"], st["live"])
    return {"pool": st["pool"], "where": where, "count": count}


_PLAIN = {"fwd": _fwd_plain, "bwd": _bwd_plain, "step": _step_plain, "norm": _norm_plain, "norm_bwd": _norm_bwd_plain,
          "copy": _copy_plain, "compact": _compact_plain}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_sequence(q, k, v, lam, scale, D):
    """The recurrence token by token over [T, heads, *]: outputs, and the state after the last token."""
    o = q.new_empty(q.shape[0], q.shape[1], v.shape[2])
    for t in range(q.shape[0]):
        D.mul_(lam).addcmul_(v[t].unsqueeze(2), k[t].unsqueeze(1))
        o[t] = torch.bmm(D, q[t].unsqueeze(2)).squeeze(2)
    return o * scale, D


def _exact_adjoint(q, k, v, do, lam, scale, D, L):
    """Gradients token by token, forwards for dq and backwards for the others, and the first state's."""
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for t in range(q.shape[0]):
        D.mul_(lam).addcmul_(v[t].unsqueeze(2), k[t].unsqueeze(1))
        dq[t] = torch.bmm(do[t].unsqueeze(1), D).squeeze(1) * scale
    for t in range(q.shape[0] - 1, -1, -1):
        L.addcmul_(do[t].unsqueeze(2), q[t].unsqueeze(1), value=scale)
        dk[t] = torch.bmm(v[t].unsqueeze(1), L).squeeze(1)
        dv[t] = torch.bmm(L, k[t].unsqueeze(2)).squeeze(2)
        L.mul_(lam)
    return dq, dk, dv, L


def _exact_attention(case, st):
    b, H, Hk, scale = case["b"], case["H"], case["Hk"], st["scale"]
    lens = st["lens"] or [case["T"]]   # rows of equal length run side by side, as b * H heads
    lam = torch.exp(st["ld"].double())[:, None, None].repeat(b, 1, 1)

    def heads(t):
        t = t.double().repeat_interleave(H // t.shape[2], 2)
        return t.transpose(0, 1).reshape(t.shape[1], b * H, t.shape[3])

    def state(name, s):
        if st.get(name) is None:
            return lam.new_zeros(b * H, case["dv"], case["dk"])
        t = st[name] if not st["lens"] else st[name][s:s + 1]
        return t.double().reshape(b * H, case["dv"], case["dk"]).clone()

    names = ("q", "k", "v", "do") if case["op"] == "bwd" else ("q", "k", "v")
    x = [heads(st[n]) for n in names]
    outs, states, a = [], [], 0
    for s, n in enumerate(lens):
        part = [t[a:a + n] for t in x]
        if case["op"] == "bwd":
            *o, last = _exact_adjoint(*part, lam, scale, state("init", s), state("dfinal", s))
        else:
            *o, last = _exact_sequence(*part, lam, scale, state("init", s))
        outs.append(o)
        states.append(last.view(-1, H, case["dv"], case["dk"]))
        a += n
    outs = [torch.cat([o[i] for o in outs]) for i in range(len(outs[0]))]
    outs = [t.view(case["T"], b, H, -1).transpose(0, 1) for t in outs]
    states = torch.cat(states)
    if case["op"] == "fwd":
        return {"o": outs[0], "final": states}
    share = lambda t: t.reshape(b, case["T"], Hk, H // Hk, t.shape[3]).sum(3)
    res = {"dq": outs[0], "dk": share(outs[1]), "dv": share(outs[2])}
    if st["init"] is not None:
        res["dinit"] = states
    return res


def _exact_norm(case, st):
    n, s, C, G = (case[k] for k in ("n", "s", "C", "G"))
    d = lambda t: None if t is None else t.double()
    x, z, w = (None if t is None else t.double() for t in (st["x"], st["z"], st["w"]))
    x = x.view(n, s, C)
    z = None if z is None else z.view(n, s, C)
    bias = torch.zeros_like(w) if st["bias"] is None else d(st["bias"])
    per_c = lambda t: t.repeat_interleave(C // G, 1)[:, None]             # [n, G] -> [n, 1, C]
    per_g = lambda t: t.sum(1).view(n, G, C // G).sum(2)                  # [n, s, C] -> [n, G]
    M = s * (C // G)
    sg = None if z is None else torch.sigmoid(z)
    u = x * z * sg if case["gate"] == "before" else x
    if case["op"] == "norm":
        mean = per_g(u) / M if case["center"] else torch.zeros(n, G, dtype=u.dtype, device=u.device)
        rstd = (per_g((u - per_c(mean)) ** 2) / M + st["eps"]) ** -0.5
    else:
        mean, rstd = d(st["stats"][..., 0]), d(st["stats"][..., 1])
    xh = (u - per_c(mean)) * per_c(rstd)
    t = xh * w + bias
    st_ = torch.sigmoid(t)
    a = t * st_ if case["act"] == "silu" else t
    if case["op"] == "norm":
        y = a * z * sg if case["gate"] == "after" else a
        return {"y": y.view(st["x"].shape), "stats": torch.stack([mean, rstd], -1)}
    dy = d(st["dy"]).view(n, s, C)
    out = {}
    dz = None
    if case["gate"] == "after":
        dz = dy * a * (sg + z * sg * (1 - sg))
        dy = dy * z * sg
    if case["act"] == "silu":
        dy = dy * (st_ + t * st_ * (1 - st_))
    out["dweight"] = (dy * xh).sum((0, 1))
    if st["bias"] is not None:
        out["dbias"] = dy.sum((0, 1))
    gx = dy * w
    du = gx - xh * per_c(per_g(gx * xh) / M)
    if case["center"]:
        du = du - per_c(per_g(gx) / M)
    du = du * per_c(rstd)
    if case["gate"] == "before":
        dz = du * x * (sg + z * sg * (1 - sg))
        du = du * z * sg
    out["dx"] = du.view(st["x"].shape)
    if dz is not None:
        out["dz"] = dz.view(st["x"].shape)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_attention(case, st)
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(case, st)
    if case["op"] == "step":
        rep = case["H"] // case["Hk"]
        lam = torch.exp(st["ld"].double())
        state = st["state"].double()
        o = torch.zeros(case["b"], case["H"], case["dv"], dtype=torch.float64, device=state.device)
        for i, s in enumerate(st["slots"].tolist()):
            k, v = (st[n][i].double().repeat_interleave(rep, 0) for n in ("k", "v"))
            state[s] = state[s] * lam[:, None, None] + torch.einsum("hi,hj->hij", v, k)
            o[i] = st["scale"] * torch.einsum("hij,hj->hi", state[s], st["q"][i].double())
        return {"o": o, "state": state}
    pool = st["pool"].double()
    if case["op"] == "copy":
        old = pool.clone()
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            pool[:, b] = old[:, a]
        return {"pool": pool}
    live = st["live"].tolist()
    count = sum(live)
    holes = [i for i in range(count) if not live[i]]
    high = [i for i in range(count, len(live)) if live[i]]
    where = [i if live[i] else -1 for i in range(len(live))]
    for a, b in zip(high, holes):
        pool[:, b] = pool[:, a]
        where[a] = b
    dev = pool.device
    return {"pool": pool, "where": torch.tensor(where, dtype=torch.int32, device=dev),
            "count": torch.tensor([count], dtype=torch.int32, device=dev)}

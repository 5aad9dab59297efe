"""Workloads of the gated delta rule and of rotary positions, for timing and checking.

The gated delta rule is linear attention whose state is corrected by what it
already answers: over prompts (a chunked form), its gradients, and one token a
stream against a pool of states. Rotary positions turn queries and keys before
such a scan, over prompts, for single tokens, and backwards.

Each case names one pass through one operator. `run` computes it in plain torch
operations, or, where `own` is true, with the library's calls.

Formulas (one value head; a = exp(log_decay), S the head's state, [dv, dk]):
  u_t = beta_t (v_t - a_t S_{t-1} k_t),  S_t = a_t S_{t-1} + u_t k_t^T,  o_t = scale S_t q_t
  value head h reads query and key head h / (H / Hk)
Rotary: a pair (x, y) of a head becomes scale (x cos - y sin, y cos + x sin) of the
angle position * freq_i; pairs are (i, i + rot / 2) or (2 i, 2 i + 1), i < rot / 2.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the longest prompt of the repository's workloads, 16 query and key heads for 32 value heads
        dict(name="delta_prompt_16k", op="fwd", b=1, T=16384, H=32, Hk=16, dk=128, dv=128, lens="", init=False, dtype="bf16"),
        # a serving batch of ragged prompts packed together, continued from kept states; one stream has no token in this
        # batch, one has a single one
        dict(name="delta_packed_ragged", op="fwd", b=1, T=5087, H=16, Hk=4, dk=64, dv=96,
             lens="701,0,1,1333,64,2047,130,811", init=True, dtype="bf16"),
        # a long document on a narrow layer (or one GPU's share of the heads): few heads, a long chain of tokens
        dict(name="delta_few_heads", op="fwd", b=1, T=8192, H=4, Hk=2, dk=128, dv=128, lens="", init=True, dtype="bf16"),
        # a short fp32 run, as a user checking numerics makes it: launch latency
        dict(name="delta_tiny_fp32", op="fwd", b=1, T=256, H=2, Hk=2, dk=16, dv=16, lens="", init=False, dtype="fp32"),
        # a training step's backward on long rows
        dict(name="delta_bwd_8k", op="bwd", b=1, T=8192, H=32, Hk=16, dk=128, dv=128, lens="", init=False, dtype="bf16"),
        # backward of a smaller layer, odd length, heads of 64, from a carried state and with its gradient
        dict(name="delta_bwd_odd", op="bwd", b=2, T=2047, H=24, Hk=24, dk=64, dv=64, lens="", init=True, dtype="bf16"),
        # one decode step of a full serving batch: 64 streams scattered over a pool of 80 states
        dict(name="delta_step_b64", op="step", b=64, slots=80, H=32, Hk=16, dk=128, dv=128, dtype="bf16"),
        # one decode step of a single stream, fp32: the smallest call
        dict(name="delta_step_b1_fp32", op="step", b=1, slots=4, H=24, Hk=24, dk=64, dv=64, dtype="fp32"),
        # queries and keys of the longest prompt, inside the rows of one projection
        dict(name="rotary_prompt_16k", op="rot", b=1, T=16384, H=32, Hk=8, d=128, rot=128, layout="half", lens="", far=0,
             gap=1024, scale=1.0, dtype="bf16"),
        # a packed batch whose sequences continue far along (positions of 10^6), a part of each head, pairs side by side,
        # amplitudes scaled as for lengthened contexts
        dict(name="rotary_packed_part", op="rot", b=1, T=5087, H=16, Hk=4, d=80, rot=48, layout="interleaved",
             lens="701,0,1,1333,64,2047,130,811", far=1000000, gap=320, scale=1.1, dtype="bf16"),
        # one token for each of 64 streams, each at its own position: the smallest call
        dict(name="rotary_step_b64", op="rot_step", b=64, H=32, Hk=8, d=128, rot=64, layout="half", far=100000, gap=1024,
             scale=1.0, dtype="bf16"),
        # gradients of rotated queries and keys in a training step
        dict(name="rotary_bwd_8k", op="rot_bwd", b=4, T=2047, H=32, Hk=32, d=64, rot=64, layout="half", lens="", far=0, gap=0,
             scale=1.0, dtype="bf16"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _some_lens(rng):
    lens = [rng.choice([0, 1, _logint(rng, 2, 4096), _logint(rng, 2, 4096)]) for _ in range(rng.randint(1, 9))]
    return lens + [_logint(rng, 1, 4096)]


def _draw(rng):
    op = rng.choice(["fwd", "fwd", "fwd", "bwd", "bwd", "bwd", "step", "step", "rot", "rot", "rot_step", "rot_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("fwd", "bwd", "step"):
        dims = [16, 24, 32, 40, 64, 64, 96, 128, 128, 200, 256]
        Hk = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
        c = dict(op=op, H=Hk * rng.choice([1, 1, 2, 3, 4]), Hk=Hk, dk=rng.choice(dims), dv=rng.choice(dims), dtype=dtype)
        if op == "step":
            c["b"] = _logint(rng, 1, 256)
            c["slots"] = c["b"] + rng.randint(0, 16)
            return c
        c["init"] = rng.random() < 0.5
        if rng.random() < 0.4:
            lens = _some_lens(rng)
            return dict(c, b=1, T=sum(lens), lens=",".join(map(str, lens)))
        return dict(c, b=rng.choice([1, 1, 2, 3, 8]), T=_logint(rng, 1, 16384), lens="")
    d = rng.choice([16, 32, 64, 64, 80, 96, 128, 128, 256])
    c = dict(op=op, H=rng.choice([1, 4, 8, 16, 32, 40]), Hk=rng.choice([1, 2, 4, 8, 16]), d=d,
             rot=rng.choice([d, d, d // 2, 8 * rng.randint(1, d // 8)]), layout=rng.choice(["half", "interleaved"]),
             far=rng.choice([0, 0, 5000, 1000000]), gap=rng.choice([0, 64, 1000]), scale=rng.choice([1.0, 1.0, 1.2]), dtype=dtype)
    if op == "rot_step":
        return dict(c, b=_logint(rng, 1, 512))
    if op == "rot" and rng.random() < 0.4:
        lens = _some_lens(rng)
        return dict(c, b=1, T=sum(lens), lens=",".join(map(str, lens)))
    return dict(c, b=rng.choice([1, 2, 3, 8]), T=_logint(rng, 1, 16384), lens="")


def draw(rng):
    cap = [max(work(c)[k] for c in listed()) for k in ("bytes", "flops")]
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= cap[0] and w["flops"] <= cap[1]:
            return c


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    H, Hk = case["H"], case["Hk"]
    if case["op"].startswith("rot"):
        tok = case["b"] * case.get("T", 1)
        return dict(bytes=tok * (H + Hk) * case["d"] * 2 * e + tok * 4, flops=tok * (H + Hk) * case["rot"] * 3)
    dk, dv = case["dk"], case["dv"]
    if case["op"] == "step":
        b = case["b"]
        return dict(bytes=b * (2 * H * dk * dv * 4 + (2 * Hk * dk + 2 * H * dv) * e + 8 * H), flops=6 * b * H * dk * dv)
    tok = case["b"] * case["T"]
    st = (len(_lens(case)) or case["b"]) * H * dk * dv * 4
    qkv, gates = tok * (2 * Hk * dk + H * dv) * e, tok * H * 8
    if case["op"] == "fwd":
        return dict(bytes=qkv + tok * H * dv * e + gates + st * (2 if case["init"] else 1), flops=6 * tok * H * dk * dv)
    return dict(bytes=2 * qkv + tok * H * dv * e + 2 * gates + (3 * st if case["init"] else 0), flops=16 * tok * H * dk * dv)


def _lens(case):
    return [int(v) for v in case["lens"].split(",")] if case.get("lens") else []


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = _DT[case["dtype"]]

    def rnd(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)

    def uni(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=dev) * (hi - lo) + lo

    def unit(*shape):   # rows of norm 1, as such layers normalise queries and keys
        x = torch.randn(*shape, generator=g, device=dev)
        return (x * torch.rsqrt((x * x).sum(-1, keepdim=True) + 1e-6)).to(dt)

    st = {"case": case}
    H, Hk = case["H"], case["Hk"]
    lens = _lens(case)
    st.update(lens=lens, cu=None)
    if lens:
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
    if case["op"] in ("fwd", "bwd", "step"):
        dk, dv = case["dk"], case["dv"]
        lead = (case["b"],) if case["op"] == "step" else (case["b"], case["T"])
        # decays of a step of U(0.001, 0.1) times a rate of U(1, 16) a head, learning rates of sigmoid(N(0, 1))
        st.update(q=unit(*lead, Hk, dk), k=unit(*lead, Hk, dk), v=rnd(*lead, H, dv),
                  ld=-uni(*lead, H, lo=0.001, hi=0.1) * uni(H, lo=1.0, hi=16.0), beta=torch.sigmoid(rnd(*lead, H, dtype=torch.float32)),
                  scale=dk ** -0.5, init=None)
        if case["op"] == "step":
            st["state"] = rnd(case["slots"], H, dv, dk, dtype=torch.float32)
            st["slots"] = torch.randperm(case["slots"], generator=g, device=dev)[:case["b"]].to(torch.int32)
            return st
        nseq = len(lens) or case["b"]
        if case["init"]:
            st["init"] = rnd(nseq, H, dv, dk, dtype=torch.float32)
        if case["op"] == "bwd":
            st["do"] = rnd(*lead, H, dv)
            st["dfinal"] = rnd(nseq, H, dv, dk, dtype=torch.float32) if case["init"] else None
        return st
    d, rot = case["d"], case["rot"]
    lead = (case["b"],) if case["op"] == "rot_step" else (case["b"], case["T"])
    rows = rnd(*lead, (H + Hk) * d + case["gap"])   # one projection; behind q and k the values
    st["q"], st["k"] = rows[..., :H * d].unflatten(-1, (H, d)), rows[..., H * d:(H + Hk) * d].unflatten(-1, (Hk, d))
    st["freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)).float()
    st.update(scale=case["scale"], layout=case["layout"], positions=None, offsets=None)
    if case["op"] == "rot_step":
        st["positions"] = torch.randint(0, case["far"] + 1, (case["b"],), generator=g, device=dev).to(torch.int32)
    elif case["far"]:
        st["offsets"] = torch.randint(0, case["far"] + 1, (len(lens) or case["b"],), generator=g, device=dev).to(torch.int32)
    return st


# ---------------------------------------------------------------- plain forms (32 bits)

_C = 64


def _pad_rows(st, x, fill=0.0):
    """[b, T, ...] to rows of equal length, a multiple of the chunk: [rows, Tp, ...], behind their ends `fill`."""
    c = st["case"]
    if not st["lens"]:
        Tp = -(-c["T"] // _C) * _C
        return torch.cat([x, x.new_full((c["b"], Tp - c["T"], *x.shape[2:]), fill)], 1) if Tp > c["T"] else x
    Tp = -(-max(max(st["lens"]), 1) // _C) * _C
    cu = st["cu"].long()
    at = cu[:-1, None] + torch.arange(Tp, device=x.device)
    inside = at < cu[1:, None]
    y = x[0, at.clamp_max(c["T"] - 1)]
    return torch.where(inside.reshape(*inside.shape, *([1] * (y.dim() - 2))), y, torch.full_like(y, fill))


def _unpad_rows(st, y):
    c = st["case"]
    if not st["lens"]:
        return y[:, :c["T"]]
    cu = st["cu"].long()
    t = torch.arange(c["T"], device=y.device)
    s = torch.searchsorted(cu[1:], t, right=True)
    return y[s, t - cu[s]].unsqueeze(0)


def _delta_chunks(st, q, k, v, ld, beta, S):
    """The chunked rule in 32 bits over rows of whole chunks: q, k [n, T, H, dk], v [n, T, H, dv], ld and beta
    [n, T, H], S [n * H, dk, dv] (transposed states). Returns o [n, T, H, dv] and the last states."""
    n, T, H, dk = q.shape
    K = T // _C

    def lay(x):   # [n * H, K, C, *]
        return x.transpose(1, 2).reshape(n * H, K, _C, *x.shape[3:])

    q, k, v, ld, beta = lay(q), lay(k), lay(v), lay(ld.unsqueeze(-1)), lay(beta.unsqueeze(-1))
    G = ld.cumsum(2)
    i = torch.arange(_C, device=q.device)
    lower = i[:, None] >= i[None, :]
    D = torch.where(lower, torch.exp(torch.where(lower, G - G.transpose(2, 3), torch.zeros((), device=q.device))),
                    torch.zeros((), device=q.device))
    kt = k.transpose(2, 3).contiguous()
    A = torch.matmul(k, kt) * D * beta * (i[:, None] > i[None, :])
    P = torch.matmul(q, kt) * D
    # (I + A)^-1 by blocks: those of 2 s from the inverses of those of s
    M = torch.eye(_C, device=q.device).expand_as(A)
    for s in (1, 2, 4, 8, 16, 32):
        cross = (i[:, None] // (2 * s) == i[None, :] // (2 * s)) & (i[:, None] // s > i[None, :] // s)
        M = M - torch.matmul(M, torch.matmul(A * cross, M))
    W = torch.matmul(M, beta * torch.exp(G) * k)
    Y = torch.matmul(M, beta * v)
    qd = q * torch.exp(G)
    end = G[:, :, -1:]
    kd = (k * torch.exp(end - G)).transpose(2, 3).contiguous()
    keep = torch.exp(end)
    out = []
    for c in range(K):
        u = Y[:, c] - torch.matmul(W[:, c], S)
        out.append(torch.matmul(qd[:, c], S) + torch.matmul(P[:, c], u))
        S = keep[:, c] * S + torch.matmul(kd[:, c], u)
    o = torch.stack(out, 1).reshape(n, H, T, -1).transpose(1, 2) * st["scale"]
    return o, S


def _delta_plain(st, q, k, v, ld, beta, init):
    c = st["case"]
    rep = c["H"] // c["Hk"]
    rows = len(st["lens"]) or c["b"]
    q, k = (_pad_rows(st, x).repeat_interleave(rep, 2) for x in (q, k))
    v, ld, beta = (_pad_rows(st, x) for x in (v, ld, beta))
    if init is None:
        S = torch.zeros(rows * c["H"], c["dk"], c["dv"], device=q.device)
    else:
        S = init.reshape(rows * c["H"], c["dv"], c["dk"]).transpose(1, 2).contiguous()
    o, S = _delta_chunks(st, q, k, v, ld, beta, S)
    return _unpad_rows(st, o), S.transpose(1, 2).reshape(rows, c["H"], c["dv"], c["dk"])


def _fwd_plain(st):
    o, fin = _delta_plain(st, st["q"].float(), st["k"].float(), st["v"].float(), st["ld"], st["beta"], st["init"])
    return {"o": o.to(st["q"].dtype), "final": fin.contiguous()}


def _bwd_plain(st):
    x = [st[n].float().detach().clone().requires_grad_() for n in ("q", "k", "v", "ld", "beta")]
    init = None if st["init"] is None else st["init"].detach().clone().requires_grad_()
    o, fin = _delta_plain(st, *x, init)
    total = (o * st["do"].float()).sum()
    if st["dfinal"] is not None:
        total = total + (fin * st["dfinal"]).sum()
    grads = torch.autograd.grad(total, x if init is None else x + [init])
    dt = st["q"].dtype
    out = {"dq": grads[0].to(dt), "dk": grads[1].to(dt), "dv": grads[2].to(dt), "dld": grads[3], "dbeta": grads[4]}
    if init is not None:
        out["dinit"] = grads[5]
    return out


def _step_plain(st):
    rep = st["case"]["H"] // st["case"]["Hk"]
    q, k = (st[n].float().repeat_interleave(rep, 1)[..., None, :] for n in ("q", "k"))
    at = st["slots"].long()
    s = st["state"][at] * torch.exp(st["ld"])[..., None, None]
    u = st["beta"][..., None] * (st["v"].float() - (s * k).sum(-1))
    s = s + u[..., None] * k
    st["state"][at] = s
    o = (s * q).sum(-1) * st["scale"]
    return {"o": o.to(st["q"].dtype), "state": st["state"]}


def _positions(st):
    """The position of every token, [b] or [b, T], in 64 bits."""
    c = st["case"]
    if st["positions"] is not None:
        return st["positions"].double()
    if st["lens"]:
        cu = st["cu"].long()
        t = torch.arange(c["T"], device=cu.device)
        s = torch.searchsorted(cu[1:], t, right=True)
        p = t - cu[s] + (0 if st["offsets"] is None else st["offsets"].long()[s])
        return p.double().unsqueeze(0)
    p = torch.arange(c["T"], device=st["q"].device).expand(c["b"], -1)
    return (p if st["offsets"] is None else p + st["offsets"].long()[:, None]).double()


def _rot_plain(st):
    rot, sign = st["case"]["rot"], -1.0 if st["case"]["op"] == "rot_bwd" else 1.0
    t = _positions(st)[..., None, None] * st["freq"].double()
    cos, sin = (st["scale"] * torch.cos(t)).float(), (sign * st["scale"] * torch.sin(t)).float()

    def turn(x):
        y = x.float()
        r = y[..., :rot]
        if st["layout"] == "half":
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([r, y[..., rot:]], -1).to(x.dtype)

    return {"q": turn(st["q"]), "k": turn(st["k"])}


# ---------------------------------------------------------------- the library's calls

def _own(st):
    import ssd_chunked_scan_fwd_amd as ssd
    op = st["case"]["op"]
    if op == "fwd":
        o, fin = ssd.gated_delta_fwd(st["q"], st["k"], st["v"], st["ld"], st["beta"], cu_seqlens=st["cu"], scale=st["scale"],
                                     initial_state=st["init"])
        return {"o": o, "final": fin}
    if op == "bwd":
        r = ssd.gated_delta_bwd(st["q"], st["k"], st["v"], st["ld"], st["beta"], st["do"], cu_seqlens=st["cu"], scale=st["scale"],
                                initial_state=st["init"], dfinal_state=st["dfinal"], want_dinit=st["init"] is not None)
        out = {"dq": r["dq"], "dk": r["dk"], "dv": r["dv"], "dld": r["dlog_decay"], "dbeta": r["dbeta"]}
        if r["dinit"] is not None:
            out["dinit"] = r["dinit"]
        return out
    if op == "step":
        o = ssd.gated_delta_step(st["state"], st["q"], st["k"], st["v"], st["ld"], st["beta"], slots=st["slots"], scale=st["scale"])
        return {"o": o, "state": st["state"]}
    turn = ssd.rotary_bwd if op == "rot_bwd" else ssd.rotary
    q, k = turn(st["q"], st["k"], st["freq"], positions=st["positions"], cu_seqlens=st["cu"], offsets=st["offsets"],
                layout=st["layout"], scale=st["scale"])
    return {"q": q, "k": k}


_PLAIN = {"fwd": _fwd_plain, "bwd": _bwd_plain, "step": _step_plain, "rot": _rot_plain, "rot_step": _rot_plain,
          "rot_bwd": _rot_plain}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_delta(case, st):
    """The rule token by token; backwards, by its adjoint from the last token to the first, the states
    between kept for 128 tokens at a time."""
    b, H, dk, dv, scale = case["b"], case["H"], case["dk"], case["dv"], st["scale"]
    lens = st["lens"] or [case["T"]]   # rows of equal length run side by side, as b * H heads
    back = case["op"] == "bwd"

    def heads(t):   # [T, b * H, *]
        t = t.double().repeat_interleave(H // t.shape[2], 2)
        return t.transpose(0, 1).reshape(t.shape[1], b * H, *t.shape[3:])

    def state(name, s):
        if st.get(name) is None:
            return torch.zeros(b * H, dv, dk, dtype=torch.float64, device=st["q"].device)
        t = st[name] if not st["lens"] else st[name][s:s + 1]
        return t.double().reshape(b * H, dv, dk).clone()

    q, k, v = (heads(st[n]) for n in ("q", "k", "v"))
    a, beta = torch.exp(heads(st["ld"][..., None])), heads(st["beta"][..., None])
    do = heads(st["do"]) if back else None

    def token(S, t):
        S = S * a[t, :, :, None]
        u = beta[t] * (v[t] - torch.bmm(S, k[t].unsqueeze(2)).squeeze(2))
        return S + u.unsqueeze(2) * k[t].unsqueeze(1), u

    o = torch.empty_like(v)
    dq, dk_, dv_ = (torch.empty_like(x) if back else None for x in (q, k, v))
    da, db = (torch.empty_like(a) if back else None for _ in range(2))
    ends, first, t0 = [], [], 0
    for s, n in enumerate(lens):
        S, kept = state("init", s), []
        for t in range(t0, t0 + n):
            if (t - t0) % 128 == 0:
                kept.append(S)
            S, _ = token(S, t)
            o[t] = scale * torch.bmm(S, q[t].unsqueeze(2)).squeeze(2)
        ends.append(S)
        if back:
            L = state("dfinal", s)
            for m in range(len(kept) - 1, -1, -1):
                lo, hi = t0 + 128 * m, min(t0 + 128 * (m + 1), t0 + n)
                before, us = [kept[m]], []
                for t in range(lo, hi):
                    S, u = token(before[-1], t)
                    before.append(S)
                    us.append(u)
                for t in range(hi - 1, lo - 1, -1):
                    S0, S1, u = before[t - lo], before[t - lo + 1], us[t - lo]
                    dq[t] = scale * torch.bmm(do[t].unsqueeze(1), S1).squeeze(1)
                    L = L + scale * do[t].unsqueeze(2) * q[t].unsqueeze(1)
                    gu = torch.bmm(L, k[t].unsqueeze(2)).squeeze(2)          # of u
                    decayed = S0 * a[t, :, :, None]
                    off = v[t] - torch.bmm(decayed, k[t].unsqueeze(2)).squeeze(2)
                    ge = beta[t] * gu                                         # of the error that u corrects
                    db[t] = (gu * off).sum(-1, keepdim=True)
                    dv_[t] = ge
                    dk_[t] = torch.bmm(u.unsqueeze(1), L).squeeze(1) - torch.bmm(ge.unsqueeze(1), decayed).squeeze(1)
                    L = L - ge.unsqueeze(2) * k[t].unsqueeze(1)               # of the decayed state
                    da[t] = (L * decayed).sum((1, 2)).unsqueeze(-1)
                    L = L * a[t, :, :, None]
            first.append(L)
        t0 += n

    def rows(x, shared=False):
        x = x.reshape(case["T"], b, H, *x.shape[2:]).transpose(0, 1)
        if shared:
            x = x.reshape(b, case["T"], case["Hk"], H // case["Hk"], x.shape[3]).sum(3)
        return x

    states = lambda x: torch.cat([y.view(-1, H, dv, dk) for y in x])
    if not back:
        return {"o": rows(o), "final": states(ends)}
    out = {"dq": rows(dq, True), "dk": rows(dk_, True), "dv": rows(dv_), "dld": rows(da).squeeze(-1), "dbeta": rows(db).squeeze(-1)}
    if st["init"] is not None:
        out["dinit"] = states(first)
    return out


def _exact_rotary(case, st):
    """Each pair as a complex number, times scale e^(i angle)."""
    if st["positions"] is not None:
        pos = st["positions"].tolist()
    else:
        off = [0] * (len(st["lens"]) or case["b"]) if st["offsets"] is None else st["offsets"].tolist()
        pos = [p for n, f in zip(st["lens"] or [case["T"]] * case["b"], off) for p in range(f, f + n)]
    pos = torch.tensor(pos, dtype=torch.float64, device=st["q"].device)
    angle = pos[:, None] * st["freq"].double()
    turn = torch.polar(torch.full_like(angle, st["scale"]), -angle if case["op"] == "rot_bwd" else angle)[:, None]
    out = {}
    for n in ("q", "k"):
        x = st[n].double().reshape(-1, *st[n].shape[-2:])
        r, rest = x[..., :case["rot"]], x[..., case["rot"]:]
        pairs = r.unflatten(-1, (2, -1)).transpose(-1, -2) if case["layout"] == "half" else r.unflatten(-1, (-1, 2))
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.transpose(-1, -2).flatten(-2) if case["layout"] == "half" else z.flatten(-2)
        out[n] = torch.cat([z, rest], -1).reshape(st[n].shape)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("fwd", "bwd"):
        return _exact_delta(case, st)
    if case["op"].startswith("rot"):
        return _exact_rotary(case, st)
    rep = case["H"] // case["Hk"]
    state = st["state"].double()
    o = torch.zeros(case["b"], case["H"], case["dv"], dtype=torch.float64, device=state.device)
    for i, s in enumerate(st["slots"].tolist()):
        q, k = (st[n][i].double().repeat_interleave(rep, 0) for n in ("q", "k"))
        S = state[s] * torch.exp(st["ld"][i].double())[:, None, None]
        u = st["beta"][i].double()[:, None] * (st["v"][i].double() - torch.bmm(S, k.unsqueeze(2)).squeeze(2))
        state[s] = S + u.unsqueeze(2) * k.unsqueeze(1)
        o[i] = st["scale"] * torch.bmm(state[s], q.unsqueeze(2)).squeeze(2)
    return {"o": o, "state": state}

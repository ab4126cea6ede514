"""Cases of the gated delta rule (a scan with a matrix state), its single-token
step and the group norm with an activation, in a plain form (elementary torch
operations in 32 bits), as calls of the package, and from the definitions in
64 bits.

Delta rule, per head: u_t = beta_t (v_t - a_t S_{t-1}^T k_t),
S_t = a_t S_{t-1} + k_t u_t^T, o_t = scale S_t^T q_t, a_t = exp(g_t), 0 where
another document starts. Group norm: statistics over one group's channels of
one row, y = act(n w + b), or (n w + b) act(gate)."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
CHUNK = 64  # steps that the plain form takes at once
EPS = 1e-5


def listed():
    return [
        # the smallest training call: the plain fp32 workload's sizes; latency
        dict(name="delta_train_small", op="delta", dtype="f32", B=2, T=16, Nk=1, N=1, Dk=32, Dv=32, reset=False),
        # packed documents, the three heads of 256 of the cluster workload
        dict(name="delta_train_packed", op="delta", dtype="bf16", B=8, T=1024, Nk=3, N=3, Dk=256, Dv=256, reset=True),
        # a training batch of long sequences with many heads
        dict(name="delta_train_large", op="delta", dtype="bf16", B=8, T=4096, Nk=8, N=8, Dk=128, Dv=128, reset=False),
        # one long document of odd length: few heads, a long axis
        dict(name="delta_train_long", op="delta", dtype="bf16", B=1, T=32771, Nk=4, N=4, Dk=128, Dv=128, reset=False),
        # query and key heads shared by three value heads, odd sizes, fp32
        dict(name="delta_train_shared", op="delta", dtype="f32", B=3, T=515, Nk=2, N=6, Dk=40, Dv=72, reset=True),
        # reading prompts of different lengths (one empty) into a state pool: forward only
        dict(name="delta_prefill_ragged", op="prefill", dtype="bf16", B=16, T=2048, Nk=4, N=4, Dk=128, Dv=128),
        # one token for each of many running requests, some rows of the batch unused
        dict(name="delta_step_batch", op="step", dtype="bf16", M=256, P=320, Nk=4, N=8, Dk=128, Dv=128),
        # one token of one request: pure latency
        dict(name="delta_step_one", op="step", dtype="bf16", M=1, P=4, Nk=4, N=4, Dk=192, Dv=192),
        # a scan's output gated head by head, a large training batch
        dict(name="norm_train_large", op="norm", dtype="bf16", rows=65536, groups=8, width=128, gate=True,
             act="silu", centered=False, affine=True, train=True),
        # between the layers of a stack of three heads of 256
        dict(name="norm_train_stack", op="norm", dtype="bf16", rows=8192, groups=3, width=256, gate=False,
             act="silu", centered=True, affine=True, train=True),
        # odd sizes, fp32, few rows
        dict(name="norm_train_odd", op="norm", dtype="f32", rows=37, groups=5, width=83, gate=False, act=None,
             centered=True, affine=True, train=True),
        # one token of one request
        dict(name="norm_one", op="norm", dtype="bf16", rows=1, groups=4, width=192, gate=True, act="silu",
             centered=True, affine=True, train=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    return 16 * rng.randint(1, 16) if rng.random() < 0.6 else _log(rng, 8, 256)


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "prefill", "step", "norm", "norm"])
    if op in ("delta", "prefill", "step"):
        Nk = rng.choice([1, 2, 3, 4])
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), Nk=Nk, N=Nk * rng.choice([1, 1, 2, 3]),
                 Dk=_width(rng), Dv=_width(rng))
        if op == "step":
            c["M"] = _log(rng, 1, max(1, 256 * 8 * 128 * 128 // (c["N"] * c["Dk"] * c["Dv"])))
            c["P"] = c["M"] + rng.randint(1, 64)
            return c
        # tokens, so that the state's products and the plain form's chunk matrices stay below the largest case's
        top = 8 * 4096 * 8 * 128 // (c["N"] * max(c["Dk"], c["Dv"], 64)) // (4 if c["dtype"] == "f32" else 2)
        c["T"] = _log(rng, 1, min(32771, top))
        c["B"] = max(1, min(_log(rng, 1, 32), top // c["T"]))
        if op == "delta":
            c["reset"] = rng.random() < 0.5
        return c
    groups = rng.choice([1, 2, 3, 4, 8, 16])
    width = _log(rng, 16, 4096 // groups) if rng.random() < 0.5 else 16 * _log(rng, 1, 256 // groups)
    return dict(op="norm", dtype=rng.choice(["bf16", "bf16", "f32"]), rows=_log(rng, 1, 30000000 // (groups * width)),
                groups=groups, width=width, gate=rng.random() < 0.5, act=rng.choice([None, "silu", "sigmoid"]),
                centered=rng.random() < 0.5, affine=rng.random() < 0.8, train=rng.random() < 0.7)


# ---- inputs --------------------------------------------------------------------
def _gen(seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    return torch.Generator(device=dev).manual_seed(seed), dev


def _randn(g, dev, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _unit(x, dtype):
    return (x / x.square().sum(-1, keepdim=True).add(1e-6).sqrt()).to(dtype)


def prepare(case, seed):
    g, dev = _gen(seed)
    op, dt = case["op"], DT[case["dtype"]]
    s = dict(case=case)
    if op == "norm":
        rows, G, W = case["rows"], case["groups"], case["width"]
        C = G * W
        # outputs of a scan: heads of different loudness, a mean of their own
        loud = torch.exp(0.5 * _randn(g, dev, (G, 1)))
        s["x"] = ((_randn(g, dev, (rows, G, W)) + 0.5 * _randn(g, dev, (G, 1))) * loud).reshape(rows, C).to(dt)
        s["gate"] = _randn(g, dev, (rows, C), dt) if case["gate"] else None
        s["w"] = (1 + 0.1 * _randn(g, dev, (C,))).to(dt) if case["affine"] else None
        s["b"] = (0.1 * _randn(g, dev, (C,))).to(dt) if case["affine"] else None
        if case["train"]:
            s["dy"] = _randn(g, dev, (rows, C), dt)
            for k in ("x", "gate", "w", "b"):
                if s[k] is not None:
                    s[k].requires_grad_(own)
        return s
    Nk, N, Dk, Dv = (case[k] for k in ("Nk", "N", "Dk", "Dv"))
    lead = (case["M"],) if op == "step" else (case["B"], case["T"])
    s["q"] = _unit(_randn(g, dev, (*lead, Nk, Dk)), dt)
    s["k"] = _unit(_randn(g, dev, (*lead, Nk, Dk)), dt)
    s["v"] = _randn(g, dev, (*lead, N, Dv), dt)
    # each head remembers 2 to 2000 steps, more or less as the token has it
    tau = 2 * torch.exp(torch.rand((N,), generator=g, device=dev) * math.log(1000.0))
    s["g"] = -torch.log1p(torch.exp(_randn(g, dev, (*lead, N)))) / tau
    s["beta"] = 1 / (1 + torch.exp(-_randn(g, dev, (*lead, N))))
    if op == "step":
        M, P = case["M"], case["P"]
        s["pool"] = _randn(g, dev, (P, N, Dk, Dv)) / math.sqrt(Dk)
        s["next"] = s["pool"].clone()
        slots = torch.randperm(P, generator=g, device=dev)[:M].to(torch.int32)
        if M > 4:  # a padded batch: every eighth row is not in use
            slots[::8] = -1
        s["slots"] = slots
        return s
    B, T = lead
    s["state"] = _randn(g, dev, (B, 1, N, Dk, Dv)) / math.sqrt(Dk)
    if op == "prefill":
        n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        n[0] = T
        if B > 1:
            n[1] = 0
        s["lengths"] = n
        return s
    s["do"] = _randn(g, dev, (B, T, N, Dv), dt)
    s["dlast"] = _randn(g, dev, (B, 1, N, Dk, Dv))
    s["reset"] = torch.rand((B, T), generator=g, device=dev) < 1 / 200 if case["reset"] else None
    for k in ("q", "k", "v", "g", "beta", "state"):
        s[k].requires_grad_(own)
    return s


# ---- the package's calls ---------------------------------------------------------
def _run_own(s):
    import recurrent_networks_gb300 as rn
    case = s["case"]
    op = case["op"]
    if op == "delta":
        leaves = [s[k] for k in ("q", "k", "v", "g", "beta", "state")]
        o, last = rn.gated_delta(*leaves, reset=s["reset"])
        return (o.detach(), last.detach()) + torch.autograd.grad((o, last), leaves, (s["do"], s["dlast"]))
    if op == "prefill":
        return rn.gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], lengths=s["lengths"])
    if op == "step":
        o = rn.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], slots=s["slots"],
                                pool_out=s["next"])
        return o, s["next"]
    y = rn.group_norm(s["x"], case["groups"], s["w"], s["b"], gate=s["gate"], activation=case["act"], eps=EPS,
                      centered=case["centered"])
    if not case["train"]:
        return y
    leaves = [s[k] for k in ("x", "gate", "w", "b") if s[k] is not None]
    return (y.detach(),) + torch.autograd.grad(y, leaves, s["dy"])


# ---- the plain form --------------------------------------------------------------
def _heads(x, N):
    """[B, T, Nk, D] -> [B, N, T, D], each head for the N / Nk that share it."""
    B, T, Nk, D = x.shape
    return x[:, :, :, None].expand(B, T, Nk, N // Nk, D).reshape(B, T, N, D).transpose(1, 2)


def _inverse(L):
    """(I + L)^-1 of strictly lower L, [..., C, C]: blocks of doubling size."""
    C = L.shape[-1]
    inv = torch.ones_like(L[..., :1, :1].expand(*L.shape[:-2], C, 1)).reshape(*L.shape[:-2], C, 1, 1)
    n = 1
    while n < C:
        low = torch.stack([L[..., k + n:k + 2 * n, k:k + n] for k in range(0, C, 2 * n)], -3)
        a, d = inv[..., 0::2, :, :], inv[..., 1::2, :, :]
        c = -(d @ low @ a)
        inv = torch.cat([torch.cat([a, torch.zeros_like(a)], -1), torch.cat([c, d], -1)], -2)
        n *= 2
    return inv[..., 0, :, :]


def _delta32(q, k, v, g, beta, state, reset, lengths):
    B, T, N, Dv = v.shape
    Dk = q.shape[-1]
    q, k, v = _heads(q, N), _heads(k, N), v.transpose(1, 2)
    g, beta = g.transpose(1, 2), beta.transpose(1, 2)
    marks = torch.zeros((B, 1, T), dtype=torch.bool, device=v.device) if reset is None else reset[:, None]
    if lengths is not None:
        off = torch.arange(T, device=v.device)[None, None] >= lengths[:, None, None]
        k, v = k.masked_fill(off[..., None], 0), v.masked_fill(off[..., None], 0)
        g, beta = g.masked_fill(off, 0), beta.masked_fill(off, 0)
        marks = marks & ~off
    n = -(-T // CHUNK)
    pad = n * CHUNK - T

    def chunks(x):
        x = torch.cat([x, x.new_zeros((*x.shape[:2], pad, *x.shape[3:]))], 2)
        return x.reshape(*x.shape[:2], n, CHUNK, *x.shape[3:])

    q, k, v, beta = chunks(q), chunks(k), chunks(v), chunks(beta)
    doc = torch.cumsum(chunks(marks.int()), 3)
    c = torch.cumsum(chunks(g.masked_fill(marks, 0)).double(), 3)
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=v.device).tril()
    on = lower & (doc[..., :, None] == doc[..., None, :])
    decay = torch.exp((c[..., :, None] - c[..., None, :]).masked_fill(~on, -math.inf)).float()
    first = torch.exp(c.masked_fill(doc > 0, -math.inf)).float()[..., None]
    rho = torch.exp((c[..., -1:] - c).masked_fill(doc != doc[..., -1:], -math.inf)).float()[..., None]
    P = (q @ k.transpose(-1, -2)) * decay
    inv = _inverse((k @ k.transpose(-1, -2) * decay * beta[..., None, :]).tril(-1))
    S = state[:, 0]
    out = []
    for i in range(n):
        z = inv[:, :, i] @ (v[:, :, i] - first[:, :, i] * (k[:, :, i] @ S))
        u = beta[:, :, i, :, None] * z
        out.append(first[:, :, i] * (q[:, :, i] @ S) + P[:, :, i] @ u)
        S = first[:, :, i, -1:] * S + k[:, :, i].transpose(-1, -2) @ (rho[:, :, i] * u)
    o = torch.cat(out, 2)[:, :, :T].transpose(1, 2) / math.sqrt(Dk)
    if lengths is not None:
        o = o.masked_fill(off.transpose(1, 2)[..., None], 0)
    return o, S[:, None]


def _act32(x, act):
    if act is None:
        return x
    sig = 1 / (1 + torch.exp(-x))
    return x * sig if act == "silu" else sig


def _act_slope32(x, act):
    if act is None:
        return torch.ones_like(x)
    sig = 1 / (1 + torch.exp(-x))
    return sig * (1 + x * (1 - sig)) if act == "silu" else sig * (1 - sig)


def _norm32(s):
    case = s["case"]
    G, W, act = case["groups"], case["width"], case["act"]
    rows, C, dt = case["rows"], G * W, s["x"].dtype
    x = s["x"].float().reshape(rows, G, W)
    if case["centered"]:
        x = x - x.sum(-1, keepdim=True) / W
    r = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / W + EPS)
    n = (x * r).reshape(rows, C)
    w = s["w"].float() if s["w"] is not None else torch.ones(C, device=x.device)
    t = n * w
    if s["b"] is not None:
        t = t + s["b"].float()
    z = s["gate"].float() if s["gate"] is not None else None
    y = (_act32(t, act) if z is None else t * _act32(z, act)).to(dt)
    if not case["train"]:
        return y
    dy = s["dy"].float()
    dt_ = dy * (_act_slope32(t, act) if z is None else _act32(z, act))
    dn = (dt_ * w).reshape(rows, G, W)
    n3 = n.reshape(rows, G, W)
    dx = dn - n3 * ((dn * n3).sum(-1, keepdim=True) / W)
    if case["centered"]:
        dx = dx - dn.sum(-1, keepdim=True) / W
    out = [y, (dx * r).reshape(rows, C).to(dt)]
    if z is not None:
        out.append((dy * t * _act_slope32(z, act)).to(dt))
    if s["w"] is not None:
        out += [(dt_ * n).sum(0).to(dt), dt_.sum(0).to(dt)]
    return tuple(out)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        return _norm32(s)
    if op == "delta":
        names = ("q", "k", "v", "g", "beta", "state")
        with torch.enable_grad():
            leaves = [s[k].detach().float().clone().requires_grad_(True) for k in names]
            o, last = _delta32(*leaves, s["reset"], None)
            grads = torch.autograd.grad((o, last), leaves, (s["do"].float(), s["dlast"]))
        return (o.detach().to(s["v"].dtype), last.detach(), *(d.to(s[k].dtype) for k, d in zip(names, grads)))
    with torch.no_grad():
        if op == "prefill":
            o, last = _delta32(*(s[k].float() for k in ("q", "k", "v", "g", "beta", "state")), None, s["lengths"])
            return o.to(s["v"].dtype), last
        N, P = case["N"], case["P"]
        use = s["slots"] >= 0
        at = s["slots"].clamp(min=0).long()
        q, k = (_heads(s[n].float()[:, None], N)[:, :, 0] for n in ("q", "k"))
        S = s["pool"][at] * torch.exp(s["g"].float())[..., None, None]
        u = s["beta"].float()[..., None] * (s["v"].float() - (k[..., None] * S).sum(-2))
        S = S + k[..., None] * u[..., None, :]
        o = (q[..., None] * S).sum(-2) / math.sqrt(case["Dk"])
        o = torch.where(use[:, None, None], o, torch.zeros_like(o)).to(s["v"].dtype)
        wide = torch.cat([s["next"], torch.zeros_like(s["next"][:1])])
        wide[torch.where(use, at, torch.full_like(at, P))] = S
        s["next"].copy_(wide[:-1])
        return o, s["next"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- from the definitions, in 64 bits --------------------------------------------
def _exact_delta(s, train):
    case = s["case"]
    B, T, Nk, N, Dk, Dv = (case[k] for k in ("B", "T", "Nk", "N", "Dk", "Dv"))
    scale = Dk ** -0.5
    share = N // Nk
    reset, lengths = s.get("reset"), s.get("lengths")

    def rows(name, t):
        """Step t of an input as [B N, width]."""
        x = s[name][:, t].double()
        if name in ("q", "k"):
            x = x.repeat_interleave(share, 1)
        return x.reshape(B * N, -1)

    g = s["g"].double()
    keep = torch.exp(g)
    if reset is not None:
        keep = keep * (~reset)[:, :, None]
    beta = s["beta"].double()
    if lengths is not None:
        live = (torch.arange(T, device=g.device)[None] < lengths[:, None])[:, :, None]
        keep = torch.where(live, keep, torch.ones_like(keep))
        beta = beta * live
    keep, beta = (x.permute(1, 0, 2).reshape(T, B * N, 1).contiguous() for x in (keep, beta))

    def step(S, t):
        """State after step t, the decayed state before it and the error v - S^T k."""
        k = rows("k", t)
        D = S * keep[t][:, :, None]
        e = rows("v", t) - torch.bmm(k[:, None], D)[:, 0]
        return torch.baddbmm(D, k[:, :, None], (beta[t] * e)[:, None]), D, e

    S = s["state"].double().reshape(B * N, Dk, Dv)
    o = torch.empty((T, B * N, Dv), dtype=torch.float64, device=S.device)
    starts = []
    for t in range(T):
        if t % 128 == 0:
            starts.append(S)
        S = step(S, t)[0]
        o[t] = torch.bmm(rows("q", t)[:, None], S)[:, 0]
    last = S.reshape(B, 1, N, Dk, Dv)
    o = (o * scale).reshape(T, B, N, Dv).transpose(0, 1)
    if lengths is not None:
        o = o * live[..., None]
    if not train:
        return o, last
    dS = s["dlast"].double().reshape(B * N, Dk, Dv)
    grads = {n: torch.empty((T, B * N, w), dtype=torch.float64, device=S.device)
             for n, w in (("q", Dk), ("k", Dk), ("v", Dv), ("g", 1), ("beta", 1))}
    for lo in reversed(range(0, T, 128)):
        S = starts.pop()
        trail = []
        for t in range(lo, min(T, lo + 128)):
            S, D, e = step(S, t)
            trail.append((S, D, e))
        for t in reversed(range(lo, min(T, lo + 128))):
            S, D, e = trail.pop()
            q, k, do = rows("q", t), rows("k", t), rows("do", t) * scale
            dS = torch.baddbmm(dS, q[:, :, None], do[:, None])
            grads["q"][t] = torch.bmm(S, do[:, :, None])[:, :, 0]
            du = torch.bmm(k[:, None], dS)[:, 0]
            dv = beta[t] * du
            grads["beta"][t] = (du * e).sum(1, keepdim=True)
            grads["v"][t] = dv
            both = torch.bmm(dS, (beta[t] * e)[:, :, None]) - torch.bmm(D, dv[:, :, None])
            grads["k"][t] = both[:, :, 0]
            dD = torch.baddbmm(dS, k[:, :, None], dv[:, None], alpha=-1)
            grads["g"][t] = (D * dD).sum((1, 2))[:, None]
            dS = dD * keep[t][:, :, None]

    def back(n):
        x = grads[n].reshape(T, B, N, -1).transpose(0, 1)
        if n in ("q", "k"):
            return x.reshape(B, T, Nk, share, Dk).sum(3)
        return x if n == "v" else x[..., 0]

    return (o, last, *(back(n) for n in ("q", "k", "v", "g", "beta")), dS.reshape(B, 1, N, Dk, Dv))


def _exact_norm(s):
    case = s["case"]
    rows, G, W, act = case["rows"], case["groups"], case["width"], case["act"]
    C = G * W
    f = {None: lambda a: (a, torch.ones_like(a)),
         "sigmoid": lambda a: (torch.sigmoid(a), torch.sigmoid(a) * torch.sigmoid(-a)),
         "silu": lambda a: (a * torch.sigmoid(a), torch.sigmoid(a) + a * torch.sigmoid(a) * torch.sigmoid(-a))}[act]
    sums = [torch.zeros(C, dtype=torch.float64, device=s["x"].device) for _ in range(2)]
    parts = []
    for lo in range(0, rows, 8192):
        x = s["x"][lo:lo + 8192].double().unflatten(1, (G, W))
        mean = x.mean(2, keepdim=True) if case["centered"] else torch.zeros_like(x[..., :1])
        var = ((x - mean) ** 2).mean(2, keepdim=True)
        n = (x - mean) / (var + EPS).sqrt()
        w = s["w"].double().view(G, W) if s["w"] is not None else 1.0
        t = n * w + (s["b"].double().view(G, W) if s["b"] is not None else 0.0)
        z = s["gate"][lo:lo + 8192].double().view(t.shape) if s["gate"] is not None else None
        if z is None:
            y, slope = f(t)
        else:
            az, dz = f(z)
            y, slope = t * az, az
        part = [y.flatten(1)]
        if case["train"]:
            dy = s["dy"][lo:lo + 8192].double().view(t.shape)
            dn = dy * slope * w
            dx = dn - n * (dn * n).mean(2, keepdim=True)
            if case["centered"]:
                dx = dx - dn.mean(2, keepdim=True)
            part.append((dx / (var + EPS).sqrt()).flatten(1))
            if z is not None:
                part.append((dy * t * dz).flatten(1))
            sums[0] += (dy * slope * n).sum(0).flatten()
            sums[1] += (dy * slope).sum(0).flatten()
        parts.append(part)
    out = [torch.cat(p) for p in zip(*parts)]
    if not case["train"]:
        return out[0]
    return tuple(out + (sums if s["w"] is not None else []))


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    with torch.no_grad():
        if op == "norm":
            return _exact_norm(s)
        if op in ("delta", "prefill"):
            return _exact_delta(s, op == "delta")
        o = torch.zeros(s["v"].shape, dtype=torch.float64, device=s["v"].device)
        nxt = s["next"].double()
        share = case["N"] // case["Nk"]
        for m, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            k, q = (s[n][m].double().repeat_interleave(share, 0) for n in ("k", "q"))
            S = s["pool"][slot].double() * torch.exp(s["g"][m].double())[:, None, None]
            e = s["v"][m].double() - torch.einsum("nkv,nk->nv", S, k)
            S = S + torch.einsum("nk,nv->nkv", k, s["beta"][m].double()[:, None] * e)
            o[m] = torch.einsum("nkv,nk->nv", S, q) * case["Dk"] ** -0.5
            nxt[slot] = S
        return o, nxt


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    op, e = case["op"], ESIZE[case["dtype"]]
    if op == "norm":
        n = case["rows"] * case["groups"] * case["width"]
        # x, dy in and y, dx out, or x in and y out; the gate in, and its gradient out
        moved = (4 if case["train"] else 2) + ((2 if case["train"] else 1) if case["gate"] else 0)
        return {"bytes": n * e * moved, "flops": n * (30 if case["train"] else 10)}
    Nk, N, Dk, Dv = (case[k] for k in ("Nk", "N", "Dk", "Dv"))
    if op == "step":
        m = case["M"] * (7 / 8 if case["M"] > 4 else 1)
        return {"bytes": m * (N * Dk * Dv * 8 + e * 2 * (Nk * Dk + N * Dv) + 8 * N), "flops": m * N * Dk * Dv * 7}
    n = case["B"] * case["T"]
    ends = case["B"] * N * Dk * Dv * 4
    if op == "prefill":  # half the steps are live on average; o is written everywhere
        return {"bytes": n * (e * (Nk * Dk + N * Dv * 1.5) + 4 * N) + 2 * ends, "flops": n / 2 * N * Dk * Dv * 6}
    # q, k, v, do, g, beta in; o and the gradients out; the state, last and their gradients
    return {"bytes": n * (e * (4 * Nk * Dk + 4 * N * Dv) + 16 * N) + 4 * ends, "flops": n * N * Dk * Dv * 20}

"""Cases of the gated linear scan, the 8-bit activation checkpoints and the
token embedding, in a plain form (elementary torch operations in 32 bits), as
calls of the package, and from the definitions in 64 bits.

Gate order of "linear": i, f, g, o; of "linear_coupled": f, g."""
import math

import numpy as np
import torch

own = False

GATES = {"linear": 4, "linear_coupled": 2}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}
BLOCK = 32   # steps (rows) that share a scale in an 8-bit checkpoint
CHUNK = 128  # steps between the carried states that a training forward keeps


def listed():
    return [
        # the smallest training call: the plain fp32 workload's sizes; latency of two short launches
        dict(name="scan_train_small", op="scan", fn="linear", dtype="f32", B=2, T=16, N=1, D=32, reset=False),
        # packed documents, three heads, the coupled gates
        dict(name="scan_train_packed", op="scan", fn="linear_coupled", dtype="bf16", B=8, T=1024, N=3, D=256,
             reset=True),
        # the benchmark workload's batch, length and width
        dict(name="scan_train_large", op="scan", fn="linear", dtype="bf16", B=32, T=4096, N=1, D=1024, reset=False),
        # one long document of odd length: few channels, a long axis
        dict(name="scan_train_long", op="scan", fn="linear", dtype="bf16", B=1, T=65537, N=4, D=192, reset=False),
        # training with the pre-activations kept in 8 bits, odd length
        dict(name="scan_train_8bit", op="scan8", fn="linear", dtype="bf16", B=8, T=4099, N=4, D=256, reset=False),
        # reading prompts of different lengths (one empty) into a state pool: forward only
        dict(name="scan_prefill_ragged", op="prefill", fn="linear", dtype="bf16", B=16, T=2048, N=4, D=128),
        # one token for each of many running requests, some slots of the batch unused
        dict(name="scan_step_batch", op="step", fn="linear", dtype="bf16", M=256, P=320, N=1, D=1024),
        # one token of one request: pure latency
        dict(name="scan_step_one", op="step", fn="linear_coupled", dtype="bf16", M=1, P=4, N=3, D=256),
        # a projection's training step whose input is kept in 8 bits for dW
        dict(name="proj_train_8bit", op="proj8", B=16, T=2047, I=1024, C=2048),
        # an activation packed to 8 bits and back, a ragged last block of rows
        dict(name="pack_unpack", op="pack", dtype="bf16", rows=65521, cols=1024),
        # a small batch of padded tokens, odd sizes, fp32
        dict(name="embed_train_small", op="embed", dtype="f32", ids="i64", n=74, V=1003, E=200, pad=True),
        # a training batch over a full vocabulary
        dict(name="embed_train_large", op="embed", dtype="bf16", ids="i32", n=131072, V=50000, E=1024, pad=False),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["scan", "scan", "scan8", "prefill", "step", "proj8", "pack", "embed", "embed"])
    if op in ("scan", "scan8", "prefill"):
        fn = rng.choice(["linear", "linear_coupled"])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        N = rng.choice([1, 2, 3, 4, 5])
        D = _log(rng, 17, 1000) if rng.random() < 0.4 else 32 * _log(rng, 1, 32)
        top = 32 * 4096 * 1024 // (2 if dtype == "f32" else 1) // 2
        T = _log(rng, 1, min(65537, top // (N * D)))
        B = max(1, min(_log(rng, 1, 64), top // (T * N * D)))
        c = dict(op=op, fn=fn, dtype=dtype, B=B, T=T, N=N, D=D)
        if op != "prefill":
            c["reset"] = rng.random() < 0.5
        return c
    if op == "step":
        M = _log(rng, 1, 512)
        return dict(op=op, fn=rng.choice(["linear", "linear_coupled"]), dtype=rng.choice(["bf16", "f32"]), M=M,
                    P=M + rng.randint(1, 64), N=rng.choice([1, 2, 3, 4, 5]), D=_log(rng, 17, 1024))
    if op == "proj8":
        return dict(op=op, B=_log(rng, 1, 16), T=_log(rng, 64, 2048), I=8 * _log(rng, 8, 128),
                    C=8 * _log(rng, 8, 256))
    if op == "pack":
        cols = _log(rng, 33, 4096)
        return dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=_log(rng, 1, 100000000 // cols), cols=cols)
    E = _log(rng, 33, 2048)
    return dict(op="embed", dtype=rng.choice(["bf16", "f32"]), ids=rng.choice(["i32", "i64"]),
                n=_log(rng, 1, 150000000 // E if E > 1150 else 131072), V=_log(rng, 100, 131072 if E < 1100 else 60000),
                E=E, pad=rng.random() < 0.5)


# ---- inputs --------------------------------------------------------------------
def _gen(seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    return torch.Generator(device=dev).manual_seed(seed), dev


def _randn(g, dev, shape, dtype):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _bias(g, dev, G, N, D, dtype):
    """N(0, 1) but for the forget gate, whose channels remember 2 to 2000 steps."""
    b = torch.randn((G, N, D), generator=g, device=dev, dtype=torch.float32)
    tau = torch.exp(torch.rand((N, D), generator=g, device=dev) * math.log(1000.0)) * 2
    b[1 if G == 4 else 0] = torch.log(tau - 1)
    return b.to(dtype)


def prepare(case, seed):
    g, dev = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("scan", "scan8", "prefill"):
        B, T, N, D, dt = case["B"], case["T"], case["N"], case["D"], DT[case["dtype"]]
        G = GATES[case["fn"]]
        s["Wx"] = _randn(g, dev, (B, T, G, N, D), dt)
        s["b"] = _bias(g, dev, G, N, D, dt)
        s["state"] = _randn(g, dev, (B, 1, N, D), torch.float32)
        if op == "prefill":
            n = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
            n[0] = T
            if B > 1:
                n[1] = 0
            s["lengths"] = n
        else:
            s["dh"] = _randn(g, dev, (B, T, N, D), dt)
            s["dlast"] = _randn(g, dev, (B, 1, N, D), torch.float32)
            s["reset"] = None
            if case["reset"]:
                s["reset"] = torch.rand((B, T), generator=g, device=dev) < 1 / 200
            for k in ("Wx", "b", "state"):
                s[k].requires_grad_(own)
    elif op == "step":
        M, P, N, D, dt = case["M"], case["P"], case["N"], case["D"], DT[case["dtype"]]
        G = GATES[case["fn"]]
        s["Wx"] = _randn(g, dev, (M, G, N, D), dt)
        s["b"] = _bias(g, dev, G, N, D, dt)
        s["pool"] = _randn(g, dev, (P, N, D), torch.float32)
        s["next"] = s["pool"].clone()
        slots = torch.randperm(P, generator=g, device=dev)[:M].to(torch.int32)
        if M > 4:  # a padded batch: every eighth row is not in use
            slots[::8] = -1
        s["slots"] = slots
    elif op == "proj8":
        B, T, I, C = case["B"], case["T"], case["I"], case["C"]
        s["x"] = _randn(g, dev, (B, T, I), torch.bfloat16)
        s["W"] = (torch.randn((C, I), generator=g, device=dev) / math.sqrt(I)).to(torch.bfloat16)
        s["bias"] = _randn(g, dev, (C,), torch.bfloat16)
        s["dy"] = _randn(g, dev, (B, T, C), torch.bfloat16)
        for k in ("x", "W", "bias"):
            s[k].requires_grad_(own)
    elif op == "pack":
        s["x"] = _randn(g, dev, (case["rows"], case["cols"]), torch.float32)
        s["x"] *= torch.exp(1.5 * torch.randn((case["cols"],), generator=g, device=dev))  # some columns are outliers
        s["x"] = s["x"].to(DT[case["dtype"]])
    else:
        n, V, E, dt = case["n"], case["V"], case["E"], DT[case["dtype"]]
        p = torch.cumsum(_zipf(V).to(dev), 0)
        rank = torch.searchsorted(p, torch.rand((n,), generator=g, device=dev, dtype=torch.float64) * p[-1])
        ids = torch.randperm(V, generator=g, device=dev)[rank.clamp_(max=V - 1)]
        s["pad"] = None
        if case["pad"]:
            s["pad"] = 0
            ids[torch.rand((n,), generator=g, device=dev) < 0.1] = 0
        s["ids"] = ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)
        s["W"] = (torch.randn((V, E), generator=g, device=dev) / math.sqrt(E)).to(dt).requires_grad_(own)
        s["scale"] = math.sqrt(E)
        s["dout"] = _randn(g, dev, (n, E), dt)
    return s


def _zipf(V):
    return 1.0 / (torch.arange(V, dtype=torch.float64) + 2.7)


# ---- the package's calls ---------------------------------------------------------
def _run_own(s):
    import recurrent_networks_gb300 as rn
    case = s["case"]
    op = case["op"]
    if op in ("scan", "scan8"):
        h, last = rn.gated_scan(s["Wx"], s["b"], s["state"], function=case["fn"], reset=s["reset"],
                                checkpoint="int8" if op == "scan8" else None)
        dWx, db, ds = torch.autograd.grad((h, last), (s["Wx"], s["b"], s["state"]), (s["dh"], s["dlast"]))
        return h.detach(), last.detach(), dWx, db, ds
    if op == "prefill":
        return rn.gated_scan(s["Wx"], s["b"], s["state"], function=case["fn"], lengths=s["lengths"])
    if op == "step":
        h = rn.gated_scan_step(s["Wx"], s["b"], s["pool"], slots=s["slots"], function=case["fn"], pool_out=s["next"])
        return h, s["next"]
    if op == "proj8":
        y = rn.input_projection(s["x"], s["W"], s["bias"], checkpoint="int8")
        dx, dW, db = torch.autograd.grad(y, (s["x"], s["W"], s["bias"]), s["dy"])
        return y.detach(), dx, dW, db
    if op == "pack":
        q, scales = rn.checkpoint_pack(s["x"])
        return rn.checkpoint_unpack(q, scales, s["x"].dtype)
    out = rn.embedding(s["ids"], s["W"], scale=s["scale"], padding_idx=s["pad"])
    (dW,) = torch.autograd.grad(out, (s["W"],), s["dout"])
    return out.detach(), dW


# ---- the plain form --------------------------------------------------------------
def _scan32(f, u, c0):
    """c_t = f_t c_{t-1} + u_t along the second axis, by doubling."""
    n, k = f.shape[1], 1
    while k < n:
        u = torch.cat([u[:, :k], u[:, k:] + f[:, k:] * u[:, :-k]], 1)
        f = torch.cat([f[:, :k], f[:, k:] * f[:, :-k]], 1)
        k *= 2
    return u + f * c0


def _sig(x):
    return 1 / (1 + torch.exp(-x))


def _pack32(x):
    """x [batch, rows, cols] in 32 bits -> the values its 8-bit checkpoint stands for."""
    n, rows, cols = x.shape
    pad = -rows % BLOCK
    v = torch.cat([x, x.new_zeros(n, pad, cols)], 1).reshape(n, -1, BLOCK, cols)
    m, ex = torch.frexp(v.abs().amax(2, keepdim=True))
    e = torch.where(m <= 127 / 128, ex - 7, ex - 6).clamp(min=-126)
    q = torch.round(torch.ldexp(v, -e))
    return torch.ldexp(q, e).reshape(n, -1, cols)[:, :rows]


def _gates32(a, fn):
    """Pre-activations [B, T, G, C] -> (f, u) of the recurrence, and the gates."""
    if fn == "linear":
        i, f, g, o = _sig(a[:, :, 0]), _sig(a[:, :, 1]), a[:, :, 2], _sig(a[:, :, 3])
        return f, i * g, (i, f, g, o)
    f, g = _sig(a[:, :, 0]), a[:, :, 1]
    return f, _sig(-a[:, :, 0]) * g, (f, g)


def _run_scan(s, eight, train):
    case, fn = s["case"], s["case"]["fn"]
    B, T, N, D = (case[k] for k in "BTND")
    C, G = N * D, GATES[fn]
    dt = s["Wx"].dtype
    x = s["Wx"].float().reshape(B, T, G, C)
    bias = s["b"].float().reshape(G, C)
    f, u, gates = _gates32(x + bias, fn)
    live = None
    if train and s["reset"] is not None:
        f = f.masked_fill(s["reset"][:, :, None], 0)
    if not train:
        live = torch.arange(T, device=x.device)[None] < s["lengths"][:, None]
        f = torch.where(live[:, :, None], f, torch.ones_like(f))
        u = torch.where(live[:, :, None], u, torch.zeros_like(u))
    c0 = s["state"].float().reshape(B, 1, C)
    c = _scan32(f, u, c0)
    last = c[:, -1:].reshape(B, 1, N, D)
    h = gates[3] * c if fn == "linear" else c
    if live is not None:
        h = torch.where(live[:, :, None], h, torch.zeros_like(h))
    h = h.reshape(B, T, N, D).to(dt)
    if not train:
        return h, last
    cprev = torch.cat([c0, c[:, :-1]], 1)
    if eight:
        x = _pack32(x.reshape(B, T, G * C)).reshape(B, T, G, C)
        f, u, gates = _gates32(x + bias, fn)
        if s["reset"] is not None:
            f = f.masked_fill(s["reset"][:, :, None], 0)
        nc = -(-T // CHUNK)
        start = cprev[:, ::CHUNK].reshape(B * nc, 1, C)
        pad = nc * CHUNK - T
        fp = torch.cat([f, f.new_zeros(B, pad, C)], 1).reshape(B * nc, CHUNK, C)
        up = torch.cat([u, u.new_zeros(B, pad, C)], 1).reshape(B * nc, CHUNK, C)
        c = _scan32(fp, up, start)
        cprev = torch.cat([start, c[:, :-1]], 1).reshape(B, -1, C)[:, :T]
        c = c.reshape(B, -1, C)[:, :T]
    if s["reset"] is not None:
        cprev = cprev.masked_fill(s["reset"][:, :, None], 0)
    dh = s["dh"].float().reshape(B, T, C)
    e = dh * gates[3] if fn == "linear" else dh
    fr = torch.cat([torch.ones_like(f[:, :1]), f.flip(1)[:, :-1]], 1)
    delta = _scan32(fr, e.flip(1), s["dlast"].float().reshape(B, 1, C)).flip(1)
    if fn == "linear":
        i, fg, g, o = gates
        da = torch.stack([delta * g * i * (1 - i), delta * cprev * fg * (1 - fg), delta * i, dh * c * o * (1 - o)], 2)
    else:
        fg, g = gates
        nf = _sig(-(x[:, :, 0] + bias[0]))
        da = torch.stack([delta * (cprev - g) * fg * nf, delta * nf], 2)
    ds = (f[:, :1] * delta[:, :1]).reshape(B, 1, N, D)
    db = da.sum((0, 1)).reshape(G, N, D).to(dt)
    return h, last, da.reshape(B, T, G, N, D).to(dt), db, ds


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op in ("scan", "scan8", "prefill"):
        return _run_scan(s, op == "scan8", op != "prefill")
    if op == "step":
        M, N, D = case["M"], case["N"], case["D"]
        a = (s["Wx"].float() + s["b"].float()).reshape(M, 1, -1, N * D)
        f, u, gates = _gates32(a, case["fn"])
        use = (s["slots"] >= 0)[:, None]
        at = s["slots"].clamp(min=0).long()
        c = f[:, 0] * s["pool"][at].reshape(M, -1) + u[:, 0]
        h = gates[3][:, 0] * c if case["fn"] == "linear" else c
        h = torch.where(use, h, torch.zeros_like(h)).reshape(M, N, D).to(s["Wx"].dtype)
        at = torch.where(s["slots"] >= 0, at, torch.full_like(at, case["P"]))
        wide = torch.cat([s["next"], torch.zeros_like(s["next"][:1])])
        wide[at] = c.reshape(M, N, D)
        s["next"].copy_(wide[:-1])
        return h, s["next"]
    if op == "proj8":
        x = s["x"].float().reshape(-1, case["I"])
        W, dy = s["W"].float(), s["dy"].float().reshape(-1, case["C"])
        y = (x @ W.T + s["bias"].float()).to(torch.bfloat16)
        dx = (dy @ W).to(torch.bfloat16)
        dW = (dy.T @ _pack32(x[None])[0]).to(torch.bfloat16)
        return y.reshape(s["dy"].shape), dx.reshape(s["x"].shape), dW, dy.sum(0).to(torch.bfloat16)
    if op == "pack":
        return _pack32(s["x"].float()[None])[0].to(s["x"].dtype)
    dt = s["W"].dtype
    ids = s["ids"].long()
    out = (s["W"][ids].float() * s["scale"]).to(dt)
    d = s["dout"].float() * s["scale"]
    if s["pad"] is not None:
        d = d.masked_fill((ids == s["pad"])[:, None], 0)
    dW = torch.zeros(s["W"].shape, device=d.device).index_add_(0, ids, d).to(dt)
    return out, dW


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- from the definitions, in 64 bits --------------------------------------------
def _e8(x):
    """The values an 8-bit checkpoint of x [rows, cols] (64 bits) stands for."""
    out = torch.empty_like(x)
    whole = x.shape[0] // BLOCK * BLOCK
    for lo, hi, rows in ((0, whole, BLOCK), (whole, x.shape[0], x.shape[0] - whole)):
        if lo == hi:
            continue
        v = x[lo:hi].reshape(-1, rows, x.shape[1])
        top = v.abs().max(1, keepdim=True).values
        step = torch.exp2(torch.ceil(torch.log2(top / 127)).clamp(min=-126))
        step = torch.where(top <= 127 * step / 2, step / 2, step)  # log2 rounds: the smallest that holds
        step = torch.where(top > 127 * step, step * 2, step).clamp(min=2.0 ** -126)
        out[lo:hi] = (torch.round(v / step) * step).reshape(-1, x.shape[1])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    s = {k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in s.items()}
    op = case["op"]
    if op in ("scan", "scan8", "prefill"):
        fn, N, D = case["fn"], case["N"], case["D"]
        B, T = case["B"], case["T"]
        C, G = N * D, GATES[fn]
        bias = s["b"].double().reshape(G, C)
        raw = s["Wx"].reshape(B, T, G, C)
        lens, reset = s.get("lengths"), s.get("reset")

        def part(x, lo):
            """Gates of the steps from lo on: f as it carries the state, u, and all of them."""
            z = x.double() + bias
            if fn == "linear":
                i, f, g, o = torch.sigmoid(z[:, :, 0]), torch.sigmoid(z[:, :, 1]), z[:, :, 2], torch.sigmoid(z[:, :, 3])
                u, gates = i * g, (i, f, g, o)
            else:
                f, g, nf = torch.sigmoid(z[:, :, 0]), z[:, :, 1], torch.sigmoid(-z[:, :, 0])
                u, gates = nf * g, (f, g, nf)
            keep = f
            if reset is not None:
                keep = f * (~reset[:, lo:lo + f.shape[1], None]).double()
            if lens is not None:
                off = (torch.arange(lo, lo + f.shape[1], device=f.device)[None] >= lens[:, None])[:, :, None]
                keep, u = keep.masked_fill(off, 1.0), u.masked_fill(off, 0.0)
            return keep, u, gates

        def follow(keep, u, c):
            """States before and after each step."""
            prev, after = torch.empty_like(u), torch.empty_like(u)
            for t in range(u.shape[1]):
                prev[:, t] = c
                c = torch.addcmul(u[:, t], keep[:, t], c)
                after[:, t] = c
            return prev, after, c

        c = s["state"].double().reshape(B, C)
        h = torch.zeros((B, T, C), dtype=torch.float64, device=c.device)
        starts = []
        for lo in range(0, T, CHUNK):
            starts.append(c)
            keep, u, gates = part(raw[:, lo:lo + CHUNK], lo)
            _, after, c = follow(keep, u, c)
            h[:, lo:lo + CHUNK] = gates[3] * after if fn == "linear" else after
        if lens is not None:
            h *= (torch.arange(T, device=h.device)[None] < lens[:, None])[:, :, None]
        last = c.reshape(B, 1, N, D)
        h = h.reshape(B, T, N, D)
        if op == "prefill":
            return h, last
        x = raw
        if op == "scan8":
            x = s["Wx"].double().reshape(B, T, G * C)
            x = torch.stack([_e8(x[b]) for b in range(B)]).reshape(B, T, G, C)
        d = s["dlast"].double().reshape(B, C)
        da = torch.empty((B, T, G, C), dtype=torch.float64, device=c.device)
        for lo in reversed(range(0, T, CHUNK)):
            keep, u, gates = part(x[:, lo:lo + CHUNK], lo)
            prev, after, _ = follow(keep, u, starts[lo // CHUNK])
            if reset is not None:
                prev = prev * (~reset[:, lo:lo + CHUNK, None]).double()
            dh = s["dh"][:, lo:lo + CHUNK].double().reshape(after.shape)
            e = dh * gates[3] if fn == "linear" else dh
            delta = torch.empty_like(e)
            for t in reversed(range(e.shape[1])):
                delta[:, t] = e[:, t] + d
                d = keep[:, t] * delta[:, t]
            if fn == "linear":
                i, f, g, o = gates
                parts = (delta * g * i * (1 - i), delta * prev * f * (1 - f), delta * i, dh * after * o * (1 - o))
            else:
                f, g, nf = gates
                parts = (delta * (prev - g) * f * nf, delta * nf)
            da[:, lo:lo + CHUNK] = torch.stack(parts, 2)
        return h, last, da.reshape(B, T, G, N, D), da.sum((0, 1)).reshape(G, N, D), d.reshape(B, 1, N, D)
    if op == "step":
        h = torch.zeros((case["M"], case["N"], case["D"]), dtype=torch.float64, device=s["Wx"].device)
        nxt = s["next"].double()
        for m, slot in enumerate(s["slots"].tolist()):
            if slot < 0:
                continue
            z = s["Wx"][m].double() + s["b"].double()
            c = s["pool"][slot].double()
            if case["fn"] == "linear":
                c = torch.sigmoid(z[1]) * c + torch.sigmoid(z[0]) * z[2]
                h[m] = torch.sigmoid(z[3]) * c
            else:
                c = torch.sigmoid(z[0]) * c + torch.sigmoid(-z[0]) * z[1]
                h[m] = c
            nxt[slot] = c
        return h, nxt
    if op == "proj8":
        x = s["x"].double().flatten(0, 1)
        W, dy = s["W"].double(), s["dy"].double().flatten(0, 1)
        y = torch.matmul(x, W.t()) + s["bias"].double()
        return (y.view(s["dy"].shape), torch.matmul(dy, W).view(s["x"].shape), torch.matmul(dy.t(), _e8(x)),
                dy.sum(0))
    if op == "pack":
        return _e8(s["x"].double())
    W = s["W"].double()
    ids = s["ids"].long()
    out = W.index_select(0, ids) * s["scale"]
    d = s["dout"].double()
    if s["pad"] is not None:
        d[ids == s["pad"]] = 0
    dW = torch.zeros_like(W)
    dW.index_put_((ids,), d, accumulate=True)
    return out, dW * s["scale"]


# ---- what a pass cannot do without --------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("scan", "scan8", "prefill"):
        e = ESIZE[case["dtype"]]
        G = GATES[case["fn"]]
        n = case["B"] * case["T"] * case["N"] * case["D"]
        ends = case["B"] * case["N"] * case["D"] * 4
        if op == "prefill":  # half the steps are live on average
            return {"bytes": n * e * (G / 2 + 1) + 2 * ends, "flops": n * 6 * G / 2}
        # Wx and dh in, h and dWx out
        return {"bytes": n * e * (2 * G + 2) + 4 * ends, "flops": n * 20 * G}
    if op == "step":
        G = GATES[case["fn"]]
        n = case["M"] * case["N"] * case["D"]
        return {"bytes": n * (ESIZE[case["dtype"]] * (G + 1) + 8), "flops": n * 6 * G}
    if op == "proj8":
        bt, i, c = case["B"] * case["T"], case["I"], case["C"]
        return {"bytes": 2 * (2 * bt * i + 2 * bt * c + 2 * i * c), "flops": 6 * bt * i * c}
    if op == "pack":
        n = case["rows"] * case["cols"]
        return {"bytes": 2 * n * ESIZE[case["dtype"]], "flops": 4 * n}
    p = _zipf(case["V"]).numpy()
    rows = float(np.sum(-np.expm1(case["n"] * np.log1p(-p / p.sum()))))  # distinct tokens, on average
    e = ESIZE[case["dtype"]]
    return {"bytes": e * case["E"] * (rows + 2 * case["n"] + case["V"]), "flops": 2 * case["n"] * case["E"]}

"""The functional entry point, shaped like the FlashRNN announcement's usage
example (hottg.com/neural/9889): ``states, last = flashrnn(Wx, R, b, states=...,
function=..., backend=...)`` with no parameters bound to the function.

PyTorch provides memory, streams and autograd bookkeeping only; the forward and
the backward through time run in librnn_gb300.so's kernels via the C ABI.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib

BACKENDS = {"auto": "auto", "cuda_fused": "fused", "fused": "fused", "cuda": "alternating",
            "alternating": "alternating", "simt": "simt", "grid": "grid"}


def _on_gpu(t, name):
    if not t.is_cuda:
        raise RuntimeError(f"{name} runs on CUDA tensors only (there is no CPU path)")


def _dims(Wx, R, function, backend):
    B, T, G, N, D = Wx.shape
    if G != _lib.rnn_num_gates(function):
        raise ValueError(f"{function} needs G={_lib.rnn_num_gates(function)} gates, Wx has {G}")
    if tuple(R.shape) != (G, N, D, D):
        raise ValueError(f"R must be [G,N,D,D]={(G, N, D, D)}, got {tuple(R.shape)}")
    if Wx.dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {Wx.dtype}")
    return _lib.make_dims(B, T, N, D, function, Wx.dtype, BACKENDS[backend])


def _ws(dims, kind, device):
    n = _lib.rnn_workspace_size(dims, kind)
    return torch.empty(n, dtype=torch.uint8, device=device)


class _ScanFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Wx, R, b, states0, function, backend):
        dims = _dims(Wx, R, function, backend)
        S = _lib.rnn_num_states(function)
        B, T, G, N, D = Wx.shape
        Wx, R, b = Wx.contiguous(), R.contiguous(), b.contiguous()
        s0 = states0.contiguous() if states0 is not None else None
        states = torch.empty((S, B, T, N, D), dtype=Wx.dtype, device=Wx.device)
        last = torch.empty((S, B, 1, N, D), dtype=Wx.dtype, device=Wx.device)
        need_grad = any(ctx.needs_input_grad[:4])
        tape = torch.empty(_lib.rnn_tape_size(dims), dtype=torch.uint8, device=Wx.device) if need_grad else None
        ws = _ws(dims, _lib.WS_FWD, Wx.device)
        _lib.rnn_fwd(dims, Wx, R, b, s0, states, last, tape, ws)
        ctx.dims = dims
        ctx.has_s0 = s0 is not None
        ctx.save_for_backward(Wx, R, b, s0, states, tape)
        return states, last

    @staticmethod
    def backward(ctx, dstates, dlast):
        Wx, R, b, s0, states, tape = ctx.saved_tensors
        dims = ctx.dims
        dstates = dstates.contiguous() if dstates is not None else None
        dlast = dlast.contiguous() if dlast is not None else None
        dWx = torch.empty_like(Wx) if ctx.needs_input_grad[0] else None
        dR = torch.empty_like(R) if ctx.needs_input_grad[1] else None
        db = torch.empty_like(b) if ctx.needs_input_grad[2] else None
        ds0 = torch.empty_like(s0) if (ctx.has_s0 and ctx.needs_input_grad[3]) else None
        ws = _ws(dims, _lib.WS_BWD, Wx.device)
        _lib.rnn_bwd(dims, Wx, R, b, s0, states, tape, dstates, dlast, dWx, dR, db, ds0, ws)
        return dWx, dR, db, ds0, None, None


def flashrnn(Wx, R, b, states=None, function: str = "lstm", backend: str = "auto"):
    """Head-wise recurrent scan. Wx [B,T,G,N,D], R [G,N,D,D], b [G,N,D],
    states [S,B,1,N,D] or None (zeros). Returns (states [S,B,T,N,D], last
    [S,B,1,N,D]). function: lstm | gru | elman | slstm. backend: auto |
    cuda_fused (fused) | cuda (alternating) | simt."""
    _on_gpu(Wx, "flashrnn")
    _lib.check_device(Wx)
    return _ScanFn.apply(Wx, R, b, states, function, backend)


class _ProjFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, W, bias, checkpoint=None):
        BT, I = x.shape
        C = W.shape[0]
        x, W = x.contiguous(), W.contiguous()
        bias = bias.contiguous() if bias is not None else None
        Wx = torch.empty((BT, C), dtype=x.dtype, device=x.device)
        ws = torch.empty(_lib.rnn_input_proj_workspace_size(BT, I, C), dtype=torch.uint8, device=x.device)
        _lib.rnn_input_proj_fwd(BT, I, C, x, W, bias, Wx, ws)
        ctx.has_bias = bias is not None
        ctx.packed = checkpoint == "int8"
        if ctx.packed:  # x is needed for dW alone
            ctx.save_for_backward(W, *(_pack(x) if ctx.needs_input_grad[1] else ()))
        else:
            ctx.save_for_backward(x, W)
        return Wx

    @staticmethod
    def backward(ctx, dWx):
        if ctx.packed:
            W, *kept = ctx.saved_tensors
            x = torch.empty((dWx.shape[0], W.shape[1]), dtype=W.dtype, device=W.device)
            if kept:
                _lib.rnn_act_unpack(x.shape[0], x.shape[1], kept[0], kept[1], x)
        else:
            x, W = ctx.saved_tensors
        BT, I = x.shape
        C = W.shape[0]
        dWx = dWx.contiguous()
        dx = torch.empty_like(x) if ctx.needs_input_grad[0] else None
        dW = torch.empty_like(W) if ctx.needs_input_grad[1] else None
        db = torch.empty((C,), dtype=x.dtype, device=x.device) if (ctx.has_bias and ctx.needs_input_grad[2]) else None
        ws = torch.empty(_lib.rnn_input_proj_workspace_size(BT, I, C), dtype=torch.uint8, device=x.device)
        _lib.rnn_input_proj_bwd(BT, I, C, x, W, dWx, dx, dW, db, ws)
        return dx, dW, db, None


def input_projection(x, W, bias=None, checkpoint=None):
    """Wx = x W^T (+ bias) on the tensor cores: x [..., I], W [C, I] (the
    weight_ih layout), bias [C] or None; returns [..., C]. bf16, CUDA only.
    checkpoint="int8" keeps x for the backward in 8 bits (checkpoint_pack over
    the flattened rows) instead of x itself: dW is then taken at the unpacked
    values; the result, dx and dbias are unchanged."""
    _on_gpu(x, "input_projection")
    _lib.check_device(x)
    if checkpoint not in _lib.CHECKPOINTS:
        raise ValueError(f"checkpoint must be one of {list(_lib.CHECKPOINTS)}, got {checkpoint!r}")
    if not torch.is_grad_enabled():  # no backward to come, nothing to keep
        checkpoint = None
    lead = x.shape[:-1]
    y = _ProjFn.apply(x.reshape(-1, x.shape[-1]), W, bias, checkpoint)
    return y.reshape(*lead, W.shape[0])


def flashrnn_stack(x, layers, function: str = "lstm", backend: str = "auto"):
    """Stacked layers: layer l projects its input (x for l = 0, the previous
    layer's h, [B, T, N*D], otherwise) with W_x [G*N*D, I_l] (+ bias_x) and
    runs the head-wise scan with R, b and initial states (or zeros).
    layers: sequence of dicts with keys W_x, bias_x (optional), R, b, states
    (optional) and norm (optional: a dict of group_norm's weight, bias,
    activation, eps and centered, with which the layer's h leaves it, normalised
    head by head). Returns (h of the last layer [B, T, N*D], [(states, last) of
    every layer]). Differentiable end to end (autograd chains the kernels'
    backward passes)."""
    B, T = x.shape[0], x.shape[1]
    h = x
    outs = []
    for layer in layers:
        R = layer["R"]
        G, N, D = R.shape[0], R.shape[1], R.shape[2]
        Wx = input_projection(h, layer["W_x"], layer.get("bias_x")).reshape(B, T, G, N, D)
        states, last = flashrnn(Wx, R, layer["b"], layer.get("states"), function, backend)
        outs.append((states, last))
        h = states[0].reshape(B, T, N * D)
        if layer.get("norm") is not None:
            h = group_norm(h, N, **layer["norm"])
    return h, outs


# ---- gated linear scan ------------------------------------------------------------
def _check_status(status, t):
    """The kernels write to the status word, so it has to be one that they can."""
    if status is None:
        return
    if status.dtype != torch.int32:
        raise TypeError(f"status must be int32, got {status.dtype}")
    if status.numel() < 1 or status.get_device() != t.get_device():
        raise ValueError(f"status must be an element on cuda:{t.get_device()}, got shape {tuple(status.shape)} "
                         f"on {status.device}")


def _any_dual(*tensors):
    if getattr(forward_ad, "_current_level", 0) < 0:  # no dual level is open (asking each tensor costs more)
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _tracked(*tensors):
    """Whether autograd has to see a call on these tensors (None: absent): for a
    gradient, or to refuse a forward-mode tangent, which the call would drop."""
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return _any_dual(*tensors)


def _first_order(*grads):
    """Refuses forward over reverse: the gradients' kernels would drop the tangent."""
    if _any_dual(*grads):
        raise NotImplementedError("the backward has no forward-mode derivative")


def _dense(t):
    """t (or None) as the library takes it: contiguous and 16-byte aligned."""
    if t is None or (t.is_contiguous() and t.data_ptr() % 16 == 0):
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _workspace(size, t, status):
    """Workspace on t's device: the kept word where the call needs no more than a
    status word and nobody asks for it."""
    if size <= 256 and status is None:
        return _lib.status_word(t)
    return torch.empty(size, dtype=torch.uint8, device=t.device)


def _add_status(status, workspace):
    """What the kernels running on the workspace report, added to the caller's word."""
    if status is not None:
        status.as_strided((1,), (1,)).bitwise_or_(workspace[:4].view(torch.int32))


def _gated_run(Wx, b, state, function, reset, lengths, checkpoint, status, keep):
    """(h, last, Wx and b as the library took them, plan, tape or None)."""
    B, T, _, N, D = Wx.shape
    plan = _lib.gated_plan(B, T, N, D, function, Wx.dtype, checkpoint, _lib.check_device(Wx))
    Wx, b, state = _dense(Wx), _dense(b), _dense(state)
    h = Wx.new_empty((B, T, N, D))
    last = torch.empty((B, 1, N, D), dtype=torch.float32, device=h.device)
    dims, size, fwd, _ = plan
    tape = torch.empty(size, dtype=torch.uint8, device=h.device) if keep else None
    ws = _workspace(fwd, h, status)
    _lib.rnn_gated_fwd(dims, Wx, b, state, reset, lengths, h, last, tape, ws)
    _add_status(status, ws)
    return h, last, Wx, b, plan, tape


class _GatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Wx, b, state, function, reset, lengths, checkpoint, status):
        h, last, Wx, b, ctx.plan, tape = _gated_run(Wx, b, state, function, reset, lengths, checkpoint, status, True)
        ctx.status = status
        ctx.shape = Wx.shape
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(Wx if checkpoint is None else None, b, reset, lengths, tape)
        return h, last

    @staticmethod
    def backward(ctx, dh, dlast):
        return (_gated_bwd_once if torch.is_grad_enabled() else _gated_bwd)(ctx, dh, dlast)


def _gated_bwd(ctx, dh, dlast):
    _first_order(dh, dlast)
    Wx, b, reset, lengths, tape = ctx.saved_tensors
    dims, _, _, size = ctx.plan
    B, _, G, N, D = ctx.shape
    need = ctx.needs_input_grad
    dtype = torch.bfloat16 if dims.dtype == _lib.DTYPES[torch.bfloat16] else torch.float32
    dWx = torch.empty(ctx.shape, dtype=dtype, device=tape.device) if need[0] else None
    db = torch.empty((G, N, D), dtype=dtype, device=tape.device) if need[1] else None
    ds = torch.empty((B, 1, N, D), dtype=torch.float32, device=tape.device) if need[2] else None
    ws = _workspace(size, tape, ctx.status)
    _lib.rnn_gated_bwd(dims, Wx, b, reset, lengths, tape, _dense(dh), _dense(dlast), dWx, db, ds, ws)
    _add_status(ctx.status, ws)
    return dWx, db, ds, None, None, None, None, None


_gated_bwd_once = once_differentiable(_gated_bwd)


def _gated_shapes(Wx, b, function, lead):
    shape, dtype = Wx.shape, Wx.dtype
    if function not in _lib.GATED_FUNCTIONS:
        raise ValueError(f"function must be one of {list(_lib.GATED_FUNCTIONS)}, got {function!r}")
    if dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if len(shape) != lead + 3:
        raise ValueError(f"Wx must have {lead + 3} dimensions, got shape {tuple(shape)}")
    G, N, D = shape[lead:]
    want = 4 if function == "linear" else 2
    if G != want:
        raise ValueError(f"{function} needs G={want} gates, Wx has {G}")
    if b is not None:
        if b.shape != (G, N, D):
            raise ValueError(f"b must be [G,N,D]={(G, N, D)}, got {tuple(b.shape)}")
        if b.dtype != dtype:
            raise TypeError(f"b is {b.dtype}, Wx is {dtype}")
        if b.get_device() != Wx.get_device():
            raise ValueError("b must be on Wx's device")
    return N, D


def _marks(reset, lengths, B, T, t, name):
    """reset and lengths as the library takes them, beside the tensor t called `name`."""
    if reset is not None:
        if reset.shape != (B, T):
            raise ValueError(f"reset must be [B,T]={(B, T)}, got {tuple(reset.shape)}")
        if reset.dtype not in (torch.bool, torch.uint8):
            raise TypeError(f"reset must be bool or uint8, got {reset.dtype}")
        if reset.device != t.device:
            raise ValueError(f"reset must be on {name}'s device")
        reset = reset.contiguous()
    if lengths is not None:
        if lengths.shape != (B,):
            raise ValueError(f"lengths must be [B]={(B,)}, got {tuple(lengths.shape)}")
        if lengths.dtype not in (torch.int32, torch.int64):
            raise TypeError(f"lengths must be integers, got {lengths.dtype}")
        if lengths.device != t.device:
            raise ValueError(f"lengths must be on {name}'s device")
        if lengths.dtype == torch.int64:
            lengths = lengths.clamp(0, T).to(torch.int32)
        lengths = lengths.contiguous()
    return reset, lengths


def _check_pool(pools, slots, M, shape, names, t, name):
    """The state pools ([P, *shape] fp32) and slots of M rows, beside the tensor t called `name`."""
    dev = t.get_device()
    for p in pools:
        if p.dtype != torch.float32:
            raise TypeError(f"the pool must be float32, got {p.dtype}")
        if p.dim() != len(shape) + 1 or p.shape != (pools[0].shape[0], *shape):
            raise ValueError(f"the pool must be [P,{names}]=[P,{','.join(map(str, shape))}], got {tuple(p.shape)}")
        if not p.is_contiguous() or p.data_ptr() % 16 or p.get_device() != dev:
            raise ValueError(f"the pool must be contiguous, 16-byte aligned and on {name}'s device")
    P = pools[0].shape[0]
    if len(pools) == 2 and 0 < abs(pools[0].data_ptr() - pools[1].data_ptr()) < 4 * pools[0].numel():
        raise ValueError("pool_out must be the pool itself or share no memory with it")
    if slots is None:
        if M > P:
            raise ValueError(f"{M} rows need as many slots, the pool has {P}")
    elif slots.shape != (M,) or slots.dtype != torch.int32 or slots.get_device() != dev:
        raise ValueError(f"slots must be [M]=[{M}] int32 on {name}'s device")
    return P


def gated_scan(Wx, b=None, state=None, function: str = "linear", reset=None, lengths=None, checkpoint=None, status=None):
    """Gated linear scan: the recurrence without R, linear in its state.

    Wx [B,T,G,N,D] (bf16 or fp32), b [G,N,D] or None, state [B,1,N,D] or None
    (zeros). function "linear" (gates i, f, g, o): c_t = s(f) c_{t-1} + s(i) g,
    h_t = s(o) c_t; "linear_coupled" (gates f, g): h_t = c_t = s(f) c_{t-1} +
    (1 - s(f)) g, s the sigmoid of the biased pre-activation. reset [B,T] (bool
    or uint8): c_{t-1} counts as zero at the marked steps (packed documents).
    lengths [B]: row b has lengths[b] steps; past them h is zero and the state
    is kept. Returns (h [B,T,N,D], last [B,1,N,D]: the state after the last
    step, fp32). Differentiable in Wx, b and state; the backward recomputes the
    states from those kept every 128 steps. checkpoint="int8" keeps Wx for the
    backward in 8 bits (a power-of-two scale per 32 steps of a channel and
    gate) instead of Wx itself; the gradient is then taken at those values.
    status: an int32 CUDA tensor of one element, zeroed by the caller, in which
    the forward and the backward record a device-side wait that ran out (their
    results are then not valid); _lib.rnn_check_status(status) raises for it."""
    _on_gpu(Wx, "gated_scan")
    N, D = _gated_shapes(Wx, b, function, 2)
    B, T = Wx.shape[:2]
    if checkpoint not in _lib.CHECKPOINTS:
        raise ValueError(f"checkpoint must be one of {list(_lib.CHECKPOINTS)}, got {checkpoint!r}")
    _check_status(status, Wx)
    if state is not None:
        if state.shape != (B, 1, N, D):
            raise ValueError(f"state must be [B,1,N,D]={(B, 1, N, D)}, got {tuple(state.shape)}")
        if state.get_device() != Wx.get_device():
            raise ValueError("state must be on Wx's device")
        if state.dtype != torch.float32:
            state = state.float()
    reset, lengths = _marks(reset, lengths, B, T, Wx, "Wx")
    if _tracked(Wx, b, state):
        return _GatedFn.apply(Wx, b, state, function, reset, lengths, checkpoint, status)
    return _gated_run(Wx, b, state, function, reset, lengths, checkpoint, status, False)[:2]


def gated_scan_step(Wx, b, pool, slots=None, function: str = "linear", pool_out=None, status=None):
    """One step of running sequences whose states live in a pool (serving; not
    differentiable). Wx [M,G,N,D], b [G,N,D] or None, pool [P,N,D] fp32, slots
    [M] int32: each row's place in the pool, or None for the row's number; no
    slot twice; a negative slot marks an unused row (h = 0, no state touched).
    The new states go to pool_out, by default the pool itself (another one shares
    no memory with it). Returns h [M,N,D]. status: an int32 CUDA tensor of one element, zeroed by the caller,
    in which a slot past the pool is recorded (such a row counts as unused);
    _lib.rnn_check_status(status) raises for it."""
    _on_gpu(Wx, "gated_scan_step")
    N, D = _gated_shapes(Wx, b, function, 1)
    _check_status(status, Wx)
    M = Wx.shape[0]
    P = _check_pool((pool,) if pool_out is None else (pool, pool_out), slots, M, (N, D), "N,D", Wx, "Wx")
    if slots is not None:
        slots = slots.contiguous()
    h = Wx.new_empty((M, N, D))
    out = pool if pool_out is None else pool_out
    _lib.rnn_gated_step(M, P, N, D, function, Wx.dtype, _dense(Wx), _dense(b), slots, pool, out, h, status)
    if not out.is_inference():  # a graph that saved the old states has to learn of the write
        torch.autograd.graph.increment_version(out)
    return h


# ---- gated delta rule ----------------------------------------------------------------
def _delta_run(q, k, v, g, beta, state, reset, lengths, scale, status, keep):
    """(o, last, q, k and v as the library took them, plan, tape)."""
    B, T, Nk, Dk = q.shape
    N, Dv = v.shape[2:]
    plan = _lib.delta_plan(B, T, Nk, N, Dk, Dv, q.dtype, _lib.check_device(q))
    q, k, v, g, beta, state = (_dense(t) for t in (q, k, v, g, beta, state))
    o = q.new_empty((B, T, N, Dv))
    last = torch.empty((B, 1, N, Dk, Dv), dtype=torch.float32, device=v.device)
    tape = torch.empty(plan[2 if keep else 1], dtype=torch.uint8, device=v.device)
    _lib.rnn_delta_fwd(plan[0], q, k, v, g, beta, state, reset, lengths, scale, o, last, keep, tape)
    _add_status(status, tape)
    return o, last, q, k, v, plan, tape


class _DeltaFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, state, reset, lengths, scale, status):
        o, last, q, k, v, ctx.plan, tape = _delta_run(q, k, v, g, beta, state, reset, lengths, scale, status, True)
        ctx.scale, ctx.status = scale, status
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(q, k, v, lengths, tape)
        return o, last

    @staticmethod
    def backward(ctx, do, dlast):
        return (_delta_bwd_once if torch.is_grad_enabled() else _delta_bwd)(ctx, do, dlast)


def _delta_grads(q, v, state, plan):
    """dq, dk, dv, dg, dbeta, dstate (or None) and the workspace."""
    B, T, N, Dv = v.shape
    dg, dbeta = (torch.empty((B, T, N), dtype=torch.float32, device=q.device) for _ in range(2))
    ds = torch.empty((B, 1, N, q.shape[3], Dv), dtype=torch.float32, device=q.device) if state else None
    return (q.new_empty(q.shape), q.new_empty(q.shape), q.new_empty(v.shape), dg, dbeta, ds,
            torch.empty(plan[3], dtype=torch.uint8, device=q.device))


def _delta_bwd(ctx, do, dlast):
    _first_order(do, dlast)
    q, k, v, lengths, tape = ctx.saved_tensors
    dq, dk, dv, dg, dbeta, ds, ws = _delta_grads(q, v, ctx.needs_input_grad[5], ctx.plan)
    _lib.rnn_delta_bwd(ctx.plan[0], q, k, v, lengths, ctx.scale, tape, _dense(do), _dense(dlast), dq, dk, dv, dg, dbeta, ds, ws)
    _add_status(ctx.status, tape)
    return dq, dk, dv, dg, dbeta, ds, None, None, None, None


_delta_bwd_once = once_differentiable(_delta_bwd)


def _delta_shapes(q, k, v, g, beta, lead):
    """Checks the inputs of the delta rule, whose leading axes are lead; returns (Nk, N, Dk, Dv)."""
    n = len(lead)
    if q.dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}")
    if q.dim() != n + 2 or v.dim() != n + 2:
        raise ValueError(f"q and v must have {n + 2} dimensions, got shapes {tuple(q.shape)} and {tuple(v.shape)}")
    (Nk, Dk), (N, Dv) = q.shape[n:], v.shape[n:]
    if q.shape[:n] != lead or k.shape != q.shape or v.shape[:n] != lead:
        raise ValueError(f"q and k must have one shape and v the same leading axes, got {tuple(q.shape)}, "
                         f"{tuple(k.shape)} and {tuple(v.shape)}")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError(f"q, k and v must have one dtype, got {q.dtype}, {k.dtype} and {v.dtype}")
    if Nk < 1 or N < 1 or N % Nk:
        raise ValueError(f"v's {N} heads must be a multiple of q's and k's {Nk}")
    if not (1 <= Dk <= _lib.DELTA_MAX_D and 1 <= Dv <= _lib.DELTA_MAX_D):
        raise ValueError(f"heads of 1 to {_lib.DELTA_MAX_D} channels, got {Dk} and {Dv}")
    for t, name in ((g, "g"), (beta, "beta")):
        if t.shape != (*lead, N):
            raise ValueError(f"{name} must be {(*lead, N)}, got {tuple(t.shape)}")
        if t.dtype not in (torch.float32, q.dtype):
            raise TypeError(f"{name} must be float32 or {q.dtype}, got {t.dtype}")
    for t, name in ((k, "k"), (v, "v"), (g, "g"), (beta, "beta")):
        if t.get_device() != q.get_device():
            raise ValueError(f"{name} must be on q's device")
    return Nk, N, Dk, Dv


def gated_delta(q, k, v, g, beta, state=None, scale=None, reset=None, lengths=None, status=None):
    """Gated delta rule: a scan whose state is a matrix S [Dk,Dv] per head,
    u_t = beta_t (v_t - a_t S_{t-1}^T k_t), S_t = a_t S_{t-1} + k_t u_t^T,
    o_t = scale S_t^T q_t, a_t = exp(g_t).

    q, k [B,T,Nk,Dk] and v [B,T,N,Dv] (bf16 or fp32; N a multiple of Nk: v head n
    goes with q and k head n // (N // Nk); Dk and Dv up to 256), g and beta
    [B,T,N] (fp32 or q's dtype), state [B,1,N,Dk,Dv] or None (zeros), scale None =
    Dk ** -0.5. Keys are taken as they are: beta |k|^2 past 2 lets the state
    grow (group_norm with centered=False and a weight of Dk ** -0.5 makes unit keys).
    reset [B,T] (bool or uint8): S_{t-1} counts as zero at the marked steps
    (packed documents), whatever it holds. lengths [B]: row b has lengths[b]
    steps; past them nothing is looked at, o is zero and the state is kept.
    Returns (o [B,T,N,Dv], last [B,1,N,Dk,Dv]: the state after the last step,
    fp32). Differentiable in q, k, v, g, beta and state; what is fp32 is fp32
    throughout. The last bits of fp32 results follow from how the steps are spread
    over the GPU: from the sizes, and from whether a gradient will be asked for;
    where one will be, bf16 takes a |beta| below 2^-60 (a shut gate) as 2^-60.
    An infinity or a NaN in q, k, v, g or beta may reach every step of its row and
    head; one in the state ends at the next reset.
    status: an int32 CUDA tensor of one element, zeroed by the caller, in which
    the forward and the backward record a device-side wait that ran out (their
    results are then not valid); _lib.rnn_check_status(status) raises for it."""
    _on_gpu(q, "gated_delta")
    if q.dim() != 4:
        raise ValueError(f"q must be [B,T,Nk,Dk], got shape {tuple(q.shape)}")
    B, T = q.shape[:2]
    _, N, Dk, Dv = _delta_shapes(q, k, v, g, beta, (B, T))
    if state is not None:
        if state.shape != (B, 1, N, Dk, Dv):
            raise ValueError(f"state must be [B,1,N,Dk,Dv]={(B, 1, N, Dk, Dv)}, got {tuple(state.shape)}")
        if state.get_device() != q.get_device():
            raise ValueError("state must be on q's device")
        if state.dtype != torch.float32:
            state = state.float()
    _check_status(status, q)
    reset, lengths = _marks(reset, lengths, B, T, q, "q")
    scale = Dk ** -0.5 if scale is None else float(scale)
    if g.dtype != torch.float32:
        g = g.float()
    if beta.dtype != torch.float32:
        beta = beta.float()
    if _tracked(q, k, v, g, beta, state):
        return _DeltaFn.apply(q, k, v, g, beta, state, reset, lengths, scale, status)
    return _delta_run(q, k, v, g, beta, state, reset, lengths, scale, status, False)[:2]


def gated_delta_step(q, k, v, g, beta, pool, slots=None, scale=None, pool_out=None, status=None):
    """One step of running sequences whose states live in a pool (serving; not
    differentiable). q, k [M,Nk,Dk], v [M,N,Dv], g and beta [M,N] as for
    gated_delta, pool [P,N,Dk,Dv] fp32; slots, pool_out and status as for
    gated_scan_step. Returns o [M,N,Dv]."""
    _on_gpu(q, "gated_delta_step")
    if q.dim() != 3:
        raise ValueError(f"q must be [M,Nk,Dk], got shape {tuple(q.shape)}")
    M = q.shape[0]
    Nk, N, Dk, Dv = _delta_shapes(q, k, v, g, beta, (M,))
    _check_status(status, q)
    P = _check_pool((pool,) if pool_out is None else (pool, pool_out), slots, M, (N, Dk, Dv), "N,Dk,Dv", q, "q")
    if slots is not None:
        slots = slots.contiguous()
    o = v.new_empty((M, N, Dv))
    out = pool if pool_out is None else pool_out
    _lib.rnn_delta_step(M, P, Nk, N, Dk, Dv, _dense(q), _dense(k), _dense(v), _dense(g.float()), _dense(beta.float()),
                        slots, pool, out, Dk ** -0.5 if scale is None else float(scale), o, status)
    if not out.is_inference():  # a graph that saved the old states has to learn of the write
        torch.autograd.graph.increment_version(out)
    return o


# ---- group norm ------------------------------------------------------------------------
def _norm_run(x, weight, bias, gate, groups, activation, eps, centered):
    """(y, and the tensors as the library took them)."""
    _lib.check_device(x)
    x, weight, bias, gate = _dense(x), _dense(weight), _dense(bias), _dense(gate)
    C = x.shape[-1]
    y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _lib.rnn_group_norm_fwd(x.numel() // C, groups, C // groups, activation, centered, eps, x, weight, bias, gate, y)
    return y, x, weight, bias, gate


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, gate, groups, activation, eps, centered):
        y, *kept = _norm_run(x, weight, bias, gate, groups, activation, eps, centered)
        ctx.args = (groups, activation, eps, centered)
        ctx.save_for_backward(*kept)
        return y

    @staticmethod
    def backward(ctx, dy):
        return (_norm_bwd_once if torch.is_grad_enabled() else _norm_bwd)(ctx, dy)


def _norm_grads(x, weight, bias, gate, groups, need):
    """dx, dweight, dbias, dgate (or None) and the workspace (or None)."""
    dx, dgate = x.new_empty(x.shape), None if gate is None else x.new_empty(x.shape)
    dw = weight.new_empty(weight.shape) if need[1] else None
    db = bias.new_empty(bias.shape) if need[2] else None
    ws = None
    if dw is not None or db is not None:
        C = x.shape[-1]
        size = _lib.rnn_group_norm_workspace_size(x.numel() // C, groups, C // groups, x.dtype, x.get_device())
        ws = torch.empty(size, dtype=torch.uint8, device=x.device)
    return dx, dw, db, dgate, ws


def _norm_bwd(ctx, dy):
    _first_order(dy)
    x, weight, bias, gate = ctx.saved_tensors
    groups, activation, eps, centered = ctx.args
    need = ctx.needs_input_grad
    dx, dw, db, dgate, ws = _norm_grads(x, weight, bias, gate, groups, need)
    C = x.shape[-1]
    _lib.rnn_group_norm_bwd(x.numel() // C, groups, C // groups, activation, centered, eps, x, weight, bias, gate,
                            _dense(dy), dx, dgate, dw, db, ws)
    return dx if need[0] else None, dw, db, dgate if need[3] else None, None, None, None, None


_norm_bwd_once = once_differentiable(_norm_bwd)


def group_norm(x, groups: int, weight=None, bias=None, gate=None, activation=None, eps: float = 1e-5,
               centered: bool = True):
    """Group norm with an activation, channels last: x [..., C] (bf16 or fp32), C
    in `groups` groups of neighbouring channels (the heads of a scan's output),
    statistics over one group's channels of one row. n = (x - mean) / sqrt(var +
    eps), t = n * weight + bias, y = act(t) or, with a gate of x's shape,
    t * act(gate). weight, bias [C] or None; activation None, "silu" or
    "sigmoid"; centered=False leaves the mean out (var is then the mean square).
    Differentiable in x, weight, bias and gate; the statistics and all sums are
    fp32. Up to 65535 groups of up to 14336 channels, 2^28 channels in all."""
    _on_gpu(x, "group_norm")
    if x.dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"x must have channels, got shape {tuple(x.shape)}")
    C = x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"{C} channels do not make {groups} groups")
    if groups > _lib.NORM_MAX_GROUPS or C > _lib.NORM_MAX_CHANNELS:
        raise ValueError(f"up to {_lib.NORM_MAX_GROUPS} groups and {_lib.NORM_MAX_CHANNELS} channels, got {groups} and {C}")
    if C // groups > _lib.NORM_MAX_WIDTH:
        raise ValueError(f"groups of up to {_lib.NORM_MAX_WIDTH} channels, got {C // groups}")
    if activation not in _lib.ACTIVATIONS:
        raise ValueError(f"activation must be one of {list(_lib.ACTIVATIONS)}, got {activation!r}")
    if not eps >= 0:
        raise ValueError(f"eps must not be negative, got {eps}")
    for t, name, shape in ((weight, "weight", (C,)), (bias, "bias", (C,)), (gate, "gate", x.shape)):
        if t is None:
            continue
        if t.shape != shape:
            raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
        if t.dtype != x.dtype:
            raise TypeError(f"{name} is {t.dtype}, x is {x.dtype}")
        if t.get_device() != x.get_device():
            raise ValueError(f"{name} must be on x's device")
    if _tracked(x, weight, bias, gate):
        return _NormFn.apply(x, weight, bias, gate, int(groups), activation, float(eps), bool(centered))
    return _norm_run(x, weight, bias, gate, int(groups), activation, float(eps), bool(centered))[0]


# ---- 8-bit activation checkpoints -----------------------------------------------------
def _pack(x):
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
    scales = torch.empty((-(-rows // _lib.ACT_BLOCK), cols), dtype=torch.uint8, device=x.device)
    _lib.rnn_act_pack(rows, cols, x, q, scales)
    return q, scales


def checkpoint_pack(x):
    """x [..., cols] (bf16 or fp32) in 8 bits: q (int8, x's shape) and scales
    (uint8, [ceil(rows / 32), cols], rows being the flattened leading axes): one
    power of two per 32 rows of a column, the smallest whose 127-fold holds the
    block's largest magnitude. Blocks with an infinity or a NaN unpack to NaN."""
    _on_gpu(x, "checkpoint_pack")
    if x.dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if not (x.dim() >= 1 and x.shape[-1] >= 1):
        raise ValueError(f"x must have a last axis, got shape {tuple(x.shape)}")
    q, scales = _pack(_dense(x.detach().reshape(-1, x.shape[-1])))
    return q.reshape(x.shape), scales


def checkpoint_unpack(q, scales, dtype=torch.bfloat16):
    """The values (exact in either dtype) that checkpoint_pack's q and scales stand for."""
    _on_gpu(q, "checkpoint_unpack")
    if dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {dtype}")
    if not (q.dtype == torch.int8 and scales.dtype == torch.uint8):
        raise TypeError("q must be int8 and scales uint8")
    if not (q.dim() >= 1 and q.shape[-1] >= 1):
        raise ValueError(f"q must have a last axis, got shape {tuple(q.shape)}")
    cols = q.shape[-1]
    rows = q.numel() // cols
    if not (tuple(scales.shape) == (-(-rows // _lib.ACT_BLOCK), cols) and scales.device == q.device):
        raise ValueError(f"scales must be [{-(-rows // _lib.ACT_BLOCK)},{cols}] on q's device, got {tuple(scales.shape)}")
    x = torch.empty(q.shape, dtype=dtype, device=q.device)
    _lib.rnn_act_unpack(rows, cols, _dense(q), _dense(scales), x)
    return x


# ---- token embedding --------------------------------------------------------------------
def _embed_run(ids, W, scale, status):
    W = _dense(W)
    V, E = W.shape
    out = W.new_empty((*ids.shape, E))
    _lib.rnn_embed_fwd(ids.numel(), V, E, ids, W, scale, out, status)
    return out


class _EmbedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, W, scale, padding_idx, status):
        ctx.save_for_backward(ids)
        ctx.args = (W.shape, W.dtype, scale, padding_idx)
        return _embed_run(ids, W, scale, status)

    @staticmethod
    def backward(ctx, dout):
        return (_embed_bwd_once if torch.is_grad_enabled() else _embed_bwd)(ctx, dout)


def _embed_bwd(ctx, dout):
    _first_order(dout)
    (ids,) = ctx.saved_tensors
    (V, E), dtype, scale, pad = ctx.args
    n = ids.numel()
    dW = torch.empty((V, E), dtype=dtype, device=ids.device)
    size = _lib.rnn_embed_bwd_workspace_size(n, V, E, ids.get_device())
    ws = _workspace(size, ids, None)
    _lib.rnn_embed_bwd(n, V, E, ids, pad, _dense(dout), scale, dW, ws)
    return None, dW, None, None, None


_embed_bwd_once = once_differentiable(_embed_bwd)


def embedding(ids, weight, scale: float = 1.0, padding_idx=None, status=None):
    """scale * weight[ids]: ids [...] int32 or int64, weight [V, E] (bf16 or
    fp32); returns [..., E]. Differentiable in weight: the gradient is dense
    [V, E], each row the scaled fp32 sum over its tokens in a fixed order,
    zero for padding_idx. Ids out of range give zero rows and no gradient;
    status: an int32 CUDA tensor of one element, zeroed by the caller, in which
    they are recorded (_lib.rnn_check_status(status) raises for it)."""
    _on_gpu(weight, "embedding")
    if weight.dim() != 2:
        raise ValueError(f"weight must be [V,E], got shape {tuple(weight.shape)}")
    if weight.dtype not in _lib.DTYPES:
        raise TypeError(f"unsupported dtype {weight.dtype}")
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"ids must be int32 or int64, got {ids.dtype}")
    if ids.get_device() != weight.get_device():
        raise ValueError("ids must be on weight's device")
    if not (padding_idx is None or 0 <= padding_idx < weight.shape[0]):
        raise ValueError(f"padding_idx must be None or in 0 .. {weight.shape[0] - 1}, got {padding_idx}")
    _check_status(status, weight)
    pad = -1 if padding_idx is None else int(padding_idx)
    ids = ids.contiguous()
    if _tracked(weight):
        return _EmbedFn.apply(ids, weight, float(scale), pad, status)
    return _embed_run(ids, weight, float(scale), status)

"""Bindings of the delta rule with one decay per head and of the operators around it
(``kda_qk_norm``, ``kda_gdr_fwd``, ``kda_gdr_step``, ``kda_verify_drafts`` and the backward
passes): argument checks and marshalling, as in the package's other calls."""
from __future__ import annotations

import ctypes
import sys

_vp, _i, _f, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_longlong
_NORMS = {"l2": 0, "rms": 1}


def declare(lib):
    """Argument and result types of these functions on a loaded library."""
    norm = [_i, _i, _f, _vp, _vp]
    turn = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _ll, _ll, _vp]
    rule = [_vp] * 5 + [_i, _f]
    sizes = [_i] * 6 + [_ll] * 3 + [_vp]
    for name, args in (
            ("kda_qk_norm", [_vp] * 4 + norm + turn),
            ("kda_qk_norm_bwd", [_vp] * 6 + norm + [_vp, _vp] + turn),
            ("kda_gdr_fwd", rule + [_vp, _vp, _i, _vp, _i, _vp, _i] + sizes),
            ("kda_gdr_bwd", rule + [_vp, _i, _vp, _vp, _i] + [_vp] * 6 + [_i, _vp, _i] + sizes),
            ("kda_gdr_step", rule + [_vp, _vp, _i, _vp, _i, _vp, _i, _vp] + sizes),
            ("kda_verify_drafts", [_vp, _vp, _i] + [_vp] * 6 + [_i] * 3 + [_vp])):
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, _i
    lib.kda_gdr_bwd_workspace_bytes.argtypes = [_i] * 6
    lib.kda_gdr_bwd_workspace_bytes.restype = ctypes.c_size_t
    return lib


# The checks below run on every call, where a decode step's whole kernel takes a few
# microseconds, so they read each attribute of a tensor once and import nothing.
def _torch():
    """The torch module: loaded already wherever a tensor has been made."""
    return sys.modules["torch"]


def _call(name, device, stream, *args):
    """One library call on `device` and `stream` (default: the current stream)."""
    torch, kda = _torch(), sys.modules[__package__]
    fn = getattr(kda._lib or kda.load_library(), name)
    index = device.index
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(index)
    else:
        s = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == index:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, s)
    if rc != 0:
        raise kda.KdaError(rc, name)


def results_on(stream, device, make):
    """The tensors that ``make()`` allocates for a call on `stream` (a torch stream or a
    handle; None: the current one) to write.  They come from that stream's memory, since what the
    current stream's pool hands out may still be read or written by work queued there; and
    memory that the current stream's work reads is not given away before that work is done."""
    torch = _torch()
    if stream is None:
        return make()
    if not hasattr(stream, "cuda_stream"):      # a handle; 0 and 1 are the default stream's
        handle = int(stream)
        stream = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else torch.cuda.default_stream(device)
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return make()
    with torch.cuda.stream(stream):
        r = make()
    for t in r.values():
        t.record_stream(current)
    return r


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cuda(t, where):
    device = t.device
    if device.type != "cuda":
        raise ValueError(f"{where} takes CUDA tensors")
    return device


def _is(t, name, dtypes, shape, device):
    """Type, shape and place of a tensor; a ``None`` stands for an optional one."""
    if t is None:
        return
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _dense(t, name, dtypes, shape, device):
    if t is None:
        return
    _is(t, name, dtypes, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _token_stride(t, name):
    """Elements from one token to the next of [..., heads, channels], whose tokens must be
    equally spaced and whose heads and channels contiguous."""
    shape, s = t.shape, t.stride()
    h, d = shape[-2], shape[-1]
    if t.is_contiguous():
        return h * d
    ok = (d == 1 or s[-1] == 1) and (h == 1 or s[-2] == d)
    step, span = None, 1
    for i in range(len(s) - 3, -1, -1):
        if shape[i] != 1:
            if step is None:
                step = s[i]
            ok = ok and s[i] == step * span
            span *= shape[i]
    if not ok or (step is not None and step < h * d):
        raise ValueError(f"{name}: heads and channels must be contiguous and tokens equally spaced, "
                         f"got strides {s}")
    return h * d if step is None else step


def _norm_args(where, q, k, norm, q_weight, k_weight, cos, sin, positions):
    torch = _torch()
    dev, qs, ks, dtype = _cuda(q, where), q.shape, k.shape, q.dtype
    if len(qs) < 3 or ks[:-2] != qs[:-2] or ks[-1] != qs[-1]:
        raise ValueError(f"q and k must be [..., heads, channels] with the same tokens and "
                         f"channels, got {tuple(qs)} and {tuple(ks)}")
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"q must be torch.bfloat16 or torch.float32, got {dtype}")
    _is(k, "k", (dtype,), ks, dev)
    if norm not in _NORMS:
        raise ValueError(f"norm must be 'l2' or 'rms', got {norm!r}")
    D = qs[-1]
    f32 = (torch.float32,)
    if q_weight is not None:
        _dense(q_weight, "q_weight", f32, (D,), dev)
    if k_weight is not None:
        _dense(k_weight, "k_weight", f32, (D,), dev)
    rows = rotary = 0
    if cos is not None:
        if sin is None or cos.dim() != 2 or 2 * cos.shape[1] > D:
            raise ValueError("cos and sin must both be [rows, rotary_dim / 2] with rotary_dim <= channels")
        rows, rotary = cos.shape[0], 2 * cos.shape[1]
        _dense(cos, "cos", f32, cos.shape, dev)
        _dense(sin, "sin", f32, cos.shape, dev)
        _dense(positions, "positions", (torch.int32,), qs[:-2], dev)
    elif sin is not None or positions is not None:
        raise ValueError("sin and positions need cos")
    head = (_ptr(q_weight), _ptr(k_weight))
    tail = (_ptr(cos), _ptr(sin), _ptr(positions), rows, rotary)
    tokens = qs[0] if len(qs) == 3 else qs[:-2].numel()
    sizes = (tokens, qs[-2], ks[-2], D, _token_stride(q, "q"), _token_stride(k, "k"))
    return dev, int(dtype is torch.float32), head, tail, sizes


def kda_qk_norm(q, k, q_out, k_out, norm: str = "l2", eps: float = 1e-6, q_weight=None,
                k_weight=None, cos=None, sin=None, positions=None, interleaved: bool = False,
                stream=None) -> None:
    """Norms of queries and keys for each head, with the position rotation in the same
    pass, on CUDA tensors (asynchronous on ``stream``).

    q [..., Hq, D] and k [..., Hk, D]: bf16 or fp32, tokens equally spaced (views of one
    projection's buffer are fine); q_out, k_out: contiguous, of the same shapes and type;
    norm: 'l2' (x / sqrt(sum x^2 + eps)) or 'rms' (mean); weights: optional fp32 [D];
    cos, sin: optional fp32 [rows, rotary_dim / 2]; positions: optional int32 [...] (default:
    token t uses row t); interleaved: neighbouring channels are pairs, else the halves of
    the rotated channels.  Raises KdaError on a rejected call.
    """
    dev, f32, w, turn, sizes = _norm_args("kda_qk_norm", q, k, norm, q_weight, k_weight, cos, sin,
                                          positions)
    _dense(q_out, "q_out", (q.dtype,), q.shape, dev)
    _dense(k_out, "k_out", (q.dtype,), k.shape, dev)
    _call("kda_qk_norm", dev, stream, _ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), f32,
          _NORMS[norm], eps, *w, *turn, int(interleaved), *sizes)


def kda_qk_norm_bwd(q, k, dq_out, dk_out, norm: str = "l2", eps: float = 1e-6, q_weight=None,
                    k_weight=None, cos=None, sin=None, positions=None, interleaved: bool = False,
                    stream=None) -> dict:
    """Gradients of ``kda_qk_norm`` from dL/d(q_out) and dL/d(k_out) (contiguous, of q's
    type): dq, dk (contiguous, of q's type) and, with weights, dq_weight, dk_weight (fp32 [D])."""
    torch = _torch()
    dev, f32, w, turn, sizes = _norm_args("kda_qk_norm_bwd", q, k, norm, q_weight, k_weight, cos, sin,
                                          positions)
    _dense(dq_out, "dq_out", (q.dtype,), q.shape, dev)
    _dense(dk_out, "dk_out", (q.dtype,), k.shape, dev)
    like = {"dq": dq_out, "dk": dk_out, "dq_weight": q_weight, "dk_weight": k_weight}
    r = results_on(stream, dev, lambda: {n: torch.empty_like(t) for n, t in like.items() if t is not None})
    _call("kda_qk_norm_bwd", dev, stream, _ptr(q), _ptr(k), _ptr(dq_out), _ptr(dk_out),
          _ptr(r["dq"]), _ptr(r["dk"]), f32, _NORMS[norm], eps, *w, _ptr(r.get("dq_weight")),
          _ptr(r.get("dk_weight")), *turn, int(interleaved), *sizes)
    return r


def _rule_args(where, q, k, v, g, beta):
    torch = _torch()
    dev, qs, vs = _cuda(q, where), q.shape, v.shape
    bf16 = (torch.bfloat16,)
    if len(qs) != 4 or len(vs) != 4:
        raise ValueError("q, k and v must be [B, T, heads, 128]")
    B, T, Hk, K = qs
    Hv, V = vs[2], vs[3]
    _is(q, "q", bf16, qs, dev)
    _is(k, "k", bf16, qs, dev)
    _is(v, "v", bf16, (B, T, Hv, V), dev)
    gate = g.dtype
    _dense(g, "g", (torch.float32, torch.bfloat16), (B, T, Hv), dev)
    _dense(beta, "beta", (gate,), (B, T, Hv), dev)
    head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), int(gate is torch.float32))
    strides = (_token_stride(q, "q"), _token_stride(k, "k"), _token_stride(v, "v"))
    return dev, head, (B, T, Hk, Hv, K, V), strides


def _states(dev, shape, **states):
    torch = _torch()
    r = []
    for name, t in states.items():
        if t is None:
            r += (None, 0)
        else:
            _dense(t, name, (torch.float32, torch.bfloat16), shape, dev)
            r += (t.data_ptr(), int(t.dtype is torch.float32))
    return r


def _sequences(cu_seqlens, B, dev):
    """(number of states, the C call's num_seqs) of a call."""
    torch = _torch()
    if cu_seqlens is None:
        return B, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a contiguous 1-D int32 tensor")
    _dense(cu_seqlens, "cu_seqlens", (torch.int32,), cu_seqlens.shape, dev)
    return cu_seqlens.numel() - 1, cu_seqlens.numel() - 1


def kda_gdr_fwd(q, k, v, g, beta, scale: float, out, initial_state=None, final_state=None,
                cu_seqlens=None, stream=None) -> None:
    """The delta rule with one decay per value head over whole sequences, on CUDA tensors
    (asynchronous on ``stream``).

    q, k: bf16 [B, T, Hk, 128], used as given; v, out: bf16 [B, T, Hv, 128], Hv a multiple of
    Hk; q, k, v may be views with equally spaced tokens; g (log decay), beta (write
    strength): fp32 or bf16 [B, T, Hv]; states: optional bf16 or fp32 [N, Hv, 128, 128];
    cu_seqlens: optional int32 [N + 1] (then B == 1).  Raises KdaError on a rejected call.
    """
    torch = _torch()
    dev, head, (B, T, Hk, Hv, K, V), strides = _rule_args("kda_gdr_fwd", q, k, v, g, beta)
    _dense(out, "out", (torch.bfloat16,), (B, T, Hv, V), dev)
    N, num = _sequences(cu_seqlens, B, dev)
    states = _states(dev, (N, Hv, K, V), initial_state=initial_state, final_state=final_state)
    _call("kda_gdr_fwd", dev, stream, *head, scale, _ptr(out), *states, _ptr(cu_seqlens), num, B, T,
          Hk, Hv, K, V, *strides)


def kda_gdr_bwd(q, k, v, g, beta, scale: float, d_out, initial_state=None, d_final_state=None,
                cu_seqlens=None, stream=None, d_initial_state: bool = True) -> dict:
    """Gradients of a loss with respect to ``kda_gdr_fwd``'s inputs, on CUDA tensors
    (asynchronous on ``stream``).

    d_out: bf16 [B, T, Hv, 128] = dL/d(out); d_final_state: optional bf16 or fp32
    [N, Hv, 128, 128] = dL/d(final state).  Other arguments as ``kda_gdr_fwd``.  Returns dq, dk
    (bf16 [B, T, Hk, 128]), dv (bf16 [B, T, Hv, 128]), dg, dbeta ([B, T, Hv] of the gates' type)
    and, with an initial state (unless d_initial_state is False), d_initial_state of its type.
    """
    torch = _torch()
    dev, head, (B, T, Hk, Hv, K, V), strides = _rule_args("kda_gdr_bwd", q, k, v, g, beta)
    _dense(d_out, "d_out", (torch.bfloat16,), (B, T, Hv, V), dev)
    N, num = _sequences(cu_seqlens, B, dev)
    states = _states(dev, (N, Hv, K, V), initial_state=initial_state, d_final_state=d_final_state)
    dense = torch.contiguous_format
    like = {"dq": q, "dk": k, "dv": d_out, "dg": g, "dbeta": beta}
    if d_initial_state and initial_state is not None:
        like["d_initial_state"] = initial_state
    r = results_on(stream, dev, lambda: {n: torch.empty_like(t, memory_format=dense) for n, t in like.items()})
    ds = r.get("d_initial_state")
    _call("kda_gdr_bwd", dev, stream, *head, scale, *states[:2], _ptr(d_out), *states[2:],
          _ptr(r["dq"]), _ptr(r["dk"]), _ptr(r["dv"]), _ptr(r["dg"]), _ptr(r["dbeta"]), _ptr(ds),
          int(ds is not None and ds.dtype == torch.float32), _ptr(cu_seqlens), num, B, T, Hk, Hv, K, V,
          *strides)
    return r


def kda_gdr_bwd_workspace_bytes(B: int, T: int, Hk: int, Hv: int, num_seqs: int = 0,
                                varlen: bool = False) -> int:
    return int(sys.modules[__package__].load_library().kda_gdr_bwd_workspace_bytes(B, T, Hk, Hv, num_seqs, int(varlen)))


def kda_gdr_step(q, k, v, g, beta, scale: float, out=None, state_in=None, state_out=None,
                 slots=None, lengths=None, stream=None) -> None:
    """The same rule for T new tokens of each of N sequences on states held in memory, on
    CUDA tensors (asynchronous on ``stream``).

    q, k: bf16 [N, T, Hk, 128]; v, out: bf16 [N, T, Hv, 128] (out optional); g, beta: fp32 or
    bf16 [N, T, Hv]; state_in / state_out: optional pools, bf16 or fp32
    [pool, Hv, 128, 128] (the same tensor updates it in place); slots: optional int32 [N], each
    sequence's state (-1: a padding entry); lengths: optional int32 [N], the tokens after
    which the state is kept (default T).  Raises KdaError on a rejected call.
    """
    torch = _torch()
    dev, head, (N, T, Hk, Hv, K, V), strides = _rule_args("kda_gdr_step", q, k, v, g, beta)
    _dense(out, "out", (torch.bfloat16,), (N, T, Hv, V), dev)
    pool = N
    if slots is not None:
        _dense(slots, "slots", (torch.int32,), (N,), dev)
        if state_in is None and state_out is None:
            raise ValueError("slots need state_in or state_out")
        pool = (state_in if state_in is not None else state_out).shape[0]
    _dense(lengths, "lengths", (torch.int32,), (N,), dev)
    states = _states(dev, (pool, Hv, K, V), state_in=state_in, state_out=state_out)
    _call("kda_gdr_step", dev, stream, *head, scale, _ptr(out), *states, _ptr(slots), pool,
          _ptr(lengths), N, T, Hk, Hv, K, V, *strides)


def kda_verify_drafts(target_probs, draft_probs, draft_tokens, uniform, noise, accepted, tokens,
                      num_drafts=None, stream=None) -> None:
    """Verification of drafted tokens against the target's probabilities from given random
    numbers, on CUDA tensors (asynchronous on ``stream``).

    target_probs: fp32 or bf16 [N, D + 1, V]; draft_probs: [N, D, V] of the same type, or None
    (the drafts were certain); draft_tokens: int32 [N, D]; uniform: fp32 [N, D] in [0, 1);
    noise: fp32 [N, V] ~ Exp(1); num_drafts: optional int32 [N]; writes accepted (int32 [N])
    and tokens (int32 [N, D + 1]: the kept drafts, the next token, then -1).
    Raises KdaError on a rejected call.
    """
    torch = _torch()
    dev = _cuda(target_probs, "kda_verify_drafts")
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise ValueError("target_probs must be [N, D + 1, V]")
    N, D, V = target_probs.shape[0], target_probs.shape[1] - 1, target_probs.shape[2]
    i32, f32 = (torch.int32,), (torch.float32,)
    _dense(target_probs, "target_probs", (torch.float32, torch.bfloat16), target_probs.shape, dev)
    _dense(draft_probs, "draft_probs", (target_probs.dtype,), (N, D, V), dev)
    _dense(draft_tokens, "draft_tokens", i32, (N, D), dev)
    _dense(uniform, "uniform", f32, (N, D), dev)
    _dense(noise, "noise", f32, (N, V), dev)
    _dense(num_drafts, "num_drafts", i32, (N,), dev)
    _dense(accepted, "accepted", i32, (N,), dev)
    _dense(tokens, "tokens", i32, (N, D + 1), dev)
    _call("kda_verify_drafts", dev, stream, _ptr(target_probs), _ptr(draft_probs),
          int(target_probs.dtype == torch.float32), _ptr(draft_tokens), _ptr(uniform), _ptr(noise),
          _ptr(num_drafts), _ptr(accepted), _ptr(tokens), N, D, V)

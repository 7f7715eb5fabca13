"""Linear attention with a decay for each head, and the norms behind it.

Thin Python binding of the C ABI in include/linear_attention.h (liblinattn.so), in the manner
of the conv's: it marshals torch tensors, passes torch's current HIP stream, and computes
nothing itself.  Calls on torch's current stream that are plainly in order are marshalled by the
call module (csrc/la_call.cpp, 12 us less a call); the Python here takes all others, and says
what is wrong with those that are refused.

    linear_attn_prefill(q, k, v, g, state, out, cu_seqlens, max_len=..., ...)
    linear_attn_update(q, k, v, g, state, out, ...)     T new tokens of each row, committed
    linear_attn_verify(q, k, v, g, state, out, ...)     T draft tokens, the state only read
    linear_attn_commit(k, v, g, state, num_tokens, ...) the accepted drafts folded in
    gated_norm(y, gate, weight, out, ...)
    residual_norm(y, residual, pre_weight, out, ...)

Tensors (all on one GPU; bf16 or fp32):
    q, k         [n_seq, T, q_heads, dk], or packed [total, q_heads, dk] (prefill)
    v, out       [n_seq, T, v_heads, dv], or packed [total, v_heads, dv]; v_heads a multiple of
                 q_heads, v head h uses q and k head h // (v_heads // q_heads)
    g            fp32 log decays [n_seq, T, v_heads] or [total, v_heads], [v_heads] (one decay
                 for each head), or None (no decay)
    state        [n_slots, v_heads, dk, dv], contiguous below the slot dimension
    slot_idx, has_initial_state, num_tokens: int32 [n_seq] or None; cu_seqlens int32 [n_seq+1]
Innermost dimensions have stride 1, other strides are free (q, k and v may be views of the
conv's output rows).
"""

from __future__ import annotations

import ctypes

from . import _lib, _linattn

__all__ = ["linear_attn_prefill", "linear_attn_update", "linear_attn_verify",
           "linear_attn_commit", "gated_norm", "residual_norm", "linear_attn_describe",
           "linear_attn_abi_version", "LinAttnError"]

ACTIVATIONS = {"silu": _linattn.LA_SILU, "sigmoid": _linattn.LA_SIGMOID}


class LinAttnError(RuntimeError):
    """A non-zero return code of the C ABI."""

    def __init__(self, code: int, message: str):
        super().__init__(message)
        self.code = code


_CODES = None


def _dtype_code(t) -> int:
    global _CODES
    if _CODES is None:
        import torch

        _CODES = {torch.float32: _lib.CV_F32, torch.bfloat16: _lib.CV_BF16}
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")
    return code


def _same_gpu(first, *others):
    dev = first.device
    if dev.type != "cuda":
        raise ValueError("all tensors must live on the same GPU (no CPU path exists)")
    for t in others:
        if t is not None and t.device != dev:
            raise ValueError("all tensors must live on the same GPU (no CPU path exists)")
    return dev


def _ptr(t):
    return None if t is None else t.data_ptr()


def _int32_vec(name, t, n):
    import torch

    if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (n,) or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor")


def _strides(t, dims):
    """Strides of dimensions dims of t; that of a dimension of one index is of no account."""
    shape, stride = t.shape, t.stride()
    return [stride[d] if shape[d] > 1 else 0 for d in dims]


def _on_stream(stream, dev):
    import torch

    if stream is None:
        stream = torch.cuda.current_stream(dev)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _attn_args(kind, q, k, v, g, state, out, *, cu_seqlens=None, max_len=None, scale=None,
               slot_idx=None, has_initial_state=None, num_tokens=None, workspace=None,
               stream=None):
    """(library, device, function, its arguments, what must stay alive)."""
    import torch

    lib = _linattn.load()
    dev = _same_gpu(state, q, k, v, g, out, cu_seqlens, slot_idx, has_initial_state, num_tokens,
                    workspace)
    packed = kind == "prefill"
    lead = 1 if packed else 2
    if k.dim() != lead + 2 or v.dim() != lead + 2 or k.shape[:lead] != v.shape[:lead]:
        raise ValueError(f"k and v must be {'[total' if packed else '[n_seq, T'}, heads, channels] "
                         f"of the same tokens (k {tuple(k.shape)}, v {tuple(v.shape)})")
    q_heads, dk = k.shape[lead:]
    v_heads, dv = v.shape[lead:]
    for name, t, like in (("q", q, k), ("out", out, v)):
        if t is not None and t.shape != like.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(like.shape)} is needed")
    for t in (q, k, v, out):
        if t is None:
            continue
        if t.dtype != v.dtype:
            raise TypeError("q, k, v and out must share one dtype")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("q, k, v and out need a contiguous channel dimension")
    if state.dim() != 4 or tuple(state.shape[1:]) != (v_heads, dk, dv) or \
            (state.shape[0] and not state[0].is_contiguous()):
        raise ValueError(f"state must be [n_slots, {v_heads}, {dk}, {dv}], contiguous below the "
                         f"slot dimension (got {tuple(state.shape)})")
    g_seq = g_tok = 0
    if g is not None:
        if g.dtype != torch.float32 or g.shape[-1] != v_heads or \
                (g.dim() > 1 and g.shape != v.shape[:-1]):
            raise ValueError(f"g must be float32 {tuple(v.shape[:-1])} or [{v_heads}]")
        if v_heads > 1 and g.stride(-1) != 1:
            raise ValueError("g needs a contiguous head dimension")
        if g.dim() > 1:
            g_tok = _strides(g, (lead - 1,))[0]
            g_seq = 0 if packed else _strides(g, (0,))[0]
    if packed:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must hold n_seq + 1 offsets")
        n_seq, T = cu_seqlens.shape[0] - 1, max(1, int(max_len))
        if T > 2 ** 31 - 1:
            raise ValueError(f"max_len ({T}) is over 2^31 - 1")
        _int32_vec("cu_seqlens", cu_seqlens, n_seq + 1)
        _int32_vec("has_initial_state", has_initial_state, n_seq)
        dims = (0, 1)
        if v.shape[0] == 0:
            # no tokens at all, though states may start from zeros: the token tensors hold no
            # element to point at, and one token that is neither read nor written stands in
            T = 1
            q, k, v, out = (t.new_empty(1, *t.shape[1:]) for t in (q, k, v, out))
    else:
        n_seq, T = v.shape[0], v.shape[1]
        _int32_vec("num_tokens", num_tokens, n_seq)
        dims = (0, 1, 2)
    _int32_vec("slot_idx", slot_idx, n_seq)

    def strides(t):
        return (0, 0, 0) if t is None else (0, *_strides(t, dims)) if packed else _strides(t, dims)

    shape = _linattn.LaShape(
        n_seq, T, q_heads, v_heads, dk, dv, dk ** -0.5 if scale is None else scale,
        _dtype_code(v), _dtype_code(state), state.shape[0], *strides(q), *strides(k),
        *strides(v), *strides(out), g_seq, g_tok, _strides(state, (0,))[0],
        v.shape[0] if packed else 0)
    handle = _on_stream(stream, dev)
    ref = ctypes.byref(shape)
    if packed:
        need = lib.linattn_prefill_workspace(ref)
        if need < 0:
            raise LinAttnError(need, _linattn.error_message(lib, need))
        if need and workspace is None:
            # a block of the stream that the call runs on: one that another stream gave up may
            # still be in use by what is queued there
            if handle == torch.cuda.current_stream(dev).cuda_stream:
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
            else:
                with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=dev) if handle
                                       else torch.cuda.default_stream(dev)):
                    workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        if workspace is not None and not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        size = 0 if workspace is None else workspace.numel() * workspace.element_size()
        fn, args = lib.linattn_prefill, (ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state),
                                         _ptr(slot_idx), _ptr(cu_seqlens), _ptr(has_initial_state),
                                         _ptr(out), _ptr(workspace), size, handle)
    elif kind == "commit":
        fn, args = lib.linattn_commit, (ref, _ptr(k), _ptr(v), _ptr(g), _ptr(state),
                                        _ptr(slot_idx), _ptr(num_tokens), handle)
    else:
        fn = lib.linattn_update if kind == "update" else lib.linattn_verify
        args = (ref, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state), _ptr(slot_idx), _ptr(out),
                handle)
    keep = (shape, q, k, v, g, state, out, cu_seqlens, slot_idx, has_initial_state, num_tokens,
            workspace)
    return lib, dev, fn, args, keep


def _gated_args(y, gate, weight, out, *, eps=1e-6, activation="silu", gate_first=False,
                stream=None):
    lib = _linattn.load()
    dev = _same_gpu(y, gate, weight, out)
    if y.dim() not in (2, 3) or out.shape != y.shape or (gate is not None and gate.shape != y.shape):
        raise ValueError("y, gate and out must be [rows, heads, dim] (or [rows, dim]) of one shape")
    dim = y.shape[-1]
    if tuple(weight.shape) != (dim,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous [{dim}] tensor")
    for t in (y, gate, weight, out):
        if t is None:
            continue
        if t.dtype != y.dtype:
            raise TypeError("y, gate, weight and out must share one dtype")
        if t.stride(-1) != 1 and dim > 1:
            raise ValueError("y, gate and out need a contiguous channel dimension")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")

    def strides(t):
        return (0, 0) if t is None else _strides(t, (0, 1)) if t.dim() == 3 else (*_strides(t, (0,)), 0)

    code = _dtype_code(y)
    shape = _linattn.LaNormShape(y.shape[0], y.shape[1] if y.dim() == 3 else 1, dim, eps, 1.0, code,
                                 code, ACTIVATIONS[activation], int(gate_first), *strides(y),
                                 *strides(gate), *strides(out), 0, 0)
    args = (ctypes.byref(shape), _ptr(y), _ptr(gate), _ptr(weight), _ptr(out),
            _on_stream(stream, dev))
    return lib, dev, lib.norm_gated, args, (shape, y, gate, weight, out)


def _residual_args(y, residual, pre_weight, out, *, post_weight=None, gate=None, scale=1.0,
                   residual_out=None, eps=1e-6, stream=None):
    lib = _linattn.load()
    if residual_out is None:
        residual_out = residual
    dev = _same_gpu(y, residual, pre_weight, out, post_weight, gate, residual_out)
    if y.dim() != 2 or residual.shape != y.shape or residual_out.shape != y.shape or \
            (out is not None and out.shape != y.shape):
        raise ValueError("y, residual, residual_out and out must be [rows, dim] of one shape")
    dim = y.shape[1]
    if gate is not None and gate.shape != y.shape and tuple(gate.shape) != (dim,):
        raise ValueError(f"gate must be [rows, {dim}] or [{dim}]")
    for name, t in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if t is not None and (tuple(t.shape) != (dim,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous [{dim}] tensor")
    if (out is None) != (pre_weight is None):
        raise ValueError("out and pre_weight go together")
    for t in (y, post_weight, gate, pre_weight, out):
        if t is not None and t.dtype != y.dtype:
            raise TypeError("y, gate, out and the weights must share one dtype")
    if residual_out.dtype != residual.dtype:
        raise TypeError("residual and residual_out must share one dtype")
    for t in (y, gate, residual, residual_out, out):
        if t is not None and t.stride(-1) != 1 and dim > 1:
            raise ValueError("tensors need a contiguous channel dimension")

    def row(t):
        return 0 if t is None or t.dim() == 1 else _strides(t, (0,))[0]

    shape = _linattn.LaNormShape(y.shape[0], 1, dim, eps, scale, _dtype_code(y),
                                 _dtype_code(residual), 0, 0, row(y), 0, row(gate), 0, row(out), 0,
                                 row(residual), row(residual_out))
    args = (ctypes.byref(shape), _ptr(y), _ptr(post_weight), _ptr(gate), _ptr(residual),
            _ptr(residual_out), _ptr(pre_weight), _ptr(out), _on_stream(stream, dev))
    return lib, dev, lib.norm_residual, args, (shape, y, post_weight, gate, residual, residual_out,
                                               pre_weight, out)


def _issue(lib, dev, fn, args, keep):
    import torch

    if torch.cuda.current_device() == dev.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != _lib.CV_OK:
        raise LinAttnError(rc, _linattn.error_message(lib, rc))


_call = None


class _NoCallModule:
    """In the call module's place: every call takes the binding's own way."""

    @staticmethod
    def attn(*args):
        return None

    gated = residual = attn


def _short():
    """The call module (csrc/la_call.cpp): the same marshalling in C for calls that are plainly in
    order; it answers None to all others, and they take the way above, as all do without it (it is
    built for one torch and one Python, and the library under both ways is not)."""
    global _call
    if _call is None:
        import torch  # noqa: F401  (its libraries, which the module is linked to)

        try:
            from . import _lacall as _call
        except ImportError as e:
            import warnings

            _call = _NoCallModule
            warnings.warn(f"calls are marshalled in Python, some 12 us each slower: {e} (build it with "
                          "`python -m causal_conv1d_verify_amd.build`)", RuntimeWarning, stacklevel=3)
    return _call


def _done(rc) -> bool:
    """Whether the call module took a call; raises on its error code."""
    if rc is None:
        return False
    if rc == _lib.CV_OK:
        return True
    raise LinAttnError(rc, _linattn.error_message(_linattn.load(), rc))


def linear_attn_prefill(q, k, v, g, state, out, cu_seqlens, *, max_len: int, scale=None,
                        slot_idx=None, has_initial_state=None, workspace=None,
                        stream=None) -> None:
    """Enqueue linear attention over packed prompts; each row's last state is left in its slot.
    max_len >= the longest prompt.  scale: dk ** -0.5 if None.  workspace: a contiguous uint8
    tensor of at least the size that the shape needs (allocated here if None)."""
    if stream is None and _done(_short().attn(0, q, k, v, g, state, out, cu_seqlens, max_len, scale,
                                              slot_idx, has_initial_state, None, workspace)):
        return
    _issue(*_attn_args("prefill", q, k, v, g, state, out, cu_seqlens=cu_seqlens, max_len=max_len,
                       scale=scale, slot_idx=slot_idx, has_initial_state=has_initial_state,
                       workspace=workspace, stream=stream))


def linear_attn_update(q, k, v, g, state, out, *, scale=None, slot_idx=None, stream=None) -> None:
    """Enqueue T (1..32) new tokens of each row: out for each, and the state after the last."""
    if stream is None and _done(_short().attn(1, q, k, v, g, state, out, None, None, scale, slot_idx,
                                              None, None, None)):
        return
    _issue(*_attn_args("update", q, k, v, g, state, out, scale=scale, slot_idx=slot_idx,
                       stream=stream))


def linear_attn_verify(q, k, v, g, state, out, *, scale=None, slot_idx=None, stream=None) -> None:
    """Enqueue the outputs of T (1..32) draft tokens of each row; the state is only read."""
    if stream is None and _done(_short().attn(2, q, k, v, g, state, out, None, None, scale, slot_idx,
                                              None, None, None)):
        return
    _issue(*_attn_args("verify", q, k, v, g, state, out, scale=scale, slot_idx=slot_idx,
                       stream=stream))


def linear_attn_commit(k, v, g, state, num_tokens=None, *, slot_idx=None, stream=None) -> None:
    """Enqueue the commit of the first num_tokens[i] (None: all) tokens of each row to its
    state."""
    if stream is None and _done(_short().attn(3, None, k, v, g, state, None, None, None, None,
                                              slot_idx, None, num_tokens, None)):
        return
    _issue(*_attn_args("commit", None, k, v, g, state, None, num_tokens=num_tokens,
                       slot_idx=slot_idx, stream=stream))


def gated_norm(y, gate, weight, out, *, eps: float = 1e-6, activation: str = "silu",
               gate_first: bool = False, stream=None) -> None:
    """Enqueue out = norm(y) * act(gate), or norm(y * act(gate)) with gate_first, the RMS norm
    (times weight) over the last dimension of y [rows, heads, dim] or [rows, dim].  gate may be
    None, out may be y."""
    act = ACTIVATIONS.get(activation)
    if stream is None and act is not None and _done(
            _short().gated(y, gate, weight, out, eps, act, gate_first)):
        return
    _issue(*_gated_args(y, gate, weight, out, eps=eps, activation=activation,
                        gate_first=gate_first, stream=stream))


def residual_norm(y, residual, pre_weight, out, *, post_weight=None, gate=None,
                  scale: float = 1.0, residual_out=None, eps: float = 1e-6, stream=None) -> None:
    """Enqueue a block's end: r = residual + scale * gate * norm(y) (norm with post_weight only,
    gate [rows, dim], [dim] or None) to residual_out (in place if None), and out = norm(r) with
    pre_weight, the next block's input (out and pre_weight may both be None)."""
    if stream is None and _done(_short().residual(y, residual, pre_weight, out, post_weight, gate,
                                                  scale, residual_out, eps)):
        return
    _issue(*_residual_args(y, residual, pre_weight, out, post_weight=post_weight, gate=gate,
                           scale=scale, residual_out=residual_out, eps=eps, stream=stream))


PREPARE = {
    "linear_attn_prefill": lambda q, k, v, g, state, out, cu_seqlens, **kw: _attn_args(
        "prefill", q, k, v, g, state, out, cu_seqlens=cu_seqlens, **kw),
    "linear_attn_update": lambda *a, **kw: _attn_args("update", *a, **kw),
    "linear_attn_verify": lambda *a, **kw: _attn_args("verify", *a, **kw),
    "linear_attn_commit": lambda k, v, g, state, num_tokens=None, **kw: _attn_args(
        "commit", None, k, v, g, state, None, num_tokens=num_tokens, **kw),
    "gated_norm": _gated_args,
    "residual_norm": _residual_args,
}


def prepared(kind, args, kwargs):
    """A zero-argument callable that issues the same launch again (see prepare)."""
    lib, _dev, fn, cargs, keep = PREPARE[kind](*args, **kwargs)

    def launch():
        rc = fn(*cargs)
        if rc != _lib.CV_OK:
            raise LinAttnError(rc, _linattn.error_message(lib, rc))

    launch.keepalive = keep
    return launch


def linear_attn_describe(call, *args, **kwargs) -> "_linattn.LaLaunchInfo":
    """How a call with these arguments is launched (host only; raises what the call raises).
    call: "prefill", "update", "verify" or "commit", with the arguments of that entry point."""
    if call == "prefill" and kwargs.get("workspace") is None:   # none is made for the asking
        cu = args[6] if len(args) > 6 else kwargs["cu_seqlens"]
        kwargs["workspace"] = cu.new_empty(0)
    lib, _dev, _fn, cargs, _keep = PREPARE["linear_attn_" + call](*args, **kwargs)
    info = _linattn.LaLaunchInfo()
    code = ("prefill", "update", "verify", "commit").index(call)
    rc = lib.linattn_describe(code, cargs[0], ctypes.byref(info))
    if rc != _lib.CV_OK:
        raise LinAttnError(rc, _linattn.error_message(lib, rc))
    return info


def linear_attn_abi_version() -> int:
    return _linattn.load().linattn_abi_version()

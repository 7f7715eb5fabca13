"""The selective state space scan, rotated q and k heads, and the verdict on drafted tokens.

Thin Python binding of the C ABI in include/sequence_ops.h (libseqops.so), in the manner of
linear_attention.py: it marshals torch tensors, passes torch's current HIP stream, and computes
nothing itself.  Calls on torch's current stream that are plainly in order are marshalled by the
call module (csrc/sq_call.cpp); the Python here takes all others, and says what is wrong with those
that are refused.

    selective_scan_prefill(x, dt, A, B, C, state, out, cu_seqlens, max_len=..., ...)
    selective_scan_update(x, dt, A, B, C, state, out, ...)   T new tokens of each row, committed
    selective_scan_verify(x, dt, A, B, C, state, out, ...)   T draft tokens, the state only read
    selective_scan_commit(x, dt, A, B, state, num_tokens, ...)   the accepted drafts folded in
    qk_norm_rotary(q, k, positions, inv_freq, q_out, k_out, ...)
    accept_drafts(tokens, target, uniform, num_tokens, next_token, ...)

The scan's tensors (all on one GPU; x, dt, z, B, C and out bf16 or fp32):
    x, dt, z, out  [n_seq, T, d], or packed [total, d] (prefill); dt before its bias and softplus
    B, C         [n_seq, T, d_state] or [total, d_state]
    A            fp32 [d, d_state], the rates of decay themselves (negative), contiguous
    D, dt_bias   fp32 [d] or None
    state        [n_slots, d, d_state], contiguous below the slot dimension
    slot_idx, has_initial_state, num_tokens: int32 [n_seq] or None; cu_seqlens int32 [n_seq+1]
Innermost dimensions have stride 1, other strides are free.
"""

from __future__ import annotations

import ctypes

from . import _lib, _seqops
from .linear_attention import _dtype_code, _int32_vec, _on_stream, _ptr, _same_gpu, _strides

__all__ = ["selective_scan_prefill", "selective_scan_update", "selective_scan_verify",
           "selective_scan_commit", "selective_scan_describe", "qk_norm_rotary", "accept_drafts",
           "sequence_ops_abi_version", "SeqOpsError"]


class SeqOpsError(RuntimeError):
    """A non-zero return code of the C ABI."""

    def __init__(self, code: int, message: str):
        super().__init__(message)
        self.code = code


def _workspace(need, workspace, handle, dev):
    """The given workspace, or one of the stream that the call runs on: a block that another stream
    gave up may still be in use by what is queued there."""
    import torch

    if need and workspace is None:
        if handle == torch.cuda.current_stream(dev).cuda_stream:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        else:
            with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=dev) if handle
                                   else torch.cuda.default_stream(dev)):
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def _need(lib, need):
    if need < 0:
        raise SeqOpsError(need, _seqops.error_message(lib, need))
    return need


def _scan_args(kind, x, dt, A, B, C, state, out, *, cu_seqlens=None, max_len=None, z=None, D=None,
               dt_bias=None, dt_softplus=True, slot_idx=None, has_initial_state=None,
               num_tokens=None, workspace=None, stream=None):
    """(library, device, function, its arguments, what must stay alive)."""
    import torch

    lib = _seqops.load()
    dev = _same_gpu(state, x, dt, A, B, C, out, z, D, dt_bias, cu_seqlens, slot_idx,
                    has_initial_state, num_tokens, workspace)
    packed = kind == "prefill"
    lead = 1 if packed else 2
    if x.dim() != lead + 1 or B.dim() != lead + 1 or B.shape[:lead] != x.shape[:lead]:
        raise ValueError(f"x and B must be {'[total' if packed else '[n_seq, T'}, channels or states] "
                         f"of the same tokens (x {tuple(x.shape)}, B {tuple(B.shape)})")
    d, d_state = x.shape[-1], B.shape[-1]
    for name, t, like in (("dt", dt, x), ("z", z, x), ("out", out, x), ("C", C, B)):
        if t is not None and t.shape != like.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(like.shape)} is needed")
    for t in (x, dt, z, B, C, out):
        if t is None:
            continue
        if t.dtype != x.dtype:
            raise TypeError("x, dt, z, B, C and out must share one dtype")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("x, dt, z, B, C and out need a contiguous last dimension")
    for name, t, size in (("A", A, (d, d_state)), ("D", D, (d,)), ("dt_bias", dt_bias, (d,))):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != size or
                              not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 {list(size)} tensor")
    if state.dim() != 3 or tuple(state.shape[1:]) != (d, d_state) or \
            (state.shape[0] and not state[0].is_contiguous()):
        raise ValueError(f"state must be [n_slots, {d}, {d_state}], contiguous below the slot "
                         f"dimension (got {tuple(state.shape)})")
    if packed:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must hold n_seq + 1 offsets")
        n_seq, T = cu_seqlens.shape[0] - 1, max(1, int(max_len))
        if T > 2 ** 31 - 1:
            raise ValueError(f"max_len ({T}) is over 2^31 - 1")
        _int32_vec("cu_seqlens", cu_seqlens, n_seq + 1)
        _int32_vec("has_initial_state", has_initial_state, n_seq)
        dims = (0,)
        if x.shape[0] == 0:
            # no tokens at all, though states may start from zeros: the token tensors hold no
            # element to point at, and one token that is neither read nor written stands in
            T = 1
            x, dt, z, B, C, out = (None if t is None else t.new_empty(1, *t.shape[1:])
                                   for t in (x, dt, z, B, C, out))
    else:
        n_seq, T = x.shape[0], x.shape[1]
        _int32_vec("num_tokens", num_tokens, n_seq)
        dims = (0, 1)
    _int32_vec("slot_idx", slot_idx, n_seq)

    def strides(t):
        return (0, 0) if t is None else (0, *_strides(t, dims)) if packed else _strides(t, dims)

    shape = _seqops.SqScanShape(
        n_seq, T, d, d_state, _dtype_code(x), _dtype_code(state), state.shape[0],
        int(bool(dt_softplus)), *strides(x), *strides(dt), *strides(z), *strides(B), *strides(C),
        *strides(out), _strides(state, (0,))[0], x.shape[0] if packed else 0)
    data = _seqops.SqScanData(_ptr(x), _ptr(dt), _ptr(z), _ptr(B), _ptr(C), _ptr(A), _ptr(D),
                              _ptr(dt_bias))
    handle = _on_stream(stream, dev)
    ref, dref = ctypes.byref(shape), ctypes.byref(data)
    if packed:
        workspace, size = _workspace(_need(lib, lib.selscan_prefill_workspace(ref)), workspace,
                                     handle, dev)
        fn, args = lib.selscan_prefill, (ref, dref, _ptr(state), _ptr(slot_idx), _ptr(cu_seqlens),
                                         _ptr(has_initial_state), _ptr(out), _ptr(workspace), size,
                                         handle)
    elif kind == "commit":
        fn, args = lib.selscan_commit, (ref, dref, _ptr(state), _ptr(slot_idx), _ptr(num_tokens),
                                        handle)
    else:
        fn = lib.selscan_update if kind == "update" else lib.selscan_verify
        args = (ref, dref, _ptr(state), _ptr(slot_idx), _ptr(out), handle)
    keep = (shape, data, x, dt, z, B, C, A, D, dt_bias, state, out, cu_seqlens, slot_idx,
            has_initial_state, num_tokens, workspace)
    return lib, dev, fn, args, keep


def _rotary_args(q, k, positions, inv_freq, q_out, k_out, *, q_weight=None, k_weight=None,
                 eps=1e-6, interleaved=False, stream=None):
    import torch

    lib = _seqops.load()
    if (k is None) != (k_out is None) or (k is None and k_weight is not None):
        raise ValueError("k, k_out (and k_weight) go together")
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq go together")
    dev = _same_gpu(q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight)
    if q.dim() != 3 or q_out.shape != q.shape:
        raise ValueError("q and q_out must be [tokens, heads, dim] of one shape")
    tokens, q_heads, dim = q.shape
    if k is not None and (k.dim() != 3 or k.shape[0] != tokens or k.shape[2] != dim or
                          k_out.shape != k.shape):
        raise ValueError(f"k and k_out must be [{tokens}, heads, {dim}] of one shape")
    for t in (q, k, q_out, k_out, q_weight, k_weight):
        if t is not None and t.dtype != q.dtype:
            raise TypeError("q, k, their outs and weights must share one dtype")
    for t in (q, k, q_out, k_out):
        if t is not None and t.stride(-1) != 1 and dim > 1:
            raise ValueError("q, k and their outs need a contiguous channel dimension")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None and (tuple(t.shape) != (dim,) or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous [{dim}] tensor")
    if positions is not None:
        if positions.dtype not in (torch.int32, torch.int64) or tuple(positions.shape) != (tokens,) \
                or not positions.is_contiguous():
            raise ValueError(f"positions must be a contiguous int32 or int64 [{tokens}] tensor")
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous() \
                or 2 * inv_freq.shape[0] > dim:
            raise ValueError(f"inv_freq must be a contiguous float32 tensor of at most {dim // 2}")

    def strides(t):
        return (0, 0) if t is None else _strides(t, (0, 1))

    shape = _seqops.SqRotaryShape(
        tokens, q_heads, 0 if k is None else k.shape[1], dim,
        0 if inv_freq is None else 2 * inv_freq.shape[0], eps, _dtype_code(q), int(bool(interleaved)),
        int(positions is not None and positions.dtype == torch.int64), *strides(q), *strides(k),
        *strides(q_out), *strides(k_out))
    args = (ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
            _ptr(inv_freq), _ptr(q_out), _ptr(k_out), _on_stream(stream, dev))
    return lib, dev, lib.norm_rotary, args, (shape, q, k, q_weight, k_weight, positions, inv_freq,
                                             q_out, k_out)


def _accept_args(tokens, target, uniform, num_tokens, next_token, *, draft=None, parent=None,
                 window_index=None, path=None, slot_idx=None, workspace=None, stream=None):
    import torch

    lib = _seqops.load()
    dev = _same_gpu(target, tokens, uniform, num_tokens, next_token, draft, parent, window_index,
                    path, slot_idx, workspace)
    if target.dim() != 3:
        raise ValueError("target must be [n_seq, T, vocab]")
    n, T, vocab = target.shape
    for name, t in (("tokens", tokens), ("parent", parent), ("path", path)):
        if t is not None and (t.dtype != torch.int32 or tuple(t.shape) != (n, T) or
                              (T > 1 and t.stride(1) != 1)):
            raise ValueError(f"{name} must be int32 [{n}, {T}] with contiguous rows")
    if uniform.dtype != torch.float32 or tuple(uniform.shape) != (n, T) or \
            (T > 1 and uniform.stride(1) != 1):
        raise ValueError(f"uniform must be float32 [{n}, {T}] with contiguous rows")
    for name, t in (("num_tokens", num_tokens), ("next_token", next_token),
                    ("window_index", window_index), ("slot_idx", slot_idx)):
        _int32_vec(name, t, n)
    if draft is not None and tuple(draft.shape) != (n, T - 1, vocab):
        raise ValueError(f"draft must be [{n}, {T - 1}, {vocab}]")
    if draft is not None and parent is not None:
        raise ValueError("a tree (parent) is verified without a draft's probabilities")
    if draft is not None and T == 1:
        draft = None                               # no draft was drawn
    for name, t in (("target", target), ("draft", draft)):
        if t is None:
            continue
        if t.dtype != target.dtype:
            raise TypeError("target and draft must share one dtype")
        if t.stride(2) != 1 and vocab > 1:
            raise ValueError(f"{name} needs a contiguous vocabulary dimension")

    def rows(t):
        return 0 if t is None else _strides(t, (0,))[0]

    shape = _seqops.SqAcceptShape(
        n, T, vocab, _dtype_code(target), rows(tokens), rows(parent), rows(uniform), rows(path),
        *_strides(target, (0, 1)), *((0, 0) if draft is None else _strides(draft, (0, 1))))
    handle = _on_stream(stream, dev)
    ref = ctypes.byref(shape)
    workspace, size = _workspace(_need(lib, lib.accept_drafts_workspace(ref)), workspace, handle, dev)
    args = (ref, _ptr(tokens), _ptr(parent), _ptr(target), _ptr(draft), _ptr(uniform),
            _ptr(slot_idx), _ptr(num_tokens), _ptr(next_token), _ptr(window_index), _ptr(path),
            _ptr(workspace), size, handle)
    return lib, dev, lib.accept_drafts, args, (shape, tokens, parent, target, draft, uniform,
                                               slot_idx, num_tokens, next_token, window_index, path,
                                               workspace)


def _issue(lib, dev, fn, args, keep):
    import torch

    if torch.cuda.current_device() == dev.index:
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != _lib.CV_OK:
        raise SeqOpsError(rc, _seqops.error_message(lib, rc))


_call = None


class _NoCallModule:
    """In the call module's place: every call takes the binding's own way."""

    @staticmethod
    def scan(*args):
        return None

    rotary = accept = scan


def _short():
    """The call module (csrc/sq_call.cpp): the same marshalling in C for calls that are plainly in
    order; it answers None to all others, and they take the way above, as all do without it (it is
    built for one torch and one Python, and the library under both ways is not)."""
    global _call
    if _call is None:
        import torch  # noqa: F401  (its libraries, which the module is linked to)

        try:
            from . import _sqcall as _call
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
    raise SeqOpsError(rc, _seqops.error_message(_seqops.load(), rc))


def selective_scan_prefill(x, dt, A, B, C, state, out, cu_seqlens, *, max_len: int, z=None, D=None,
                           dt_bias=None, dt_softplus: bool = True, slot_idx=None,
                           has_initial_state=None, workspace=None, stream=None) -> None:
    """Enqueue the scan of packed prompts; each row's last state is left in its slot.  max_len >=
    the longest prompt.  workspace: a contiguous uint8 tensor of at least the size that the shape
    needs (allocated here if None)."""
    if stream is None and _done(_short().scan(0, x, dt, A, B, C, state, out, cu_seqlens, max_len, z, D,
                                              dt_bias, dt_softplus, slot_idx, has_initial_state, None,
                                              workspace)):
        return
    _issue(*_scan_args("prefill", x, dt, A, B, C, state, out, cu_seqlens=cu_seqlens, max_len=max_len,
                       z=z, D=D, dt_bias=dt_bias, dt_softplus=dt_softplus, slot_idx=slot_idx,
                       has_initial_state=has_initial_state, workspace=workspace, stream=stream))


def selective_scan_update(x, dt, A, B, C, state, out, *, z=None, D=None, dt_bias=None,
                          dt_softplus: bool = True, slot_idx=None, stream=None) -> None:
    """Enqueue T (1..32) new tokens of each row: out for each, and the state after the last."""
    if stream is None and _done(_short().scan(1, x, dt, A, B, C, state, out, None, None, z, D, dt_bias,
                                              dt_softplus, slot_idx, None, None, None)):
        return
    _issue(*_scan_args("update", x, dt, A, B, C, state, out, z=z, D=D, dt_bias=dt_bias,
                       dt_softplus=dt_softplus, slot_idx=slot_idx, stream=stream))


def selective_scan_verify(x, dt, A, B, C, state, out, *, z=None, D=None, dt_bias=None,
                          dt_softplus: bool = True, slot_idx=None, stream=None) -> None:
    """Enqueue the outputs of T (1..32) draft tokens of each row; the state is only read."""
    if stream is None and _done(_short().scan(2, x, dt, A, B, C, state, out, None, None, z, D, dt_bias,
                                              dt_softplus, slot_idx, None, None, None)):
        return
    _issue(*_scan_args("verify", x, dt, A, B, C, state, out, z=z, D=D, dt_bias=dt_bias,
                       dt_softplus=dt_softplus, slot_idx=slot_idx, stream=stream))


def selective_scan_commit(x, dt, A, B, state, num_tokens=None, *, dt_bias=None,
                          dt_softplus: bool = True, slot_idx=None, stream=None) -> None:
    """Enqueue the commit of the first num_tokens[i] (None: all) tokens of each row to its state."""
    if stream is None and _done(_short().scan(3, x, dt, A, B, None, state, None, None, None, None, None,
                                              dt_bias, dt_softplus, slot_idx, None, num_tokens, None)):
        return
    _issue(*_scan_args("commit", x, dt, A, B, None, state, None, dt_bias=dt_bias,
                       dt_softplus=dt_softplus, slot_idx=slot_idx, num_tokens=num_tokens,
                       stream=stream))


def qk_norm_rotary(q, k, positions, inv_freq, q_out, k_out, *, q_weight=None, k_weight=None,
                   eps: float = 1e-6, interleaved: bool = False, stream=None) -> None:
    """Enqueue the RMS norm (times weight; no norm where the weight is None) of each head of q and k
    [tokens, heads, dim] and the rotation of its first 2 * len(inv_freq) channels by the angles
    positions[t] * inv_freq: of channels i and i + len(inv_freq), or with interleaved 2i and 2i + 1.
    positions int32 or int64 [tokens], inv_freq fp32; both None: no rotation.  k and k_out may both
    be None; q_out may be q, and k_out k."""
    if stream is None and _done(_short().rotary(q, k, positions, inv_freq, q_out, k_out, q_weight,
                                                k_weight, eps, interleaved)):
        return
    _issue(*_rotary_args(q, k, positions, inv_freq, q_out, k_out, q_weight=q_weight,
                         k_weight=k_weight, eps=eps, interleaved=interleaved, stream=stream))


def accept_drafts(tokens, target, uniform, num_tokens, next_token, *, draft=None, parent=None,
                  window_index=None, path=None, slot_idx=None, workspace=None, stream=None) -> None:
    """Enqueue the verdict on each row's drafts tokens[i, 1:] (token 0 is certain) and draw the token
    behind the accepted ones.

    target [n_seq, T, vocab]: the target's probabilities of what follows each token.  draft
    [n_seq, T-1, vocab]: those that drafts 1..T-1 were drawn from, or None (certain drafts: a greedy
    draft model, or a tree of candidates).  parent int32 [n_seq, T]: a tree (-1 for token 0), None:
    a chain.  uniform fp32 [n_seq, T] in [0, 1): uniform[i, t-1] tries draft t, uniform[i, T-1] draws
    the next token.  A draft outside [0, vocab) (a pad) is not tried, a row of a negative slot is not
    written.

    Written, int32: num_tokens [n_seq], 1..T; next_token [n_seq]; window_index [n_seq] (if given), the
    last accepted token's place, as conv_verify_restore takes it; path [n_seq, T] (if given), the
    accepted places, then -1.

    linear_attn_commit and selective_scan_commit fold a row's first num_tokens tokens.  Of a chain those
    are the accepted ones; of a tree they are not: gather the commit's inputs along path first (its -1
    as any place), x.gather(1, path.clamp(min=0)...), and each row starts with its accepted tokens.
    (Both layers' verifies follow a row's tokens in order; a tree goes through them branch by branch.)"""
    if stream is None and _done(_short().accept(tokens, target, uniform, num_tokens, next_token, draft,
                                                parent, window_index, path, slot_idx, workspace)):
        return
    _issue(*_accept_args(tokens, target, uniform, num_tokens, next_token, draft=draft, parent=parent,
                         window_index=window_index, path=path, slot_idx=slot_idx,
                         workspace=workspace, stream=stream))


PREPARE = {
    "selective_scan_prefill": lambda x, dt, A, B, C, state, out, cu_seqlens, **kw: _scan_args(
        "prefill", x, dt, A, B, C, state, out, cu_seqlens=cu_seqlens, **kw),
    "selective_scan_update": lambda *a, **kw: _scan_args("update", *a, **kw),
    "selective_scan_verify": lambda *a, **kw: _scan_args("verify", *a, **kw),
    "selective_scan_commit": lambda x, dt, A, B, state, num_tokens=None, **kw: _scan_args(
        "commit", x, dt, A, B, None, state, None, num_tokens=num_tokens, **kw),
    "qk_norm_rotary": _rotary_args,
    "accept_drafts": _accept_args,
}


def prepared(kind, args, kwargs):
    """A zero-argument callable that issues the same launch again (see prepare)."""
    lib, _dev, fn, cargs, keep = PREPARE[kind](*args, **kwargs)

    def launch():
        rc = fn(*cargs)
        if rc != _lib.CV_OK:
            raise SeqOpsError(rc, _seqops.error_message(lib, rc))

    launch.keepalive = keep
    return launch


def selective_scan_describe(call, *args, **kwargs) -> "_seqops.SqScanInfo":
    """How a call with these arguments is launched (host only; raises what the call raises).
    call: "prefill", "update", "verify" or "commit", with the arguments of that entry point."""
    if call == "prefill" and kwargs.get("workspace") is None:   # none is made for the asking
        cu = args[7] if len(args) > 7 else kwargs["cu_seqlens"]
        kwargs["workspace"] = cu.new_empty(0)
    lib, _dev, _fn, cargs, _keep = PREPARE["selective_scan_" + call](*args, **kwargs)
    info = _seqops.SqScanInfo()
    code = ("prefill", "update", "verify", "commit").index(call)
    rc = lib.selscan_describe(code, cargs[0], ctypes.byref(info))
    if rc != _lib.CV_OK:
        raise SeqOpsError(rc, _seqops.error_message(lib, rc))
    return info


def sequence_ops_abi_version() -> int:
    return _seqops.load().seqops_abi_version()

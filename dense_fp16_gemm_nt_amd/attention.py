"""Attention beside the products: ctypes binding of ``include/attention.h``.

``attention_prompt`` attends over whole prompts packed without padding,
``attention_shared_prefix`` over one new token for each sequence of a batch
with a common prefix.  Both take fp16 or bf16 device tensors, check their
metadata, pass device pointers and the current HIP stream, and raise on a
non-zero status.  Lengths and offsets stay on the device: neither call
synchronises.
"""
from __future__ import annotations

import ctypes
import math

F16 = 0
BF16 = 1


class PromptDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("dtype", "causal", "heads", "kv_heads", "head_dim", "batch")]
                + [(n, ctypes.c_int64) for n in ("total_q", "total_k")]
                + [(n, ctypes.c_void_p) for n in ("Q", "K", "V", "O", "lse", "cu_q", "cu_k")]
                + [(n, ctypes.c_int64) for n in ("q_row", "q_head", "k_row", "k_head", "v_row", "v_head", "o_row", "o_head")]
                + [("scale", ctypes.c_float)])


class SharedPrefixDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("dtype", "heads", "kv_heads", "head_dim")]
                + [(n, ctypes.c_int64) for n in ("batch", "prefix", "slot_rows")]
                + [(n, ctypes.c_void_p) for n in ("Q", "Kp", "Vp", "Ks", "Vs", "O", "lse", "lens")]
                + [(n, ctypes.c_int64) for n in ("q_row", "q_head", "kp_row", "kp_head", "vp_row", "vp_head", "ks_slot",
                                                 "ks_row", "ks_head", "vs_slot", "vs_row", "vs_head", "o_row", "o_head")]
                + [("scale", ctypes.c_float)])


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the attention entry points of the library."""
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name, desc in (("attn_prompt", PromptDesc), ("attn_shared_prefix", SharedPrefixDesc)):
        p = ctypes.POINTER(desc)
        f = getattr(L, name)
        f.restype, f.argtypes = i32, [p, vp, i64, vp]
        f = getattr(L, name + "_workspace")
        f.restype, f.argtypes = i64, [p]
        f = getattr(L, name + "_check")
        f.restype, f.argtypes = i32, [p]


def _dtype(Q):
    import torch

    if Q.dtype == torch.float16:
        return F16
    if Q.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"attention takes torch.float16 or torch.bfloat16, not {Q.dtype}")


def _like(Q, name, X, dim):
    """X is a device tensor of Q's type and device with `dim` dimensions, the last contiguous."""
    if X.dtype != Q.dtype:
        raise TypeError(f"{name} must be {Q.dtype} like Q, not {X.dtype}")
    if X.device != Q.device:
        raise ValueError(f"{name} is on {X.device}, Q on {Q.device}")
    if X.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions; got {tuple(X.shape)}")
    if X.stride(-1) != 1 and X.shape[-1] > 1:
        raise ValueError(f"{name}: last dimension must be contiguous")


def _ints(Q, name, X, n):
    import torch

    if X.dtype != torch.int32:
        raise TypeError(f"{name} must be torch.int32")
    if X.device != Q.device or X.dim() != 1 or (n is not None and X.numel() != n) or not X.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor{'' if n is None else f' of {n} values'} on {Q.device}")


def _strides(X):
    """Strides of the dimensions before the last; 0 where a dimension has one entry and its stride says nothing."""
    return [s if n > 1 else 0 for n, s in zip(X.shape[:-1], X.stride()[:-1])]


def _heads(H, Hk):
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"{H} query heads do not divide among {Hk} key/value heads")


def _scale(scale, d):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _outputs(Q, O, lse, return_lse):
    import torch

    if O is None:
        O = torch.empty(Q.shape, dtype=Q.dtype, device=Q.device)
    else:
        _like(Q, "O", O, 3)
        if O.shape != Q.shape:
            raise ValueError(f"O must be {tuple(Q.shape)}; got {tuple(O.shape)}")
    if lse is None:
        if return_lse:
            lse = torch.empty(Q.shape[:2], dtype=torch.float32, device=Q.device)
    elif lse.dtype != torch.float32 or lse.shape != Q.shape[:2] or not lse.is_contiguous() or lse.device != Q.device:
        raise ValueError(f"lse must be a contiguous float32 {tuple(Q.shape[:2])} tensor on {Q.device}")
    return O, lse


def _call(name, desc, Q, workspace):
    """Runs an entry point on Q's device and current stream, with a workspace if it needs one."""
    import torch

    from . import OK, GemmError, lib

    L = lib()
    ref = ctypes.byref(desc)
    dev = Q.device
    if dev.index != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(name, desc, Q, workspace)
    need = getattr(L, name + "_workspace")(ref)
    if need < 0:
        raise GemmError(int(need), name)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    ws, have = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel() * workspace.element_size())
    st = getattr(L, name)(ref, ws, have, torch.cuda.current_stream(dev).cuda_stream)
    if st != OK:
        raise GemmError(st, name)


def _workspace_bytes(name, desc, Q):
    import torch

    from . import GemmError, lib

    with torch.cuda.device(Q.device):
        n = getattr(lib(), name + "_workspace")(ctypes.byref(desc))
    if n < 0:
        raise GemmError(int(n), name + "_workspace")
    return int(n)


def _prompt_desc(Q, K, V, cu_q, cu_k, causal, scale, O, lse):
    dtype = _dtype(Q)
    if not Q.is_cuda:
        raise ValueError("Q must be a device tensor")
    _like(Q, "Q", Q, 3)
    _like(Q, "K", K, 3)
    _like(Q, "V", V, 3)
    Tq, H, d = Q.shape
    Tk, Hk, dk = K.shape
    if dk != d or V.shape != K.shape:
        raise ValueError(f"Q, K and V do not match: {tuple(Q.shape)}, {tuple(K.shape)}, {tuple(V.shape)}")
    _heads(H, Hk)
    _ints(Q, "cu_q", cu_q, None)
    if cu_q.numel() < 1:
        raise ValueError("cu_q needs a value more than there are sequences")
    _ints(Q, "cu_k", cu_k, cu_q.numel())
    qs, ks, vs, os = _strides(Q), _strides(K), _strides(V), _strides(O)
    return PromptDesc(dtype, int(bool(causal)), H, Hk, d, cu_q.numel() - 1, Tq, Tk, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                      O.data_ptr(), None if lse is None else lse.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
                      qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1], _scale(scale, d))


def attention_prompt(Q, K, V, cu_q, cu_k=None, *, causal=True, scale=None, O=None, lse=None, return_lse=False, workspace=None):
    """softmax(scale * Q K^T) V for sequences packed along the first dimension.

    Q (tokens, heads, d) and K, V (key tokens, kv heads, d), fp16 or bf16, any
    strides the C-ABI takes (so views of a fused projection work); heads is a
    multiple of kv heads, d a multiple of 8 up to 128.  Sequence b has the
    query rows cu_q[b] .. cu_q[b+1] and the key rows cu_k[b] .. cu_k[b+1]
    (int32 device tensors; cu_k defaults to cu_q).  With `causal`, query i of n
    reads keys j <= i + (keys - n).  `scale` defaults to 1 / sqrt(d).

    Returns O (tokens, heads, d), or (O, lse) with `return_lse`: lse (tokens,
    heads) fp32 is the natural log-sum-exp of a row's scaled scores.  Rows
    without a key get 0 and -inf; rows of no sequence are left as they were in
    O and lse, where those are given (O and lse allocated here hold arbitrary
    values there).  `workspace`: a device tensor of at least
    attention_prompt_workspace(...) bytes, 16-byte aligned; allocated here
    when not given."""
    O, lse = _outputs(Q, O, lse, return_lse)
    desc = _prompt_desc(Q, K, V, cu_q, cu_q if cu_k is None else cu_k, causal, scale, O, lse)
    _call("attn_prompt", desc, Q, workspace)
    return (O, lse) if return_lse else O


def attention_prompt_workspace(Q, K, V, cu_q, cu_k=None) -> int:
    """Bytes of workspace attention_prompt needs for tensors of these shapes (0: none)."""
    desc = _prompt_desc(Q, K, V, cu_q, cu_q if cu_k is None else cu_k, True, None, Q, None)
    desc.O, desc.o_row, desc.o_head = 16, desc.heads * desc.head_dim, desc.head_dim   # no output is looked at
    return _workspace_bytes("attn_prompt", desc, Q)


def _shared_desc(Q, Kp, Vp, Ks, Vs, lens, scale, O, lse):
    dtype = _dtype(Q)
    if not Q.is_cuda:
        raise ValueError("Q must be a device tensor")
    _like(Q, "Q", Q, 3)
    for name, X, dim in (("Kp", Kp, 3), ("Vp", Vp, 3), ("Ks", Ks, 4), ("Vs", Vs, 4)):
        _like(Q, name, X, dim)
    B, H, d = Q.shape
    P, Hk, dk = Kp.shape
    N = Ks.shape[1]
    if dk != d or Vp.shape != Kp.shape or tuple(Ks.shape) != (B, N, Hk, d) or Vs.shape != Ks.shape:
        raise ValueError(f"Q, Kp, Vp, Ks and Vs do not match: {[tuple(X.shape) for X in (Q, Kp, Vp, Ks, Vs)]}")
    _heads(H, Hk)
    _ints(Q, "lens", lens, B)
    q, kp, vp, ks, vs, o = (_strides(X) for X in (Q, Kp, Vp, Ks, Vs, O))
    return SharedPrefixDesc(dtype, H, Hk, d, B, P, N, Q.data_ptr(), Kp.data_ptr(), Vp.data_ptr(), Ks.data_ptr(),
                            Vs.data_ptr(), O.data_ptr(), None if lse is None else lse.data_ptr(), lens.data_ptr(),
                            q[0], q[1], kp[0], kp[1], vp[0], vp[1], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], o[0], o[1],
                            _scale(scale, d))


def attention_shared_prefix(Q, Kp, Vp, Ks, Vs, lens, *, scale=None, O=None, lse=None, return_lse=False, workspace=None):
    """One new token for each sequence of a batch behind a common prefix.

    Row b of Q (batch, heads, d) attends to all rows of Kp, Vp (prefix, kv
    heads, d), which are read once for the whole batch, and to the first
    lens[b] rows of its slot of Ks, Vs (batch, slot rows, kv heads, d), any
    strides the C-ABI takes (a cache laid out head by head is passed as its
    transposed view).  lens: int32 device tensor; more than a slot's rows
    counts as all of them, and a negative length says that the slot is not in
    use: its row of O and lse is left as it was.

    Returns O (batch, heads, d), or (O, lse) with `return_lse`, as
    attention_prompt does, with the same `scale`, `O`, `lse` and `workspace`
    (attention_shared_prefix_workspace(...) bytes)."""
    O, lse = _outputs(Q, O, lse, return_lse)
    desc = _shared_desc(Q, Kp, Vp, Ks, Vs, lens, scale, O, lse)
    _call("attn_shared_prefix", desc, Q, workspace)
    return (O, lse) if return_lse else O


def attention_shared_prefix_workspace(Q, Kp, Vp, Ks, Vs, lens) -> int:
    """Bytes of workspace attention_shared_prefix needs for tensors of these shapes (0: none)."""
    desc = _shared_desc(Q, Kp, Vp, Ks, Vs, lens, None, Q, None)
    desc.O, desc.o_row, desc.o_head = 16, desc.heads * desc.head_dim, desc.head_dim   # no output is looked at
    return _workspace_bytes("attn_shared_prefix", desc, Q)

"""Attention beside the products: ctypes binding of ``include/attention.h``.

``attention_prompt`` attends over whole prompts packed without padding,
``attention_shared_prefix`` over one new token for each sequence of a batch
with a common prefix.  Both take fp16 or bf16 device tensors, check their
metadata, pass device pointers and the current HIP stream, and raise on a
non-zero status.  Lengths and offsets stay on the device: neither call
synchronises.  Neither has a gradient: results are not part of an autograd
graph.
"""
from __future__ import annotations

import ctypes
import math
import struct

from . import OK, GemmError, lib

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


def _packer(desc):
    """The descriptor's layout as a struct.Struct: packing its fields into bytes takes a fifth of the time of building
    the ctypes.Structure, which is most of what a small call costs on the host."""
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_float: "f"}
    return struct.Struct("@" + "".join(codes[t] for _, t in desc._fields_)).pack


_pack_prompt, _pack_shared_prefix = _packer(PromptDesc), _packer(SharedPrefixDesc)


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the attention entry points of the library; descriptors are passed as their bytes or by reference."""
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name in ("attn_prompt", "attn_shared_prefix"):
        f = getattr(L, name)
        f.restype, f.argtypes = i32, [vp, vp, i64, vp]
        f = getattr(L, name + "_workspace")
        f.restype, f.argtypes = i64, [vp]
        f = getattr(L, name + "_check")
        f.restype, f.argtypes = i32, [vp]


_torch = None


def _module():
    """torch, which the package loads with the first call that needs it.  Not by an import statement in each function:
    with those and a second look at tensors made here a call of 128 tokens took 10.6 us on the host instead of 9.7."""
    global _torch
    import torch

    _torch = torch
    return torch


def _query(Q):
    """Type code and device of Q."""
    torch = _torch or _module()
    dtype = Q.dtype
    if dtype is torch.float16:
        code = F16
    elif dtype is torch.bfloat16:
        code = BF16
    else:
        raise TypeError(f"attention takes torch.float16 or torch.bfloat16, not {dtype}")
    if not Q.is_cuda:
        raise ValueError("Q must be a device tensor")
    if Q.dim() != 3:
        raise ValueError(f"Q must have 3 dimensions; got {tuple(Q.shape)}")
    return code, Q.device


def _strides(name, X, shape, dtype, device):
    """Strides of a tensor that has to have this shape and type, as _steps has them."""
    if X.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} like Q, not {X.dtype}")
    if X.device != device:
        raise ValueError(f"{name} is on {X.device}, Q on {device}")
    if X.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}; got {tuple(X.shape)}")
    return _steps(name, X, shape)


def _steps(name, X, shape):
    """Strides of the dimensions before the last, which has to be contiguous; 0 where a dimension has one entry and its
    stride says nothing."""
    *st, last = X.stride()
    if last != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    return st if min(shape) > 1 else [s if n > 1 else 0 for n, s in zip(shape, st)]


def _ints(name, X, n, device):
    if X.dtype is not (_torch or _module()).int32:
        raise TypeError(f"{name} must be torch.int32")
    if X.device != device or X.shape != (n,) or not X.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} values on {device}")
    return X.data_ptr()


def _heads(H, Hk):
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"{H} query heads do not divide among {Hk} key/value heads")


def _scale(scale, d):
    if scale is None:
        return 1.0 / math.sqrt(d) if d else 1.0   # heads without elements are refused by the library
    scale = float(scale)
    return scale if abs(scale) < 3.4e38 else math.inf   # what fp32 does not hold is refused by the library


def _outputs(Q, O, lse, return_lse):
    """(O, lse), allocated where they are not given; lse may be None."""
    torch = _torch or _module()
    if O is None:
        O = torch.empty_like(Q) if Q.is_contiguous() else torch.empty_like(Q, memory_format=torch.contiguous_format)
    if lse is None:
        if return_lse:
            lse = torch.empty(tuple(Q.shape)[:2], dtype=torch.float32, device=Q.device)   # a slice of a torch.Size costs 0.5 us
    elif lse.dtype != torch.float32 or lse.shape != Q.shape[:2] or not lse.is_contiguous() or lse.device != Q.device:
        raise ValueError(f"lse must be a contiguous float32 {tuple(Q.shape[:2])} tensor on {Q.device}")
    return O, lse


_entries = {}   # name -> (entry point, its workspace query) of the loaded library


def _call(name, desc, device, workspace):
    """Runs an entry point on a device's current stream, with a workspace if it needs one."""
    torch = _torch or _module()
    if device.index != torch.cuda.current_device():   # launches go to the current device
        with torch.cuda.device(device):
            return _call(name, desc, device, workspace)
    if name not in _entries:
        L = lib()
        _entries[name] = getattr(L, name), getattr(L, name + "_workspace")
    run, size = _entries[name]
    ws, have = None, 0
    if workspace is None:
        have = size(desc)
        if have < 0:
            raise GemmError(int(have), name)
        if have:
            workspace = torch.empty(have, dtype=torch.uint8, device=device)
            ws = workspace.data_ptr()
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    else:
        ws, have = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = run(desc, ws, have, torch._C._cuda_getCurrentRawStream(device.index))
    if st != OK:
        raise GemmError(st, name)


def _workspace_bytes(name, desc, device):
    with (_torch or _module()).cuda.device(device):
        n = getattr(lib(), name + "_workspace")(desc)
    if n < 0:
        raise GemmError(int(n), name + "_workspace")
    return int(n)


def _prompt_desc(Q, K, V, cu_q, cu_k, causal, scale, O, lse, given):
    """Descriptor bytes and device; an O that was not given is contiguous, and without one the address is one that no
    tensor has."""
    code, device = _query(Q)
    dtype, shape = Q.dtype, Q.shape
    Tq, H, d = shape
    if K.dim() != 3:
        raise ValueError(f"K must have 3 dimensions; got {tuple(K.shape)}")
    kv = K.shape
    Tk, Hk, dk = kv
    if dk != d:
        raise ValueError(f"Q and K do not match: {tuple(shape)}, {tuple(kv)}")
    _heads(H, Hk)
    n = cu_q.numel()
    if n < 1:
        raise ValueError("cu_q needs a value more than there are sequences")
    cq = _ints("cu_q", cu_q, n, device)
    ck = cq if cu_k is cu_q else _ints("cu_k", cu_k, n, device)
    qs, ks, vs = _steps("Q", Q, shape), _strides("K", K, kv, dtype, device), _strides("V", V, kv, dtype, device)
    os = _strides("O", O, shape, dtype, device) if given else (H * d, d)
    return _pack_prompt(code, 1 if causal else 0, H, Hk, d, n - 1, Tq, Tk, Q.data_ptr(), K.data_ptr(), V.data_ptr(),
                        16 if O is None else O.data_ptr(), 0 if lse is None else lse.data_ptr(), cq, ck, *qs, *ks, *vs, *os, _scale(scale, d)), device


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
    given = O is not None
    O, lse = _outputs(Q, O, lse, return_lse)
    desc, device = _prompt_desc(Q, K, V, cu_q, cu_q if cu_k is None else cu_k, causal, scale, O, lse, given)
    _call("attn_prompt", desc, device, workspace)
    return (O, lse) if return_lse else O


def attention_prompt_workspace(Q, K, V, cu_q, cu_k=None, *, causal=None) -> int:
    """Bytes of workspace attention_prompt needs for tensors of these shapes (0: none): with a causal mask, without one,
    or, when `causal` is not given, enough for either."""
    masks = (True, False) if causal is None else (causal,)
    return max(_workspace_bytes("attn_prompt", *_prompt_desc(Q, K, V, cu_q, cu_q if cu_k is None else cu_k, m, None, None, None, False))
               for m in masks)


def _shared_desc(Q, Kp, Vp, Ks, Vs, lens, scale, O, lse, given):
    code, device = _query(Q)
    dtype, shape = Q.dtype, Q.shape
    B, H, d = shape
    if Kp.dim() != 3 or Ks.dim() != 4:
        raise ValueError(f"Kp must have 3 and Ks 4 dimensions; got {tuple(Kp.shape)} and {tuple(Ks.shape)}")
    kv, own = Kp.shape, Ks.shape
    P, Hk, dk = kv
    N = own[1]
    if dk != d or own != (B, N, Hk, d):
        raise ValueError(f"Q, Kp and Ks do not match: {tuple(shape)}, {tuple(kv)}, {tuple(own)}")
    _heads(H, Hk)
    ln = _ints("lens", lens, B, device)
    q, kp, vp = _steps("Q", Q, shape), _strides("Kp", Kp, kv, dtype, device), _strides("Vp", Vp, kv, dtype, device)
    ks, vs = _strides("Ks", Ks, own, dtype, device), _strides("Vs", Vs, own, dtype, device)
    os = _strides("O", O, shape, dtype, device) if given else (H * d, d)
    return _pack_shared_prefix(code, H, Hk, d, B, P, N, Q.data_ptr(), Kp.data_ptr(), Vp.data_ptr(), Ks.data_ptr(),
                               Vs.data_ptr(), 16 if O is None else O.data_ptr(), 0 if lse is None else lse.data_ptr(), ln, *q, *kp, *vp, *ks, *vs, *os,
                               _scale(scale, d)), device


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
    given = O is not None
    O, lse = _outputs(Q, O, lse, return_lse)
    desc, device = _shared_desc(Q, Kp, Vp, Ks, Vs, lens, scale, O, lse, given)
    _call("attn_shared_prefix", desc, device, workspace)
    return (O, lse) if return_lse else O


def attention_shared_prefix_workspace(Q, Kp, Vp, Ks, Vs, lens) -> int:
    """Bytes of workspace attention_shared_prefix needs for tensors of these shapes (0: none)."""
    return _workspace_bytes("attn_shared_prefix", *_shared_desc(Q, Kp, Vp, Ks, Vs, lens, None, None, None, False))

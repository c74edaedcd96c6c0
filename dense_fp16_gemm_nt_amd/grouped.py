"""Products of many matrices in one call: ctypes binding of ``include/grouped.h``.

``grouped_product`` multiplies rows that are sorted by the matrix they go
through (a layer of experts), ``grouped_product_grad_input`` and
``grouped_product_grad_weight`` are its gradients, and ``adapter_product`` is
one projection for all rows with the low-rank adapters of many requests beside
it.  All take fp16 or bf16 device tensors, check their metadata, pass device
pointers and the current HIP stream, and raise on a non-zero status.  Offsets
stay on the device: no call synchronises.  None is part of an autograd graph.
"""
from __future__ import annotations

import ctypes
import struct

from . import OK, GemmError, lib

F16 = 0
BF16 = 1


class GroupedDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("dtype", "b_fp32")]
                + [(n, ctypes.c_int64) for n in ("groups", "rows", "N", "K")]
                + [(n, ctypes.c_void_p) for n in ("A", "B", "D")]
                + [(n, ctypes.c_int64) for n in ("lda", "ldb", "stride_b", "ldd")]
                + [("cu", ctypes.c_void_p)])


class AdapterDesc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("dtype", "rank")]
                + [(n, ctypes.c_int64) for n in ("adapters", "requests", "rows", "N", "K")]
                + [(n, ctypes.c_void_p) for n in ("A", "B", "D", "down", "up", "scales", "cu", "ids")]
                + [(n, ctypes.c_int64) for n in ("lda", "ldb", "ldd", "ld_down", "stride_down", "ld_up", "stride_up")])


def _packer(desc):
    """The descriptor's layout as a struct.Struct: packing bytes takes a fifth of the time of a ctypes.Structure."""
    codes = {ctypes.c_int32: "i", ctypes.c_int64: "q", ctypes.c_void_p: "P"}
    return struct.Struct("@" + "".join(codes[t] for _, t in desc._fields_)).pack


_pack_grouped, _pack_adapter = _packer(GroupedDesc), _packer(AdapterDesc)


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the entry points of the library; descriptors are passed as their bytes or by reference."""
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    for name in ("grouped_nt", "grouped_nn", "grouped_tn", "adapter_nt"):
        f = getattr(L, name)
        f.restype, f.argtypes = i32, [vp, vp, i64, vp]
        f = getattr(L, name + "_workspace")
        f.restype, f.argtypes = i64, [vp]
        f = getattr(L, name + "_check")
        f.restype, f.argtypes = i32, [vp]
    ip, i64p = ctypes.POINTER(i32), ctypes.POINTER(i64)
    L.gemm_f16_nt_grouped_plan.restype, L.gemm_f16_nt_grouped_plan.argtypes = i32, [vp, i32, i32, ip, i64p]
    L.gemm_f16_nt_adapter_plan.restype, L.gemm_f16_nt_adapter_plan.argtypes = i32, [vp, i32, ip, ip, i64p, ip, i64p]


def plan(product: str, desc: GroupedDesc, cus: int):
    """(tile rows, tile columns, parts of the contraction) that "nt", "nn" or "tn" runs with on a device with `cus` compute
    units (host evaluation, no GPU needed); 0 parts: the device divides a small last round of large tiles."""
    tile, parts = (ctypes.c_int * 2)(), ctypes.c_int64()
    st = lib().gemm_f16_nt_grouped_plan(ctypes.byref(desc), ("nt", "nn", "tn").index(product), int(cus), tile, ctypes.byref(parts))
    if st != OK:
        raise GemmError(st, "gemm_f16_nt_grouped_plan")
    return tile[0], tile[1], parts.value


ONE_LAUNCH, DOTS, SUMS, TILES, EACH = 1, 2, 3, 4, 5   # ways of an adapter_nt call


def adapter_plan(desc: AdapterDesc, cus: int):
    """(way, (tile rows, tile columns, parts), the same of the projections) of an adapter_nt call, as `plan`."""
    way, tile, low, parts, low_parts = ctypes.c_int(), (ctypes.c_int * 2)(), (ctypes.c_int * 2)(), ctypes.c_int64(), ctypes.c_int64()
    st = lib().gemm_f16_nt_adapter_plan(ctypes.byref(desc), int(cus), ctypes.byref(way), tile, ctypes.byref(parts), low, ctypes.byref(low_parts))
    if st != OK:
        raise GemmError(st, "gemm_f16_nt_adapter_plan")
    return way.value, (tile[0], tile[1], parts.value), (low[0], low[1], low_parts.value)


_torch = None


def _module():
    """torch, which the package loads with the first call that needs it (and not by an import statement in each function,
    which is slower)."""
    global _torch
    import torch

    _torch = torch
    return torch


def _first(name, X, dims):
    """Type code, type and device of the tensor that the others have to match."""
    torch = _torch or _module()
    dtype = X.dtype
    code = F16 if dtype is torch.float16 else BF16 if dtype is torch.bfloat16 else None
    if code is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, not {dtype}")
    if not X.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if X.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions; got {tuple(X.shape)}")
    return code, dtype, X.device


def _rows(name, X, shape, dtype, device):
    """Elements from a row to the next of a 2-D tensor that has to have this shape and type."""
    st = X.stride()
    if X.shape == shape and st[1] == 1 and st[0] >= shape[1] > 0 and shape[0] > 1 and X.dtype is dtype and X.device == device:
        return st[0]
    return _explain(name, X, shape, dtype, device)[-1]


def _matrices(name, X, shape, dtype, device):
    """Elements from a row to the next, and from a matrix to the next, of a 3-D tensor that has to have this shape and type."""
    st = X.stride()
    if X.shape == shape and st[2] == 1 and st[1] >= shape[2] > 0 and shape[1] > 1 and shape[0] > 1 and X.dtype is dtype and X.device == device:
        return st[1], st[0]
    between, ld = _explain(name, X, shape, dtype, device)
    return ld, between


def _explain(name, X, shape, dtype, device):
    """(stride of the first dimension, row pitch), where a look at the tensor does not settle them: says what is wrong, and
    leaves out strides of dimensions with one entry, which say nothing."""
    if X.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, not {X.dtype}")
    if X.device != device:
        raise ValueError(f"{name} is on {X.device}, the other tensors on {device}")
    if X.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}; got {tuple(X.shape)}")
    st, width, there = X.stride(), shape[-1], X.numel() > 0
    if there and width > 1 and st[-1] != 1:
        raise ValueError(f"{name}: last dimension must be contiguous")
    ld = width
    if there and shape[-2] > 1:
        ld = st[-2]
        if ld < width:
            raise ValueError(f"{name}: rows must not overlap")
    return st[0] if there and shape[0] > 1 else shape[-2] * ld, ld


def _ints(name, X, n, device):
    if X.dtype is not _torch.int32:
        raise TypeError(f"{name} must be torch.int32")
    if X.device != device or X.shape != (n,) or not X.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} values on {device}")
    return X.data_ptr()


_entries = {}   # name -> (entry point, its workspace query) of the loaded library


def _run(name, desc, device, workspace):
    """Runs an entry point on a device's current stream, with a workspace if it needs one."""
    torch = _torch or _module()
    if device.index != torch.cuda.current_device():   # launches go to the current device
        with torch.cuda.device(device):
            return _run(name, desc, device, workspace)
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


def _groups(cu):
    n = cu.numel()
    if n < 1:
        raise ValueError("cu needs a value more than there are groups")
    return n - 1


def _product_desc(A, B, cu, D):
    """Descriptor bytes and device; without a D its address is one that no tensor has."""
    code, dtype, device = _first("A", A, 2)
    rows, K = A.shape
    if B.dim() != 3:
        raise ValueError(f"B must have 3 dimensions; got {tuple(B.shape)}")
    G, N = _groups(cu), B.shape[1]
    ldb, sb = _matrices("B", B, (G, N, K), dtype, device)
    return _pack_grouped(code, 0, G, rows, N, K, A.data_ptr(), B.data_ptr(), 16 if D is None else D.data_ptr(),
                         _rows("A", A, (rows, K), dtype, device), ldb, sb, N if D is None else _rows("D", D, (rows, N), dtype, device),
                         _ints("cu", cu, G + 1, device)), device


def grouped_product(A, B, cu, *, D=None, workspace=None):
    """D[r] = B[e] @ A[r] for the rows r = cu[e] .. cu[e + 1] - 1 of each group e.

    A (rows, K) and B (groups, N, K), fp16 or bf16, last dimensions contiguous,
    other strides as the C-ABI takes them; cu: groups + 1 int32 offsets on the
    device, not decreasing.  N and K are multiples of 8.  Returns D (rows, N).
    Rows of no group are left as they were in a given D (one allocated here
    holds arbitrary values there).  `workspace`: a device tensor of at least
    grouped_product_workspace(...) bytes, 16-byte aligned; allocated here when
    not given."""
    if D is None and A.dim() == 2 and B.dim() == 3:   # other tensors are refused below
        D = A.new_empty(A.shape[0], B.shape[1])
    _run("grouped_nt", *_product_desc(A, B, cu, D), workspace)
    return D


def grouped_product_workspace(A, B, cu) -> int:
    """Bytes of workspace grouped_product needs for tensors of these shapes (0: none)."""
    return _workspace_bytes("grouped_nt", *_product_desc(A, B, cu, None))


def _grad_input_desc(G, B, cu, dA):
    code, dtype, device = _first("G", G, 2)
    rows, N = G.shape
    if B.dim() != 3:
        raise ValueError(f"B must have 3 dimensions; got {tuple(B.shape)}")
    groups, K = _groups(cu), B.shape[2]
    ldb, sb = _matrices("B", B, (groups, N, K), dtype, device)
    return _pack_grouped(code, 0, groups, rows, N, K, 16 if dA is None else dA.data_ptr(), B.data_ptr(), G.data_ptr(),
                         K if dA is None else _rows("dA", dA, (rows, K), dtype, device), ldb, sb, _rows("G", G, (rows, N), dtype, device),
                         _ints("cu", cu, groups + 1, device)), device


def grouped_product_grad_input(G, B, cu, *, dA=None, workspace=None):
    """The gradient of grouped_product for A: dA[r] = B[e].T @ G[r], G (rows, N)
    being the gradient for D and B (groups, N, K) the matrices.  Returns dA
    (rows, K); rows of no group are left as they were in a given dA.
    `workspace` as for grouped_product."""
    if dA is None and G.dim() == 2 and B.dim() == 3:   # other tensors are refused below
        dA = G.new_empty(G.shape[0], B.shape[2])
    _run("grouped_nn", *_grad_input_desc(G, B, cu, dA), workspace)
    return dA


def grouped_product_grad_input_workspace(G, B, cu) -> int:
    """Bytes of workspace grouped_product_grad_input needs for tensors of these shapes (0: none)."""
    return _workspace_bytes("grouped_nn", *_grad_input_desc(G, B, cu, None))


def _grad_weight_desc(G, A, cu, dB, dtype):
    code, own, device = _first("G", G, 2)
    rows, N = G.shape
    if A.dim() != 2:
        raise ValueError(f"A must have 2 dimensions; got {tuple(A.shape)}")
    groups, K = _groups(cu), A.shape[1]
    if dtype is not own and dtype is not _torch.float32:
        raise TypeError(f"dB must be {own} or torch.float32, not {dtype}")
    ldb, sb = K, N * K
    if dB is not None:
        ldb, sb = _matrices("dB", dB, (groups, N, K), dtype, device)
    return _pack_grouped(code, 0 if dtype is own else 1, groups, rows, N, K, A.data_ptr(), 16 if dB is None else dB.data_ptr(), G.data_ptr(),
                         _rows("A", A, (rows, K), own, device), ldb, sb, _rows("G", G, (rows, N), own, device),
                         _ints("cu", cu, groups + 1, device)), device


def grouped_product_grad_weight(G, A, cu, *, dB=None, dtype=None, workspace=None):
    """The gradient of grouped_product for B: dB[e] = sum of the outer products
    of G[r] and A[r] over the rows of group e (zeros without rows), G (rows, N)
    being the gradient for D and A (rows, K) its input.  Returns dB (groups, N,
    K) in the operands' type, or in torch.float32 where `dtype` or a given dB
    says so.  `workspace` as for grouped_product."""
    if dtype is None:
        dtype = G.dtype if dB is None else dB.dtype
    if dB is None and G.dim() == 2 and A.dim() == 2 and dtype in (G.dtype, (_torch or _module()).float32):   # others are refused below
        dB = G.new_empty(_groups(cu), G.shape[1], A.shape[1], dtype=dtype)
    _run("grouped_tn", *_grad_weight_desc(G, A, cu, dB, dtype), workspace)
    return dB


def grouped_product_grad_weight_workspace(G, A, cu, *, dtype=None) -> int:
    """Bytes of workspace grouped_product_grad_weight needs for tensors of these shapes (0: none), and a dB, if one is given,
    whose rows begin less than 2^21 elements apart."""
    return _workspace_bytes("grouped_tn", *_grad_weight_desc(G, A, cu, None, G.dtype if dtype is None else dtype))


def _adapter_desc(A, B, down, up, cu, adapters, scales, D):
    """As _product_desc."""
    code, dtype, device = _first("A", A, 2)
    rows, K = A.shape
    if B.dim() != 2 or down.dim() != 3 or up.dim() != 3:
        raise ValueError(f"B must have 2, down and up 3 dimensions; got {tuple(B.shape)}, {tuple(down.shape)}, {tuple(up.shape)}")
    N, (count, rank, _), requests = B.shape[0], down.shape, _groups(cu)
    ldb = _rows("B", B, (N, K), dtype, device)
    ldn, sdn = _matrices("down", down, (count, rank, K), dtype, device)
    lup, sup = _matrices("up", up, (count, N, rank), dtype, device)
    factors = 0
    if scales is not None:
        if scales.dtype is not _torch.float32 or scales.device != device or scales.shape != (count,) or not scales.is_contiguous():
            raise ValueError(f"scales must be a contiguous float32 tensor of {count} values on {device}")
        factors = scales.data_ptr()
    desc = _pack_adapter(code, rank, count, requests, rows, N, K, A.data_ptr(), B.data_ptr(), 16 if D is None else D.data_ptr(), down.data_ptr(),
                         up.data_ptr(), factors, _ints("cu", cu, requests + 1, device), _ints("adapters", adapters, requests, device),
                         _rows("A", A, (rows, K), dtype, device), ldb, N if D is None else _rows("D", D, (rows, N), dtype, device), ldn, sdn,
                         lup, sup)
    return desc, device


def adapter_product(A, B, down, up, cu, adapters, scales=None, *, D=None, workspace=None):
    """D[r] = B @ A[r] + scales[a] * up[a] @ (down[a] @ A[r]), a = adapters[b] for the
    rows r = cu[b] .. cu[b + 1] - 1 of request b.

    A (rows, K), B (N, K) shared by all rows, down (adapters, rank, K) and up
    (adapters, N, rank), fp16 or bf16; rank is a multiple of 8 up to 128
    (adapters of a smaller rank are padded with zeros).  cu: requests + 1 int32
    offsets, adapters: int32, both on the device; -1 means no adapter.  scales:
    float32 for each adapter, 1 when not given.  Returns D (rows, N); rows of
    no request are left as they were in a given D.  `workspace`: a device
    tensor of at least adapter_product_workspace(...) bytes, 16-byte aligned;
    allocated here when not given."""
    if D is None and A.dim() == 2 and B.dim() == 2:   # other tensors are refused below
        D = A.new_empty(A.shape[0], B.shape[0])
    _run("adapter_nt", *_adapter_desc(A, B, down, up, cu, adapters, scales, D), workspace)
    return D


def adapter_product_workspace(A, B, down, up, cu, adapters, scales=None) -> int:
    """Bytes of workspace adapter_product needs for tensors of these shapes."""
    return _workspace_bytes("adapter_nt", *_adapter_desc(A, B, down, up, cu, adapters, scales, None))

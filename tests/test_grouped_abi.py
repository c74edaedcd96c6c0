"""The grouped entry points on the CPU: exported, and refusing what they do not take before any HIP call."""
import ctypes
import os
import re
import subprocess

import pytest

import dense_fp16_gemm_nt_amd as g
from dense_fp16_gemm_nt_amd import grouped as gr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "grouped.h")
BASE = 1 << 36   # fake, aligned, far apart
OK, INVALID, UNSUPPORTED = g.OK, g.INVALID_ARG, g.UNSUPPORTED


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b((?:grouped|adapter)_\w+)\s*\(", text))
    assert len(names) == 12
    L = ctypes.CDLL(g.LIB_PATH)
    for n in names:
        assert hasattr(L, n), n


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "user.c"
    src.write_text('#include "grouped.h"\nint main(void) { grouped_desc d = {0}; adapter_desc a = {0}; '
                   'return grouped_tn_check(&d) + adapter_nt_check(&a) + GROUPED_BF16; }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


@pytest.mark.parametrize("struct,desc", [("grouped_desc", gr.GroupedDesc), ("adapter_desc", gr.AdapterDesc)])
def test_binding_has_the_headers_fields(struct, desc):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\}" % struct, text, flags=re.S).group(1)
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64}
    want = []
    for line in body.split(";"):
        line = line.replace("const", "").strip()
        if line:
            kind, names = line.split(None, 1)
            for n in names.split(","):
                pointer = "*" in kind or "*" in n
                want.append((n.replace("*", "").strip(), ctypes.c_void_p if pointer else kinds[kind]))
    assert [(n, t) for n, t in desc._fields_] == want


def grouped(**kw):
    d = dict(dtype=0, b_fp32=0, groups=3, rows=100, N=64, K=32, A=BASE, B=2 * BASE, D=3 * BASE, lda=32, ldb=32, stride_b=64 * 32, ldd=64,
             cu=4 * BASE)
    d.update(kw)
    return gr.GroupedDesc(**d)


def adapter(**kw):
    d = dict(dtype=1, rank=16, adapters=4, requests=3, rows=100, N=64, K=32, A=BASE, B=2 * BASE, D=3 * BASE, down=4 * BASE, up=5 * BASE,
             scales=6 * BASE, cu=7 * BASE, ids=8 * BASE, lda=32, ldb=32, ldd=64, ld_down=32, stride_down=512, ld_up=16, stride_up=1024)
    d.update(kw)
    return gr.AdapterDesc(**d)


ALL = ("grouped_nt", "grouped_nn", "grouped_tn")
# (change, statuses of nt, nn and tn)
CHANGES = [
    ({}, (OK, OK, OK)),
    ({"dtype": 1}, (OK, OK, OK)),
    ({"dtype": 2}, (INVALID,) * 3),
    ({"b_fp32": 1}, (UNSUPPORTED, UNSUPPORTED, OK)),
    ({"b_fp32": 2}, (INVALID,) * 3),
    ({"groups": -1}, (INVALID,) * 3),
    ({"rows": -1}, (INVALID,) * 3),
    ({"N": -8}, (INVALID,) * 3),
    ({"K": -8}, (INVALID,) * 3),
    ({"lda": 24}, (INVALID,) * 3),
    ({"ldb": 24}, (INVALID,) * 3),
    ({"ldd": 56}, (INVALID,) * 3),
    ({"ldb": -32}, (INVALID,) * 3),
    ({"stride_b": -8}, (INVALID,) * 3),
    ({"stride_b": 0}, (OK, OK, INVALID)),             # a matrix repeated; matrices written on top of each other
    ({"stride_b": 63 * 32}, (OK, OK, INVALID)),
    ({"stride_b": 0, "groups": 1}, (OK, OK, OK)),
    ({"A": 0}, (INVALID,) * 3),
    ({"B": 0}, (INVALID,) * 3),
    ({"D": 0}, (INVALID,) * 3),
    ({"cu": 0}, (INVALID,) * 3),
    ({"cu": 4 * BASE + 2}, (UNSUPPORTED,) * 3),
    ({"A": BASE + 8}, (UNSUPPORTED,) * 3),
    ({"B": 2 * BASE + 2}, (UNSUPPORTED,) * 3),
    ({"D": 3 * BASE + 1}, (UNSUPPORTED,) * 3),
    ({"lda": 36}, (UNSUPPORTED,) * 3),
    ({"ldd": 68}, (UNSUPPORTED,) * 3),
    ({"ldb": 34, "stride_b": 64 * 40}, (UNSUPPORTED,) * 3),
    ({"stride_b": 64 * 32 + 4}, (UNSUPPORTED,) * 3),
    ({"N": 60}, (UNSUPPORTED,) * 3),
    ({"K": 31}, (UNSUPPORTED,) * 3),
    ({"lda": 1 << 22}, (UNSUPPORTED,) * 3),
    ({"ldd": 1 << 22}, (UNSUPPORTED,) * 3),
    ({"lda": 1 << 41}, (INVALID,) * 3),
    ({"D": BASE}, (INVALID, INVALID, OK)),            # what is read may overlap
    ({"A": 2 * BASE}, (OK, INVALID, INVALID)),
    ({"B": 3 * BASE + 1024}, (INVALID, OK, INVALID)),
    ({"cu": 3 * BASE + 64}, (INVALID, OK, OK)),
    ({"cu": 2 * BASE + 64}, (OK, OK, INVALID)),
    ({"rows": 0, "A": 0, "D": 0}, (OK, OK, OK)),
    ({"rows": 0, "A": 0, "D": 0, "B": 0}, (OK, OK, INVALID)),   # matrices of zeros have to be written
    ({"groups": 0, "A": 0, "B": 0, "D": 0, "cu": 0}, (OK, OK, OK)),
    ({"N": 0, "D": 0, "B": 0, "cu": 0}, (OK, INVALID, OK)),
    ({"K": 0, "A": 0, "B": 0}, (OK, OK, OK)),
    ({"rows": (1 << 31) - 1000, "A": 1 << 50, "D": 1 << 52}, (UNSUPPORTED,) * 3),
    ({"groups": 1 << 22, "D": 1 << 50, "A": 1 << 51}, (UNSUPPORTED,) * 3),
]


@pytest.mark.parametrize("change,want", CHANGES)
def test_grouped_arguments(change, want):
    L = g.lib()
    d = grouped(**change)
    for name, status in zip(ALL, want):
        assert getattr(L, name + "_check")(ctypes.byref(d)) == status, name
        if status != OK:
            assert getattr(L, name)(ctypes.byref(d), None, 0, None) == status, name
            assert getattr(L, name + "_workspace")(ctypes.byref(d)) == status, name


@pytest.mark.parametrize("change,want", [
    ({}, OK),
    ({"dtype": 0}, OK),
    ({"dtype": -1}, INVALID),
    ({"rank": -8}, INVALID),
    ({"rank": 12, "ld_up": 16}, UNSUPPORTED),
    ({"rank": 136, "ld_up": 136, "stride_up": 1 << 20, "stride_down": 1 << 20}, UNSUPPORTED),
    ({"rank": 128, "ld_up": 128, "stride_up": 1 << 20, "stride_down": 1 << 20}, OK),
    ({"rank": 0, "down": 0, "up": 0}, OK),
    ({"adapters": -1}, INVALID),
    ({"adapters": 0, "down": 0, "up": 0, "scales": 0}, OK),
    ({"requests": -1}, INVALID),
    ({"requests": 0, "cu": 0, "ids": 0, "D": 0}, OK),
    ({"rows": -1}, INVALID),
    ({"rows": 0, "A": 0, "D": 0}, OK),
    ({"N": 0, "B": 0, "D": 0, "up": 0}, OK),
    ({"K": 0, "A": 0, "B": 0, "down": 0}, OK),
    ({"N": 60}, UNSUPPORTED),
    ({"K": 30}, UNSUPPORTED),
    ({"A": 0}, INVALID),
    ({"B": 0}, INVALID),
    ({"D": 0}, INVALID),
    ({"down": 0}, INVALID),
    ({"up": 0}, INVALID),
    ({"cu": 0}, INVALID),
    ({"ids": 0}, INVALID),
    ({"scales": 0}, OK),
    ({"scales": 6 * BASE + 2}, UNSUPPORTED),
    ({"ids": 8 * BASE + 1}, UNSUPPORTED),
    ({"down": 4 * BASE + 8}, UNSUPPORTED),
    ({"up": 5 * BASE + 2}, UNSUPPORTED),
    ({"ld_down": 24}, INVALID),
    ({"ld_up": 8}, INVALID),
    ({"ld_up": 20}, UNSUPPORTED),
    ({"stride_up": 1028}, UNSUPPORTED),
    ({"stride_down": 0, "stride_up": 0}, OK),
    ({"stride_down": -8}, INVALID),
    ({"lda": 24}, INVALID),
    ({"ldd": 1 << 22}, UNSUPPORTED),
    ({"ld_up": 1 << 22, "stride_up": 1 << 30, "up": 1 << 50}, UNSUPPORTED),
    ({"D": BASE + 1024}, INVALID),
    ({"D": 2 * BASE}, INVALID),
    ({"D": 4 * BASE + 512}, INVALID),
    ({"D": 5 * BASE}, INVALID),
    ({"cu": 3 * BASE}, INVALID),
    ({"ids": 3 * BASE + 4}, INVALID),
    ({"scales": 3 * BASE}, INVALID),
    ({"adapters": 1 << 22, "stride_down": 0, "stride_up": 0}, UNSUPPORTED),
])
def test_adapter_arguments(change, want):
    L = g.lib()
    d = adapter(**change)
    assert L.adapter_nt_check(ctypes.byref(d)) == want
    if want != OK:
        assert L.adapter_nt(ctypes.byref(d), None, 0, None) == want
        assert L.adapter_nt_workspace(ctypes.byref(d)) == want


def test_workspaces_of_calls_that_write_nothing():
    L = g.lib()
    for none in ({"rows": 0}, {"requests": 0}, {"N": 0}):
        assert L.adapter_nt_workspace(ctypes.byref(adapter(**none))) == 0
    for name in ALL:
        assert getattr(L, name + "_workspace")(ctypes.byref(grouped(groups=0))) == 0


def test_null_descriptors():
    L = g.lib()
    for name in ALL:
        assert getattr(L, name)(None, None, 0, None) == INVALID and getattr(L, name + "_check")(None) == INVALID
    assert L.adapter_nt(None, None, 0, None) == INVALID and L.adapter_nt_check(None) == INVALID
    assert L.adapter_nt_workspace(None) == INVALID


def test_host_tensors_are_refused():
    torch = pytest.importorskip("torch")
    t = torch.float16
    A, B, G, cu = torch.zeros(4, 16, dtype=t), torch.zeros(2, 8, 16, dtype=t), torch.zeros(4, 8, dtype=t), torch.tensor([0, 1, 4], dtype=torch.int32)
    down, up, ids = torch.zeros(3, 8, 16, dtype=t), torch.zeros(3, 8, 8, dtype=t), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: g.grouped_product(A, B, cu), lambda: g.grouped_product_grad_input(G, B, cu), lambda: g.grouped_product_grad_weight(G, A, cu),
                 lambda: g.adapter_product(A, B[0], down, up, cu, ids), lambda: g.grouped_product_workspace(A, B, cu),
                 lambda: g.grouped_product_grad_input_workspace(G, B, cu), lambda: g.grouped_product_grad_weight_workspace(G, A, cu),
                 lambda: g.adapter_product_workspace(A, B[0], down, up, cu, ids)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
    with pytest.raises(TypeError):
        g.grouped_product(A.float(), B, cu)

"""The attention entry points on the CPU: exported, and refusing what they do not take before any HIP call."""
import ctypes
import os
import re
import subprocess

import pytest

import dense_fp16_gemm_nt_amd as g
from dense_fp16_gemm_nt_amd import attention as a

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "attention.h")
BASE = 1 << 32   # fake, aligned, far apart


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(attn_\w+)\s*\(", text))
    assert len(names) == 6
    L = ctypes.CDLL(g.LIB_PATH)
    for n in names:
        assert hasattr(L, n), n


def test_header_is_plain_c(tmp_path):
    src = tmp_path / "user.c"
    src.write_text('#include "attention.h"\nint main(void) { attn_prompt_desc d = {0}; return sizeof d == 0 ? ATTN_BF16 : attn_prompt_check(&d); }\n')
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                   check=True)


@pytest.mark.parametrize("struct,desc", [("attn_prompt_desc", a.PromptDesc), ("attn_shared_prefix_desc", a.SharedPrefixDesc)])
def test_binding_has_the_headers_fields(struct, desc):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct %s \{(.*?)\}" % struct, text, flags=re.S).group(1)
    kinds = {"int32_t": ctypes.c_int32, "int64_t": ctypes.c_int64, "float": ctypes.c_float}
    want = []
    for line in body.split(";"):
        line = line.replace("const", "").strip()
        if line:
            kind, names = line.split(None, 1)
            for n in names.split(","):
                pointer = "*" in kind or "*" in n
                want.append((n.replace("*", "").strip(), ctypes.c_void_p if pointer else kinds[kind]))
    assert [(n, t) for n, t in desc._fields_] == want


def prompt(**kw):
    d = dict(dtype=0, causal=1, heads=8, kv_heads=2, head_dim=128, batch=2, total_q=100, total_k=200,
             Q=BASE, K=2 * BASE, V=3 * BASE, O=4 * BASE, lse=None, cu_q=5 * BASE, cu_k=6 * BASE,
             q_row=1024, q_head=128, k_row=256, k_head=128, v_row=256, v_head=128, o_row=1024, o_head=128, scale=0.1)
    d.update(kw)
    return a.PromptDesc(**d)


def shared(**kw):
    d = dict(dtype=1, heads=8, kv_heads=2, head_dim=64, batch=3, prefix=100, slot_rows=50,
             Q=BASE, Kp=2 * BASE, Vp=3 * BASE, Ks=4 * BASE, Vs=5 * BASE, O=6 * BASE, lse=None, lens=7 * BASE,
             q_row=512, q_head=64, kp_row=128, kp_head=64, vp_row=128, vp_head=64, ks_slot=6400, ks_row=128, ks_head=64,
             vs_slot=6400, vs_row=128, vs_head=64, o_row=512, o_head=64, scale=0.1)
    d.update(kw)
    return a.SharedPrefixDesc(**d)


OK, INVALID, UNSUPPORTED = g.OK, g.INVALID_ARG, g.UNSUPPORTED


@pytest.mark.parametrize("change,want", [
    ({}, OK),
    ({"dtype": 1}, OK),
    ({"dtype": 2}, INVALID),
    ({"causal": 2}, INVALID),
    ({"heads": 0}, INVALID),
    ({"heads": 7}, INVALID),
    ({"kv_heads": 0}, INVALID),
    ({"head_dim": 0}, INVALID),
    ({"head_dim": 100}, UNSUPPORTED),
    ({"head_dim": 136, "q_head": 136, "o_head": 136, "k_head": 136, "v_head": 136, "q_row": 1088, "o_row": 1088}, UNSUPPORTED),
    ({"batch": -1}, INVALID),
    ({"batch": 0}, OK),
    ({"total_q": -1}, INVALID),
    ({"total_q": 0, "Q": 0, "O": 0}, OK),
    ({"total_k": 0, "K": 0, "V": 0}, OK),
    ({"Q": 0}, INVALID),
    ({"K": 0}, INVALID),
    ({"V": 0}, INVALID),
    ({"O": 0}, INVALID),
    ({"cu_q": 0}, INVALID),
    ({"cu_k": 0}, INVALID),
    ({"cu_k": 6 * BASE + 2}, UNSUPPORTED),
    ({"lse": 7 * BASE}, OK),
    ({"lse": 7 * BASE + 1}, UNSUPPORTED),
    ({"lse": 4 * BASE}, INVALID),                # lse over O
    ({"lse": 2 * BASE + 1024}, INVALID),
    ({"Q": BASE + 8}, UNSUPPORTED),
    ({"Q": BASE + 1}, UNSUPPORTED),
    ({"K": 2 * BASE + 2}, UNSUPPORTED),
    ({"q_row": 1028}, UNSUPPORTED),
    ({"v_head": 132}, UNSUPPORTED),
    ({"q_row": -1024}, INVALID),
    ({"k_row": 1 << 23}, UNSUPPORTED),
    ({"k_row": (1 << 23) - 8, "O": 1 << 50}, OK),
    ({"k_head": 0, "v_head": 0}, OK),            # one kv head repeated
    ({"o_head": 0}, INVALID),                    # heads of O on top of each other
    ({"o_row": 128}, INVALID),
    ({"o_row": 128, "o_head": 12800}, OK),       # heads first
    ({"O": BASE}, INVALID),
    ({"O": 3 * BASE + 1024}, INVALID),
    ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID),
    ({"scale": 3e38}, INVALID),
    ({"scale": -1.0}, OK),
    ({"scale": 0.0}, OK),
    ({"total_q": 1 << 30, "q_row": 0, "o_row": 1 << 10, "O": 1 << 50}, UNSUPPORTED),   # 2^32 rows of one kv head
    ({"total_k": 1 << 31, "O": 1 << 50}, UNSUPPORTED),
    ({"k_row": 1 << 41}, INVALID),
])
def test_prompt_arguments(change, want):
    L = g.lib()
    d = prompt(**change)
    assert L.attn_prompt_check(ctypes.byref(d)) == want
    if want != OK:
        assert L.attn_prompt(ctypes.byref(d), None, 0, None) == want
        assert L.attn_prompt_workspace(ctypes.byref(d)) == want


@pytest.mark.parametrize("change,want", [
    ({}, OK),
    ({"dtype": -1}, INVALID),
    ({"heads": 3}, INVALID),
    ({"head_dim": 4}, UNSUPPORTED),
    ({"batch": -1}, INVALID),
    ({"batch": 0, "Q": 0}, OK),
    ({"prefix": -1}, INVALID),
    ({"prefix": 0, "Kp": 0, "Vp": 0}, OK),
    ({"slot_rows": -1}, INVALID),
    ({"slot_rows": 0, "Ks": 0, "Vs": 0}, OK),
    ({"Q": 0}, INVALID),
    ({"Kp": 0}, INVALID),
    ({"Vs": 0}, INVALID),
    ({"lens": 0}, INVALID),
    ({"lens": 7 * BASE + 1}, UNSUPPORTED),
    ({"lse": 6 * BASE}, INVALID),
    ({"lse": 8 * BASE}, OK),
    ({"Ks": 4 * BASE + 4}, UNSUPPORTED),
    ({"ks_slot": 6404}, UNSUPPORTED),
    ({"vs_slot": -8}, INVALID),
    ({"ks_row": 1 << 23}, UNSUPPORTED),
    ({"ks_slot": 0, "vs_slot": 0}, OK),
    ({"O": 4 * BASE + 6400}, INVALID),
    ({"o_head": 32}, INVALID),
    ({"scale": float("nan")}, INVALID),
    ({"batch": 1 << 30, "q_row": 0, "ks_slot": 0, "vs_slot": 0, "O": 1 << 50}, UNSUPPORTED),
])
def test_shared_prefix_arguments(change, want):
    L = g.lib()
    d = shared(**change)
    assert L.attn_shared_prefix_check(ctypes.byref(d)) == want
    if want != OK:
        assert L.attn_shared_prefix(ctypes.byref(d), None, 0, None) == want
        assert L.attn_shared_prefix_workspace(ctypes.byref(d)) == want


FAR = 1 << 50   # O above everything the inputs span
MANY = dict(q_row=0, o_row=1 << 10, O=FAR, k_row=0, v_row=0)


@pytest.mark.parametrize("change,want", [
    # kv_heads (2) x (total_q * group (4) / 128 + sequences) units, at most 2^22
    (dict(MANY, batch=1, total_q=(1 << 26) - 32), OK),
    (dict(MANY, batch=1, total_q=1 << 26), UNSUPPORTED),
    (dict(MANY, batch=1 << 20, total_q=1 << 20), OK),
    (dict(MANY, batch=1 << 21, total_q=1 << 21), UNSUPPORTED),
    (dict(MANY, batch=1 << 30, total_q=5), OK),    # at most five of them have a query
    (dict(MANY, batch=(1 << 31) - 1, total_q=5), UNSUPPORTED),   # a count of them by 64 would pass 32 bits
])
def test_prompt_most_work(change, want):
    assert g.lib().attn_prompt_check(ctypes.byref(prompt(**change))) == want


ONE_SLOT = dict(q_row=0, ks_slot=0, vs_slot=0, ks_row=0, vs_row=0, O=FAR)


@pytest.mark.parametrize("change,want", [
    # kv_heads (2) x (batch * group (4) / 128 + batch * (slot_rows / 2048 + 1)) units, at most 2^22
    (dict(ONE_SLOT, batch=1 << 20), OK),
    (dict(ONE_SLOT, batch=1 << 21), UNSUPPORTED),
    (dict(ONE_SLOT, batch=1 << 20, slot_rows=2047), OK),
    (dict(ONE_SLOT, batch=1 << 20, slot_rows=2048), UNSUPPORTED),
    (dict(ONE_SLOT, batch=4, slot_rows=1 << 30), UNSUPPORTED),
    (dict(ONE_SLOT, batch=3, slot_rows=1 << 30), OK),
])
def test_shared_prefix_most_work(change, want):
    assert g.lib().attn_shared_prefix_check(ctypes.byref(shared(**change))) == want


def test_null_descriptors():
    L = g.lib()
    assert L.attn_prompt_check(None) == INVALID and L.attn_shared_prefix_check(None) == INVALID
    assert L.attn_prompt(None, None, 0, None) == INVALID and L.attn_shared_prefix(None, None, 0, None) == INVALID


def test_empty_calls_launch_nothing():
    # nothing to do: no device is needed
    L = g.lib()
    assert L.attn_prompt(ctypes.byref(prompt(total_q=0)), None, 0, None) == OK
    assert L.attn_prompt(ctypes.byref(prompt(batch=0)), None, 0, None) == OK
    assert L.attn_shared_prefix(ctypes.byref(shared(batch=0)), None, 0, None) == OK
    assert L.attn_prompt_workspace(ctypes.byref(prompt(batch=0))) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    c = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.attention_prompt(q, q, q, c)
    with pytest.raises(ValueError):
        g.attention_shared_prefix(q, q, q, q[:, None], q[:, None], c)

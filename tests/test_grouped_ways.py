"""Which ways through the kernels the GPU tests' cases take: the library's own choice, evaluated on the host for the 256 compute
units of an MI355X.  A changed rate of its model must not leave a kernel without a test."""
import ctypes

import pytest

import dense_fp16_gemm_nt_amd as g
from dense_fp16_gemm_nt_amd import grouped as gr

pytest.importorskip("torch")

from tests.adapter_cases import EVERY_WAY  # noqa: E402
from tests.test_gpu_grouped import CASES  # noqa: E402
from tests.test_gpu_grouped_ways import MORE  # noqa: E402

CUS = 256
FAR = 1 << 50   # addresses that no two of which reach each other


def adapter_desc(case, dtype=0):
    lens, ids, n, k, rank = case
    count = max(4, max(ids) + 1 if max(ids) < 9 else 4)
    return gr.AdapterDesc(dtype=dtype, rank=rank, adapters=count, requests=len(lens), rows=sum(lens), N=n, K=k, A=FAR, B=2 * FAR, D=3 * FAR, down=4 * FAR,
                          up=5 * FAR, scales=0, cu=6 * FAR, ids=7 * FAR, lda=k, ldb=k, ldd=n, ld_down=k, stride_down=rank * k, ld_up=rank,
                          stride_up=n * rank)


def grouped_desc(case, dtype=0, b_fp32=0):
    lens, n, k = case
    return gr.GroupedDesc(dtype=dtype, b_fp32=b_fp32, groups=len(lens), rows=sum(lens), N=n, K=k, A=FAR, B=2 * FAR, D=3 * FAR, lda=k, ldb=k, stride_b=n * k,
                          ldd=n, cu=4 * FAR)


def divided(parts):
    return "whole" if parts == 1 else "in parts"


def ways(cases):
    """A name for each kernel, or pair of kernels, of the cases' calls."""
    out = set()
    for case in cases:
        if sum(case[0]) == 0:
            continue
        way, (rows, cols, parts), (low_rows, low_cols, low_parts) = gr.adapter_plan(adapter_desc(case), CUS)
        if way == gr.ONE_LAUNCH:
            out.add(("one launch", min(1, len(case[0]) * -(-case[4] // 16) - 1)))
        elif way == gr.EACH:
            assert (rows, cols) == (256, 256) and parts in (0, 1)
            out.add(("each", "one step" if case[4] <= 32 else "two steps"))
            out.add(("each", divided(parts)))
        else:
            out.add((("dots", "sums", "tiles")[way - gr.DOTS], rows, cols, divided(parts)))
        if way in (gr.TILES, gr.EACH):
            out.add(("projections", low_rows, low_cols, divided(low_parts)))
    return out


def test_adapter_cases_reach_every_way():
    got = ways(EVERY_WAY)
    print(sorted(map(str, got)))
    assert got >= {("one launch", 0), ("one launch", 1), ("each", "one step"), ("each", "two steps"), ("each", "in parts"), ("each", "whole")}
    assert got >= {("projections", r, c, "whole") for r, c in ((16, 16), (32, 32), (64, 64), (64, 128))}
    assert got >= {("projections", r, c, "in parts") for r, c in ((64, 64), (64, 128))}
    assert got >= {("dots", 16, 16, p) for p in ("whole", "in parts")} | {("dots", 32, 32, p) for p in ("whole", "in parts")}
    assert got >= {("dots", 64, c, p) for c in (64, 128) for p in ("whole", "in parts")} | {("sums", 64, 128, p) for p in ("whole", "in parts")}
    assert got >= {("tiles", r, c, "whole") for r, c in ((16, 16), (32, 32), (64, 64), (64, 128), (128, 128), (256, 256))}
    assert got >= {("tiles", r, c, "in parts") for r, c in ((64, 64), (64, 128), (128, 128))}


SPLIT = {"nt": {(64, 128), (128, 128)}, "nn": {(64, 64), (64, 128), (128, 128)}, "tn": {(64, 64), (128, 128)}}   # forms that can be in parts
WHOLE = {p: {(64, 64), (128, 128), (256, 256)} | (set() if p == "tn" else {(16, 16), (32, 32), (32, 128), (64, 128)}) for p in SPLIT}


@pytest.mark.parametrize("product", sorted(SPLIT))
def test_grouped_cases_reach_every_tile(product):
    got = set()
    for case in CASES + MORE:
        rows, cols, parts = gr.plan(product, grouped_desc(case), CUS)
        got.add(((rows, cols), divided(parts)))
    print(sorted(got))
    assert got >= {(t, "whole") for t in WHOLE[product]} | {(t, "in parts") for t in SPLIT[product] | {(256, 256)}}


def test_plans_refuse_what_calls_refuse():
    bad, fine = grouped_desc(([5, 3], 64, 60)), grouped_desc(([5, 3], 64, 64))
    for call in (lambda: gr.plan("nt", bad, CUS), lambda: gr.plan("nt", fine, 0), lambda: gr.adapter_plan(adapter_desc(([5], [0], 64, 64, 12)), CUS)):
        with pytest.raises(g.GemmError):
            call()
    L = g.lib()
    i, two, n = ctypes.c_int(), (ctypes.c_int * 2)(), ctypes.c_int64()
    assert L.gemm_f16_nt_grouped_plan(ctypes.byref(fine), 3, CUS, two, ctypes.byref(n)) == g.INVALID_ARG
    assert L.gemm_f16_nt_grouped_plan(ctypes.byref(fine), 0, CUS, None, ctypes.byref(n)) == g.INVALID_ARG
    assert L.gemm_f16_nt_adapter_plan(None, CUS, ctypes.byref(i), two, ctypes.byref(n), two, ctypes.byref(n)) == g.INVALID_ARG
    assert gr.plan("nt", grouped_desc(([0, 0], 64, 64)), CUS) == (0, 0, 0)
    assert gr.adapter_plan(adapter_desc(([0], [0], 64, 64, 8)), CUS) == (0, (0, 0, 0), (0, 0, 0))

"""Adapters' low-rank values between the two products keep more bits than the operands have, on every way through the kernels.

The shared matrix cancels all but a small part of the adapters': for row n of it, with j = n % rank,

    B[n] = -base[j],   down_a[j] = base[j] + delta_a[j],   up_a[n] = e_j   =>   D[r, n] = delta_a[j] . A[r]

All are whole numbers.  The values down_a A[r] between the products need up to 15 bits, more than a term of either type has;
two hold them (16 bits in bf16, and 21 and more in fp16), so what is left is exact.
"""
import math
import sys

import pytest

import dense_fp16_gemm_nt_amd as g
from tests import grouped_ref as ref
from tests.adapter_cases import EVERY_WAY
from tests.test_gpu_grouped import DEV, TYPES, adapter_inputs, ints, kept, real, starts, whole

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def cancelling(seed, dtype, case):
    lens, ids, n, k, rank = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    count = max(4, max(ids) + 1 if max(ids) < 9 else 4)
    # |down A| has a standard deviation of 0.82 top sqrt(k) < 6600 of the values -2 .. 2 of A: below 2^15 to five of these
    top = min(120, int(8000 / math.sqrt(k)))
    base = whole(gen, dtype, rank, k, top=top)
    down = (base.float()[None] + whole(gen, dtype, count, rank, k, top=1).float()).to(TYPES[dtype])
    j = torch.arange(n, device=DEV) % rank
    up = torch.nn.functional.one_hot(j, rank).to(TYPES[dtype]).expand(count, n, rank).contiguous()
    return whole(gen, dtype, sum(lens), k), -base[j], down, up, starts(lens), ids


@pytest.mark.parametrize("case", range(len(EVERY_WAY)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_low_rank_values_are_held_in_two_terms(dtype, case):
    A, B, down, up, cu, ids = cancelling(700 + case, dtype, EVERY_WAY[case])
    print(f"[gpu] cancelling adapters {dtype} {EVERY_WAY[case][2:]}", file=sys.stderr, flush=True)
    D = g.adapter_product(A, B, down, up, ints(cu), ints(ids), D=kept(dtype, A.shape[0], B.shape[0]))
    torch.cuda.synchronize()
    want, _ = ref.adapters(A, B, down, up, cu, ids, None, kept(dtype, A.shape[0], B.shape[0]))
    assert torch.equal(D, want.to(TYPES[dtype]))


@pytest.mark.parametrize("case", range(len(EVERY_WAY)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_values_on_every_way(dtype, case):
    A, B, down, up, cu, ids = adapter_inputs(real, 750 + case, dtype, EVERY_WAY[case], 3, 5, 8)
    scales = torch.linspace(-1.5, 2.0, down.shape[0], device=DEV)
    down = down / 8
    print(f"[gpu] adapter values {dtype} {EVERY_WAY[case][2:]}", file=sys.stderr, flush=True)
    D = kept(dtype, A.shape[0], B.shape[0], 8)
    g.adapter_product(A, B, down, up, ints(cu), ints(ids), scales, D=D)
    torch.cuda.synchronize()
    # rows of no request keep what they held; the others' bound is that of products whose low-rank values are off by 2^-16 of
    # themselves in bf16, and in fp16 by 2^-20 or 2^-25
    own = slice(cu[0], cu[-1])
    assert bool((D[:cu[0]] == 7).all()) and bool((D[cu[-1]:] == 7).all())
    t, rank = TYPES[dtype], down.shape[1]
    want, bound = kept(dtype, A.shape[0], B.shape[0]).double(), torch.zeros(D.shape, dtype=torch.float64, device=DEV)
    for q, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if a == b:
            continue
        x, i = A[a:b].double(), ids[q]
        want[a:b], bound[a:b] = ref._sum(x, B.double().t(), A.shape[1])
        if 0 <= i < down.shape[0]:
            h, off = ref._sum(x, down[i].double().t(), A.shape[1])
            s = float(scales[i])
            h, off = h * s, off * abs(s) + h.abs() * abs(s) * ref.STEP
            off = off + (2.0 ** -16 if t is torch.bfloat16 else 2.0 ** -20) * (h.abs() + off) + (2.0 ** -25 if t is torch.float16 else 0.0)
            w = up[i].double().t()
            want[a:b] += torch.mm(h, w)
            bound[a:b] += torch.mm(off, w.abs()) + (2 * rank + 8) * ref.STEP * torch.mm(h.abs() + off, w.abs())
    ref.check(D[own], want[own], bound[own], "adapters")

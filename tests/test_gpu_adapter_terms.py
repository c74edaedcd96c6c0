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
from tests.test_gpu_grouped import ADAPTERS, DEV, TYPES, ints, kept, starts, whole

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


@pytest.mark.parametrize("case", range(len(ADAPTERS)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_low_rank_values_are_held_in_two_terms(dtype, case):
    A, B, down, up, cu, ids = cancelling(700 + case, dtype, ADAPTERS[case])
    print(f"[gpu] cancelling adapters {dtype} {ADAPTERS[case][2:]}", file=sys.stderr, flush=True)
    D = g.adapter_product(A, B, down, up, ints(cu), ints(ids), D=kept(dtype, A.shape[0], B.shape[0]))
    torch.cuda.synchronize()
    want, _ = ref.adapters(A, B, down, up, cu, ids, None, kept(dtype, A.shape[0], B.shape[0]))
    assert torch.equal(D, want.to(TYPES[dtype]))

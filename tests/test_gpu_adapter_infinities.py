"""Adapters beside values that are not finite, on every way through the kernels: an output is what the formula gives for its
own row, whatever the rank is padded to inside."""
import sys

import pytest

import dense_fp16_gemm_nt_amd as g
from tests.adapter_cases import EVERY_WAY
from tests.test_gpu_grouped import DEV, TYPES, adapter_inputs, ints, real

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
INF = float("inf")


@pytest.mark.parametrize("case", range(len(EVERY_WAY)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_an_infinity_in_a_row_of_positive_values(dtype, case):
    # everything that the infinity meets is positive, so its row is infinite, and no number anywhere is missing
    lens, ids, n, k, rank = EVERY_WAY[case]
    A, B, down, up, cu, ids = adapter_inputs(real, 800 + case, dtype, EVERY_WAY[case])
    if A.shape[0] == 0:
        pytest.skip("no rows")
    B, down, up = B.abs() + 0.25, down.abs() / 8 + 0.25, up.abs() + 0.25
    print(f"[gpu] an infinity in A, {dtype} {EVERY_WAY[case][2:]}", file=sys.stderr, flush=True)
    clean = g.adapter_product(A, B, down, up, ints(cu), ints(ids))
    hit = sorted({0, A.shape[0] // 2, A.shape[0] - 1})
    A = A.clone()
    for i, r in enumerate(hit):
        A[r, (7 * r) % k] = INF if i % 2 == 0 else -INF
    D = g.adapter_product(A, B, down, up, ints(cu), ints(ids))
    torch.cuda.synchronize()
    for i, r in enumerate(hit):
        assert bool((D[r] == (INF if i % 2 == 0 else -INF)).all()), r
    others = torch.ones(A.shape[0], dtype=torch.bool, device=DEV)
    others[hit] = False
    assert torch.equal(D[others], clean[others])


@pytest.mark.parametrize("case", range(len(EVERY_WAY)))
@pytest.mark.parametrize("sign", [1, -1])
def test_an_infinite_adapter_beside_sums_beyond_the_largest_value(sign, case):
    # the shared product alone is 131008 or so, finite in the sums and infinite when rounded to fp16: an adapter's infinity of
    # the other sign decides, as it does before any rounding
    lens, ids, n, k, rank = EVERY_WAY[case]
    A, B, down, up, cu, ids = adapter_inputs(real, 850 + case, "fp16", EVERY_WAY[case])
    owners = [a for ln, a in zip(lens, ids) if ln and 0 <= a < down.shape[0]]
    if not owners:
        pytest.skip("no row has an adapter")
    A, B = torch.ones_like(A), torch.full_like(B, sign * 2 * 65504 / k)
    down, up = down.abs() / (8 * k) + 1 / k, up.abs() / 8
    up[owners[0], 1::3, rank // 2] = -sign * INF
    print(f"[gpu] sums beyond the largest value, {EVERY_WAY[case][2:]}", file=sys.stderr, flush=True)
    D = g.adapter_product(A, B, down, up, ints(cu), ints(ids))
    torch.cuda.synchronize()
    whose = torch.repeat_interleave(torch.tensor(ids[:len(lens)], device=DEV), torch.tensor(lens, device=DEV))
    hit = (whose == owners[0])[:, None] & (torch.arange(n, device=DEV) % 3 == 1)[None]
    assert bool(hit.any()) and bool((D[hit] == -sign * INF).all()) and bool((D[~hit] == sign * INF).all())


@pytest.mark.parametrize("case", range(len(EVERY_WAY)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("bad", [INF, float("nan")])
def test_an_adapter_that_is_not_finite_has_its_own_rows_alone(bad, dtype, case):
    # down positive and A too, so that an infinity of `up` is met by positive values: it is the output's, and a NaN is one
    lens, ids, n, k, rank = EVERY_WAY[case]
    A, B, down, up, cu, ids = adapter_inputs(real, 880 + case, dtype, EVERY_WAY[case])
    owners = [a for ln, a in zip(lens, ids) if ln and 0 <= a < down.shape[0]]
    if not owners:
        pytest.skip("no row has an adapter")
    A, down = A.abs() / 8 + 1 / 64, down.abs() / 8 + 1 / 64
    clean = g.adapter_product(A, B, down, up, ints(cu), ints(ids))
    up = up.clone()
    up[owners[-1], 1::3, rank - 1] = bad
    print(f"[gpu] adapter {owners[-1]} holds {bad}, {dtype} {EVERY_WAY[case][2:]}", file=sys.stderr, flush=True)
    D = g.adapter_product(A, B, down, up, ints(cu), ints(ids))
    torch.cuda.synchronize()
    whose = torch.repeat_interleave(torch.tensor(ids[:len(lens)], device=DEV), torch.tensor(lens, device=DEV))
    hit = (whose == owners[-1])[:, None] & (torch.arange(n, device=DEV) % 3 == 1)[None]
    assert bool(hit.any()) and bool((D[hit] == INF).all() if bad == INF else torch.isnan(D[hit]).all())
    assert torch.equal(D[~hit], clean[~hit])

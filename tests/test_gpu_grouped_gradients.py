"""Gradients of grouped products against differences, where nothing is rounded: values -1, 0 and 1 have sums below 256, which both
types hold, and the products are linear in each operand, so a step's difference is the gradient's product with it exactly."""
import pytest

import dense_fp16_gemm_nt_amd as g
from tests.test_gpu_grouped import TYPES, inputs, ints, whole

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def signs(gen, dtype, *shape):
    return whole(gen, dtype, *shape, top=1)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,n,k", [([3, 0, 30, 7], 72, 136), ([1], 8, 8), ([40, 60, 0, 70], 200, 248)])
def test_gradients_are_the_differences(lens, n, k, dtype):
    A, G, B, cu_host = inputs(signs, 52, dtype, lens, n, k)
    cu, rows = ints(cu_host), sum(lens)
    dA, dB = g.grouped_product_grad_input(G, B, cu).double(), g.grouped_product_grad_weight(G, A, cu).double()
    assert torch.equal(g.grouped_product_grad_weight(G, A, cu, dtype=torch.float32).double(), dB)
    base = g.grouped_product(A, B, cu).double()
    pick = torch.Generator().manual_seed(n)
    some = [(int(torch.randint(rows, (1,), generator=pick)), int(torch.randint(k, (1,), generator=pick))) for _ in range(12)]
    found = []
    for r, c in some:
        step = torch.zeros_like(A)
        step[r, c] = 2
        found.append(float(((g.grouped_product(A + step, B, cu).double() - base) * G.double()).sum()) / 2)
        assert found[-1] == float(dA[r, c])
    for r, c in some:
        e, row = next(e for e in range(len(lens)) if cu_host[e] <= r < cu_host[e + 1]), (7 * r + c) % n
        step = torch.zeros_like(B)
        step[e, row, c] = -2
        found.append(float(((g.grouped_product(A, B + step, cu).double() - base) * G.double()).sum()) / -2)
        assert found[-1] == float(dB[e, row, c])
    # a gradient of zeros, or of another sign, would have been found
    assert any(x > 0 for x in found) and any(x < 0 for x in found)
    # a matrix without rows has no gradient, and a step of it changes nothing
    for e in [e for e in range(len(lens)) if lens[e] == 0]:
        step = torch.zeros_like(B)
        step[e] = 1
        assert not bool(dB[e].any()) and torch.equal(g.grouped_product(A, B + step, cu).double(), base)

"""Grouped products on the tiles, and parts of a contraction, that the cases of test_gpu_grouped.py leave out (test_grouped_ways.py
checks which are reached): whole numbers, bit by bit."""
import pytest

import dense_fp16_gemm_nt_amd as g
from tests import grouped_ref as ref
from tests.test_gpu_grouped import NAN, TYPES, inputs, ints, kept, say, whole

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

# (rows of each group, N, K)
MORE = [
    ([8, 3], 608, 9824),                          # nt: 64 x 128 in parts
    ([44, 367, 4, 0, 261, 170, 7, 34], 584, 5128),   # nt: 128 x 128 in parts
    ([3], 5712, 16),                              # nn: 64 x 64 in parts
    ([2, 0, 1], 5712, 24),
    ([66], 6936, 6768),                           # nn: 128 x 128 in parts
]


@pytest.mark.parametrize("case", range(len(MORE)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pad", [0, 24])
def test_whole_numbers(pad, dtype, case):
    lens, n, k = MORE[case]
    A, G, B, cu = inputs(whole, 160 + case, dtype, lens, n, k, before=3 if pad else 0, behind=5 if pad else 0, pad=pad)
    rows, t = A.shape[0], TYPES[dtype]
    say(f"[gpu] grouped {dtype} N={n} K={k} pad={pad} lens={lens}")
    D, dA = kept(dtype, rows, n, pad), kept(dtype, rows, k, pad)
    dB = torch.full((len(lens), n, k), NAN, dtype=torch.float32, device=A.device)
    g.grouped_product(A, B, ints(cu), D=D)
    g.grouped_product_grad_input(G, B, ints(cu), dA=dA)
    g.grouped_product_grad_weight(G, A, ints(cu), dB=dB)
    torch.cuda.synchronize()
    assert torch.equal(D, ref.product(A, B, cu, kept(dtype, rows, n))[0].to(t))
    assert torch.equal(dA, ref.grad_input(G, B, cu, kept(dtype, rows, k))[0].to(t))
    assert torch.equal(dB, ref.grad_weight(G, A, cu)[0].float())

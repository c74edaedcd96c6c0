"""The grouped products and the product with adapters on the GPU against the plain 64-bit forms (grouped_ref.py derives the
bounds; whole numbers have to come out bit by bit)."""
import sys

import pytest

import dense_fp16_gemm_nt_amd as g
from tests import grouped_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def starts(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def whole(gen, dtype, *shape, top=2):
    """Small whole numbers."""
    return torch.randint(-top, top + 1, shape, generator=gen, device=DEV).to(TYPES[dtype])


def real(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(TYPES[dtype])


def padded(x, pad):
    """The same values in rows that are `pad` elements longer, NaN in between; matrices of a 3-D tensor lie apart too."""
    if pad == 0:
        return x
    shape = list(x.shape)
    shape[-1] += pad
    if len(shape) == 3:
        shape[1] += 1
    out = torch.full(shape, NAN, dtype=x.dtype, device=x.device)
    view = out[..., :x.shape[-1]] if len(shape) == 2 else out[:, :x.shape[1], :x.shape[2]]
    view.copy_(x)
    return view


def inputs(make, seed, dtype, lens, n, k, before=0, behind=0, pad=0):
    """A, G, B and offsets; rows of no group hold NaN."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows = before + sum(lens) + behind
    A, G, B = make(gen, dtype, rows, k), make(gen, dtype, rows, n), make(gen, dtype, len(lens), n, k)
    for X in (A, G):
        X[:before] = NAN
        X[rows - behind:] = NAN
    return padded(A, pad), padded(G, pad), padded(B, pad), starts(lens, before)


def kept(dtype, rows, width, pad=0):
    return padded(torch.full((rows, width), 7.0, dtype=TYPES[dtype], device=DEV), pad)


# (lens, N, K): every shape of tile, sizes at and beside the edges of tiles and steps
CASES = [
    ([1], 8, 8),
    ([1], 32, 64),
    ([5], 64, 8),
    ([0, 3, 0, 0, 33, 1], 40, 264),
    ([31, 32, 33, 0, 2], 136, 256),
    ([1] * 9, 1000, 520),
    ([3, 17, 0, 40, 1, 9, 2, 30] * 9, 1032, 72),           # 72 groups
    ([10] * 64, 1024, 192),
    ([64, 65, 127, 128, 129, 0, 300], 264, 200),
    ([130, 77], 128, 128),
    ([1000, 3, 257, 0, 255, 900, 256, 1500], 2056, 136),
    ([1111, 2222], 8, 64),
    ([5000], 2048, 328),
    ([1000, 3, 257, 0, 255, 900, 256, 1500, 2000, 513], 4104, 264),   # large tiles: rows, or both sides, by columns too
    ([1000, 3, 257, 0, 255, 900, 256, 1500, 2000, 513], 264, 4104),
    ([3000, 1, 64, 65, 129, 2900], 4096, 72),
    ([3000, 1, 64, 65, 129, 2900], 320, 4096),
    ([300] * 70, 1024, 256),
    ([207, 50], 264, 6152),                                # few tiles, a long contraction: in parts
    ([100, 0, 33], 6152, 264),
    ([3000, 0, 2500, 7], 72, 136),
    ([4352], 4104, 2056),                                  # a small last round of large tiles, in parts
    ([4352], 2056, 4104),
    ([700], 4352, 4352),
    ([2200], 4352, 4352),
    ([4000, 9, 352], 1032, 4104),
]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pad", [0, 24])
def test_whole_numbers(pad, dtype, case):
    lens, n, k = CASES[case]
    A, G, B, cu = inputs(whole, 100 + case, dtype, lens, n, k, before=3 if pad else 0, behind=5 if pad else 0, pad=pad)
    rows, t = A.shape[0], TYPES[dtype]
    say(f"[gpu] grouped {dtype} N={n} K={k} pad={pad} lens={lens[:9]}")
    D, dA = kept(dtype, rows, n, pad), kept(dtype, rows, k, pad)
    assert g.grouped_product(A, B, ints(cu), D=D) is D
    torch.cuda.synchronize()
    say("[gpu] grad_input")
    assert g.grouped_product_grad_input(G, B, ints(cu), dA=dA) is dA
    torch.cuda.synchronize()
    want, _ = ref.product(A, B, cu, kept(dtype, rows, n))
    assert torch.equal(D, want.to(t))
    want, _ = ref.grad_input(G, B, cu, kept(dtype, rows, k))
    assert torch.equal(dA, want.to(t))
    want, _ = ref.grad_weight(G, A, cu)
    for out in (t, torch.float32):
        say(f"[gpu] grad_weight {out}")
        dB = padded(torch.full((len(lens), n, k), NAN, dtype=out, device=DEV), pad)
        assert g.grouped_product_grad_weight(G, A, ints(cu), dB=dB) is dB
        torch.cuda.synchronize()
        assert torch.equal(dB, want.to(out))
        if pad:   # what lies between rows and matrices
            whole_dB = dB._base
            assert bool(torch.isnan(whole_dB[:, n:]).all()) and bool(torch.isnan(whole_dB[:, :, k:]).all())
    if pad:
        assert bool(torch.isnan(D._base[:, n:]).all()) and bool(torch.isnan(dA._base[:, k:]).all())


def test_parts_are_reached():
    # among the cases above are some, for each direction, whose contraction is divided: they need room for the parts
    need = {"nt": [], "nn": [], "tn": []}
    for lens, n, k in CASES:
        A, G, B = (torch.empty(s, dtype=torch.float16, device=DEV) for s in ((sum(lens), k), (sum(lens), n), (len(lens), n, k)))
        cu = ints(starts(lens))
        need["nt"].append(g.grouped_product_workspace(A, B, cu))
        need["nn"].append(g.grouped_product_grad_input_workspace(G, B, cu))
        need["tn"].append(g.grouped_product_grad_weight_workspace(G, A, cu))
    say(f"[gpu] workspaces {need}")
    for name, sizes in need.items():
        large = torch.cuda.get_device_properties(DEV).multi_processor_count << 18   # a part of a large tile for each compute unit
        assert any(0 < s < large for s in sizes) and large in sizes and sizes[0] == 0, name


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,n,k", [([7], 96, 1000), ([3, 0, 40], 136, 520), ([100, 90], 264, 328), ([700, 300, 411], 2048, 2056), ([3000, 2500, 1], 4096, 4104)])
def test_values(lens, n, k, dtype):
    A, G, B, cu = inputs(real, 5, dtype, lens, n, k)
    say(f"[gpu] grouped values {dtype} N={n} K={k} lens={lens}")
    D, dA = g.grouped_product(A, B, ints(cu)), g.grouped_product_grad_input(G, B, ints(cu))
    dB, dB32 = g.grouped_product_grad_weight(G, A, ints(cu)), g.grouped_product_grad_weight(G, A, ints(cu), dtype=torch.float32)
    torch.cuda.synchronize()
    ref.check(D, *ref.product(A, B, cu, D), "product")
    ref.check(dA, *ref.grad_input(G, B, cu, dA), "grad_input")
    ref.check(dB, *ref.grad_weight(G, A, cu), "grad_weight")
    ref.check(dB32, *ref.grad_weight(G, A, cu), "grad_weight, fp32")
    assert torch.equal(dB32.to(TYPES[dtype]), dB)   # one rounding of the same sums


# (lens, ids, N, K, rank)
ADAPTERS = [
    ([1], [0], 8, 8, 8),
    ([1], [-1], 64, 72, 16),
    ([16], [2], 40, 2000, 16),                             # one request of few rows
    ([3], [1], 4104, 1032, 48),
    ([7], [3], 264, 256, 24),
    ([0], [1], 64, 64, 8),
    ([2, 0, 5, 1, 1, 0, 3], [1, 0, -1, 3, 7, 2, 0], 72, 264, 16),
    ([1, 1], [2, 2], 520, 1024, 40),
    ([1] * 7 + [0, 5], [0, 1, 2, 3, -1, 9, 3, 1, 2], 2056, 4096, 16),   # up to 16, 32 and 64 rows
    ([20, 1, 3], [3, -1, 1], 1032, 2056, 128),
    ([1] * 64, [b % 4 for b in range(64)], 4104, 520, 24),
    ([64], [2], 72, 8200, 64),
    ([17], [2], 136, 520, 40),
    ([1] * 40, [b % 7 - 1 for b in range(40)], 136, 264, 16),
    ([1] * 130, [b % 3 for b in range(130)], 264, 128, 24),
    ([3, 0, 40, 1, 1, 0, 0, 17], [1, 0, 2, 2, -1, 9, 1, 0], 520, 520, 128),
    ([200, 1, 0, 77, 400], [0, 1, 2, -5, 3], 264, 136, 64),
    ([1500, 300, 1, 2, 700], [3, 3, 0, 1, 2], 4104, 200, 40),
    ([2100, 0, 900, 3, 1500], [1, 0, -1, 2, 3], 4104, 1032, 64),   # large tiles of one request each
    ([4352], [2], 4104, 2056, 24),                                 # and of a small last round, in parts
    ([257, 4000, 255], [2, 3, 0], 4096, 2048, 8),
]


def adapter_inputs(make, seed, dtype, case, before=0, behind=0, pad=0):
    lens, ids, n, k, rank = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows = before + sum(lens) + behind
    A = make(gen, dtype, rows, k)
    A[:before] = NAN
    A[rows - behind:] = NAN
    count = max(4, max(ids) + 1 if max(ids) < 9 else 4)
    B, down, up = make(gen, dtype, n, k), make(gen, dtype, count, rank, k), make(gen, dtype, count, n, rank)
    return [padded(x, pad) for x in (A, B, down, up)] + [starts(lens, before), ids]


@pytest.mark.parametrize("case", range(len(ADAPTERS)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("pad", [0, 8])
def test_adapters_whole_numbers(pad, dtype, case):
    A, B, down, up, cu, ids = adapter_inputs(whole, 300 + case, dtype, ADAPTERS[case], 3 if pad else 0, 5 if pad else 0, pad)
    # few enough products for low-rank values that both types hold: at most 8 of 2 * 2, times 2
    keep = torch.zeros(down.shape[-1], dtype=torch.bool, device=DEV)
    keep[torch.randperm(down.shape[-1], generator=torch.Generator().manual_seed(case))[:8].to(DEV)] = True
    down *= keep
    scales = torch.tensor([0.5, 1.0, 2.0, -1.0], device=DEV)[torch.arange(down.shape[0], device=DEV) % 4]
    n = B.shape[0]
    say(f"[gpu] adapters {dtype} {ADAPTERS[case][2:]} pad={pad} rows={A.shape[0]}")
    for s in (scales, None):
        D = kept(dtype, A.shape[0], n, pad)
        assert g.adapter_product(A, B, down, up, ints(cu), ints(ids), s, D=D) is D
        torch.cuda.synchronize()
        want, _ = ref.adapters(A, B, down, up, cu, ids, s, kept(dtype, A.shape[0], n))
        assert torch.equal(D, want.to(TYPES[dtype]))


@pytest.mark.parametrize("case", range(len(ADAPTERS)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_adapters_values(dtype, case):
    A, B, down, up, cu, ids = adapter_inputs(real, 400 + case, dtype, ADAPTERS[case])
    scales = torch.linspace(-1.5, 2.0, down.shape[0], device=DEV)
    say(f"[gpu] adapter values {dtype} {ADAPTERS[case][2:]}")
    D = g.adapter_product(A, B, down / 8, up, ints(cu), ints(ids), scales)
    torch.cuda.synchronize()
    ref.check(D, *ref.adapters(A, B, down / 8, up, cu, ids, scales, D), "adapters")

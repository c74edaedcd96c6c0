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
    ([150, 120, 140, 90], 8200, 200),
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
    ([100, 0, 60, 35], [1, 0, -1, 3], 520, 2056, 16),              # projections beside the shared product
    ([1] * 90, [b % 5 - 1 for b in range(90)], 264, 4104, 40),
    ([70], [2], 2056, 2048, 8),
    ([300, 1, 411], [3, 3, 0], 1032, 4104, 128),
    ([65, 2, 700, 0, 1], [-1, 0, 2, 1, 9], 264, 7688, 24),
    ([1] * 300, [b % 5 - 1 for b in range(300)], 4104, 2056, 64),   # more single tokens than tiles have rows
    ([2, 1, 0, 3] * 25, [b * 7 % 4 for b in range(100)], 1032, 1032, 128),
    ([1] * 100, [b % 6 - 1 for b in range(100)], 14344, 520, 8),
    ([200, 200], [1, 0], 2048, 4096, 64),                           # few tiles, requests of many rows
    ([128, 70, 1, 57], [2, 0, -1, 3], 520, 4104, 64),
    ([100, 90], [3, 1], 1032, 1544, 128),
    ([4096, 2, 4094], [1, 3, 2], 4096, 2048, 128),                  # large tiles of several requests, a rank above 64
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


# ------------------------------------------------------------------ corners
def test_nothing_to_do():
    for t in TYPES.values():
        A, B, G = torch.zeros(4, 16, dtype=t, device=DEV), torch.zeros(2, 8, 16, dtype=t, device=DEV), torch.zeros(4, 8, dtype=t, device=DEV)
        cu = ints([0, 1, 4])
        none = ints([0, 0, 0])
        assert g.grouped_product(A[:0], B, none).shape == (0, 8)
        assert g.grouped_product_grad_input(G[:0], B, none).shape == (0, 16)
        assert bool((g.grouped_product_grad_weight(G[:0], A[:0], none) == 0).all())      # every matrix is written
        assert bool((g.grouped_product_grad_weight(G, A, none, dtype=torch.float32) == 0).all())
        assert g.grouped_product(A, B[:, :0], cu).shape == (4, 0)
        assert bool((g.grouped_product(A[:, :0], B[:, :, :0], cu) == 0).all())            # a contraction of nothing
        assert bool((g.grouped_product_grad_input(G[:, :0], B[:, :0], cu) == 0).all())
        kept_D, kept_A = torch.full_like(G, 3.0), torch.full_like(A, 3.0)
        g.grouped_product(A, B[:0], ints([0]), D=kept_D)                                 # no group
        g.grouped_product_grad_input(G, B, none, dA=kept_A)                              # no rows in any
        ad = [torch.zeros(3, 8, 16, dtype=t, device=DEV), torch.zeros(3, 8, 8, dtype=t, device=DEV)]
        g.adapter_product(A, B[0], *ad, ints([2, 2]), ints([0]), D=kept_D)
        g.adapter_product(A, B[0], *ad, ints([0]), ints([]), D=kept_D)
        out = g.adapter_product(A, B[0], ad[0][:, :0], ad[1][:, :, :0], ints([0, 4]), ints([0]))   # rank 0
        torch.cuda.synchronize()
        assert bool((kept_D == 3).all()) and bool((kept_A == 3).all()) and bool((out == 0).all())


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("lens,n,k", [([3, 2], 64, 72), ([40, 50], 264, 520), ([2100, 1300], 4104, 264), ([2100, 1300], 264, 4104)])
def test_what_is_not_finite_stays_where_it_is(lens, n, k, dtype):
    # a row with NaN and infinities spoils itself, a matrix with them its own group
    A, G, B, cu = inputs(whole, 7, dtype, lens, n, k)
    bad = lens[0] - 1
    clean = [g.grouped_product(A, B, ints(cu)), g.grouped_product_grad_input(G, B, ints(cu)), g.grouped_product_grad_weight(G, A, ints(cu))]
    A2, G2, B2 = A.clone(), G.clone(), B.clone()
    A2[bad, ::3], G2[bad, ::3], B2[1, ::2] = NAN, float("inf"), float("-inf")
    D, dA = g.grouped_product(A2, B, ints(cu)), g.grouped_product_grad_input(G2, B, ints(cu))
    D2, dA2 = g.grouped_product(A, B2, ints(cu)), g.grouped_product_grad_input(G, B2, ints(cu))
    dB = g.grouped_product_grad_weight(G, A2, ints(cu))
    torch.cuda.synchronize()
    rest = [r for r in range(sum(lens)) if r != bad]
    assert torch.equal(D[rest], clean[0][rest]) and bool(torch.isnan(D[bad]).all())
    assert torch.equal(dA[rest], clean[1][rest]) and not bool(torch.isfinite(dA[bad]).any())
    assert torch.equal(D2[:lens[0]], clean[0][:lens[0]]) and torch.equal(dA2[:lens[0]], clean[1][:lens[0]])
    assert not bool(torch.isfinite(D2[lens[0]:, ::2]).any())
    assert torch.equal(D2[lens[0]:, 1::2], clean[0][lens[0]:, 1::2])   # other rows of the matrix
    assert torch.equal(dB[1], clean[2][1]) and torch.equal(dB[0][:, 1], clean[2][0][:, 1])


@pytest.mark.parametrize("case", [2, 4, 5, 8, 11, 13, 18, 22, 23, 25])
def test_adapters_that_no_row_asks_for(case):
    lens, ids, n, k, rank = ADAPTERS[case]
    ids = [i if i % 2 == 0 else -1 for i in ids]
    A, B, down, up, cu, _ = adapter_inputs(whole, 500 + case, "fp16", (lens, ids, n, k, rank))
    down[..., 8:] = 0
    want, _ = ref.adapters(A, B, down, up, cu, ids, None, kept("fp16", A.shape[0], n))
    down[1::2], up[1::2] = NAN, float("inf")
    D = g.adapter_product(A, B, down, up, ints(cu), ints(ids))
    torch.cuda.synchronize()
    assert torch.equal(D, want.to(torch.float16))


SPOILT = [ADAPTERS[i] for i in (6, 7, 8, 9, 10, 13, 14, 15, 16, 17, 18, 20, 21, 22, 24, 25, 26, 27, 28, 29, 30, 31)] + [
    ([1, 2], [0, 1], 264, 1032, 16), ([2, 1, 1], [2, 0, 1], 72, 520, 8), ([3, 90], [1, 2], 136, 200, 8), ([1] * 200, [b % 4 for b in range(200)], 136, 72, 8)]


@pytest.mark.parametrize("case", range(len(SPOILT)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("bad", [NAN, float("inf")])
def test_an_adapter_that_is_not_finite_spoils_its_own_rows_alone(bad, dtype, case):
    lens, ids, n, k, rank = SPOILT[case]
    A, B, down, up, cu, ids = adapter_inputs(real, 900 + case, dtype, SPOILT[case])
    spoilt = next(a for ln, a in zip(lens, ids) if ln and 0 <= a < down.shape[0])
    clean = g.adapter_product(A, B, down / 8, up, ints(cu), ints(ids))
    up = up.clone()
    up[spoilt, 1::3, rank // 2] = bad
    say(f"[gpu] adapter {spoilt} holds {bad}, {dtype} {SPOILT[case][2:]}")
    D = g.adapter_product(A, B, down / 8, up, ints(cu), ints(ids))
    torch.cuda.synchronize()
    whose = torch.repeat_interleave(torch.tensor(ids[:len(lens)], device=DEV), torch.tensor(lens, device=DEV))
    hit = (whose == spoilt)[:, None] & (torch.arange(n, device=DEV) % 3 == 1)[None]
    assert bool(hit.any()) and not bool(torch.isfinite(D[hit]).any())
    assert torch.equal(D[~hit], clean[~hit])


def test_tables_that_decrease_or_run_past_the_rows():
    # not a valid call; it has to stay inside its tensors all the same
    gen = torch.Generator(device=DEV).manual_seed(3)
    for rows, n, k, tables in ((50, 72, 264, ([0, 90, -5, 60], [40, 30, 20, 10], [7, 7, 1 << 30, 50], [-1, -1, -1, -1])),
                               (700, 264, 4104, ([0, 700, 0, 700], [900, 10, 800, 5])), (5000, 2056, 2056, ([0, 5000, 1, 9000],))):
        A, G, B = whole(gen, "bf16", rows, k), whole(gen, "bf16", rows, n), whole(gen, "bf16", 3, n, k)
        down, up = whole(gen, "bf16", 2, 16, k), whole(gen, "bf16", 2, n, 16)
        for table in tables:
            say(f"[gpu] table {table} of {rows} rows")
            cu = ints(table)
            guard = [torch.full((rows + 2, w), 5.0, dtype=torch.bfloat16, device=DEV) for w in (n, k, n)]
            g.grouped_product(A, B, cu, D=guard[0][1:-1])
            g.grouped_product_grad_input(G, B, cu, dA=guard[1][1:-1])
            g.grouped_product_grad_weight(G, A, cu)
            g.adapter_product(A, B[0], down, up, cu, ints([1, 0, 1]), D=guard[2][1:-1])
            torch.cuda.synchronize()
            for x in guard:
                assert bool((x[0] == 5).all()) and bool((x[-1] == 5).all())


def test_offsets_beyond_32_bits():
    gen = torch.Generator(device=DEV).manual_seed(9)
    n, k, lens, t = 136, 264, [700, 0, 300], torch.float16
    rows, cu = 1000, starts(lens)
    pitch = 1 << 21   # 1000 rows of 4 MiB: 4 GiB
    A, G, B = whole(gen, "fp16", rows, k), whole(gen, "fp16", rows, n), whole(gen, "fp16", 3, n, k)

    def spread(x, step):
        shape = list(x.shape)
        base = torch.empty((shape[0] - 1) * step + shape[-1] * (shape[1] if len(shape) == 3 else 1), dtype=x.dtype, device=DEV)
        view = base.as_strided(shape, [step, shape[-1], 1][:1] + ([shape[-1], 1] if len(shape) == 3 else [1]))
        view.copy_(x)
        return view

    A2, G2, B2 = spread(A, pitch), spread(G, pitch), spread(B, 3 << 30)
    D = spread(torch.zeros(rows, n, dtype=t, device=DEV), pitch)
    say("[gpu] far rows and matrices")
    g.grouped_product(A2, B2, ints(cu), D=D)
    dA = g.grouped_product_grad_input(G2, B2, ints(cu), dA=spread(torch.zeros(rows, k, dtype=t, device=DEV), pitch))
    dB = g.grouped_product_grad_weight(G2, A2, ints(cu), dB=spread(torch.zeros(3, n, k, dtype=t, device=DEV), 3 << 30))
    ids = [1, 0, 2]
    down, up = whole(gen, "fp16", 3, 8, k), whole(gen, "fp16", 3, n, 8)
    E = g.adapter_product(A2, B2[1], spread(down, 3 << 30), spread(up, 3 << 30), ints(cu), ints(ids))
    torch.cuda.synchronize()
    assert torch.equal(D, ref.product(A, B, cu, D)[0].to(t)) and torch.equal(dA, ref.grad_input(G, B, cu, dA)[0].to(t))
    assert torch.equal(dB, ref.grad_weight(G, A, cu)[0].to(t))
    ref.check(E, *ref.adapters(A, B[1], down, up, cu, ids, None, E), "adapters")


def test_many_rows_of_a_long_group():
    # a contraction over rows whose offsets pass 2^32 bytes: not the large tiles' kernel
    rows, n, k = 140000, 264, 256
    gen = torch.Generator(device=DEV).manual_seed(10)
    A = torch.zeros(rows, 16384, dtype=torch.bfloat16, device=DEV)[:, :k]
    A.copy_(whole(gen, "bf16", rows, k))
    G = whole(gen, "bf16", rows, n)
    dB = g.grouped_product_grad_weight(G, A, ints([0, rows - 5, rows]), dtype=torch.float32)
    torch.cuda.synchronize()
    want, _ = ref.grad_weight(G, A, [0, rows - 5, rows])
    assert torch.equal(dB, want.float())


# -------------------------------------------- streams, graphs, calls together
def layer(dtype, seed, lens, n, k):
    A, G, B, cu = inputs(whole, seed, dtype, lens, n, k)
    return A, G, B, ints(cu)


def all_three(A, G, B, cu):
    return (g.grouped_product(A, B, cu), g.grouped_product_grad_input(G, B, cu), g.grouped_product_grad_weight(G, A, cu, dtype=torch.float32))


@pytest.mark.parametrize("lens,n,k", [([5, 0, 9], 72, 264), ([207, 50], 264, 6152), ([2200], 4104, 2056)])
def test_another_stream_and_two_at_once(lens, n, k):
    first, second = layer("fp16", 20, lens, n, k), layer("fp16", 21, lens, n, k)
    want = [all_three(*first), all_three(*second)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, args in enumerate((first, second)):
            with torch.cuda.stream(streams[i]):
                got[i] = all_three(*args)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("lens,n,k", [([5, 0, 9], 72, 264), ([207, 50, 0], 264, 6152), ([2200, 0, 100], 2056, 4104)])
def test_captured_graph(lens, n, k):
    # replays see new values and new offsets, with eager calls of the same between them
    A, G, B, cu = layer("bf16", 30, lens, n, k)
    gen = torch.Generator(device=DEV).manual_seed(31)
    down, up = whole(gen, "bf16", 3, 16, k), whole(gen, "bf16", 3, n, 16)
    down[..., 8:] = 0
    ids, rows = ints([2, 0, 1][:len(lens)]), sum(lens)
    D, dA = torch.zeros(rows, n, dtype=A.dtype, device=DEV), torch.zeros(rows, k, dtype=A.dtype, device=DEV)

    def run(D, dA):
        return (g.grouped_product(A, B, cu, D=D), g.grouped_product_grad_input(G, B, cu, dA=dA), g.grouped_product_grad_weight(G, A, cu),
                g.adapter_product(A, B[0], down, up, cu, ids))

    run(D, dA)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(D, dA)
    for step, share in enumerate((0.5, 0.0, 1.0, 0.25)):
        A.copy_(whole(gen, "bf16", rows, k))
        G.copy_(whole(gen, "bf16", rows, n))
        cut = int(rows * share)
        cu.copy_(ints([0, cut, rows, rows][:len(lens) + 1]))
        D.fill_(7)
        dA.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        want = run(torch.full_like(D, 7), torch.full_like(dA, 7))
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y), step


def test_given_workspaces():
    A, G, B, cu = layer("fp16", 40, [207, 50], 264, 6152)
    need = g.grouped_product_workspace(A, B, cu)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)   # NaN as fp32
    D = g.grouped_product(A, B, cu, workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.equal(D, g.grouped_product(A, B, cu)) and bool((ws[need:] == 0xff).all())
    with pytest.raises(g.GemmError):
        g.grouped_product(A, B, cu, workspace=ws[:need - 1])
    with pytest.raises(g.GemmError):
        g.grouped_product(A, B, cu, workspace=ws[8:])
    with pytest.raises(g.GemmError):   # over an input
        g.grouped_product(A, B, cu, workspace=B.view(torch.uint8))
    for rows in (9, 50, 300, 5000):
        A, B = torch.ones(rows, 520, dtype=torch.float16, device=DEV), torch.ones(264, 520, dtype=torch.float16, device=DEV)
        down, up = torch.ones(2, 40, 520, dtype=torch.float16, device=DEV), torch.ones(2, 264, 40, dtype=torch.float16, device=DEV)
        cu, ids = ints([0, 5, rows]), ints([1, 0])
        need = g.adapter_product_workspace(A, B, down / 64, up, cu, ids)
        assert need > 0
        ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)
        D = g.adapter_product(A, B, down / 64, up, cu, ids, workspace=ws[:need])
        torch.cuda.synchronize()
        assert bool((D == 520 + 40 * 520 / 64).all()) and bool((ws[need:] == 0xff).all())
        with pytest.raises(g.GemmError):
            g.adapter_product(A, B, down, up, cu, ids, workspace=ws[:need - 16])


def test_refused_tensors():
    t = torch.float16
    A, B, G, cu = (torch.zeros(4, 16, dtype=t, device=DEV), torch.zeros(2, 8, 16, dtype=t, device=DEV), torch.zeros(4, 8, dtype=t, device=DEV),
                   ints([0, 1, 4]))
    down, up, ids = torch.zeros(3, 8, 16, dtype=t, device=DEV), torch.zeros(3, 8, 8, dtype=t, device=DEV), ints([0, 1])
    refused = [
        lambda: g.grouped_product(A.float(), B, cu), lambda: g.grouped_product(A.cpu(), B, cu), lambda: g.grouped_product(A[0], B, cu),
        lambda: g.grouped_product(A, B[0], cu), lambda: g.grouped_product(A, B.bfloat16(), cu), lambda: g.grouped_product(A, B, cu[:2]),
        lambda: g.grouped_product(A, B, cu.long()), lambda: g.grouped_product(A, B, cu.cpu()), lambda: g.grouped_product(A, B, ints([])),
        lambda: g.grouped_product(A[:, :8], B, cu), lambda: g.grouped_product(A, B.transpose(1, 2), cu),
        lambda: g.grouped_product(A, B, cu, D=G[:3]), lambda: g.grouped_product(A, B, cu, D=G.float()),
        lambda: g.grouped_product(A[:1].expand(4, 16), B, cu),                                             # rows on top of each other
        lambda: g.grouped_product(A, B, cu, D=A[:, :8]), lambda: g.grouped_product(A[:, :12], B[..., :12], cu),
        lambda: g.grouped_product(A.t().contiguous().t(), B, cu),
        lambda: g.grouped_product_grad_input(G.float(), B, cu), lambda: g.grouped_product_grad_input(G, B[0], cu),
        lambda: g.grouped_product_grad_input(G[:, :4], B, cu), lambda: g.grouped_product_grad_input(G, B, cu, dA=A[:2]),
        lambda: g.grouped_product_grad_input(A[:, 8:], B, cu, dA=A),
        lambda: g.grouped_product_grad_weight(G, A[:3], cu), lambda: g.grouped_product_grad_weight(G, A[0], cu),
        lambda: g.grouped_product_grad_weight(G, A, cu, dtype=torch.float64), lambda: g.grouped_product_grad_weight(G, A, cu, dB=B.double()),
        lambda: g.grouped_product_grad_weight(G, A, cu, dB=B[:1].expand(2, 8, 16)), lambda: g.grouped_product_grad_weight(G.bfloat16(), A, cu),
        lambda: g.grouped_product_grad_weight(G, A, cu, dB=B, dtype=torch.float32),
        lambda: g.adapter_product(A, B, down, up, cu, ids), lambda: g.adapter_product(A, B[0], down[0], up, cu, ids),
        lambda: g.adapter_product(A, B[0], down, up[:2], cu, ids), lambda: g.adapter_product(A, B[0], down[:, :4], up[..., :4], cu, ids),
        lambda: g.adapter_product(A, B[0], down, up, cu, ids[:1]), lambda: g.adapter_product(A, B[0], down, up, cu, ids.long()),
        lambda: g.adapter_product(A, B[0], down, up, cu, ids, torch.ones(2, device=DEV)),
        lambda: g.adapter_product(A, B[0], down, up, cu, ids, torch.ones(3, device=DEV, dtype=t)),
        lambda: g.adapter_product(A, B[0], down, up, cu, ids, torch.ones(3)),
        lambda: g.adapter_product(A, B[0], down, up, cu, ids, D=A[:, :8]),
        lambda: g.adapter_product(A, B[0], down, up, cu, ids, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
    ]
    for i, call in enumerate(refused):
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            call()
            pytest.fail(f"call {i} was taken")
    torch.cuda.synchronize()


# ------------------------------------------------------------- used together
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_gradients_against_differences(dtype):
    # the products are linear in each operand: a step's difference is the gradient's product with it, exactly for whole numbers
    lens, n, k = [3, 0, 30, 7], 72, 136
    gen = torch.Generator(device=DEV).manual_seed(50)
    A, G, B, cu = inputs(whole, 51, dtype, lens, n, k)
    cu = ints(cu)
    dA, dB = g.grouped_product_grad_input(G, B, cu).double(), g.grouped_product_grad_weight(G, A, cu, dtype=torch.float32).double()
    step_A, step_B = torch.zeros_like(A), torch.zeros_like(B)
    step_A[5, 11], step_A[39, 0] = 1, -2
    step_B[2, 8, 9], step_B[1, 0, 0], step_B[3, 71, 135] = 1, 5, -1
    base = g.grouped_product(A, B, cu).double()
    by_A = ((g.grouped_product(A + step_A, B, cu).double() - base) * G.double()).sum()
    by_B = ((g.grouped_product(A, B + step_B, cu).double() - base) * G.double()).sum()
    bound = 2.0 ** -8 * float((base.abs() + 4 * k).max()) * float(G.double().abs().sum()) if dtype == "bf16" else 0.0   # bf16 outputs above 256 are rounded
    assert abs(float(by_A - (dA * step_A.double()).sum())) <= bound + (2.0 ** -8 * float((dA.abs() * step_A.double().abs()).sum()) if dtype == "bf16" else 0)
    assert abs(float(by_B - (dB * step_B.double()).sum())) <= bound


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_a_layer_of_experts(dtype):
    # forward and backward of two products with an activation between them, tokens sent to two experts each and joined again,
    # against 64 bits; each product's own rounding is taken from its own output, so that the bounds stay those of one product
    gen = torch.Generator(device=DEV).manual_seed(60)
    tokens, d, hidden, experts, t = 150, 136, 264, 6, TYPES[dtype]
    X, W1, W2 = real(gen, dtype, tokens, d), real(gen, dtype, experts, hidden, d) / 8, real(gen, dtype, experts, d, hidden) / 8
    choice = torch.stack([torch.randperm(experts, generator=torch.Generator().manual_seed(i))[:2] for i in range(tokens)]).flatten()
    order = torch.argsort(choice, stable=True).to(DEV)
    counts = torch.bincount(choice, minlength=experts)
    cu_host = [0] + torch.cumsum(counts, 0).tolist()
    cu = ints(cu_host)
    A = X[order // 2]
    H = g.grouped_product(A, W1, cu)
    ref.check(H, *ref.product(A, W1, cu_host, H), "first product")
    R = torch.relu(H)
    Y = g.grouped_product(R, W2, cu)
    ref.check(Y, *ref.product(R, W2, cu_host, Y), "second product")
    out = torch.zeros(tokens, d, dtype=torch.float32, device=DEV).index_add_(0, order // 2, Y.float())
    gY = out.to(t)[order // 2]          # the gradient of half the outputs' squares
    gR = g.grouped_product_grad_input(gY, W2, cu)
    ref.check(gR, *ref.grad_input(gY, W2, cu_host, gR), "gradient for the second input")
    gW2 = g.grouped_product_grad_weight(gY, R, cu, dtype=torch.float32)
    ref.check(gW2, *ref.grad_weight(gY, R, cu_host), "gradient for the second weights")
    gH = torch.where(H > 0, gR, torch.zeros_like(gR))
    gW1 = g.grouped_product_grad_weight(gH, A, cu)
    ref.check(gW1, *ref.grad_weight(gH, A, cu_host), "gradient for the first weights")
    gA = g.grouped_product_grad_input(gH, W1, cu)
    ref.check(gA, *ref.grad_input(gH, W1, cu_host, gA), "gradient for the first input")
    # the whole, in 64 bits with the activations' signs of above: errors of 1 part in 2^6 of the largest, 2^-8 for each of
    # the roundings behind one another (H, Y, out, gR) and as much again for their way through 264 products of random sign
    A64, W1_64, W2_64 = A.double().requires_grad_(), W1.double().requires_grad_(), W2.double().requires_grad_()
    ys = []
    for e in range(experts):
        rows = slice(cu_host[e], cu_host[e + 1])
        ys.append((A64[rows] @ W1_64[e].t() * (H[rows] > 0).double()) @ W2_64[e].t())
    total = torch.zeros(tokens, d, dtype=torch.float64, device=DEV).index_add_(0, order // 2, torch.cat(ys))
    (total ** 2).sum().div(2).backward()
    for got, want in ((gA, A64.grad), (gW1, W1_64.grad), (gW2, W2_64.grad)):
        assert float((got.double() - want).abs().max()) <= float(want.abs().max()) / 64


def test_a_serving_step():
    # projections with the requests' adapters feed the attention over their prompts
    gen = torch.Generator(device=DEV).manual_seed(70)
    heads, kv, hd, d, lens, ids = 4, 2, 64, 256, [5, 1, 40], [1, -1, 0]
    t, rows, cu_host = torch.float16, sum(lens), starts(lens)
    X, W = real(gen, "fp16", rows, d), real(gen, "fp16", (heads + 2 * kv) * hd, d) / 16
    down, up, scales = real(gen, "fp16", 2, 16, d) / 16, real(gen, "fp16", 2, W.shape[0], 16) / 4, torch.tensor([0.5, 2.0], device=DEV)
    cu = ints(cu_host)
    qkv = g.adapter_product(X, W, down, up, cu, ints(ids), scales)
    ref.check(qkv, *ref.adapters(X, W, down, up, cu_host, ids, scales, qkv), "adapters")
    q, k, v = qkv.view(rows, heads + 2 * kv, hd).split([heads, kv, kv], 1)
    O, lse = g.attention_prompt(q, k, v, cu, return_lse=True)
    torch.cuda.synchronize()
    from tests import attention_ref

    attention_ref.prompt(q.cpu(), k.cpu(), v.cpu(), cu_host, cu_host, True, hd ** -0.5, O.cpu(), lse.cpu(), "attention of the projections")


@pytest.mark.parametrize("lens", [[1], [3, 37], [100, 1, 60], [700, 0, 1500], [4352]])
def test_adapters_of_no_contraction(lens):
    rows, n, rank = sum(lens), 264, 16
    A, B = torch.empty(rows, 0, dtype=torch.float16, device=DEV), torch.empty(n, 0, dtype=torch.float16, device=DEV)
    down, up = torch.empty(2, rank, 0, dtype=torch.float16, device=DEV), torch.full((2, n, rank), 3.0, dtype=torch.float16, device=DEV)
    D = g.adapter_product(A, B, down, up, ints(starts(lens)), ints([b % 3 - 1 for b in range(len(lens))]), D=kept("fp16", rows, n))
    torch.cuda.synchronize()
    assert bool((D == 0).all())


@pytest.mark.parametrize("lens,n,k", [([5, 0, 9], 72, 264), ([300, 411, 77], 1032, 520), ([2100, 900, 2000], 4104, 264)])
def test_one_matrix_for_all_groups(lens, n, k):
    # matrices that are read may repeat
    A, G, B, cu = inputs(whole, 17, "bf16", lens, n, k)
    same, first = B[:1].expand(len(lens), n, k), B[:1]
    D, dA = g.grouped_product(A, same, ints(cu)), g.grouped_product_grad_input(G, same, ints(cu))
    one = ints([0, sum(lens)])
    want, want_A = ref.product(A, first, [0, sum(lens)], D)[0], ref.grad_input(G, first, [0, sum(lens)], dA)[0]
    torch.cuda.synchronize()
    assert torch.equal(D, want.to(torch.bfloat16)) and torch.equal(dA, want_A.to(torch.bfloat16))
    assert torch.equal(g.grouped_product(A, first, one), D)
    with pytest.raises(g.GemmError):   # but not those that are written
        g.grouped_product_grad_weight(G, A, ints(cu), dB=torch.empty_like(first).expand(len(lens), n, k))


@pytest.mark.parametrize("rows", [64, 500, 6000])
def test_few_rows_of_a_long_tensor(rows):
    # a batch padded to its largest size: the tables say how many rows there are
    gen = torch.Generator(device=DEV).manual_seed(rows)
    n, k = 1032, 2056
    A, B, down, up = whole(gen, "fp16", rows, k), whole(gen, "fp16", 2, n, k), whole(gen, "fp16", 2, 24, k), whole(gen, "fp16", 2, n, 24)
    down[:, 8:] = 0
    A[5:], G = NAN, whole(gen, "fp16", rows, n)
    G[5:] = NAN
    for cu in ([0, 2, 5], [0, 0, 0]):
        D, E, dA = kept("fp16", rows, n), kept("fp16", rows, n), kept("fp16", rows, k)
        g.grouped_product(A, B, ints(cu), D=D)
        g.grouped_product_grad_input(G, B, ints(cu), dA=dA)
        dB = g.grouped_product_grad_weight(G, A, ints(cu))
        g.adapter_product(A / 8, B[0], down, up, ints(cu), ints([1, 0]), D=E)
        torch.cuda.synchronize()
        assert torch.equal(D, ref.product(A, B, cu, kept("fp16", rows, n))[0].to(torch.float16))
        assert torch.equal(dA, ref.grad_input(G, B, cu, kept("fp16", rows, k))[0].to(torch.float16))
        assert torch.equal(dB, ref.grad_weight(G, A, cu)[0].to(torch.float16))
        assert bool((E[cu[-1]:] == 7).all())
        if cu[-1]:
            ref.check(E[:5], *[x[:5] for x in ref.adapters(A / 8, B[0], down, up, cu, [1, 0], None, kept("fp16", rows, n))], "adapters")


@pytest.mark.parametrize("lens,n,k,rank", [([1], 264, 1032, 16), ([1] * 8, 264, 520, 24), ([1] * 100, 1032, 2056, 16), ([200, 200], 2048, 4096, 64), ([700, 3, 90], 520, 264, 40), ([2100, 900], 4104, 1032, 64)])
def test_adapters_captured_and_on_two_streams(lens, n, k, rank):
    gen = torch.Generator(device=DEV).manual_seed(51)
    rows = sum(lens)
    A, B, down, up = whole(gen, "fp16", rows, k), whole(gen, "fp16", n, k), whole(gen, "fp16", 4, rank, k), whole(gen, "fp16", 4, n, rank)
    down[:, 8:] = 0
    cu, ids = ints(starts(lens)), ints([b % 5 - 1 for b in range(len(lens))])
    scales = torch.tensor([1.0, 0.5, 0.25, -0.125], device=DEV)
    D = torch.zeros(rows, n, dtype=torch.float16, device=DEV)
    g.adapter_product(A, B, down, up, cu, ids, scales, D=D)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.adapter_product(A, B, down, up, cu, ids, scales, D=D)
    other = torch.cuda.Stream()
    for step in range(4):
        A.copy_(whole(gen, "fp16", rows, k))
        ids.copy_(torch.randint(-1, 5, ids.shape, generator=gen, device=DEV))
        if step > 1:   # fewer rows in use
            cu.clamp_(max=max(1, rows // step))
        D.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):   # at the same time
            beside = g.adapter_product(A, B, down, up, cu, ids, scales, D=torch.full_like(D, 7))
        torch.cuda.synchronize()
        alone = g.adapter_product(A, B, down, up, cu, ids, scales, D=torch.full_like(D, 7))
        torch.cuda.synchronize()
        assert torch.equal(D, alone) and torch.equal(beside, alone), step

"""The attention operators far from ordinary values, each on every way that a call can take through the kernels."""
import math
import sys

import pytest

import dense_fp16_gemm_nt_amd as g
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}

# (queries, keys, heads, kv heads, d, causal) of one prompt
PROMPTS = {
    "tiles": (150, 210, 4, 2, 128, True),
    "tiles, no mask": (150, 210, 2, 2, 64, False),
    "tiles, parts": (200, 1500, 2, 1, 96, False),
    "eight waves": (2048, 3001, 32, 32, 128, True),
    "eight waves, parts": (2048, 4099, 16, 16, 96, False),
    "few rows": (5, 170, 4, 1, 64, True),
    "few rows, parts": (3, 3001, 4, 2, 128, False),
}
# (batch, prefix, slot rows, heads, kv heads, d)
SHARED = {
    "one run": (3, 100, 70, 8, 2, 128),
    "one run, a wave each": (65, 61, 40, 32, 16, 64),
    "one run, parts": (1, 3001, 5, 4, 1, 96),
    "few rows": (4, 2000, 40, 4, 2, 64),
    "row tiles": (40, 1000, 300, 4, 2, 128),
    "row tiles, a wave each": (131, 600, 60, 10, 5, 80),
}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def lens_of(B, N):
    return [(N, 1, N // 2, N - 1, N + 3)[b % 5] for b in range(B)]


class Case:
    """One call: its keys laid out as the operator takes them, and for each kv head the plain problems it stands for."""

    def __init__(self, way):
        self.way = way
        kind, name = way.split(": ")
        self.prompt = kind == "prompt"
        if self.prompt:
            self.n, self.m, self.heads, self.kv_heads, self.d, self.causal = PROMPTS[name]
            self.rows, self.keys = self.n, self.m
        else:
            self.B, self.P, self.N, self.heads, self.kv_heads, self.d = SHARED[name]
            self.rows, self.keys = self.B, self.P + self.B * self.N
        self.G = self.heads // self.kv_heads

    def run(self, q, k, v, scale, **kw):
        """q (rows, heads, d), k and v (keys, kv heads, d) on the host; a batch's keys are the prefix, then the slots."""
        print(f"[gpu] {self.way} {q.dtype} scale {scale}", file=sys.stderr, flush=True)
        q, k, v = (x.to(DEV) for x in (q, k, v))
        if self.prompt:
            O, lse = g.attention_prompt(q, k, v, ints([0, self.n]), ints([0, self.m]), causal=self.causal, scale=scale,
                                        return_lse=True, **kw)
        else:
            def slots(x):
                return x[self.P:].reshape(self.B, self.N, self.kv_heads, self.d)
            O, lse = g.attention_shared_prefix(q, k[:self.P], v[:self.P], slots(k), slots(v), ints(lens_of(self.B, self.N)),
                                               scale=scale, return_lse=True, **kw)
        torch.cuda.synchronize()
        return O.cpu(), lse.cpu()

    def problems(self, q, k, v):
        """(rows of O, heads, q, k, v, allowed) in 64 bits; of many heads and rows a few."""
        for j in sorted({0, self.kv_heads - 1}):
            h = slice(j * self.G, (j + 1) * self.G)
            if self.prompt:
                rows = torch.arange(self.n) if self.n <= 300 else torch.arange(self.n - 150, self.n)
                qq = q[rows][:, h].double().reshape(-1, self.d)
                allowed = torch.ones(len(rows), self.m, dtype=torch.bool)
                if self.causal:
                    allowed = torch.arange(self.m)[None, :] <= rows[:, None] + (self.m - self.n)
                yield rows, h, qq, k[:, j].double(), v[:, j].double(), allowed.repeat_interleave(self.G, 0)
                continue
            for b, n in enumerate(lens_of(self.B, self.N)):
                if b % 7 not in (0, 1, 4) and b != self.B - 1:
                    continue
                at = self.P + b * self.N
                kk, vv = (torch.cat([x[:self.P, j], x[at:at + min(n, self.N), j]]).double() for x in (k, v))
                yield torch.tensor([b]), h, q[b, h].double(), kk, vv, torch.ones(self.G, kk.shape[0], dtype=torch.bool)


WAYS = [f"prompt: {x}" for x in PROMPTS] + [f"shared: {x}" for x in SHARED]


def rand(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float32).to(TYPES[dtype])


def check(case, q, k, v, scale, O, lse, e_weight=None):
    """Against the 64-bit form.  e_weight: how far a weight may be off, relative, where the scores are exact."""
    for rows, h, qq, kk, vv, allowed in case.problems(q, k, v):
        o, l, parts, lb = ref.attend(qq, kk, vv, scale, allowed)
        if e_weight is not None:
            mass = parts[0]
            parts = (mass, (e_weight + 2 * (kk.shape[0] + 8) * 2.0 ** -22) * mass + allowed.double() @ vv.abs() * 2.0 ** -32)
        ref.check_rows(O[rows][:, h].reshape(-1, case.d), lse[rows][:, h].reshape(-1), o, l, parts, lb, q.dtype, case.way)


# ---------------------------------------------------------------- large scores
@pytest.mark.parametrize("x", [5748, 16256, -65504])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("way", WAYS)
def test_equal_large_scores(way, dtype, x):
    """All scores of a row are the same 10^8 to 10^11 in size: its weights are the same, whatever an fp32 step is there."""
    case = Case(way)
    gen = torch.Generator().manual_seed(71)
    q = torch.full((case.rows, case.heads, case.d), float(abs(x))).to(TYPES[dtype])
    k = torch.full((case.keys, case.kv_heads, case.d), float(x)).to(TYPES[dtype])
    v = rand(gen, dtype, case.keys, case.kv_heads, case.d)
    O, lse = case.run(q, k, v, None)
    check(case, q, k, v, case.d ** -0.5, O, lse, 2.0 ** -20)


@pytest.mark.parametrize("far", [2048, -2048])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("way", WAYS)
def test_large_scores_that_rise(way, dtype, far):
    """Scores of +-2^22 plus whole numbers that rise from key to key, every one exact in fp32, so that softmax goes by
    their differences.  Every second row has ordinary scores.

    A weight's exponent x = (score - maximum) log2 e is off by 3 roundings of 2^-24 |x|, where |x| <= 40 counts: 2^-17 of
    the weight, with the exponential and the rescalings of a running maximum, which fall by 2^-8 each."""
    case = Case(way)
    gen = torch.Generator().manual_seed(73)
    q = torch.zeros(case.rows, case.heads, case.d)
    q[..., 0], q[..., 1], q[..., 2] = far, 256, 1
    q[1::2, :, :2] = 0
    q[1::2, :, 2] = 1 / 64
    level = torch.arange(case.keys)
    if not case.prompt:   # the slots go on from the prefix's last key
        level[case.P:] = case.P + (level[case.P:] - case.P) % case.N
    level = (level // 3)[:, None] + torch.randint(0, 6, (case.keys, case.kv_heads), generator=gen)
    k = torch.zeros(case.keys, case.kv_heads, case.d)
    k[..., 0], k[..., 1], k[..., 2] = 2048, level // 256, level % 256
    q, k = q.to(TYPES[dtype]), k.to(TYPES[dtype])
    v = rand(gen, dtype, case.keys, case.kv_heads, case.d)
    O, lse = case.run(q, k, v, 1.0)
    check(case, q, k, v, 1.0, O, lse, 2.0 ** -17)
    O, lse = case.run(q, k.flip(0), v, 1.0)
    check(case, q, k.flip(0), v, 1.0, O, lse, 2.0 ** -17)


# ---------------------------------------------------------------- values near the ends of the range
@pytest.mark.parametrize("exponent", [120, -60])
@pytest.mark.parametrize("way", WAYS)
def test_values_times_a_power_of_two(way, exponent):
    """V times 2^e gives O times 2^e, bit for bit, as long as 2^e V is well inside bf16's range."""
    case = Case(way)
    gen = torch.Generator().manual_seed(79)
    q, k = rand(gen, "bf16", case.rows, case.heads, case.d) * 2, rand(gen, "bf16", case.keys, case.kv_heads, case.d)
    v = rand(gen, "bf16", case.keys, case.kv_heads, case.d)
    one, lse = case.run(q, k, v, None)
    check(case, q, k, v, case.d ** -0.5, one, lse)
    far, lse2 = case.run(q, k, (v.double() * 2.0 ** exponent).bfloat16(), None)
    assert torch.equal(far.double(), one.double() * 2.0 ** exponent) and torch.equal(lse, lse2)


@pytest.mark.parametrize("way", WAYS)
def test_small_values(way):
    """V times 2^-100 against the plain form.  A product is off by 2^-150 at most where O's sum has no smaller bits; beside
    a largest weight of 2^-16 at least, and times 2^100 again, that is 2^-34 for each key, 2^-22 for 4099 of them, where
    the bound has 2^-9 of the weighted sum of |v|."""
    case = Case(way)
    gen = torch.Generator().manual_seed(79)
    q, k = rand(gen, "bf16", case.rows, case.heads, case.d) * 2, rand(gen, "bf16", case.keys, case.kv_heads, case.d)
    v = rand(gen, "bf16", case.keys, case.kv_heads, case.d)
    far, lse = case.run(q, k, (v.double() * 2.0 ** -100).bfloat16(), None)
    check(case, q, k, v, case.d ** -0.5, (far.double() * 2.0 ** 100).bfloat16(), lse)


@pytest.mark.parametrize("keys", [1, 2, 100])
@pytest.mark.parametrize("queries", [1, 40])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_largest_values(dtype, queries, keys):
    """Up to 100 keys of the type's largest value: their mean, which is that value again; with signs in turn, 0 for two."""
    gen = torch.Generator().manual_seed(83)
    top = torch.finfo(TYPES[dtype]).max
    q = rand(gen, dtype, queries, 2, 64).to(DEV)
    k = torch.zeros(keys, 2, 64, dtype=TYPES[dtype], device=DEV)
    v = torch.full_like(k, top)
    cq, ck = ints([0, queries]), ints([0, keys])
    print(f"[gpu] largest values {dtype} {queries} {keys}", file=sys.stderr, flush=True)
    O = g.attention_prompt(q, k, v, cq, ck, causal=False)
    assert bool((O == top).all())
    none = torch.empty(queries, 0, 2, 64, dtype=TYPES[dtype], device=DEV)
    assert bool((g.attention_shared_prefix(q, k, v, none, none, ints([0] * queries)) == top).all())
    if keys == 2:
        v[1] = -top
        assert bool((g.attention_prompt(q, k, v, cq, ck, causal=False) == 0).all())


# ---------------------------------------------------------------- scale 0
@pytest.mark.parametrize("scale", [0.0, 1e-39])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("way", WAYS)
def test_scale_zero_whatever_q_and_k_hold(way, dtype, scale):
    case = Case(way)
    gen = torch.Generator().manual_seed(89)
    q, k, v = (rand(gen, dtype, *s, case.d) for s in ((case.rows, case.heads), (case.keys, case.kv_heads),
                                                      (case.keys, case.kv_heads)))
    zeros = torch.zeros_like(k)
    k[::3, :, 1], k[1::3, :, 2], k[2::5] = math.inf, math.nan, -math.inf
    q[::2, :, 3], q[1::4] = math.nan, math.inf
    O, lse = case.run(q, k, v, scale)
    check(case, torch.zeros_like(q), zeros, v, 1.0, O, lse)


# ---------------------------------------------------------------- rows that overlap
@pytest.mark.parametrize("step", [0, 8])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m", [(150, 210), (3, 45), (130, 1500), (2, 2990)])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_prompt_rows_of_values_that_overlap(d, n, m, causal, dtype, step):
    """V's rows a step apart that is shorter than they are (0: one row for all keys).  The last row ends with an infinity;
    no key behind it, of the tile's rest, may bring it to another element."""
    gen = torch.Generator().manual_seed(97)
    H = 2
    q, k = rand(gen, dtype, n, H, d), rand(gen, dtype, m, H, d)
    flat = rand(gen, dtype, H, (m - 1) * step + d)

    def view(x):
        return x.as_strided((m, H, d), (step, x.shape[1], 1))

    flat[:, -1] = math.inf
    print(f"[gpu] overlapping values {n} {m} {causal} {dtype} {step}", file=sys.stderr, flush=True)
    O, lse = g.attention_prompt(q.to(DEV), k.to(DEV), view(flat.to(DEV)), ints([0, n]), ints([0, m]), causal=causal, return_lse=True)
    O, lse = O.cpu(), lse.cpu()
    # it stands in the last element of the last key alone (step 0: of every key)
    sees = torch.zeros(n, dtype=torch.bool)
    sees[-1 if causal and step else 0:] = True
    assert not bool(torch.isfinite(O[sees][..., -1]).any()) and bool(torch.isfinite(O[~sees]).all())
    v = view(flat).clone()
    v[..., -1], O[..., -1] = 0, 0
    ref.prompt(q, k, v, [0, n], [0, m], causal, d ** -0.5, O, lse, "overlapping values")


@pytest.mark.parametrize("step", [0, 8])
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("B,P,N,heads,kv_heads", [(3, 100, 70, 4, 2), (65, 61, 40, 32, 16), (1, 3001, 5, 4, 1), (4, 2001, 40, 4, 2),
                                                  (40, 1001, 301, 4, 2), (131, 601, 61, 10, 5)])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_shared_prefix_rows_of_values_that_overlap(d, B, P, N, heads, kv_heads, dtype, step):
    gen = torch.Generator().manual_seed(101)
    q, kp, ks = rand(gen, dtype, B, heads, d), rand(gen, dtype, P, kv_heads, d), rand(gen, dtype, B, N, kv_heads, d)
    fp, fs = rand(gen, dtype, kv_heads, (P - 1) * step + d), rand(gen, dtype, B, kv_heads, (N - 1) * step + d)
    lens = [(N, N - 1, N // 2, 1)[b % 4] for b in range(B)]

    def views(p, s):
        return (p.as_strided((P, kv_heads, d), (step, p.shape[1], 1)),
                s.as_strided((B, N, kv_heads, d), (kv_heads * s.shape[2], step, s.shape[2], 1)))

    fp[:, -1] = math.inf
    for b, n in enumerate(lens):   # the last element of the slot's last readable row, and all behind it
        fs[b, :, (n - 1) * step + d - 1:] = math.inf
    print(f"[gpu] overlapping values B={B} P={P} N={N} {dtype} {step}", file=sys.stderr, flush=True)
    vp, vs = views(fp.to(DEV), fs.to(DEV))
    O, lse = g.attention_shared_prefix(q.to(DEV), kp.to(DEV), vp, ks.to(DEV), vs, ints(lens), return_lse=True)
    O, lse = O.cpu(), lse.cpu()
    assert not bool(torch.isfinite(O[..., -1]).any())
    vp, vs = (x.clone() for x in views(fp, fs))
    O[..., -1], vp[..., -1], vs[..., -1] = 0, 0, 0
    ref.shared_prefix(q, kp, vp, ks, vs, lens, d ** -0.5, O, lse, "overlapping values")


# ---------------------------------------------------------------- workspace
@pytest.mark.parametrize("n,m,heads,kv_heads", [(1024, 3072, 32, 8), (960, 3072, 32, 8), (3328, 3328, 32, 32), (1, 5000, 8, 2),
                                                (40, 40, 2, 2)])
def test_prompt_takes_the_workspace_that_was_asked_for(n, m, heads, kv_heads):
    """Exactly as many bytes as attention_prompt_workspace names are enough with and without a mask."""
    gen = torch.Generator().manual_seed(103)
    q, k, v = (rand(gen, "bf16", x, h, 128).to(DEV) for x, h in ((n, heads), (m, kv_heads), (m, kv_heads)))
    cq, ck = ints([0, n]), ints([0, m])
    either = g.attention_prompt_workspace(q, k, v, cq, ck)
    for causal in (True, False):
        need = g.attention_prompt_workspace(q, k, v, cq, ck, causal=causal)
        print(f"[gpu] workspace {n} {m} causal={causal}: {need} bytes, {either} for either", file=sys.stderr, flush=True)
        assert need <= either
        b = g.attention_prompt(q, k, v, cq, ck, causal=causal)
        for size in (need, either):
            ws = torch.full((size + 64,), 0x7F, dtype=torch.uint8, device=DEV)
            a = g.attention_prompt(q, k, v, cq, ck, causal=causal, workspace=ws[:size])
            torch.cuda.synchronize()
            assert torch.equal(a, b) and bool((ws[size:] == 0x7F).all())


# ---------------------------------------------------------------- refusals
def test_heads_without_elements_are_refused_by_the_library():
    x = torch.zeros(4, 2, 0, dtype=torch.float16, device=DEV)
    with pytest.raises(g.GemmError):
        g.attention_prompt(x, x, x, ints([0, 4]))
    with pytest.raises(g.GemmError):
        g.attention_shared_prefix(x, x, x, x[:, None], x[:, None], ints([0] * 4))

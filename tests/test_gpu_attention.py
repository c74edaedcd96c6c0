"""The attention operators on the GPU against the plain 64-bit form (attention_ref.py derives the bounds)."""
import math
import sys

import pytest

import dense_fp16_gemm_nt_amd as g
from tests import attention_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DEV = "cuda:0"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def rand(gen, dtype, *shape):
    return torch.randn(*shape, generator=gen, dtype=torch.float32).to(TYPES[dtype])


def cu(lens, first=0):
    out = [first]
    for n in lens:
        out.append(out[-1] + n)
    return out


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def run_prompt(q, k, v, cq, ck, causal, scale=None, **kw):
    say(f"[gpu] prompt q={tuple(q.shape)} k={tuple(k.shape)} {q.dtype} causal={causal} cu_q={cq[:9]} cu_k={ck[:9]}")
    O, lse = g.attention_prompt(q.to(DEV), k.to(DEV), v.to(DEV), ints(cq), ints(ck), causal=causal, scale=scale,
                                return_lse=True, **kw)
    torch.cuda.synchronize()
    return O.cpu(), lse.cpu()


def check_prompt(q, k, v, cq, ck, causal, scale=None, **kw):
    O, lse = run_prompt(q, k, v, cq, ck, causal, scale, **kw)
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    return ref.prompt(q, k, v, cq, ck, causal, s, O, lse, f"prompt {q.dtype} d={q.shape[2]} causal={causal}")


LENS = [
    ([1], [1]),
    ([33], [33]),
    ([1, 0, 2, 63, 64, 65, 127, 128, 129], [1, 0, 2, 63, 64, 65, 127, 128, 129]),
    ([5, 40, 1, 0, 130], [200, 41, 700, 3, 131]),        # chunks behind earlier keys, single tokens, keys without queries
    ([40, 3, 100, 7], [10, 0, 99, 1]),                   # fewer keys than queries, none at all
]


@pytest.mark.parametrize("lens", range(len(LENS)))
@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("heads,kv_heads,d", [(4, 1, 128), (2, 2, 64), (6, 2, 96), (5, 5, 80), (3, 1, 8), (2, 1, 40), (1, 1, 120)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(causal, heads, kv_heads, d, dtype, lens):
    gen = torch.Generator().manual_seed(1000 + 7 * lens + d)
    cq, ck = cu(LENS[lens][0]), cu(LENS[lens][1])
    q, k, v = rand(gen, dtype, cq[-1], heads, d), rand(gen, dtype, ck[-1], kv_heads, d), rand(gen, dtype, ck[-1], kv_heads, d)
    check_prompt(q, k, v, cq, ck, causal)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_many_sequences(d, dtype):
    # more sequences than lanes look at in one go, some without a token
    gen = torch.Generator().manual_seed(5)
    lens = [(7 * i) % 23 for i in range(150)]
    c = cu(lens)
    q, k, v = (rand(gen, dtype, c[-1], h, d) for h in (4, 2, 2))
    check_prompt(q, k, v, c, c, True)


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n,m,heads,kv_heads,d", [(700, 700, 2, 1, 128), (1, 3000, 8, 2, 128), (3, 2501, 4, 4, 64),
                                                  (130, 1999, 2, 2, 96), (65, 1030, 64, 1, 64)])
def test_prompt_long_keys(n, m, heads, kv_heads, d, causal, dtype):
    # few row tiles: the keys are split and joined
    gen = torch.Generator().manual_seed(n + m)
    q, k, v = rand(gen, dtype, n, heads, d), rand(gen, dtype, m, kv_heads, d), rand(gen, dtype, m, kv_heads, d)
    need = g.attention_prompt_workspace(q.to(DEV), k.to(DEV), v.to(DEV), ints([0, n]), ints([0, m]))
    assert need > 0 or m < 1000
    check_prompt(q, k, v, [0, n], [0, m], causal)


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (96, "fp16"), (64, "fp16")])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_mixed_batch(causal, d, dtype):
    # a long prompt, chunks and single tokens behind long caches in one call
    gen = torch.Generator().manual_seed(d)
    cq, ck = cu([1500, 1, 3, 70, 1]), cu([2600, 3000, 2500, 2111, 1])
    q, k, v = rand(gen, dtype, cq[-1], 4, d), rand(gen, dtype, ck[-1], 2, d), rand(gen, dtype, ck[-1], 2, d)
    check_prompt(q, k, v, cq, ck, causal)


def test_prompt_without_keys():
    q = torch.ones(5, 2, 64, dtype=torch.float16, device=DEV)
    none = torch.empty(0, 2, 64, dtype=torch.float16, device=DEV)
    O, lse = g.attention_prompt(q, none, none, ints([0, 2, 5]), ints([0, 0, 0]), return_lse=True)
    torch.cuda.synchronize()
    assert bool((O == 0).all()) and bool((lse == -float("inf")).all())
    assert g.attention_prompt(q[:0], none, none, ints([0, 0])).shape == (0, 2, 64)
    kept = torch.full_like(q, 3.0)
    g.attention_prompt(q, none, none, ints([0]), O=kept)   # no sequence
    torch.cuda.synchronize()
    assert bool((kept == 3).all())


def test_rows_do_not_depend_on_their_neighbours():
    # the same sequence alone and packed between others: the same bits where the same kernel takes it
    gen = torch.Generator().manual_seed(59)
    lens = [300, 180, 300]
    c = cu(lens)
    q, k, v = (rand(gen, "bf16", c[-1], 2, 128).to(DEV) for _ in range(3))
    packed = g.attention_prompt(q, k, v, ints(c))
    q[:c[1]] *= 30   # other values around it
    k[c[2]:] *= 30
    again = g.attention_prompt(q, k, v, ints(c))
    torch.cuda.synchronize()
    assert torch.equal(packed[c[1]:c[2]], again[c[1]:c[2]])


def test_prompt_peaked_and_large_scores():
    # maxima that rise from tile to tile, scores of several hundred
    gen = torch.Generator().manual_seed(9)
    n, d = 300, 128
    q, k, v = (rand(gen, "fp16", n, 2, d) for _ in range(3))
    k = (k.float() * torch.linspace(0.1, 6, n)[:, None, None]).half()
    check_prompt(q * 4, k, v, [0, n], [0, n], True)
    check_prompt(q * 4, k.flip(0).contiguous(), v, [0, n], [0, n], False)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 0.5])
def test_prompt_scales(scale):
    gen = torch.Generator().manual_seed(11)
    q, k, v = (rand(gen, "bf16", 150, h, 64) for h in (4, 2, 2))
    check_prompt(q, k, v, [0, 150], [0, 150], True, scale=scale)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_prompt_strides(dtype):
    gen = torch.Generator().manual_seed(13)
    c = cu([70, 129, 1])
    H, Hk, d = 6, 2, 64
    want = None
    qkv = rand(gen, dtype, c[-1], H + 2 * Hk, d)
    for layout in ("fused", "heads_first", "padded", "broadcast"):
        x = qkv.to(DEV)
        q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
        O = torch.full((c[-1], H, d), float("nan"), dtype=TYPES[dtype], device=DEV)
        if layout == "heads_first":
            q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
            O = O.transpose(0, 1).contiguous().transpose(0, 1)
        elif layout == "padded":
            pad = [torch.full((c[-1], t.shape[1], d + 24), float("nan"), dtype=t.dtype, device=DEV) for t in (q, k, v)]
            for p, t in zip(pad, (q, k, v)):
                p[:, :, 8:8 + d] = t
            q, k, v = (p[:, :, 8:8 + d] for p in pad)
            O = torch.full((c[-1], H, d + 8), float("nan"), dtype=TYPES[dtype], device=DEV)[:, :, :d]
        elif layout == "broadcast":   # every query head of its own kv head, repeated without a copy
            k, v = (t[:, :, None, :].expand(-1, -1, H // Hk, -1).as_strided(
                (c[-1], Hk, H // Hk, d), (t.stride(0), t.stride(1), 0, 1)) for t in (k, v))
            k, v = k[:, 0], v[:, 0]   # kv head 0 for the first H // Hk heads, head stride 0
            q, O = q[:, :H // Hk], O[:, :H // Hk]
        say(f"[gpu] prompt strides {layout} {dtype}")
        out = g.attention_prompt(q, k, v, ints(c), causal=True, O=O)
        torch.cuda.synchronize()
        assert out is O
        if want is None:
            want = O.cpu()
            ref.prompt(qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:], c, c, True, 1 / 8, want, None, "fused")
        elif layout == "broadcast":
            assert torch.equal(O.cpu(), want[:, :H // Hk])
        else:
            assert torch.equal(O.cpu(), want)


@pytest.mark.parametrize("splits", [False, True])
def test_prompt_rows_of_no_sequence(splits):
    # tokens before the first and behind the last sequence: left as they were
    gen = torch.Generator().manual_seed(17)
    n, m, H, d = 200, 2000 if splits else 180, 2, 64
    q, k, v = rand(gen, "fp16", n, H, d), rand(gen, "fp16", m, H, d), rand(gen, "fp16", m, H, d)
    cq, ck = [20, 90, 90, 150], [5, m // 2, m // 2, m - 30]
    O = torch.full((n, H, d), 7.0, dtype=torch.float16, device=DEV)
    lse = torch.full((n, H), 7.0, device=DEV)
    poison = torch.full_like(k, float("nan"))
    poison[5:m - 30] = k[5:m - 30]
    poison_v = torch.full_like(v, float("inf"))
    poison_v[5:m - 30] = v[5:m - 30]
    got, got_lse = run_prompt(q, poison, poison_v, cq, ck, False, O=O, lse=lse)
    ref.prompt(q, k, v, cq, ck, False, 1 / 8, got, got_lse, "inner rows")
    for x in (got, got_lse):
        assert bool((x[:20] == 7).all()) and bool((x[150:] == 7).all())


@pytest.mark.parametrize("d,dtype", [(128, "fp16"), (64, "bf16"), (96, "fp16")])
def test_prompt_neighbours_with_infinities(d, dtype):
    # every second sequence holds NaN and infinities: the others do not see them
    gen = torch.Generator().manual_seed(19)
    lens = [50, 30, 64, 10, 33, 100, 3]
    c = cu(lens)
    q, k, v = (rand(gen, dtype, c[-1], 2, d) for _ in range(3))
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    for b in range(1, len(lens), 2):
        for x, bad in ((q2, float("nan")), (k2, float("inf")), (v2, float("nan"))):
            x[c[b]:c[b + 1]] = bad
    O, lse = run_prompt(q2, k2, v2, c, c, True)
    for b in range(0, len(lens), 2):
        s = slice(c[b], c[b + 1])
        ref.prompt(q[s], k[s], v[s], [0, lens[b]], [0, lens[b]], True, 1 / math.sqrt(d), O[s], lse[s], f"sequence {b}")


@pytest.mark.parametrize("d,dtype", [(128, "fp16"), (64, "bf16"), (96, "bf16"), (72, "fp16")])
@pytest.mark.parametrize("n,m,heads,kv_heads", [(300, 300, 2, 1), (40, 700, 4, 4), (9, 300, 2, 1), (5, 2500, 4, 2), (600, 4000, 2, 2)])
def test_prompt_infinities_behind_the_mask(n, m, heads, kv_heads, d, dtype):
    """Values that are not finite, at keys that early rows of the sequence may not read: those rows do not see them, the
    later ones get infinity or NaN in the elements where they stand and finite sums in the others."""
    gen = torch.Generator().manual_seed(n + m + d)
    q, k, v = rand(gen, dtype, n, heads, d), rand(gen, dtype, m, kv_heads, d), rand(gen, dtype, m, kv_heads, d)
    inf = float("inf")
    base = m - n   # key of query 0
    bad = [(base + n // 4, 1, inf), (base + n // 3, 2, -inf), (base + n // 2, 3, float("nan")), (base + n - 1, 1, -inf),
           (base + n // 2 + 1, d - 1, inf), (base + n - 2, 2, -inf)]
    poisoned = v.clone()
    clean = v.clone()
    expect = torch.zeros(n, kv_heads, d)   # what the odd values add
    for key, e, x in bad:
        poisoned[key, 0, e] = x
        clean[key, 0, e] = 0
        expect[max(0, key - base):, 0, e] += x
    O, lse = run_prompt(q, k, poisoned, [0, n], [0, m], True)
    odd = ~torch.isfinite(expect.repeat_interleave(heads // kv_heads, 1))
    want = expect.repeat_interleave(heads // kv_heads, 1)
    assert torch.equal(torch.isnan(O) & odd, torch.isnan(want)) and torch.equal(torch.isfinite(O), ~odd)
    assert torch.equal(O.float()[torch.isinf(want)], want[torch.isinf(want)])
    # the rest against the sums without them
    full, flse = run_prompt(q, k, clean, [0, n], [0, m], True)
    ref.prompt(q, k, clean, [0, n], [0, m], True, 1 / math.sqrt(d), full, flse, "without the odd values")
    ref.prompt(q, k, clean, [0, n], [0, m], True, 1 / math.sqrt(d), torch.where(odd, full, O), lse, "beside the odd values")


# Enough rows and keys that eight waves share a tile (on 256 compute units): unsplit, split, and a batch whose short
# sequences run beside long ones in workgroups of that size.
LONG = {
    "unsplit": ([1800], [2700], 32, 16),
    "split": ([300], [6500], 48, 12),
    "batch": ([2000, 1, 40, 900, 0], [3500, 3000, 2111, 900, 40], 18, 9),
}


@pytest.mark.parametrize("kind", sorted(LONG))
@pytest.mark.parametrize("d,dtype", [(128, "fp16"), (96, "bf16"), (120, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_long_workgroups(causal, d, dtype, kind):
    q_lens, k_lens, heads, kv_heads = LONG[kind]
    gen = torch.Generator().manual_seed(67 + d)
    cq, ck = cu(q_lens), cu(k_lens)
    q, k, v = rand(gen, dtype, cq[-1], heads, d), rand(gen, dtype, ck[-1], kv_heads, d), rand(gen, dtype, ck[-1], kv_heads, d)
    O, lse = run_prompt(q, k, v, cq, ck, causal)
    # the 64-bit form for two kv heads
    G = heads // kv_heads
    for j in (0, kv_heads - 1):
        h = slice(j * G, (j + 1) * G)
        ref.prompt(q[:, h], k[:, j:j + 1], v[:, j:j + 1], cq, ck, causal, d ** -0.5, O[:, h], lse[:, h], f"{kind}, kv head {j}")
    # a head's result does not depend on the others: the same with two kv heads alone, by smaller workgroups
    two = [0, kv_heads - 1]
    hs = [j * G + i for j in two for i in range(G)]
    O2, lse2 = run_prompt(q[:, hs], k[:, two], v[:, two], cq, ck, causal)
    # each is off by u of the weights' sum of |v| and u of the output, twice that between them, and as much again for fp32
    u = torch.finfo(TYPES[dtype]).eps / 2
    assert bool(((O[:, hs].double() - O2.double()).abs() <= 4 * u * (O2.double().abs() + v.double().abs().max())).all())


@pytest.mark.parametrize("kind,d,dtype", [("unsplit", 128, "bf16"), ("split", 96, "fp16")])
def test_prompt_long_workgroups_with_infinities(kind, d, dtype):
    (n,), (m,), heads, kv_heads = LONG[kind]
    test_prompt_infinities_behind_the_mask(n, m, heads, kv_heads, d, dtype)


@pytest.mark.parametrize("n,m", [(200, 200), (6, 900)])
def test_prompt_keys_that_are_not_numbers_behind_the_mask(n, m):
    gen = torch.Generator().manual_seed(n)
    q, k, v = (rand(gen, "bf16", x, 2, 64) for x in (n, m, m))
    at = m - 3
    k[at] = float("nan")
    O, lse = run_prompt(q, k, v, [0, n], [0, m], True)
    keep = n - (m - at)   # rows that do not read it
    ref.prompt(q[:keep], k[:at], v[:at], [0, keep], [0, at], True, 1 / 8, O[:keep], lse[:keep], "rows before it")
    assert bool(torch.isnan(O[keep:].float()).all()) and bool(torch.isnan(lse[keep:]).all())


def test_prompt_offsets_that_make_no_sense():
    # tables that fall, run past the tensors or are negative: clamped, and nothing outside is written
    gen = torch.Generator().manual_seed(23)
    q, k, v = (rand(gen, "fp16", 100, 2, 64).to(DEV) for _ in range(3))
    whole = torch.full((140, 2, 64), 3.0, dtype=torch.float16, device=DEV)
    for cq, ck in (([0, 1000, 50, 70], [0, 100, 100, 2 ** 31 - 1]), ([-5, 30, 20, 2 ** 31 - 1], [90, 10, -7, 50]),
                   ([2 ** 31 - 1, -2 ** 31, 5, 5], [0, 0, 0, 0])):
        say(f"[gpu] offsets {cq} {ck}")
        g.attention_prompt(q, k, v, ints(cq), ints(ck), causal=True, O=whole[20:120])
        torch.cuda.synchronize()
        assert bool((whole[:20] == 3).all()) and bool((whole[120:] == 3).all())


def test_prompt_past_32_bits():
    # one sequence's keys span more than 4 GiB
    gen = torch.Generator().manual_seed(29)
    rows, stride, d = 700, 1 << 22, 64
    big = torch.empty(rows * stride, dtype=torch.float16, device=DEV)
    k, v = (big.as_strided((rows, 1, d), (stride, d, 1), o) for o in (0, 1 << 20))
    hk, hv, q = (rand(gen, "fp16", n, 1, d) for n in (rows, rows, 40))
    k.copy_(hk)
    v.copy_(hv)
    O, lse = g.attention_prompt(q.to(DEV), k, v, ints([0, 40]), ints([0, rows]), causal=True, return_lse=True)
    torch.cuda.synchronize()
    ref.prompt(q, hk, hv, [0, 40], [0, rows], True, 1 / 8, O.cpu(), lse.cpu(), "4 GiB cache")


# ---------------------------------------------------------------------- shared prefix
def shared_inputs(gen, dtype, B, P, N, H, Hk, d):
    return (rand(gen, dtype, B, H, d), rand(gen, dtype, P, Hk, d), rand(gen, dtype, P, Hk, d), rand(gen, dtype, B, N, Hk, d),
            rand(gen, dtype, B, N, Hk, d))


def check_shared(q, kp, vp, ks, vs, lens, scale=None, dev=None, **kw):
    say(f"[gpu] shared prefix q={tuple(q.shape)} kp={tuple(kp.shape)} ks={tuple(ks.shape)} {q.dtype} lens={lens[:9]}")
    x = dev or [t.to(DEV) for t in (q, kp, vp, ks, vs)]
    O, lse = g.attention_shared_prefix(*x, ints(lens), scale=scale, return_lse=True, **kw)
    torch.cuda.synchronize()
    s = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    ref.shared_prefix(q, kp, vp, ks, vs, lens, s, O.cpu(), lse.cpu(), f"shared prefix {q.dtype}")
    return O.cpu(), lse.cpu()


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("heads,kv_heads,d", [(8, 2, 128), (3, 3, 64), (7, 1, 96), (40, 1, 128), (2, 2, 24), (150, 1, 64)])
@pytest.mark.parametrize("B,P,N", [(1, 1, 1), (3, 64, 70), (5, 1000, 33), (2, 0, 40), (4, 130, 0), (2, 0, 0), (20, 65, 300), (1, 3001, 5)])
def test_shared_prefix(B, P, N, heads, kv_heads, d, dtype):
    gen = torch.Generator().manual_seed(B + P + N + d)
    lens = [(N - 3 * b) % (N + 1) for b in range(B)]
    check_shared(*shared_inputs(gen, dtype, B, P, N, heads, kv_heads, d), lens)


@pytest.mark.parametrize("B,heads,kv_heads,P,lens", [
    (130, 256, 256, 600, [0, 5, -1]),    # enough row tiles and kv heads that the prefix is one part
    (2, 512, 512, 550, [0, -1]),         # the same by the few-rows way
])
def test_shared_prefix_without_slot_rows(B, heads, kv_heads, P, lens):
    gen = torch.Generator().manual_seed(P)
    q, kp, vp = rand(gen, "fp16", B, heads, 8), rand(gen, "fp16", P, kv_heads, 8), rand(gen, "fp16", P, kv_heads, 8)
    none = torch.empty(B, 0, kv_heads, 8, dtype=torch.float16)
    lens = [lens[b % len(lens)] for b in range(B)]
    O = torch.full((B, heads, 8), 3.0, dtype=torch.float16, device=DEV)
    say(f"[gpu] shared prefix without slot rows B={B} heads={heads} P={P}")
    need = g.attention_shared_prefix_workspace(q.to(DEV), kp.to(DEV), vp.to(DEV), none.to(DEV), none.to(DEV), ints(lens))
    assert need >= B * heads * 10 * 4, "no room for the prefix's part"
    _, lse = g.attention_shared_prefix(q.to(DEV), kp.to(DEV), vp.to(DEV), none.to(DEV), none.to(DEV), ints(lens), O=O,
                                       return_lse=True)
    torch.cuda.synchronize()
    for b in range(B):
        if lens[b] < 0:
            assert bool((O[b] == 3).all())
    # a head's keys are one sequence's for all rows of the batch
    for h in range(0, heads, 17):
        used = [b for b in range(B) if lens[b] >= 0]
        o, l, parts, lb = ref.attend(q[used, h].double(), kp[:, h].double(), vp[:, h].double(), 8 ** -0.5, None)
        ref.check_rows(O[used, h].cpu(), lse[used, h].cpu(), o, l, parts, lb, torch.float16, f"head {h}")


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("B,heads,kv_heads,d,P,N", [(65, 24, 8, 128, 530, 70), (131, 10, 5, 80, 600, 256), (37, 32, 16, 64, 1000, 1),
                                                    (130, 66, 2, 96, 520, 33)])
def test_shared_prefix_many_short_slots(B, heads, kv_heads, d, P, N, dtype):
    # a wave to a slot and kv head; some slots empty, full, longer than there are rows, or not in use
    gen = torch.Generator().manual_seed(B)
    lens = [(0, N, 1, -1, N + 5, N // 2, N - 1)[b % 7] for b in range(B)]
    q, kp, vp, ks, vs = shared_inputs(gen, dtype, B, P, N, heads, kv_heads, d)
    for b, n in enumerate(lens):
        ks[b, max(n, 0):] = float("nan")
        vs[b, max(n, 0):] = float("inf")
    O, lse = (torch.full((B, heads) + s, 3.0, dtype=t, device=DEV) for s, t in (((d,), TYPES[dtype]), ((), torch.float32)))
    say(f"[gpu] many short slots B={B} heads={heads}/{kv_heads} d={d} P={P} N={N} {dtype}")
    g.attention_shared_prefix(*[t.to(DEV) for t in (q, kp, vp, ks, vs)], ints(lens), O=O, lse=lse)
    torch.cuda.synchronize()
    ref.shared_prefix(q, kp, vp, ks, vs, lens, d ** -0.5, O.cpu(), lse.cpu(), f"many short slots {dtype} d={d}")
    for b, n in enumerate(lens):
        assert n >= 0 or (bool((O[b] == 3).all()) and bool((lse[b] == 3).all()))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("B,heads,kv_heads,d,P,N", [(65, 32, 16, 128, 61, 40), (131, 16, 8, 80, 0, 200), (33, 32, 32, 64, 200, 30),
                                                    (65, 264, 8, 96, 33, 1), (128, 8, 8, 128, 256, 0)])
def test_shared_prefix_many_slots_behind_a_short_prefix(B, heads, kv_heads, d, P, N, dtype):
    test_shared_prefix_many_short_slots(B, heads, kv_heads, d, P, N, dtype)


def test_shared_prefix_slots():
    # unused slots keep their rows, lengths past the slot count as all of it, stale rows hold NaN
    gen = torch.Generator().manual_seed(31)
    B, P, N, H, Hk, d = 7, 200, 90, 4, 2, 128
    q, kp, vp, ks, vs = shared_inputs(gen, "bf16", B, P, N, H, Hk, d)
    lens = [5, -1, 0, 90, 1000, -2 ** 31, 64]
    for b, n in enumerate(lens):
        ks[b, max(0, n):] = float("nan")
        vs[b, max(0, n):] = float("inf")
    O = torch.full((B, H, d), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, H), 5.0, device=DEV)
    got, got_lse = check_shared(q, kp, vp, ks, vs, lens, O=O, lse=lse)
    for b in (1, 5):
        assert bool((got[b] == 5).all()) and bool((got_lse[b] == 5).all())


def test_shared_prefix_strides():
    gen = torch.Generator().manual_seed(37)
    B, P, N, H, Hk, d = 4, 129, 65, 8, 2, 64
    q, kp, vp, ks, vs = shared_inputs(gen, "fp16", B, P, N, H, Hk, d)
    lens = [65, 1, 0, 33]
    a = check_shared(q, kp, vp, ks, vs, lens)
    x = [t.to(DEV) for t in (q, kp, vp, ks, vs)]
    x[1:3] = [t.transpose(0, 1).contiguous().transpose(0, 1) for t in x[1:3]]
    x[3:5] = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in x[3:5]]
    b = check_shared(q, kp, vp, ks, vs, lens, dev=x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_shared_prefix_past_32_bits():
    gen = torch.Generator().manual_seed(41)
    rows, stride, d = 600, 1 << 22, 64
    big = torch.empty(rows * stride, dtype=torch.float16, device=DEV)
    kp, vp = (big.as_strided((rows, 1, d), (stride, d, 1), o) for o in (0, 1 << 20))
    q, hk, hv, ks, vs = shared_inputs(gen, "fp16", 3, rows, 4, 2, 1, d)
    kp.copy_(hk)
    vp.copy_(hv)
    check_shared(q, hk, hv, ks, vs, [4, 0, 2], dev=[q.to(DEV), kp, vp, ks.to(DEV), vs.to(DEV)])


# ---------------------------------------------------------------------- together, streams, graphs
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_prefill_then_single_tokens(dtype):
    """As they are used: a prompt read once, then every sequence's next tokens behind it.  Each single-token row is also
    the last row of the whole sequence's prompt."""
    gen = torch.Generator().manual_seed(43)
    P, B, N, H, Hk, d = 333, 5, 6, 8, 2, 128
    qkv = rand(gen, dtype, P, H + 2 * Hk, d)
    own = rand(gen, dtype, B, N, H + 2 * Hk, d)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    check_prompt(q, k, v, [0, P], [0, P], True)
    for n in range(1, N + 1):
        lens = [n] * B
        tok = own[:, n - 1, :H]
        O, lse = check_shared(tok.contiguous(), k.contiguous(), v.contiguous(), own[:, :, H:H + Hk], own[:, :, H + Hk:], lens)
        # the same rows through attention_prompt: one query against prefix and own keys
        K = torch.cat([torch.cat([k, own[b, :n, H:H + Hk]]) for b in range(B)])
        V = torch.cat([torch.cat([v, own[b, :n, H + Hk:]]) for b in range(B)])
        check_prompt(tok.contiguous(), K, V, cu([1] * B), cu([P + n] * B), True)


def _calls():
    gen = torch.Generator().manual_seed(47)
    c = cu([100, 40])
    a = [rand(gen, "fp16", c[-1], h, 128).to(DEV) for h in (4, 2, 2)]
    split = [rand(gen, "fp16", n, h, 128).to(DEV) for n, h in ((9, 4), (2000, 2), (2000, 2))]
    s = [t.to(DEV) for t in shared_inputs(gen, "bf16", 6, 500, 40, 8, 2, 64)]
    cua, cq, ck, lens = ints(c), ints([0, 9]), ints([0, 2000]), ints([40, 1, 0, 7, 40, 22])
    return [lambda O=None: g.attention_prompt(*a, cua, O=O), lambda O=None: g.attention_prompt(*split, cq, ck, O=O),
            lambda O=None: g.attention_shared_prefix(*s, lens, O=O)], [a, split, s]


def test_repeats_and_side_stream():
    calls, _ = _calls()
    for f in calls:
        want = f()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = [f() for _ in range(3)]
        side.synchronize()
        for x in got:
            assert torch.equal(x, want)


def test_captured_and_replayed():
    """All calls in one graph, replayed with new inputs and eager calls between the replays."""
    calls, inputs = _calls()
    outs = [torch.empty_like(f()) for f in calls]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for f, O in zip(calls, outs):
            f(O)
    for turn in range(4):
        say(f"[gpu] replay {turn}")
        for group in inputs:
            for i, x in enumerate(group):
                x.copy_(x.roll(1 + turn + i, 0))
        want = [f() for f in calls]
        torch.cuda.synchronize()
        for O in outs:
            O.fill_(float("nan"))
        graph.replay()
        extra = [f() for f in calls]   # eager calls behind the replay
        torch.cuda.synchronize()
        for a, b, e in zip(outs, want, extra):
            assert torch.equal(a, b) and torch.equal(e, b)


def test_captured_with_other_lengths():
    """The lengths are device tensors: a graph captured for a padded batch serves others, single tokens, empty sequences
    and slots not in use, and leaves the rows behind the last sequence alone."""
    gen = torch.Generator().manual_seed(61)
    q, k, v = (rand(gen, "bf16", n, h, 96) for n, h in ((300, 6), (2400, 2), (2400, 2)))
    s = shared_inputs(gen, "fp16", 5, 700, 90, 4, 2, 128)
    cq, ck, lens = ints([0, 300, 300, 300, 300]), ints([0, 2400, 2400, 2400, 2400]), ints([90] * 5)
    dq, dk, dv = q.to(DEV), k.to(DEV), v.to(DEV)
    ds = [t.to(DEV) for t in s]
    O, Os = torch.empty_like(dq), torch.empty_like(ds[0])
    lse, ls = torch.empty(300, 6, device=DEV), torch.empty(5, 4, device=DEV)

    def both():
        g.attention_prompt(dq, dk, dv, cq, ck, O=O, lse=lse)
        g.attention_shared_prefix(*ds, lens, O=Os, lse=ls)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for a, b, c in [([0, 1, 2, 3, 4], [0, 700, 700, 1500, 2399], [0, 1, 90, -1, 33]),
                    ([0, 0, 129, 129, 200], [0, 5, 600, 601, 700], [-1, -1, -1, -1, -1]),
                    ([0, 300, 300, 300, 300], [0, 2400, 2400, 2400, 2400], [90, 500, 3, 64, 32]),
                    ([0, 0, 0, 0, 0], [0, 0, 0, 0, 0], [0, 0, 0, 0, 0])]:
        say(f"[gpu] replay with cu_q={a} cu_k={b} lens={c}")
        for x, y in ((cq, a), (ck, b), (lens, c)):
            x.copy_(ints(y))
        for x in (O, Os, lse, ls):
            x.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        ref.prompt(q, k, v, a, b, True, 96 ** -0.5, O.cpu(), lse.cpu(), "replayed prompt")
        assert bool((O[a[-1]:] == 3).all()) and bool((lse[a[-1]:] == 3).all())
        ref.shared_prefix(*s, c, 128 ** -0.5, Os.cpu(), ls.cpu(), "replayed shared prefix")
        for i, n in enumerate(c):
            assert n >= 0 or (bool((Os[i] == 3).all()) and bool((ls[i] == 3).all()))


def test_calls_that_overlap_in_time():
    """Split calls on two streams at once, each with parts of its own."""
    calls, _ = _calls()
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for turn in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append([f() for f in (calls if i == 0 else calls[::-1])])
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for a, b in zip(outs if i == 0 else outs[::-1], want):
                assert torch.equal(a, b)


def test_given_workspace():
    gen = torch.Generator().manual_seed(53)
    q, k, v = (rand(gen, "fp16", n, h, 64).to(DEV) for n, h in ((3, 2), (3000, 1), (3000, 1)))
    cq, ck = ints([0, 3]), ints([0, 3000])
    need = g.attention_prompt_workspace(q, k, v, cq, ck)
    assert need > 0
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device=DEV)
    a = g.attention_prompt(q, k, v, cq, ck, workspace=ws[:need])
    b = g.attention_prompt(q, k, v, cq, ck)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and bool((ws[need:] == 0x7F).all())
    with pytest.raises(g.GemmError):
        g.attention_prompt(q, k, v, cq, ck, workspace=ws[:need - 16])


def test_python_refusals():
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device=DEV)
    k = torch.zeros(4, 1, 64, dtype=torch.float16, device=DEV)
    c = ints([0, 4])
    with pytest.raises(TypeError):
        g.attention_prompt(q.float(), k.float(), k.float(), c)
    with pytest.raises(TypeError):
        g.attention_prompt(q, k.bfloat16(), k, c)
    with pytest.raises(TypeError):
        g.attention_prompt(q, k, k, c.long())
    with pytest.raises(ValueError):
        g.attention_prompt(q, k, k[:3], c)
    with pytest.raises(ValueError):
        g.attention_prompt(q, k, k.cpu(), c)
    with pytest.raises(ValueError):
        g.attention_prompt(q, torch.zeros(4, 3, 64, dtype=torch.float16, device=DEV), k, c)
    with pytest.raises(ValueError):
        g.attention_prompt(q.transpose(0, 2), k, k, c)
    with pytest.raises(g.GemmError):
        g.attention_prompt(q, k, k, c, O=q)                       # O overlaps Q
    with pytest.raises(g.GemmError):
        g.attention_prompt(q, k, k, c, scale=float("inf"))
    with pytest.raises(g.GemmError):
        x = torch.zeros(4, 2, 72, dtype=torch.float16, device=DEV)[:, :, 4:68]   # rows off 16-byte boundaries
        g.attention_prompt(x, k, k, c)
    with pytest.raises(ValueError):
        g.attention_shared_prefix(q, k, k, torch.zeros(3, 2, 1, 64, dtype=torch.float16, device=DEV), k, ints([0] * 4))

"""The attention operators as workloads: what each is given, its plain form, and what one pass cannot do without.

Two operators, each in fp16 and bf16:

  prompt         attention of whole prompts, packed without padding: sequence b's queries are rows
                 cu_q[b] .. cu_q[b+1] of Q (tokens, heads, d), its keys rows cu_k[b] .. cu_k[b+1] of K and V
                 (tokens, kv heads, d); query head h reads kv head h / (heads / kv heads); causal masks are
                 aligned to each sequence's last key
  shared_prefix  one new token for each sequence of a batch: all of them attend to one common prefix
                 (Kp, Vp), and each to the first lens[b] rows of its own cache slot (Ks, Vs)

`own` chooses between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # a short chat turn of one user: what counts is the latency of the call
        {"name": "prompt_128", "op": "prompt", "dtype": "fp16", "heads": 32, "kv_heads": 8, "d": 128, "causal": True,
         "q_lens": "128", "k_lens": "128", "fused": True, "lse": False},
        # the attention-score product of this repository's suite (32 heads of 4096 x 4096, d 128) carried to its end
        {"name": "prompt_4096_h32", "op": "prompt", "dtype": "fp16", "heads": 32, "kv_heads": 32, "d": 128, "causal": True,
         "q_lens": "4096", "k_lens": "4096", "fused": False, "lse": False},
        # its d = 64 form without a mask: an encoder's layer
        {"name": "prompt_4096_h32_d64_full", "op": "prompt", "dtype": "bf16", "heads": 32, "kv_heads": 32, "d": 64, "causal": False,
         "q_lens": "4096", "k_lens": "4096", "fused": False, "lse": False},
        # a serving step's prompts of many lengths packed together, read from the fused projection's output
        {"name": "packed_ragged", "op": "prompt", "dtype": "bf16", "heads": 32, "kv_heads": 8, "d": 128, "causal": True,
         "q_lens": "1,2047,17,1000,64,65,2900,512,129,701", "k_lens": "1,2047,17,1000,64,65,2900,512,129,701", "fused": True, "lse": False},
        # one chunk of a long prompt against everything before it; the log-sum-exp lets a caller join it with other keys
        {"name": "chunk_512_of_20000", "op": "prompt", "dtype": "fp16", "heads": 32, "kv_heads": 8, "d": 128, "causal": True,
         "q_lens": "512", "k_lens": "20000", "fused": False, "lse": True},
        # an uncommon head size, odd lengths, seven query heads to a kv head
        {"name": "packed_d96_g7", "op": "prompt", "dtype": "fp16", "heads": 28, "kv_heads": 4, "d": 96, "causal": True,
         "q_lens": "1999,333,1001", "k_lens": "1999,1500,1001", "fused": False, "lse": False},
        # a long document read at once: the largest amount of work
        {"name": "prompt_16384", "op": "prompt", "dtype": "bf16", "heads": 32, "kv_heads": 8, "d": 128, "causal": True,
         "q_lens": "16384", "k_lens": "16384", "fused": True, "lse": False},
        # a few samples of one short instruction, just begun: latency
        {"name": "shared_3x500", "op": "shared_prefix", "dtype": "fp16", "heads": 32, "kv_heads": 8, "d": 128,
         "batch": 3, "prefix": 500, "slots": 64, "head_major": False, "lse": False},
        # a batch of users behind one long system prompt
        {"name": "shared_64x8192", "op": "shared_prefix", "dtype": "bf16", "heads": 32, "kv_heads": 8, "d": 128,
         "batch": 64, "prefix": 8192, "slots": 1000, "head_major": False, "lse": False},
        # as many kv heads as heads, odd sizes, the cache laid out head by head
        {"name": "shared_33x4095_mha_d64", "op": "shared_prefix", "dtype": "fp16", "heads": 32, "kv_heads": 32, "d": 64,
         "batch": 33, "prefix": 4095, "slots": 257, "head_major": True, "lse": True},
        # one sequence behind a very long document: few rows, a long axis
        {"name": "shared_1x100000", "op": "shared_prefix", "dtype": "bf16", "heads": 32, "kv_heads": 8, "d": 128,
         "batch": 1, "prefix": 100000, "slots": 128, "head_major": False, "lse": False},
        # a full batch, a long document and long answers: the largest
        {"name": "shared_256x32768", "op": "shared_prefix", "dtype": "bf16", "heads": 32, "kv_heads": 8, "d": 128,
         "batch": 256, "prefix": 32768, "slots": 2048, "head_major": True, "lse": False},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    dtype = rng.choice(["fp16", "bf16"])
    heads, kv_heads = rng.choice([(32, 8), (32, 32), (16, 2), (8, 1), (40, 8), (28, 4), (12, 12), (5, 5)])
    d = rng.choice([64, 128, 128, 128, 96, 80])
    if rng.random() < 0.5:
        causal = rng.random() < 0.75
        seqs = rng.choice([1, 1, 2, 3, 5, 8])
        q_lens, k_lens = [], []
        for _ in range(seqs):
            q = _spread(rng, 1, 8000 // seqs)
            k = q
            if rng.random() < 0.3:  # a chunk behind earlier keys
                k = q + _spread(rng, 1, 12000 // seqs)
            q_lens.append(q)
            k_lens.append(k)
        return {"op": "prompt", "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "d": d, "causal": causal,
                "q_lens": ",".join(map(str, q_lens)), "k_lens": ",".join(map(str, k_lens)),
                "fused": q_lens == k_lens and rng.random() < 0.5, "lse": rng.random() < 0.3}
    batch = _spread(rng, 1, 128)
    return {"op": "shared_prefix", "dtype": dtype, "heads": heads, "kv_heads": kv_heads, "d": d, "batch": batch,
            "prefix": _spread(rng, 1, 32000), "slots": _spread(rng, 1, 1500), "head_major": rng.random() < 0.5,
            "lse": rng.random() < 0.3}


def _lens(text):
    return [int(t) for t in text.split(",")]


def _suffix_lens(case):
    """The lengths of the sequences' own parts: spread over 1 .. slots in a fixed scattered order, the first one full."""
    n = case["slots"]
    return [n - (b * 2654435761 % (1 << 32)) * n // (1 << 32) for b in range(case["batch"])]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, h, hk, d = DTYPES[case["dtype"]], case["heads"], case["kv_heads"], case["d"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    s = {"case": case, "scale": 1.0 / math.sqrt(d)}
    if case["op"] == "prompt":
        ql, kl = _lens(case["q_lens"]), _lens(case["k_lens"])
        tq, tk = sum(ql), sum(kl)
        if case["fused"]:  # one projection's output holds Q, K and V of a token side by side
            qkv = normal(tq, h + 2 * hk, d)
            s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + hk], qkv[:, h + hk:]
        else:
            s["q"], s["k"], s["v"] = normal(tq, h, d), normal(tk, hk, d), normal(tk, hk, d)
        for name, lens in (("cu_q", ql), ("cu_k", kl)):
            s[name] = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).to(dev)
        s["max_q"], s["max_k"] = max(ql), max(kl)
        return s
    b, p, n = case["batch"], case["prefix"], case["slots"]
    s["q"] = normal(b, h, d)
    s["kp"], s["vp"] = normal(p, hk, d), normal(p, hk, d)
    if case["head_major"]:
        s["ks"], s["vs"] = normal(b, hk, n, d).transpose(1, 2), normal(b, hk, n, d).transpose(1, 2)
    else:
        s["ks"], s["vs"] = normal(b, n, hk, d), normal(b, n, hk, d)
    s["lens"] = torch.tensor(_suffix_lens(case), dtype=torch.int32, device=dev)
    return s


def _softmax_parts(scores, keep):
    """exp(scores - row maximum) where `keep`, its row sums and the row maxima; rows without a key give zeros."""
    if keep is not None:
        scores = scores.masked_fill_(~keep, float("-inf"))
    m = scores.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = scores.sub_(m).exp_()
    return p, p.sum(-1, keepdim=True), m


def _plain_prompt(s):
    c = s["case"]
    hk, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"]
    dev = s["q"].device
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    b, mq, mk = cu_q.numel() - 1, s["max_q"], s["max_k"]
    iq, ik = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    nq, nk = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    rows_q = (cu_q[:-1, None] + iq).clamp_(max=s["q"].shape[0] - 1)
    rows_k = (cu_k[:-1, None] + ik).clamp_(max=s["k"].shape[0] - 1)
    # (sequence, kv head, query head of it and token, d), padded to the longest sequence
    q = s["q"].float()[rows_q].reshape(b, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(b, hk, g * mq, d)
    k = s["k"].float()[rows_k].permute(0, 2, 3, 1).contiguous()
    v = s["v"].float()[rows_k].permute(0, 2, 1, 3).contiguous()
    scores = torch.matmul(q, k).mul_(s["scale"]).reshape(b, hk, g, mq, mk)
    keep = (ik < nk[:, None])[:, None, :].expand(b, mq, mk)
    if c["causal"]:
        keep = keep & (ik <= iq[:, None] + (nk - nq)[:, None, None])
    p, l, m = _softmax_parts(scores, keep[:, None, None])
    o = torch.matmul(p.reshape(b, hk, g * mq, mk), v).reshape(b, hk, g, mq, d) / torch.where(l > 0, l, torch.ones_like(l))
    real = iq < nq[:, None]
    out = o.permute(0, 3, 1, 2, 4)[real].reshape(-1, c["heads"], d).to(s["q"].dtype)
    if not c["lse"]:
        return out
    return out, (m + l.log()).squeeze(-1).permute(0, 3, 1, 2)[real].reshape(-1, c["heads"])


def _plain_shared_prefix(s):
    c = s["case"]
    hk, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["d"]
    b, n = s["ks"].shape[:2]
    q = s["q"].float().reshape(b, hk, g, d)
    kp, vp = s["kp"].float().permute(1, 2, 0).contiguous(), s["vp"].float().permute(1, 0, 2).contiguous()
    ks, vs = s["ks"].float().permute(0, 2, 3, 1).contiguous(), s["vs"].float().permute(0, 2, 1, 3).contiguous()
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hk, b * g, d), kp).reshape(hk, b, g, -1).permute(1, 0, 2, 3)
    ss = torch.matmul(q, ks)
    own_keys = torch.arange(n, device=q.device) < s["lens"][:, None]
    keep = torch.cat([own_keys.new_ones(b, sp.shape[-1]), own_keys], 1)
    p, l, m = _softmax_parts(torch.cat([sp, ss], -1).mul_(s["scale"]), keep[:, None, None])
    pp, ps = p[..., :sp.shape[-1]], p[..., sp.shape[-1]:]
    o = torch.matmul(pp.permute(1, 0, 2, 3).reshape(hk, b * g, -1), vp).reshape(hk, b, g, d).permute(1, 0, 2, 3)
    o = (o + torch.matmul(ps, vs)) / torch.where(l > 0, l, torch.ones_like(l))
    out = o.reshape(b, c["heads"], d).to(s["q"].dtype)
    return (out, (m + l.log()).reshape(b, c["heads"])) if c["lse"] else out


def run(state):
    s, c = state, state["case"]
    if c["op"] == "prompt":
        if own:
            import dense_fp16_gemm_nt_amd as fw
            return fw.attention_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=c["causal"], scale=s["scale"],
                                       return_lse=c["lse"])
        return _plain_prompt(s)
    if own:
        import dense_fp16_gemm_nt_amd as fw
        return fw.attention_shared_prefix(s["q"], s["kp"], s["vp"], s["ks"], s["vs"], s["lens"], scale=s["scale"],
                                          return_lse=c["lse"])
    return _plain_shared_prefix(s)


def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["d"]
    if case["op"] == "prompt":
        ql, kl = _lens(case["q_lens"]), _lens(case["k_lens"])
        # pairs of a query and a key that it may read: a causal query i of n reads the keys up to k - n + i
        pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in zip(ql, kl))
        rows, keys = sum(ql), sum(kl)
    else:
        lens = _suffix_lens(case)
        rows, keys = case["batch"], case["prefix"] + sum(lens)
        pairs = rows * case["prefix"] + sum(lens)
    # Q, K and V read once, the output written once; a product with K and one with V for each pair and head
    return {"bytes": 2 * d * (2 * rows * h + 2 * keys * hk) + (4 * rows * h if case["lse"] else 0), "flops": 4 * d * h * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    h, hk, d = case["heads"], case["kv_heads"], case["d"]
    g = h // hk
    rows = s["q"].shape[0]
    out = torch.zeros((rows, h, d), dtype=torch.float64, device=s["q"].device)
    lse = torch.full((rows, h), float("-inf"), dtype=torch.float64, device=s["q"].device)

    def attend(q, k, v, keep):
        """softmax(q k^T / sqrt(d)) v in 64 bits for 2-D q, k and v; `keep` says which pairs count."""
        a = torch.mm(q, k.t()) / math.sqrt(d)
        if keep is not None:
            a = torch.where(keep, a, torch.full_like(a, float("-inf")))
        z = torch.logsumexp(a, 1)
        return torch.mm(torch.exp(a - z[:, None]), v), z

    if case["op"] == "prompt":
        at_q = at_k = 0
        for n, k_len in zip(_lens(case["q_lens"]), _lens(case["k_lens"])):
            keep = None
            if case["causal"]:
                last = torch.arange(n, device=out.device) + (k_len - n)
                keep = torch.arange(k_len, device=out.device)[None, :] <= last[:, None]
            for j in range(h):
                q = s["q"][at_q:at_q + n, j].double()
                k = s["k"][at_k:at_k + k_len, j // g].double()
                v = s["v"][at_k:at_k + k_len, j // g].double()
                out[at_q:at_q + n, j], lse[at_q:at_q + n, j] = attend(q, k, v, keep)
            at_q, at_k = at_q + n, at_k + k_len
    else:
        lens = torch.tensor(_suffix_lens(case), device=out.device)
        p, n = case["prefix"], case["slots"]
        mine = torch.arange(n, device=out.device)[None, None, :] < lens[:, None, None]
        for j in range(hk):
            q = s["q"][:, j * g:(j + 1) * g].double()
            # scores against the prefix for all rows at once, and against each sequence's own rows
            a = torch.mm(q.reshape(-1, d), s["kp"][:, j].double().t()).reshape(rows, g, p) / math.sqrt(d)
            own_k, own_v = s["ks"][:, :, j].double(), s["vs"][:, :, j].double()
            c = (q[:, :, None, :] * own_k[:, None, :, :]).sum(-1) / math.sqrt(d)
            c = torch.where(mine, c, torch.full_like(c, float("-inf")))
            z = torch.logsumexp(torch.cat([a, c], 2), 2)
            o = torch.mm(torch.exp(a - z[..., None]).reshape(-1, p), s["vp"][:, j].double()).reshape(rows, g, d)
            o = o + (torch.exp(c - z[..., None])[..., None] * own_v[:, None, :, :]).sum(2)
            out[:, j * g:(j + 1) * g], lse[:, j * g:(j + 1) * g] = o, z
    return (out, lse) if case["lse"] else out

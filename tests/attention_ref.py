"""Plain 64-bit attention and its error bounds (test infrastructure).

Bounds, with u = eps / 2 of the tensors' type (half a step of a rounding) and
w_j a row's softmax weights:

* each weight is rounded to the type once: at most u * sum_j w_j |v_j|; below
  fp16's normal numbers the step is absolute, 2^-25 beside a largest weight
  of at least 2^7: 2^-32 * sum_j |v_j|;
* the output is rounded once: u * |o|, or half the smallest step, 2^-25;
* fp32: a score is a sum of d products, off by at most (d + 8) * 2^-22 *
  scale * sum |q k| (2^-22: two fp32 steps for an addition inside a matrix
  instruction); an error e of the scores moves every weight by a factor
  e^(+-2e); the exponential and its argument add 2^-20 * (1 + |score|); the sum
  over n keys, of weights and of products, adds 2 * n * 2^-22 at most, and
  joining parts a few more steps, which the 8s cover.
"""
import torch


def attend(q, k, v, scale, allowed):
    """One head: q (n, d), k, v (m, d) in 64 bits, allowed (n, m) or None.
    Returns (o, lse, bound of o without the final rounding, bound of lse)."""
    n, m = q.shape[0], k.shape[0]
    d = q.shape[1]
    if allowed is None:
        allowed = torch.ones(n, m, dtype=torch.bool)
    inf = float("inf")
    s = (q @ k.t()) * scale
    s = torch.where(allowed, s, torch.full_like(s, -inf))
    lse = torch.logsumexp(s, 1) if m else torch.full((n,), -inf, dtype=torch.float64)
    w = torch.where(allowed, torch.exp(s - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]), torch.zeros_like(s))
    o = w @ v
    qk = (q.abs() @ k.abs().t()) * abs(scale)
    qk = torch.where(allowed, qk, torch.zeros_like(qk))
    top = qk.amax(1) if m else torch.zeros(n, dtype=torch.float64)
    e_score = (d + 8) * 2.0 ** -22 * top
    e_weight = 2 * e_score + 2.0 ** -20 * (1 + 2 * top) + 2 * (m + 8) * 2.0 ** -22
    mass = w @ v.abs()
    tiny = allowed.double() @ v.abs() * 2.0 ** -32
    return o, lse, (mass, e_weight[:, None] * mass + tiny), e_score + 2.0 ** -20 * (1 + top) + (m + 8) * 2.0 ** -22


def check_rows(got, lse_got, o, lse, parts, lse_bound, dtype, what):
    u = torch.finfo(dtype).eps / 2
    mass, rest = parts
    bound = (u * mass + rest) * (1 + u) + u * o.abs() + 2.0 ** -25
    off = (got.double() - o).abs()
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound at {divmod(int((off / bound).argmax()), o.shape[-1])}"
    if lse_got is not None:
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(lse_got) & (lse_got < 0), empty), f"{what}: rows without a key"
        off = (lse_got.double() - lse).abs()[~empty]
        assert bool((off <= lse_bound[~empty]).all()), f"{what}: lse off by {float(off.max())}"
    return worst


def prompt(q, k, v, cu_q, cu_k, causal, scale, got, lse_got, what):
    """Checks attention_prompt's outputs, all on the host; returns the largest share of a bound."""
    H, Hk, d = q.shape[1], k.shape[1], q.shape[2]
    G = H // Hk
    worst = 0.0
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        n, m = q1 - q0, k1 - k0
        if n == 0:
            continue
        allowed = None
        if causal:
            allowed = (torch.arange(m)[None, :] <= torch.arange(n)[:, None] + (m - n)).repeat_interleave(G, 0)
        for j in range(Hk):
            h = slice(j * G, (j + 1) * G)
            o, lse, parts, lb = attend(q[q0:q1, h].double().reshape(n * G, d), k[k0:k1, j].double(), v[k0:k1, j].double(),
                                       scale, allowed)
            worst = max(worst, check_rows(got[q0:q1, h].reshape(n * G, d),
                                          None if lse_got is None else lse_got[q0:q1, h].reshape(n * G), o, lse, parts, lb,
                                          q.dtype, f"{what}, sequence {b} of {n} queries and {m} keys, kv head {j}"))
    return worst


def shared_prefix(q, kp, vp, ks, vs, lens, scale, got, lse_got, what):
    H, Hk = q.shape[1], kp.shape[1]
    G = H // Hk
    worst = 0.0
    for b, n in enumerate(lens):
        if n < 0:
            continue
        n = min(n, ks.shape[1])
        for j in range(Hk):
            h = slice(j * G, (j + 1) * G)
            k = torch.cat([kp[:, j], ks[b, :n, j]]).double()
            v = torch.cat([vp[:, j], vs[b, :n, j]]).double()
            o, lse, parts, lb = attend(q[b, h].double(), k, v, scale, None)
            worst = max(worst, check_rows(got[b, h], None if lse_got is None else lse_got[b, h], o, lse, parts, lb,
                                          q.dtype, f"{what}, slot {b} with {n} own keys, kv head {j}"))
    return worst

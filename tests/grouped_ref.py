"""Plain 64-bit grouped products and products with adapters, and their error bounds (test infrastructure).

Bounds, with u = eps / 2 of an output's type (half a step of a rounding):

* an output is rounded once: u * |d|, or half the smallest step of fp16, 2^-25;
* fp32: a sum of n products is off by at most n * 2^-22 * sum |x y| (2^-22: two
  fp32 steps for an addition inside a matrix instruction), and the sums of four
  waves are added in three more steps, which the 8 covers;
* an adapter's low-rank values h are scaled (one fp32 step) and rounded to the
  operands' type: u * |h| each, or 2^-25 in fp16, on top of their own sum's
  bound; an error of h reaches the output as sum |up| * error.

Inputs of small whole numbers have sums that fp32 holds, so results are equal
to the rounded exact ones, bit by bit.
"""
import torch

STEP = 2.0 ** -22


def clamp_rows(cu, rows):
    """The rows of each group, as the kernels clamp offsets."""
    out = []
    for a, b in zip(cu[:-1], cu[1:]):
        a = min(max(a, 0), rows)
        out.append((a, min(max(b, a), rows)))
    return out


def _sum(x, y, n):
    """x @ y in 64 bits, and the bound of its fp32 sums."""
    return torch.mm(x, y), (n + 8) * STEP * torch.mm(x.abs(), y.abs())


def product(A, B, cu, kept):
    d, e = kept.double(), torch.zeros_like(kept, dtype=torch.float64)
    for g, (a, b) in enumerate(clamp_rows(cu, A.shape[0])):
        if b > a:
            d[a:b], e[a:b] = _sum(A[a:b].double(), B[g].double().t(), A.shape[1])
    return d, e


def grad_input(G, B, cu, kept):
    d, e = kept.double(), torch.zeros_like(kept, dtype=torch.float64)
    for g, (a, b) in enumerate(clamp_rows(cu, G.shape[0])):
        if b > a:
            d[a:b], e[a:b] = _sum(G[a:b].double(), B[g].double(), G.shape[1])
    return d, e


def grad_weight(G, A, cu):
    n = len(cu) - 1
    d = torch.zeros(n, G.shape[1], A.shape[1], dtype=torch.float64, device=G.device)
    e = torch.zeros_like(d)
    for g, (a, b) in enumerate(clamp_rows(cu, G.shape[0])):
        if b > a:
            d[g], e[g] = _sum(G[a:b].double().t(), A[a:b].double(), b - a)
    return d, e


def adapters(A, B, down, up, cu, ids, scales, kept):
    u = torch.finfo(A.dtype).eps / 2
    d, e = kept.double(), torch.zeros_like(kept, dtype=torch.float64)
    for q, (a, b) in enumerate(clamp_rows(cu, A.shape[0])):
        if b <= a:
            continue
        x = A[a:b].double()
        d[a:b], e[a:b] = _sum(x, B.double().t(), A.shape[1])
        i = ids[q]
        if not 0 <= i < down.shape[0] or down.shape[1] == 0:
            continue
        s = 1.0 if scales is None else float(scales[i])
        h, eh = _sum(x, down[i].double().t(), A.shape[1])
        h, eh = h * s, eh * abs(s) + h.abs() * abs(s) * STEP
        eh = eh + u * (h.abs() + eh) + (2.0 ** -25 if A.dtype == torch.float16 else 0.0)
        w = up[i].double().t()
        d[a:b] += torch.mm(h, w)
        e[a:b] += torch.mm(eh, w.abs()) + (down.shape[1] + 8) * STEP * torch.mm(h.abs() + eh, w.abs())
    return d, e


def check(got, d, e, what):
    """Largest share of the bound; raises above 1."""
    u = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 2.0 ** -24
    bound = e * (1 + u) + u * d.abs() + 2.0 ** -25
    assert bool(torch.isfinite(got).all()), f"{what}: not finite"
    off = (got.double() - d).abs()
    worst = float((off / bound).max()) if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound at {int((off / bound).argmax())} of {tuple(got.shape)}"
    return worst

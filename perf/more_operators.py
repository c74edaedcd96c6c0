"""Products of many matrices in one call as workloads: what each is given, its plain form, and what one pass cannot do without.

Four operators, each in fp16 and bf16:

  product      D[r] = B_e A[r] for the rows r = cu[e] .. cu[e + 1] - 1 of group e: the rows of A (rows, K) are sorted by
               the matrix of B (groups, N, K) that they go through, as a router of experts leaves them
  grad_input   its gradient for A: dA[r] = B_e^T G[r], G (rows, N) being the gradient for D
  grad_weight  its gradient for B: dB_e = sum over the group's rows of G[r] A[r]^T; 0 for a group without rows
  adapters     D[r] = W X[r] + scale_a up_a (down_a X[r]): one projection W (N, K) shared by all rows, and beside it the
               low-rank adapter a of the request that the row belongs to; requests are runs of rows, cu[b] .. cu[b + 1] - 1

`own` chooses between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math
import random

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # four tokens of one user, two experts each, at the smallest layer: what counts is the latency of the call
        {"name": "product_8_rows", "op": "product", "dtype": "bf16", "groups": 16, "rows": 8, "n": 1024, "k": 2048},
        # a decoding step of 64 users, eight of 64 experts each: the weights are read once, each for a few rows
        {"name": "product_512_of_64", "op": "product", "dtype": "fp16", "groups": 64, "rows": 512, "n": 2048, "k": 4096},
        # odd sizes, uneven groups, some of them without a row
        {"name": "product_odd", "op": "product", "dtype": "fp16", "groups": 13, "rows": 5003, "n": 1416, "k": 1000},
        # a training step's tokens over eight large experts: the largest amount of work
        {"name": "product_16384_of_8", "op": "product", "dtype": "bf16", "groups": 8, "rows": 16384, "n": 14336, "k": 4096},
        # the gradients of such a layer with half as many tokens
        {"name": "grad_input_8192_of_8", "op": "grad_input", "dtype": "bf16", "groups": 8, "rows": 8192, "n": 14336, "k": 4096},
        {"name": "grad_weight_8192_of_8", "op": "grad_weight", "dtype": "bf16", "groups": 8, "rows": 8192, "n": 4096, "k": 14336,
         "out": "bf16"},
        # fine-grained experts with few rows each, odd sizes; weights' gradients kept in 32 bits for accumulation
        {"name": "grad_input_odd", "op": "grad_input", "dtype": "fp16", "groups": 40, "rows": 2999, "n": 1000, "k": 2056},
        {"name": "grad_weight_1500_of_64", "op": "grad_weight", "dtype": "fp16", "groups": 64, "rows": 1500, "n": 2048, "k": 1024,
         "out": "fp32"},
        # one user's next token through one adapter: latency
        {"name": "adapters_1", "op": "adapters", "dtype": "fp16", "n": 4096, "k": 4096, "rank": 16, "adapters": 4, "lens": "1"},
        # a decoding step of 64 users, most with an adapter of their own
        {"name": "adapters_64_tokens", "op": "adapters", "dtype": "bf16", "n": 14336, "k": 4096, "rank": 16, "adapters": 48,
         "lens": ",".join(["1"] * 64)},
        # prompts and single tokens side by side, odd sizes
        {"name": "adapters_mixed_odd", "op": "adapters", "dtype": "fp16", "n": 2056, "k": 1000, "rank": 24, "adapters": 7,
         "lens": "1,1,333,1,64,1,900,17,1,1,128,1,1,250,33"},
        # a serving step full of prompts, adapters of high rank
        {"name": "adapters_prompts", "op": "adapters", "dtype": "bf16", "n": 4096, "k": 4096, "rank": 64, "adapters": 6,
         "lens": "512,1000,77,2048,300,129,1500,640"},
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    dtype = rng.choice(["fp16", "bf16"])
    op = rng.choice(["product", "product", "grad_input", "grad_weight", "adapters", "adapters"])
    while True:
        n, k = 8 * _spread(rng, 16, 1792), 8 * _spread(rng, 16, 1792)   # 128 .. 14336
        if rng.random() < 0.5:   # most layers are multiples of 256
            n, k = max(256, n // 256 * 256), max(256, k // 256 * 256)
        if op == "adapters":
            requests = _spread(rng, 1, 100)
            if rng.random() < 0.4:
                lens = [1] * requests
            else:
                lens = [_spread(rng, 1, max(1, 8000 // requests)) for _ in range(requests)]
            if sum(lens) * n * k > 8000 * 8192 * 8192:
                continue
            return {"op": op, "dtype": dtype, "n": n, "k": k, "rank": rng.choice([8, 16, 16, 32, 64, 128, 24]),
                    "adapters": _spread(rng, 1, 60), "lens": ",".join(map(str, lens))}
        groups, rows = rng.choice([1, 2, 5, 8, 8, 16, 27, 64, 128]), _spread(rng, 1, 16384)
        if groups * n * k > 8 * 14336 * 4096 or rows * n * k > 16384 * 14336 * 4096:
            continue
        case = {"op": op, "dtype": dtype, "groups": groups, "rows": rows, "n": n, "k": k}
        if op == "grad_weight":
            case["out"] = rng.choice([dtype, "fp32"])
        return case


def _group_lens(case):
    """Rows of each group: every row goes through a matrix of its own choice, some matrices being chosen more often."""
    rng = random.Random(1000003 * case["groups"] + case["rows"])
    likely = [rng.uniform(0.2, 1.8) if rng.random() < 0.9 else 0.0 for _ in range(case["groups"])]
    if not any(likely):
        likely[0] = 1.0
    lens = [0] * case["groups"]
    for e in rng.choices(range(case["groups"]), weights=likely, k=case["rows"]):
        lens[e] += 1
    return lens


def _requests(case):
    """(rows, adapter) of each request; every seventh request has no adapter (-1)."""
    lens = [int(t) for t in case["lens"].split(",")]
    return [(n, -1 if b % 7 == 6 else (b * 2654435761 >> 7) % case["adapters"]) for b, n in enumerate(lens)]


def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, n, k = DTYPES[case["dtype"]], case["n"], case["k"]

    def normal(*shape, std=1.0):
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.float32)
        return (x.mul_(std) if std != 1.0 else x).to(dt)

    def matrices(count):   # of K inputs each, which keep the size of what they are given
        out = torch.empty((count, n, k), dtype=dt, device=dev)
        for e in range(count):
            out[e] = normal(n, k, std=1.0 / math.sqrt(k))
        return out

    def ints(values):
        return torch.tensor(values, dtype=torch.int32).to(dev)

    s = {"case": case}
    if case["op"] == "adapters":
        requests = _requests(case)
        r, count = case["rank"], case["adapters"]
        s["cu"] = ints(_starts([m for m, _ in requests]))
        s["adapter"] = ints([a for _, a in requests])
        s["requests"] = requests   # the same on the host, as a scheduler has them
        s["x"] = normal(sum(m for m, _ in requests), k)
        s["w"] = matrices(1)[0]
        s["down"] = normal(count, r, k, std=1.0 / math.sqrt(k))
        s["up"] = normal(count, n, r, std=0.5 / math.sqrt(r))
        s["scales"] = torch.rand(count, generator=gen, device=dev, dtype=torch.float32) + 0.5
        return s
    s["lens"] = _group_lens(case)   # as a router's counts
    s["cu"] = ints(_starts(s["lens"]))
    if case["op"] != "grad_input":
        s["a"] = normal(case["rows"], k)
    if case["op"] != "product":
        s["g"] = normal(case["rows"], n)
    if case["op"] != "grad_weight":
        s["b"] = matrices(case["groups"])
    return s


def _plain_groups(s):
    c, at = s["case"], _starts(s["lens"])
    dt, dev = DTYPES[c["dtype"]], s["cu"].device
    if c["op"] == "grad_weight":
        out = torch.zeros((c["groups"], c["n"], c["k"]), dtype=DTYPES[c["out"]], device=dev)
    else:
        out = torch.empty((c["rows"], c["n"] if c["op"] == "product" else c["k"]), dtype=dt, device=dev)
    for e, m in enumerate(s["lens"]):
        if m == 0:
            continue
        rows = slice(at[e], at[e + 1])
        if c["op"] == "product":
            out[rows] = torch.matmul(s["a"][rows].float(), s["b"][e].float().t())
        elif c["op"] == "grad_input":
            out[rows] = torch.matmul(s["g"][rows].float(), s["b"][e].float())
        else:
            out[e] = torch.matmul(s["g"][rows].float().t(), s["a"][rows].float())
    return out


def _plain_adapters(s):
    x = s["x"].float()
    y = torch.matmul(x, s["w"].float().t())
    if all(m == 1 for m, _ in s["requests"]):   # single tokens: all requests at once
        a = s["adapter"].long()
        on = a.clamp(min=0)
        h = (s["down"][on].float() * x[:, None, :]).sum(-1) * torch.where(a < 0, 0.0, s["scales"][on])[:, None]
        y += (s["up"][on].float() * h[:, None, :]).sum(-1)
    else:
        at = 0
        for m, a in s["requests"]:
            if a >= 0 and m > 0:
                h = torch.matmul(x[at:at + m], s["down"][a].float().t()) * s["scales"][a]
                y[at:at + m] += torch.matmul(h, s["up"][a].float().t())
            at += m
    return y.to(s["x"].dtype)


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _plain_adapters(s) if op == "adapters" else _plain_groups(s)
    import dense_fp16_gemm_nt_amd as fw
    if op == "product":
        return fw.grouped_product(s["a"], s["b"], s["cu"])
    if op == "grad_input":
        return fw.grouped_product_grad_input(s["g"], s["b"], s["cu"])
    if op == "grad_weight":
        return fw.grouped_product_grad_weight(s["g"], s["a"], s["cu"], dtype=DTYPES[s["case"]["out"]])
    return fw.adapter_product(s["x"], s["w"], s["down"], s["up"], s["cu"], s["adapter"], s["scales"])


def work(case):
    n, k = case["n"], case["k"]
    if case["op"] == "adapters":
        requests = _requests(case)
        rows, used = sum(m for m, _ in requests), {a for m, a in requests if a >= 0 and m > 0}
        adapted = sum(m for m, a in requests if a >= 0)
        return {"bytes": 2 * (rows * (k + n) + n * k + len(used) * case["rank"] * (n + k)) + 4 * (2 * len(requests) + 1 + len(used)),
                "flops": 2 * rows * n * k + 2 * adapted * case["rank"] * (n + k)}
    lens = _group_lens(case)
    rows, used = sum(lens), sum(m > 0 for m in lens)
    if case["op"] == "grad_weight":   # every matrix is written, zeros where no row chose it
        matrices = case["groups"] * n * k * (4 if case["out"] == "fp32" else 2)
    else:
        matrices = used * n * k * 2
    return {"bytes": 2 * rows * (n + k) + matrices + 4 * (case["groups"] + 1), "flops": 2 * rows * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    cu = s["cu"].tolist()
    if case["op"] == "adapters":
        out = torch.mm(s["x"].double(), s["w"].double().t())
        for b, a in enumerate(s["adapter"].tolist()):
            x = s["x"][cu[b]:cu[b + 1]].double()
            if a >= 0 and len(x):
                low = torch.mm(x, s["down"][a].double().t())
                out[cu[b]:cu[b + 1]] += torch.mm(low, s["up"][a].double().t()) * s["scales"][a].double()
        return out
    dev = s["cu"].device
    shape = {"product": (case["rows"], case["n"]), "grad_input": (case["rows"], case["k"]),
             "grad_weight": (case["groups"], case["n"], case["k"])}[case["op"]]
    out = torch.zeros(shape, dtype=torch.float64, device=dev)
    for e in range(case["groups"]):
        lo, hi = cu[e], cu[e + 1]
        if lo == hi:
            continue
        if case["op"] == "product":
            torch.mm(s["a"][lo:hi].double(), s["b"][e].double().t(), out=out[lo:hi])
        elif case["op"] == "grad_input":
            torch.mm(s["g"][lo:hi].double(), s["b"][e].double(), out=out[lo:hi])
        else:
            torch.mm(s["g"][lo:hi].double().t(), s["a"][lo:hi].double(), out=out[e])
    return out

"""Measured cases of the expert operators: products over row groups, their weight gradients, and the 8-bit product.

Rows of a token matrix are sorted by expert; ``offsets`` (int32, on the device) marks where each expert's rows begin, and an expert
may have none.  ``run`` computes an operator in plain torch, or through the library where ``own`` is set.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # generation, one token routed to 8 of the 64 experts of 1024 x 4096: latency, and 8 weight matrices read
        dict(name="product_one_token", op="product", n=64, active=8, rows=8, k=1024, m=4096, trans=False, dtype="bf16", out="bf16"),
        # generation, a batch of sequences: a few rows for most experts, the whole weight set read once
        dict(name="product_batch", op="product", n=64, active=56, rows=256, k=4096, m=1024, trans=True, dtype="bf16", out="bf16"),
        # a training step's forward product, ragged groups
        dict(name="product_forward", op="product", n=64, active=61, rows=16381, k=1024, m=4096, trans=False, dtype="bf16", out="bf16"),
        # the gradient of the same product's input, fp16
        dict(name="product_input_grad", op="product", n=64, active=64, rows=32768, k=4096, m=1024, trans=True, dtype="fp16", out="fp16"),
        # odd sizes, experts in allocations of their own, fp32 result
        dict(name="product_odd", op="product", n=7, active=6, rows=1531, k=1100, m=2050, trans=False, dtype="bf16", out="fp32", separate=True),
        # one group: the up projection of the 4096 / 11008 block over a long sequence
        dict(name="product_dense", op="product", n=1, active=1, rows=8192, k=4096, m=11008, trans=False, dtype="bf16", out="bf16"),
        # the experts' weight gradients in bf16
        dict(name="gradient_train", op="gradient", n=64, active=64, rows=32768, k=1024, m=4096, dtype="bf16", out="bf16", add=False),
        # the same added to an fp32 gradient of earlier micro-batches; one expert got no rows
        dict(name="gradient_accumulate", op="gradient", n=64, active=63, rows=16381, k=1024, m=4096, dtype="bf16", out="fp32", add=True),
        # small odd matrices
        dict(name="gradient_odd", op="gradient", n=7, active=6, rows=999, k=520, m=771, dtype="fp16", out="fp16", add=True),
        # generation in 8 bits: a few rows for half the experts
        dict(name="int8_batch", op="int8", n=64, active=32, rows=64, k=1024, m=4096, dtype="bf16", out="bf16"),
        # a prompt in 8 bits, ragged groups
        dict(name="int8_prompt", op="int8", n=64, active=62, rows=16381, k=4096, m=1024, dtype="bf16", out="bf16"),
        # one group: the down projection of the 4096 / 11008 block
        dict(name="int8_dense", op="int8", n=1, active=1, rows=8192, k=11008, m=4096, dtype="bf16", out="bf16"),
    ]


MOST_FLOPS = 7.3e11
MOST_WEIGHTS = 64 * 1024 * 4096


def draw(rng):
    spread = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    while True:
        op = rng.choice(["product", "product", "gradient", "int8"])
        n = rng.choice([1, spread(2, 96), spread(2, 96)])
        k, m, rows = spread(64, 11008), spread(64, 11008), spread(1, 32768)
        if rng.random() < 0.6:  # most matrices have sides that are multiples of 64
            k, m = 64 * max(1, k // 64), 64 * max(1, m // 64)
        flops, weights = 2.0 * rows * k * m, n * k * m
        moved = weights * (6 if op == "gradient" else 2) + rows * (k + m) * 2
        if flops > MOST_FLOPS or weights > MOST_WEIGHTS or flops + 100.0 * moved < 1e8:
            continue
        active = max(1, min(n, rows, n - rng.randint(0, n // 4)))
        case = dict(op=op, n=n, active=active, rows=rows, k=k, m=m, dtype=rng.choice(["bf16", "bf16", "fp16"]))
        case["out"] = rng.choice([case["dtype"], case["dtype"], "fp32"])
        if op == "product":
            case["trans"] = rng.random() < 0.5
            case["separate"] = n <= 32 and rng.random() < 0.3
        if op == "gradient":
            case["add"] = rng.random() < 0.5
        return case


def _counts(case, seed):
    """Rows of each expert: `active` experts of unequal popularity, one row at least for each of them."""
    rng = np.random.default_rng(seed)
    n, active, rows = case["n"], case["active"], case["rows"]
    p = np.exp(0.5 * rng.standard_normal(active))
    got = np.zeros(n, dtype=np.int64)
    got[rng.permutation(n)[:active]] = 1 + rng.multinomial(rows - active, p / p.sum())
    return got


def _matrix(gen, shape, dtype, scale, lead):
    """Normal values, in rows that begin at multiples of 16 bytes."""
    pitch = -(-shape[-1] // lead) * lead
    base = torch.empty(*shape[:-1], pitch, dtype=dtype, device="cuda")
    view = base[..., :shape[-1]]
    if len(shape) == 3:
        for part in view:
            part.copy_(torch.randn(*shape[1:], generator=gen, device="cuda").mul_(scale))
    else:
        view.copy_(torch.randn(*shape, generator=gen, device="cuda").mul_(scale))
    return view


def _empty(shape, dtype, lead=8):
    pitch = -(-shape[-1] // lead) * lead
    return torch.zeros(*shape[:-1], pitch, dtype=dtype, device="cuda")[..., :shape[-1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    counts = _counts(case, seed)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n, rows, k, m = case["n"], case["rows"], case["k"], case["m"]
    dt, out = DTYPES[case["dtype"]], DTYPES[case["out"]]
    s = dict(case=case, offsets=torch.from_numpy(offsets).cuda(), most=int(counts.max()))
    if case["op"] == "product":
        shape = (m, k) if case["trans"] else (k, m)
        s["X"] = _matrix(gen, (rows, k), dt, 1.0, 8)
        if case.get("separate"):
            s["W"] = [_matrix(gen, shape, dt, 0.02, 8) for _ in range(n)]
        else:
            s["W"] = _matrix(gen, (n, *shape), dt, 0.02, 8)
        s["Y"] = _empty((rows, m), out)
    elif case["op"] == "gradient":
        s["A"] = _matrix(gen, (rows, k), dt, 1.0, 8)
        s["B"] = _matrix(gen, (rows, m), dt, 0.01, 8)
        s["C"] = _matrix(gen, (n, k, m), out, 0.1, 8) if case["add"] else None
        s["G"] = _empty((n, k, m), out)
    else:
        s["X"] = _matrix(gen, (rows, k), dt, 1.0, 8)
        # the channels' codes and scales, laid out once when the weights were loaded
        pitch = -(-k // 16) * 16
        s["W"] = torch.zeros(n, m, pitch, dtype=torch.int8, device="cuda")[..., :k]
        s["w_scale"] = torch.empty(n, m, dtype=torch.float32, device="cuda")
        for e in range(n):
            w = torch.randn(m, k, generator=gen, device="cuda").mul_(0.02)
            top = w.abs().amax(1)
            s["w_scale"][e] = top / 127
            s["W"][e] = torch.round(w * (127 / top)[:, None]).to(torch.int8)
        s["Xq"] = torch.zeros(rows, pitch, dtype=torch.int8, device="cuda")[:, :k]
        s["x_scale"] = torch.empty(rows, dtype=torch.float32, device="cuda")
        s["Y"] = _empty((rows, m), out)
    return s


def _places(s, rows):
    """Each row's expert, and its place among that expert's rows."""
    at = torch.arange(rows, device="cuda")
    expert = torch.searchsorted(s["offsets"][1:], at, right=True)
    return expert, at - s["offsets"][expert]


def _spread(x, expert, place, n, most):
    """The rows of each expert as a matrix of their own, zeros below."""
    padded = torch.zeros(n, most, x.shape[1], dtype=x.dtype, device="cuda")
    padded[expert, place] = x
    return padded


def run(s):
    case = s["case"]
    n, most = case["n"], s["most"]
    if case["op"] == "product":
        if own:
            from tiled_newton_schulz_b200 import himuon as hm
            hm.expert_product(s["X"], s["W"], s["Y"], s["offsets"], w_trans=case["trans"])
            return s["Y"]
        expert, place = _places(s, case["rows"])
        W = (torch.stack(s["W"]) if case.get("separate") else s["W"]).float()
        Y = _spread(s["X"].float(), expert, place, n, most) @ (W.mT if case["trans"] else W)
        return Y[expert, place].to(DTYPES[case["out"]])
    if case["op"] == "gradient":
        if own:
            from tiled_newton_schulz_b200 import himuon as hm
            hm.expert_gradient(s["A"], s["B"], s["G"], s["offsets"], beta=1.0 if case["add"] else 0.0, C=s["C"])
            return s["G"]
        expert, place = _places(s, case["rows"])
        G = _spread(s["A"].float(), expert, place, n, most).mT @ _spread(s["B"].float(), expert, place, n, most)
        return (G + s["C"].float() if case["add"] else G).to(DTYPES[case["out"]])
    if own:
        from tiled_newton_schulz_b200 import himuon as hm
        hm.quantize([s["X"]], [s["Xq"]], [s["x_scale"]])
        hm.expert_product_i8(s["Xq"], s["x_scale"], s["W"], s["w_scale"], s["Y"], s["offsets"])
        return s["Y"]
    X = s["X"].float()
    top = X.abs().amax(1)
    codes = torch.round(127 * X / top[:, None])  # 127 x is whole in 32 bits for 16-bit x, so halves are met exactly
    expert, place = _places(s, case["rows"])
    # whole numbers beyond 2^24: the sums need 64 bits
    sums = (_spread(codes.double(), expert, place, n, most) @ s["W"].double().mT)[expert, place]
    return (sums.float() * (top / 127)[:, None] * s["w_scale"][expert]).to(DTYPES[case["out"]])


def work(case):
    n, active, rows, k, m = case["n"], case["active"], case["rows"], case["k"], case["m"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    i, o = size[case["dtype"]], size[case["out"]]
    flops = 2.0 * rows * k * m
    if case["op"] == "product":
        return {"bytes": rows * k * i + active * k * m * i + rows * m * o, "flops": flops}
    if case["op"] == "gradient":
        return {"bytes": rows * (k + m) * i + n * k * m * o * (2 if case["add"] else 1), "flops": flops}
    return {"bytes": rows * k * i + active * (k * m + 4 * m) + rows * m * o, "flops": flops}


def exact(case, seed):
    """From the definitions, expert by expert, in 64 bits."""
    s = prepare(case, seed)
    ends = s["offsets"].tolist()
    groups = [slice(a, b) for a, b in zip(ends, ends[1:])]
    if case["op"] == "product":
        Y = torch.zeros(case["rows"], case["m"], dtype=torch.float64, device="cuda")
        for e, g in enumerate(groups):
            w = s["W"][e].double()
            Y[g] = torch.einsum("rk,mk->rm" if case["trans"] else "rk,km->rm", s["X"][g].double(), w)
        return Y
    if case["op"] == "gradient":
        G = torch.zeros(case["n"], case["k"], case["m"], dtype=torch.float64, device="cuda")
        for e, g in enumerate(groups):
            G[e] = torch.einsum("rk,rm->km", s["A"][g].double(), s["B"][g].double())
            if case["add"]:
                G[e] += s["C"][e].double()
        return G
    Y = torch.zeros(case["rows"], case["m"], dtype=torch.float64, device="cuda")
    X = s["X"].double()
    top = X.abs().max(dim=1).values
    codes = torch.round(127 * X / top[:, None])
    for e, g in enumerate(groups):
        Y[g] = torch.einsum("rk,mk->rm", codes[g], s["W"][e].double()) * (top[g] / 127)[:, None] * s["w_scale"][e].double()
    return Y


if __name__ == "__main__":
    for c in listed() + [draw(random.Random(i)) for i in range(8)]:
        print(c, work(c))

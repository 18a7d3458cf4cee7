"""Cases, inputs and plain forms of the INT8 operators around the experts and of the norm before them: the root-mean-square
norm with the residual's addition and an 8-bit output, rows quantised to INT8 with a scale each, and the experts'
products on such rows with scales for each token and channel.

``run`` computes each operator with elementary torch operations in 32 bits, or, where ``own`` is set, through the
library's prepared calls.  ``exact`` computes the definitions in 64 bits.  INT8 rows are returned as the numbers that
their codes are (BF16 holds every one of them), beside their scales.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
E4M3_MAX, INT8_MAX = 448.0, 127.0
EPS = 1e-6
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn,
      "int8": torch.int8}


def listed():
    return [
        # one token of a decode step, on its way into an INT8 batching: launch latency
        dict(name="norm 1x7168 bf16 int8", op="norm", rows=1, hidden=7168, dtype="bf16", q="int8", residual=True, y=False),
        # no size is a multiple of anything; rows in 32 bits, no residual
        dict(name="norm 333x4095 fp32 int8", op="norm", rows=333, hidden=4095, dtype="fp32", q="int8", residual=False, y=True),
        # a worker's tokens before the e4m3 products
        dict(name="norm 4608x7168 bf16 fp8", op="norm", rows=4608, hidden=7168, dtype="bf16", q="fp8", residual=True, y=False),
        # a prefill of 16384 tokens; the router takes the 16-bit rows beside the INT8 ones
        dict(name="norm 16384x4096 fp16 int8 y", op="norm", rows=16384, hidden=4096, dtype="fp16", q="int8", residual=True, y=True),
        # one decode step of two sessions: 48 slots of a small hidden size, launch latency
        dict(name="quant 48x128 fp16", op="quant", rows=48, actual=43, hidden=128, dtype="fp16"),
        # a batching worker's 16-bit output, 16 x 32 x 9 slots with 5% masked, on its way into the first product
        dict(name="quant 4608x7168 bf16", op="quant", rows=4608, actual=4377, hidden=7168, dtype="bf16"),
        # one token through a dense expert: the weights are read once for a single row
        dict(name="matmul 1x4096x7168", op="matmul", rows=1, actual=1, experts=0, k=7168, n=4096,
             epilogue="none", out="bf16", skew=0.0),
        # ragged in every direction: no size is a multiple of a tile
        dict(name="matmul 100x1000x1040 fp32", op="matmul", rows=100, actual=100, experts=0, k=1040, n=1000,
             epilogue="none", out="fp32", skew=0.0),
        # a dense product of a prefill, one row short of a round number
        dict(name="matmul 8191x7168x5120", op="matmul", rows=8191, actual=8191, experts=0, k=5120, n=7168,
             epilogue="none", out="bf16", skew=0.0),
        # gate and up products of an INT8 batching: 256 experts with a skewed load, a few rows for most of them
        dict(name="gate_up 256e 4377 int8", op="matmul", rows=4608, actual=4377, experts=256, k=7168, n=2048,
             epilogue="swiglu", out="int8", skew=1.1),
        # the down product that follows it
        dict(name="down 256e 4377 bf16", op="matmul", rows=4608, actual=4377, experts=256, k=1024, n=7168,
             epilogue="none", out="bf16", skew=1.1),
        # gate and up products of a prefill: 16384 tokens with 8 experts each
        dict(name="gate_up 128e 131072 int8", op="matmul", rows=131072, actual=131072, experts=128, k=4096, n=2048,
             epilogue="swiglu", out="int8", skew=0.0),
    ]


def draw(rng):
    def log(lo, hi, step=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)

    op = rng.choice(["norm", "norm", "quant", "matmul", "matmul", "matmul"])
    if op == "norm":
        return dict(op=op, rows=log(1, 16384), hidden=log(16, 8192, rng.choice([1, 8, 16])),
                    dtype=rng.choice(["fp16", "bf16", "fp32"]), q=rng.choice(["int8", "fp8"]),
                    residual=rng.random() < 0.7, y=rng.random() < 0.5)
    if op == "quant":
        rows, hidden = log(1, 8192), log(16, 8192, rng.choice([1, 8, 16]))
        return dict(op=op, rows=rows, actual=rng.randint((rows + 1) // 2, rows), hidden=hidden,
                    dtype=rng.choice(["fp16", "bf16", "fp32"]))
    experts = rng.choice([0, log(1, 256)])
    epilogue = rng.choice(["none", "swiglu"])
    while True:
        rows, k = log(1, 65536), log(16, 8192, 16)
        n = 2 * log(16, 4096, 16) if epilogue == "swiglu" else log(1, 8192)
        if max(experts, 1) * n * k <= 3_700_000_000 and rows * n * k <= 600_000_000_000:
            break
    return dict(op=op, rows=rows, actual=rng.randint((rows + 1) // 2, rows) if experts else rows, experts=experts,
                k=k, n=n, epilogue=epilogue,
                out=rng.choice(["bf16", "fp16", "fp32"] + (["int8", "int8"] if epilogue == "swiglu" else [])),
                skew=rng.choice([0.0, 0.6, 1.1]))


# ------------------------------------------------------------------------------ inputs

def _activations(rows, hidden, gen, dtype):
    """Rows of different size, some columns far larger than the rest."""
    x = torch.randn((rows, hidden), generator=gen, device=DEV)
    x *= torch.exp(torch.randn((rows, 1), generator=gen, device=DEV))
    x *= torch.exp(0.5 * torch.randn((1, hidden), generator=gen, device=DEV))
    return x.to(DT[dtype])


def _codes(shape, gen, out=None):
    """INT8 codes as a normal row quantised by its largest value holds them."""
    out = torch.empty(shape, dtype=torch.int8, device=DEV) if out is None else out
    out.copy_((torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16) * 34).round_().clamp_(-127, 127))
    return out


def _counts(case, seed):
    """Rows of each expert: a seeded draw from uniform or Zipf-like shares, every row placed."""
    experts, rng = case["experts"], torch.Generator().manual_seed(seed)
    share = torch.arange(1, experts + 1, dtype=torch.float64) ** -case["skew"]
    share = share[torch.randperm(experts, generator=rng)]
    pick = torch.multinomial(share, case["actual"], replacement=True, generator=rng)
    return torch.bincount(pick, minlength=experts)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        s["x"] = _activations(case["rows"], case["hidden"], gen, case["dtype"])
        s["gamma"] = (1 + 0.2 * torch.randn(case["hidden"], generator=gen, device=DEV)).to(DT[case["dtype"]])
        s["res"] = _activations(case["rows"], case["hidden"], gen, case["dtype"]) if case["residual"] else None
        return s
    if case["op"] == "quant":
        s["x"] = _activations(case["rows"], case["hidden"], gen, case["dtype"])
        s["actual_rows"] = torch.tensor([case["actual"]], dtype=torch.int64, device=DEV)
        return s
    rows, k, n, experts = case["rows"], case["k"], case["n"], max(case["experts"], 1)
    s["x"] = _codes((rows, k), gen)
    s["x_scale"] = (torch.rand(rows, generator=gen, device=DEV) + 0.5) / 34
    s["w"] = torch.empty((experts, n, k), dtype=torch.int8, device=DEV)
    for e in range(experts):
        _codes((n, k), gen, s["w"][e])
    s["w_scale"] = (torch.rand((experts, n), generator=gen, device=DEV) + 0.5) * (k ** -0.5 / 34)
    s["group_list"] = None
    if case["experts"]:
        counts = _counts(case, seed)
        present = counts.nonzero().flatten()
        group_list = torch.zeros((case["experts"], 2), dtype=torch.int64)
        group_list[:len(present), 0] = present
        group_list[:len(present), 1] = counts[present]
        s["group_list"], s["most"] = group_list.to(DEV), int(counts.max())
    return s


# ------------------------------------------------------------------------------ plain forms

def _quantised(x, q="int8"):
    """Rows in 32 bits -> INT8 with a scale for each row, or e4m3 with one for each 128 elements of a row."""
    if q == "int8":
        amax = x.abs().amax(1)
        scale = (amax / torch.full_like(amax, INT8_MAX)).clamp_min(2.0 ** -126)
        return (x / scale[:, None]).round().to(torch.int8), scale
    rows, n = x.shape
    blocks = -(-n // BLOCK)
    x = torch.nn.functional.pad(x, (0, blocks * BLOCK - n)).view(rows, blocks, BLOCK)
    amax = x.abs().amax(2)
    scale = (amax / torch.full_like(amax, E4M3_MAX)).clamp_min(2.0 ** -126)
    codes = (x / scale[:, :, None]).to(torch.float8_e4m3fn).view(rows, blocks * BLOCK)
    return codes[:, :n].contiguous(), scale


def _norm_plain(s):
    t = s["x"].float()
    if s["residual"]:
        t = t + s["res"].float()
    n = t * s["gamma"].float() * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
    q, scale = _quantised(n, s["q"])
    out = dict(q=q, scale=scale)
    if s["residual"]:
        out["residual_out"] = t.to(DT[s["dtype"]])
    if s["y"]:
        out["y"] = n.to(DT[s["dtype"]])
    return out


def _matmul_plain(s):
    x, w = s["x"].float(), s["w"].float()
    if s["group_list"] is None:
        y = x @ w[0].t() * s["x_scale"][:, None] * s["w_scale"]
    else:
        # rows laid out as [experts, most, k], one batched product, and back
        keys, counts = s["group_list"][:, 0], s["group_list"][:, 1]
        first = torch.cumsum(counts, 0) - counts
        i = torch.arange(s["actual"], device=x.device)
        group = torch.searchsorted(first + counts, i, right=True)
        at = keys[group] * s["most"] + i - first[group]
        padded = x.new_zeros((s["experts"] * s["most"], s["k"]))
        padded[at] = x[:s["actual"]]
        padded = padded.view(s["experts"], s["most"], s["k"]).transpose(1, 2).contiguous()
        y = torch.bmm(w, padded).transpose(1, 2).reshape(s["experts"] * s["most"], s["n"])[at]
        y = y * s["x_scale"][:s["actual"], None] * s["w_scale"][keys[group]]
    if s["epilogue"] == "swiglu":
        gate, up = y.split(s["n"] // 2, dim=1)
        y = gate * torch.sigmoid(gate) * up
    if s["out"] == "int8":
        q, scale = _quantised(y)
        return dict(y=q, y_scale=scale)
    return dict(y=y.to(DT[s["out"]]))


def _own(s):
    import unpermute_ffnwb_batching_amd as F
    # a serving loop prepares its calls once and runs them on the same buffers
    if "call" not in s:
        if s["op"] == "norm":
            s["call"] = F.RmsNormQuantCall(s["x"], s["gamma"], residual=s["res"], eps=EPS, q_dtype=DT[s["q"]], with_y=s["y"])
        elif s["op"] == "quant":
            s["call"] = F.QuantInt8Call(s["x"], actual_rows=s["actual_rows"])
        else:
            s["call"] = F.GroupedMatmulInt8Call(
                s["x"], s["x_scale"], s["w"], s["w_scale"], group_list=s["group_list"],
                epilogue=F.FFNWB_EPI_SWIGLU if s["epilogue"] == "swiglu" else F.FFNWB_EPI_NONE, out_dtype=DT[s["out"]])
    out = s["call"].run()
    if s.get("actual", s["rows"]) == s["rows"]:
        return out
    return {k: v[:s["actual"]] for k, v in out.items()}


def run(state):
    s = state
    if own:
        out = _own(s)
    elif s["op"] == "norm":
        out = _norm_plain(s)
    elif s["op"] == "quant":
        out = dict(zip(("q", "scale"), _quantised(s["x"][:s["actual"]].float())))
    else:
        out = _matmul_plain(s)
    return {k: v.to(torch.bfloat16) if v.dtype == torch.int8 else v for k, v in out.items()}


# ------------------------------------------------------------------------------ work

def _size(dtype):
    return torch.empty(0, dtype=DT[dtype]).element_size()


def work(case):
    if case["op"] == "norm":
        rows, hidden, elt = case["rows"], case["hidden"], _size(case["dtype"])
        scales = rows * (1 if case["q"] == "int8" else -(-hidden // BLOCK)) * 4
        moved = 1 + 2 * case["residual"] + case["y"]  # x, the residual and its sum, the rows in their own type
        return {"bytes": rows * hidden * (moved * elt + 1) + scales + hidden * elt, "flops": 10 * rows * hidden}
    if case["op"] == "quant":
        cells = case["actual"] * case["hidden"]
        return {"bytes": cells * (_size(case["dtype"]) + 1) + case["actual"] * 4, "flops": 4 * cells}
    m, n, k, experts = case["actual"], case["n"], case["k"], max(case["experts"], 1)
    share = [(i + 1) ** -case["skew"] for i in range(experts)]
    present = sum(1 - (1 - p / sum(share)) ** m for p in share)  # experts that get a row, on average
    cols = n // 2 if case["epilogue"] == "swiglu" else n
    out = m * cols * _size(case["out"]) + (m * 4 if case["out"] == "int8" else 0)
    return {"bytes": m * (k + 4) + present * n * (k + 4) + out, "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------ exact

def _exact_int8(v):
    scale = (v.abs().max(1).values / INT8_MAX).clamp_min(2.0 ** -126)
    return torch.round(v / scale[:, None]), scale


def _to_e4m3(v):
    """float64 -> the nearest e4m3 value, ties to even (|v| <= 448 up to rounding)."""
    exponent = torch.frexp(v.abs()).exponent.clamp_min(-5).long() - 1
    step = ((exponent - 3 + 1023) << 52).view(torch.float64)  # 2^(exponent - 3), exactly
    return (torch.round(v / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_fp8(v):
    q, scales = torch.empty_like(v), []
    for b in range(0, v.shape[1], BLOCK):
        part = v[:, b:b + BLOCK]
        scales.append((part.abs().max(1, keepdim=True).values / E4M3_MAX).clamp_min(2.0 ** -126))
        q[:, b:b + BLOCK] = _to_e4m3(part / scales[-1])
    return q, torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return dict(zip(("q", "scale"), _exact_int8(s["x"][:case["actual"]].double())))
    if case["op"] == "norm":
        out = dict(q=[], scale=[], residual_out=[], y=[])
        for i in range(0, case["rows"], 2048):
            v = s["x"][i:i + 2048].double()
            if case["residual"]:
                v = v + s["res"][i:i + 2048].double()
                out["residual_out"].append(v)
            mean = v.square().sum(1, keepdim=True) / case["hidden"]
            n = v / (mean + EPS).sqrt() * s["gamma"].double()
            q, scale = (_exact_int8 if case["q"] == "int8" else _exact_fp8)(n)
            out["q"].append(q)
            out["scale"].append(scale)
            if case["y"]:
                out["y"].append(n)
        return {k: torch.cat(v) for k, v in out.items() if v}
    groups = [(0, case["actual"])] if s["group_list"] is None else [tuple(g) for g in s["group_list"].tolist()]
    done, at = [], 0
    for e, count in groups:
        if count == 0:
            continue
        w = s["w"][e].double() * s["w_scale"][e].double()[:, None]
        x = s["x"][at:at + count].double() * s["x_scale"][at:at + count].double()[:, None]
        y = x @ w.t()
        if case["epilogue"] == "swiglu":
            gate, up = y[:, :case["n"] // 2], y[:, case["n"] // 2:]
            y = gate / (1 + torch.exp(-gate)) * up
        done.append(y)
        at += count
    y = torch.cat(done)
    return dict(zip(("y", "y_scale"), _exact_int8(y))) if case["out"] == "int8" else dict(y=y)

"""Cases of the microscaled 4-bit operators: rows kept in 4 bits and read back, products, the memory projection.

A row is cut into blocks of values that share a scale; a value is an e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4 or 6, with a
sign) times its block's scale, rounded to nearest with ties to the even code.

- mxfp4: blocks of 32, scale 2^(floor(log2(amax)) - 2), not below 2^-127; larger quotients than 6 become 6.
- nvfp4: blocks of 16, scale r * e4m3(amax / (6 r)) with r = 2^(floor(log2(amax of the row)) - 10), not below 2^-126.

The last block of a row may be short.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = {"mxfp4": 32, "nvfp4": 16}
EPS = 1e-5  # of the memory LayerNorm


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a chunk of 64 streamed memory rows, kept and read back
        dict(name="keep_chunk_64", op="keep", format="nvfp4", rows=64, cols=4096, dtype="bf16", out="bf16"),
        # a weight matrix of the 5120-wide head in fp32, as a program quantises its weights
        dict(name="keep_weight_fp32", op="keep", format="mxfp4", rows=4096, cols=5120, dtype="fp32", out="fp32"),
        # ragged rows of an odd width in fp16
        dict(name="keep_odd", op="keep", format="nvfp4", rows=3001, cols=1111, dtype="fp16", out="fp32"),
        # the memory rows of 8 records of 16384
        dict(name="keep_memory_8x16k", op="keep", format="nvfp4", rows=131072, cols=4096, dtype="bf16", out="bf16"),
        # one token through a square layer: latency
        dict(name="linear_one_token", op="linear", format="nvfp4", rows=1, cols=4096, outs=4096, dtype="bf16", out="bf16"),
        # a serving batch of 24 tokens through a wide layer
        dict(name="linear_step_24", op="linear", format="mxfp4", rows=24, cols=4096, outs=16384, dtype="bf16", out="bf16"),
        # the options of 8 records through the feed-forward layer of the head
        dict(name="linear_options_511", op="linear", format="nvfp4", rows=511, cols=1024, outs=4096, dtype="fp16", out="fp16"),
        # odd sizes all round, sums kept in fp32
        dict(name="linear_odd", op="linear", format="mxfp4", rows=333, cols=1000, outs=777, dtype="fp32", out="fp32"),
        # a prompt of 8192 tokens through a wide layer
        dict(name="linear_prompt_8k", op="linear", format="mxfp4", rows=8192, cols=5120, outs=5120, dtype="bf16", out="bf16"),
        # 64 streamed memory rows to the keys and values of both routing layers
        dict(name="project_chunk_64", op="project", format="nvfp4", rows=64, cols=4096, outs=4096, dtype="bf16", out="bf16"),
        # a ragged record of the 5120-wide head in fp16
        dict(name="project_record_5k", op="project", format="mxfp4", rows=5003, cols=5120, outs=4096, dtype="fp16", out="bf16"),
        # the memory of 8 records of 16384 rows to keys and values: the head's largest product
        dict(name="project_memory_8x16k", op="project", format="nvfp4", rows=131072, cols=4096, outs=4096, dtype="bf16",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["keep", "linear", "linear", "project"])
    cols = _log(rng, 32, 8192)
    if rng.random() < 0.6:
        cols = max(32, cols // 64 * 64)
    case = dict(op=op, format=rng.choice(["mxfp4", "nvfp4"]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                out=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if op == "keep":
        return dict(case, rows=_log(rng, 1, min(131072, 200_000_000 // cols)), cols=cols)
    outs = _log(rng, 16, 16384)
    if rng.random() < 0.7:
        outs = max(16, outs // 16 * 16)
    return dict(case, rows=_log(rng, 1, min(131072, 200_000_000 // cols, 400_000_000 // outs)), cols=cols, outs=outs)


def _kept_bytes(case, rows):
    """Codes and scales of `rows` rows."""
    return rows * (-(-case["cols"] // 2) + -(-case["cols"] // BLOCK[case["format"]]) + (4 if case["format"] == "nvfp4" else 0))


def work(case):
    rows, cols = case["rows"], case["cols"]
    size, to = TYPES[case["dtype"]].itemsize, TYPES[case["out"]].itemsize
    if case["op"] == "keep":  # in, kept, and what it stands for read back
        return {"bytes": rows * cols * (size + to) + 2 * _kept_bytes(case, rows), "flops": 0}
    outs = case["outs"]
    more = 12 * outs + 8 * rows if case["op"] == "project" else 4 * outs
    return {"bytes": rows * cols * size + _kept_bytes(case, outs) + rows * outs * to + more, "flops": 2 * rows * cols * outs}


# --------------------------------------------------------------------- inputs

def _rows(rows, cols, dtype, g):
    """Hidden rows as a backbone leaves them: rows of uneven size, a few strong channels, a small offset."""
    x = torch.randn(rows, cols, generator=g, device=DEVICE)
    strong = 1 + 7 * (torch.rand(cols, generator=g, device=DEVICE) < 0.01)
    size = torch.exp(0.4 * torch.randn(rows, 1, generator=g, device=DEVICE))
    return x.mul_(strong).add_(0.1).mul_(size).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    s = dict(case=case, x=_rows(case["rows"], case["cols"], TYPES[case["dtype"]], g))
    if case["op"] != "keep":
        w = torch.randn(case["outs"], case["cols"], generator=g, device=DEVICE) * case["cols"] ** -0.5
        s["w"] = w.bfloat16()
        s["bias"] = 0.1 * torch.randn(case["outs"], generator=g, device=DEVICE)
        _kept_weights(s)
    return s


def _kept_weights(s):
    """The weights as a program keeps them: in 4 bits, or as the numbers that they stand for."""
    if own:
        from structured_decision_model_gb300.microscaled import Fp4Linear
        s["layer"] = Fp4Linear(s["w"], s["bias"], s["case"]["format"])
    else:
        s["kept"] = _plain_kept(s["w"], s["case"]["format"])


# ------------------------------------------------------------------ plain forms

def _power(x, least):
    """2^floor(log2 x), not below 2^least; x >= 0.  A number over its own fraction is a power of two, without rounding."""
    part, _ = torch.frexp(x)
    return torch.where(x > 0, x / torch.where(x > 0, 2 * part, 1), 0).clamp(min=2.0 ** least)


def _plain_kept(x, form):
    """What the rows of x stand for once kept, in 32 bits (64 for fp32 rows, whose quotients lie next to the borders)."""
    wide = torch.float64 if x.dtype == torch.float32 else torch.float32
    rows, cols, n = *x.shape, BLOCK[form]
    y = torch.nn.functional.pad(x.to(wide), (0, -cols % n)).view(rows, -1, n)
    top = y.abs().amax(-1, keepdim=True)
    if form == "mxfp4":
        scale = _power(top, -125) * 0.25
    else:
        r = _power(top.amax(1, keepdim=True), -116) * 2.0 ** -10
        q = top / r / 6
        # e4m3: 3 bits behind the point, steps of 2^-9 below 2^-6
        step = _power(q, -6) * 0.125
        scale = (q / step).round() * step * r
    q = y.abs() / torch.where(scale == 0, 1, scale)
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))
    q = ((q / step).round() * step).clamp(max=6) * (scale != 0)
    return (q * torch.sign(y) * scale).view(rows, -1)[:, :cols].float()


def _plain_keep(s):
    return {"values": _plain_kept(s["x"], s["case"]["format"]).to(TYPES[s["case"]["out"]])}


def _plain_linear(s):
    x = _plain_kept(s["x"], s["case"]["format"])
    return {"y": (torch.matmul(x, s["kept"].T) + s["bias"]).to(TYPES[s["case"]["out"]])}


def _plain_project(s):
    x, w = s["x"].float(), s["kept"]
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    del x
    y = torch.matmul(_plain_kept(s["x"], s["case"]["format"]), w.T)
    y = rstd * (y - mean * w.sum(1)) + s["bias"]
    return {"y": y.to(TYPES[s["case"]["out"]]), "mean": mean.squeeze(1), "rstd": rstd.squeeze(1)}


def run(state):
    case = state["case"]
    if own:
        from structured_decision_model_gb300.microscaled import quantize
        out = TYPES[case["out"]]
        if case["op"] == "keep":
            return {"values": quantize(state["x"], case["format"]).dequantize(out)}
        if case["op"] == "linear":
            return {"y": state["layer"](state["x"], out)}
        y, mean, rstd = state["layer"].normalized(state["x"], out)
        return {"y": y, "mean": mean, "rstd": rstd}
    return {"keep": _plain_keep, "linear": _plain_linear, "project": _plain_project}[case["op"]](state)


# ------------------------------------------------- the definition, in 64 bits

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_power(x):
    """The power of two at or below fp64 x >= 0 (0 for 0): its exponent's bits alone."""
    return (x.contiguous().view(torch.int64) & (0x7FF << 52)).view(torch.float64)


def _exact_kept(x, form):
    """What the rows of x stand for, block by block, each quotient compared with the borders between numbers."""
    x = x.double()
    y = torch.zeros_like(x)
    row = x.abs().amax(1)
    r = (_exact_power(row) / 1024).clamp(min=2.0 ** -126)
    levels = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    for a in range(0, x.shape[1], BLOCK[form]):
        part = x[:, a:a + BLOCK[form]]
        top = part.abs().amax(1)
        if form == "mxfp4":
            scale = (_exact_power(top) / 4).clamp(min=2.0 ** -127)
        else:
            # every e4m3 number that is not negative, and the nearest of them
            low = (top / (6 * r)).contiguous()
            grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] +
                                [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8)][:-1],
                                dtype=torch.float64, device=x.device)
            i = torch.searchsorted(grid, low).clamp(1, len(grid) - 1)
            below, above = low - grid[i - 1], grid[i] - low
            i = torch.where((below < above) | ((below == above) & ((i - 1) % 2 == 0)), i - 1, i)
            scale = grid[i] * r
        size = part.abs() / torch.where(scale > 0, scale, torch.inf)[:, None]
        code = torch.zeros_like(size, dtype=torch.long)
        for c in range(7):  # a tie goes to the even code
            border = (_E2M1[c] + _E2M1[c + 1]) / 2
            code += (size > border) if c % 2 == 0 else (size >= border)
        y[:, a:a + BLOCK[form]] = torch.where(part < 0, -levels[code], levels[code]) * scale[:, None]
    return y


def exact(case, seed):
    if case["op"] != "keep" and 2.0 * case["rows"] * case["cols"] * case["outs"] > 1e13:
        return None
    s = prepare(case, seed)
    x = s["x"]
    step = max(1, 30_000_000 // case["cols"])
    parts = []
    w = _exact_kept(s["w"], case["format"]) if case["op"] != "keep" else None
    for a in range(0, len(x), step):
        rows = x[a:a + step].double()
        kept = _exact_kept(rows, case["format"])
        if case["op"] == "keep":
            parts.append((kept,))
            continue
        y = kept @ w.T
        if case["op"] == "project":
            mean = rows.sum(1) / rows.shape[1]
            var = ((rows - mean[:, None]) ** 2).sum(1) / rows.shape[1]
            rstd = (var + EPS) ** -0.5
            y = (y - torch.outer(mean, w.sum(1))) * rstd[:, None]
            parts.append((y + s["bias"].double(), mean, rstd))
        else:
            parts.append((y + s["bias"].double(),))
    names = {"keep": ("values",), "linear": ("y",), "project": ("y", "mean", "rstd")}[case["op"]]
    return {k: torch.cat(v) for k, v in zip(names, zip(*parts))}

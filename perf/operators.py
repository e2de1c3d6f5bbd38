"""Cases of the 8-bit integer and the expert-grouped products, for measuring them.

Four operators: the per-token int8 quantiser, the int8 product with a scale
per token and per channel, the product of ragged groups of rows with one
weight per group ("experts"), and that product's weight gradient. `run` makes
the library's calls where `own` is true, and computes the same with elementary
torch operations in 32 bits where it is false; `exact` has the values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

# Sizes: 4096, 7168, 2048, 14336 and 18432 are the projection, FFN and decode
# widths of this repository's own workloads; the others are generic.
_CASES = [
    # One token of a decode step: latency alone.
    {"name": "quant_token", "op": "quant", "rows": 1, "k": 4096},
    # A prompt's FFN activations: bandwidth.
    {"name": "quant_prompt", "op": "quant", "rows": 8192, "k": 14336},
    # Decode, one token against the widest weight: the weight is streamed once.
    {"name": "int8_decode", "op": "int8", "m": 1, "n": 18432, "k": 4096, "out": "bf16",
     "bias": False, "gelu": False, "zero": False},
    # Prefill projection with its bias and activation.
    {"name": "int8_projection", "op": "int8", "m": 4096, "n": 7168, "k": 2048, "out": "bf16",
     "bias": True, "gelu": True, "zero": False},
    # Asymmetric activations (a zero point per token), no size a multiple of anything.
    {"name": "int8_zero_odd", "op": "int8", "m": 1001, "n": 4093, "k": 4099, "out": "f32",
     "bias": True, "gelu": False, "zero": True},
    # Decode of a batch through an expert layer: a row or two per expert, many experts idle.
    {"name": "experts_bf16_decode", "op": "grouped", "type": "bf16", "layout": "col", "t": 32,
     "g": 64, "live": 24, "cap": 4, "n": 2048, "k": 4096, "out": "bf16", "bias": False,
     "gelu": False},
    # The forward pass of a training step: many rows per expert.
    {"name": "experts_bf16_forward", "op": "grouped", "type": "bf16", "layout": "col", "t": 16384,
     "g": 8, "live": 8, "cap": 4096, "n": 14336, "k": 4096, "out": "bf16", "bias": True,
     "gelu": True},
    # Input gradient: the same weights read along their other axis; uneven groups, some empty.
    {"name": "experts_bf16_dgrad", "op": "grouped", "type": "bf16", "layout": "row", "t": 5000,
     "g": 16, "live": 13, "cap": 1000, "n": 4096, "k": 2048, "out": "bf16", "bias": False,
     "gelu": False},
    # Weight gradient of the training step, kept in FP32.
    {"name": "experts_wgrad", "op": "wgrad", "t": 16384, "g": 8, "live": 8, "cap": 4096,
     "n": 14336, "k": 4096, "out": "f32"},
    # Weight gradient of many small experts, a few rows each, some without any.
    {"name": "experts_wgrad_small", "op": "wgrad", "t": 777, "g": 32, "live": 27, "cap": 100,
     "n": 1000, "k": 2048, "out": "bf16"},
    # Decode of a larger batch with 8-bit experts.
    {"name": "experts_int8_decode", "op": "grouped", "type": "int8", "layout": "col", "t": 128,
     "g": 32, "live": 30, "cap": 16, "n": 4096, "k": 2048, "out": "bf16", "bias": True,
     "gelu": False},
    # Prefill through 8-bit experts.
    {"name": "experts_int8_prefill", "op": "grouped", "type": "int8", "layout": "col", "t": 8192,
     "g": 32, "live": 31, "cap": 768, "n": 4096, "k": 4096, "out": "bf16", "bias": True,
     "gelu": True},
]

_MOST_FLOPS = 2.0 * 16384 * 14336 * 4096
_MOST_WEIGHTS = 8 * 14336 * 4096


def listed():
    return [dict(c) for c in _CASES]


def _spread(rng, lo, hi, multiple):
    """A size between lo and hi, spread over its logarithm; a multiple of `multiple` three times in four."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.75:
        v = v // multiple * multiple
    return max(lo, min(hi, v))


def draw(rng):
    while True:
        op = rng.choice(("quant", "int8", "int8", "grouped", "grouped", "grouped", "wgrad", "wgrad"))
        if op == "quant":
            return {"op": op, "rows": _spread(rng, 1, 8192, 1), "k": _spread(rng, 64, 14336, 64)}
        n, k = _spread(rng, 256, 18432, 64), _spread(rng, 256, 14336, 64)
        if op == "int8":
            c = {"op": op, "m": _spread(rng, 1, 8192, 1), "n": n, "k": k,
                 "out": rng.choice(("bf16", "f32")), "bias": rng.random() < 0.5,
                 "gelu": rng.random() < 0.3, "zero": rng.random() < 0.3}
            if 2.0 * c["m"] * n * k <= _MOST_FLOPS:
                return c
            continue
        t = _spread(rng, 1, 16384, 1)
        g = int(round(math.exp(rng.uniform(0, math.log(64)))))
        live = rng.randint(max(1, min(g, t) // 2), min(g, t))
        cap = min(t, max(1, math.ceil(t / live * rng.uniform(1.1, 2.5))))
        # The plain form computes every group at its capacity: bounded with it.
        if g * n * k > _MOST_WEIGHTS or 2.0 * g * max(cap, t / g) * n * k > 2 * _MOST_FLOPS:
            continue
        c = {"op": op, "t": t, "g": g, "live": live, "cap": cap, "n": n, "k": k,
             "out": rng.choice(("bf16", "f32"))}
        if 2.0 * t * n * k > _MOST_FLOPS:
            continue
        if op == "grouped":
            c["type"] = rng.choice(("bf16", "bf16", "int8", "fp8"))
            c["layout"] = rng.choice(("col", "row")) if c["type"] == "bf16" else "col"
            c["bias"], c["gelu"] = rng.random() < 0.5, rng.random() < 0.3
            if c["type"] == "fp8":
                c["out"] = "bf16"  # the matrix cores' E4M3 sums keep fewer bits than an FP32 result shows
        return c


def _sizes(case, seed):
    """Rows per group: `live` groups get at least one row and at most `cap`, unevenly; the others none."""
    rng = np.random.default_rng(seed)
    live, t, cap = case["live"], case["t"], case["cap"]
    p = rng.lognormal(0.0, 0.6, live)
    n = np.minimum(cap, 1 + np.floor((t - live) * p / p.sum()).astype(np.int64))
    for i in rng.permutation(live):
        n[i] += min(cap - n[i], t - n.sum())
    sizes = np.zeros(case["g"], dtype=np.int64)
    sizes[rng.permutation(case["g"])[:live]] = n
    return sizes


def _quantised(x, top, dtype):
    """Rows of x (last axis) as codes of a symmetric 8-bit type and one scale per row."""
    s = x.abs().amax(-1) / top
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = x / s.unsqueeze(-1)
    return (q.round().clamp(-top, top) if dtype == torch.int8 else q.clamp(-top, top)).to(dtype), s


def _plain(n):
    return torch.float32 if n == "f32" else torch.bfloat16


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": dict(case)}
    op = case["op"]
    if op == "quant":
        m, k = case["rows"], case["k"]
        # Activations: every token has a level of its own.
        level = torch.exp(normal(m, 1, dtype=torch.float32))
        s["x"] = (normal(m, k, dtype=torch.float32) * level).to(torch.bfloat16)
        s["q"] = torch.empty(m, k, device="cuda", dtype=torch.int8)
        s["scale"] = torch.empty(m, device="cuda")
        return s
    n, k = case["n"], case["k"]
    if op == "int8":
        m = case["m"]
        x = normal(m, k, dtype=torch.float32)
        if case["zero"]:
            # Activations around a mean of their own: codes over the whole range, and a zero point.
            x = x.abs_()
            s["sa"] = x.amax(-1) / 255
            s["za"] = torch.full((m,), -128, device="cuda", dtype=torch.int32)
            s["a"] = ((x / s["sa"][:, None]).round() - 128).clamp_(-128, 127).to(torch.int8)
        else:
            s["a"], s["sa"] = _quantised(x, 127, torch.int8)
            s["za"] = None
        s["b"], s["sb"] = _quantised(normal(n, k, std=0.02, dtype=torch.float32), 127, torch.int8)
        s["sumb"] = s["b"].sum(1, dtype=torch.int32) if case["zero"] else None
        s["bias"] = normal(n, std=0.1) if case["bias"] else None
        s["c"] = torch.empty(m, n, device="cuda", dtype=_plain(case["out"]))
        return s
    t, g = case["t"], case["g"]
    sizes = _sizes(case, seed)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    s["off"] = torch.from_numpy(off).cuda()
    if op == "wgrad":
        s["d"], s["x"] = normal(t, n), normal(t, k)
        s["c"] = torch.empty(g, n, k, device="cuda", dtype=_plain(case["out"]))
        return s
    s["bias"] = normal(g, n, std=0.1) if case["bias"] else None
    s["c"] = torch.empty(t, n, device="cuda", dtype=_plain(case["out"]))
    x = normal(t, k, dtype=torch.float32)
    w = torch.empty(0)
    if case["type"] == "bf16":
        s["a"] = x.to(torch.bfloat16)
        s["b"] = normal(*((g, n, k) if case["layout"] == "col" else (g, k, n)), std=0.02)
    else:
        top, kind = (127, torch.int8) if case["type"] == "int8" else (448, torch.float8_e4m3fn)
        s["a"], s["sa"] = _quantised(x, top, kind)
        w = normal(g, n, k, std=0.02, dtype=torch.float32)
        s["b"], s["sb"] = _quantised(w, top, kind)
    return s


# ------------------------------------------------------------------ the library's calls

def _run_own(s):
    import dense_gemm_09_amd as lib
    case = s["case"]
    op = case["op"]
    if op == "quant":
        m, k = case["rows"], case["k"]
        lib.quantize_int8_rows(m, k, s["x"], k, s["q"], k, s["scale"])
        return {"q": s["q"], "scale": s["scale"]}
    n, k, c = case["n"], case["k"], s["c"]
    out = lib.OUT_F32 if case["out"] == "f32" else lib.OUT_BF16
    if op == "wgrad":
        lib.gemm_grouped_bf16_wgrad(case["g"], case["t"], n, k, 1.0, s["d"], n, s["x"], k, s["off"],
                                    0.0, c, k, n * k, out)
        return c
    act = lib.ACT_GELU_ERF if case["gelu"] else lib.ACT_NONE
    if op == "int8":
        lib.gemm_int8_scaled(case["m"], n, k, 1.0, s["a"], k, lib.ROW, s["b"], k, lib.COL, s["sa"],
                             s["za"], s["sb"], s["sumb"], 0.0, c, n, out, s["bias"], act)
    elif case["type"] == "bf16":
        col = case["layout"] == "col"
        lib.gemm_grouped_bf16(case["g"], case["t"], n, k, 1.0, s["a"], k, s["off"], s["b"],
                              k if col else n, lib.COL if col else lib.ROW, n * k, 0.0, c, n, out,
                              s["bias"], act)
    elif case["type"] == "int8":
        lib.gemm_grouped_int8_scaled(case["g"], case["t"], n, k, 1.0, s["a"], k, s["off"], s["b"], k,
                                     lib.COL, n * k, s["sa"], None, s["sb"], None, 0.0, c, n, out,
                                     s["bias"], act)
    else:
        lib.gemm_grouped_fp8_scaled(case["g"], case["t"], n, k, 1.0, s["a"], k, s["off"], s["b"], k,
                                    lib.COL, n * k, s["sa"], s["sb"], 0.0, c, n, out, s["bias"], act)
    return c


# ------------------------------------------------------------------ the plain forms

def _gelu(z):
    return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))


def _padded(x, off, cap):
    """Rows of each group as [groups, cap, width] in FP32, zeros past a group's end."""
    at = torch.arange(cap, device=x.device)
    rows = off[:-1, None].long() + at
    ok = at < (off[1:] - off[:-1])[:, None]
    return x.float()[rows.clamp(max=x.shape[0] - 1)] * ok[..., None]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        x = s["x"].float()
        amax = x.abs().amax(1)
        # Tensor divisors: dividing by a number may be computed as a product with its reciprocal.
        scale = torch.where(amax > 0, amax / torch.full_like(amax, 127.0), torch.ones_like(amax))
        q = torch.round(x / scale[:, None]).clamp(-127, 127).to(torch.int8)
        return {"q": q, "scale": scale}
    if op == "int8":
        a = s["a"].float()
        if s["za"] is not None:
            a = a - s["za"].float()[:, None]
        z = (a @ s["b"].float().t()) * (s["sa"][:, None] * s["sb"])
        z = z if s["bias"] is None else z + s["bias"].float()
        return (_gelu(z) if case["gelu"] else z).to(_plain(case["out"]))
    off, cap, t = s["off"], case["cap"], case["t"]
    if op == "wgrad":
        d, x = _padded(s["d"], off, cap), _padded(s["x"], off, cap)
        return torch.bmm(d.transpose(1, 2).contiguous(), x).to(_plain(case["out"]))
    x = _padded(s["a"], off, cap)
    w = s["b"].float()
    if case["layout"] == "col":
        y = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)
    else:
        y = torch.bmm(x, w)
    # Back to rows of tokens: row r is row r - off[group] of its group.
    r = torch.arange(t, device=off.device)
    group = torch.searchsorted(off[1:].long(), r, right=True)
    z = y[group, r - off.long()[group]]
    if case["type"] != "bf16":
        z = z * (s["sa"][:, None] * s["sb"][group])
    z = z if s["bias"] is None else z + s["bias"].float()[group]
    return (_gelu(z) if case["gelu"] else z).to(_plain(case["out"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "quant":
        e = case["rows"] * case["k"]
        return {"bytes": 3 * e + 4 * case["rows"], "flops": 3 * e}
    n, k = case["n"], case["k"]
    size = 4 if case["out"] == "f32" else 2
    if op == "int8":
        m = case["m"]
        extra = (4 * m + 4 * n if case["zero"] else 0) + (2 * n if case["bias"] else 0)
        return {"bytes": m * k + n * k + 4 * (m + n) + extra + size * m * n, "flops": 2 * m * n * k}
    t, g, live = case["t"], case["g"], case["live"]
    if op == "wgrad":
        return {"bytes": 2 * t * (n + k) + size * g * n * k + 4 * (g + 1), "flops": 2 * t * n * k}
    wide = 2 if case["type"] == "bf16" else 1
    extra = (0 if wide == 2 else 4 * (t + live * n)) + (2 * live * n if case["bias"] else 0)
    return {"bytes": wide * (t * k + live * n * k) + size * t * n + 4 * (g + 1) + extra,
            "flops": 2 * t * n * k}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        top = s["x"].double().abs().max(dim=1).values
        # A code next to a border is decided by the FP32 quotient: no 64-bit value stands in its place.
        return {"q": None, "scale": torch.where(top == 0, 1.0, top / 127)}

    def last(z, bias):
        z = z if bias is None else z + bias.double()
        if case.get("gelu"):
            z = z * torch.special.ndtr(z)
        return z

    if op == "int8":
        zero = 0.0 if s["za"] is None else s["za"].double().unsqueeze(1)
        z = torch.mm(s["a"].double() - zero, s["b"].double().t())
        return last(z * s["sa"].double().unsqueeze(1) * s["sb"].double(), s["bias"])
    ends = s["off"].tolist()
    if op == "wgrad":
        c = torch.zeros(case["g"], case["n"], case["k"], device="cuda", dtype=torch.float64)
        for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
            c[g] = torch.mm(s["d"][lo:hi].double().t(), s["x"][lo:hi].double())
        return c
    c = torch.zeros(case["t"], case["n"], device="cuda", dtype=torch.float64)
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        w = s["b"][g].double()
        z = torch.mm(s["a"][lo:hi].double(), w.t() if case["layout"] == "col" else w)
        if case["type"] != "bf16":
            z = z * s["sa"][lo:hi].double().unsqueeze(1) * s["sb"][g].double()
        c[lo:hi] = last(z, None if s["bias"] is None else s["bias"][g])
    return c

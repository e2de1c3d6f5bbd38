"""Cases of the operators by which rows choose a weight of their own, for measuring them.

Three operators: routing of tokens to experts (and the gradient of its weights), the
way of rows to their experts and back (sort, copies, weighted sums and their gradients),
and a shared projection with a low-rank adapter per row. `run` makes the library's
calls where `own` is true, and computes the same with elementary torch operations where
it is false; `exact` has the values in 64 bits.
"""
import math

import numpy as np
import torch

own = False

# Widths (2048, 4096, 14336, 18432) are this repository's own projection, FFN and decode
# widths; numbers of experts, ranks and tokens are generic.
_CASES = [
    # One token of a decode step through a small router: latency alone.
    {"name": "route_token", "op": "route", "t": 1, "e": 64, "k": 6, "type": "bf16", "score": "softmax",
     "bias": False, "groups": 1, "kept": 1, "best": 1, "renorm": False, "scale": 1.0, "masked": 0.0, "grad": False},
    # A decode batch through a wide router whose experts are kept in balance by a bias, a few groups each.
    {"name": "route_batch", "op": "route", "t": 128, "e": 256, "k": 8, "type": "f32", "score": "sigmoid",
     "bias": True, "groups": 8, "kept": 4, "best": 2, "renorm": True, "scale": 2.5, "masked": 0.0, "grad": False},
    # The same router in a training step, with the gradient of its logits.
    {"name": "route_train", "op": "route", "t": 16384, "e": 256, "k": 8, "type": "f32", "score": "sigmoid",
     "bias": True, "groups": 8, "kept": 4, "best": 2, "renorm": True, "scale": 2.5, "masked": 0.0, "grad": True},
    # Odd numbers of tokens and experts, BF16 logits with equal values, experts masked out, weights that do not
    # sum to one: the gradient reaches every logit.
    {"name": "route_odd_train", "op": "route", "t": 5003, "e": 60, "k": 4, "type": "bf16", "score": "softmax",
     "bias": False, "groups": 1, "kept": 1, "best": 1, "renorm": False, "scale": 1.0, "masked": 0.1, "grad": True},
    # A decode batch on its way to the experts and back.
    {"name": "rows_decode", "op": "rows", "t": 32, "k": 8, "e": 256, "n": 4096, "out": "bf16", "none": 0.0,
     "grad": False},
    # The same of a training step, with every gradient.
    {"name": "rows_train", "op": "rows", "t": 8192, "k": 4, "e": 64, "n": 4096, "out": "bf16", "none": 0.0,
     "grad": True},
    # A width and numbers that are multiples of nothing; some slots have no expert.
    {"name": "rows_odd_train", "op": "rows", "t": 1001, "k": 3, "e": 9, "n": 4093, "out": "f32", "none": 0.1,
     "grad": True},
    # One token of one request.
    {"name": "lora_token", "op": "lora", "m": 1, "n": 4096, "k": 4096, "r": 16, "g": 8, "live": 1, "out": "bf16",
     "bias": False, "gelu": False, "none": 0.0},
    # A decode step of sixteen requests, an adapter each, on the widest projection.
    {"name": "lora_decode", "op": "lora", "m": 16, "n": 18432, "k": 4096, "r": 16, "g": 64, "live": 16, "out": "bf16",
     "bias": False, "gelu": False, "none": 0.0},
    # A larger decode batch on the FFN's second product: long rows, higher rank, some requests without an adapter.
    {"name": "lora_batch", "op": "lora", "m": 64, "n": 4096, "k": 14336, "r": 64, "g": 32, "live": 24, "out": "bf16",
     "bias": False, "gelu": False, "none": 0.1},
    # Prompts of a few requests at once, through the FFN's first product.
    {"name": "lora_prompts", "op": "lora", "m": 4096, "n": 14336, "k": 4096, "r": 16, "g": 8, "live": 6,
     "out": "bf16", "bias": True, "gelu": True, "none": 0.0},
    # No size a multiple of anything, FP32 results.
    {"name": "lora_odd", "op": "lora", "m": 777, "n": 4093, "k": 4099, "r": 20, "g": 16, "live": 9, "out": "f32",
     "bias": True, "gelu": False, "none": 0.1},
]

_MOST_FLOPS = 2.0 * 4096 * 14336 * 4096
_MOST_ROWS = 8192 * 4 * 4096
_MOST_LOGITS = 16384 * 256


def listed():
    return [dict(c) for c in _CASES]


def _spread(rng, lo, hi, multiple=1):
    """A size between lo and hi, spread over its logarithm; a multiple of `multiple` three times in four."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.75:
        v = v // multiple * multiple
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(("route", "rows", "lora"))
    if op == "route":
        while True:
            t, e = _spread(rng, 1, 16384), _spread(rng, 8, 512, 8)
            groups = rng.choice([d for d in (1, 1, 2, 4, 8, 16) if e % d == 0 and e // d >= 2])
            kept = rng.randint(max(1, groups // 2), groups)
            k = rng.randint(1, min(12, e // groups * kept))
            if t * e > _MOST_LOGITS:
                continue
            bias = rng.random() < 0.5
            return {"op": op, "t": t, "e": e, "k": k, "type": rng.choice(("f32", "bf16")),
                    "score": rng.choice(("softmax", "sigmoid")), "bias": bias, "groups": groups, "kept": kept,
                    "best": rng.choice((1, 2)) if bias else 1, "renorm": rng.random() < 0.5,
                    "scale": rng.choice((1.0, 2.5)), "masked": rng.choice((0.0, 0.0, 0.1)),
                    "grad": rng.random() < 0.6}
    if op == "rows":
        while True:
            c = {"op": op, "t": _spread(rng, 1, 16384), "k": rng.choice((1, 2, 3, 4, 6, 8)),
                 "e": _spread(rng, 8, 256, 8), "n": _spread(rng, 256, 14336, 64), "out": rng.choice(("bf16", "f32")),
                 "none": rng.choice((0.0, 0.0, 0.1)), "grad": rng.random() < 0.6}
            if c["t"] * c["k"] * c["n"] <= _MOST_ROWS:
                return c
    while True:
        m = _spread(rng, 1, 4096)
        g = _spread(rng, 1, 64)
        c = {"op": op, "m": m, "n": _spread(rng, 256, 18432, 64), "k": _spread(rng, 256, 14336, 64),
             "r": rng.choice((4, 8, 8, 16, 16, 16, 20, 32, 64)), "g": g, "live": rng.randint(1, min(g, m, 24)),
             "out": rng.choice(("bf16", "bf16", "f32")), "bias": rng.random() < 0.4, "gelu": rng.random() < 0.3,
             "none": rng.choice((0.0, 0.0, 0.1))}
        if 2.0 * m * c["n"] * c["k"] <= _MOST_FLOPS:
            return c


def _dtype(n):
    return torch.float32 if n == "f32" else torch.bfloat16


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, device="cuda", generator=gen, dtype=torch.float32).mul_(std).to(dtype)

    s = {"case": dict(case)}
    op = case["op"]
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        # Logits: some experts are asked for more than others.
        x = normal(t, e, std=1.5, dtype=torch.float32) + normal(e, std=0.5, dtype=torch.float32)
        if case["masked"]:
            x[torch.rand(t, e, device="cuda", generator=gen) < case["masked"]] = -math.inf
        s["x"] = x.to(_dtype(case["type"]))
        s["bias"] = normal(e, std=0.05, dtype=torch.float32) if case["bias"] else None
        s["expert"] = torch.empty(t, k, device="cuda", dtype=torch.int32)
        s["weight"] = torch.empty(t, k, device="cuda")
        if case["grad"]:
            s["dw"] = normal(t, k, dtype=torch.float32)
            s["dx"] = torch.empty_like(s["x"])
        return s
    if op == "rows":
        t, k, e, n = case["t"], case["k"], case["e"], case["n"]
        # k different experts for every token, some experts preferred.
        level = normal(t, e, dtype=torch.float32) + normal(e, std=0.5, dtype=torch.float32)
        expert = torch.sort(level, dim=1, descending=True).indices[:, :k].to(torch.int32)
        w = torch.rand(t, k, device="cuda", generator=gen) + 0.05
        w = w / w.sum(1, keepdim=True)
        if case["none"]:
            gone = torch.rand(t, k, device="cuda", generator=gen) < case["none"]
            expert = torch.where(gone, -1, expert)
            w = torch.where(gone, 0.0, w)
        s["expert"], s["weight"] = expert.contiguous(), w.contiguous()
        s["x"], s["y"] = normal(t, n), normal(t * k, n)
        i32 = lambda *shape: torch.empty(*shape, device="cuda", dtype=torch.int32)  # noqa: E731
        s["offsets"], s["position"], s["order"] = i32(e + 1), i32(t, k), i32(t * k)
        s["rows"] = torch.zeros(t * k, n, device="cuda", dtype=torch.bfloat16)
        s["c"] = torch.empty(t, n, device="cuda", dtype=_dtype(case["out"]))
        if case["grad"]:
            s["d"], s["drows"] = normal(t, n, dtype=_dtype(case["out"])), normal(t * k, n)
            s["dy"] = torch.zeros_like(s["y"])
            s["dweight"] = torch.empty(t, k, device="cuda")
            s["dx"] = torch.empty_like(s["x"])
        return s
    m, n, k, r, g = case["m"], case["n"], case["k"], case["r"], case["g"]
    s["a"] = normal(m, k)
    s["b"] = normal(n, k, std=0.02)
    s["down"] = normal(g, r, k, std=0.02)
    s["up"] = normal(g, n, r, std=0.05)
    s["scale"] = torch.rand(g, device="cuda", generator=gen) + 0.5
    # Rows of one request are neighbours and share its adapter; a decode batch has one row each.
    live = rng.permutation(g)[:case["live"]]
    ids = np.sort(np.concatenate([np.arange(case["live"]), rng.integers(0, case["live"], m - case["live"])]))
    ids = live[ids]
    if case["none"]:
        ids = np.where(rng.random(m) < case["none"], -1, ids)
    s["adapter"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    s["bias"] = normal(n, std=0.1) if case["bias"] else None
    s["c"] = torch.empty(m, n, device="cuda", dtype=_dtype(case["out"]))
    if own:
        import dense_gemm_09_amd as lib
        # A serving program allocates its workspace once.
        size = lib.lora_workspace_size(m, n, k, r)
        s["workspace"] = torch.empty(max(16, size), device="cuda", dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ the library's calls

def _run_own(s):
    import dense_gemm_09_amd as lib
    case = s["case"]
    op = case["op"]
    kind = lambda name: lib.OUT_F32 if name == "f32" else lib.OUT_BF16  # noqa: E731
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        score = lib.SCORE_SOFTMAX if case["score"] == "softmax" else lib.SCORE_SIGMOID
        lib.route(t, e, k, s["x"], e, kind(case["type"]), score, s["bias"], case["groups"], case["kept"],
                  case["best"], case["renorm"], case["scale"], s["expert"], s["weight"])
        out = {"expert": s["expert"], "weight": s["weight"]}
        if case["grad"]:
            lib.route_grad(t, e, k, s["x"], e, kind(case["type"]), score, case["renorm"], case["scale"], s["expert"],
                           s["dw"], s["dx"], e)
            out["dx"] = s["dx"]
        return out
    if op == "rows":
        t, k, e, n = case["t"], case["k"], case["e"], case["n"]
        lib.route_order(t * k, e, s["expert"], s["offsets"], s["position"], s["order"])
        lib.dispatch_rows(t, k, t * k, n, s["x"], n, 2, s["position"], s["rows"], n)
        lib.combine_rows(t, k, t * k, n, s["y"], n, lib.OUT_BF16, s["position"], s["weight"], 0.0, s["c"], n,
                         kind(case["out"]))
        out = {name: s[name] for name in ("offsets", "position", "order", "rows", "c")}
        if case["grad"]:
            lib.combine_rows_grad(t, k, t * k, n, s["d"], n, kind(case["out"]), s["y"], n, lib.OUT_BF16,
                                  s["position"], s["weight"], s["dy"], n, s["dweight"])
            lib.combine_rows(t, k, t * k, n, s["drows"], n, lib.OUT_BF16, s["position"], None, 0.0, s["dx"], n,
                             lib.OUT_BF16)
            out.update({name: s[name] for name in ("dy", "dweight", "dx")})
        return out
    m, n, k, r, g = case["m"], case["n"], case["k"], case["r"], case["g"]
    lib.gemm_lora_bf16(m, n, k, g, r, 1.0, s["a"], k, s["b"], k, s["adapter"], s["down"], k, r * k, s["up"], r, n * r,
                       s["scale"], 0.0, s["c"], n, kind(case["out"]), s["bias"],
                       lib.ACT_GELU_ERF if case["gelu"] else lib.ACT_NONE, s["workspace"])
    return s["c"]


# ------------------------------------------------------------------ the plain forms

def _gelu(z):
    return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))


def _route_plain(s):
    case = s["case"]
    t, e, k, groups = case["t"], case["e"], case["k"], case["groups"]
    # 64 bits: experts next to a border are told apart by the last bits of their scores.
    x = s["x"].double()
    out_there = x > -math.inf
    if case["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
        log_sum = torch.log(p.sum(1, keepdim=True))
        score = p / p.sum(1, keepdim=True)
        log_score = x - torch.where(top > -math.inf, top, 0.0) - log_sum
    else:
        score = 1 / (1 + torch.exp(-x))
        log_score = torch.clamp(x, max=0.0) - torch.log1p(torch.exp(-x.abs()))
    # Without a bias the order is that of the logits.
    c = x if s["bias"] is None else score + s["bias"].double()
    c = torch.where(out_there, c, -math.inf)
    if groups > 1:
        best = torch.sort(c.view(t, groups, e // groups), dim=2, descending=True).values[..., :case["best"]]
        first = best[..., 0] > -math.inf
        total = torch.where(first, torch.where(best > -math.inf, best, 0.0).sum(2), -math.inf)
        rank = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = (rank[:, :, None] == torch.arange(groups, device=x.device)).any(1)
        c = torch.where(keep.repeat_interleave(e // groups, dim=1), c, -math.inf)
    c, ids = torch.sort(c, dim=1, descending=True, stable=True)
    chosen = c[:, :k] > -math.inf
    ids = ids[:, :k]
    w = torch.where(chosen, score.gather(1, ids), 0.0)
    # Shares of the chosen from the scores' logarithms: scores that are all tiny still have them.
    logs = torch.where(chosen, log_score.gather(1, ids), -math.inf)
    top = logs.amax(1, keepdim=True)
    share = torch.exp(logs - torch.where(top > -math.inf, top, 0.0))
    total = share.sum(1, keepdim=True)
    share = share / torch.where(total > 0, total, 1.0)
    weight = case["scale"] * (share if case["renorm"] else w)
    out = {"expert": torch.where(chosen, ids, -1).to(torch.int32), "weight": weight.float()}
    if not case["grad"]:
        return out
    dw = torch.where(chosen, s["dw"].double(), 0.0) * case["scale"]
    if case["renorm"]:
        d = share * (dw - (dw * share).sum(1, keepdim=True))
        d = d if case["score"] == "softmax" else d * (1 - w)
        dx = torch.zeros_like(x).scatter_add_(1, ids, torch.where(chosen, d, 0.0))
    elif case["score"] == "softmax":
        dx = torch.zeros_like(x).scatter_add_(1, ids, w * dw) - torch.where(out_there, score, 0.0) * (w * dw).sum(
            1, keepdim=True)
    else:
        dx = torch.zeros_like(x).scatter_add_(1, ids, dw * w * (1 - w))
    out["dx"] = dx.to(s["x"].dtype)
    return out


def _rows_plain(s):
    case = s["case"]
    t, k, e, n = case["t"], case["k"], case["e"], case["n"]
    expert = s["expert"].view(-1)
    key = torch.where(expert < 0, e, expert)
    in_order, order = torch.sort(key, stable=True)
    offsets = (key[None, :] < torch.arange(e + 1, device=key.device)[:, None]).sum(1)
    position = torch.empty_like(order)
    position[order] = torch.arange(t * k, device=key.device)
    there = expert >= 0
    out = {"offsets": offsets.to(torch.int32),
           "position": torch.where(there, position, -1).view(t, k).to(torch.int32),
           "order": torch.where(in_order < e, order, -1).to(torch.int32)}
    live = (in_order < e)[:, None]
    out["rows"] = torch.where(live, s["x"][order // k], 0)
    there = there.view(t, k, 1)
    back = s["y"].float()[position.view(t, k)]
    w = s["weight"][..., None]
    out["c"] = torch.where(there, w * back, 0.0).sum(1).to(_dtype(case["out"]))
    if case["grad"]:
        d = s["d"].float()
        dy = torch.where(there, w * d[:, None, :], 0.0).view(t * k, n)
        out["dy"] = torch.where(live, dy[order], 0.0).to(torch.bfloat16)
        out["dweight"] = torch.where(there[..., 0], (back * d[:, None, :]).sum(2), 0.0)
        out["dx"] = torch.where(there, s["drows"].float()[position.view(t, k)], 0.0).sum(1).to(torch.bfloat16)
    return out


def _lora_plain(s):
    case = s["case"]
    g, r, n = case["g"], case["r"], case["n"]
    a = s["a"].float()
    # Every row against every adapter's first factor, then its own alone.
    h = (a @ s["down"].float().view(g * r, -1).t()).view(-1, g, r)
    mine = s["adapter"][:, None] == torch.arange(g, device=a.device)
    h = torch.where(mine[..., None], h * s["scale"][:, None], 0.0).view(-1, g * r)
    z = a @ s["b"].float().t() + h @ s["up"].float().permute(0, 2, 1).reshape(g * r, n)
    z = z if s["bias"] is None else z + s["bias"].float()
    return (_gelu(z) if case["gelu"] else z).to(_dtype(case["out"]))


def run(state):
    if own:
        return _run_own(state)
    return {"route": _route_plain, "rows": _rows_plain, "lora": _lora_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["t"], case["e"], case["k"]
        size = 4 if case["type"] == "f32" else 2
        total = size * t * e + 8 * t * k + (4 * e if case["bias"] else 0)
        if case["grad"]:
            # The logits once for both passes; the gradient is written whole.
            total += size * t * e + 4 * t * k
        return {"bytes": total, "flops": (10 if case["grad"] else 6) * t * e}
    if op == "rows":
        t, k, e, n = case["t"], case["k"], case["e"], case["n"]
        size = 4 if case["out"] == "f32" else 2
        slots = int(round(t * k * (1 - case["none"])))
        total = 4 * t * k + 8 * t * k + 4 * (e + 1) + 4 * t * k
        total += 2 * t * n + 2 * slots * n + 2 * slots * n + size * t * n
        flops = 2 * slots * n
        if case["grad"]:
            total += size * t * n + 2 * slots * n + 4 * t * k + 2 * slots * n + 2 * t * n
            flops += 3 * slots * n + slots * n
        return {"bytes": total, "flops": flops}
    m, n, k, r, live = case["m"], case["n"], case["k"], case["r"], case["live"]
    size = 4 if case["out"] == "f32" else 2
    total = 2 * (m * k + n * k + live * r * (n + k)) + 4 * m + 4 * live + size * m * n + (2 * n if case["bias"] else 0)
    return {"bytes": total, "flops": 2 * m * n * k + 2 * m * r * (n + k)}


# ------------------------------------------------------------------ the definition in 64 bits

def _route_exact(s):
    case = s["case"]
    t, e, k = case["t"], case["e"], case["k"]
    x = s["x"].double().requires_grad_(case["grad"])
    dead = (x == -math.inf).detach()
    empty = dead.all(1, keepdim=True)
    safe = torch.where(empty, torch.zeros_like(x), x)
    if case["score"] == "softmax":
        logs = torch.log_softmax(safe, 1)
    else:
        logs = torch.nn.functional.logsigmoid(torch.where(dead, torch.zeros_like(x), x))
    with torch.no_grad():
        c = x.detach().clone() if s["bias"] is None else torch.exp(logs) + s["bias"].double()
        c[dead] = -math.inf
        per = e // case["groups"]
        number = torch.arange(e, device=x.device)

        def take(v):
            """The largest of each row, the first where several are; its index and whether there is one."""
            top = v.max(1, keepdim=True).values
            at = torch.where(v == top, torch.arange(v.shape[1], device=v.device), v.shape[1]).min(1).values
            return at, top[:, 0] > -math.inf

        if case["groups"] > 1:
            parts = []
            for i in range(case["groups"]):
                part = c[:, i * per:(i + 1) * per].clone()
                best = torch.full((t,), -math.inf, device=x.device, dtype=torch.float64)
                for j in range(case["best"]):
                    at, found = take(part)
                    v = part.gather(1, at[:, None])[:, 0]
                    best = torch.where(found, v if j == 0 else best + v, best)
                    part.scatter_(1, at[:, None], -math.inf)
                parts.append(best)
            score = torch.stack(parts, 1)
            kept = torch.zeros(t, case["groups"], device=x.device, dtype=torch.bool)
            for _ in range(case["kept"]):
                at, _found = take(score)
                kept.scatter_(1, at[:, None], True)
                score.scatter_(1, at[:, None], -math.inf)
            c[~kept[:, number // per]] = -math.inf
        ids = []
        for _ in range(k):
            at, found = take(c)
            ids.append(torch.where(found, at, -1))
            c.scatter_(1, at[:, None], -math.inf)
        ids = torch.stack(ids, 1)
    there = ids >= 0
    picked = logs.gather(1, ids.clamp(min=0))
    if case["renorm"]:
        picked = torch.where(there, picked, -math.inf)
        none = ~there.any(1, keepdim=True)
        weight = torch.softmax(torch.where(none, torch.zeros_like(picked), picked), 1)
    else:
        weight = torch.exp(picked)
    weight = torch.where(there, weight, 0.0) * case["scale"]
    out = {"expert": ids.to(torch.int32), "weight": weight.detach()}
    if case["grad"]:
        (weight * s["dw"].double()).sum().backward()
        out["dx"] = torch.nan_to_num(x.grad, nan=0.0)
    return out


def _rows_exact(s):
    case = s["case"]
    t, k, e, n = case["t"], case["k"], case["e"], case["n"]
    expert = s["expert"].reshape(-1).cpu().numpy()
    slots = [np.flatnonzero(expert == g) for g in range(e)]
    order = np.concatenate(slots)
    live = len(order)
    position = np.full(t * k, -1, np.int32)
    position[order] = np.arange(live)
    whole = np.full(t * k, -1, np.int32)
    whole[:live] = order
    dev = lambda v: torch.from_numpy(np.ascontiguousarray(v)).cuda()  # noqa: E731
    out = {"offsets": dev(np.concatenate([[0], np.cumsum([len(v) for v in slots])]).astype(np.int32)),
           "position": dev(position.reshape(t, k)), "order": dev(whole)}
    token, slot = dev(order // k).long(), dev(order).long()
    rows = torch.zeros(t * k, n, device="cuda", dtype=torch.float64)
    rows[:live] = s["x"].double()[token]
    w = s["weight"].double().view(-1)[slot]
    y = s["y"][:live].double()
    out["rows"] = rows
    out["c"] = torch.zeros(t, n, device="cuda", dtype=torch.float64).index_add_(0, token, y * w[:, None])
    if case["grad"]:
        d = s["d"].double()[token]
        dy = torch.zeros_like(rows)
        dy[:live] = d * w[:, None]
        dw = torch.zeros(t * k, device="cuda", dtype=torch.float64)
        dw[slot] = (d * y).sum(1)
        out["dy"], out["dweight"] = dy, dw.view(t, k)
        out["dx"] = torch.zeros(t, n, device="cuda", dtype=torch.float64).index_add_(
            0, token, s["drows"][:live].double())
    return out


def _lora_exact(s):
    case = s["case"]
    a = s["a"].double()
    z = torch.mm(a, s["b"].double().t())
    adapter = s["adapter"].cpu().numpy()
    for i in sorted(set(adapter[adapter >= 0].tolist())):
        rows = torch.from_numpy(np.flatnonzero(adapter == i)).cuda()
        h = torch.mm(a[rows], s["down"][i].double().t()) * s["scale"][i].double()
        z[rows] += torch.mm(h, s["up"][i].double().t())
    if s["bias"] is not None:
        z += s["bias"].double()
    return z * torch.special.ndtr(z) if case["gelu"] else z


def exact(case, seed):
    return {"route": _route_exact, "rows": _rows_exact, "lora": _lora_exact}[case["op"]](prepare(case, seed))

"""The operators of rows that choose their weights, as workloads to be timed.

Rows of one batch that go through different weights: tokens routed to experts and requests with adapters of
their own.  Five kinds of pass, each a call a serving program makes:

  route    router logits -> expert ids and weights, and the row groups that the experts' products read
           (``route`` + ``group_rows``)
  gated    the experts' gate and up products with the activation, from packed int8 rows
           (``linear_gated_grouped``)
  down     the experts' down product, back in the order of the (row, choice) pairs (``linear_grouped``)
  combine  the weighted sum of every row's expert outputs (``combine_rows``)
  lora     the low-rank correction of a batch whose rows use different adapters (``lora_add_grouped``)

``run`` computes a pass in elementary torch operations, or with the package's operators where ``own`` is
true.  ``exact`` states the same results from the definitions in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------------

def _route(name, M, E, k, score, dt="f32", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0, masked=0.0):
    return {"name": name, "op": "route", "M": M, "E": E, "k": k, "score": score, "dt": dt, "bias": bias,
            "groups": groups, "top_groups": top_groups, "renorm": renorm, "scale": scale, "masked": masked}


def _gated(name, M, E, k, K, N, G, act, bias=False, dt="bf16"):
    return {"name": name, "op": "gated", "M": M, "E": E, "k": k, "K": K, "N": N, "G": G, "act": act, "bias": bias,
            "dt": dt}


def _down(name, M, E, k, K, N, G, bias=False, dt="bf16"):
    return {"name": name, "op": "down", "M": M, "E": E, "k": k, "K": K, "N": N, "G": G, "bias": bias, "dt": dt}


def _combine(name, M, E, k, N, dt="bf16", unused=0.0):
    return {"name": name, "op": "combine", "M": M, "E": E, "k": k, "N": N, "dt": dt, "unused": unused}


def _lora(name, M, E, K, N, r, dt="bf16", unused=0.0, runs=1):
    return {"name": name, "op": "lora", "M": M, "E": E, "K": K, "N": N, "r": r, "dt": dt, "unused": unused,
            "runs": runs}


def listed():
    return [
        # one token of a served stream: the router's latency
        _route("route_one_token", 1, 128, 8, "softmax"),
        # a long prompt through a router with a balance bias and groups of experts
        _route("route_prompt_grouped", 8192, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, scale=2.5),
        # one token: eight small experts are read whole
        _gated("gated_one_token", 1, 128, 8, 2048, 768, 256, "silu"),
        # a decode batch over few wide experts (the width of the decode workload's gated layer)
        _gated("gated_decode_batch", 16, 8, 2, 1152, 6912, 64, "gelu_tanh"),
        # a mixed batch with ragged sizes: few rows per expert, all experts read
        _gated("gated_ragged_batch", 257, 64, 6, 1408, 1000, 64, "silu", bias=True),
        # a long prompt: the products are bound by the matrix cores
        _gated("gated_prompt", 8192, 128, 8, 2048, 768, 256, "silu"),
        # the decode batch's way back
        _down("down_decode_batch", 16, 8, 2, 6912, 1152, 64),
        # the long prompt's way back
        _down("down_prompt", 8192, 128, 8, 768, 2048, 256),
        # a decode batch, some of whose choices were dropped
        _combine("combine_decode_batch", 33, 8, 2, 1152, "f32", unused=0.1),
        # the long prompt's rows, each the sum of eight
        _combine("combine_prompt", 8192, 128, 8, 2048),
        # decode: many requests, each with its own small adapter
        _lora("lora_decode_batch", 48, 64, 4096, 4096, 16, unused=0.1),
        # prompts of several requests side by side, ragged, some without an adapter
        _lora("lora_prompts", 4099, 24, 2048, 6144, 64, unused=0.1, runs=150),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "gated", "gated", "down", "combine", "lora", "lora"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, 8, 384 // groups)
        k = rng.randint(1, min(8, E // groups))
        return _route("", _log_int(rng, 1, 8192), E, k, rng.choice(["softmax", "sigmoid"]),
                      rng.choice(["f32", "bf16"]), rng.random() < 0.5, groups, rng.randint(1, groups),
                      rng.random() < 0.7, rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.3]))
    if op in ("gated", "down"):
        G = rng.choice([16, 64, 256])
        lo = max(1, 256 // G)
        K = G * _log_int(rng, lo, 4096 // G)
        N = _log_int(rng, 64, 3000)
        E = _log_int(rng, 2, 128)
        k = rng.randint(1, min(8, E))
        M = _log_int(rng, 1, 4096)
        # no more than the long prompt's products, and weights that are quick to make
        while M * k * N * K > 8192 * 8 * 2048 * 768:
            M = (M + 1) // 2
        while E * N * K > 128 * 2048 * 768:
            E = (E + 1) // 2
        k = min(k, E)
        dt = rng.choice(["bf16", "bf16", "f32"])
        if op == "gated":
            return _gated("", M, E, k, K, N, G, rng.choice(["silu", "gelu_tanh", "gelu_erf"]), rng.random() < 0.3, dt)
        return _down("", M, E, k, K, N, G, rng.random() < 0.3, dt)
    if op == "combine":
        k = rng.randint(1, 8)
        N = _log_int(rng, 64, 4096)
        M = _log_int(rng, 1, 8192)
        while M * k * N > 8192 * 8 * 2048:
            M = (M + 1) // 2
        return _combine("", M, 128, k, N, rng.choice(["bf16", "f32"]), rng.choice([0.0, 0.2]))
    K, N = 16 * _log_int(rng, 16, 384), _log_int(rng, 64, 6144)
    M = _log_int(rng, 1, 4096)
    return _lora("", M, _log_int(rng, 1, 64), K, N, 16 * rng.choice([1, 1, 2, 3, 4, 8]), rng.choice(["bf16", "f32"]),
                 rng.choice([0.0, 0.2]), rng.choice([1, 40]))


# ----------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------

def _codes(shape, g):
    """Codes of rotated, quantised rows: near normal, the largest of a row near 127."""
    x = torch.empty(shape, device=DEV, dtype=torch.bfloat16).normal_(0.0, 36.0, generator=g)
    return x.round_().clamp_(-127, 127).to(torch.int8)


def _choices(M, E, k, g):
    """Expert ids [M, k] of a router whose experts are not equally popular."""
    logits = torch.randn(M, E, device=DEV, generator=g) + 0.7 * torch.randn(E, device=DEV, generator=g)
    return logits.topk(k, dim=1).indices.to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    M, E, op = case["M"], case["E"], case["op"]
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    uni = lambda *s: torch.rand(*s, device=DEV, generator=g)
    t = {}
    if op == "route":
        x = 1.5 * rnd(M, E)
        if case["masked"]:
            x = x.masked_fill(uni(M, E) < case["masked"], float("-inf"))
            x[:: 17] = x[:: 17].masked_fill(uni(*x[:: 17].shape) < 0.98, float("-inf"))
        t["logits"] = x.to(_DT[case["dt"]])
        t["bias"] = 0.1 * rnd(E) if case["bias"] else None
        return t
    if op in ("gated", "down"):
        k, K, N = case["k"], case["K"], case["N"]
        ids = _choices(M, E, k, g)
        t["ids"] = ids
        rows = M if op == "gated" else M * k
        t["x"], t["sx"] = _codes((rows, K), g), (0.5 + uni(rows)) * (3.0 / 127)
        for w in (("wg", "wu") if op == "gated" else ("w",)):
            t[w] = _codes((E * N, K), g)
            t["s_" + w] = (0.5 + uni(E * N)) * (0.08 / 127)
            t["b_" + w] = 0.1 * rnd(E * N) if case["bias"] else None
        return t
    if op == "combine":
        k, N = case["k"], case["N"]
        ids = torch.randint(0, E, (M, k), device=DEV, generator=g, dtype=torch.int32)
        ids = ids.masked_fill(uni(M, k) < case["unused"], -1)
        t["ids"] = ids
        t["y"] = rnd(M * k, N).to(_DT[case["dt"]])
        t["weights"] = uni(M, k)
        return t
    K, N, r = case["K"], case["N"], case["r"]
    # prompts are runs of rows of one request; decode has one row for each
    n = (M + case["runs"] - 1) // case["runs"]
    req = torch.randint(0, E, (n,), device=DEV, generator=g, dtype=torch.int32)
    req = req.masked_fill(uni(n) < case["unused"], -1)
    t["ids"] = req.repeat_interleave(case["runs"])[:M].contiguous()
    t["x"] = rnd(M, K).to(torch.bfloat16)
    t["a"] = (rnd(E, r, K) / math.sqrt(K)).to(torch.bfloat16)
    t["b"] = (rnd(E, N, r) / math.sqrt(r)).to(torch.bfloat16)
    t["scales"] = 0.25 + uni(E)
    t["y"] = rnd(M, N).to(_DT[case["dt"]])
    return t


def _plan(ids, E):
    """Where every group's pairs are, for the plain form: order and sizes."""
    flat = ids.reshape(-1).to(torch.int64)
    flat = torch.where((flat < 0) | (flat >= E), torch.full_like(flat, E), flat)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)
    return order, counts


def prepare(case, seed):
    s = dict(case)
    s.update(_inputs(case, seed))
    op, E = case["op"], case["E"]
    if op in ("gated", "down", "lora"):
        order, counts = _plan(s["ids"], E)
        s["order"], s["counts"] = order, counts.tolist()
    if own:
        import w8a8_int8_linear_amd as cr

        s["cr"] = cr
        if op in ("gated", "down"):
            G = case["G"]
            s["px"] = cr.Packed(s["x"], s["sx"], G)
            for w in (("wg", "wu") if op == "gated" else ("w",)):
                s["p_" + w] = cr.Packed(s[w], s["s_" + w], G)
        if op in ("gated", "down", "lora"):
            s["groups"] = cr.group_rows(s["ids"], E)
    return s


# ----------------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------------

def _activation(x, act):
    if act == "silu":
        return x / (1 + torch.exp(-x))
    if act == "gelu_tanh":
        return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))
    return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))


def _spans(counts, E):
    p = 0
    for e in range(E):
        if counts[e]:
            yield e, p, p + counts[e]
        p += counts[e]


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    cr, op, E = s["cr"], s["op"], s["E"]
    if op == "route":
        ids, weights = cr.route(s["logits"], s["k"], score=s["score"], bias=s["bias"], groups=s["groups"],
                                top_groups=s["top_groups"], renormalise=s["renorm"], scale=s["scale"])
        g = cr.group_rows(ids, E)
        return ids, weights, g.order, g.offsets
    if op == "gated":
        return cr.linear_gated_grouped(s["px"], s["p_wg"], s["p_wu"], s["groups"], b_gate=s["b_wg"], b_up=s["b_wu"],
                                       act=s["act"], source=cr.BY_ROW, dest=cr.SORTED, out_dtype=_DT[s["dt"]])
    if op == "down":
        return cr.linear_grouped(s["px"], s["p_w"], s["groups"], bias=s["b_w"], source=cr.SORTED, dest=cr.BY_PAIR,
                                 out_dtype=_DT[s["dt"]])
    if op == "combine":
        return cr.combine_rows(s["y"], s["weights"], s["ids"], E)
    return cr.lora_add_grouped(s["x"], s["a"], s["b"], s["scales"], s["y"], s["groups"], out=torch.empty_like(s["y"]))


def _run_plain(s):
    op, E = s["op"], s["E"]
    if op == "route":
        # the choice falls between values that may lie closer than 32 bits resolve
        return _route_rows(s, s["logits"].double())
    if op == "combine":
        M, k, N = s["M"], s["k"], s["N"]
        y = s["y"].float().reshape(M, k, N)
        used = (s["ids"] >= 0) & (s["ids"] < E)
        y = torch.where(used[..., None], y, torch.zeros_like(y))
        return (y * s["weights"][..., None]).sum(1).to(s["y"].dtype)
    order, counts = s["order"], s["counts"]
    if op == "lora":
        out = s["y"].float()
        for e, p0, p1 in _spans(counts, E):
            rows = order[p0:p1]
            t = s["x"][rows].float() @ s["a"][e].float().T
            out[rows] += s["scales"][e] * (t @ s["b"][e].float().T)
        return out.to(s["y"].dtype)
    N, dt = s["N"], _DT[s["dt"]]
    out = torch.empty(s["M"] * s["k"], N, device=DEV, dtype=dt)

    def product(x, sx, w, e):
        rows = slice(e * N, (e + 1) * N)
        y = (x @ s[w][rows].float().T) * (sx[:, None] * s["s_" + w][rows])
        return y if s["b_" + w] is None else y + s["b_" + w][rows]

    for e, p0, p1 in _spans(counts, E):
        if op == "gated":
            src = order[p0:p1] // s["k"]
            x, sx = s["x"][src].float(), s["sx"][src]
            out[p0:p1] = (_activation(product(x, sx, "wg", e), s["act"]) * product(x, sx, "wu", e)).to(dt)
        else:
            out[order[p0:p1]] = product(s["x"][p0:p1].float(), s["sx"][p0:p1], "w", e).to(dt)
    return out


def _route_rows(s, x):
    """Scores, choice, weights and row groups from 64-bit logits."""
    E, k = s["E"], s["k"]
    low = float("-inf")
    if s["score"] == "softmax":
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    c = p if s["bias"] is None else p + s["bias"]
    c = c.masked_fill((x == low) | torch.isnan(p), low)
    if s["groups"] > 1:
        per = E // s["groups"]
        best = torch.sort(c.reshape(-1, s["groups"], per), dim=2, descending=True).values[..., :2]
        first = best[..., 0]
        value = first + torch.where(best[..., -1] == low, torch.zeros_like(first), best[..., -1]) if per > 1 else first
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        c = c.masked_fill(~keep.repeat_interleave(per, 1), low)
    v, ids = torch.sort(c, dim=1, descending=True, stable=True)
    v, ids = v[:, :k], ids[:, :k]
    gone = v == low
    w = p.gather(1, ids).masked_fill(gone, 0.0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    ids = ids.masked_fill(gone, -1).to(torch.int32)
    order, counts = _plan(ids, E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = counts[:E].cumsum(0)
    return ids, (w * s["scale"]).float(), order.to(torch.int32), offsets


# ----------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------------------------------

def exact(case, seed):
    t = _inputs(case, seed)
    op, M, E = case["op"], case["M"], case["E"]
    if op == "route":
        k = case["k"]
        x = t["logits"].double().cpu()
        open_ = x > float("-inf")
        if case["score"] == "softmax":
            p = torch.softmax(x.masked_fill(~open_, -1e300), dim=1) * open_
        else:
            p = torch.sigmoid(x) * open_
        c = p if t["bias"] is None else p + t["bias"].double().cpu()
        ids = torch.full((M, k), -1, dtype=torch.int64)
        weights = torch.zeros(M, k, dtype=torch.float64)
        per = E // case["groups"]
        # rows one at a time, from the definition
        for m, (cm, om) in enumerate(zip(c.tolist(), open_.tolist())):
            cand = [i for i in range(E) if om[i]]
            if case["groups"] > 1:
                value = {}
                for gi in range(case["groups"]):
                    vals = sorted((cm[i] for i in range(gi * per, (gi + 1) * per) if om[i]), reverse=True)
                    if vals:
                        value[gi] = sum(vals[:2])
                kept = set(sorted(value, key=lambda gi: (-value[gi], gi))[:case["top_groups"]])
                cand = [i for i in cand if i // per in kept]
            for j, i in enumerate(sorted(cand, key=lambda i: (-cm[i], i))[:k]):
                ids[m, j] = i
                weights[m, j] = p[m, i]
        if case["renorm"]:
            weights /= weights.sum(1, keepdim=True).clamp_min(1e-300)
        weights *= case["scale"]
        flat = ids.reshape(-1)
        key = torch.where(flat < 0, torch.full_like(flat, E), flat)
        order = torch.argsort(key * key.numel() + torch.arange(key.numel()))
        offsets = torch.tensor([int((key < e).sum()) for e in range(E + 1)])
        return (ids.int().to(DEV), weights.to(DEV), order.int().to(DEV), offsets.int().to(DEV))
    if op == "combine":
        ids = t["ids"].reshape(-1)
        out = torch.zeros(M, case["N"], dtype=torch.float64, device=DEV)
        w = (t["weights"].double().reshape(-1) * ((ids >= 0) & (ids < E))).reshape(M, case["k"])
        y = t["y"].reshape(M, case["k"], case["N"])
        for j in range(case["k"]):
            out += w[:, j:j + 1] * y[:, j].double()
        return out
    if op == "lora":
        out = t["y"].double()
        for e in range(E):
            rows = (t["ids"] == e).nonzero().reshape(-1)
            if rows.numel():
                low = torch.matmul(t["x"][rows].double(), t["a"][e].double().t().contiguous())
                out[rows] += t["scales"][e].double() * torch.matmul(low, t["b"][e].double().t().contiguous())
        return out
    k, K, N = case["k"], case["K"], case["N"]
    flat = t["ids"].reshape(-1)
    out = torch.empty(M * k, N, dtype=torch.float64, device=DEV)

    def affine(x, sx, w, e):
        y = torch.matmul(x, t[w].view(E, N, K)[e].double().t().contiguous())
        y = y * sx[:, None] * t["s_" + w].view(E, N)[e].double()
        return y if t["b_" + w] is None else y + t["b_" + w].view(E, N)[e].double()

    at = 0
    for e in range(E):
        pairs = (flat == e).nonzero().reshape(-1)
        n = pairs.numel()
        if not n:
            continue
        if op == "gated":
            x, sx = t["x"][pairs // k].double(), t["sx"][pairs // k].double()
            z = affine(x, sx, "wg", e)
            if case["act"] == "silu":
                z = z * torch.sigmoid(z)
            elif case["act"] == "gelu_tanh":
                z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
            else:
                z = z * 0.5 * torch.erfc(-z / math.sqrt(2.0))
            out[at:at + n] = z * affine(x, sx, "wu", e)
        else:
            out[pairs] = affine(t["x"][at:at + n].double(), t["sx"][at:at + n].double(), "w", e)
        at += n
    return out


# ----------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ----------------------------------------------------------------------------------------------------

def _used(M, E, k):
    """Expected number of different groups that M rows of k choices use."""
    return E * (1 - (1 - k / E) ** M)


def work(case):
    op, M, E = case["op"], case["M"], case["E"]
    size = {"f32": 4, "bf16": 2}[case["dt"]]
    if op == "route":
        k = case["k"]
        return {"bytes": M * E * size + M * k * 12 + 4 * (E + 1), "flops": 8 * M * E}
    if op == "combine":
        return {"bytes": (M * case["k"] + M) * case["N"] * size, "flops": 2 * M * case["k"] * case["N"]}
    if op == "lora":
        K, N, r = case["K"], case["N"], case["r"]
        rows = M * (1 - case["unused"])
        used = _used(rows / case["runs"], E, 1)
        return {"bytes": M * K * 2 + 2 * M * N * size + used * r * (K + N) * 2 + 4 * M,
                "flops": 2 * rows * r * (K + N)}
    k, K, N = case["k"], case["K"], case["N"]
    weights = 2 if op == "gated" else 1
    rows = M if op == "gated" else M * k
    return {"bytes": rows * (K + 4) + weights * _used(M, E, k) * N * (K + 4) + M * k * N * size + 4 * M * k,
            "flops": 2 * weights * M * k * N * K}

"""What is measured of the operators that surround the FP4 linear in 16 (or
32) bits: the normalization in front of it and its gradient, the low-rank
adapters of many requests beside it, and the mixture-of-experts token order
around the grouped linear (tokens sorted by expert, and back with weights, and
its gradient).

listed() gives the cases, draw() more of the same ranges; prepare() makes the
inputs on the GPU from a seed, run() is one pass: with own = True through the
public calls of sparsity_gemm_b200, else in elementary torch operations in 32
bits rounded once at the end. exact() gives a pass's results in 64 bits, and
work() the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # the norm in front of the attention projections while decoding: 16
        # sequences, one token each, hidden 4096
        {"name": "norm_decode", "op": "norm", "rows": 16, "k": 4096, "dtype": "fp16", "kind": "rms", "affine": True,
         "stats": False},
        # the same norm over a prompt of 8192 tokens, statistics kept for a
        # backward pass
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "k": 4096, "dtype": "fp16", "kind": "layer",
         "affine": True, "stats": True},
        # a training step's backward pass of that norm
        {"name": "norm_grad_train", "op": "norm_grad", "rows": 8192, "k": 4096, "dtype": "bf16", "kind": "layer",
         "affine": True},
        # an odd number of tokens through an RMSNorm of hidden 3584
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 1021, "k": 3584, "dtype": "fp16", "kind": "rms",
         "affine": True},
        # one token of one request through the up projection's adapter
        {"name": "adapters_one_token", "op": "adapters", "rows": 1, "requests": 1, "k": 4096, "n": 14336, "rank": 64,
         "adapters": 1, "dtype": "bf16"},
        # 64 decoding requests over 32 adapters beside the q projection
        {"name": "adapters_decode", "op": "adapters", "rows": 64, "requests": 64, "k": 4096, "n": 4096, "rank": 16,
         "adapters": 32, "dtype": "fp16"},
        # a prompt batch of 16 requests over 8 adapters, same projection
        {"name": "adapters_prompt", "op": "adapters", "rows": 8192, "requests": 16, "k": 4096, "n": 4096, "rank": 16,
         "adapters": 8, "dtype": "fp16"},
        # ragged prompts of many requests beside the down projection, a
        # larger rank
        {"name": "adapters_ragged", "op": "adapters", "rows": 4099, "requests": 75, "k": 14336, "n": 4096, "rank": 64,
         "adapters": 64, "dtype": "bf16"},
        # one decoding step of 16 sequences into 128 experts, top 8
        {"name": "dispatch_decode", "op": "dispatch", "tokens": 16, "padded": 0, "k": 2048, "experts": 128, "top_k": 8,
         "dtype": "fp16"},
        # a prompt batch of 4096 tokens (the last 100 are padding)
        {"name": "dispatch_prompt", "op": "dispatch", "tokens": 4096, "padded": 100, "k": 2048, "experts": 128,
         "top_k": 8, "dtype": "fp16"},
        # the experts' results of that batch back into the residual stream
        {"name": "combine_prompt", "op": "combine", "tokens": 4096, "padded": 100, "k": 2048, "experts": 128,
         "top_k": 8, "dtype": "fp16", "residual": True},
        # the gradient of the way back in a training step
        {"name": "combine_grad_train", "op": "combine_grad", "tokens": 4096, "padded": 0, "k": 2048, "experts": 128,
         "top_k": 8, "dtype": "bf16"},
    ]


def _log(rng, lo, hi, step=1):
    """A size spread over its logarithm, a multiple of step."""
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def _draw_once(rng):
    op = rng.choice(["norm", "norm_grad", "adapters", "dispatch", "combine", "combine_grad"])
    if op in ("norm", "norm_grad"):
        # most hidden sizes are multiples of 16 bytes; some are not
        k = _log(rng, 64, 20000, 1 if rng.random() < 0.2 else 8)
        c = {"op": op, "rows": _log(rng, 1, 16384), "k": k, "dtype": rng.choice(["fp16", "bf16", "fp32"]),
             "kind": rng.choice(["layer", "rms"]), "affine": rng.random() < 0.8}
        if op == "norm":
            c["stats"] = rng.random() < 0.5
        return c
    if op == "adapters":
        rows = _log(rng, 1, 8192)
        requests = rows if rng.random() < 0.4 else rng.randint(1, min(rows, 100))
        return {"op": op, "rows": rows, "requests": min(requests, 512), "k": _log(rng, 256, 14336, 8),
                "n": _log(rng, 256, 14336, 8), "rank": rng.choice([8, 16, 24, 32, 64, 128]),
                "adapters": rng.randint(1, 32), "dtype": rng.choice(["fp16", "bf16"])}
    experts = rng.choice([8, 60, 64, 128, 256])
    tokens = _log(rng, 1, 8192)
    c = {"op": op, "tokens": tokens, "padded": rng.choice([0, 0, tokens // 7]), "k": _log(rng, 256, 8192, 8),
         "experts": experts, "top_k": rng.choice([1, 2, 4, 6, 8]), "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    if op == "combine":
        c["residual"] = rng.random() < 0.5
    return c


def draw(rng):
    # a drawn case costs no more than the largest listed ones
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] <= 2.2e8 and w["flops"] <= 9e9:
            return c


def _adapted(case):
    """Requests and rows that have an adapter (every eighth request has none)."""
    ends = _request_ends(case)
    have = [i for i in range(case["requests"]) if i % 8 != 7]
    rows = sum(ends[i] - (ends[i - 1] if i else 0) for i in have)
    return have, rows


def _request_ends(case):
    """Where each request's rows end: ragged lengths, the same for every seed."""
    n = case["requests"]
    w = [1 if case["rows"] == n else 1 + (7 * i) % 5 for i in range(n)]
    total, acc, ends = sum(w), 0, []
    for v in w:
        acc += v
        ends.append(case["rows"] * acc // total)
    return ends


def work(case):
    e = {"fp16": 2, "bf16": 2, "fp32": 4}[case["dtype"]]
    op, k = case["op"], case["k"]
    if op == "norm":
        rms = case["kind"] == "rms"
        params = (1 if rms else 2) * k * e if case["affine"] else 0
        stats = case["rows"] * (4 if rms else 8) if case["stats"] else 0
        return {"bytes": 2 * case["rows"] * k * e + params + stats, "flops": 8 * case["rows"] * k}
    if op == "norm_grad":
        rms = case["kind"] == "rms"
        params = (k * e + (1 if rms else 2) * k * 4) if case["affine"] else 0
        stats = case["rows"] * (4 if rms else 8)
        return {"bytes": 3 * case["rows"] * k * e + params + stats, "flops": 14 * case["rows"] * k}
    if op == "adapters":
        have, rows = _adapted(case)
        used = min(case["adapters"], len(have))
        n, r = case["n"], case["rank"]
        return {"bytes": rows * k * e + used * r * (k + n) * e + 2 * case["rows"] * n * e + 4 * case["rows"],
                "flops": 2 * rows * r * (k + n)}
    t, top_k, g = case["tokens"], case["top_k"], case["experts"]
    kept = (t - case["padded"]) * top_k
    if op == "dispatch":
        return {"bytes": (t - case["padded"]) * k * e + t * top_k * k * e + 3 * 4 * t * top_k + 4 * (g + 1),
                "flops": 0}
    if op == "combine":
        return {"bytes": kept * k * e + (2 if case["residual"] else 1) * t * k * e + 8 * t * top_k,
                "flops": 2 * kept * k}
    return {"bytes": (t - case["padded"]) * k * e + (kept + t * top_k) * k * e + 12 * t * top_k, "flops": 3 * kept * k}


# ---------------------------------------------------------------------------
# Inputs

def _activations(gen, rows, k):
    """Outlier-heavy activations: Student-t(3) values, 1% of the channels 20
    to 100 times larger (the distribution of the repository's bench)."""
    z = torch.randn((rows, k), generator=gen, device="cuda")
    c = sum(torch.randn((rows, k), generator=gen, device="cuda").square() for _ in range(3)) / 3
    gains = torch.where(torch.rand(k, generator=gen, device="cuda") < 0.01,
                        20 + 80 * torch.rand(k, generator=gen, device="cuda"), torch.ones(k, device="cuda"))
    return (z / c.clamp_min(1e-3).sqrt() * gains).clamp(-6e4, 6e4)


def _expert_choice(gen, case):
    """top_k distinct experts per token (some experts busier than others),
    -1 for the padding tokens at the end of the batch, and the weights."""
    t, g = case["tokens"], case["experts"]
    logits = torch.randn((t, g), generator=gen, device="cuda")
    logits += 0.5 * torch.randn(g, generator=gen, device="cuda")
    top, ids = torch.topk(logits, case["top_k"], dim=1)
    ids = ids.to(torch.int32)
    ids[t - case["padded"]:] = -1
    return ids, torch.softmax(top, 1)


def _sorted_by_group(ids, groups):
    """(offsets, rows, slots) of entries sorted by group, first come first."""
    top_k = ids.shape[1]
    flat = ids.reshape(-1).long()
    key = torch.where(flat >= 0, flat, groups)
    order = torch.argsort(key, stable=True)
    total = int((flat >= 0).sum())
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    rows = torch.div(order, top_k, rounding_mode="floor").to(torch.int32)
    rows[total:] = -1
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=flat.device)
    slots = torch.where(flat >= 0, slots, -1).to(torch.int32).view_as(ids)
    return offsets, rows, slots


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op, k = DTYPES[case["dtype"]], case["op"], case["k"]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    s = {"case": case}
    if op in ("norm", "norm_grad"):
        rms = case["kind"] == "rms"
        s["x"] = _activations(gen, case["rows"], k).to(dt)
        s["w"] = (1 + 0.1 * randn(k)).to(dt) if case["affine"] else None
        s["b"] = (0.1 * randn(k)).to(dt) if case["affine"] and not rms else None
        if op == "norm_grad":  # the forward pass's statistics and the gradient of its output
            xd = s["x"].double()
            mean = torch.zeros_like(xd[:, :1]) if rms else xd.mean(1, keepdim=True)
            var = (xd - mean).square().mean(1, keepdim=True)
            s["mean"] = None if rms else mean.view(-1).float()
            s["rstd"] = (var + EPS).rsqrt().view(-1).float()
            s["dy"] = (0.01 * randn(case["rows"], k)).to(dt)
    elif op == "adapters":
        rows, r, g, n = case["rows"], case["rank"], case["adapters"], case["n"]
        have, _ = _adapted(case)
        perm = torch.randperm(g, generator=gen, device="cuda").tolist()
        of_request = [-1] * case["requests"]
        for j, i in enumerate(have):
            of_request[i] = perm[j % g]
        ends = _request_ends(case)
        lengths = torch.tensor([ends[i] - (ends[i - 1] if i else 0) for i in range(len(ends))], device="cuda")
        s["ids"] = torch.repeat_interleave(torch.tensor(of_request, device="cuda"), lengths).to(torch.int32)
        # the plan of a serving step, made once and used by every layer
        s["offsets"], s["rows"], s["slots"] = _sorted_by_group(s["ids"].view(-1, 1), g)
        x = _activations(gen, rows, k)
        s["x"] = (x / x.square().mean(1, keepdim=True).sqrt()).to(dt)
        s["a"] = (randn(g, r, k) / math.sqrt(k)).to(dt)
        s["b"] = (0.5 * randn(g, n, r) / math.sqrt(r)).to(dt)
        s["scales"] = 0.5 + torch.rand(g, generator=gen, device="cuda")
        s["base"] = randn(rows, n).to(dt)
    else:
        t = case["tokens"]
        s["ids"], s["weights"] = _expert_choice(gen, case)
        if op == "dispatch":
            s["x"] = _activations(gen, t, k).to(dt)
        else:
            s["offsets"], s["rows"], s["slots"] = _sorted_by_group(s["ids"], case["experts"])
            s["y"] = randn(t * case["top_k"], k).to(dt)
            if op == "combine":
                s["residual"] = randn(t, k).to(dt) if case["residual"] else None
            else:
                s["dout"] = (0.01 * randn(t, k)).to(dt)
    return s


# ---------------------------------------------------------------------------
# One pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import sparsity_gemm_b200 as sq
    c = s["case"]
    op = c["op"]
    if op == "norm":
        return sq.layer_norm(s["x"], s["w"], s["b"], EPS, norm=c["kind"], stats=c["stats"])
    if op == "norm_grad":
        return sq.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], norm=c["kind"])
    if op == "dispatch":
        routing = sq.route(s["ids"], c["experts"])
        return [routing.offsets, routing.rows, routing.slots, sq.permute_rows(s["x"], routing)]
    routing = sq.Routing(s["offsets"], s["rows"], s["slots"])
    if op == "adapters":
        return sq.lora(s["x"], s["a"], s["b"], routing, scales=s["scales"], base=s["base"])
    if op == "combine":
        return sq.combine(s["y"], routing, s["weights"], residual=s["residual"])
    return sq.combine_backward(s["dout"], s["y"], routing, s["weights"])


def _run_plain(s):
    c = s["case"]
    op, dt = c["op"], DTYPES[c["dtype"]]
    rms = c.get("kind") == "rms"
    if op == "norm":
        x = s["x"].float()
        mean = None if rms else x.mean(1, keepdim=True)
        xc = x if rms else x - mean
        rstd = (xc.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = xc * rstd
        if s["w"] is not None:
            y = y * s["w"].float()
        if s["b"] is not None:
            y = y + s["b"].float()
        y = y.to(dt)
        return (y, None if rms else mean.view(-1), rstd.view(-1)) if c["stats"] else y
    if op == "norm_grad":
        dy, x, rstd = s["dy"].float(), s["x"].float(), s["rstd"].view(-1, 1)
        xhat = x * rstd if rms else (x - s["mean"].view(-1, 1)) * rstd
        g = dy if s["w"] is None else dy * s["w"].float()
        dx = g - xhat * (g * xhat).mean(1, keepdim=True)
        if not rms:
            dx = dx - g.mean(1, keepdim=True)
        dx = (rstd * dx).to(dt)
        dw = None if s["w"] is None else (dy * xhat).sum(0)
        db = None if rms or s["w"] is None else dy.sum(0)
        return dx, dw, db
    if op == "adapters":
        # every row against every adapter, then the row's own kept
        g, r, n = c["adapters"], c["rank"], c["n"]
        h = s["x"].float() @ s["a"].float().reshape(g * r, -1).t()
        ids = s["ids"].long()
        mine = (ids.view(-1, 1) == torch.arange(g, device=ids.device)).float() * s["scales"]
        h = (h.view(-1, g, r) * mine.unsqueeze(2)).reshape(-1, g * r)
        return (s["base"].float() + h @ s["b"].float().transpose(1, 2).reshape(g * r, n)).to(dt)
    if op == "dispatch":
        ids, top_k, g = s["ids"], c["top_k"], c["experts"]
        flat = ids.reshape(-1).long()
        key = torch.where(flat >= 0, flat, g)
        order = torch.argsort(key, stable=True)
        bounds = (key.view(1, -1) < torch.arange(g + 1, device=key.device).view(-1, 1)).sum(1)
        kept = torch.arange(flat.numel(), device=key.device) < bounds[g]
        rows = torch.where(kept, torch.div(order, top_k, rounding_mode="floor"), -1)
        slots = torch.empty_like(flat)
        slots[order] = torch.arange(flat.numel(), device=flat.device)
        slots = torch.where(flat >= 0, slots, -1).view_as(ids)
        moved = torch.where(kept.view(-1, 1), s["x"][rows.clamp_min(0)], 0)
        return [bounds.to(torch.int32), rows.to(torch.int32), slots.to(torch.int32), moved]
    there = (s["slots"] >= 0)
    at = s["slots"].clamp_min(0).long()
    y = s["y"][at].float()
    if op == "combine":
        out = (torch.where(there, s["weights"], 0).unsqueeze(2) * y).sum(1)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return out.to(dt)
    dout = s["dout"].float().unsqueeze(1)
    dw = torch.where(there, (dout * y).sum(2), 0)
    dy = torch.zeros_like(s["y"])
    dy[s["slots"][there].long()] = (s["weights"].unsqueeze(2) * dout).to(dt)[there]
    return dy, dw


# ---------------------------------------------------------------------------
# The definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, n_rows = case["op"], case.get("rows")
    f64 = lambda t: None if t is None else t.double()  # noqa: E731
    if op in ("norm", "norm_grad"):
        x, w, b, k = f64(s["x"]), f64(s["w"]), f64(s["b"]), case["k"]
        if op == "norm":
            mu = torch.zeros(n_rows, 1, dtype=torch.float64, device="cuda") if case["kind"] == "rms" \
                else x.sum(1, keepdim=True) / k
            sd = torch.sqrt(torch.einsum("ij,ij->i", x - mu, x - mu) / k + EPS).view(-1, 1)
            y = (x - mu) / sd
            y = y if w is None else torch.einsum("ij,j->ij", y, w)
            y = y if b is None else y + b
            if not case["stats"]:
                return y
            return y, None if case["kind"] == "rms" else mu.flatten(), 1 / sd.flatten()
        # the Jacobian of y = w (x - mu) rstd with the statistics as given
        r, dy = f64(s["rstd"]), f64(s["dy"])
        z = x if s["mean"] is None else x - f64(s["mean"])[:, None]
        t = dy if w is None else torch.einsum("ij,j->ij", dy, w)
        along = torch.einsum("ij,ij->i", t, z) * r ** 3 / k
        dx = r[:, None] * t - along[:, None] * z
        if s["mean"] is not None:
            dx -= (r * t.sum(1) / k)[:, None]
        if w is None:
            return dx, None, None
        dw = torch.einsum("ij,ij,i->j", dy, z, r)
        return dx, dw, dy.sum(0) if case["kind"] == "layer" else None
    if op == "adapters":
        out = f64(s["base"])
        for g in range(case["adapters"]):
            at = torch.nonzero(s["ids"] == g).flatten()
            h = torch.einsum("mk,rk->mr", f64(s["x"][at]), f64(s["a"][g]))
            out[at] += f64(s["scales"][g]) * torch.einsum("mr,nr->mn", h, f64(s["b"][g]))
        return out
    if op == "dispatch":
        ids = s["ids"].cpu().tolist()
        entries = sorted((e, t, j) for t, row in enumerate(ids) for j, e in enumerate(row) if e >= 0)
        top_k, g = case["top_k"], case["experts"]
        offsets = [0] * (g + 1)
        rows, slots = [-1] * (len(ids) * top_k), [[-1] * top_k for _ in ids]
        for i, (e, t, j) in enumerate(entries):
            offsets[e + 1] += 1
            rows[i], slots[t][j] = t, i
        for e in range(g):
            offsets[e + 1] += offsets[e]
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        moved = torch.zeros(len(rows), case["k"], dtype=torch.float64, device="cuda")
        moved[:len(entries)] = f64(s["x"])[i32(rows[:len(entries)]).long()]
        return [i32(offsets), i32(rows), i32(slots), moved]
    tokens, top_k = case["tokens"], case["top_k"]
    if op == "combine":
        out = torch.zeros(tokens, case["k"], dtype=torch.float64, device="cuda")
        if s["residual"] is not None:
            out += f64(s["residual"])
        for j in range(top_k):
            at = torch.nonzero(s["slots"][:, j] >= 0).flatten()
            out[at] += f64(s["weights"][at, j])[:, None] * f64(s["y"][s["slots"][at, j].long()])
        return out
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(tokens, top_k, dtype=torch.float64, device="cuda")
    for j in range(top_k):
        at = torch.nonzero(s["slots"][:, j] >= 0).flatten()
        slot = s["slots"][at, j].long()
        dy[slot] = f64(s["weights"][at, j])[:, None] * f64(s["dout"][at])
        dw[at, j] = torch.einsum("mk,mk->m", f64(s["y"][slot]), f64(s["dout"][at]))
    return dy, dw

"""The training-step operators of the two towers, as they are measured.

Each case is one call of one operator: embedding lookup and its gradient by
sorted ids, layer norm and its gradient, the gradient of the L2 normalisation,
the gradient of the in-batch sampled softmax, and the global gradient norm with
clipping. With ``own`` false a case runs in its plain form (elementary torch
operations); with ``own`` true it calls the library's entry point.
"""
import math
import random

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i32": torch.int32, "i64": torch.int64}
SIZE = {"f32": 4, "bf16": 2, "i32": 4, "i64": 8}
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the vectors of the candidates that a batch of 1024 searches with k = 1000 returned (-1: padding)
        {"name": "lookup_results", "op": "embedding", "m": 1_024_000, "rows": 4_000_000, "d": 128, "table": "bf16",
         "out": "bf16", "ids": "i32", "scale": 1.0},
        # the gradient of a small table (one categorical feature) over one batch of histories, dense
        {"name": "embedding_grad_feature", "op": "embedding_grad", "m": 4_097, "rows": 50_000, "d": 64, "table": "f32",
         "out": "f32", "ids": "i64", "scale": 8.0},
        # the gradient of a catalogue of items, as the rows that the batch touched
        {"name": "embedding_grad_catalogue", "op": "embedding_grad_rows", "m": 1_000_003, "rows": 10_000_000, "d": 128,
         "table": "bf16", "out": "f32", "ids": "i64", "scale": 1.0},
        # the input norm of a user tower, for one request
        {"name": "layernorm_request", "op": "layernorm", "n": 37, "d": 256, "x": "bf16", "w": "f32"},
        # the norm of a candidate tower that embeds a slice of the corpus
        {"name": "layernorm_corpus", "op": "layernorm", "n": 200_003, "d": 512, "x": "f32", "w": "f32"},
        # its backward pass over a training batch, with an odd width of the hidden layer
        {"name": "layernorm_grad_batch", "op": "layernorm_grad", "n": 65_536, "d": 1000, "x": "bf16", "w": "f32"},
        # the backward pass of the L2 normalisation: a small batch, and a global batch with its shared negatives
        {"name": "normalize_grad_small", "op": "normalize_grad", "n": 300, "d": 96, "x": "f32", "g": "bf16"},
        {"name": "normalize_grad_batch", "op": "normalize_grad", "n": 1_000_000, "d": 128, "x": "bf16", "g": "bf16"},
        # the gradients of two small towers, and of large towers with their embedding tables
        {"name": "clip_towers", "op": "clip", "count": 14, "f32": 300_001, "bf16": 0, "shapes": 5, "max_norm": 1.0},
        {"name": "clip_tables", "op": "clip", "count": 160, "f32": 150_000_000, "bf16": 250_000_001, "shapes": 6,
         "max_norm": 1.0},
        # the loss's gradient: a small batch with few shared negatives, and a global batch with as many as it has rows
        {"name": "inbatch_grad_small", "op": "inbatch_grad", "b": 500, "nc": 1100, "d": 96, "tau": 0.05, "masks": True},
        {"name": "inbatch_grad_batch", "op": "inbatch_grad", "b": 16_384, "nc": 32_768, "d": 128, "tau": 0.05,
         "masks": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embedding", "embedding_grad", "embedding_grad_rows", "layernorm", "layernorm_grad",
                     "normalize_grad", "clip", "inbatch_grad"])
    if op.startswith("embedding"):
        d = _log_int(rng, 1, 2048)
        m = _log_int(rng, 1, min(1_200_000, 150_000_000 // d))
        rows = _log_int(rng, 1, min(10_000_000, (200_000_000 if op == "embedding_grad" else 500_000_000) // d))
        t = rng.choice(["f32", "bf16"])
        return {"op": op, "m": m, "rows": rows, "d": d, "table": t, "out": rng.choice(["f32", t]),
                "ids": rng.choice(["i32", "i64"]), "scale": rng.choice([1.0, round(math.sqrt(d), 3)])}
    if op.startswith("layernorm"):
        d = _log_int(rng, 8, 8192)
        return {"op": op, "n": _log_int(rng, 1, min(500_000, 100_000_000 // d)), "d": d,
                "x": rng.choice(["f32", "bf16"]), "w": rng.choice(["f32", "bf16"])}
    if op == "normalize_grad":
        d = 16 * rng.randint(1, 32)
        return {"op": op, "n": _log_int(rng, 1, 200_000_000 // d), "d": d, "x": rng.choice(["f32", "bf16"]),
                "g": rng.choice(["f32", "bf16"])}
    if op == "clip":
        return {"op": op, "count": _log_int(rng, 1, 400), "f32": _log_int(rng, 1, 150_000_000),
                "bf16": _log_int(rng, 1, 200_000_000), "shapes": rng.randint(1, 1 << 20),
                "max_norm": rng.choice([0.5, 1.0, 1e9])}
    b = _log_int(rng, 1, 16_384)
    return {"op": op, "b": b, "nc": b + rng.choice([0, _log_int(rng, 1, 16_384)]), "d": 16 * rng.randint(4, 16),
            "tau": rng.choice([0.05, 0.1, 1.0]), "masks": rng.random() < 0.7}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _zipf(g, m, rows):
    """Ids of [0, rows), popular ones low: log-uniform, which is close to Zipf's law with exponent 1."""
    u = torch.rand(m, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(rows + 1.0)).to(torch.int64) - 1).clamp_(0, rows - 1)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _clip_sizes(case):
    """Element counts of the tensors: `count` in all, shared between the two types by their totals."""
    r = random.Random(case["shapes"])

    def split(total, parts):
        if total <= 0:
            return []
        weights = [math.exp(r.uniform(0.0, 6.0)) for _ in range(parts)]
        cuts = [int(total * w / sum(weights)) for w in weights]
        cuts[-1] += total - sum(cuts)
        return cuts

    parts16 = 0 if case["bf16"] == 0 else max(1, case["count"] // 2)
    parts32 = 0 if case["f32"] == 0 else max(1, case["count"] - parts16)
    return split(case["f32"], parts32), split(case["bf16"], parts16)


def _inbatch_inputs(g, case):
    """Vectors of length about 1, item ids with Zipf popularity, log q of the ids, 1% padding; the loss's lse and loss."""
    b, nc, d = case["b"], case["nc"], case["d"]
    s = {"users": _randn(g, b, d).div_(math.sqrt(d)).bfloat16(), "logq": None, "item_ids": None, "valid": None}
    items = _randn(g, nc, d).div_(math.sqrt(d)).bfloat16()
    if case["masks"]:
        catalogue = 1_000_000
        ids = _zipf(g, nc, catalogue)
        _, inverse = torch.unique(ids, return_inverse=True)
        first = torch.full((nc,), nc, dtype=torch.int64, device="cuda")
        first.scatter_reduce_(0, inverse, torch.arange(nc, device="cuda"), reduce="amin")
        items = items[first[inverse]].contiguous()  # a repeated item has one vector
        s["item_ids"] = ids
        s["logq"] = torch.log(torch.log1p(1.0 / (ids + 1.0)) / math.log(catalogue + 1.0)).float()
        s["valid"] = torch.rand(nc, generator=g, device="cuda") >= 0.01
    s["items"] = items
    lse, own_logit = [], []
    for r0 in range(0, b, 2048):
        rows = torch.arange(r0, min(b, r0 + 2048), device="cuda")
        logits, keep = _logits(s, rows, case["tau"], torch.float64)
        own_logit.append(logits.gather(1, rows[:, None])[:, 0])
        lse.append(torch.logsumexp(logits.masked_fill_(~keep, -math.inf), 1))
    s["lse"] = torch.cat(lse).float()
    s["loss"] = torch.cat(lse).sub_(torch.cat(own_logit)).float()
    if s["valid"] is not None:
        s["loss"] = torch.where(s["valid"][:b], s["loss"], 0.0)
    s["grad_mean"] = torch.ones((), device="cuda")
    return s


def _logits(s, rows, tau, dtype):
    """Logits of the listed rows against every column, and which of them enter the row's sum."""
    logits = s["users"][rows].to(dtype) @ s["items"].to(dtype).T
    logits /= tau
    if s["logq"] is not None:
        logits -= s["logq"].to(dtype)
    nc = logits.shape[1]
    keep = torch.ones_like(logits, dtype=torch.bool)
    if s["item_ids"] is not None:
        keep = s["item_ids"][rows][:, None] != s["item_ids"][None, :]
        keep |= rows[:, None] == torch.arange(nc, device="cuda")[None, :]
    if s["valid"] is not None:
        keep &= s["valid"][None, :]
    return logits, keep


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1_000_003 + 17)
    op = case["op"]
    s = {"case": case, "op": op}
    if op.startswith("embedding"):
        m, rows, d = case["m"], case["rows"], case["d"]
        ids = _zipf(g, m, rows)
        ids[torch.rand(m, generator=g, device="cuda") < 0.02] = -1  # padding
        s["ids"] = ids.to(DT[case["ids"]])
        if op == "embedding":
            s["table"] = _randn(g, rows, d, dtype=DT[case["table"]])
        else:
            s["grad"] = _randn(g, m, d, dtype=DT[case["table"]])
        if op == "embedding_grad_rows":  # places behind the last row are left as they are
            s["row_ids"] = torch.full((m,), -1, dtype=DT[case["ids"]], device="cuda")
            s["row_grads"] = torch.zeros((m, d), dtype=DT[case["out"]], device="cuda")
    elif op.startswith("layernorm"):
        n, d = case["n"], case["d"]
        s["x"] = (_randn(g, n, d) * (0.5 + torch.rand(n, 1, generator=g, device="cuda"))
                  + _randn(g, n, 1)).to(DT[case["x"]])
        s["w"] = (1.0 + 0.1 * _randn(g, d)).to(DT[case["w"]])
        s["bias"] = (0.1 * _randn(g, d)).to(DT[case["w"]])
        if op == "layernorm_grad":
            s["grad"] = _randn(g, n, d, dtype=DT[case["x"]])
            x = s["x"].float()
            mean = x.mean(1, keepdim=True)
            s["mean"] = mean[:, 0].contiguous()
            s["rstd"] = torch.rsqrt((x - mean).square().mean(1) + EPS)
    elif op == "normalize_grad":
        s["x"] = _randn(g, case["n"], case["d"], dtype=DT[case["x"]])
        s["grad"] = _randn(g, case["n"], case["d"], dtype=DT[case["g"]])
    elif op == "clip":
        sizes = _clip_sizes(case)
        s["in"] = [1e-3 * _randn(g, sum(sizes[0])), (1e-3 * _randn(g, sum(sizes[1]))).bfloat16()]
        s["out"] = [torch.empty_like(t) for t in s["in"]]
        views = [[v for t, z in zip(flat, sizes) for v in t.split(z or [0])] for flat in (s["in"], s["out"])]
        s["grads"], s["clipped"] = views
    else:
        s.update(_inbatch_inputs(g, case))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import exact_inner_product_b200 as tt
    op, case = s["op"], s["case"]
    if op == "embedding":
        return tt.tt_embedding(s["table"], s["ids"], scale=case["scale"], out_dtype=DT[case["out"]])
    if op == "embedding_grad":
        return tt.tt_embedding_grad(s["ids"], s["grad"], case["rows"], scale=case["scale"], out_dtype=DT[case["out"]])
    if op == "embedding_grad_rows":
        ids, rows, count = tt.tt_embedding_grad_rows(s["ids"], s["grad"], case["rows"], scale=case["scale"],
                                                     out=(s["row_ids"], s["row_grads"]))
        return {"ids": ids, "rows": rows, "count": count}
    if op == "layernorm":
        y, mean, rstd = tt.tt_layernorm(s["x"], s["w"], s["bias"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "layernorm_grad":
        gx, gw, gb = tt.tt_layernorm_grad(s["grad"], s["x"], s["w"], s["mean"], s["rstd"])
        return {"x": gx, "w": gw, "bias": gb}
    if op == "normalize_grad":
        return tt.tt_normalize_grad(s["grad"], s["x"])
    if op == "clip":
        norm = tt.tt_clip_grad_norm(s["grads"], case["max_norm"], out=s["clipped"])
        return {"norm": norm, "f32": s["out"][0], "bf16": s["out"][1]}
    gu, gv = tt.tt_inbatch_softmax_grad(s["users"], s["items"], s["lse"], s["loss"], case["tau"], logq=s["logq"],
                                        item_ids=s["item_ids"], valid=s["valid"], grad_mean=s["grad_mean"])
    return {"users": gu, "items": gv}


def _plain(s):
    op, case = s["op"], s["case"]
    if op == "embedding":
        ids = s["ids"].long()
        rows = s["table"][ids.clamp(min=0)].float() * case["scale"]
        return torch.where((ids >= 0)[:, None], rows, 0.0).to(DT[case["out"]])
    if op == "embedding_grad":
        keep = s["ids"] >= 0
        total = torch.zeros(case["rows"], case["d"], dtype=torch.float64, device="cuda")
        grad = torch.where(keep[:, None], s["grad"].double(), 0.0)
        total.index_add_(0, s["ids"].long().clamp(min=0), grad)
        return (total * case["scale"]).to(DT[case["out"]])
    if op == "embedding_grad_rows":
        ids, order = torch.sort(s["ids"], stable=True)
        new = torch.ones_like(ids, dtype=torch.bool)
        new[1:] = ids[1:] != ids[:-1]
        new &= ids >= 0
        place = (torch.cumsum(new, 0) - 1).clamp(min=0)
        count = new.sum(dtype=torch.int32).reshape(1)
        m, d = s["grad"].shape
        total = torch.zeros(m, d, dtype=torch.float64, device="cuda")
        total.index_add_(0, place, torch.where((ids >= 0)[:, None], s["grad"][order].double(), 0.0))
        row_ids = torch.full((m,), -1, dtype=ids.dtype, device="cuda")
        row_ids.scatter_reduce_(0, place, torch.where(ids >= 0, ids, -1), "amax")
        return {"ids": row_ids, "rows": (total * case["scale"]).to(DT[case["out"]]), "count": count}
    if op == "layernorm":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        centred = x - mean
        rstd = torch.rsqrt(centred.square().mean(1, keepdim=True) + EPS)
        y = centred * rstd * s["w"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "layernorm_grad":
        xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        grad = s["grad"].float()
        gw, gb = (grad * xhat).sum(0), grad.sum(0)
        grad = grad * s["w"].float()
        gx = grad - grad.mean(1, keepdim=True) - xhat * (grad * xhat).mean(1, keepdim=True)
        return {"x": (gx * s["rstd"][:, None]).to(s["x"].dtype), "w": gw, "bias": gb}
    if op == "normalize_grad":
        x, grad = s["x"].float(), s["grad"].float()
        square = x.square().sum(1, keepdim=True)
        norm = torch.sqrt(square.clamp(min=1e-12))
        inner = torch.where(square >= 1e-12, (x * grad).sum(1, keepdim=True), 0.0)
        return ((grad - x * (inner / (norm * norm))) / norm).to(s["x"].dtype)
    if op == "clip":
        norm = torch.sqrt(torch.stack([t.double().square().sum() for t in s["in"]]).sum()).float()
        scale = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
        f32, bf16 = [(t.float() * scale).to(t.dtype) for t in s["in"]]
        return {"norm": norm, "f32": f32, "bf16": bf16}
    b = case["b"]
    rows = torch.arange(b, device="cuda")
    p, keep = _logits(s, rows, case["tau"], torch.float32)
    p = torch.where(keep, torch.exp_(p.sub_(s["lse"][:, None])), 0.0)
    p[rows, rows] = torch.expm1(-s["loss"])
    weight = s["grad_mean"] / (b * case["tau"]) * torch.ones(b, device="cuda")
    if s["valid"] is not None:
        ok = s["valid"][:b]
        weight = torch.where(ok, s["grad_mean"] / (ok.sum().clamp(min=1) * case["tau"]), 0.0)
        p = torch.where(ok[:, None], p, 0.0)
    p *= weight[:, None]
    return {"users": (p @ s["items"].float()).bfloat16(), "items": (p.T @ s["users"].float()).bfloat16()}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op.startswith("embedding"):
        m, d, e_in, e_out, e_id = case["m"], case["d"], SIZE[case["table"]], SIZE[case["out"]], SIZE[case["ids"]]
        # ids that differ, in the mean: a row with the probability p is among m draws with 1 - (1 - p)^m
        edges = [int(round(math.exp(math.log(case["rows"] + 1.0) * i / 400))) for i in range(401)]
        touched = sum((hi - lo) * -math.expm1(m * 0.98 * math.log1p(-min(
            1 - 1e-12, math.log1p(1.0 / ((lo + hi) / 2)) / math.log(case["rows"] + 1.0))))
            for lo, hi in zip(edges, edges[1:]) if hi > lo)
        if op == "embedding":
            return {"bytes": m * e_id + touched * d * e_in + m * d * e_out, "flops": m * d}
        written = (case["rows"] if op == "embedding_grad" else touched) * d * e_out
        return {"bytes": m * e_id + m * d * e_in + written, "flops": m * d}
    if op == "layernorm":
        n, d = case["n"], case["d"]
        return {"bytes": 2 * n * d * SIZE[case["x"]] + 8 * n + 2 * d * SIZE[case["w"]], "flops": 8 * n * d}
    if op == "layernorm_grad":
        n, d = case["n"], case["d"]
        return {"bytes": 3 * n * d * SIZE[case["x"]] + 8 * n + d * SIZE[case["w"]] + 8 * d, "flops": 14 * n * d}
    if op == "normalize_grad":
        return {"bytes": case["n"] * case["d"] * (2 * SIZE[case["x"]] + SIZE[case["g"]]),
                "flops": 8 * case["n"] * case["d"]}
    if op == "clip":
        total = case["f32"] * 4 + case["bf16"] * 2
        return {"bytes": 2 * total + 4, "flops": 3 * (case["f32"] + case["bf16"])}
    b, nc, d = case["b"], case["nc"], case["d"]
    # the logits again, and the two products with the probabilities
    return {"bytes": 4 * (b + nc) * d + 8 * b + (13 * nc if case["masks"] else 0), "flops": 6.0 * b * nc * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, d = case["op"], case.get("d")
    f8 = torch.float64
    if op == "embedding":
        out = torch.zeros(case["m"], d, dtype=f8, device="cuda")
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        out[at] = s["table"].index_select(0, s["ids"][at].long()).to(f8).mul_(case["scale"])
        return out
    if op.startswith("embedding_grad"):
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        present, group, runs = torch.unique(s["ids"][at].long(), return_inverse=True, return_counts=True)
        order = torch.argsort(group, stable=True)
        total = torch.segment_reduce(s["grad"][at][order].to(f8), "sum", lengths=runs, axis=0).mul_(case["scale"]) \
            if at.numel() else torch.zeros(0, d, dtype=f8, device="cuda")
        if op == "embedding_grad":
            out = torch.zeros(case["rows"], d, dtype=f8, device="cuda")
            out[present] = total
            return out
        out = torch.zeros(case["m"], d, dtype=f8, device="cuda")
        out[:present.numel()] = total
        return {"ids": None, "rows": out, "count": None}
    if op.startswith("layernorm"):
        x, w = s["x"].to(f8), s["w"].to(f8)
        if op == "layernorm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = 1.0 / torch.sqrt(var + EPS)
            return {"y": torch.addcmul(s["bias"].to(f8), (x - mean[:, None]).mul_(rstd[:, None]), w), "mean": mean,
                    "rstd": rstd}
        grad, rstd = s["grad"].to(f8), s["rstd"].to(f8)[:, None]
        x = (x - s["mean"].to(f8)[:, None]).mul_(rstd)
        along = torch.einsum("nd,nd,d->n", grad, x, w) / d
        ahead = (grad @ w) / d
        gx = (grad * w - ahead[:, None] - along[:, None] * x) * rstd
        return {"x": gx, "w": torch.einsum("nd,nd->d", grad, x), "bias": grad.sum(0)}
    if op == "normalize_grad":
        x, grad = s["x"].to(f8), s["grad"].to(f8)
        square = torch.einsum("nd,nd->n", x, x)
        y = x / square.clamp(min=1e-12).sqrt()[:, None]
        along = torch.einsum("nd,nd->n", y, grad) * (square >= 1e-12)
        return (grad - along[:, None] * y) / square.clamp(min=1e-12).sqrt()[:, None]
    if op == "clip":
        total = sum(torch.linalg.vector_norm(t.to(f8)) ** 2 for t in s["in"] if t.numel())
        norm = total ** 0.5
        scale = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm, "f32": s["in"][0].to(f8) * scale, "bf16": s["in"][1].to(f8) * scale}
    b, nc, tau = case["b"], case["nc"], case["tau"]
    users, items, lse = s["users"].to(f8), s["items"].to(f8), s["lse"].to(f8)
    ok = torch.ones(nc, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    weight = ok[:b].to(f8) * (float(s["grad_mean"]) / (max(1, int(ok[:b].sum())) * tau))
    gu, gv = torch.zeros_like(users), torch.zeros_like(items)
    for r0 in range(0, b, 1024):
        r1 = min(b, r0 + 1024)
        p = torch.addmm(-lse[r0:r1, None].expand(-1, nc), users[r0:r1], items.T, alpha=1.0 / tau)
        if s["logq"] is not None:
            p -= s["logq"].to(f8)[None, :]
        p = p.exp_() * ok[None, :].to(f8)
        if s["item_ids"] is not None:
            p[s["item_ids"][r0:r1, None] == s["item_ids"][None, :]] = 0.0
        p[:, r0:r1].diagonal().copy_(torch.expm1(-s["loss"][r0:r1].to(f8)))
        p = torch.nan_to_num(p, nan=0.0, posinf=0.0) * weight[r0:r1, None]
        gu[r0:r1] = p @ items
        gv += p.T @ users[r0:r1]
    return {"users": gu, "items": gv}

"""The training-step operators in one run, as a user strings them together:
embedding rows, layer norm, L2 normalisation, the in-batch loss, and the
gradients back to the tables and the norm's weights, then clipping. (GPU)

The reference is the same chain in float64 by automatic differentiation. The
normalised vectors are stored in bf16, so the reference takes the stored
values (a straight-through rounding); the loss's gradient comes back in bf16.
Bounds: that rounding and the products' (bounds of the loss's gradient, see
test_gpu_softmax_grad) are carried through the linear maps behind it with
absolute values; the fp32 steps after it add less than 1e-4 of the terms."""
import pytest
import torch

import train_ref as R
from test_gpu_softmax_grad import reference as softmax_reference

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

BF16 = torch.bfloat16
EPS = 1e-5


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def make(seed, b=260, extra=140, d=64, users=500, items=300):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    nc = b + extra
    return {
        "user_table": torch.randn((users, d), generator=g, device="cuda"),
        "item_table": torch.randn((items, d), generator=g, device="cuda"),
        "w": 1 + 0.1 * torch.randn(d, generator=g, device="cuda"),
        "bias": 0.1 * torch.randn(d, generator=g, device="cuda"),
        "user_ids": torch.randint(0, users, (b,), generator=g, device="cuda"),
        "item_ids": (torch.rand(nc, generator=g, device="cuda") ** 2 * items).long(),
        "logq": torch.randn(nc, generator=g, device="cuda"),
        "valid": torch.rand(nc, generator=g, device="cuda") > 0.05,
        "tau": 0.2, "scale": 0.5, "max_norm": 0.05,
    }


def tower(x, p):
    y, mean, rstd = tt.tt_layernorm(x, p["w"], p["bias"], EPS)
    z = torch.empty(y.shape, dtype=BF16, device="cuda")
    tt.tt_normalize_candidates(y, z, make_index=False)
    return z, (x, y, mean, rstd)


def tower_grad(gz, saved, p):
    x, y, mean, rstd = saved
    return tt.tt_layernorm_grad(tt.tt_normalize_grad(gz, y), x, p["w"], mean, rstd)


def step(p):
    """One step: the loss, the clipped gradients and their norm before the clipping."""
    xu = tt.tt_embedding(p["user_table"], p["user_ids"], scale=p["scale"])
    xi = tt.tt_embedding(p["item_table"], p["item_ids"], scale=p["scale"])
    zu, su = tower(xu, p)
    zi, si = tower(xi, p)
    masks = {"logq": p["logq"], "item_ids": p["item_ids"], "valid": p["valid"]}
    lse, loss, mean = tt.tt_inbatch_softmax(zu, zi, p["tau"], check=False, **masks)
    one = torch.ones((), device="cuda")
    gzu, gzi = tt.tt_inbatch_softmax_grad(zu, zi, lse, loss, p["tau"], grad_mean=one, **masks)
    gxu, gwu, gbu = tower_grad(gzu, su, p)
    gxi, gwi, gbi = tower_grad(gzi, si, p)
    grads = [tt.tt_embedding_grad(p["user_ids"], gxu, p["user_table"].shape[0], scale=p["scale"]),
             tt.tt_embedding_grad(p["item_ids"], gxi, p["item_table"].shape[0], scale=p["scale"]), gwu + gwi, gbu + gbi]
    raw = [g.clone() for g in grads]
    norm = tt.tt_clip_grad_norm(grads, p["max_norm"])
    return {"mean": mean, "grads": grads, "raw": raw, "norm": norm, "zu": zu, "zi": zi, "lse": lse, "loss": loss,
            "saved": (su, si)}


def reference_step(p, out):
    leaves = [p[k].double().requires_grad_(True) for k in ("user_table", "item_table", "w", "bias")]
    ut, it, w, bias = leaves

    def embed(table, ids, stored):
        x = table[ids] * p["scale"]
        c = x - x.mean(1, keepdim=True)
        y = c / (c.square().mean(1, keepdim=True) + EPS).sqrt() * w + bias
        z = y / y.square().sum(1, keepdim=True).clamp(min=1e-12).sqrt()
        return z + (stored.double() - z).detach()  # the value as stored

    zu, zi = embed(ut, p["user_ids"], out["zu"]), embed(it, p["item_ids"], out["zi"])
    b = zu.shape[0]
    logits = zu @ zi.T / p["tau"] - p["logq"].double()
    rows = torch.arange(b, device="cuda")
    same = p["item_ids"][:b, None] == p["item_ids"][None, :]
    same[rows, rows] = False
    keep = p["valid"][None, :] & ~same
    ok = p["valid"][:b]
    lse = torch.logsumexp(logits.masked_fill(~keep, float("-inf")), 1)
    mean = (lse - logits[rows, rows])[ok].mean()
    mean.backward()
    return mean.detach(), [x.grad for x in leaves]


def carried(p, out):
    """The bounds of the loss's gradients, through the maps behind them."""
    ok = p["valid"][:out["zu"].shape[0]]
    weight = ok.double() / int(ok.sum())
    inp = {"users": out["zu"], "items": out["zi"], "logq": p["logq"], "item_ids": p["item_ids"], "valid": p["valid"]}
    grads, bounds = softmax_reference(inp, p["tau"], out["lse"], out["loss"], weight, ("logq", "ids", "valid"))
    total = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (p["user_table"], p["item_table"], p["w"],
                                                                                p["bias"])]
    for k, ids in ((0, p["user_ids"]), (1, p["item_ids"])):
        x, y, mean, rstd = (t.double() for t in out["saved"][k])
        e = bounds[k] + 1e-4 * grads[k].abs()  # and the fp32 steps'
        norm = y.square().sum(1, keepdim=True).sqrt()
        z = (y / norm).abs()
        e = (e + z * (z * e).sum(1, keepdim=True)) / norm
        xh = ((x - mean[:, None]) * rstd[:, None]).abs()
        w = p["w"].double().abs()
        total[2] += (e * xh).sum(0)
        total[3] += e.sum(0)
        e = rstd[:, None] * (e * w + (e * w).mean(1, keepdim=True) + xh * (e * w * xh).mean(1, keepdim=True))
        total[k].index_add_(0, ids, e * p["scale"])
    return total


@pytest.mark.parametrize("shape", [{}, {"b": 33, "extra": 0, "d": 80, "users": 10, "items": 7},
                                   {"b": 1000, "extra": 3000, "d": 128, "users": 50, "items": 4000}])
def test_a_step_against_automatic_differentiation(shape):
    _cuda()
    p = make(3, **shape)
    out = step(p)
    mean, want = reference_step(p, out)
    assert abs(float(out["mean"]) - float(mean)) <= 1e-4 * (1 + abs(float(mean)))
    for name, got, w, tol in zip(("user_table", "item_table", "w", "bias"), out["raw"], want, carried(p, out)):
        R.close(got, w, tol + 1e-12, name)
    norm = sum(float(g.double().square().sum()) for g in out["raw"]) ** 0.5
    assert abs(float(out["norm"]) - norm) <= 5 * R.U * norm
    scale = min(1.0, p["max_norm"] / (norm + 1e-6))
    for g, r in zip(out["grads"], out["raw"]):
        R.close(g, r.double() * scale, r.double().abs() * scale * 10 * R.U, "clipped")


def test_row_form_gives_the_same_table_gradient():
    _cuda()
    p = make(5)
    out = step(p)
    gx = tower_grad(tt.tt_inbatch_softmax_grad(out["zu"], out["zi"], out["lse"], out["loss"], p["tau"],
                                               grad_mean=torch.ones((), device="cuda"), logq=p["logq"],
                                               item_ids=p["item_ids"], valid=p["valid"])[1], out["saved"][1], p)[0]
    ids, rows, count = tt.tt_embedding_grad_rows(p["item_ids"], gx, p["item_table"].shape[0], scale=p["scale"])
    n = int(count)
    assert torch.equal(rows[:n], out["raw"][1][ids[:n]])


def test_a_captured_step_replays_on_new_data():
    """The whole step as one graph: replayed on other tables and ids it gives the
    bits of an eager step."""
    _cuda()
    p = make(7)
    step(p)  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(p)
    q = make(8)
    for k, v in q.items():
        if isinstance(v, torch.Tensor):
            p[k].copy_(v)
    graph.replay()
    torch.cuda.synchronize()
    want = step(q)
    assert torch.equal(out["mean"], want["mean"]) and torch.equal(out["norm"], want["norm"])
    assert all(torch.equal(a, b) for a, b in zip(out["grads"], want["grads"]))


def test_two_streams_at_once():
    """Two steps in flight on two streams, each with its own buffers."""
    _cuda()
    ps = [make(11), make(12)]
    want = [step(p) for p in ps]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [None, None]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                outs[k] = step(ps[k])
    torch.cuda.synchronize()
    for k in range(2):
        assert all(torch.equal(a, b) for a, b in zip(outs[k]["grads"], want[k]["grads"]))

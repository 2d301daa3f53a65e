"""The gradient of the in-batch softmax on the GPU against float64. (GPU)

The bound of an element, from the roundings: P enters the products as bf16,
off by at most half a bf16 step (2^-8 relative to the value); its exponent is
off by the fp32 logit (gamma_d |u| |v| / tau), by the roundings of the biased
logit and of lse (a few U times their size) and ex2 (2^-22). The products are
exact and add in fp32 over at most b or nc terms in chains per tile:
(n / 16 + 64) U of the sum of the terms' sizes. The diagonal's coefficient is
off by a few U of itself, and the result is rounded to bf16 once."""
import math

import numpy as np
import pytest
import torch

import train_ref as R
import workloads as W

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

BF16 = torch.bfloat16


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def reference(inp, tau, lse, loss, w, use):
    """grad_users, grad_items and their bounds in float64, from the lse and loss given."""
    u, v = inp["users"].double(), inp["items"].double()
    b, nc, d = u.shape[0], v.shape[0], u.shape[1]
    ok = inp["valid"].bool() if "valid" in use else torch.ones(nc, dtype=torch.bool, device=u.device)
    u = torch.where(ok[:b, None], u, 0.0)
    v = torch.where(ok[:, None], v, 0.0)
    logit = u @ v.T / tau
    if "logq" in use:
        logit = logit - inp["logq"].double()
    keep = ok[None, :].expand(b, nc).clone()
    if "ids" in use:
        keep &= inp["item_ids"][:b, None] != inp["item_ids"][None, :]
    rows = torch.arange(b, device=u.device)
    keep[rows, rows] = False
    w = torch.where(ok[:b], w.double(), 0.0)
    keep &= (w != 0)[:, None]
    p = torch.where(keep, torch.exp(logit - lse.double()[:, None]), 0.0)
    diag = torch.where(w != 0, torch.expm1(-loss.double()), 0.0)
    gu = w[:, None] / tau * (p @ v + diag[:, None] * v[:b])
    wp = w[:, None] * p
    gv = wp.T @ u
    gv[:b] += (w * diag)[:, None] * u
    gv /= tau
    gamma = d * R.U / (1 - d * R.U)
    x_err = gamma * u.norm(dim=1).max() * v.norm(dim=1).max() / tau \
        + 6 * R.U * (logit.abs().max() + torch.where(w != 0, lse.double().abs(), 0.0).max() + 10) + 2.0 ** -22
    rel = R.half_step(BF16) * (1 + 2.0 ** -7) + 1.1 * float(x_err)
    add_u, add_v = (nc / 16 + 64) * R.U, (b / 16 + 64) * R.U
    eu = w.abs()[:, None] / tau * ((rel + add_u) * (p @ v.abs()) + 8 * R.U * diag.abs()[:, None] * v[:b].abs())
    ev = (rel + add_v + 4 * R.U) * (wp.abs().T @ u.abs())
    ev[:b] += 8 * R.U * (w * diag).abs()[:, None] * u.abs()
    ev /= tau
    half = R.half_step(BF16)
    return (gu, gv), (eu + (gu.abs() + eu) * half, ev + (gv.abs() + ev) * half)


def _args(inp, use):
    return {"logq": inp["logq"] if "logq" in use else None, "item_ids": inp["item_ids"] if "ids" in use else None,
            "valid": inp["valid"] if "valid" in use else None}


def _check(inp, tau, use, grad_loss=None, grad_mean=1.0):
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], tau, **_args(inp, use))
    gm = None if grad_mean is None else torch.tensor(grad_mean, device="cuda")
    gu, gv = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, tau, grad_loss=grad_loss, grad_mean=gm,
                                        check=True, **_args(inp, use))
    b = inp["users"].shape[0]
    ok = inp["valid"][:b].bool() if "valid" in use else torch.ones(b, dtype=torch.bool, device="cuda")
    w = torch.zeros(b, dtype=torch.float64, device="cuda")
    if grad_loss is not None:
        w += grad_loss.double()
    if grad_mean is not None:
        w += grad_mean / max(1, int(ok.sum()))
    (wu, wv), (eu, ev) = reference(inp, tau, lse, loss, w, use)
    assert gu.dtype == gv.dtype == BF16
    R.close(gu, wu, eu + 1e-37, "grad_users")
    R.close(gv, wv, ev + 1e-37, "grad_items")
    return gu, gv


FULL = ("logq", "ids", "valid")


@pytest.mark.parametrize("over,use", [
    ({"b": 128, "nc": 128, "d": 64}, ()),
    ({"b": 1, "nc": 1, "d": 64}, ()),
    ({"b": 1, "nc": 300, "d": 64}, ("logq",)),
    ({"b": 129, "nc": 257, "d": 64, "catalogue": 50}, FULL),  # one row and one column past a tile
    ({"b": 384, "nc": 384, "d": 64, "catalogue": 500}, FULL),  # many accidental hits
    ({"b": 300, "nc": 1100, "d": 96, "catalogue": 3000}, FULL),
    ({"b": 500, "nc": 900, "d": 80}, ("logq", "valid")),
    ({"b": 640, "nc": 2000, "d": 112, "tau": 1.0}, ("logq",)),
    ({"b": 1000, "nc": 3000, "d": 128}, FULL),
    ({"b": 700, "nc": 705, "d": 144}, FULL),  # tiles of 64 columns
    ({"b": 400, "nc": 1300, "d": 192, "catalogue": 600}, FULL),
    ({"b": 257, "nc": 513, "d": 256}, FULL),
    ({"b": 200, "nc": 700, "d": 272, "catalogue": 400}, FULL),  # two halves, the second 16 wide
    ({"b": 300, "nc": 300, "d": 320}, ()),
    ({"b": 200, "nc": 700, "d": 384, "catalogue": 400}, FULL),
    ({"b": 130, "nc": 1000, "d": 448}, ("ids",)),
    ({"b": 200, "nc": 700, "d": 512, "catalogue": 400}, FULL),
    ({"b": 512, "nc": 512, "d": 64, "pad_rate": 0.3}, ("ids", "valid")),
    ({"b": 2048, "nc": 6000, "d": 64, "catalogue": 20}, FULL),  # groups of hundreds of rows
    ({"b": 3000, "nc": 3500, "d": 64, "zipf_s": 0.0}, FULL),
    ({"b": 64, "nc": 20000, "d": 64}, FULL),  # one row tile, its columns over the whole GPU
])
def test_every_row(over, use):
    _cuda()
    w = W.batch("inbatch_b8192_d64", oracle_rows=0, **over)
    _check(W.batch_inputs(w, "cuda"), w.tau, use)


def test_weights_per_row():
    """A gradient per loss row: any sign, zeros among them, with and without the mean's."""
    _cuda()
    w = W.batch("inbatch_b8192_d64", b=300, nc=700, d=64, catalogue=300)
    inp = W.batch_inputs(w, "cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    gl = torch.randn(300, generator=g, device="cuda")
    gl[::7] = 0.0
    _check(inp, w.tau, FULL, grad_loss=gl, grad_mean=None)
    _check(inp, w.tau, FULL, grad_loss=gl, grad_mean=-2.5)
    gu, gv = _check(inp, w.tau, FULL, grad_loss=torch.zeros(300, device="cuda"), grad_mean=None)
    assert bool((gu == 0).all()) and bool((gv == 0).all())


def test_padding_holds_anything():
    """What padded rows hold does not matter: NaN, infinities, any lse. Their gradients are zero."""
    _cuda()
    w = W.batch("inbatch_b8192_d64", b=400, nc=900, d=96, catalogue=300, pad_rate=0.2)
    inp = W.batch_inputs(w, "cuda")
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], w.tau, **_args(inp, FULL))
    one = torch.ones((), device="cuda")
    want = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, w.tau, grad_mean=one, **_args(inp, FULL))
    bad = ~inp["valid"].bool()
    users, items, lse2, loss2 = inp["users"].clone(), inp["items"].clone(), lse.clone(), loss.clone()
    users[bad[:400]] = float("nan")
    items[bad] = float("inf")
    lse2[bad[:400]] = float("nan")
    loss2[bad[:400]] = float("nan")
    lq = inp["logq"].clone()
    lq[bad] = float("nan")
    got = tt.tt_inbatch_softmax_grad(users, items, lse2, loss2, w.tau, grad_mean=one,
                                     **{**_args(inp, FULL), "logq": lq})
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert bool((got[0][bad[:400]] == 0).all()) and bool((got[1][bad] == 0).all())


@pytest.mark.parametrize("shift", [1, 4, 8, 16])
def test_masks_that_begin_anywhere(shift):
    """valid, logq and item_ids as views into longer tensors, at any element."""
    _cuda()
    w = W.batch("inbatch_b8192_d64", b=333, nc=700, d=64, catalogue=300, pad_rate=0.2)
    inp = W.batch_inputs(w, "cuda")
    for name in ("valid", "logq", "item_ids"):
        long = torch.zeros(700 + shift, dtype=inp[name].dtype, device="cuda")
        long[shift:] = inp[name]
        inp[name] = long[shift:]
    _check(inp, w.tau, FULL)


def test_edge_batches():
    _cuda()
    d = 64
    one = torch.ones((), device="cuda")
    none = torch.empty(0, device="cuda")
    u = torch.empty((0, d), dtype=BF16, device="cuda")
    v = torch.randn((5, d), device="cuda").to(BF16)
    gu, gv = tt.tt_inbatch_softmax_grad(u, v, none, none, 0.5, grad_mean=one, check=True)
    assert gu.shape == (0, d) and bool((gv == 0).all())
    gu, gv = tt.tt_inbatch_softmax_grad(u, v[:0], none, none, 0.5, grad_mean=one, check=True)
    assert gv.shape == (0, d)
    # every row invalid
    w = W.batch("inbatch_b8192_d64", b=70, nc=90, d=d)
    inp = W.batch_inputs(w, "cuda")
    inp["valid"] = torch.zeros(90, dtype=torch.bool, device="cuda")
    gu, gv = _check(inp, w.tau, FULL)
    assert bool((gu == 0).all()) and bool((gv == 0).all())
    # all columns hold one item: each row keeps only its own positive, and the loss is flat
    inp = W.batch_inputs(w, "cuda")
    inp["item_ids"] = torch.full((90,), 7, dtype=torch.int64, device="cuda")
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], w.tau, item_ids=inp["item_ids"])
    gu, gv = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], torch.zeros_like(lse), torch.zeros_like(loss), w.tau,
                                        item_ids=inp["item_ids"], grad_mean=one)
    assert bool((gu == 0).all()) and bool((gv == 0).all())
    # the id that marks a free slot of the library's table is an ordinary id
    inp["item_ids"] = torch.arange(90, device="cuda")
    inp["item_ids"][3] = inp["item_ids"][11] = -(2 ** 63)
    _check(inp, w.tau, FULL)


@pytest.mark.parametrize("tau", [0.01, 5.0])
def test_temperatures(tau):
    """A sharp softmax, where one column takes nearly all, and a flat one."""
    _cuda()
    w = W.batch("inbatch_b8192_d64", b=300, nc=600, d=64, catalogue=2000)
    inp = W.batch_inputs(w, "cuda")
    _check(inp, tau, FULL)


def test_against_differences():
    """sum(grad . v) against central differences of the mean loss in float64.
    Difference error: h^2 third derivatives (|u| <= 2, 1/tau = 2: below 1e-6)
    and 1e-15 / h."""
    _cuda()
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    b, nc, d, tau, h = 40, 70, 64, 0.5, 1e-4
    u = (torch.randn((b, d), generator=g, device="cuda") / 8).to(BF16)
    v = (torch.randn((nc, d), generator=g, device="cuda") / 8).to(BF16)
    ids = torch.randint(0, 30, (nc,), generator=g, device="cuda")
    valid = torch.rand(nc, generator=g, device="cuda") > 0.1
    logq = torch.randn(nc, generator=g, device="cuda")
    rows = torch.arange(b, device="cuda")
    keep = ((ids[:b, None] != ids[None, :]) | (rows[:, None] == torch.arange(nc, device="cuda")[None, :])) & valid[None, :]

    def mean_loss(u, v):
        logit = u @ v.T / tau - logq.double()
        lse = torch.logsumexp(logit.masked_fill(~keep, -math.inf), 1)
        return float((lse - logit[rows, rows])[valid[:b]].mean())

    lse, loss, _ = tt.tt_inbatch_softmax(u, v, tau, logq=logq, item_ids=ids, valid=valid)
    one = torch.ones((), device="cuda")
    grads = tt.tt_inbatch_softmax_grad(u, v, lse, loss, tau, logq=logq, item_ids=ids, valid=valid, grad_mean=one)
    inp = {"users": u, "items": v, "item_ids": ids, "valid": valid, "logq": logq}
    weight = torch.full((b,), 1.0 / int(valid[:b].sum()), dtype=torch.float64, device="cuda")
    _, bounds = reference(inp, tau, lse, loss, weight, FULL)
    for k in range(2):
        z = torch.randn(grads[k].shape, generator=g, device="cuda", dtype=torch.float64)
        at = [u.double(), v.double()]
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + h * z, at[k] - h * z
        diff = (mean_loss(*up) - mean_loss(*down)) / (2 * h)
        along = float((grads[k].double() * z).sum())
        # lse and loss are fp32: 1e-5 relative on what they scale
        tol = float((bounds[k] * z.abs()).sum()) + 1e-5 * float((grads[k].double() * z).abs().sum()) + 1e-6
        assert abs(along - diff) <= tol, (k, along, diff, tol)


def test_batch_of_8192_rows():
    """The whole batch: sampled rows and columns in float64, and the same bits on a second run."""
    _cuda()
    w = W.batch("inbatch_b8192_d64")
    inp = W.batch_inputs(w, "cuda")
    gu, gv = _check(inp, w.tau, FULL)
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], w.tau, **_args(inp, FULL))
    again = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, w.tau,
                                       grad_mean=torch.ones((), device="cuda"), **_args(inp, FULL))
    assert torch.equal(gu, again[0]) and torch.equal(gv, again[1])


def test_side_stream_and_graph():
    _cuda()
    w = W.batch("inbatch_b8192_d64", b=300, nc=700, d=64, catalogue=300)
    inp = W.batch_inputs(w, "cuda")
    args = _args(inp, FULL)
    one = torch.ones((), device="cuda")
    fwd = (torch.empty(300, device="cuda"), torch.empty(300, device="cuda"), torch.empty((), device="cuda"))
    grads = (torch.empty_like(inp["users"]), torch.empty_like(inp["items"]))
    ws_f = torch.empty(tt.tt_inbatch_softmax_workspace(300, 700, 64, True), dtype=torch.uint8, device="cuda")
    ws_b = torch.empty(tt.tt_inbatch_softmax_grad_workspace(300, 700, 64, True, True), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        tt.tt_inbatch_softmax(inp["users"], inp["items"], w.tau, workspace=ws_f, out=fwd, check=False, stream=stream, **args)
        tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], fwd[0], fwd[1], w.tau, grad_mean=one, workspace=ws_b,
                                   out=grads, stream=stream, **args)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    inp["users"].copy_(W.batch_inputs(W.batch("inbatch_b8192_d64", b=300, nc=700, d=64, seed=5), "cuda")["users"])
    ws_f.fill_(255)
    ws_b.fill_(255)
    graph.replay()
    torch.cuda.synchronize()
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], w.tau, **args)
    want = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, w.tau, grad_mean=one, **args)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_memory_made_for_another_stream():
    """A call on a stream of its own: the workspace it makes is not handed out
    again on the current stream while its kernels still use it."""
    _cuda()
    w = W.batch("inbatch_b8192_d64", b=2000, nc=4000, d=128, catalogue=300)
    inp = W.batch_inputs(w, "cuda")
    args = _args(inp, FULL)
    one = torch.ones((), device="cuda")
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], w.tau, **args)
    want = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, w.tau, grad_mean=one, **args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    need = tt.tt_inbatch_softmax_grad_workspace(2000, 4000, 128, True, True)
    for _ in range(10):
        got = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, w.tau, grad_mean=one, stream=side, **args)
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)  # on the current stream, at once
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals():
    _cuda()
    u = torch.randn((8, 64), device="cuda").to(BF16)
    v = torch.randn((6, 64), device="cuda").to(BF16)
    s = torch.zeros(8, device="cuda")
    one = torch.ones((), device="cuda")
    with pytest.raises(tt.TTError) as err:  # nc < b
        tt.tt_inbatch_softmax_grad(u, v, s, s, 1.0, grad_mean=one)
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        tt.tt_inbatch_softmax_grad(u, u.clone(), s, s, 1.0)  # no gradient given
    with pytest.raises(TypeError):
        tt.tt_inbatch_softmax_grad(u, u.clone(), s.double(), s, 1.0, grad_mean=one)
    with pytest.raises(ValueError):
        tt.tt_inbatch_softmax_grad(u, u.clone(), s[:7], s, 1.0, grad_mean=one)
    with pytest.raises(tt.TTError) as err:  # fp32 rows: cast to bf16 first
        tt.tt_inbatch_softmax_grad(u.float(), u.float(), s, s, 1.0, grad_mean=one)
    assert err.value.status == tt.TT_ERR_UNSUPPORTED
    with pytest.raises(tt.TTError) as err:
        tt.tt_inbatch_softmax_grad(u, u.clone(), s, s, 0.0, grad_mean=one)
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(tt.TTError) as err:  # the gradient over its input
        tt.tt_inbatch_softmax_grad(u, u.clone(), s, s, 1.0, grad_mean=one, out=(u, torch.empty_like(u)))
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(tt.TTError) as err:
        tt.tt_inbatch_softmax_grad(u, u.clone(), s, s, 1.0, grad_mean=one,
                                   workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.status == tt.TT_ERR_INVALID_ARG

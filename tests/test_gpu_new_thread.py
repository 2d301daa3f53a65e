"""Calls whose host thread has not used CUDA before: the first call of a worker
thread of a data loader or a server. (GPU)"""
import threading

import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

BF16 = torch.bfloat16


def _in_new_thread(call):
    errors = []

    def work():
        try:
            call()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert errors == []


def _like(tensors):
    return tuple(torch.zeros_like(t) for t in tensors)


def test_in_batch_loss():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    inp = W.batch_inputs(W.batch("inbatch_b8192_d64", b=130, nc=200, d=64, catalogue=300), "cuda")
    args = {k: inp[k] for k in ("logq", "item_ids", "valid")}
    want = tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.1, **args)
    out = _like(want)
    ws = torch.empty(tt.tt_inbatch_softmax_workspace(130, 200, 64, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _in_new_thread(lambda: tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.1, workspace=ws, out=out, check=False, **args))
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    one = torch.ones((), device="cuda")
    want_g = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], want[0], want[1], 0.1, grad_mean=one, **args)
    out_g = _like(want_g)
    ws_g = torch.empty(tt.tt_inbatch_softmax_grad_workspace(130, 200, 64, True, True), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    _in_new_thread(lambda: tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], want[0], want[1], 0.1, grad_mean=one,
                                                      workspace=ws_g, out=out_g, **args))
    assert all(torch.equal(a, b) for a, b in zip(out_g, want_g))


@pytest.mark.parametrize("b", [1, 48, 300])
def test_search(b):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda")
    g.manual_seed(b)
    index = tt.tt_index_wrap(torch.randn((40_000, 64), generator=g, device="cuda").to(BF16))
    queries = torch.randn((b, 64), generator=g, device="cuda").to(BF16)
    want = tt.tt_score_topk(index, queries, 20)
    out = _like(want)
    torch.cuda.synchronize()
    _in_new_thread(lambda: tt.tt_score_topk(index, queries, 20, out_ids=out[0], out_scores=out[1]))
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_rows_and_lists():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.randn((50, 96), device="cuda")
    ids = torch.randint(0, 50, (200,), device="cuda")
    norm_out = torch.zeros((), device="cuda")
    want = tt.tt_layernorm(x)
    out = _like(want)
    rows = torch.zeros((200, 96), device="cuda")
    torch.cuda.synchronize()

    def call():
        tt.tt_grad_norm([x, rows[:0]], norm=norm_out, workspace=ws)
        tt.tt_layernorm(x, out=out)
        tt.tt_embedding(x, ids, out=rows)

    ws = torch.empty(tt.tt_clip_grad_norm_workspace([x, rows[:0]]), dtype=torch.uint8, device="cuda")
    _in_new_thread(call)
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(rows, x[ids])
    assert abs(float(norm_out) - float(x.double().norm())) <= 1e-5 * float(norm_out)

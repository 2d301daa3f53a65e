"""The in-batch gradient's copies of padded batches: calls right behind one
another in one workspace, with other rows and other padding each time. (GPU)"""
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")


@pytest.mark.parametrize("b,nc,d", [(300, 700, 64), (2000, 4000, 128), (200, 500, 320)])
def test_calls_in_one_workspace(b, nc, d):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    one = torch.ones((), device="cuda")
    ws = torch.empty(tt.tt_inbatch_softmax_grad_workspace(b, nc, d, True, True), dtype=torch.uint8, device="cuda")
    calls, want = [], []
    for seed in range(6):
        inp = W.batch_inputs(W.batch("inbatch_b8192_d64", b=b, nc=nc, d=d, catalogue=300, pad_rate=0.3, seed=seed), "cuda")
        args = {k: inp[k] for k in ("logq", "item_ids", "valid")}
        lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.2, **args)
        calls.append(lambda inp=inp, args=args, lse=lse, loss=loss: tt.tt_inbatch_softmax_grad(
            inp["users"], inp["items"], lse, loss, 0.2, grad_mean=one, workspace=ws, **args))
        torch.cuda.synchronize()
        ws.fill_(255)
        want.append(calls[-1]())
        torch.cuda.synchronize()
    for _ in range(5):
        got = [call() for call in calls]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])

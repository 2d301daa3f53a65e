"""The in-batch loss on a stream of its own, without a wait: the workspace that
the call makes is not handed out again on the current stream while its kernels
still use it. (GPU)"""
import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")


def test_workspace_stays_with_the_call():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    b, nc, d = 4000, 8000, 128
    inp = W.batch_inputs(W.batch("inbatch_b8192_d64", b=b, nc=nc, d=d, catalogue=3000), "cuda")
    args = {k: inp[k] for k in ("logq", "item_ids", "valid")}
    want = tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.1, **args)
    need = tt.tt_inbatch_softmax_workspace(b, nc, d, True)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        got = tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.1, stream=side, check=False, **args)
        torch.empty(need, dtype=torch.uint8, device="cuda").fill_(255)  # on the current stream, at once
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))

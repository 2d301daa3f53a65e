"""Training calls of two host threads at once, at different widths, each with a
stream and a workspace of its own. (GPU)

The kernels' shared memory grows with the width; a call must not take back what
another thread's call has just asked for."""
import threading

import pytest
import torch

import workloads as W

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

CALLS = 400


def _at_once(calls):
    """Run the calls, each CALLS times in a thread of its own; the errors."""
    errors = []
    start = threading.Barrier(len(calls))

    def work(call):
        stream = torch.cuda.Stream()
        try:
            start.wait()
            for _ in range(CALLS):
                call(stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return errors


@pytest.mark.parametrize("widths", [(64, 128), (256, 192), (320, 512)])
def test_in_batch_loss_and_gradient(widths):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    calls, checks = [], []
    for d in widths:
        inp = W.batch_inputs(W.batch("inbatch_b8192_d64", b=130, nc=200, d=d, catalogue=300), "cuda")
        args = {k: inp[k] for k in ("logq", "item_ids", "valid")}
        one = torch.ones((), device="cuda")
        want_f = tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.1, **args)
        want_b = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], want_f[0], want_f[1], 0.1, grad_mean=one, **args)
        fwd, bwd = tuple(map(torch.empty_like, want_f)), tuple(map(torch.empty_like, want_b))
        ws_f = torch.empty(tt.tt_inbatch_softmax_workspace(130, 200, d, True), dtype=torch.uint8, device="cuda")
        ws_b = torch.empty(tt.tt_inbatch_softmax_grad_workspace(130, 200, d, True, True), dtype=torch.uint8, device="cuda")

        def call(stream, inp=inp, args=args, one=one, fwd=fwd, bwd=bwd, ws_f=ws_f, ws_b=ws_b):
            tt.tt_inbatch_softmax(inp["users"], inp["items"], 0.1, workspace=ws_f, out=fwd, check=False, stream=stream, **args)
            tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], fwd[0], fwd[1], 0.1, grad_mean=one, workspace=ws_b,
                                       out=bwd, stream=stream, **args)

        calls.append(call)
        checks.append((fwd + bwd, want_f + want_b))
    torch.cuda.synchronize()
    assert _at_once(calls) == []
    for got, want in checks:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("widths", [(5001, 9001), (1031, 16383)])
def test_layer_norm(widths):
    """Widths that are no multiple of 8 keep their weights in shared memory."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    calls, checks = [], []
    for d in widths:
        x = torch.randn((40, d), device="cuda")
        w, bias, dy = torch.randn(d, device="cuda"), torch.randn(d, device="cuda"), torch.randn((40, d), device="cuda")
        want = tt.tt_layernorm(x, w, bias)
        want_g = tt.tt_layernorm_grad(dy, x, w, want[1], want[2])
        out, out_g = tuple(map(torch.empty_like, want)), tuple(map(torch.empty_like, want_g))
        ws = torch.empty(tt.tt_layernorm_grad_workspace(40, d), dtype=torch.uint8, device="cuda")

        def call(stream, x=x, w=w, bias=bias, dy=dy, out=out, out_g=out_g, ws=ws):
            tt.tt_layernorm(x, w, bias, out=out, stream=stream)
            tt.tt_layernorm_grad(dy, x, w, out[1], out[2], out=out_g, workspace=ws, stream=stream)

        calls.append(call)
        checks.append((out + out_g, want + want_g))
    torch.cuda.synchronize()
    assert _at_once(calls) == []
    for got, want in checks:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_searches():
    """Two handles, one per thread, at different widths: the tensor-core search and
    the streaming one with its sampled threshold."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    calls, checks = [], []
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for d in (64, 384):
        rows = torch.randn((40_000, d), generator=g, device="cuda").to(torch.bfloat16)
        index = tt.tt_index_wrap(rows)
        many = torch.randn((48, d), generator=g, device="cuda").to(torch.bfloat16)
        few = torch.randn((1, d), generator=g, device="cuda")
        want = [tt.tt_score_topk(index, q, 20) for q in (many, few)]
        out = [tuple(map(torch.empty_like, x)) for x in want]

        def call(stream, index=index, many=many, few=few, out=out):
            tt.tt_score_topk(index, many, 20, out_ids=out[0][0], out_scores=out[0][1], stream=stream)
            tt.tt_score_topk(index, few, 20, out_ids=out[1][0], out_scores=out[1][1], stream=stream)

        calls.append(call)
        checks.append((out[0] + out[1], want[0] + want[1]))
    torch.cuda.synchronize()
    assert _at_once(calls) == []
    for got, want in checks:
        assert all(torch.equal(a, b) for a, b in zip(got, want))

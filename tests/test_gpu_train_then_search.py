"""A search right behind a training call, on its outputs: as queries, and as the
corpus. The search's kernels start early and read their rows before they wait for
one another, but not before the training call's writes. (GPU)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

BF16 = torch.bfloat16


def _check(index, queries, write, inputs):
    """For each input: the call and the search one after the other on the stream,
    against the same with a wait between them."""
    want = []
    for x in inputs:
        write(x)
        torch.cuda.synchronize()
        want.append(tt.tt_score_topk(index, queries, 10))
        torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for x in inputs:
            write(x)
            got.append(tt.tt_score_topk(index, queries, 10))
        torch.cuda.synchronize()
        for (gi, gs), (wi, ws) in zip(got, want):
            assert torch.equal(gi, wi) and torch.equal(gs, ws)


@pytest.mark.parametrize("dtype", [BF16, torch.int8])
@pytest.mark.parametrize("n", [200_000, 1_000_000])
@pytest.mark.parametrize("b", [1, 2])
def test_gradient_rows_as_queries(n, b, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda")
    g.manual_seed(n + b)
    d, m, nc = 64, 300, 700
    raw = torch.randn((n, d), generator=g, device="cuda")
    if dtype == BF16:
        index = tt.tt_normalize_candidates(raw, torch.empty((n, d), dtype=BF16, device="cuda"))
    else:
        index = tt.tt_quantize_candidates(raw, torch.empty((n, d), dtype=torch.int8, device="cuda"),
                                          torch.empty(n, device="cuda"))
    one = torch.ones((), device="cuda")
    out = (torch.empty((m, d), dtype=BF16, device="cuda"), torch.empty((nc, d), dtype=BF16, device="cuda"))
    ws = torch.empty(tt.tt_inbatch_softmax_grad_workspace(m, nc, d, False, False), dtype=torch.uint8, device="cuda")
    inputs = []
    for _ in range(6):
        u, v = (torch.randn((k, d), generator=g, device="cuda").to(BF16) for k in (m, nc))
        lse, loss, _ = tt.tt_inbatch_softmax(u, v, 4.0)
        inputs.append((u, v, lse, loss))

    def write(x):
        tt.tt_inbatch_softmax_grad(*x, tau=4.0, grad_mean=one, workspace=ws, out=out)

    _check(index, out[0][m - b:], write, inputs)


@pytest.mark.parametrize("m", [3, 200, 256, 257, 2000])
def test_embedding_gradient_as_queries_and_as_corpus(m):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda")
    g.manual_seed(m)
    d, rows = 64, 100_000
    corpus = torch.randn((1_000_000, d), generator=g, device="cuda").to(BF16)
    table, by_row = torch.zeros((rows, d), device="cuda"), (torch.zeros(m, dtype=torch.int64, device="cuda"),
                                                             torch.zeros((m, d), device="cuda"))
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(tt.tt_embedding_grad_workspace(m, rows, d), dtype=torch.uint8, device="cuda")
    inputs = [(torch.randperm(rows, generator=g, device="cuda")[:m], torch.randn((m, d), generator=g, device="cuda"))
              for _ in range(6)]
    _check(tt.tt_index_wrap(corpus), by_row[1][:1],
           lambda x: tt.tt_embedding_grad_rows(*x, rows, out=by_row, count=count, workspace=ws), inputs)
    _check(tt.tt_index_wrap(table), torch.randn((1, d), generator=g, device="cuda"),
           lambda x: tt.tt_embedding_grad(*x, rows, out=table, workspace=ws), inputs)

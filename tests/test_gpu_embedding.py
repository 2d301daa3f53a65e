"""Embedding lookup and its gradient by sorted ids on the GPU against
float64. (GPU)

Bounds: the lookup is one fp32 product and one rounding. A row of the gradient
is a sum along chains of at most 32 tokens, then 64 partial rows (or m / 256
of them and 8 warps), then one product: (D + 2) U sum|g|, and one rounding."""
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("d", [1, 3, 8, 10, 16, 33, 64, 96, 128, 200, 257, 512, 1000, 4096, 16384])
@pytest.mark.parametrize("dtype,out_dtype,idt", [(F32, F32, I64), (BF16, BF16, I32), (BF16, F32, I64), (F32, BF16, I32)])
def test_lookup(d, dtype, out_dtype, idt):
    _cuda()
    g = _gen(d)
    rows, m = 77, 131
    table = torch.randn((rows, d), generator=g, device="cuda").to(dtype)
    table[5] = float("inf")
    ids = torch.randint(-2, rows + 2, (m,), generator=g, device="cuda").to(idt)  # some outside the table
    ids[:3] = torch.tensor([0, rows - 1, -1])
    got = tt.tt_embedding(table, ids, scale=1.5, out_dtype=out_dtype)
    inside = (ids >= 0) & (ids < rows)
    want = torch.where(inside[:, None], table[ids.long().clamp(0, rows - 1)].double() * 1.5, 0.0)
    assert got.dtype == out_dtype
    R.close(got, want, want.abs().nan_to_num(posinf=0.0) * (R.U + R.half_step(out_dtype) * 1.001), "rows")


def test_lookup_shapes_and_far_rows():
    _cuda()
    # any shape of ids; offsets past 2^31 elements
    rows, d = (1 << 22) + 3, 512
    table = torch.zeros((rows, d), dtype=BF16, device="cuda")
    table[-1], table[1 << 22] = 2.0, 3.0
    ids = torch.tensor([[rows - 1, 0], [1 << 22, -1], [-(1 << 40), 1 << 40]], device="cuda")
    got = tt.tt_embedding(table, ids)
    assert got.shape == (3, 2, d)
    assert [float(v) for v in got[..., 7].flatten()] == [2.0, 0.0, 3.0, 0.0, 0.0, 0.0]
    assert tt.tt_embedding(table, ids[:0]).shape == (0, 2, d)
    empty = torch.empty((0, 16), device="cuda")
    assert bool((tt.tt_embedding(empty, ids) == 0).all())  # a table without rows: every id is outside


def test_lookup_of_search_results():
    """The rows of a search's ids, with its padding (fewer eligible rows than k)."""
    _cuda()
    g = _gen(1)
    corpus = torch.randn((50, 64), generator=g, device="cuda")
    index = tt.tt_normalize_candidates(corpus, torch.empty((50, 64), device="cuda"))
    ids, scores = tt.tt_score_topk(index, index.rows[:3].contiguous(), 60)
    got = tt.tt_embedding(index.rows, ids)
    assert bool((ids[:, 50:] == -1).all()) and bool((got[:, 50:] == 0).all())
    again = (got[:, :50].double() * index.rows[:3, None].double()).sum(-1)
    assert float((again - scores[:, :50].double()).abs().max()) < 1e-5


def _grad_ref(ids, grad, rows, scale):
    inside = (ids >= 0) & (ids < rows)
    at = torch.where(inside, ids, 0).long().flatten()
    g = torch.where(inside.flatten()[:, None], grad.reshape(-1, grad.shape[-1]).double(), 0.0)
    want = torch.zeros((rows, g.shape[1]), dtype=torch.float64, device="cuda").index_add_(0, at, g) * scale
    mag = torch.zeros_like(want).index_add_(0, at, g.abs()) * abs(scale)
    D = 32 + 64 + ids.numel() / 256 + 8
    return want, (D + 2) * R.U * mag


def _check_grad(ids, grad, rows, scale, out_dtype):
    want, tol = _grad_ref(ids, grad, rows, scale)
    tol = tol + (want.abs() + tol) * R.half_step(out_dtype)
    got = tt.tt_embedding_grad(ids, grad, rows, scale=scale, out_dtype=out_dtype)
    assert got.dtype == out_dtype
    R.close(got, want, tol, "dense")
    m, d = ids.numel(), grad.shape[-1]
    flat = ids.flatten()
    present = torch.unique(flat[(flat >= 0) & (flat < rows)])
    n = present.numel()
    out_ids = torch.full((m,), -77, dtype=ids.dtype, device="cuda")
    out_rows = torch.full((m, d), -77.0, dtype=out_dtype, device="cuda")
    _, _, count = tt.tt_embedding_grad_rows(ids, grad, rows, scale=scale, out=(out_ids, out_rows))
    assert int(count) == n
    assert torch.equal(out_ids[:n], present) and bool((out_ids[n:] == -77).all())
    assert bool((out_rows[n:] == -77).all())
    assert torch.equal(out_rows[:n], got[present.long()])  # both forms add in the same order
    return got


@pytest.mark.parametrize("d", [1, 2, 3, 12, 32, 33, 64, 96, 100, 128, 200, 257, 512, 1000])
@pytest.mark.parametrize("dtype,out_dtype,idt", [(F32, F32, I64), (BF16, F32, I32), (BF16, BF16, I64), (F32, BF16, I32)])
def test_gradient_widths(d, dtype, out_dtype, idt):
    _cuda()
    g = _gen(d + 100)
    rows, m = 23, 301
    ids = torch.randint(-1, rows, (m,), generator=g, device="cuda").to(idt)
    grad = torch.randn((m, d), generator=g, device="cuda").to(dtype)
    _check_grad(ids, grad, rows, 0.5, out_dtype)


@pytest.mark.parametrize("d", [1001, 2049, 4096, 8190, 16383, 16384])
@pytest.mark.parametrize("dtype,out_dtype", [(F32, F32), (BF16, BF16)])
def test_wide_rows(d, dtype, out_dtype):
    _cuda()
    g = _gen(d)
    rows, m = 19, 300
    ids = torch.randint(-1, rows, (m,), generator=g, device="cuda")
    grad = torch.randn((m, d), generator=g, device="cuda").to(dtype)
    _check_grad(ids, grad, rows, 1.0, out_dtype)
    table = torch.randn((rows, d), generator=g, device="cuda").to(dtype)
    want = torch.where((ids >= 0)[:, None], table[ids.clamp(min=0)], torch.zeros((), dtype=dtype, device="cuda"))
    assert torch.equal(tt.tt_embedding(table, ids), want)


# one token, one warp-chunk and one more, a block's sort and one more, tiles of the larger sort
LENGTHS = [1, 2, 31, 32, 33, 64, 255, 1023, 1025, 4096, 4097, 16383, 16384, 16385, 20480, 40001]


@pytest.mark.parametrize("m,rows", [(m, r) for r in (1, 2, 255, 256, 257, 70_000) for m in LENGTHS]
                         + [(m, (1 << 24) + 1) for m in (33, 16384, 40001)])
def test_gradient_sizes(m, rows):
    _cuda()
    g = _gen(m * 7 + rows % 1000)
    u = torch.rand(m, generator=g, device="cuda", dtype=torch.float64)
    ids = ((rows + 1) ** u - 1).long().clamp(0, rows - 1)  # popular low ids: long and short runs
    ids[torch.rand(m, generator=g, device="cuda") < 0.05] = -1
    grad = torch.randn((m, 8), generator=g, device="cuda")
    _check_grad(ids, grad, rows, 1.0, F32)


@pytest.mark.parametrize("kind", ["one id", "two ids", "all outside", "all differ", "runs of 32", "runs of 33"])
@pytest.mark.parametrize("m", [500, 70_000])
def test_gradient_runs(kind, m):
    _cuda()
    g = _gen(m)
    rows = m + 5
    t = torch.arange(m, device="cuda")
    ids = {"one id": torch.full((m,), 3, device="cuda"), "two ids": 1 + (t % 2) * (rows - 2),
           "all outside": torch.where(t % 2 == 0, -1, rows), "all differ": torch.randperm(m, generator=g, device="cuda"),
           "runs of 32": t // 32, "runs of 33": (m - 1 - t) // 33}[kind]
    grad = torch.randn((m, 20), generator=g, device="cuda")
    grad[(ids < 0) | (ids >= rows)] = float("nan")  # rows that no id points to are not read
    got = _check_grad(ids, grad.nan_to_num(0.0), rows, 2.0, F32)
    same = tt.tt_embedding_grad(ids, grad, rows, scale=2.0)
    assert torch.equal(same, got)
    assert torch.equal(tt.tt_embedding_grad(ids, grad, rows, scale=2.0), same)  # the same bits on every run


def test_gradient_no_tokens_and_no_rows():
    _cuda()
    ids = torch.empty(0, dtype=I64, device="cuda")
    grad = torch.empty((0, 24), device="cuda")
    assert bool((tt.tt_embedding_grad(ids, grad, 7) == 0).all())
    assert int(tt.tt_embedding_grad_rows(ids, grad, 7)[2]) == 0
    ids = torch.tensor([0, 3, -1], device="cuda")
    assert tt.tt_embedding_grad(ids, torch.ones((3, 24), device="cuda"), 0).shape == (0, 24)
    assert int(tt.tt_embedding_grad_rows(ids, torch.ones((3, 24), device="cuda"), 0)[2]) == 0


def test_gradient_against_differences():
    """The lookup is linear in the table: (f(T + h v) - f(T - h v)) / 2h in float64 is its derivative."""
    _cuda()
    g = _gen(8)
    rows, m, d = 9, 40, 16
    ids = torch.randint(-1, rows, (3, m), generator=g, device="cuda")
    dy = torch.randn((3, m, d), generator=g, device="cuda")
    table = torch.randn((rows, d), generator=g, device="cuda", dtype=torch.float64)
    v = torch.randn((rows, d), generator=g, device="cuda", dtype=torch.float64)

    def loss(t):
        return float((dy.double() * torch.where((ids >= 0)[..., None], t[ids.clamp(min=0)] * 3.0, 0.0)).sum())

    diff = (loss(table + 1e-3 * v) - loss(table - 1e-3 * v)) / 2e-3
    grad = tt.tt_embedding_grad(ids, dy, rows, scale=3.0)
    _, tol = _grad_ref(ids, dy, rows, 3.0)
    assert abs(float((grad.double() * v).sum()) - diff) <= float(((tol + R.U * grad.double().abs()) * v.abs()).sum()) + 1e-8


def test_catalogue_scale():
    """A million tokens over ten million rows, three digits, long popular runs."""
    _cuda()
    g = _gen(77)
    rows, m, d = 10_000_000, 1_000_003, 16
    u = torch.rand(m, generator=g, device="cuda", dtype=torch.float64)
    ids = ((rows + 1) ** u - 1).long().clamp(0, rows - 1)
    grad = torch.randn((m, d), generator=g, device="cuda").to(BF16)
    _check_grad(ids, grad, rows, 1.0, F32)


def test_side_stream_and_graph():
    _cuda()
    g = _gen(31)
    rows, m, d = 5000, 20_000, 40
    table = torch.randn((rows, d), generator=g, device="cuda")
    ids = torch.randint(0, rows, (m,), generator=g, device="cuda")
    dy = torch.randn((m, d), generator=g, device="cuda")
    look, dense = torch.empty((m, d), device="cuda"), torch.empty((rows, d), device="cuda")
    by_row = (torch.zeros(m, dtype=I64, device="cuda"), torch.zeros((m, d), device="cuda"))
    count = torch.zeros(1, dtype=I32, device="cuda")
    ws = torch.empty(tt.tt_embedding_grad_workspace(m, rows, d), dtype=torch.uint8, device="cuda")

    def call(stream=None):
        tt.tt_embedding(table, ids, out=look, stream=stream)
        tt.tt_embedding_grad(ids, dy, rows, out=dense, workspace=ws, stream=stream)
        tt.tt_embedding_grad_rows(ids, dy, rows, out=by_row, count=count, workspace=ws, stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    ids.copy_(torch.randint(-1, 50, (m,), generator=g, device="cuda"))
    ws.fill_(255)
    graph.replay()
    assert torch.equal(look, tt.tt_embedding(table, ids))
    assert torch.equal(dense, tt.tt_embedding_grad(ids, dy, rows))
    n = int(count)
    assert n == 50 and torch.equal(by_row[0][:n], torch.arange(n, device="cuda"))
    assert torch.equal(by_row[1][:n], dense[:n])


def test_refusals():
    _cuda()
    table = torch.randn((10, 16), device="cuda")
    ids = torch.zeros(4, dtype=I64, device="cuda")
    with pytest.raises(TypeError):
        tt.tt_embedding(table.half(), ids)
    with pytest.raises(TypeError):
        tt.tt_embedding(table, ids.to(torch.int16))
    with pytest.raises(ValueError):
        tt.tt_embedding(table.t(), ids)
    with pytest.raises(ValueError):
        tt.tt_embedding(table, ids.cpu())
    with pytest.raises(ValueError):
        tt.tt_embedding(table, ids, out=torch.empty((4, 15), device="cuda"))
    with pytest.raises(tt.TTError) as err:
        tt.tt_embedding(table, ids, scale=float("nan"))
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        tt.tt_embedding_grad(ids, torch.empty((5, 16), device="cuda"), 10)
    with pytest.raises(tt.TTError) as err:
        tt.tt_embedding_grad(ids, torch.empty((4, 16), device="cuda"), 10,
                             workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(tt.TTError):
        tt.tt_embedding_grad_workspace(4, 10, 20000)

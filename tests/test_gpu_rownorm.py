"""Layer norm, its gradient and the gradient of the L2 normalisation on the
GPU against float64 forms, with bounds that count roundings. (GPU)"""
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

F32, BF16 = torch.float32, torch.bfloat16


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, n, d, dtype, spread=True):
    x = torch.randn((n, d), generator=g, device="cuda")
    if spread:
        x = x * torch.exp(torch.randn((n, 1), generator=g, device="cuda")) + 2 * torch.randn((n, 1), generator=g,
                                                                                             device="cuda")
    return x.to(dtype)


# every way a row is laid on threads: groups of 8, 16 and 32 lanes, several chunks
# per lane, blocks of 256 and 512 threads; multiples of 8 and odd widths
WIDTHS = [1, 2, 3, 7, 8, 16, 24, 31, 33, 64, 96, 127, 128, 200, 256, 257, 504, 512, 513, 1000, 1024, 1032, 1500, 2048,
          2049, 4096, 5000, 8191, 8192, 8200, 12345, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype,wdtype", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
def test_layernorm_and_gradient(d, dtype, wdtype):
    _cuda()
    g = _gen(d * 4 + (dtype == BF16))
    n = 45 if d < 2000 else 5
    x, dy = _rows(g, n, d, dtype), _rows(g, n, d, dtype, spread=False)
    w = (1 + 0.5 * torch.randn(d, generator=g, device="cuda")).to(wdtype)
    bias = torch.randn(d, generator=g, device="cuda").to(wdtype)
    eps = 1e-5
    y, mean, rstd = tt.tt_layernorm(x, w, bias, eps)
    (y8, m8, r8), (ey, em, er) = R.layernorm(x, w, bias, eps)
    assert y.dtype == dtype and mean.dtype == rstd.dtype == F32
    R.close(y, y8, ey + (y8.abs() + ey) * R.half_step(dtype), "y")
    R.close(mean, m8, em, "mean")
    R.close(rstd, r8, er, "rstd")
    gx, gw, gb = tt.tt_layernorm_grad(dy, x, w, mean, rstd)
    (x8, w8, b8), (ex, ew, eb) = R.layernorm_grad(dy, x, w, mean, rstd)
    R.close(gx, x8, ex + (x8.abs() + ex) * R.half_step(dtype), "grad_x")
    R.close(gw, w8, ew, "grad_w")
    R.close(gb, b8, eb, "grad_bias")


@pytest.mark.parametrize("n,d", [(1, 64), (7, 96), (8, 256), (9, 256), (2500, 40), (5000, 64), (20011, 128), (3001, 1000),
                                 (1200, 2048), (700, 2049)])
def test_layernorm_many_rows(n, d):
    """Several rows per lane group and per block, and a last block that is not full."""
    _cuda()
    g = _gen(n)
    x, dy = _rows(g, n, d, BF16), _rows(g, n, d, BF16, spread=False)
    w = (1 + 0.5 * torch.randn(d, generator=g, device="cuda"))
    y, mean, rstd = tt.tt_layernorm(x, w, None, 1e-5)
    (y8, _, _), (ey, _, _) = R.layernorm(x, w, None, 1e-5)
    R.close(y, y8, ey + (y8.abs() + ey) * R.half_step(BF16), "y")
    got = tt.tt_layernorm_grad(dy, x, w, mean, rstd)
    want, tol = R.layernorm_grad(dy, x, w, mean, rstd)
    R.close(got[0], want[0], tol[0] + (want[0].abs() + tol[0]) * R.half_step(BF16), "grad_x")
    R.close(got[1], want[1], tol[1], "grad_w")
    R.close(got[2], want[2], tol[2], "grad_bias")
    again = tt.tt_layernorm_grad(dy, x, w, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, again))  # the same bits on every run


@pytest.mark.parametrize("n,d", [(2000, 1536), (1999, 2401), (2600, 1033), (700, 4097), (450, 8192), (310, 12288), (5, 16378),
                                 (301, 16383)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_layernorm_wide_rows(n, d, dtype):
    """Several rows per team of warps, one to three teams per block, and the
    widest rows that do not begin on 16 bytes; also without weights."""
    _cuda()
    g = _gen(n + d)
    x, dy = _rows(g, n, d, dtype), _rows(g, n, d, dtype, spread=False)
    w = (1 + 0.5 * torch.randn(d, generator=g, device="cuda"))
    y, mean, rstd = tt.tt_layernorm(x, w, None, 1e-5)
    (y8, _, _), (ey, _, _) = R.layernorm(x, w, None, 1e-5)
    R.close(y, y8, ey + (y8.abs() + ey) * R.half_step(dtype), "y")
    for weights in (w, None):
        got = tt.tt_layernorm_grad(dy, x, weights, mean, rstd)
        want, tol = R.layernorm_grad(dy, x, weights, mean, rstd)
        R.close(got[0], want[0], tol[0] + (want[0].abs() + tol[0]) * R.half_step(dtype), "grad_x")
        R.close(got[1], want[1], tol[1], "grad_w")
        R.close(got[2], want[2], tol[2], "grad_bias")
    sums = tt.tt_layernorm_grad(dy, x, None, mean, rstd, out=(None, torch.empty_like(got[1]), torch.empty_like(got[2])))
    assert torch.equal(sums[1], got[1]) and torch.equal(sums[2], got[2])


def test_layernorm_without_weights_and_parts():
    _cuda()
    g = _gen(3)
    x, dy = _rows(g, 33, 200, F32), _rows(g, 33, 200, F32, spread=False)
    y, mean, rstd = tt.tt_layernorm(x)
    (y8, _, _), (ey, _, _) = R.layernorm(x, None, None, 1e-5)
    R.close(y, y8, ey + y8.abs() * R.U, "y")
    whole = tt.tt_layernorm_grad(dy, x, None, mean, rstd)
    want, tol = R.layernorm_grad(dy, x, None, mean, rstd)
    R.close(whole[0], want[0], tol[0] + want[0].abs() * R.U, "grad_x")
    # only some of the outputs: the same bits, the others untouched
    only = tt.tt_layernorm_grad(dy, x, None, mean, rstd, out=(None, torch.empty_like(whole[1]), None))
    assert only[0] is None and only[2] is None and torch.equal(only[1], whole[1])
    only = tt.tt_layernorm_grad(dy, x, None, mean, rstd, out=(torch.empty_like(x), None, None))
    assert torch.equal(only[0], whole[0])


def test_layernorm_no_rows():
    _cuda()
    x = torch.empty((0, 96), device="cuda")
    y, mean, rstd = tt.tt_layernorm(x)
    assert y.shape == (0, 96) and mean.numel() == rstd.numel() == 0
    gx, gw, gb = tt.tt_layernorm_grad(x, x, None, mean, rstd)
    assert gx.shape == (0, 96) and bool((gw == 0).all()) and bool((gb == 0).all())


def test_layernorm_special_rows():
    """A constant row has xhat = 0; a large mean loses nothing but what the
    input lost; NaN and infinity stay in their row (and in the column sums)."""
    _cuda()
    g = _gen(9)
    x = torch.randn((6, 64), generator=g, device="cuda")
    x[0] = 3.0
    x[1] += 4096.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    y, mean, rstd = tt.tt_layernorm(x, eps=1e-5)
    ok = [0, 1, 4, 5]
    (y8, m8, r8), (ey, em, er) = R.layernorm(x[ok], None, None, 1e-5)
    R.close(y[ok], y8, ey + y8.abs() * R.U, "y")
    R.close(rstd[ok], r8, er, "rstd")
    assert bool((y[0] == 0).all())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[3]).all())
    gx, gw, gb = tt.tt_layernorm_grad(torch.ones_like(x), x, None, mean, rstd)
    assert bool(torch.isfinite(gx[ok]).all()) and bool(torch.isnan(gx[2]).all()) and bool(torch.isnan(gx[3]).all())
    assert bool(torch.isnan(gw).all()) and bool((gb == 6).all())


def test_layernorm_gradient_against_differences():
    """sum(grad . v) against the central difference of sum(dy y) along v, in
    float64. The difference's own error: h^2 / 6 times the third derivative
    (at most a few hundred here) plus 1e-16 / h times the sum: below 1e-6."""
    _cuda()
    g = _gen(21)
    n, d, h = 3, 40, 1e-5
    x, dy = _rows(g, n, d, F32, spread=False), _rows(g, n, d, F32, spread=False)
    w, bias = 1 + torch.randn(d, generator=g, device="cuda"), torch.randn(d, generator=g, device="cuda")

    def loss(x, w, bias):
        c = x - x.mean(1, keepdim=True)
        return float((dy.double() * (c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * w + bias)).sum())

    y, mean, rstd = tt.tt_layernorm(x, w, bias, 1e-5)
    grads = tt.tt_layernorm_grad(dy, x, w, mean, rstd)
    at = [x.double(), w.double(), bias.double()]
    _, bounds = R.layernorm_grad(dy, x, w, mean, rstd)
    for k in range(3):
        v = torch.randn(at[k].shape, generator=g, device="cuda", dtype=torch.float64)
        up, down = list(at), list(at)
        up[k], down[k] = at[k] + h * v, at[k] - h * v
        diff = (loss(*up) - loss(*down)) / (2 * h)
        along = float((grads[k].double() * v).sum())
        # mean and rstd are rounded too: 100 U relative on what they enter
        tol = float((bounds[k] * v.abs()).sum()) + 200 * R.U * float((grads[k].double() * v).abs().sum()) + 1e-6
        assert abs(along - diff) <= tol, (k, along, diff, tol)


@pytest.mark.parametrize("d", [16, 48, 64, 80, 96, 128, 144, 256, 272, 400, 512])
@pytest.mark.parametrize("dtype,gdtype", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16)])
def test_normalize_gradient(d, dtype, gdtype):
    _cuda()
    g = _gen(d)
    n = 301
    x, dy = _rows(g, n, d, dtype), _rows(g, n, d, gdtype, spread=False)
    x[0] = 0                       # the norm is the constant 1e-6
    x[1] = 1e-8                    # so it is here: sum x^2 <= 512e-16
    got = tt.tt_normalize_grad(dy, x)
    want, tol = R.normalize_grad(dy, x)
    assert got.dtype == dtype
    R.close(got, want, tol + (want.abs() + tol) * R.half_step(dtype), "grad_x")


def test_normalize_gradient_against_differences():
    _cuda()
    g = _gen(5)
    x, dy = _rows(g, 5, 32, F32), _rows(g, 5, 32, F32, spread=False)
    v = torch.randn((5, 32), generator=g, device="cuda", dtype=torch.float64)
    h = 1e-6
    diff = float((dy.double() * (R.normalize(x.double() + h * v) - R.normalize(x.double() - h * v))).sum()) / (2 * h)
    got = tt.tt_normalize_grad(dy, x)
    _, tol = R.normalize_grad(dy, x)
    scale = float((got.double() * v).abs().sum())
    assert abs(float((got.double() * v).sum()) - diff) <= float((tol * v.abs()).sum()) + 1e-6 * (1 + scale)
    # what the forward call does is what is differentiated
    y = torch.empty_like(x)
    tt.tt_normalize_candidates(x, y, make_index=False)
    R.close(y, R.normalize(x), (R.D_ROW + 4) * R.U * R.normalize(x).abs(), "y")


def test_rows_past_2_31_elements():
    """Offsets past 32 bits: the last rows of a tensor of 2^31 + elements."""
    _cuda()
    n, d = (1 << 22) + 5, 512
    x = torch.zeros((n, d), dtype=BF16, device="cuda")
    tail = torch.randn((3, d), generator=_gen(1), device="cuda").to(BF16)
    x[-3:] = tail
    y, mean, rstd = tt.tt_layernorm(x)
    y3, _, _ = tt.tt_layernorm(tail)
    assert torch.equal(y[-3:], y3) and bool((y[:4] == 0).all())
    gx = tt.tt_normalize_grad(x, x, out=y)
    assert torch.equal(gx[-3:], tt.tt_normalize_grad(tail, tail))


def test_stream_capture_and_replay():
    """On a side stream, then captured in a graph and replayed on new data:
    the same bits as eager calls."""
    _cuda()
    g = _gen(12)
    n, d = 130, 384
    x, dy = _rows(g, n, d, BF16), _rows(g, n, d, BF16, spread=False)
    w = torch.randn(d, generator=g, device="cuda")
    outs = (torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda"))
    grads = (torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda"))
    ws = torch.empty(tt.tt_layernorm_grad_workspace(n, d), dtype=torch.uint8, device="cuda")

    def call():
        tt.tt_layernorm(x, w, None, 1e-5, out=outs)
        tt.tt_layernorm_grad(dy, x, w, outs[1], outs[2], out=grads, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(_rows(g, n, d, BF16))
    graph.replay()
    torch.cuda.synchronize()
    y, mean, rstd = tt.tt_layernorm(x, w, None, 1e-5)
    want = tt.tt_layernorm_grad(dy, x, w, mean, rstd)
    assert torch.equal(outs[0], y) and all(torch.equal(a, b) for a, b in zip(grads, want))


def test_refusals():
    _cuda()
    x = torch.randn((4, 64), device="cuda")
    s = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        tt.tt_layernorm(x.t())
    with pytest.raises(ValueError):
        tt.tt_layernorm(x.cpu())
    with pytest.raises(TypeError):
        tt.tt_layernorm(x.half())
    with pytest.raises(ValueError):
        tt.tt_layernorm(x, torch.ones(63, device="cuda"))
    with pytest.raises(TypeError):
        tt.tt_layernorm(x, torch.ones(64, device="cuda"), torch.ones(64, device="cuda", dtype=BF16))
    with pytest.raises(tt.TTError) as err:
        tt.tt_layernorm(x, out=(x, s, torch.empty_like(s)))  # in place
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        tt.tt_layernorm_grad(x, x, None, s[:3], s)
    with pytest.raises(tt.TTError) as err:
        tt.tt_layernorm_grad(x, x, None, s, s, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    with pytest.raises(tt.TTError) as err:
        tt.tt_normalize_grad(x, x, out=x)
    assert err.value.status == tt.TT_ERR_INVALID_ARG
    y = torch.randn((4, 40), device="cuda")
    with pytest.raises(tt.TTError) as err:
        tt.tt_normalize_grad(y, y)  # d is not a multiple of 16
    assert err.value.status == tt.TT_ERR_UNSUPPORTED

"""The global gradient norm and clipping on the GPU against float64. (GPU)

Bounds: a group of 8 squares in fp32 is off by at most 8 roundings, so the sum
of squares by 8 U relative, the norm by 4 U and one rounding to fp32: 5 U. The
scale adds three fp32 operations, the product one, then the output's rounding."""
import math

import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

F32, BF16 = torch.float32, torch.bfloat16


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _tensors(sizes, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(scale * torch.randn(n, generator=g, device="cuda")).to(dt) for n, dt in sizes]


def _norm(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def _check(grads, max_norm, norm, outs):
    want = _norm(grads)
    assert abs(float(norm) - want) <= 5 * R.U * want + 1e-45
    scale = min(1.0, max_norm / (want + 1e-6))
    for x, y in zip(grads, outs):
        w = x.double() * scale
        rel = 0.0 if scale == 1.0 else 10 * R.U
        R.close(y, w, w.abs() * (rel + (0.0 if scale == 1.0 else R.half_step(y.dtype) * 1.01)), "out")


SETS = {
    "one element": [(1, F32)],
    "small": [(5, F32), (8, BF16), (3, BF16), (1, F32), (4097, F32)],
    "chunks": [(4096, F32), (4097, F32), (8192, BF16), (8193, BF16), (16384, BF16), (7, F32)],
    "empty among them": [(0, F32), (100, BF16), (0, BF16), (33, F32)],
    "33 tensors": [(1000 + i, F32 if i % 2 else BF16) for i in range(33)],
    "1003 tensors": [(17 + 3 * i, F32 if i % 3 else BF16) for i in range(1003)],
    "large": [(9_000_001, F32), (30_000_003, BF16), (11, F32)],
}


@pytest.mark.parametrize("max_norm", [0.75, 1e9, 0.0, float("inf")])
@pytest.mark.parametrize("name", sorted(SETS))
def test_norm_and_clip(name, max_norm):
    _cuda()
    grads = _tensors(SETS[name], seed=len(name))
    outs = [torch.full_like(t, 7.0) for t in grads]
    norm = tt.tt_clip_grad_norm(grads, max_norm, out=outs)
    assert norm.dtype == F32 and norm.shape == ()
    _check(grads, max_norm, norm, outs)
    alone = tt.tt_grad_norm(grads)
    assert torch.equal(alone, norm)
    # in place: the same values
    same = [t.clone() for t in grads]
    assert torch.equal(tt.tt_clip_grad_norm(same, max_norm), norm)
    assert all(torch.equal(a, b) for a, b in zip(same, outs))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (3, 3), (1, 0), (0, 5), (2, 7)])
def test_views_that_begin_anywhere(dtype, shift_in, shift_out):
    """Tensors inside flat buffers, at any element; nothing outside them is written."""
    _cuda()
    sizes = [1, 2, 9, 4096, 20_011, 5]
    total = sum(sizes) + 16
    flat = _tensors([(total, dtype)], seed=4)[0]
    flat_out = torch.full((total,), -9.0, dtype=dtype, device="cuda")
    grads, outs = [], []
    at = 0
    for n in sizes:
        grads.append(flat[shift_in + at:shift_in + at + n])
        outs.append(flat_out[shift_out + at:shift_out + at + n])
        at += n
    norm = tt.tt_clip_grad_norm(grads, 0.5, out=outs)
    _check(grads, 0.5, norm, outs)
    assert bool((flat_out[:shift_out] == -9).all()) and bool((flat_out[shift_out + at:] == -9).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-20, 1e18, 1e25])
def test_squares_outside_fp32(scale):
    """Values whose squares underflow or overflow fp32 still give the norm."""
    _cuda()
    grads = _tensors([(5000, F32), (777, BF16)], seed=6, scale=scale)
    grads[0][::3] *= 1e-6  # mixed magnitudes in a group
    norm = tt.tt_grad_norm(grads)
    want = _norm(grads)
    assert abs(float(norm) - want) <= 5 * R.U * want + 1e-45
    norm = tt.tt_clip_grad_norm(grads, 1.0)
    assert abs(float(norm) - want) <= 5 * R.U * want + 1e-45


def test_not_finite():
    _cuda()
    grads = _tensors([(100, F32), (100, BF16)])
    grads[0][7] = float("nan")
    norm = tt.tt_clip_grad_norm(grads, 1.0)
    assert math.isnan(float(norm)) and all(bool(torch.isnan(t).all()) for t in grads)
    grads = _tensors([(100, F32), (100, BF16)])
    grads[1][3] = float("-inf")
    norm = tt.tt_clip_grad_norm(grads, 1.0)
    assert float(norm) == math.inf and bool((grads[0] == 0).all()) and bool(torch.isnan(grads[1][3]))
    assert float(tt.tt_grad_norm([])) == 0.0
    assert float(tt.tt_grad_norm([torch.zeros(300, device="cuda")])) == 0.0
    zeros = [torch.zeros(300, device="cuda")]
    assert float(tt.tt_clip_grad_norm(zeros, 1.0)) == 0.0 and bool((zeros[0] == 0).all())


def test_no_limit_and_an_infinite_norm():
    """An infinite max_norm only measures: the tensors stay as they are."""
    _cuda()
    grads = _tensors([(100, F32), (100, BF16)])
    grads[1][3] = float("inf")
    before = [t.clone() for t in grads]
    assert float(tt.tt_clip_grad_norm(grads, float("inf"))) == math.inf
    assert all(torch.equal(a, b) for a, b in zip(grads, before))


def test_tensor_past_2_31_elements():
    _cuda()
    t = torch.zeros((1 << 31) + 9, dtype=BF16, device="cuda")
    t[0], t[-1] = 3.0, 4.0
    norm = tt.tt_clip_grad_norm([t], 2.5)
    assert float(norm) == 5.0
    assert float(t[0]) == 1.5 and float(t[-1]) == 2.0 and float(t[1 << 30]) == 0.0


def test_side_stream_and_graph():
    _cuda()
    grads = _tensors(SETS["33 tensors"], seed=2)
    outs = [torch.empty_like(t) for t in grads]
    norm = torch.empty((), device="cuda")
    ws = torch.empty(tt.tt_clip_grad_norm_workspace(grads), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tt.tt_clip_grad_norm(grads, 1.0, out=outs, norm=norm, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    _check(grads, 1.0, norm, outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tt.tt_clip_grad_norm(grads, 1.0, out=outs, norm=norm, workspace=ws)
    for t in grads:
        t.mul_(3)
    ws.fill_(255)  # its contents do not matter
    graph.replay()
    _check(grads, 1.0, norm, outs)


def test_refusals():
    _cuda()
    a, b = torch.ones(10, device="cuda"), torch.ones(10, device="cuda")
    with pytest.raises(TypeError):
        tt.tt_grad_norm([a.half()])
    with pytest.raises(ValueError):
        tt.tt_grad_norm([a.cpu()])
    with pytest.raises(ValueError):
        tt.tt_grad_norm([torch.ones((4, 4), device="cuda").t()[:, :2]])
    with pytest.raises(ValueError):
        tt.tt_clip_grad_norm([a, b], 1.0, out=[a])
    with pytest.raises(ValueError):
        tt.tt_clip_grad_norm([a], 1.0, out=[torch.empty(9, device="cuda")])
    with pytest.raises(tt.TTError) as err:
        tt.tt_clip_grad_norm([a, a], 1.0)  # would be scaled twice
    assert err.value.status == tt.TT_ERR_INVALID_ARG and bool((a == 1).all())
    with pytest.raises(tt.TTError) as err:
        tt.tt_clip_grad_norm([a], -1.0)
    assert err.value.status == tt.TT_ERR_INVALID_ARG

"""Layer norm of rows that hold one number: where fp32 holds the row's sum, the
mean is that number and the row minus its mean is zero, whatever the width. (GPU)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

F32, BF16 = torch.float32, torch.bfloat16
# lane groups and chunks of every width class; most of their inverses are rounded up or down
WIDTHS = [1, 3, 7, 41, 49, 56, 61, 104, 112, 120, 208, 224, 240, 257, 500, 501, 513, 776, 777, 1000, 1023, 1032, 1128, 1129,
          2400, 2401, 4104, 5000, 8191, 8200, 12345, 16376, 16383, 16384]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_constant_rows(d, dtype):
    """Whole numbers whose sums stay below 2^24, so that every partial sum is exact."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    values = [1.0, 3.0, -7.0, 255.0, 1000.0, 12289.0, -5.0, 96.0, 129.0]
    values = [v for v in values if abs(v) * d < 2 ** 24 and float(torch.tensor(v, dtype=dtype)) == v]
    x = torch.tensor(values, device="cuda").to(dtype)[:, None].expand(-1, d).contiguous()
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    w = torch.randn(d, generator=g, device="cuda")
    bias = torch.randn(d, generator=g, device="cuda")
    y, mean, rstd = tt.tt_layernorm(x, w, bias, 1e-5)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, bias.to(dtype).expand_as(y))
    # of a variance of zero: eps in fp32 (half a U after the root) and rsqrtf's two units in the last place (4 U)
    assert bool(((rstd.double() * 1e-5 ** 0.5 - 1).abs() <= 5 * 2.0 ** -24).all())
    y, mean, rstd = tt.tt_layernorm(x, eps=0.0)
    assert bool(torch.isnan(y).all()) and bool(torch.isinf(rstd).all())


@pytest.mark.parametrize("d", [7, 56, 500, 777, 1128, 2401])
def test_infinite_and_huge_means(d):
    """The mean of a row with an infinity is that infinity, of one with NaN NaN; a sum near the largest
    fp32 number keeps its mean."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.ones((4, d), device="cuda")
    x[0, d // 2], x[1, 0], x[2, d - 1] = float("inf"), float("-inf"), float("nan")
    x[3] = 2.0 ** 127 / 2 ** (d - 1).bit_length()  # every partial sum is exact
    _, mean, _ = tt.tt_layernorm(x)
    assert float(mean[0]) == float("inf") and float(mean[1]) == float("-inf") and bool(torch.isnan(mean[2]))
    assert float(mean[3]) == float(x[3, 0])

"""The embedding gradient at the token counts where its sort changes form, and
the sort by tiles with its scan over more types and widths. (GPU)"""
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

F32, BF16, I32, I64 = torch.float32, torch.bfloat16, torch.int32, torch.int64


def _check(m, rows, d, dtype, out_dtype, idt, scale=1.0):
    """Both forms against float64. A run of n tokens adds along a chain of at most
    n, and of 32 in a warp, 8 in a block, n / 256 partial rows and 8 joins."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda")
    g.manual_seed(m + rows + d)
    u = torch.rand(m, generator=g, device="cuda", dtype=torch.float64)
    ids = ((rows + 1) ** u - 1).long().clamp(0, rows - 1)  # popular low ids: long and short runs
    ids[torch.rand(m, generator=g, device="cuda") < 0.05] = -1
    ids[-1], ids[0] = rows - 1, 0
    grad = torch.randn((m, d), generator=g, device="cuda").to(dtype)
    keep = ids >= 0
    present, where = torch.unique(ids[keep], return_inverse=True)
    n = present.numel()
    want = torch.zeros((n, d), dtype=torch.float64, device="cuda").index_add_(0, where, grad[keep].double()) * scale
    size = torch.zeros((n, d), dtype=torch.float64, device="cuda").index_add_(0, where, grad[keep].double().abs()) * scale
    runs = torch.bincount(where, minlength=n).double()[:, None]
    tol = (torch.minimum(runs, 48 + runs / 256) + 2) * R.U * size
    tol = tol + (want.abs() + tol) * R.half_step(out_dtype)
    ids = ids.to(idt)
    got_ids = torch.full((m,), -9, dtype=idt, device="cuda")
    got_rows = torch.full((m, d), -77.0, dtype=out_dtype, device="cuda")
    _, _, count = tt.tt_embedding_grad_rows(ids, grad, rows, scale=scale, out=(got_ids, got_rows))
    assert int(count) == n
    assert torch.equal(got_ids[:n].long(), present) and bool((got_ids[n:] == -9).all())
    R.close(got_rows[:n], want, tol, "rows")
    assert bool((got_rows[n:] == -77.0).all())
    dense = tt.tt_embedding_grad(ids, grad, rows, scale=scale, out_dtype=out_dtype)
    assert torch.equal(dense[present], got_rows[:n])
    rest = torch.ones(rows, dtype=torch.bool, device="cuda")
    rest[present] = False
    assert not bool(dense[rest].any())


# a smaller block's sort and a larger one's, sort by tiles, tiles whose counts are scanned
@pytest.mark.parametrize("m", [4095, 4096, 4097, 8191, 8192, 8193, 131_071, 131_072, 131_073, 133_121])
@pytest.mark.parametrize("rows", [1, 3, 255, 300, 65_535, 70_000])  # digits of 1 to 8 bits, one to three of them
def test_sort_borders(m, rows):
    _check(m, rows, 8, F32, F32, I64)


@pytest.mark.parametrize("d,dtype,out_dtype,idt", [(64, F32, F32, I32), (40, BF16, BF16, I64), (77, BF16, F32, I32),
                                                   (300, F32, BF16, I64), (1, F32, F32, I32)])
@pytest.mark.parametrize("m", [140_001, 300_000])
def test_scanned_tiles(m, d, dtype, out_dtype, idt):
    _check(m, 50_001, d, dtype, out_dtype, idt, scale=0.5)


def test_widest_ids():
    """Ids of four digits."""
    _check(200_003, (1 << 27) + 5, 1, F32, BF16, I64)

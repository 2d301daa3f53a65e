"""The gradient of the in-batch softmax where the vectors share a large common
component, against float64. (GPU)

The gradient of a user row is a sum over differences of items (and that of an
item nearly one over differences of users), so what all vectors have in common
leaves it; the rounding of P to bf16 must not bring it back. Hence a bound that
goes by the spread of the vectors, not by their size.

With h = 2^-8 (half a bf16 step): the product's coefficients are P (1 + e), |e|
<= h, times f, the ratio of the sums of P before and after the rounding, |f - 1|
<= h / (1 - h). Each differs from P by at most (2 h + 4 h^2) P, and together they
add up to sum P but for the fp32 sums' own error: at most (n / 4 + 200) U each (a
thread adds a quarter of a row or less, then 2 shuffle steps, 2 groups of warps
and at most 148 parts). So for any m the rounding changes sum P v by at most
  (2 h + 4 h^2) sum P |v - m| + 2 (n / 4 + 200) U sum P |v|.
The other terms are those of test_gpu_softmax_grad: the fp32 logit and
exponential, the products' sums, the diagonal, the result's own rounding."""
import pytest
import torch

import train_ref as R

pytestmark = pytest.mark.gpu

tt = pytest.importorskip("exact_inner_product_b200")

BF16 = torch.bfloat16
H = 2.0 ** -8


def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def spread(p, rows):
    """sum_j p_ij |rows_j - m_i| with m_i the p-weighted mean of the rows: [len(p), d]."""
    m = p @ rows / p.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.stack([(p[i][:, None] * (rows - m[i]).abs()).sum(0) for i in range(p.shape[0])])


def make(seed, b, nc, d, noise, masks):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    common = torch.randn((2, d), generator=g, device="cuda")
    common /= common.norm(dim=1, keepdim=True)

    def vectors(n, c):
        x = c + noise * torch.randn((n, d), generator=g, device="cuda") / d ** 0.5
        return (x / x.norm(dim=1, keepdim=True)).to(BF16)

    inp = {"users": vectors(b, common[0]), "items": vectors(nc, common[1]), "logq": None, "item_ids": None, "valid": None}
    if masks:
        inp["item_ids"] = torch.randint(0, 4 * nc, (nc,), generator=g, device="cuda")
        inp["logq"] = 0.1 * torch.randn(nc, generator=g, device="cuda")
        inp["valid"] = torch.rand(nc, generator=g, device="cuda") > 0.05
    return inp


@pytest.mark.parametrize("b,nc,d,noise,masks,per_row", [
    (500, 512, 64, 0.1, False, False),
    (500, 1500, 64, 0.05, False, False),
    (512, 512, 64, 0.05, False, False),    # the items' sums are near one too
    (512, 700, 128, 0.05, True, False),
    (512, 700, 128, 0.05, True, True),     # a weight per row
    (300, 1100, 96, 0.02, True, False),
    (700, 705, 256, 0.05, False, True),
    (300, 600, 320, 0.05, True, False),    # two halves of the columns
    (200, 700, 512, 0.05, False, False),
    (130, 9000, 64, 0.05, False, False),   # a row's sum in many parts
])
def test_common_component(b, nc, d, noise, masks, per_row):
    _cuda()
    tau = 1.0
    inp = make(b + nc + d, b, nc, d, noise, masks)
    mask_args = {k: inp[k] for k in ("logq", "item_ids", "valid")}
    lse, loss, _ = tt.tt_inbatch_softmax(inp["users"], inp["items"], tau, **mask_args)
    ok = torch.ones(nc, dtype=torch.bool, device="cuda") if inp["valid"] is None else inp["valid"]
    w = ok[:b].double() / int(ok[:b].sum())
    grad_loss = None
    if per_row:
        g = torch.Generator(device="cuda")
        g.manual_seed(b)
        grad_loss = 0.5 + torch.rand(b, generator=g, device="cuda")
        w = torch.where(ok[:b], grad_loss.double(), 0.0)
    got = tt.tt_inbatch_softmax_grad(inp["users"], inp["items"], lse, loss, tau, grad_loss=grad_loss,
                                     grad_mean=None if per_row else torch.ones((), device="cuda"), check=True, **mask_args)

    u = torch.where(ok[:b, None], inp["users"].double(), 0.0)
    v = torch.where(ok[:, None], inp["items"].double(), 0.0)
    logit = u @ v.T / tau
    if inp["logq"] is not None:
        logit = logit - inp["logq"].double()
    keep = ok[None, :].expand(b, nc).clone()
    if inp["item_ids"] is not None:
        keep &= inp["item_ids"][:b, None] != inp["item_ids"][None, :]
    rows = torch.arange(b, device="cuda")
    keep[rows, rows] = False
    keep &= ok[:b, None]
    p = torch.where(keep, torch.exp(logit - lse.double()[:, None]), 0.0)
    diag = torch.where(ok[:b], torch.expm1(-loss.double()), 0.0)
    gamma = d * R.U / (1 - d * R.U)
    x_err = 1.1 * (gamma * 1.01 / tau + 6 * R.U * float(logit.abs().max() + lse.abs().max() + 10) + 2.0 ** -22)

    def bound(p, own, others, want, n):
        """own: the diagonal's rows with their coefficients; others: the rows that are added."""
        sums = p @ others.abs()
        e = (2 * H + 4 * H * H) * spread(p, others) + (2 * (n / 4 + 200) * R.U + x_err + (n / 16 + 64) * R.U + 8 * R.U) * sums
        e = (e + 8 * R.U * own.abs()) / tau
        return e + (want.abs() + e) * R.half_step(BF16)

    want_u = w[:, None] / tau * (p @ v + diag[:, None] * v[:b])
    R.close(got[0], want_u, bound(w[:, None] * p, w[:, None] * diag[:, None] * v[:b], v, want_u, nc) + 1e-37, "grad_users")
    wp = (w[:, None] * p).T
    own = torch.zeros_like(v)
    own[:b] = (w * diag)[:, None] * u
    want_v = (wp @ u + own) / tau
    R.close(got[1], want_v, bound(wp, own, u, want_v, b) + 1e-37, "grad_items")

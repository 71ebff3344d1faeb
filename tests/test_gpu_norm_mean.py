"""LayerNorm of rows whose mean is far above their spread, down to rows of one
value, against the formula in binary64, at widths that are not powers of two.

Tolerances, with u = 2^-24 and SUM = 100 u the error of a row's sum relative to
the sum of magnitudes (64 terms in a thread, then 10 levels of pairs, and the
terms' own rounding): the first mean is off by at most D = SUM |mu|. The second
pass sums terms of at most |x - mu| + D, so the mean is known to E = SUM (mean|x -
mu| + D) + u D, and the variance to SUM (var + D^2), which is half of that in rstd.
x - mu, the shift by the mean's rest and the product with rstd add 8 u of
their values; the output's rounding adds half a step of its type."""
import pytest
import torch

import sparsity_gemm_b200 as sq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 100 * U
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
WIDTHS = [3, 60, 999, 1000, 3584, 3585, 8201, 14336, 20000, 40000]


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("dt", list(DTYPES))
def test_rows_of_one_value(dt, k):
    """The mean is the value, the output zero (b, where there is one)."""
    values = torch.tensor([65504.0, 60000.0, 50016.0, -12344.0, 1000.0, 0.1, 1 / 3, -3e-5], device="cuda").to(DTYPES[dt])
    x = values.view(-1, 1).expand(-1, k).contiguous()
    b = torch.randn(k, generator=torch.Generator(device="cuda").manual_seed(k), device="cuda").to(DTYPES[dt])
    for eps in (1e-5, 1e-12):
        y, mean, rstd = sq.layer_norm(x, None, None, eps, stats=True)
        assert torch.equal(mean, values.float())
        assert not bool(y.any())
        # eps and what rounding leaves of the variance: at most SUM D^2
        top = torch.full_like(mean, eps, dtype=torch.float64).rsqrt()
        low = (eps + SUM * (SUM * values.double().abs()).square()).rsqrt()
        assert bool((rstd <= top * (1 + 8 * U)).all()) and bool((rstd >= low * (1 - 8 * U)).all())
        assert torch.equal(sq.layer_norm(x, None, b, eps), b.expand(8, k))


@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("center", [1000.0, 60000.0])
def test_mean_far_above_the_spread(center, dt, k):
    """Values within 16 steps of the type around the center."""
    gen = torch.Generator(device="cuda").manual_seed(k)
    step = torch.finfo(DTYPES[dt]).eps * 2.0 ** (9 if center == 1000.0 else 15)
    x = (center + step * torch.randint(-16, 17, (6, k), generator=gen, device="cuda")).to(DTYPES[dt])
    w = (1 + 0.2 * torch.randn(k, generator=gen, device="cuda")).to(DTYPES[dt])
    y, mean, rstd = sq.layer_norm(x, w, None, 1e-5, stats=True)
    xd, wd = x.double(), w.double()
    mu = xd.mean(1, keepdim=True)
    var = (xd - mu).square().mean(1, keepdim=True)
    rs = (var + 1e-5).rsqrt()
    d = SUM * mu.abs()
    e = SUM * ((xd - mu).abs().mean(1, keepdim=True) + d) + U * d
    rel = SUM * (1 + d.square() / (var + 1e-5)) + 8 * U
    assert bool(((mean.double() - mu.view(-1)).abs() <= (e + U * mu.abs()).view(-1)).all())
    assert bool(((rstd.double() / rs.view(-1) - 1).abs() <= rel.view(-1)).all())
    want = (xd - mu) * rs * wd
    fin = torch.finfo(DTYPES[dt])
    tol = wd.abs() * rs * (e + (xd - mu).abs() * (rel + 8 * U)) + 2 * U * want.abs() + want.abs() * fin.eps / 2 \
        + fin.smallest_normal * fin.eps / 2
    err = (y.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).max()):.3g} of the tolerance"


def test_rows_that_are_not_finite():
    """As the formula: an infinite row has that mean and no other result."""
    x = torch.randn(4, 1000, device="cuda")
    x[0, 7], x[1, 9], x[2, 11] = float("inf"), float("-inf"), float("nan")
    y, mean, rstd = sq.layer_norm(x, stats=True)
    assert bool(y[:3].isnan().all()) and bool(rstd[:3].isnan().all()) and bool(y[3].isfinite().all())
    assert float(mean[0]) == float("inf") and float(mean[1]) == float("-inf") and bool(mean[2].isnan())

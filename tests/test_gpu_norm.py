"""LayerNorm and RMSNorm in 16 and 32 bits and their backward pass, against
the formulas in binary64.

Tolerances, with u = 2^-24 (binary32) and r = eps / 2 of the output's type:
a binary32 sum of a row adds at most 64 terms in a thread and then 10 levels
of pairs, so its error is at most SUM = 100 u times the sum of magnitudes; the
few operations after it add 8 u of each term; the output's rounding adds r of
the value (and half the smallest subnormal). The weight gradients add rows in
chains no longer than the number of rows plus 40."""
import numpy as np
import pytest
import torch

import sparsity_gemm_b200 as sq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
SUM = 100 * U
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _round(v, dt):
    return v.abs() * torch.finfo(dt).eps / 2 + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def _close(name, got, want, tol):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} off, worst {float((err / tol).nan_to_num(1e30).max()):.3g} of the tolerance"


def _inputs(seed, rows, k, dt, mean=0.5, offset=0):
    """x with per-row means and a few large channels, and the affine weights;
    offset: elements by which the buffers miss their alignment."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    x = r(rows, k) + mean * r(rows, 1)
    x[:, ::37] *= 20
    def place(t):
        buf = torch.empty(t.numel() + offset, dtype=dt, device="cuda")
        buf[offset:] = t.to(dt).flatten()
        return buf[offset:].view(t.shape)
    return place(x), place(1 + 0.2 * r(k)), place(0.3 * r(k)), place(r(rows, k))


def _forward(x, w, b, eps, norm):
    x = x.double()
    mu = x.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(x[:, :1])
    rstd = ((x - mu).square().mean(1, keepdim=True) + eps).rsqrt()
    y = (x - mu) * rstd
    y = y if w is None else y * w.double()
    y = y if b is None else y + b.double()
    return y, mu, rstd


def _check_forward(x, w, b, eps, norm):
    dt = x.dtype
    y, mean, rstd = sq.layer_norm(x, w, b, eps, norm=norm, stats=True)
    want, mu, rs = _forward(x, w, b, eps, norm)
    xd = x.double()
    wa = 1.0 if w is None else w.double().abs()
    off = SUM * xd.abs().mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(mu)  # the mean's error
    rel = SUM + 8 * U + 0.5 * (off * rs).square()  # rstd's relative error
    if norm == "layer":
        _close("mean", mean, mu.view(-1), off.view(-1) + 2 * U * mu.view(-1).abs())
    else:
        assert mean is None
    _close("rstd", rstd, rs.view(-1), (rel * rs).view(-1))
    ba = 0.0 if b is None else b.double().abs()
    tol = wa * rs * (off + (xd - mu).abs() * (rel + 8 * U)) + 2 * U * (want.abs() + ba) + _round(want, dt)
    _close("y", y, want, tol)
    assert torch.equal(y, sq.layer_norm(x, w, b, eps, norm=norm))  # same bits without statistics
    return mean, rstd


def _check_backward(dy, x, mean, rstd, w, norm):
    dt, k, rows = x.dtype, x.shape[1], x.shape[0]
    dx, dw, db = sq.layer_norm_backward(dy, x, mean, rstd, w, norm=norm)
    rs = rstd.double().view(-1, 1)
    h = x.double() * rs if mean is None else (x.double() - mean.double().view(-1, 1)) * rs
    g = dy.double() if w is None else dy.double() * w.double()
    m1 = g.mean(1, keepdim=True) if norm == "layer" else torch.zeros_like(rs)
    m2 = (g * h).mean(1, keepdim=True)
    want = rs * (g - m1 - h * m2)
    ga, ha = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    tol = rs * (8 * U * (g.abs() + m1.abs() + (h * m2).abs()) + (SUM + 8 * U) * (ga + h.abs() * ha)) + _round(want, dt)
    _close("dx", dx, want, tol)
    if w is None:
        assert dw is None and db is None
        return
    n = (rows + 40 + 8) * U
    _close("dw", dw, (dy.double() * h).sum(0), n * (dy.double() * h).abs().sum(0) + 1e-300)
    if norm == "layer":
        _close("db", db, dy.double().sum(0), n * dy.double().abs().sum(0) + 1e-300)
    else:
        assert db is None


# widths: a warp's row, a few warps, a CTA's register rows and their ends
# (4096 vectors; scalar rows of odd widths), rows streamed from L2 and rows
# split over a cluster in the backward pass
WIDTHS = [1, 7, 8, 64, 129, 256, 512, 520, 1000, 2048, 4096, 4097, 8200, 14336, 16384 + 8, 33000, 65536]


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("k", WIDTHS)
@pytest.mark.parametrize("dt", list(DTYPES))
def test_widths(dt, k, norm):
    x, w, b, dy = _inputs(k, 5, k, DTYPES[dt])
    b = b if norm == "layer" else None
    mean, rstd = _check_forward(x, w, b, 1e-5, norm)
    _check_backward(dy, x, mean, rstd, w, norm)


@pytest.mark.parametrize("norm", ["layer", "rms"])
@pytest.mark.parametrize("rows,k", [(1, 4096), (2, 128), (601, 128), (3001, 256), (1500, 768), (1021, 3584), (777, 8192),
                                    (301, 14336), (90, 20000)])
def test_row_counts(rows, k, norm):
    x, w, b, dy = _inputs(rows + k, rows, k, torch.bfloat16)
    mean, rstd = _check_forward(x, w, b if norm == "layer" else None, 1e-6, norm)
    _check_backward(dy, x, mean, rstd, w, norm)


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("with_w,with_b", [(False, False), (True, False), (False, True)])
def test_without_affine_parameters(dt, with_w, with_b):
    x, w, b, dy = _inputs(5, 33, 640, DTYPES[dt])
    w, b = (w if with_w else None), (b if with_b else None)
    mean, rstd = _check_forward(x, w, b, 1e-5, "layer")
    _check_backward(dy, x, mean, rstd, w, "layer")


@pytest.mark.parametrize("norm", ["layer", "rms"])
def test_long_rows_without_weights(norm):
    for k in (8200, 9001, 20000):
        x, _, _, dy = _inputs(k, 9, k, torch.float16)
        mean, rstd = _check_forward(x, None, None, 1e-5, norm)
        _check_backward(dy, x, mean, rstd, None, norm)


@pytest.mark.parametrize("dt", list(DTYPES))
def test_buffers_that_miss_16_byte_alignment(dt):
    x, w, b, dy = _inputs(6, 21, 1024, DTYPES[dt], offset=1)
    mean, rstd = _check_forward(x, w, b, 1e-5, "layer")
    _check_backward(dy, x, mean, rstd, w, "layer")


def test_mean_far_above_the_spread():
    """The variance is taken around the mean, so a mean 1000 times the spread
    costs no digits beyond the mean's own error."""
    x, w, b, _ = _inputs(7, 16, 4096, torch.float32, mean=0.0)
    _check_forward((x + 1000.0).contiguous(), w, b, 1e-5, "layer")


def test_degenerate_rows():
    x = torch.zeros(4, 512, dtype=torch.float16, device="cuda")
    x[1] = 3.0
    x[2] = 65504.0
    x[3, 0] = 6e-8
    y, mean, rstd = sq.layer_norm(x, None, None, 1e-5, stats=True)
    assert torch.equal(y[:3], torch.zeros_like(y[:3]))  # constant rows: exact mean, no spread
    assert torch.equal(mean[:3].cpu(), torch.tensor([0.0, 3.0, 65504.0]))
    assert bool(torch.isfinite(y).all()) and bool(torch.isfinite(rstd).all())


def test_gradient_against_differences():
    """<dx, d> equals the forward pass's difference quotient along d, in
    binary32; the error of a central difference with step 2^-6 is the step
    squared times third derivatives (under 1e-2 here) plus rounding of y over
    the step (under 1e-3)."""
    x, w, b, dy = _inputs(8, 7, 300, torch.float32)
    x = (x / x.std(1, keepdim=True)).contiguous()
    for norm in ("layer", "rms"):
        _, mean, rstd = sq.layer_norm(x, w, None, 1e-5, norm=norm, stats=True)
        dx, dw, db = sq.layer_norm_backward(dy, x, mean, rstd, w, norm=norm)
        gen = torch.Generator(device="cuda").manual_seed(9)
        d = torch.randn(x.shape, generator=gen, device="cuda")
        s = 2.0 ** -6
        f = lambda t: sq.layer_norm(t, w, None, 1e-5, norm=norm).double()  # noqa: E731
        want = ((f(x + s * d) - f(x - s * d)) * dy.double()).sum(1) / (2 * s)
        got = (dx.double() * d.double()).sum(1)
        scale = (dy.double().norm(dim=1) * d.double().norm(dim=1))
        assert bool(((got - want).abs() <= 1e-2 * scale).all())
        dirw = torch.randn(w.shape, generator=gen, device="cuda")
        lin = (sq.layer_norm(x, dirw, None, 1e-5, norm=norm).double() * dy.double()).sum()
        assert abs(float((dw.double() * dirw.double()).sum() - lin)) <= 1e-4 * float(dy.double().norm() * dirw.double().norm() * 3)


def test_no_rows():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = sq.layer_norm(x, w, w, stats=True)
    assert y.shape == x.shape and mean.numel() == 0
    dx, dw, db = sq.layer_norm_backward(x, x, mean, rstd, w)
    assert dx.shape == x.shape and not bool(dw.any()) and not bool(db.any())


def test_backward_in_place_of_dy_and_repeatable():
    x, w, b, dy = _inputs(10, 1021, 3584, torch.float16)
    _, mean, rstd = sq.layer_norm(x, w, b, stats=True)
    dx, dw, db = sq.layer_norm_backward(dy, x, mean, rstd, w)
    again = dy.clone()
    out, dw2, db2 = sq.layer_norm_backward(again, x, mean, rstd, w, out=again)
    assert out is again and torch.equal(out, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)


def test_long_row_offsets_pass_32_bits():
    """Rows whose element offsets pass 2^31: the last rows are right."""
    rows, k = 33000, 65536  # 2.16e9 elements, 4.3 GB each
    x = torch.empty(rows, k, dtype=torch.float16, device="cuda")
    x[:8], x[-8:] = torch.randn(8, k, device="cuda"), torch.randn(8, k, device="cuda")
    x[8:-8] = 0
    y = sq.layer_norm(x, norm="rms")
    want, _, _ = _forward(x[-8:], None, None, 1e-5, "rms")
    _close("y", y[-8:], want, 4 * SUM * want.abs() + _round(want, torch.float16))
    del y, x


@pytest.mark.parametrize("rows,k", [(33000, 65536), (270000, 8192), (270000, 8193)])
def test_gradient_row_offsets_pass_32_bits(rows, k):
    """The gradient where offsets pass 2^31: the last rows are those of a call
    on these rows alone, bit for bit (a row's sums do not depend on its place)."""
    x = torch.zeros(rows, k, dtype=torch.float16, device="cuda")
    dy = torch.zeros(rows, k, dtype=torch.float16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x[-8:] = torch.randn(8, k, generator=gen, device="cuda").half()
    dy[-8:] = torch.randn(8, k, generator=gen, device="cuda").half()
    _, mean, rstd = sq.layer_norm(x[-8:], stats=True)
    means, rstds = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    means[-8:], rstds[-8:] = mean, rstd
    dx, _, _ = sq.layer_norm_backward(dy, x, means, rstds, out=dy.clone())
    want, _, _ = sq.layer_norm_backward(dy[-8:], x[-8:], mean, rstd)
    assert torch.equal(dx[-8:], want) and not bool(dx[:8].any())
    del dx, dy, x


def test_other_streams_and_graph_replay():
    x, w, b, dy = _inputs(11, 64, 1536, torch.float16)
    want = sq.layer_norm(x, w, b, stats=True)
    wb = sq.layer_norm_backward(dy, x, want[1], want[2], w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sq.layer_norm(x, w, b, stats=True, stream=s)
    gb = sq.layer_norm_backward(dy, x, got[1], got[2], w, stream=s)
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want + wb, got + gb))
    static = x.clone()
    with torch.cuda.stream(s):
        sq.layer_norm_backward(dy, static, want[1], want[2], w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, mean, rstd = sq.layer_norm(static, w, b, stats=True)
        outs = sq.layer_norm_backward(dy, static, mean, rstd, w)
    for seed in (12, 13):
        x2, _, _, _ = _inputs(seed, 64, 1536, torch.float16)
        static.copy_(x2)
        g.replay()
        torch.cuda.synchronize()
        ey = sq.layer_norm(x2, w, b, stats=True)
        eb = sq.layer_norm_backward(dy, x2, ey[1], ey[2], w)
        assert all(torch.equal(a, c) for a, c in zip((y, mean, rstd) + outs, ey + eb))
    assert sq.get_last_error() == sq.OK


def test_norm_agrees_with_the_preparation_operator():
    """layer_norm is the normalization that prepare applies: the mean and rstd
    of the exact statistics agree within the sums' error."""
    x, w, b, _ = _inputs(14, 40, 1024, torch.float16)
    ex = sq.prep_export(sq.prepare(x, w, b))
    _, mean, rstd = sq.layer_norm(x, w, b, stats=True)
    xd = x.double().abs().mean(1).cpu().numpy()
    assert np.all(np.abs(mean.cpu().numpy().astype(np.float64) - ex["mu"]) <= (SUM + 2 * U) * xd + 2 * U * np.abs(ex["mu"]))
    assert np.all(np.abs(rstd.cpu().numpy().astype(np.float64) / ex["rstd"] - 1) <= SUM + 16 * U)

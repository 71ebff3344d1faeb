"""Low-rank adapters where a result hangs on the last bits of x A^T, and where
values are infinite or NaN, in the one-launch and the two-launch form."""
import pytest
import torch

import sparsity_gemm_b200 as sq

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
# (rows, rank): one launch up to rank 128, two launches after these
FORMS = [(1, 8), (40, 16), (300, 32), (300, 64), (100, 128), (3600, 16), (2600, 32), (1100, 64), (1300, 120)]


def _digits(m, rank, dt, big):
    """x, A, B whose h = x A^T is, per row, integers H (23 bits in bf16, 22 in
    fp16), d - H with d below 256, and, if big, a third value 2^11 to 2^18 times
    larger that B leaves out: x A^T B^T = d."""
    gen = torch.Generator(device="cuda").manual_seed(m + rank)
    part = lambda hi: torch.randint(0, hi, (m,), generator=gen, device="cuda")  # noqa: E731
    a2, a1, a0, d = part(128 if dt == torch.bfloat16 else 64), part(256), part(256), part(256)
    x = torch.zeros(m, 64, device="cuda")
    x[:, 3], x[:, 17], x[:, 40], x[:, 41], x[:, 63] = 2 * a2, a1, a0, d, 2.0 ** (25 if dt == torch.bfloat16 else 15)
    a = torch.zeros(1, rank, 64, device="cuda")
    for col, v in ((3, 2.0 ** 15), (17, 256.0), (40, 1.0)):
        a[0, 1, col], a[0, rank - 2, col] = v, -v
    a[0, rank - 2, 41] = 1.0
    if big:
        a[0, 4, 63] = 2.0 ** 15
    b = torch.zeros(1, 72, rank, device="cuda")
    b[0, :, 1] = b[0, :, rank - 2] = 1.0
    assert torch.equal(x, x.to(dt).float()) and torch.equal(a, a.to(dt).float())
    return x.to(dt), a.to(dt), b.to(dt), d.to(dt).view(-1, 1).expand(m, 72)


@pytest.mark.parametrize("big", [False, True])
@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("m,rank", FORMS)
def test_products_keep_the_digits_of_binary32(m, rank, dt, big):
    """Every sum of both products is an integer below 2^24 (times a power of
    two), so binary32 holds it and the result is exact."""
    x, a, b, want = _digits(m, rank, DTYPES[dt], big)
    r = sq.route(torch.zeros(m, dtype=torch.int32, device="cuda"), 1)
    assert torch.equal(sq.lora(x, a, b, r), want)
    assert sq.get_last_error() == sq.OK


def _formula(x, a, b):
    """x A^T B^T of one adapter in binary64, term by term (0 times infinity is
    NaN, and nothing else is)."""
    h = (x.double().unsqueeze(1) * a.double()).sum(2)
    return (h.unsqueeze(1) * b.double()).sum(2)


def _same(got, want, tol):
    nan, inf = want.isnan(), want.isinf()
    assert torch.equal(got.isnan(), nan)
    assert torch.equal(got[inf].double(), want[inf])
    fine = ~nan & ~inf
    assert bool(((got.double() - want).abs()[fine] <= tol * want.abs().clamp_min(1.0)[fine]).all())


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("m,rank", FORMS)
def test_infinities_come_out_as_in_the_formula(m, rank, dt):
    """An infinite x makes every column of its row infinite (by the signs of A
    and B) or NaN, an infinite A the columns of its adapter's rows; other rows,
    and the rows of an adapter beside one of NaN, are as they were. Tolerance:
    the finite results are below 64 and rounded to 8 or 11 bits; their sums are
    good to 1e-3 in any order."""
    gen = torch.Generator(device="cuda").manual_seed(m + rank)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    k, n, groups = 72, 72, 3
    x, a, b = r(m, k), r(groups, rank, k) / k ** 0.5, r(groups, n, rank) / rank ** 0.5
    a[0, :, 5] = a[0, :, 5].abs() + 0.1           # all of x[., 5]'s products have its sign
    b[0, :24], b[0, 24:48] = b[0, :24].abs() + 0.01, -b[0, 24:48].abs() - 0.01
    a[1, 3, 7] = float("inf")
    a[2] = float("nan")
    b[1] = torch.where(b[1].abs() < 0.01, 0.01, b[1])
    ids = torch.arange(m, device="cuda", dtype=torch.int32) % groups
    x[0, 5] = float("inf")
    if m > 9:
        x[3, 5], x[6, 11], x[9, 5] = float("-inf"), float("nan"), 1.0
    x, a, b = x.to(DTYPES[dt]), a.to(DTYPES[dt]), b.to(DTYPES[dt])
    got = sq.lora(x, a, b, sq.route(ids, groups))
    for g in (0, 1, 2):
        at = torch.nonzero(ids == g).flatten()
        at = torch.cat([at[:40], at[-40:]])
        if at.numel():
            _same(got[at], _formula(x[at], a[g], b[g]), 2.0 ** (-8 if dt == "bf16" else -11) + 1e-3)
    rows = torch.ones(m, dtype=torch.bool, device="cuda")
    rows[0] = False
    if m > 9:
        rows[3] = rows[6] = False
    assert bool(got[rows & (ids == 0)].isfinite().all())
    assert sq.get_last_error() == sq.OK


@pytest.mark.parametrize("m,rank", FORMS)
def test_the_largest_finite_products(m, rank):
    """bf16: x A^T that rounds to infinity in 16 bits but not in 32."""
    x = torch.zeros(m, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 1], x[:, 9] = 2.0 ** 127, 1.5 * 2.0 ** 119
    a = torch.zeros(1, rank, 64, dtype=torch.bfloat16, device="cuda")
    a[0, 2, 1], a[0, 2, 9] = 255 / 128, 1.0
    b = torch.zeros(1, 40, rank, dtype=torch.bfloat16, device="cuda")
    b[0, :, 2] = 2.0 ** -100
    got = sq.lora(x, a, b, sq.route(torch.zeros(m, dtype=torch.int32, device="cuda"), 1))
    want = torch.full((m, 40), 255.75 * 2.0 ** 20, device="cuda").bfloat16()
    assert torch.equal(got, want)


# (rows, rank, adapters) of both forms, the two-launch one with padded ranks and
# with tiles that end early
BOTH = [(30, 16, 3), (100, 24, 5), (1100, 72, 3), (2700, 24, 4), (3600, 8, 3), (130, 64, 200)]


def _adapter_case(m, rank, groups, dt, none):
    gen = torch.Generator(device="cuda").manual_seed(m + rank)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    k, n = 136, 72
    ids = torch.randint(0, groups, (m,), generator=gen, device="cuda", dtype=torch.int32)
    ids[torch.rand(m, generator=gen, device="cuda") < none] = -1
    return r(m, k), r(groups, rank, k) / k ** 0.5, r(groups, n, rank) / rank ** 0.5, r(m, n), ids


@pytest.mark.parametrize("m,rank,groups", BOTH)
def test_bad_routing_is_reported_in_both_forms(m, rank, groups):
    x, a, b, base, ids = _adapter_case(m, rank, groups, torch.float16, 0.1)
    r = sq.route(ids, groups)
    good = sq.lora(x, a, b, r, base=base)
    assert sq.get_last_error() == sq.OK
    total = int(r.offsets[-1])
    bare = ids < 0
    edits = [(0, 1), (-1, m + 1), (1, -5), (1, total + 7 if groups > 1 else m + 7)]
    for at, value in edits:
        offsets = r.offsets.clone()
        offsets[at] = value
        out = torch.full_like(base, 7.0)
        sq.lora(x, a, b, sq.Routing(offsets, r.rows, r.slots), base=base, out=out)
        assert sq.get_last_error() == sq.ERR_INVALID_ARG
        assert bool((out[~bare] == 7.0).all()) and torch.equal(out[bare], base[bare])
    for bad in (m, m + 100, -1, -(2 ** 31)):  # rows out of range are left out, the others are as before
        rows = r.rows.clone()
        at = torch.tensor([0, total // 2, total - 1], device="cuda")
        lost = rows[at].long()
        rows[at] = bad
        out = torch.full_like(base, 7.0)
        sq.lora(x, a, b, sq.Routing(r.offsets, rows, r.slots), base=base, out=out)
        assert sq.get_last_error() == sq.ERR_INVALID_ARG
        keep = torch.ones(m, dtype=torch.bool, device="cuda")
        keep[lost] = False
        assert torch.equal(out[keep], good[keep]) and bool((out[lost] == 7.0).all())
    assert torch.equal(sq.lora(x, a, b, r, base=base), good) and sq.get_last_error() == sq.OK


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("m,rank,groups", BOTH)
def test_nothing_leaks_between_adapters_and_rows(m, rank, groups, dt):
    """NaN and infinity in every second adapter (behind the padded rank of the
    one before it) and in the last rows of a group: the rows of the others keep
    their bits."""
    x, a, b, base, ids = _adapter_case(m, rank, groups, DTYPES[dt], 0.1)
    r = sq.route(ids, groups)
    good = sq.lora(x, a, b, r, base=base)
    clean = (ids < 0) | (ids % 2 == 0)
    ends = r.offsets[1:][r.offsets[1:] > r.offsets[:-1]].long() - 1  # each group's last grouped row
    last = r.rows[ends].long()
    x[last[0::2]] = float("nan")
    x[last[1::2]] = float("inf")
    clean[last] = False
    clean |= ids < 0
    a[1::2, 0], a[1::2, -1], b[1::2] = float("nan"), float("inf"), float("nan")
    got = sq.lora(x, a, b, r, base=base)
    assert torch.equal(got[clean], good[clean])
    assert bool(got[last].isnan().any(1).all())
    assert sq.get_last_error() == sq.OK

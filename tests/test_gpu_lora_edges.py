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

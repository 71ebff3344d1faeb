"""The operators whose kernels wait for copies and products of their own, with
the shortest wait limit: a call either gets its result or reports that it gave
up, and leaves nothing in flight behind, so that the next calls are right."""
import pytest
import torch

import sparsity_gemm_b200 as sq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,k", [(2000, 4096), (300, 8192), (5000, 520)])
def test_norm_gradient_with_the_shortest_wait_limit(rows, k):
    gen = torch.Generator(device="cuda").manual_seed(k)
    x, dy = (torch.randn(rows, k, generator=gen, device="cuda").half() for _ in range(2))
    w = torch.ones(k, dtype=torch.float16, device="cuda")
    _, mean, rstd = sq.layer_norm(x, w, stats=True)
    want = sq.layer_norm_backward(dy, x, mean, rstd, w)
    assert sq.get_last_error() == sq.OK
    old = sq.set_wait_limit_ns(1)
    try:
        got = [sq.layer_norm_backward(dy, x, mean, rstd, w) for _ in range(8)]
        status = sq.get_last_error()
    finally:
        sq.set_wait_limit_ns(old)
    assert status in (sq.OK, sq.ERR_TIMEOUT)
    if status == sq.OK:
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    assert all(torch.equal(a, b) for a, b in zip(sq.layer_norm_backward(dy, x, mean, rstd, w), want))
    assert sq.get_last_error() == sq.OK


@pytest.mark.parametrize("m,rank,groups", [(4000, 16, 3), (1500, 64, 3), (1300, 128, 2)])
def test_adapters_with_the_shortest_wait_limit(m, rank, groups):
    gen = torch.Generator(device="cuda").manual_seed(m)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").half()  # noqa: E731
    x, a, b, base = r(m, 1024), r(groups, rank, 1024) / 32, r(groups, 264, rank), r(m, 264)
    q = sq.route(torch.randint(-1, groups, (m,), generator=gen, device="cuda", dtype=torch.int32), groups)
    want = sq.lora(x, a, b, q, base=base)
    assert sq.get_last_error() == sq.OK
    old = sq.set_wait_limit_ns(1)
    try:
        got = [sq.lora(x, a, b, q, base=base) for _ in range(8)]
        status = sq.get_last_error()
    finally:
        sq.set_wait_limit_ns(old)
    assert status in (sq.OK, sq.ERR_TIMEOUT)
    if status == sq.OK:
        assert all(torch.equal(g, want) for g in got)
    assert torch.equal(sq.lora(x, a, b, q, base=base), want)
    assert sq.get_last_error() == sq.OK

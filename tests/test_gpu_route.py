"""Entries sorted by group, rows moved into that order and back with weights,
and the gradient, against plain restatements (integers equal, values in
binary64).

Tolerances, with u = 2^-24 and r = eps / 2 of the output's type: combine adds
at most top_k + 1 products in a chain, (top_k + 3) u of the sum of magnitudes;
a dot product over k adds at most 256 terms in a thread and 13 levels after
it, 300 u of the sum of magnitudes; results are rounded once (r)."""
import numpy as np
import pytest
import torch

import sparsity_gemm_b200 as sq
import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _round(v, dt):
    return v.abs() * torch.finfo(dt).eps / 2 + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


def _close(name, got, want, tol):
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{name}: worst {float((err / tol).nan_to_num(1e30).max()):.3g} of the tolerance"


def plain_route(ids, groups):
    """offsets, rows, slots by the definition, entry after entry."""
    flat = ids.reshape(-1)
    top_k = ids.shape[1] if ids.ndim == 2 else 1
    lists = [[] for _ in range(groups)]
    for e, g in enumerate(flat.tolist()):
        if 0 <= g < groups:
            lists[g].append(e)
    offsets = np.zeros(groups + 1, np.int32)
    offsets[1:] = np.cumsum([len(v) for v in lists])
    rows, slots = np.full(flat.size, -1, np.int32), np.full(flat.size, -1, np.int32)
    order = np.concatenate([np.asarray(v, np.int64) for v in lists]) if flat.size else np.zeros(0, np.int64)
    rows[:order.size] = order // top_k
    slots[order] = np.arange(order.size)
    return offsets, rows, slots.reshape(-1, top_k)


def check_route(ids, groups):
    r = sq.route(ids, groups)
    for name, got, want in zip(("offsets", "rows", "slots"), (r.offsets, r.rows, r.slots),
                               plain_route(ids.cpu().numpy(), groups)):
        assert np.array_equal(got.cpu().numpy(), want), name
    return r


def random_ids(seed, tokens, top_k, groups, none=0.0, dtype=np.int32):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, groups, size=(tokens, top_k))
    ids[rng.random(ids.shape) < none] = -1
    return torch.from_numpy(ids.astype(dtype)).cuda()


@pytest.mark.parametrize("dtype", [np.int32, np.int64])
@pytest.mark.parametrize("tokens,top_k,groups", [
    (1, 1, 1), (1, 8, 128), (3, 5, 7), (31, 1, 32), (33, 1, 33), (128, 8, 128), (1024, 2, 1024), (1023, 3, 60),
    (2049, 1, 1000), (4096, 8, 128), (5000, 4, 8), (16384, 8, 256), (40000, 6, 64)])
def test_route(tokens, top_k, groups, dtype):
    check_route(random_ids(tokens, tokens, top_k, groups, 0.0, dtype), groups)
    check_route(random_ids(tokens + 1, tokens, top_k, groups, 0.3, dtype), groups)


def test_route_edges():
    none = torch.full((37, 4), -1, dtype=torch.int32, device="cuda")
    r = check_route(none, 5)  # nobody has a group
    assert int(r.offsets[-1]) == 0 and bool((r.rows == -1).all())
    check_route(torch.full((3000, 1), 2, dtype=torch.int32, device="cuda"), 4)  # all in one
    ids = random_ids(3, 500, 2, 16)
    ids[::7, 0], ids[::5, 1] = 16, 2 ** 31 - 1  # ids past the last group
    ids[3] = -2 ** 31
    check_route(ids, 16)
    big = torch.tensor([[2 ** 40], [2 ** 32], [1], [-2 ** 33], [0]], device="cuda")  # int64 ids that truncate to a group
    check_route(big, 2)
    check_route(random_ids(4, 700, 1, 9)[:, 0].contiguous(), 9)  # a vector of ids
    r = sq.route(torch.empty(0, 8, dtype=torch.int64, device="cuda"), 12)
    assert not bool(r.offsets.any()) and r.rows.numel() == 0
    ids = random_ids(5, 50, 4, 6)
    ids[:, 1] = ids[:, 0]  # the same expert twice
    check_route(ids, 6)


def test_route_equals_the_workload_generator():
    row_idx, offsets = synth.moe_routing(3, 700, 128, 8)
    logits = synth.normal(3, synth.S_GATE, 700 * 128).reshape(700, 128)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :8].astype(np.int32)
    r = sq.route(torch.from_numpy(ids).cuda(), 128)
    assert np.array_equal(r.rows.cpu().numpy(), row_idx) and np.array_equal(r.offsets.cpu().numpy(), offsets)


def _values(seed, shape, dt, offset=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = int(np.prod(shape))
    buf = torch.empty(n + offset, dtype=dt, device="cuda")
    buf[offset:] = torch.randn(n, generator=gen, device="cuda").to(dt)
    return buf[offset:].view(shape)


def check_moves(tokens, top_k, groups, k, dt, none=0.2, offset=0, extra=0):
    ids = random_ids(tokens + k, tokens, top_k, groups, none)
    r = sq.route(ids, groups)
    total = int(r.offsets[-1])
    rows, slots = r.rows.long(), r.slots.long()
    x = _values(1, (tokens, k), dt, offset)
    moved = sq.permute_rows(x, r)
    assert torch.equal(moved[:total], x[rows[:total]]) and not bool(moved[total:].any())

    y = _values(2, (tokens * top_k + extra, k), dt, offset)
    w = _values(3, (tokens, top_k), torch.float32)
    res, dout = _values(4, (tokens, k), dt, offset), _values(5, (tokens, k), dt, offset)
    there = (slots >= 0).double()
    yd = y.double()[slots.clamp_min(0)] * there.unsqueeze(2)
    for weights, residual in ((w, res), (w, None), (None, None)):
        wd = torch.ones_like(w) if weights is None else weights
        terms = wd.double().unsqueeze(2) * yd
        want, mag = terms.sum(1), terms.abs().sum(1)
        if residual is not None:
            want, mag = want + residual.double(), mag + residual.double().abs()
        out = sq.combine(y, r, weights, residual)
        _close("combine", out, want, (top_k + 3) * U * mag + _round(want, dt))
        if residual is not None:
            inplace = residual.clone()
            assert torch.equal(sq.combine(y, r, weights, inplace, out=inplace), out)
    # the gradient of permute is combine without weights
    dy, dw = sq.combine_backward(dout, y, r, w)
    want = torch.zeros_like(y, dtype=torch.float64)
    want[slots[slots >= 0]] = (w.double().unsqueeze(2) * dout.double().unsqueeze(1))[slots >= 0]
    _close("dy", dy, want, 2 * U * want.abs() + _round(want, dt))
    assert not bool(dy[total:].any())
    prod = dout.double().unsqueeze(1) * yd
    _close("dweights", dw, prod.sum(2), 300 * U * prod.abs().sum(2) + 1e-300)
    again = sq.combine_backward(dout, y, r, w)
    assert torch.equal(again[0], dy) and torch.equal(again[1], dw)
    assert sq.get_last_error() == sq.OK


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("tokens,top_k,groups,k", [(1, 1, 1, 8), (1, 8, 128, 2048), (16, 8, 128, 4096), (7, 3, 5, 1), (5, 9, 16, 129),
                                                   (64, 2, 8, 2056), (300, 8, 60, 1000), (33, 17, 64, 7000), (2, 64, 70, 640)])
def test_rows_there_and_back(tokens, top_k, groups, k, dt):
    check_moves(tokens, top_k, groups, k, DTYPES[dt])


def test_rows_there_and_back_other_layouts():
    check_moves(50, 4, 8, 512, torch.float16, offset=1)            # buffers that miss 16-byte alignment
    check_moves(50, 4, 8, 512, torch.bfloat16, none=1.0)           # nobody has a group
    check_moves(50, 4, 8, 512, torch.float32, none=0.0, extra=13)  # grouped rows behind the last group


@pytest.mark.parametrize("top_k,k", [(1, 65536), (2, 32768), (1, 32771)])
def test_row_offsets_pass_32_bits(top_k, k):
    """Grouped rows and tokens whose element offsets pass 2^31: copies and sums
    with powers of two as weights are exact, so every bit is known."""
    tokens = 33000 if k == 65536 else 66000 // top_k if k == 32768 else 65600
    ids = torch.arange(tokens * top_k, device="cuda", dtype=torch.int32).view(tokens, top_k) % 2
    r = sq.route(ids, 2)
    pick = torch.tensor([0, 1, tokens // 2, tokens - 2, tokens - 1], device="cuda")
    x = torch.zeros(tokens, k, dtype=torch.float16, device="cuda")
    x[pick] = _values(1, (5, k), torch.float16)
    moved = sq.permute_rows(x, r)
    slots = r.slots.long()[pick]
    for j in range(top_k):
        assert torch.equal(moved[slots[:, j]], x[pick])
    w = torch.full((tokens, top_k), 1.0 / top_k, device="cuda")
    assert torch.equal(sq.combine(moved, r, w)[pick], x[pick])
    dy, dw = sq.combine_backward(x, moved, r, w)
    for j in range(top_k):
        assert torch.equal(dy[slots[:, j]], (x[pick].float() / top_k).half())
    sq2 = (x[pick].double() ** 2).sum(1, keepdim=True).expand(5, top_k)
    _close("dweights", dw[pick], sq2, (k / 256 + 16) * U * sq2)
    assert sq.get_last_error() == sq.OK


def test_values_nobody_asked_for_do_not_leak():
    """NaN and infinity in grouped rows without an entry stay there."""
    ids = random_ids(6, 40, 2, 4, 0.4)
    r = sq.route(ids, 4)
    total = int(r.offsets[-1])
    y = _values(7, (80, 256), torch.bfloat16)
    y[total:] = float("nan")
    y[total + 1:total + 2] = float("inf")
    w = _values(8, (40, 2), torch.float32)
    w[r.slots < 0] = float("nan")
    out = sq.combine(y, r, w)
    dy, dw = sq.combine_backward(out, y, r, w)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(dy).all()) and bool(torch.isfinite(dw).all())


def test_no_tokens():
    r = sq.route(torch.empty(0, 2, dtype=torch.int32, device="cuda"), 3)
    x = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    assert sq.permute_rows(x, r).shape == (0, 64)
    assert sq.combine(x, r).shape == (0, 64)
    y = torch.ones(5, 64, dtype=torch.float16, device="cuda")
    dy, dw = sq.combine_backward(x, y, r, torch.empty(0, 2, device="cuda"))
    assert not bool(dy.any()) and dw.shape == (0, 2)


def test_gradient_of_combine_against_differences():
    """combine is linear in y and in the weights: a difference along a
    direction is the operator itself, so <dy, d> = <combine(d), dout> and
    <dw, e> = <combine with weights e, dout> up to the sums' error."""
    r = sq.route(random_ids(9, 60, 4, 8, 0.1), 8)
    y, d = _values(10, (240, 320), torch.float32), _values(11, (240, 320), torch.float32)
    w, e = _values(12, (60, 4), torch.float32), _values(13, (60, 4), torch.float32)
    dout = _values(14, (60, 320), torch.float32)
    dy, dw = sq.combine_backward(dout, y, r, w)
    e = torch.where(r.slots >= 0, e, 0)
    for got, want, size in (((dy.double() * d.double()).sum(), (sq.combine(d, r, w).double() * dout.double()).sum(), d.norm()),
                            ((dw.double() * e.double()).sum(), (sq.combine(y, r, e).double() * dout.double()).sum(), y.norm())):
        assert abs(float(got - want)) <= 1e-5 * float(size * dout.norm())
    dx = _values(15, (60, 320), torch.float32)  # permute and its gradient
    lhs = (sq.permute_rows(dx, r).double() * y.double()).sum()
    rhs = (dx.double() * sq.combine(y, r).double()).sum()
    assert abs(float(lhs - rhs)) <= 1e-5 * float(dx.norm() * y.norm())


def test_bad_slots_are_skipped_and_reported():
    r = sq.route(random_ids(16, 12, 2, 3), 3)
    x = _values(17, (12, 64), torch.float16)
    good = sq.permute_rows(x, r)
    bad = sq.Routing(r.offsets, r.rows, r.slots.clone())
    bad.slots[4, 1] = 24
    out = torch.zeros_like(good)
    sq.permute_rows(x, bad, out=out)
    assert sq.get_last_error() == sq.ERR_INVALID_ARG and sq.get_last_error() == sq.OK
    keep = torch.ones(24, dtype=torch.bool)
    keep[int(r.slots[4, 1])] = False
    assert torch.equal(out[keep.cuda()], good[keep.cuda()])
    y = _values(18, (24, 64), torch.float16)
    sq.combine(y, bad)
    assert sq.get_last_error() == sq.ERR_INVALID_ARG
    sq.combine_backward(x, y, bad, torch.ones(12, 2, device="cuda"))
    assert sq.get_last_error() == sq.ERR_INVALID_ARG


def test_moe_layer_runs_on_the_grouped_linear():
    """As they are used together: route, rows into expert order, the grouped
    preparation and linear, and back with weights and the residual, against
    the gather path on the same routing and a binary64 combine; captured into
    a graph and replayed on new tokens and choices."""
    tokens, top_k, groups, k, n_out = 96, 4, 8, 256, 512
    wq = sq.quantize_weight_grouped(torch.from_numpy(
        np.stack([synth.weights(50 + g, n_out, k) for g in range(groups)]).view(np.float16)).cuda())
    x_of = lambda s: torch.from_numpy(synth.activations_student(s, tokens, k).view(np.float16)).cuda()  # noqa: E731
    x, ids = x_of(60), random_ids(61, tokens, top_k, groups)
    w, res = torch.rand(tokens, top_k, device="cuda"), _values(62, (tokens, n_out), torch.float16)
    rows = tokens * top_k

    def layer():
        r = sq.route(ids, groups)
        moved = sq.permute_rows(x, r)
        p = sq.prepare_grouped(moved, r.offsets)
        y = sq.linear_grouped(p, r.offsets, wq, rows)
        return r, y, sq.combine(y, r, w, res)

    def check(r, y, out):
        g = sq.gather_rows(sq.prepare(x), r.rows, r.offsets, rows)
        assert torch.equal(y, sq.linear_grouped(g, r.offsets, wq, rows))  # same rows, same bits
        terms = w.double().unsqueeze(2) * y.double()[r.slots.long()]
        want = terms.sum(1) + res.double()
        mag = terms.abs().sum(1) + res.double().abs()
        _close("layer", out, want, (top_k + 3) * U * mag + _round(want, torch.float16))
        assert sq.get_last_error() == sq.OK

    check(*layer())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer()
    for seed in (70, 80):
        x.copy_(x_of(seed))
        ids.copy_(random_ids(seed + 1, tokens, top_k, groups))
        graph.replay()
        torch.cuda.synchronize()
        check(*got)

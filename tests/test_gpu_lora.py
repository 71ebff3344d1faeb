"""Low-rank adapters of many requests beside a shared projection, against the
formula in binary64.

Tolerance, with v = 2^-22 for one binary32 addition on the tensor cores (two
units of the last place), r = eps / 2 of the output's type and t = 2^-16
(bf16) or 2^-22 (fp16) for the two-term form of h:
  h = x A^T adds k / 16 + 32 partial sums:  (k/16 + 32) v sum|x a|;
  its two terms: t times the row's largest |h|;
  h B^T adds 2 rank / 16 + 4 partial sums: (rank/8 + 4) v sum|h b|;
  the sum with base: 2^-23 of the magnitudes, and r of the result."""
import numpy as np
import pytest
import torch

import sparsity_gemm_b200 as sq
import synth

pytestmark = pytest.mark.gpu

V = 2.0 ** -22
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _case(seed, m, k, n, rank, groups, dt, none=0.2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    ids = torch.randint(0, groups, (m,), generator=gen, device="cuda", dtype=torch.int32)
    ids[torch.rand(m, generator=gen, device="cuda") < none] = -1
    return dict(x=r(m, k).to(dt), a=(r(groups, rank, k) / k ** 0.5).to(dt), b=(r(groups, n, rank) / rank ** 0.5).to(dt),
                scales=0.5 + torch.rand(groups, generator=gen, device="cuda"), base=r(m, n).to(dt), ids=ids)


def _want(c, with_scales=True, with_base=True):
    """(result, tolerance) in binary64."""
    dt = c["x"].dtype
    m, n = c["base"].shape
    rank, k = c["a"].shape[1:]
    out = c["base"].double() if with_base else torch.zeros(m, n, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    for g in range(c["a"].shape[0]):
        at = torch.nonzero(c["ids"] == g).flatten()
        x, a, b = c["x"][at].double(), c["a"][g].double(), c["b"][g].double()
        s = c["scales"][g].double() if with_scales else 1.0
        h, ha = x @ a.t(), x.abs() @ a.abs().t()
        t = 2.0 ** (-16 if dt == torch.bfloat16 else -22)
        eh = (k / 16 + 32) * V * ha + t * (h.abs() + 0).amax(1, keepdim=True)
        d, mag = s * (h @ b.t()), s * (h.abs() @ b.abs().t())
        tol[at] = s * (eh @ b.abs().t()) + (rank / 8 + 4) * V * mag + 2.0 ** -23 * (d.abs() + out[at].abs())
        out[at] = out[at] + d
    fin = torch.finfo(dt)
    return out, tol + out.abs() * fin.eps / 2 + fin.smallest_normal * fin.eps / 2


def _check(c, got, with_scales=True, with_base=True):
    want, tol = _want(c, with_scales, with_base)
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"worst {float((err / tol).nan_to_num(1e30).max()):.3g} of the tolerance"
    bare = c["ids"] < 0
    assert torch.equal(got[bare], c["base"][bare] if with_base else torch.zeros_like(got[bare]))
    assert sq.get_last_error() == sq.OK


def _run(c, **kw):
    r = sq.route(c["ids"], c["a"].shape[0])
    return sq.lora(c["x"], c["a"], c["b"], r, scales=c["scales"], base=c["base"], **kw)


# (rows, k, n, rank, adapters): one token, decode batches, tiles of many rows
# and their ends, ranks that fill a block of 8 or of 16, widths that end inside
# a step of 32
SHAPES = [(1, 256, 256, 16, 1), (1, 4096, 14336, 64, 3), (2, 8, 8, 8, 1), (5, 264, 40, 24, 2), (16, 1024, 512, 8, 16),
          (64, 512, 768, 16, 32), (17, 768, 1000, 32, 1), (33, 520, 328, 40, 1), (63, 256, 264, 16, 1), (64, 256, 256, 16, 1),
          (65, 256, 256, 16, 1), (129, 304, 96, 48, 2), (300, 512, 512, 64, 3), (300, 512, 520, 72, 3), (200, 640, 640, 128, 2),
          (40, 640, 640, 120, 40), (1000, 256, 512, 16, 1), (1000, 384, 320, 32, 7), (777, 512, 256, 64, 100),
          (500, 256, 256, 8, 1024), (4099, 256, 264, 56, 5), (1100, 256, 264, 16, 2), (2100, 328, 512, 32, 5),
          (1500, 136, 200, 8, 1), (64, 4096, 256, 96, 1), (70000, 64, 32, 64, 3), (20000, 72, 40, 40, 1000),
          (2600, 328, 512, 32, 5), (2700, 136, 200, 24, 3), (1100, 256, 264, 72, 2), (1300, 520, 328, 120, 3),
          (3600, 256, 264, 16, 2), (3500, 8, 8, 8, 1), (130, 256, 264, 64, 200)]


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("m,k,n,rank,groups", SHAPES)
def test_adapters(m, k, n, rank, groups, dt):
    c = _case(m + k + rank, m, k, n, rank, groups, DTYPES[dt])
    _check(c, _run(c))


@pytest.mark.parametrize("m,rank,groups", [(300, 16, 700), (8100, 64, 500), (8100, 64, 40), (4000, 16, 100)])
def test_many_adapters_few_of_them_used(m, rank, groups):
    """As a server has them: hundreds loaded, two in the batch (the launch
    knows only how many are loaded)."""
    c = _case(m + groups, m, 264, 72, rank, groups, torch.bfloat16)
    c["ids"] = torch.where(c["ids"] % 3 == 0, groups - 1, torch.where(c["ids"] >= 0, 3, c["ids"])).int()
    _check(c, _run(c))


@pytest.mark.parametrize("dt", list(DTYPES))
def test_with_and_without_base_scales_and_in_place(dt):
    c = _case(1, 150, 320, 416, 16, 4, DTYPES[dt])
    r = sq.route(c["ids"].view(-1, 1).long(), 4)
    _check(c, sq.lora(c["x"], c["a"], c["b"], r, base=c["base"]), with_scales=False)
    _check(c, sq.lora(c["x"], c["a"], c["b"], r, scales=c["scales"]), with_base=False)
    full = sq.lora(c["x"], c["a"], c["b"], r, scales=c["scales"], base=c["base"])
    y = c["base"].clone()
    assert sq.lora(c["x"], c["a"], c["b"], r, scales=c["scales"], base=y, out=y) is y
    assert torch.equal(y, full)
    _check(c, y)


def test_column_slices():
    """q, k and v in one buffer: the adapter of one of them on its columns, x
    a slice as well; the other columns stay as they were."""
    c = _case(2, 70, 256, 128, 16, 3, torch.float16)
    wide = torch.randn(70, 512, device="cuda").half()
    wide[:, 256:384] = c["base"]
    keep = wide.clone()
    xs = torch.randn(70, 1024, device="cuda").half()
    xs[:, 8:264] = c["x"]
    r = sq.route(c["ids"], 3)
    view = wide[:, 256:384]
    sq.lora(xs[:, 8:264], c["a"], c["b"], r, scales=c["scales"], base=view, out=view)
    _check(c, view)
    assert torch.equal(wide[:, :256], keep[:, :256]) and torch.equal(wide[:, 384:], keep[:, 384:])
    # x, base and out as disjoint column slices of one buffer
    c = _case(3, 20, 64, 32, 8, 2, torch.bfloat16, none=0.0)
    buf = torch.zeros(20, 128, device="cuda", dtype=torch.bfloat16)
    buf[:, :64], buf[:, 64:96] = c["x"], c["base"]
    sq.lora(buf[:, :64], c["a"], c["b"], sq.route(c["ids"], 2), scales=c["scales"], base=buf[:, 64:96], out=buf[:, 96:])
    _check(c, buf[:, 96:])


@pytest.mark.parametrize("m,rank", [(40000, 16), (40000, 64)])
def test_row_offsets_pass_32_bits(m, rank):
    """Columns of buffers whose element offsets pass 2^31 (65536 a row): the
    last rows are those of compact copies, bit for bit."""
    c = _case(m + rank, m, 64, 96, rank, 4, torch.float16)
    xs = torch.empty(m, 65536, dtype=torch.float16, device="cuda")
    ys = torch.empty(m, 65536, dtype=torch.float16, device="cuda")
    x, y = xs[:, 65536 - 64:], ys[:, 65536 - 96:]
    x.copy_(c["x"])
    y.copy_(c["base"])
    r = sq.route(c["ids"], 4)
    sq.lora(x, c["a"], c["b"], r, scales=c["scales"], base=y, out=y)
    assert torch.equal(y, _run(c))
    _check(c, y.contiguous())
    del x, y, xs, ys


@pytest.mark.parametrize("m", [24, 17000])
def test_adapter_offsets_pass_32_bits(m):
    """A thousand adapters of 2^21 elements: the last ones' offsets pass 2^31.
    A's rows are unit vectors, so h picks columns of x and is exact."""
    groups, rank, k, n = 1024, 128, 16400, 32
    a = torch.zeros(groups, rank, k, dtype=torch.float16, device="cuda")
    cols = torch.arange(rank, device="cuda") * 128
    a[:, torch.arange(rank, device="cuda"), cols] = 1.0
    b = torch.zeros(groups, n, rank, dtype=torch.float16, device="cuda")
    b[:, torch.arange(n, device="cuda"), torch.arange(n, device="cuda") * 3] = 1.0
    gen = torch.Generator(device="cuda").manual_seed(m)
    x = torch.randint(-64, 64, (m, k), generator=gen, device="cuda").half()
    ids = torch.randint(groups - 9, groups, (m,), generator=gen, device="cuda", dtype=torch.int32)
    r = sq.route(ids, groups)
    scales = torch.ones(groups, device="cuda") * 2.0
    out = sq.lora(x, a, b, r, scales=scales)
    assert torch.equal(out, 2 * x[:, cols[torch.arange(n, device="cuda") * 3]])
    assert sq.get_last_error() == sq.OK
    del a, b, x


def test_nobody_or_everybody_has_an_adapter():
    for none in (0.0, 1.0):
        c = _case(4, 90, 256, 256, 16, 5, torch.float16, none=none)
        _check(c, _run(c))
    c = _case(5, 0, 256, 256, 16, 5, torch.float16)
    assert _run(c).shape == (0, 256)


def test_large_and_small_products_keep_their_digits():
    """h far outside the 16-bit range of fp16 on either side: its rows are
    scaled by powers of two before they become two fp16 terms."""
    for f in (1e4, 1e-4):
        c = _case(6, 40, 256, 128, 16, 2, torch.float16)
        c["a"] = (c["a"].float() * (8 * f if f > 1 else f)).half()
        c["scales"] = c["scales"] / (8 * f if f > 1 else f)
        if f > 1:
            assert float((c["x"].float() @ c["a"][0].float().t()).abs().max()) > 65504
        _check(c, _run(c))


def test_rows_of_other_requests_do_not_leak():
    """NaN in a row, and in an adapter, stays with that row and that
    adapter's rows."""
    c = _case(7, 100, 256, 256, 16, 4, torch.bfloat16)
    c["x"][11] = float("nan")
    c["a"][2, 3, 7] = float("inf")
    got = _run(c)
    touched = (c["ids"] == 2)
    touched[11] = c["ids"][11] >= 0
    c["x"][11] = 0
    c["a"][2] = 0
    want, tol = _want(c)
    ok = (got.double() - want).abs() <= tol
    assert bool(ok[~touched].all())


def test_repeatable_and_graph_replay():
    c = _case(8, 64, 1024, 512, 16, 8, torch.float16)
    first = _run(c)
    assert torch.equal(first, _run(c))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = _run(c)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(c)
    for seed in (9, 10):
        d = _case(seed, 64, 1024, 512, 16, 8, torch.float16)
        for key in c:
            c[key].copy_(d[key])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _run(d))
        _check(d, out)


def test_bad_routing_is_reported():
    c = _case(11, 30, 256, 256, 16, 3, torch.float16, none=0.0)
    r = sq.route(c["ids"], 3)
    out = torch.full((30, 256), 7.0, dtype=torch.float16, device="cuda")
    for bad in ([0, 20, 10, 30], [0, 10, 20, 31], [1, 10, 20, 30], [0, -5, 20, 30]):
        broken = sq.Routing(torch.tensor(bad, dtype=torch.int32, device="cuda"), r.rows, r.slots)
        sq.lora(c["x"], c["a"], c["b"], broken, base=c["base"], out=out)
        assert sq.get_last_error() == sq.ERR_INVALID_ARG
        assert bool((out == 7.0).all())  # nothing written
    rows = r.rows.clone()
    rows[3], rows[5] = 30, -1
    skipped = r.rows[[3, 5]].long()
    sq.lora(c["x"], c["a"], c["b"], sq.Routing(r.offsets, rows, r.slots), scales=c["scales"], base=c["base"], out=out)
    assert sq.get_last_error() == sq.ERR_INVALID_ARG
    want, tol = _want(c)
    ok = torch.ones(30, dtype=torch.bool, device="cuda")
    ok[skipped] = False
    assert bool(((out.double() - want).abs() <= tol)[ok].all())


def test_beside_the_fp4_linear():
    """As it is used: the norm's output feeds the adapters, the preparation of
    the same rows the shared FP4 projection, and the adapters add to its
    output in place."""
    m, k, n, rank, groups = 48, 512, 256, 16, 4
    x = torch.from_numpy(synth.activations_student(20, m, k).view(np.float16)).cuda()
    g, b = (torch.from_numpy(v.view(np.float16)).cuda() for v in synth.ln_params(21, k))
    qw = sq.quantize_weight(torch.from_numpy(synth.weights(22, n, k).view(np.float16)).cuda())
    c = _case(23, m, k, n, rank, groups, torch.float16)
    base = sq.linear(sq.prepare(x, g, b), qw)
    c["x"], c["base"] = sq.layer_norm(x, g, b), base.clone()
    r = sq.route(c["ids"], groups)
    out = sq.lora(c["x"], c["a"], c["b"], r, scales=c["scales"], base=base, out=base)
    _check(c, out)

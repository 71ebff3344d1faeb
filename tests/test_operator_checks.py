"""Refusals of the operators around the FP4 linear, without a GPU: the C ABI
returns SHARQ_ERR_INVALID_ARG (or SHARQ_ERR_UNSUPPORTED) before it touches
CUDA, the binding raises ValueError before any library call, and valid
arguments pass the binding's checks with the values the library expects."""
import ctypes as C
from unittest import mock

import pytest
import torch

import sparsity_gemm_b200 as sq
from test_binding_checks import _AsCuda


class _OnCuda(_AsCuda):
    def get_device(self):
        return 0


def _as_cuda(t):
    return t.as_subclass(_OnCuda)


P = lambda i, off=0: C.c_void_p((i << 32) + off)  # noqa: E731  far apart, aligned, never dereferenced
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    from sparsity_gemm_b200 import build
    build.build()
    return sq.lib()


def test_layer_norm_refusals(L):
    def call(x=P(1), m=4, k=256, w=P(2), b=P(3), eps=1e-5, norm=0, dt=0, y=P(4), mean=P(5), rstd=P(6)):
        return L.sharq_layer_norm(x, m, k, w, b, eps, norm, dt, y, mean, rstd, None)

    for bad in (dict(k=0), dict(k=65537), dict(m=-1), dict(m=BIG + 1), dict(dt=3), dict(norm=2), dict(norm=1, mean=None),
                dict(norm=1, b=None), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(y=None),
                dict(x=P(1, 1)), dict(dt=2, y=P(4, 2)), dict(w=P(2, 1)), dict(mean=P(5, 2)), dict(y=P(1)),
                dict(y=P(1, 4 * 512 - 2)), dict(y=P(2)), dict(y=P(3, 510))):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad
    assert call(m=0, x=None, y=None, mean=None, rstd=None) == sq.OK


def test_layer_norm_backward_refusals(L):
    need = L.sharq_layer_norm_backward_bytes(4, 256)
    assert need >= 2 * 256 * 4 and L.sharq_layer_norm_backward_bytes(4, 0) == 0
    assert L.sharq_layer_norm_backward_bytes(-1, 256) == 0 and L.sharq_layer_norm_backward_bytes(0, 256) > 0

    def call(dy=P(1), x=P(2), m=4, k=256, w=P(3), mean=P(4), rstd=P(5), norm=0, dt=1, dx=P(6), dw=P(7), db=P(8), ws=P(9),
             n=need):
        return L.sharq_layer_norm_backward(dy, x, m, k, w, mean, rstd, norm, dt, dx, dw, db, ws, n, None)

    for bad in (dict(k=0), dict(k=65537), dict(m=-1), dict(dt=-1), dict(norm=1), dict(norm=0, mean=None), dict(rstd=None),
                dict(dy=None), dict(x=None), dict(dx=None), dict(dx=P(2)), dict(dx=P(1, 2)), dict(dx=P(3)), dict(ws=None),
                dict(ws=P(9, 128)), dict(n=need - 1), dict(dw=P(7, 2)), dict(db=P(7)), dict(db=P(7, 1020)), dict(x=P(2, 1)),
                dict(k=9000, dw=None, db=None, ws=None, dx=P(10))):  # rows in two passes need the workspace in any case
        assert call(**bad) == sq.ERR_INVALID_ARG, bad


def test_route_refusals(L):
    def call(ids=P(1), nb=4, m=10, top=2, g=8, off=P(2), rows=P(3), slots=P(4)):
        return L.sharq_route(ids, nb, m, top, g, off, rows, slots, None)

    for bad in (dict(nb=2), dict(m=-1), dict(top=0), dict(top=65), dict(g=0), dict(g=1025), dict(m=BIG, top=2), dict(ids=None),
                dict(off=None), dict(rows=None), dict(slots=None), dict(nb=8, ids=P(1, 4)), dict(off=P(2, 2)),
                dict(rows=P(1)), dict(slots=P(3, 76)), dict(off=P(4, 60)), dict(off=P(1))):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad


def test_moves_refusals(L):
    def permute(x=P(1), m=10, k=64, slots=P(2), top=2, off=P(3), g=4, dt=0, out=P(4)):
        return L.sharq_permute_rows(x, m, k, slots, top, off, g, dt, out, None)

    for bad in (dict(x=None), dict(out=None), dict(slots=None), dict(off=None), dict(k=0), dict(k=65537), dict(top=0), dict(g=0),
                dict(dt=5), dict(m=BIG), dict(out=P(1)), dict(x=P(1, 1)), dict(dt=2, out=P(4, 2))):
        assert permute(**bad) == sq.ERR_INVALID_ARG, bad
    assert permute(m=0, x=None, out=None) == sq.OK

    def combine(y=P(1), rows=20, m=10, k=64, slots=P(2), w=P(3), top=2, res=P(4), dt=0, out=P(5)):
        return L.sharq_combine(y, rows, m, k, slots, w, top, res, dt, out, None)

    for bad in (dict(y=None), dict(out=None), dict(slots=None), dict(rows=-1), dict(k=0), dict(out=P(1)), dict(out=P(4, 2)),
                dict(w=P(3, 2)), dict(res=P(4, 1)), dict(dt=3), dict(top=65)):
        assert combine(**bad) == sq.ERR_INVALID_ARG, bad
    assert combine(m=0) == sq.OK

    def backward(dout=P(1), y=P(2), rows=20, m=10, k=64, slots=P(3), w=P(4), top=2, off=P(5), g=4, dt=0, dy=P(6), dw=P(7)):
        return L.sharq_combine_backward(dout, y, rows, m, k, slots, w, top, off, g, dt, dy, dw, None)

    for bad in (dict(dout=None), dict(y=None), dict(slots=None), dict(w=None), dict(off=None), dict(dy=None), dict(dw=None),
                dict(dy=P(2)), dict(dy=P(1)), dict(dw=P(4)), dict(k=0), dict(rows=-2), dict(g=1025), dict(dy=P(6, 1))):
        assert backward(**bad) == sq.ERR_INVALID_ARG, bad
    assert backward(m=0, rows=0) == sq.OK


def test_lora_refusals(L):
    def call(x=P(1), ldx=256, m=10, k=256, a=P(2), b=P(3), n=128, r=16, g=4, s=P(4), off=P(5), rows=P(6), slots=P(7), dt=0,
             base=P(8), ldb=128, out=P(9), ldo=128, ws=None, nws=0):
        return L.sharq_lora(x, ldx, m, k, a, b, n, r, g, s, off, rows, slots, dt, base, ldb, out, ldo, ws, nws, None)

    for bad in (dict(k=252, ldx=252), dict(n=124), dict(r=12), dict(r=0), dict(r=136), dict(g=0), dict(g=1025), dict(m=-1),
                dict(ldx=248), dict(ldx=260), dict(ldo=120), dict(ldo=132), dict(ldb=64), dict(ldb=1 << 25), dict(x=None),
                dict(a=None), dict(b=None), dict(off=None), dict(rows=None), dict(slots=None), dict(out=None), dict(x=P(1, 8)),
                dict(base=P(8, 8)), dict(out=P(9, 8)), dict(s=P(4, 2)), dict(dt=3), dict(out=P(1)), dict(out=P(8, 16)),
                dict(out=P(8), ldo=256), dict(out=P(2)), dict(out=P(3, 16)), dict(k=65544, ldx=65544), dict(n=(1 << 20) + 8)):
        assert call(**bad) == sq.ERR_INVALID_ARG, bad
    need = L.sharq_lora_bytes(4096, 16, 4)
    assert need >= 4096 * 64 and L.sharq_lora_bytes(10, 16, 4) == 0 and L.sharq_lora_bytes(4096, 136, 4) == 0
    for bad in (dict(ws=None, nws=need), dict(ws=P(10), nws=need - 1), dict(ws=P(10, 64), nws=need)):
        assert call(m=4096, **bad) == sq.ERR_INVALID_ARG, bad
    assert call(dt=2) == sq.ERR_UNSUPPORTED
    assert call(m=0) == sq.OK
    # slices of one buffer whose columns overlap are refused, like whole ones
    assert call(x=P(1), ldx=512, out=P(1, 2 * 248), ldo=512) == sq.ERR_INVALID_ARG
    assert call(x=P(1), ldx=512, out=P(1, 2 * 400), ldo=512) == sq.ERR_INVALID_ARG  # wraps into the next row's x


def test_outputs_share_nothing(L):
    """Outputs, workspaces among them, that reach into any other buffer."""
    norm = lambda y=P(4), mean=P(5), rstd=P(6): L.sharq_layer_norm(  # noqa: E731
        P(1), 8, 256, P(2), P(3), 1e-5, 0, 0, y, mean, rstd, None)
    for bad in (dict(mean=P(1, 4092)), dict(rstd=P(2)), dict(rstd=P(5, 28)), dict(mean=P(4, 16)), dict(y=P(6, 16))):
        assert norm(**bad) == sq.ERR_INVALID_ARG, bad
    need = L.sharq_layer_norm_backward_bytes(8, 256)
    back = lambda dx=P(6), dw=P(7), db=P(8), ws=P(9): L.sharq_layer_norm_backward(  # noqa: E731
        P(1), P(2), 8, 256, P(3), P(4), P(5), 0, 0, dx, dw, db, ws, need, None)
    for bad in (dict(dx=P(4)), dict(dx=P(5, 16)), dict(dw=P(1)), dict(dw=P(1), dx=P(1)), dict(db=P(2, 4)), dict(dw=P(3)),
                dict(db=P(5)), dict(dw=P(6, 4092)), dict(ws=P(1)), dict(ws=P(2, 256)), dict(ws=P(3)), dict(ws=P(6)),
                dict(ws=P(7)), dict(db=P(9, 2044))):
        assert back(**bad) == sq.ERR_INVALID_ARG, bad
    for bad in (P(2), P(2, 64), P(3)):
        assert L.sharq_permute_rows(P(1), 10, 64, P(2), 2, P(3), 4, 0, bad, None) == sq.ERR_INVALID_ARG
    for bad in (P(2, 64), P(3)):
        assert L.sharq_combine(P(1), 20, 10, 64, P(2), P(3), 2, P(4), 0, bad, None) == sq.ERR_INVALID_ARG
    grad = lambda dy=P(6), dw=P(7): L.sharq_combine_backward(  # noqa: E731
        P(1), P(2), 20, 10, 64, P(3), P(4), 2, P(5), 4, 0, dy, dw, None)
    for bad in (dict(dy=P(3)), dict(dy=P(4)), dict(dy=P(5)), dict(dw=P(1)), dict(dw=P(2, 128)), dict(dw=P(3, 76)),
                dict(dw=P(5, 16)), dict(dw=P(6, 1024))):
        assert grad(**bad) == sq.ERR_INVALID_ARG, bad
    need = L.sharq_lora_bytes(4096, 16, 4)
    lora = lambda out=P(9), ws=P(10): L.sharq_lora(  # noqa: E731
        P(1), 512, 4096, 256, P(2), P(3), 128, 16, 4, P(4), P(5), P(6), P(7), 0, P(8), 256, out, 256, ws, need, None)
    for bad in (dict(out=P(4)), dict(out=P(5)), dict(out=P(6, 16)), dict(out=P(7)), dict(out=P(10, 512)), dict(ws=P(1, 256)),
                dict(ws=P(2)), dict(ws=P(3)), dict(ws=P(4)), dict(ws=P(5)), dict(ws=P(6)), dict(ws=P(7)), dict(ws=P(8))):
        assert lora(**bad) == sq.ERR_INVALID_ARG, bad


def _t(*shape, dtype=torch.float16):
    return _as_cuda(torch.zeros(shape, dtype=dtype))


@pytest.fixture
def here(monkeypatch):
    """The binding on host tensors that say they are on cuda:0, over a library
    that records its calls."""
    fake = mock.MagicMock()
    fake.sharq_layer_norm_backward_bytes.return_value = 4096
    fake.sharq_lora_bytes.return_value = 0
    for name in ("layer_norm", "layer_norm_backward", "route", "permute_rows", "combine", "combine_backward", "lora"):
        getattr(fake, "sharq_" + name).return_value = sq.OK
    monkeypatch.setattr(sq, "lib", lambda: fake)
    monkeypatch.setattr(sq, "_lib", None)
    monkeypatch.setattr(sq, "_new", lambda like, shape, dtype, stream: _as_cuda(torch.zeros(shape, dtype=dtype)))
    monkeypatch.setattr(sq, "_new_like", lambda t, stream: _as_cuda(torch.zeros(t.shape, dtype=t.dtype)))
    monkeypatch.setattr(sq, "_raw", lambda stream, dev: 0)
    sq._lora_bytes.cache_clear()
    sq._norm_backward_bytes.cache_clear()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    yield fake
    sq._lora_bytes.cache_clear()
    sq._norm_backward_bytes.cache_clear()


def _routing(m=6, top_k=2, groups=3):
    i32 = torch.int32
    return sq.Routing(_t(groups + 1, dtype=i32), _t(m * top_k, dtype=i32), _t(m, top_k, dtype=i32))


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 64, dtype=torch.float16)
    for f in (lambda: sq.layer_norm(x), lambda: sq.layer_norm_backward(x, x, x[0], x[0]),
              lambda: sq.route(torch.zeros(4, 2, dtype=torch.int32), 3),
              lambda: sq.Routing(torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32)),
              lambda: sq.lora(x, torch.zeros(1, 8, 64).half(), torch.zeros(1, 32, 8).half(), None)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            f()


def test_binding_refuses_other_devices(here, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for f in (lambda: sq.layer_norm(_t(4, 64)), lambda: _routing(), lambda: sq.route(_t(4, 2, dtype=torch.int32), 3)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            f()


def test_binding_refuses_bad_shapes_and_types(here):
    r, x = _routing(), _t(6, 64)
    bad = [lambda: sq.layer_norm(_t(64)), lambda: sq.layer_norm(_t(64, 6).t()), lambda: sq.layer_norm(_t(6, 64, dtype=torch.int32)),
           lambda: sq.layer_norm(x, _t(32)), lambda: sq.layer_norm(x, _t(64, dtype=torch.float32)),
           lambda: sq.layer_norm(x, None, _t(64), norm="rms"), lambda: sq.layer_norm(x, norm="batch"),
           lambda: sq.layer_norm(x, out=_t(6, 32)), lambda: sq.layer_norm(x, out=_t(6, 64, dtype=torch.float32)),
           lambda: sq.layer_norm_backward(_t(5, 64), x, _t(6, dtype=torch.float32), _t(6, dtype=torch.float32)),
           lambda: sq.layer_norm_backward(x, x, None, _t(6, dtype=torch.float32)),
           lambda: sq.layer_norm_backward(x, x, _t(6, dtype=torch.float32), _t(6, dtype=torch.float32), norm="rms"),
           lambda: sq.layer_norm_backward(x, x, _t(6, dtype=torch.float32), _t(5, dtype=torch.float32)),
           lambda: sq.route(_t(6, 2), 3), lambda: sq.route(_t(6, 65, dtype=torch.int32), 3),
           lambda: sq.route(_t(6, 2, dtype=torch.int32), 0), lambda: sq.route(_t(6, 2, dtype=torch.int32), 1025),
           lambda: sq.route(_t(4, 6, dtype=torch.int32).t(), 3),
           lambda: sq.Routing(r.offsets, r.rows[:-1], r.slots), lambda: sq.Routing(r.offsets[:1], r.rows, r.slots),
           lambda: sq.Routing(r.offsets.long(), r.rows, r.slots), lambda: sq.Routing(r.offsets, r.rows, r.rows),
           lambda: sq.permute_rows(_t(5, 64), r), lambda: sq.permute_rows(x, (r.offsets, r.rows, r.slots)),
           lambda: sq.permute_rows(x, r, out=_t(6, 64)), lambda: sq.combine(_t(12, 64), r, _t(6, 2)),
           lambda: sq.combine(_t(12, 64), r, _t(6, 3, dtype=torch.float32)), lambda: sq.combine(_t(12, 64), r, residual=_t(12, 64)),
           lambda: sq.combine_backward(_t(12, 64), _t(12, 64), r, _t(6, 2, dtype=torch.float32)),
           lambda: sq.combine_backward(x, _t(12, 64), r, None)]
    a, b, r1 = _t(3, 16, 64), _t(3, 32, 16), _routing(6, 1)
    bad += [lambda: sq.lora(x, a, b, r), lambda: sq.lora(x, a[:2], b, r1), lambda: sq.lora(x, a, b[:, :30], r1),
            lambda: sq.lora(x.float(), a.float(), b.float(), r1), lambda: sq.lora(x, a.float(), b, r1),
            lambda: sq.lora(x, a, b, r1, scales=_t(3)), lambda: sq.lora(x, a, b, r1, base=_t(6, 64)),
            lambda: sq.lora(x, _t(3, 12, 64), _t(3, 32, 12), r1), lambda: sq.lora(x, _t(3, 136, 64), _t(3, 32, 136), r1),
            lambda: sq.lora(_t(6, 128)[:, ::2], a, b, r1), lambda: sq.lora(_t(1, 64).expand(6, 64), a, b, r1),
            lambda: sq.lora(_t(6, 100)[:, :64], a, b, r1), lambda: sq.lora(x, a, b, _routing(5, 1)),
            lambda: sq.lora(x, a, b, _routing(6, 1, 4)), lambda: sq.lora(x, a, b, r1, out=_t(6, 64)[:, 4:36])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was taken")
    assert not [c for c in here.mock_calls if "bytes" not in str(c)]


def test_binding_refuses_to_lose_a_gradient(here):
    x = _t(6, 64)
    w = _as_cuda(torch.zeros(64, dtype=torch.float16, requires_grad=True))
    with pytest.raises(ValueError, match="require a gradient"):
        sq.layer_norm(x, w)
    with torch.no_grad():
        sq.layer_norm(x, w)
    assert here.sharq_layer_norm.called


def test_binding_refuses_outputs_that_require_a_gradient(here):
    x, r, r1 = _t(6, 64), _routing(), _routing(6, 1)
    stat = _t(6, dtype=torch.float32)

    def leaf(*shape):
        return _as_cuda(torch.zeros(shape, dtype=torch.float16, requires_grad=True))

    for f in (lambda: sq.layer_norm(x, out=leaf(6, 64)), lambda: sq.layer_norm_backward(x, x, stat, stat, out=leaf(6, 64)),
              lambda: sq.permute_rows(x, r, out=leaf(12, 64)), lambda: sq.combine(_t(12, 64), r, out=leaf(6, 64)),
              lambda: sq.lora(x, _t(3, 16, 64), _t(3, 32, 16), r1, out=leaf(6, 32))):
        with pytest.raises(ValueError, match="require a gradient"):
            f()


def test_routing_refuses_other_objects(here):
    r = _routing()
    for args in ((None, r.rows, r.slots), (r.offsets, None, r.slots), (r.offsets, r.rows, None), ([0, 1], r.rows, r.slots)):
        with pytest.raises(ValueError):
            sq.Routing(*args)


def test_valid_calls_reach_the_library(here):
    f32 = torch.float32
    x, r, r1 = _t(6, 64), _routing(), _routing(6, 1)
    y, mean, rstd = sq.layer_norm(x, _t(64), _t(64), stats=True)
    assert mean.shape == rstd.shape == (6,)
    assert sq.layer_norm(x, _t(64), norm="rms", stats=True)[1] is None
    dx, dw, db = sq.layer_norm_backward(x, x, mean, rstd, _t(64))
    assert dx.shape == x.shape and dw.shape == db.shape == (64,) and dw.dtype == f32
    assert sq.layer_norm_backward(x, x, None, rstd, _t(64), norm="rms")[2] is None
    assert sq.layer_norm_backward(x, x, mean, rstd)[1:] == (None, None)
    q = sq.route(_t(6, 2, dtype=torch.int64), 3)
    assert (q.groups, q.m_tok, q.top_k) == (3, 6, 2)
    assert here.sharq_route.call_args[0][1] == 8  # int64 ids
    assert sq.permute_rows(x, r).shape == (12, 64)
    w = _t(6, 2, dtype=f32)
    assert sq.combine(_t(12, 64), r, w, residual=x).shape == (6, 64)
    dy, dw = sq.combine_backward(x, _t(12, 64), r, w)
    assert dy.shape == (12, 64) and dw.shape == (6, 2)
    wide = _t(6, 128)
    a, b = _t(3, 16, 64), _t(3, 32, 16)
    sq.lora(wide[:, 64:], a, b, r1, scales=_t(3, dtype=f32), base=_t(6, 32))
    args = here.sharq_lora.call_args[0]
    assert args[1:4] == (128, 6, 64) and args[6:9] == (32, 16, 3) and args[15] == 32 and args[17] == 32
    one = sq.lora(_t(1, 128)[:, :64], a, b, _routing(1, 1))  # a single row has no stride of its own
    assert one.shape == (1, 32) and here.sharq_lora.call_args[0][1] == 64

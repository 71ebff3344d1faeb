"""More refusals of the operators around the FP4 linear, without a GPU: calls
that would leave an output unwritten or lose a derivative."""
import ctypes as C

import pytest
import torch
from torch.autograd import forward_ad

import sparsity_gemm_b200 as sq
from test_operator_checks import _as_cuda, _routing, _t, here  # noqa: F401  (here: a fixture)

P = lambda i: C.c_void_p(i << 32)  # noqa: E731  far apart, aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from sparsity_gemm_b200 import build
    build.build()
    return sq.lib()


@pytest.mark.parametrize("m", [0, 4])
def test_rms_norm_has_no_gradient_of_b(L, m):
    """No db where there is no b: it would come back unwritten."""
    ws = L.sharq_layer_norm_backward_bytes(m, 256)
    call = lambda dw, db: L.sharq_layer_norm_backward(  # noqa: E731
        P(1), P(2), m, 256, P(3), None, P(5), 1, 0, P(6), dw, db, P(9), ws, None)
    assert call(P(7), P(8)) == sq.ERR_INVALID_ARG
    assert call(None, P(8)) == sq.ERR_INVALID_ARG


def _calls():
    """Every call with each of its floating tensors in turn, as (name, function
    of that tensor, the tensor's shape and type)."""
    x, f32, f16 = _t(6, 64), torch.float32, torch.float16
    r, r1, y = _routing(), _routing(6, 1), _t(12, 64)
    stat, ew = _t(6, dtype=f32), _t(6, 2, dtype=f32)
    a, b, sc = _t(3, 16, 64), _t(3, 32, 16), _t(3, dtype=f32)
    return {
        "layer_norm": [(lambda t: sq.layer_norm(t), (6, 64), f16), (lambda t: sq.layer_norm(x, t), (64,), f16),
                       (lambda t: sq.layer_norm(x, None, t), (64,), f16), (lambda t: sq.layer_norm(x, out=t), (6, 64), f16)],
        "layer_norm_backward": [(lambda t: sq.layer_norm_backward(t, x, stat, stat), (6, 64), f16),
                                (lambda t: sq.layer_norm_backward(x, t, stat, stat), (6, 64), f16),
                                (lambda t: sq.layer_norm_backward(x, x, t, stat), (6,), f32),
                                (lambda t: sq.layer_norm_backward(x, x, stat, t), (6,), f32),
                                (lambda t: sq.layer_norm_backward(x, x, stat, stat, t), (64,), f16),
                                (lambda t: sq.layer_norm_backward(x, x, stat, stat, out=t), (6, 64), f16)],
        "permute_rows": [(lambda t: sq.permute_rows(t, r), (6, 64), f16), (lambda t: sq.permute_rows(x, r, out=t), (12, 64), f16)],
        "combine": [(lambda t: sq.combine(t, r), (12, 64), f16), (lambda t: sq.combine(y, r, t), (6, 2), f32),
                    (lambda t: sq.combine(y, r, residual=t), (6, 64), f16), (lambda t: sq.combine(y, r, out=t), (6, 64), f16)],
        "combine_backward": [(lambda t: sq.combine_backward(t, y, r, ew), (6, 64), f16),
                             (lambda t: sq.combine_backward(x, t, r, ew), (12, 64), f16),
                             (lambda t: sq.combine_backward(x, y, r, t), (6, 2), f32)],
        "lora": [(lambda t: sq.lora(t, a, b, r1), (6, 64), f16), (lambda t: sq.lora(x, t, b, r1), (3, 16, 64), f16),
                 (lambda t: sq.lora(x, a, t, r1), (3, 32, 16), f16), (lambda t: sq.lora(x, a, b, r1, scales=t), (3,), f32),
                 (lambda t: sq.lora(x, a, b, r1, base=t), (6, 32), f16), (lambda t: sq.lora(x, a, b, r1, out=t), (6, 32), f16)],
    }


@pytest.mark.parametrize("name", ["layer_norm", "layer_norm_backward", "permute_rows", "combine", "combine_backward", "lora"])
def test_tensors_whose_derivative_would_be_lost(here, name):
    """A tensor that requires a gradient, and one that carries a forward-mode
    tangent, also under no_grad, which does not end forward mode."""
    for i, (f, shape, dtype) in enumerate(_calls()[name]):
        leaf = _as_cuda(torch.zeros(shape, dtype=dtype, requires_grad=True))
        with pytest.raises(ValueError, match="require a gradient"):
            f(leaf)
            pytest.fail(f"case {i} was taken")
        with forward_ad.dual_level():
            dual = _as_cuda(forward_ad.make_dual(torch.zeros(shape, dtype=dtype), torch.ones(shape, dtype=dtype)))
            assert forward_ad.unpack_dual(dual).tangent is not None
            for mode in (torch.enable_grad, torch.no_grad):
                with mode(), pytest.raises(ValueError, match="tangent"):
                    f(dual)
                    pytest.fail(f"case {i} was taken")
            assert not getattr(here, "sharq_" + name).called
            f(_t(*shape, dtype=dtype))  # others are taken inside a dual level
            assert getattr(here, "sharq_" + name).called
            here.reset_mock()

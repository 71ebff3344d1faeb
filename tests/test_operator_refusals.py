"""More refusals of the operators around the FP4 linear, without a GPU: calls
that would leave an output unwritten or lose a derivative."""
import ctypes as C

import pytest

import sparsity_gemm_b200 as sq

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

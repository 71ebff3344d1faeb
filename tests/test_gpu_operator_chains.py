"""Calls that write in place of an input, each followed at once by kernels that
read the result and start before the writer has ended: the bits are those of
calls on copies with a pause after each. Widths of odd rows make neighbouring
rows share a memory sector."""
import pytest
import torch

import sparsity_gemm_b200 as sq

pytestmark = pytest.mark.gpu

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def _inputs(seed, m, k, top_k, dt):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)  # noqa: E731
    ids = torch.randint(-1, 5, (m, top_k), generator=gen, device="cuda", dtype=torch.int32)
    c = dict(x=r(m, k), h=r(m, k), dy=r(m, k), w=r(k), b=r(k), y=r(m * top_k, k), ids=ids,
             ew=torch.rand(m, top_k, generator=gen, device="cuda"), aids=ids[:, 0].contiguous())
    if dt != torch.float32 and k % 8 == 0:
        c["a"], c["bb"] = r(5, 16, k), r(5, k, 16)
    return c


def _chain(c, pause):
    """Each result in place of the buffer before it, read by the next calls."""
    def at(t):  # a buffer to write to: the tensor itself, or a copy after all that ran
        if not pause:
            return t
        torch.cuda.synchronize()
        t = t.clone()
        torch.cuda.synchronize()
        return t

    h, dy = c["h"].clone(), c["dy"].clone()
    e = sq.route(c["ids"], 5)
    n, mean, rstd = sq.layer_norm(c["x"], c["w"], c["b"], stats=True)
    # residual stream: h += what the experts give, then the norm of it
    out = at(h)
    h1 = sq.combine(c["y"], e, c["ew"], residual=out, out=out)
    n1, mean1, rstd1 = sq.layer_norm(h1, c["w"], c["b"], stats=True)
    back = sq.permute_rows(h1, e)
    keep1 = h1.clone()
    # the gradient in place of dy, then the gradient of the way back from it
    out = at(dy)
    dx, dw, db = sq.layer_norm_backward(out, h1, mean1, rstd1, c["w"], out=out)
    ey, ew = sq.combine_backward(dx, c["y"], e, c["ew"])
    dx2 = sq.layer_norm(dx, c["w"], c["b"])
    keep = dx.clone()
    res = [n, n1, mean1, rstd1, back, keep1, keep, dw, db, ey, ew, dx2]
    if "a" in c:  # the adapters on top of h in place, the norm and the way there of that
        r = sq.route(c["aids"], 5)
        out = at(h1)
        o = sq.lora(n1, c["a"], c["bb"], r, base=out, out=out)
        res += [sq.layer_norm(o, c["w"], c["b"]), sq.permute_rows(o, e), sq.lora(o, c["a"], c["bb"], r, base=o), o.clone()]
    return res


@pytest.mark.parametrize("dt", list(DTYPES))
@pytest.mark.parametrize("m,k,top_k", [(64, 256, 2), (700, 1000, 4), (700, 999, 4), (40, 4099, 1), (4000, 136, 2), (3, 8201, 9),
                                       (1500, 24, 2), (301, 9000, 1)])
def test_results_in_place_are_read_at_once(m, k, top_k, dt):
    for seed in range(6):
        c = _inputs(seed, m, k, top_k, DTYPES[dt])
        want = _chain(c, True)
        torch.cuda.synchronize()
        for _ in range(3):
            got = _chain(c, False)
        torch.cuda.synchronize()
        for i, (g, w) in enumerate(zip(got, want)):
            assert torch.equal(g, w), i
    assert sq.get_last_error() == sq.OK

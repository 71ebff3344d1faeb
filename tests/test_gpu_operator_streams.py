"""The operators around the FP4 linear on streams other than the current one,
on two streams at once, from two host threads, and in two captured graphs that
share a memory pool and replay in turn, and on inputs rewritten right before:
always the bits of a plain call."""
import threading

import pytest
import torch

import sparsity_gemm_b200 as sq

pytestmark = pytest.mark.gpu


def _inputs(seed, m=1500, k=256, n=264, rank=48, groups=6, top_k=4, experts=9):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").half()  # noqa: E731
    ids = torch.randint(-1, groups, (m,), generator=gen, device="cuda", dtype=torch.int32)
    return dict(x=r(m, k), dy=r(m, k), w=r(k), b=r(k), a=r(groups, rank, k), bb=r(groups, n, rank), base=r(m, n), ids=ids,
                eids=torch.randint(-1, experts, (m, top_k), generator=gen, device="cuda"), y=r(m * top_k, k),
                ew=torch.rand(m, top_k, generator=gen, device="cuda"), groups=groups, experts=experts)


def _all(c, stream=None):
    """Every operator once; the two-launch adapters and the gradients use
    workspaces of their own."""
    y, mean, rstd = sq.layer_norm(c["x"], c["w"], c["b"], stats=True, stream=stream)
    grads = sq.layer_norm_backward(c["dy"], c["x"], mean, rstd, c["w"], stream=stream)
    r = sq.route(c["ids"], c["groups"], stream=stream)
    out = sq.lora(y, c["a"], c["bb"], r, base=c["base"], stream=stream)
    few = sq.lora(y[:5], c["a"], c["bb"], sq.route(c["ids"][:5], c["groups"], stream=stream), base=c["base"][:5], stream=stream)
    e = sq.route(c["eids"], c["experts"], stream=stream)
    moved = sq.permute_rows(c["x"], e, stream=stream)
    back = sq.combine(c["y"], e, c["ew"], c["x"], stream=stream)
    eg = sq.combine_backward(c["dy"], c["y"], e, c["ew"], stream=stream)
    return [y, mean, rstd, *grads, r.offsets, r.rows, r.slots, out, few, e.offsets, e.rows, e.slots, moved, back, *eg]


def _same(got, want):
    assert len(got) == len(want)
    for i, (g, w) in enumerate(zip(got, want)):
        assert torch.equal(g, w), i


def test_another_stream():
    c = _inputs(1)
    want = _all(c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = _all(c, stream=s)
    s.synchronize()
    _same(got, want)
    with torch.cuda.stream(s):  # as the current stream
        got = _all(c)
    s.synchronize()
    _same(got, want)
    assert sq.get_last_error() == sq.OK


def test_two_streams_at_once():
    cs = [_inputs(2), _inputs(3)]
    want = [_all(c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(4):
        for i in (0, 1):
            got[i] = _all(cs[i], stream=streams[i])
    for s in streams:
        s.synchronize()
    for i in (0, 1):
        _same(got[i], want[i])
    assert sq.get_last_error() == sq.OK


def test_two_host_threads():
    cs = [_inputs(4), _inputs(5)]
    want = [_all(c) for c in cs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(6):
                got = _all(cs[i], stream=s)
            s.synchronize()
            _same(got, want[i])
        except Exception as e:  # noqa: BLE001  reported by the main thread
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad
    assert sq.get_last_error() == sq.OK


def test_two_graphs_of_one_pool():
    cs = [_inputs(6), _inputs(7)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for c in cs:
            _all(c)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            outs.append(_all(c))
        graphs.append(g)
    for seed in (8, 10):
        for i in (0, 1):
            new = _inputs(seed + i)
            for key, v in new.items():
                if isinstance(v, torch.Tensor):
                    cs[i][key].copy_(v)
            graphs[i].replay()
            torch.cuda.synchronize()
            got = [t.clone() for t in outs[i]]  # the other graph may use the same memory
            _same(got, _all(new))
    assert sq.get_last_error() == sq.OK


@pytest.mark.parametrize("m,rank,groups", [(96, 64, 3), (1100, 16, 5), (40, 16, 3), (1100, 64, 3), (130, 64, 160)])
def test_inputs_changed_right_before_a_call(m, rank, groups):
    """Weights, adapters' ids, base and statistics that a small kernel rewrites
    in place right before each call (the next one's first loads may already be
    on their way): the results are those of tensors that were never touched."""
    k, n, top_k, steps = 192, 328, 2, 48
    gen = torch.Generator(device="cuda").manual_seed(m)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").half()  # noqa: E731
    x, a = r(m, k), r(groups, rank, k)
    bs, bases, ws = r(steps, groups, n, rank), r(steps, m, n), r(steps, k)
    ids = torch.randint(-1, groups, (steps, m), generator=gen, device="cuda", dtype=torch.int32)
    eids = torch.randint(-1, groups, (steps, m, top_k), generator=gen, device="cuda", dtype=torch.int32)
    ew = torch.rand(steps, m, top_k, generator=gen, device="cuda")

    def step(b, base, w, i, e, v):
        y, mean, rstd = sq.layer_norm(x, w, stats=True)
        dx, dw, db = sq.layer_norm_backward(y, x, mean, rstd, w)
        out = sq.lora(x, a, b, sq.route(i, groups), base=base)
        q = sq.route(e, groups)
        g = sq.permute_rows(y, q)
        back = sq.combine(g, q, v, x)
        return [y, dx, dw, db, out, g, back, *sq.combine_backward(y, g, q, v)]

    mine = [t[0].clone() for t in (bs, bases, ws, ids, eids, ew)]
    got = []
    for s in range(steps):
        for t, from_ in zip(mine, (bs, bases, ws, ids, eids, ew)):
            t.copy_(from_[s])
        got.append(step(*mine))
    torch.cuda.synchronize()
    for s in range(steps):
        _same(got[s], step(bs[s], bases[s], ws[s], ids[s], eids[s], ew[s]))
    assert sq.get_last_error() == sq.OK


def test_a_stream_of_another_device_is_refused():
    class Elsewhere:
        device_index = torch.cuda.current_device() + 1
        cuda_stream = 0

    x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
    with pytest.raises(ValueError, match="stream is on cuda"):
        sq.layer_norm(x, out=torch.empty_like(x), stream=Elsewhere())

"""The mixture-of-experts layer on a batch with padding tokens (id -1), the two
ways the README gives, against the same layer without those tokens: the real
tokens' rows come out with the same bits, padding tokens keep their residual."""
import numpy as np
import pytest
import torch

import sparsity_gemm_b200 as sq
import synth

pytestmark = pytest.mark.gpu

TOKENS, TOP_K, GROUPS, K, N_OUT = 96, 4, 8, 256, 512


def _experts():
    return sq.quantize_weight_grouped(torch.from_numpy(
        np.stack([synth.weights(150 + g, N_OUT, K) for g in range(GROUPS)]).view(np.float16)).cuda())


def _batch(seed, padded, single=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.from_numpy(synth.activations_student(seed, TOKENS, K).view(np.float16)).cuda()
    ids = torch.randint(0, GROUPS, (TOKENS, TOP_K), generator=gen, device="cuda", dtype=torch.int32)
    at = torch.randperm(TOKENS, generator=gen, device="cuda")[:padded]
    ids[at] = -1
    if single and padded < TOKENS:
        ids[ids >= 0] = 0  # the last expert has no entry of its own
    w = torch.rand(TOKENS, TOP_K, generator=gen, device="cuda")
    res = torch.randn(TOKENS, N_OUT, generator=gen, device="cuda").half()
    return x, ids, w, res


def _with_count(x, ids, w, res, experts):
    r = sq.route(ids, GROUPS)
    n = int(r.offsets[-1])
    p = sq.gather_rows(sq.prepare(x), r.rows[:n], r.offsets, n)
    return sq.combine(sq.linear_grouped(p, r.offsets, experts, n), r, w, residual=res)


def _without_wait(x, ids, w, res, experts):
    r = sq.route(ids, GROUPS)
    offsets = r.offsets.clone()
    offsets[-1:] = r.rows.numel()
    p = sq.gather_rows(sq.prepare(x), r.rows.clamp_min(0), offsets, r.rows.numel())
    return sq.combine(sq.linear_grouped(p, offsets, experts, r.rows.numel()), r, w, residual=res)


def _want(x, ids, w, res, experts):
    """The real tokens alone; their preparation is the batch's."""
    real = torch.nonzero(ids[:, 0] >= 0).flatten()
    out = res.clone()
    if real.numel():
        r = sq.route(ids[real], GROUPS)
        n = r.rows.numel()
        p = sq.gather_rows(sq.prepare(x), real[r.rows.long()].int(), r.offsets, n)
        out[real] = sq.combine(sq.linear_grouped(p, r.offsets, experts, n), r, w[real], residual=res[real])
    return out


@pytest.mark.parametrize("layer", [_with_count, _without_wait])
@pytest.mark.parametrize("padded,single", [(0, False), (13, False), (95, False), (13, True), (96, False)])
def test_padding_tokens(layer, padded, single):
    experts = _experts()
    c = _batch(3 + padded, padded, single)
    want = _want(*c, experts)
    assert torch.equal(layer(*c, experts), want)
    assert torch.equal(want[c[1][:, 0] < 0], c[3][c[1][:, 0] < 0])
    assert sq.get_last_error() == sq.OK


def test_in_a_graph():
    experts = _experts()
    c = _batch(20, 9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _without_wait(*c, experts)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _without_wait(*c, experts)
    for seed, padded in ((21, 0), (22, 40), (23, 96)):
        d = _batch(seed, padded)
        for have, new in zip(c, d):
            have.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, _want(*d, experts))
    assert sq.get_last_error() == sq.OK


def test_a_routing_with_padding_is_refused_as_it_is():
    """The grouped calls want every row in a group, and say so."""
    x, ids, w, res = _batch(30, 13)
    r = sq.route(ids, GROUPS)
    sq.gather_rows(sq.prepare(x), r.rows, r.offsets, r.rows.numel())
    assert sq.get_last_error() == sq.ERR_INVALID_ARG

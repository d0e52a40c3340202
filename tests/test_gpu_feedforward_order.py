"""Stream order of the feed-forward operators' weights on a B200: fp16 weights
that the kernel right before the call writes -- an ordinary one, or one of the
library's own, which lets its successor start early -- are the ones the call
uses, on every kernel that the number of tokens selects, eager and captured.
All factors are powers of two, so the results are compared byte for byte."""
import pytest
import torch

import int8_int4_b200 as aq
from test_gpu_feedforward import normal, weight

pytestmark = pytest.mark.gpu

N, K = 1536, 512
FACTORS = (1.0, 0.5, -2.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    aq.load_library()
    yield
    aq.device_status()


def calls(M):
    X, b, R = normal(1, M, K), normal(2, N), normal(3, M, N)
    return {
        "plain": lambda Wg, Wu: aq.qgemm_act("f16", X, Wg, None, bias=b),
        "act": lambda Wg, Wu: aq.qgemm_act("f16", X, Wg, None, bias=b, act="gelu"),
        "residual": lambda Wg, Wu: aq.qgemm_act("f16", X, Wg, None, residual=R),
        "gated": lambda Wg, Wu: aq.qgemm_gated("f16", X, Wg, None, Wu, None),
    }


def check(call, write):
    """`write(k)` fills both weights with k times a fixed pair."""
    refs = []
    for k in FACTORS:
        Wg, Wu = write(k)
        torch.cuda.synchronize()
        refs.append(call(Wg, Wu).clone())
        torch.cuda.synchronize()
    assert not torch.equal(refs[0], refs[1])
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        for k in FACTORS:
            outs.append(call(*write(k)))
    for _ in range(20):
        for ref, k in zip(refs, FACTORS):
            assert torch.equal(call(*write(k)), ref)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, refs))


@pytest.mark.parametrize("M", [1, 16, 64, 100, 300])
@pytest.mark.parametrize("name", ["plain", "act", "residual", "gated"])
def test_written_by_an_ordinary_kernel(M, name):
    g0, u0 = normal(4, N, K, std=0.05), normal(5, N, K, std=0.05)
    Wg, Wu = torch.empty_like(g0), torch.empty_like(u0)

    def write(k):
        torch.mul(u0, k, out=Wu)
        torch.mul(g0, k, out=Wg)
        return Wg, Wu
    check(calls(M)[name], write)


@pytest.mark.parametrize("M", [1, 16, 64, 100, 300])
@pytest.mark.parametrize("name", ["plain", "act", "residual", "gated"])
def test_written_by_a_call_of_the_library(M, name):
    """The weight is another call's result: a product of two factors added to it (a
    low-rank update)."""
    A, B = normal(6, N, 64, std=0.2), normal(7, K, 64, std=0.05)
    g0, Wg, Wu = normal(8, N, K, std=0.05), *(torch.empty(N, K, dtype=torch.float16, device="cuda") for _ in range(2))
    scaled = {k: (A * k, g0 * k) for k in FACTORS}

    def write(k):
        a, g = scaled[k]
        aq.qgemm_act("f16", a, B, None, residual=g, out=Wu)
        aq.qgemm_act("f16", a, B, None, residual=g, out=Wg)
        return Wg, Wu
    check(calls(M)[name], write)


@pytest.mark.parametrize("fmt", ["q8", "q4", "w8a8"])
@pytest.mark.parametrize("M", [1, 16, 64, 300])
def test_packed_by_the_preceding_kernel(fmt, M):
    """Packed weights: pack-then-call on one stream, without and with G and U."""
    X, sx = (normal(1, M, K), None) if fmt != "w8a8" else aq.act_quant(normal(1, M, K))
    g0, u0 = normal(4, N, K, std=0.05), normal(5, N, K, std=0.05)
    scaled = {k: (g0 * k, u0 * k) for k in FACTORS}
    pf = "q4" if fmt == "q4" else "q8"
    Pg, Pu = weight(pf, 9, N, K)[:2], weight(pf, 10, N, K)[:2]
    G, U = (torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(2))
    for save in (None, (G, U)):
        def write(k):
            aq.qpack(pf, scaled[k][1], out=Pu)
            aq.qpack(pf, scaled[k][0], out=Pg)
            return Pg, Pu
        check(lambda g, u: aq.qgemm_gated(fmt, X, *g, *u, sx=sx, save=save), write)


@pytest.mark.parametrize("fmt", ["q8", "q4", "w8a8"])
@pytest.mark.parametrize("M", [1, 16, 64, 300, 1100])
def test_packed_weights_written_by_an_ordinary_kernel(fmt, M):
    """A call that keeps G and U: packed weights and scales that plain copies
    right before it write, the scales last."""
    X, sx = (normal(1, M, K), None) if fmt != "w8a8" else aq.act_quant(normal(1, M, K))
    pf = "q4" if fmt == "q4" else "q8"
    g0, u0 = normal(4, N, K, std=0.05), normal(5, N, K, std=0.05)
    packs = {k: (aq.qpack(pf, g0 * k), aq.qpack(pf, u0 * k)) for k in FACTORS}
    Pg, Pu = weight(pf, 9, N, K)[:2], weight(pf, 10, N, K)[:2]
    G, U = (torch.empty(M, N, dtype=torch.float16, device="cuda") for _ in range(2))

    def write(k):
        for i in (0, 1):
            for dst, src in zip((Pu[i], Pg[i]), (packs[k][1][i], packs[k][0][i])):
                dst.copy_(src)
        return Pg, Pu
    check(lambda g, u: aq.qgemm_gated(fmt, X, *g, *u, sx=sx, save=(G, U)), write)

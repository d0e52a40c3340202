"""Infinities and NaN in the feed-forward epilogues on a B200: an activation
follows its formula in 64 bits (torch's relu, z sigmoid(z), z Phi(z) and
z (1 + tanh w) / 2), so a NaN stays one and act(+inf) is +inf, on every kernel."""
import pytest
import torch

import int8_int4_b200 as aq
from test_gpu_feedforward import ACTS, FMTS, act64, acts, bwd_inputs, grads64, normal, project, weight

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# fp16 half step, the kernels' 2^-16 for an activation, fp32 sums
RTOL = 2.0 ** -11 + 2.0 ** -16 + 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _lib():
    aq.load_library()
    yield
    aq.device_status()


def same(got, ref, tol):
    """NaN and infinities where the reference has them, the rest within tol."""
    got, ref = got.double(), ref
    assert torch.equal(got.isnan(), ref.isnan()), (got.isnan() ^ ref.isnan()).nonzero()[:4].tolist()
    inf = ref.isinf()
    assert torch.equal(got[inf], ref[inf])
    fin = ref.isfinite()
    assert ((got - ref).abs() <= tol)[fin].all()


def poisoned(t):
    """Three entries of a vector's last dimension become +inf, -inf and NaN."""
    t = t.clone()
    t[..., 3], t[..., 17], t[..., t.shape[-1] - 5] = INF, -INF, NAN
    return t


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,N,K", [(3, 208, 512), (12, 64, 256), (40, 400, 512), (300, 1552, 512), (1100, 1040, 2560)])
def test_forward(fmt, act, M, N, K):
    X, sx, x = acts(fmt, 1, M, K)
    Wg, sg, wg = weight(fmt, 2, N, K)
    Wu, su, wu = weight(fmt, 3, N, K)
    b, bu = poisoned(normal(4, N)), normal(5, N)
    R = normal(6, M, N)
    R[M - 1] = poisoned(R[M - 1].roll(1))
    if fmt != "w8a8":
        X[M // 2, 5], X[0, 7] = NAN, INF
        x = X.double()
    z = x @ wg.t() + b.double()
    fin = torch.nan_to_num
    dz = project(fin(x, 0, 0, 0), wg, fin(b, 0, 0, 0))[1]
    a = act64(z, act)
    slack = 1.13 * dz + RTOL * a.abs() + 2.0 ** -25
    same(aq.qgemm_act(fmt, X, Wg, sg, sx=sx, bias=b, act=act, residual=R), a + R.double(),
         slack + RTOL * R.double().abs())
    u, du = x @ wu.t() + bu.double(), project(fin(x, 0, 0, 0), wu, bu)[1]
    G, U = torch.empty_like(R), torch.empty_like(R)
    H = aq.qgemm_gated(fmt, X, Wg, sg, Wu, su, sx=sx, bias_g=b, bias_u=bu, act=act, save=(G, U))
    same(H, a * u, slack * (u.abs() + du) + a.abs() * du + RTOL * (a * u).abs())
    same(G, z, dz + RTOL * z.abs())
    same(U, u, du + RTOL * u.abs())


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [40, 1000])
def test_backward(act, M):
    """Pre-activations that passed fp16's range, or a NaN, in single tokens: the
    bias gradients of their channels, and no other's."""
    N, K = 208, 144
    dH, X, Wg, Wu, G, U = bwd_inputs(M, N, K)
    G[M // 3] = poisoned(G[M // 3])
    dg, du = grads64(dH, G, U, act)
    r = aq.gated_backward(dH, X, Wg, Wu, G, U, act=act)
    for got, d in ((r[3], dg), (r[4], du)):
        s = torch.nan_to_num(d.abs(), 0, 0, 0).sum(0)
        same(got, d.sum(0), (M * 2.0 ** -24 + 2.0 ** -16) * s + RTOL * d.sum(0).abs() + 2.0 ** -25
             + 2.0 ** -16 * (dH.double() * U.double()).abs().sum(0))

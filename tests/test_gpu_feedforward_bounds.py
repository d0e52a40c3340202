"""Where the feed-forward operators' stated error bounds are tight, on a B200:
a W8A8 product that its bias nearly cancels, and gradients among fp16's
subnormals."""
import pytest
import torch

import int8_int4_b200 as aq
from test_gpu_feedforward import H16, SUB, acts, bwd_inputs, close, grads64, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    aq.load_library()
    yield
    aq.device_status()


@pytest.mark.parametrize("M,N,K", [(3, 256, 512), (64, 400, 1040), (130, 1536, 6144), (1100, 1040, 2576)])
def test_w8a8_bias_cancels_the_product(M, N, K):
    """The pre-activation is off by at most 2^-22 (|product| + |bias|): the
    int32 sum becomes fp32 (2^-24 relative), meets the token's scale (2^-24)
    and in one fused step the channel's scale and the bias (2^-24 of the
    result). Here the result is 2^-12 of the product, so this error is as
    large as the result's own fp16 step."""
    X, sx, x = acts("w8a8", 1, M, K)
    W, s, w = weight("w8a8", 2, N, K)
    s = s * 100
    w = W.double() * s.double()[:, None]
    main = x @ w.t()
    row = M // 2
    b = (-main[row]).half()
    z = main + b.double()
    assert float((z[row].abs() / main[row].abs()).median()) < 2.0 ** -11
    tol = 2.0 ** -22 * (main.abs() + b.double().abs())
    Y = aq.qgemm_act("w8a8", X, W, s, sx=sx, bias=b, residual=torch.zeros(M, N, dtype=torch.float16, device="cuda"))
    close(Y, z, tol + H16 * z.abs() + SUB)
    Y = aq.qgemm_act("w8a8", X, W, s, sx=sx, bias=b, act="relu")
    close(Y, z.clamp_min(0), tol + H16 * z.abs() + SUB)
    G, U = torch.empty_like(Y), torch.empty_like(Y)
    aq.qgemm_gated("w8a8", X, W, s, W, s, sx=sx, bias_g=b, act="none", save=(G, U))
    close(G, z, tol + H16 * z.abs() + SUB)


@pytest.mark.parametrize("scale", [2.0 ** -16, 2.0 ** -20, 1.0])
def test_gradients_among_the_subnormals(scale):
    """dG and dU are rounded to fp16: by half a step, 2^-11 of an element of at
    least 2^-14 and 2^-25 of any smaller one, whatever its size. With dH at
    2^-16 the sums over the tokens are normal numbers again, and this error
    of theirs is about 2^-25 / sqrt(3) over the operands' mean square root."""
    M, N, K = 2048, 256, 272
    dH, X, Wg, Wu, G, U = bwd_inputs(M, N, K)
    dH = (torch.sign(dH.double()) * (dH.double().abs() * 10).clamp(0.25, 4) * scale).half()
    dg, du = grads64(dH, G, U, "silu")
    r = aq.gated_backward(dH, X, Wg, Wu, G, U)
    x = X.double()
    for got, d, extra in ((r[1], dg, (dH.double() * U.double()).abs()), (r[2], du, 0)):
        e = (H16 + 2.0 ** -16) * d.abs() + 2.0 ** -16 * extra + SUB
        ref = d.t() @ x
        close(got, ref, e.t() @ x.abs() + (M / 16 + 16) * 2.0 ** -23 * (d.abs().t() @ x.abs()) + H16 * ref.abs() + SUB)
        rms = float(d.pow(2).mean().sqrt())
        rel = float((got.double() - ref).norm() / ref.norm())
        out = SUB / 3 ** 0.5 / float(ref.pow(2).mean().sqrt())
        assert rel <= 1.5 * (SUB / 3 ** 0.5 / rms + out) + 2 * H16

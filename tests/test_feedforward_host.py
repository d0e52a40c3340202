"""Refusals of the feed-forward operators, and their plain forms' agreement
with their definitions, on the host: nothing here reaches a GPU."""
import ctypes

import pytest
import torch

import int8_int4_b200 as aq

P = ctypes.c_void_p
A = 0x100000000          # aligned fake device addresses, far apart: every call below fails validation
BAD = P(A + 8)


def ptr(i):
    return P(A + (i << 36))


@pytest.fixture(scope="module")
def lib():
    from int8_int4_b200 import build
    build.build()
    return aq.load_library()


X, SX, W, S, B, R, V, AL, Y, WU, SU, BU, G, U, DH, DX, DG, DU, DBG, DBU, WS = (ptr(i) for i in range(1, 22))


def act(lib, fmt=4, group=0, M=4, N=32, K=64, x=X, sx=None, w=W, s=None, b=None, a=1, r=None, v=None, alpha=0.0,
        ad=None, y=Y):
    return lib.aria_qgemm_act(fmt, group, M, N, K, x, sx, w, s, b, a, r, v, alpha, ad, y, None)


def gated(lib, fmt=4, group=0, M=4, N=32, K=64, x=X, sx=None, wg=W, sg=None, wu=WU, su=None, bg=None, bu=None, a=2,
          h=Y, g=None, u=None):
    return lib.aria_qgemm_gated(fmt, group, M, N, K, x, sx, wg, sg, wu, su, bg, bu, a, h, g, u, None)


def bwd(lib, a=2, M=4, N=32, K=64, dh=DH, g=G, u=U, x=X, wg=W, wu=WU, dx=DX, dwg=DG, dwu=DU, dbg=DBG, dbu=DBU, ws=WS,
        n=1 << 30):
    return lib.aria_gated_bwd(a, M, N, K, dh, g, u, x, wg, wu, dx, dwg, dwu, dbg, dbu, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1),
    (dict(a=5), 1), (dict(a=-1), 1), (dict(fmt=9), 1),
    (dict(s=S), 1), (dict(sx=SX), 1), (dict(fmt=1), 1), (dict(fmt=3, s=S), 1),
    (dict(r=BAD), 3), (dict(y=BAD), 3), (dict(v=BAD), 3), (dict(v=V, ad=P(A + 2)), 3),
    (dict(M=0), 1), (dict(N=24), 2), (dict(K=24), 2), (dict(fmt=2, group=32, s=S, K=128), 2),
    (dict(fmt=2, group=16, s=S, K=256), 2), (dict(fmt=3, s=S, sx=SX, K=133152), 2), (dict(M=2 ** 31), 1),
    (dict(y=X), 1), (dict(y=W), 1), (dict(y=P(X.value + 4 * 64 * 2 - 16)), 1), (dict(r=P(Y.value + 16)), 1), (dict(r=P(Y.value - 4 * 32 * 2 + 16)), 1),
])
def test_act_refusals(lib, kw, status):
    assert act(lib, **kw) == status
    assert lib.aria_last_error_message()


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(wg=None), 1), (dict(wu=None), 1), (dict(h=None), 1),
    (dict(a=7), 1), (dict(fmt=0), 1), (dict(fmt=1, sg=S), 1), (dict(fmt=1, su=SU), 1), (dict(sg=S), 1), (dict(su=SU), 1),
    (dict(h=X), 1), (dict(h=W), 1), (dict(h=WU), 1), (dict(g=X, u=U), 1), (dict(g=G, u=WU), 1),
    (dict(g=G), 1), (dict(u=U), 1), (dict(g=G, u=G), 1), (dict(g=Y, u=U), 1), (dict(g=G, u=P(Y.value + 16)), 1),
    (dict(g=BAD, u=U), 3), (dict(g=G, u=BAD), 3), (dict(bu=BAD), 3), (dict(wu=BAD), 3),
    (dict(M=-1), 1), (dict(N=8), 2), (dict(K=8), 2), (dict(fmt=2, group=32, sg=S, su=SU, K=128), 2),
    (dict(fmt=1, group=32, sg=S, su=SU), 2), (dict(N=2 ** 30 + 16), 2), (dict(fmt=3, sg=S, su=SU), 1),
])
def test_gated_refusals(lib, kw, status):
    assert gated(lib, **kw) == status
    assert lib.aria_last_error_message()


@pytest.mark.parametrize("kw,status", [
    (dict(dh=None), 1), (dict(g=None), 1), (dict(u=None), 1), (dict(ws=None), 1),
    (dict(dwg=None), 1), (dict(dwu=None), 1), (dict(dbg=None), 1), (dict(dbu=None), 1),
    (dict(dx=None, dwg=None, dwu=None, dbg=None, dbu=None), 1),
    (dict(wg=None), 1), (dict(wu=None), 1), (dict(x=None), 1), (dict(a=9), 1),
    (dict(dh=BAD), 3), (dict(dx=BAD), 3), (dict(dbu=BAD), 3), (dict(ws=P(WS.value + 128)), 3),
    (dict(M=0), 1), (dict(N=24), 2), (dict(K=8), 2), (dict(n=16), 1),
    (dict(dx=X), 1), (dict(dx=DH), 1), (dict(dwg=W), 1), (dict(dwg=DU), 1), (dict(ws=G), 1), (dict(ws=DX), 1),
    (dict(dbg=P(DX.value + 256)), 1),
])
def test_backward_refusals(lib, kw, status):
    assert bwd(lib, **kw) == status
    assert lib.aria_last_error_message()


def test_backward_workspace_size(lib):
    n = ctypes.c_size_t()
    assert lib.aria_gated_bwd_workspace_size(4, 32, 64, None) == 1
    assert lib.aria_gated_bwd_workspace_size(0, 32, 64, ctypes.byref(n)) == 1
    assert lib.aria_gated_bwd_workspace_size(4, 2 ** 31, 64, ctypes.byref(n)) == 1
    assert lib.aria_gated_bwd_workspace_size(4, 32, 0, ctypes.byref(n)) == 1
    assert lib.aria_gated_bwd_workspace_size(2 ** 31 - 1, 2 ** 29, 64, ctypes.byref(n)) == 2
    # dG and dU, 256-byte aligned, then one row of column partials
    assert aq.gated_backward_workspace_size(1, 16, 16) == 256 + 256 + 256
    up = lambda v: (v + 255) // 256 * 256
    for M in (1, 15, 16, 17, 1023, 1024, 1025, 4096, 1 << 20):
        for N, K in ((16, 16), (4096, 1024), (6144, 1536), (1024, 4096)):
            extra = aq.gated_backward_workspace_size(M, N, K) - 2 * up(M * N * 2)
            # at most 64 column partials, and up to 16 partials of dX
            assert 0 < extra <= up(64 * 2 * N * 4) + up(16 * M * K * 4)


def half(*s):
    return torch.zeros(*s, dtype=torch.float16)


def test_no_cpu_path():
    with pytest.raises(ValueError, match="CUDA"):
        aq.qgemm_act("f16", half(4, 64), half(32, 64), None)
    with pytest.raises(ValueError, match="CUDA"):
        aq.qgemm_gated("f16", half(4, 64), half(32, 64), None, half(32, 64), None)
    with pytest.raises(ValueError, match="CUDA"):
        aq.gated_backward(half(4, 32), half(4, 64), half(32, 64), half(32, 64), half(4, 32), half(4, 32))


def meta(*s, dtype=torch.float16):
    """A tensor that says it is on a CUDA device, for the checks that run
    before any pointer is used."""
    class T:
        shape, device, is_cuda = torch.Size(s), torch.device("cuda:0"), True
        dim = staticmethod(lambda: len(s))
        get_device = staticmethod(lambda: 0)
        numel = staticmethod(lambda: torch.Size(s).numel())
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: A)
    T.dtype = dtype
    return T()


@pytest.mark.parametrize("kw,err", [
    (dict(fmt="q5"), ValueError), (dict(act="tanh"), ValueError), (dict(scales=meta(32, dtype=torch.float32)), ValueError),
    (dict(X=meta(4, 64, dtype=torch.float32)), TypeError), (dict(X=meta(64)), ValueError), (dict(Wq=meta(32, 80)), ValueError),
    (dict(bias=meta(33)), ValueError), (dict(bias=meta(32, dtype=torch.float32)), TypeError),
    (dict(residual=meta(4, 33)), ValueError), (dict(residual=meta(4, 32, dtype=torch.bfloat16)), TypeError),
    (dict(steer_vec=meta(32)), TypeError), (dict(out=meta(5, 32)), ValueError), (dict(sx=meta(4, dtype=torch.float32)), ValueError),
    (dict(alpha_dev=meta(2, dtype=torch.float32)), ValueError), (dict(alpha_dev=meta(1)), TypeError),
    (dict(fmt="q8"), ValueError), (dict(fmt="w8a8"), ValueError),
])
def test_act_binding_refusals(kw, err):
    args = dict(fmt="f16", X=meta(4, 64), Wq=meta(32, 64), scales=None)
    with pytest.raises(err):
        aq.qgemm_act(**{**args, **kw})


def test_binding_refuses_strides_and_other_devices():
    t = meta(4, 32)
    type(t).is_contiguous = staticmethod(lambda: False)
    with pytest.raises(ValueError, match="contiguous"):
        aq.qgemm_act("f16", meta(4, 64), meta(32, 64), None, residual=t)
    t = meta(4, 32)
    type(t).device = torch.device("cuda:1")
    type(t).get_device = staticmethod(lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        aq.qgemm_act("f16", meta(4, 64), meta(32, 64), None, residual=t)


@pytest.mark.parametrize("kw,err", [
    (dict(Wu=meta(33, 64)), ValueError), (dict(scales_u=meta(32, dtype=torch.float32)), ValueError),
    (dict(bias_g=meta(31)), ValueError), (dict(bias_u=meta(32, dtype=torch.float32)), TypeError),
    (dict(save=(meta(4, 31), meta(4, 32))), ValueError),
    (dict(act="swiglu"), ValueError),
])
def test_gated_binding_refusals(kw, err):
    args = dict(fmt="f16", X=meta(4, 64), Wg=meta(32, 64), scales_g=None, Wu=meta(32, 64), scales_u=None)
    with pytest.raises(err):
        aq.qgemm_gated(**{**args, **kw})


@pytest.mark.parametrize("kw,err", [
    (dict(X=None), ValueError), (dict(Wg=None), ValueError), (dict(Wu=None), ValueError), (dict(G=None), ValueError),
    (dict(U=meta(4, 31)), ValueError), (dict(dH=meta(4, 32, 1)), ValueError), (dict(act="x"), ValueError),
    (dict(input_grad=False, weight_grad=False, bias_grad=False), ValueError),
    (dict(out=(None,) * 5), ValueError), (dict(out=(None,) * 4), ValueError),
    (dict(workspace=meta(16, dtype=torch.uint8)), ValueError), (dict(workspace=meta(1 << 20)), TypeError),
    (dict(bias_grad=False, out=(meta(4, 64), meta(32, 64), meta(32, 64), meta(32), None)), ValueError),
])
def test_backward_binding_refusals(lib, kw, err):
    args = dict(dH=meta(4, 32), X=meta(4, 64), Wg=meta(32, 64), Wu=meta(32, 64), G=meta(4, 32), U=meta(4, 32))
    with pytest.raises(err):
        aq.gated_backward(**{**args, **kw})


def test_binding_refuses_a_stream_of_another_device(lib):
    class S:
        device, cuda_stream = torch.device("cuda:1"), 0
    with pytest.raises(ValueError, match="cuda:1"):
        aq.qgemm_act("f16", meta(4, 64), meta(32, 64), None, stream=S())
    with pytest.raises(ValueError, match="cuda:1"):
        aq.qgemm_gated("f16", meta(4, 64), meta(32, 64), None, meta(32, 64), None, stream=S())
    with pytest.raises(ValueError, match="cuda:1"):
        aq.gated_backward(meta(4, 32), meta(4, 64), meta(32, 64), meta(32, 64), meta(4, 32), meta(4, 32), stream=S())


@pytest.mark.parametrize("save", [(), (meta(4, 32),), (meta(4, 32), None), (None, None)])
def test_gated_keeps_both_or_neither(save):
    with pytest.raises(ValueError, match="save"):
        aq.qgemm_gated("f16", meta(4, 64), meta(32, 64), None, meta(32, 64), None, save=save)

"""The binding of the feed-forward operators on the host: a stand-in library
and stand-in tensors, nothing reaches a GPU."""
import contextlib
import ctypes

import pytest
import torch

import int8_int4_b200 as aq


def fake(*s, dtype=torch.float16, di=0):
    """A contiguous tensor that says it is on cuda:`di`."""
    class T:
        shape, device, is_cuda = torch.Size(s), torch.device("cuda", di), True
        dim = staticmethod(lambda: len(s))
        get_device = staticmethod(lambda: di)
        numel = staticmethod(lambda: torch.Size(s).numel())
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 0x100000000)
    T.dtype = dtype
    return T()


class Lib:
    """Records each call with the device that was current, which decides the plan:
    device 1 needs a larger workspace than device 0."""

    def __init__(self, monkeypatch, current=0):
        self.current, self.calls = current, []
        monkeypatch.setattr(aq, "load_library", lambda: self)
        monkeypatch.setattr(aq, "_here", lambda di, stream: 77 if stream is None and di == self.current else None)
        monkeypatch.setattr(aq, "_running_on", self.running_on)
        monkeypatch.setattr(torch.cuda, "device", self.device)

    @contextlib.contextmanager
    def device(self, d):
        before, self.current = self.current, d if isinstance(d, int) else d.index
        yield
        self.current = before

    @contextlib.contextmanager
    def running_on(self, di, stream):
        with self.device(di):
            yield 77

    def aria_gated_bwd_workspace_size(self, M, N, K, out):
        self.calls.append(("size", self.current, K))
        ctypes.cast(out, ctypes.POINTER(ctypes.c_size_t))[0] = 4 * M * N + 1000 * (1 + self.current)
        return 0

    def aria_gated_bwd(self, *a):
        self.calls.append(("bwd", self.current, a[3]))
        return 0


M, N, K = 4, 32, 64


def backward(di, ws, **kw):
    t = lambda *s, dtype=torch.float16: fake(*s, dtype=dtype, di=di)
    args = dict(dH=t(M, N), X=t(M, K), Wg=t(N, K), Wu=t(N, K), G=t(M, N), U=t(M, N),
                out=(t(M, K), t(N, K), t(N, K), t(N), t(N)))
    if ws:
        args["workspace"] = t(ws, dtype=torch.uint8)
    return aq.gated_backward(**{**args, **kw})


@pytest.mark.parametrize("current", [0, 1])
def test_backward_plans_for_the_device_of_its_tensors(monkeypatch, current):
    lib = Lib(monkeypatch, current)
    backward(1, 4 * M * N + 2000)
    assert lib.calls == [("size", 1, K), ("bwd", 1, K)]
    with pytest.raises(ValueError, match="workspace"):
        backward(1, 4 * M * N + 1999)
    backward(0, 4 * M * N + 1000)
    with pytest.raises(ValueError, match="workspace"):
        backward(0, 4 * M * N + 999)
    with pytest.raises(ValueError, match="workspace"):
        backward(0, 16)


def test_workspace_size_of_a_device(monkeypatch):
    Lib(monkeypatch, current=0)
    assert aq.gated_backward_workspace_size(M, N, K) == 4 * M * N + 1000
    for d in (1, "cuda:1", torch.device("cuda:1")):
        assert aq.gated_backward_workspace_size(M, N, K, device=d) == 4 * M * N + 2000
    assert aq.gated_backward_workspace_size(M, N, K) == 4 * M * N + 1000


@pytest.mark.parametrize("given", ["X", "Wg", "Wu"])
def test_bias_gradients_accept_any_of_the_inputs(monkeypatch, given):
    """K comes from whichever of X and the weights is given; none is needed."""
    lib = Lib(monkeypatch)
    only = dict(X=None, Wg=None, Wu=None, input_grad=False, weight_grad=False, out=(None,) * 3 + (fake(N), fake(N)))
    backward(0, 4 * M * N + 1000, **only)
    backward(0, 4 * M * N + 1000, **{**only, given: fake(*((M, K) if given == "X" else (N, K)))})
    assert [c[2] for c in lib.calls if c[0] == "bwd"] == [16, K]

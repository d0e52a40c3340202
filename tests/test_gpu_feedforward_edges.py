"""The feed-forward operators' epilogues where a CTA takes several tiles, and the
int8 linear's token-major tiles, on a B200, against 64 bits (bounds as derived
in test_gpu_feedforward)."""
import pytest

import int8_int4_b200 as aq
from test_gpu_feedforward import FMTS, check_act, check_gated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    aq.load_library()
    yield
    aq.device_status()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N", [(4096, 6144), (2800, 4096), (1200, 1552)])
def test_store_boxes_over_several_tiles(fmt, M, N):
    """Tiles of an odd number of 16-token chunks (4096 x 6144: 15), several per
    CTA: the next tile starts with the box that the last one ended with."""
    check_act(fmt, M, N, 256, "gelu", residual=True, steer=True)
    check_act(fmt, M, N, 256, "relu", residual=False, steer=False)
    check_gated(fmt, M, N, 256, "silu", save=True)


# the planner gives these W8A8 linears token-major tiles of 128, 192 and 256
# columns (on 148 SMs); the last row and column tiles are partial
@pytest.mark.parametrize("M,N,K", [(300, 1040, 592), (3000, 1040, 6160), (1100, 3088, 2576)])
@pytest.mark.parametrize("act,residual,steer", [("gelu", True, True), ("silu", False, False), ("none", True, False),
                                                ("relu", False, True)])
def test_w8a8_linear_token_major(M, N, K, act, residual, steer):
    check_act("w8a8", M, N, K, act, residual, steer)
    check_act("w8a8", M, N, K, act, residual, steer, bias=False, seed=70)

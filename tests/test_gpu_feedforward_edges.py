"""The feed-forward operators' epilogues where a CTA takes several tiles, on a
B200, against 64 bits (bounds as derived in test_gpu_feedforward)."""
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

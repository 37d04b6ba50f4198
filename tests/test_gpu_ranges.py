"""The calls around the cache at the ends of their ranges: caps and values far
from one, what a row does not see, rows past 31 bits, every share of the key
heads among the waves."""
import pytest

from test_gpu_kv import aq  # noqa: F401  (aq: the module's fixture)
from test_gpu_scores import _check_prompt

pytestmark = pytest.mark.gpu


# ---- caps -------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,D,cap,scale", [
    ("f16", 128, 1e4, None), ("bf16", 128, 3e4, None), ("bf16", 64, 1e5, None), ("bf16", 128, 1e5, None),
    ("bf16", 256, 1e5, None), ("bf16", 128, 1e6, None), ("bf16", 64, 4e6, None), ("f16", 128, 50.0, 1e-4),
    ("bf16", 128, 50.0, 1e-5), ("f16", 128, 1e3, None), ("f16", 64, 50.0, 1e-3), ("f16", 256, 1e-4, None)])
def test_scores_near_caps_of_any_size(aq, dtype, D, cap, scale):
    """Scores of 0.13 of the cap times a normal variable, so up to 0.6 of it, in
    tiles that all rows see and in those that only some do."""
    size = 0.13 * cap if scale is None else 0.13 * cap / (scale * D ** 0.5)
    _check_prompt(aq, [150], [200], 2, 1, D, dtype, seed=D, softcap=cap, scale=scale, size=size)

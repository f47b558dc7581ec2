"""Rows of an odd number of warps, whose sums of two values end in the middle of 16 bytes: one norm, RMS, no
other features, so that a batch's two rows are all that is summed."""
import pytest

from tests import test_block_norm_gpu as bn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [520, 768, 1100, 1280, 1792, 2816])
@pytest.mark.parametrize("x,res", [("bf16", "bf16"), ("f16", "f32"), ("f32", None)])
@pytest.mark.parametrize("post", [False, True])
def test_odd_warps(gpu_lib, D, x, res, post):
    bn.test_against_the_formulas(gpu_lib, (701, D, x, res, "rms", post, 0, "none", False))

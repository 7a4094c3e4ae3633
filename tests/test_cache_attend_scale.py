"""Score scales of the attention whose base-2 form FP32 does not hold (no GPU needed:
a refused call launches nothing)."""

import pytest
import torch

from tests.test_cache_arguments import ECUDA, EINVAL, I, _attend  # noqa: F401


@pytest.mark.parametrize("scale", [3.0e38, -3.4e38, 2.4e38])
def test_scale_beyond_fp32_in_base_2_is_refused(I, scale):  # noqa: F811
    assert _attend(I, att=dict(scale=scale)) == EINVAL


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 0.0, 1e-45])
def test_other_finite_scales_are_taken(I, scale):  # noqa: F811
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: only where no GPU can follow them")
    assert _attend(I, att=dict(scale=scale)) == ECUDA

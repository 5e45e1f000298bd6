"""Arguments at the ends of what the calls on cached sequences and between blocks take, without a GPU."""
import pytest

import normalization_layernorm_rmsnorm_gb300 as nrm
from test_served_host import attend, lib  # noqa: F401


@pytest.mark.parametrize("scale", [3.0e38, -3.4e38, float("inf"), float("nan")])
def test_a_scale_that_leaves_float32_in_base_two_is_refused(lib, scale):  # noqa: F811
    # exp(scale x) is 2^(scale log2(e) x)
    assert attend(lib, scale=scale) == nrm.NRM_ERR_INVALID_ARG
    assert "scale" in nrm.nrm_last_error_message()


@pytest.mark.parametrize("scale", [2.3e38, -2.3e38, 0.0, 1e-40])
def test_other_scales_are_not(lib, scale):  # noqa: F811
    assert attend(lib, scale=scale) != nrm.NRM_ERR_INVALID_ARG

"""Arguments of paged attention at the ends of their ranges, refused before any device work
(no GPU)."""
import pytest

from test_attn_abi import NAMES, call, dims, moe  # noqa: F401  (a fixture)


@pytest.mark.parametrize("name", NAMES)
def test_scales_whose_product_with_log2_e_is_not_finite(moe, name):
    for scale in (3e38, -3e38, 2.37e38):
        assert call(moe, name, d=dims(moe, scale=scale)) == moe.MOE_ERR_INVALID_ARG
        assert moe.moe_attn_workspace_bytes(dims(moe, scale=scale)) == 0
    for scale in (2.3e38, -2.3e38, 1e-45, 0.0):
        assert moe.moe_attn_workspace_bytes(dims(moe, scale=scale)) > 0

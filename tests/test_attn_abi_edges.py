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


def test_numbers_that_the_dims_cannot_hold(moe):
    """(ctypes keeps the lower 32 bits of them: a window of 2^32 + 5 was one of 5.)"""
    pytest.importorskip("torch")
    good = dict(q_heads=8, kv_heads=2, head_dim=128, page_size=64, window=0, device="cpu")
    assert moe.PagedAttention(**{**good, "window": 2 ** 31 - 1}).dims.window == 2 ** 31 - 1
    for name, value in good.items():
        if name == "device":
            continue
        for x in (value + 2 ** 32, value - 2 ** 32, 2 ** 31, 2 ** 64 + value, -1):
            with pytest.raises(moe.MoEError):
                moe.PagedAttention(**{**good, name: x})
    with pytest.raises(moe.MoEError):
        moe.PagedAttention(**{**good, "head_dim": 0})

"""Sizes and packing of the dense block refuse the configs that its calls refuse, and the header's
limits are the code's."""
import pytest

B = pytest.importorskip("expert_cached_moe_amd.binding")

P = 1 << 20            # a plausible, aligned address; refused calls never follow it


def _status(f, *args):
    with pytest.raises(B.MoeError) as e:
        f(*args)
    return e.value.status


@pytest.mark.parametrize("H,I", [(131072, 64), (64, 131072)])
def test_8bit_widths(H, I):
    cfg = B.make_config(H, I, 1, 1, w_dtype=B.MOE_W_BF16)
    assert B.moe_dense_workspace_bytes(cfg, 3) > 0 and B.moe_dense_save_bytes(cfg, 3) > 0
    assert _status(B.moe_i8_blob_bytes, cfg) == B.MOE_ESHAPE
    ctx = B.moe_create(cfg)
    assert _status(B.moe_i8_pack, ctx, P, P) == B.MOE_ESHAPE
    assert _status(B.moe_i8_ffn, ctx, P, 3, P, P, P) == B.MOE_ESHAPE
    assert "131056" in B.moe_last_error(ctx)
    B.moe_destroy(ctx)


@pytest.mark.parametrize("H,I", [(2 ** 20 + 64, 64), (64, 2 ** 20 + 32)])
@pytest.mark.parametrize("w", [B.MOE_W_F32, B.MOE_W_BF16])
def test_block_widths(H, I, w):
    cfg = B.make_config(H, I, 1, 1, w_dtype=w)
    for f in (B.moe_dense_workspace_bytes, B.moe_dense_save_bytes):
        assert _status(f, cfg, 3) == B.MOE_ESHAPE
    ctx = B.moe_create(cfg)
    assert _status(B.moe_dense_ffn, ctx, P, 3, P, None, P, P) == B.MOE_ESHAPE
    assert _status(B.moe_dense_ffn_backward, ctx, P, P, 3, P, P, P, P, P) == B.MOE_ESHAPE
    B.moe_destroy(ctx)


def test_weight_types():
    mx = B.make_config(256, 64, 1, 1, w_dtype=B.MOE_W_MXFP4)
    for f in (B.moe_dense_workspace_bytes, B.moe_dense_save_bytes):
        assert _status(f, mx, 3) == B.MOE_EUNSUPPORTED
    assert _status(B.moe_i8_blob_bytes, mx) == B.MOE_EUNSUPPORTED
    f32 = B.make_config(128, 64, 1, 1, w_dtype=B.MOE_W_F32)
    assert _status(B.moe_i8_blob_bytes, f32) == B.MOE_EUNSUPPORTED
    assert B.moe_dense_workspace_bytes(f32, 3) > 0 and B.moe_dense_save_bytes(f32, 3) > 0

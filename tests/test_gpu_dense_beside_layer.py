"""The dense block and the layer's shared expert are the same function of the same blob; 8-bit
products take rows of any alignment."""
import numpy as np
import pytest
import torch

from expert_cached_moe_amd.runtime import LayerBuffers
from oracle import dense_oracle as D
from test_gpu_dense import BF16, F32, NAME, TORCH, Ctx, Guarded, _blob, _block_inputs, _check, f64, normal
from test_gpu_dense import B  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 8, 9, 200])
@pytest.mark.parametrize("w", [BF16, F32])
def test_block_is_the_shared_expert(B, w, T):
    H, I = (512, 256) if w == BF16 else (256, 128)         # widths that the layer takes
    rng = np.random.default_rng(T)
    x, _, wg, wu, wd = _block_inputs(rng, T, H, I, w)
    with Ctx(B, H, I, w) as c:
        blob = _blob(B, c, wg, wu, wd)
        work = torch.empty(B.moe_dense_workspace_bytes(c.cfg, T), dtype=torch.uint8, device="cuda")
        y = torch.empty_like(x)
        B.moe_dense_ffn(c.p, x, T, blob, None, y, work)
        torch.cuda.synchronize()
    L = LayerBuffers(B.make_config(H, I, 1, 1, n_shared=1, w_dtype=w), T)
    for t in (L.offsets, L.perm):
        t.zero_()
    ids = np.zeros(T, np.int32)
    L.ffn(x, T, None, [], [], blob, 1, h_ids=ids if T <= 8 else None)
    torch.cuda.synchronize()
    shared = f64(L.o.view(TORCH[w])[T * H: 2 * T * H]).reshape(T, H)
    L.close()
    args = [f64(t) for t in (x, wg, wu, wd)]
    ref, bound = D.block(*args)[0], D.block_bounds(None, *args, NAME[w])["y"]
    _check("block", f64(y), ref, bound)
    _check("shared expert", shared, ref, bound)


@pytest.mark.parametrize("T", [1, 8, 20, 300])
@pytest.mark.parametrize("x_type,y_type,x_off,y_off", [(BF16, BF16, 1, 1), (BF16, BF16, 8, 1), (F32, F32, 1, 3),
                                                       (F32, BF16, 3, 2)])
def test_i8_matmul_any_alignment(B, T, x_type, y_type, x_off, y_off):
    """x and y begin on any element, with rows of odd lengths: the same as from aligned rows."""
    N, K, ldx, ldy = 133, 1040, 1047 if x_off != 8 else 1048, 141
    rng = np.random.default_rng(T)
    flat = normal(rng, x_off + T * ldx, x_type)
    x = flat[x_off:].as_strided((T, K), (ldx, 1))
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda")
    ws = torch.rand(N, device="cuda") * 0.01
    with Ctx(B) as c:
        out = Guarded(y_off + (T - 1) * ldy + N, TORCH[y_type])
        work = torch.empty(B.moe_i8_workspace_bytes(T, K), dtype=torch.uint8, device="cuda")
        B.moe_i8_matmul(c.p, flat[x_off:], x_type, ldx, None, T, w, ws, N, K, out.t[y_off:], y_type, ldy, work)
        torch.cuda.synchronize()
    out.check()
    got = torch.full((T * ldy,), float("nan"), dtype=TORCH[y_type], device="cuda")
    got[: (T - 1) * ldy + N] = out.t[y_off:]
    got = got.view(T, ldy)
    assert torch.isnan(got[:, N:]).all() and torch.isnan(out.t[:y_off]).all()
    q, s = D.quantize_rows(f64(x))
    ref = D.i8_matmul(q, s, w.cpu().numpy(), ws.cpu().numpy())
    _check("y", f64(got[:, :N]), ref, D.i8_bound(ref, NAME[y_type]))

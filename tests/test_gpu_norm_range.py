"""moe_norm at the ends of the range: products h * weight next to nothing.

Bounds (fixed before the first run): as in test_gpu_norm.py; y below 2^-126 is off by up to 2^-134, half a step of the
smallest bf16 numbers, besides."""
import numpy as np
import pytest
import torch

import oracle
from biased_top_routing_amd import _lib as L
from biased_top_routing_amd.runner import to_device
from gpu_util import host, say
from workloads.inputs import f32_to_bf16_bits, rng

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.mark.parametrize("codes,H", [("fp8_e4m3", 256), ("fp8_e4m3", 2048), ("fp8_e4m3", 7168), ("fp8_e4m3", 8192),
                                     ("int8", 256), ("int8", 7168), ("int8", 17408)])
@pytest.mark.parametrize("e", [-100, -116, -122, -124, -126, -130, -136, -141, -145, -149])
def test_vanishing_products(codes, H, e):
    """Rows of magnitudes about 2^e, one of them beside a tile of ordinary ones: codes are numbers, scales finite, and
    codes * scale is the normed row within half a step of its format."""
    say(f"norm of 2^{e} H={H} {codes}")
    T = 5
    g = rng(241, H, e + 200)
    h = np.exp2(max(e, -110)) * g.uniform(1, 2, (T, H)) * g.choice([-1, 1], (T, H))
    h[2, :128] = g.standard_normal(128)
    h[3, :128] = 0
    hb = f32_to_bf16_bits(h.astype(np.float32))
    wb = f32_to_bf16_bits(np.full(H, np.exp2(min(e + 110, 0)), np.float32))
    y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")
    q = torch.full((T, H), 77, dtype=torch.int8, device="cuda")
    s = torch.full((T,) if codes == "int8" else (T, H // 128), float("nan"), device="cuda")
    cfg = L.make_cfg(T, H, 1, 1, 1, 1, 0, 128, 1, 1.0, "bf16", codes)
    L.moe_norm(cfg, None, to_device(hb), None, to_device(wb), EPS, None, y, q, s)
    torch.cuda.synchronize()
    h, w = oracle.decode_act(hb).astype(np.float64), oracle.decode_act(wb).astype(np.float64)
    yr, r = oracle.rms_norm(h, w, EPS)
    yv, sv = host(y).astype(np.float64), host(s).astype(np.float64)
    assert (np.abs(yv - yr) <= np.abs(yr) * (2.0 ** -8 + 2.0 ** -15) + 2.0 ** -134 + 2.0 ** -149 * r[:, None]).all()
    assert np.isfinite(sv).all() and (sv >= 0).all()
    if codes == "int8":
        v, step = host(q) * sv[:, None], sv[:, None] / 2
    else:
        c = host(q).view(np.uint8)
        assert ((c & 0x7F) != 0x7F).all()
        v = torch.from_numpy(c.copy()).view(torch.float8_e4m3fn).double().numpy()
        sc = np.repeat(sv, 128, axis=1)
        v, step = v * sc, np.maximum(np.abs(v) * 2.0 ** -4, 2.0 ** -10) * sc
    # (half a step of the code; a scale below 2^-126 is off by half of 2^-149 of itself; a tile below 2^-133 is 0)
    most = np.abs(h * w).reshape(T, -1, 128).max(2).repeat(128, axis=1) if codes != "int8" else 0
    lost = np.where(most < 2.0 ** -133, np.abs(yr), 0.0) if codes != "int8" else 0.0
    assert (np.abs(v - yr) <= step * (1 + 2.0 ** -12) + np.abs(yr) * 2.0 ** -12
            + 448 * (2.0 ** -149 * r[:, None] + 2.0 ** -149) + lost).all()

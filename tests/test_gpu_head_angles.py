"""Angles of the rotation of query and key heads on the GPU: how near their cosines and sines are, and heads at position 0.

E = 2^-24, a rounding of 1 in fp32.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_gpu_dense_ops import E, rng_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs", [0, moe.MOE_ROPE_PAIRS])
@pytest.mark.parametrize("far", [64, 1 << 20])
def test_cosines_and_sines(pairs, far):
    """Of a pair (1, 0) the rotation gives (cos, sin) themselves. The angle's rest of an eighth of a turn, below 0.8, is rounded
    once (E / 2); the sine adds its last rounding (E / 2) and those of a cubic term below 0.09 (E / 4); the cosine its
    last (E / 2), the square's (E / 3) and the polynomial's (E / 6), and the angle counts 0.71 of itself: 1.4 E each."""
    T, D = 4096, 64
    g = rng_of(71, far)
    pos = torch.from_numpy(g.integers(-far, far, T)).int()
    inv = torch.from_numpy(np.concatenate([10000.0 ** (-np.arange(0, D - 8, 2) / D), 3.0 * g.random(4)])).float()
    a = slice(0, D, 2) if pairs else slice(0, D // 2)
    b = slice(1, D, 2) if pairs else slice(D // 2, D)
    x = torch.zeros((T, 1, D))
    x[..., a] = 1
    x, y = x.cuda(), torch.empty((T, 1, D), device="cuda")
    moe.moe_qk_norm_rope(x, None, y, None, flags=moe.MOE_NO_NORM | pairs, inv_freq=inv.cuda(), positions=pos.cuda())
    y = y[:, 0].double().cpu().numpy()
    angle = pos.double().numpy()[:, None] * inv.double().numpy()  # 21 and 24 bits: exact
    assert abs(y[:, a] - np.cos(angle)).max() <= 1.4 * E
    assert abs(y[:, b] - np.sin(angle)).max() <= 1.4 * E


@pytest.mark.parametrize("D,R", [(64, 64), (72, 72), (30, 30), (80, 60)])
@pytest.mark.parametrize("pairs", [0, moe.MOE_ROPE_PAIRS])
@pytest.mark.parametrize("norm", [True, False])
def test_position_0_leaves_each_value_alone(D, R, pairs, norm):
    """Nothing turns at position 0, so a value that is not finite does not reach its partner; axes that are all 0 say the
    same as none."""
    T, H = 3, 2
    g = rng_of(72, D, R)
    x = torch.from_numpy(g.standard_normal((T, H, D))).float().cuda()
    gr = torch.from_numpy(g.standard_normal((T, H, D))).float().cuda()
    bad = x if not norm else gr  # in a norm, one such value spoils its head; a gradient's only where it is mixed or summed
    bad[0, 0, 1], bad[0, 1, D - 1], bad[2, 1, 0] = float("nan"), float("inf"), -float("inf")
    pos = torch.tensor([0, 3, 0], dtype=torch.int32, device="cuda")
    inv = torch.from_numpy(100.0 ** (-np.arange(0, R, 2) / D)).float().cuda()
    flags = pairs | (0 if norm else moe.MOE_NO_NORM)
    outs = []
    for axis in (None, torch.zeros(R // 2, dtype=torch.uint8, device="cuda")):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        kw = dict(flags=flags, inv_freq=inv, positions=pos, pair_axis=axis)
        dw = torch.zeros(D, device="cuda") if norm else None
        moe.moe_qk_norm_rope(x, None, y, None, **kw)
        moe.moe_qk_norm_rope_grad(x, None, gr if norm else x, None, dx, None, dq_weight=dw, **kw)
        outs.append([y, dx] + ([dw] if norm else []))
    for one, other in zip(*outs):
        assert torch.equal(torch.isnan(one), torch.isnan(other))
        assert torch.equal(torch.nan_to_num(one, 0, 1, -1), torch.nan_to_num(other, 0, 1, -1))
    y, dx = outs[0][:2]
    if norm:
        # the weights' gradient: sums over the heads of each value's own
        dw = outs[0][2]
        spoilt = torch.zeros(D, dtype=torch.bool, device="cuda")
        spoilt[[0, 1, D - 1]] = True
        assert torch.equal(~torch.isfinite(dw), spoilt)
        return
    for t in (0, 2):
        for out in (y, dx):
            assert torch.equal(torch.nan_to_num(out[t], 7, 8, 9), torch.nan_to_num(x[t], 7, 8, 9))

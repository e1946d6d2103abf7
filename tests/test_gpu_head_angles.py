"""Angles of the rotation of query and key heads on the GPU: how near their cosines and sines are.

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

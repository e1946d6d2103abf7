"""What the operators beside the experts refuse, before any device call (CPU
only), and the host-side split of canonical 4-bit blocks."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from workload import q4_matrix  # noqa: E402

P = 0x10000  # an address no call here may touch

NORM = dict(device=0, stream=None, n_tokens=2, hidden=64, x_type=moe.MOE_F32, x=P, x_stride=64, res_type=moe.MOE_F32,
            residual=2 * P, res_stride=64, residual_out=3 * P, res_out_stride=64, weight=4 * P, eps=1e-6,
            out_type=moe.MOE_BF16, out=5 * P, out_stride=64, scales=None, scales_stride=0)
Q4 = dict(device=0, stream=None, n_tokens=2, n_out=8, k=64, x_type=moe.MOE_F32, x=P, x_stride=64, x_scales=None,
          x_scales_stride=0, nibbles=2 * P, w_scales=3 * P, y_type=moe.MOE_F32, y=4 * P, y_stride=8, workspace=5 * P,
          workspace_bytes=1 << 30, flags=0)
BAL = dict(device=0, stream=None, n_tokens=2, n_experts=8, top_k=2, z_type=moe.MOE_F32, logits=P, z_stride=8,
           valid=None, balance=1.0, z=0.0, counts=2 * P, load=3 * P, stats=4 * P, lse=5 * P, workspace=6 * P,
           workspace_bytes=1 << 30, flags=0)
GRAD = dict(device=0, stream=None, n_tokens=2, n_experts=8, z_type=moe.MOE_F32, logits=P, z_stride=8, load=3 * P,
            stats=4 * P, lse=5 * P, dloss=None, balance=1.0, z=0.0, d_type=moe.MOE_F32, dlogits=7 * P, d_stride=8,
            flags=0)


def _refused(name, args, what):
    assert getattr(moe.lib(), name)(*args.values()) == moe.MOE_E_INVAL
    msg = moe.moe_last_error(None)
    assert msg.startswith(name) and what in msg, msg


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_tokens=(1 << 24) + 1), "out of range"),
    (dict(hidden=0), "out of range"), (dict(hidden=(1 << 24) + 1), "out of range"),
    (dict(x_type=moe.MOE_Q8_32), "type"), (dict(x_type=9), "type"), (dict(out_type=-1), "type"),
    (dict(res_type=moe.MOE_Q8_32), "residual"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(x=None), "x null"), (dict(x=P + 2), "unaligned"), (dict(x_stride=63), "stride"),
    (dict(out=None), "out null"), (dict(out_stride=63), "stride"), (dict(out=P + 1), "unaligned"),
    (dict(residual=None), "together"), (dict(residual_out=None), "together"), (dict(res_stride=1), "stride"),
    (dict(residual_out=2 * P, res_out_stride=65), "two strides"), (dict(out=P), "in place"),
    (dict(out_type=moe.MOE_F32, out=P, out_stride=65), "in place"), (dict(out=3 * P), "overlap"),
    (dict(out=2 * P), "overlap"), (dict(residual_out=P), "overlap"), (dict(scales=6 * P), "scales"),
    (dict(out_type=moe.MOE_Q8_32), "scales"), (dict(weight=P + 2), "weight"),
    (dict(out_type=moe.MOE_Q8_32, hidden=48, scales=6 * P, scales_stride=2), "multiple of 32"),
    (dict(out_type=moe.MOE_Q8_32, scales=6 * P, scales_stride=1), "scales"),
    (dict(out_type=moe.MOE_Q8_32, scales=6 * P + 2, scales_stride=2), "scales"),
])
def test_add_rmsnorm_refuses(change, what):
    _refused("moe_add_rmsnorm", {**NORM, **change}, what)


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_tokens=(1 << 24) + 1), "out of range"), (dict(n_out=0), "out of range"),
    (dict(n_out=(1 << 22) + 1), "out of range"),
    (dict(k=0), "out of range"), (dict(k=48), "out of range"), (dict(k=(1 << 20) + 32), "out of range"),
    (dict(x_type=4), "out of range"), (dict(y_type=moe.MOE_Q8_32), "type of y"), (dict(flags=2), "flags"),
    (dict(x=None), "x null"), (dict(x=P + 2), "unaligned"), (dict(x_stride=32), "stride"), (dict(y=None), "y null"),
    (dict(y_stride=7), "stride"), (dict(x_scales=6 * P, x_scales_stride=2), "x_scales"),
    (dict(x_type=moe.MOE_Q8_32), "x_scales"),
    (dict(x_type=moe.MOE_Q8_32, x_scales=6 * P, x_scales_stride=1), "x_scales"),
    (dict(nibbles=None), "weight planes"), (dict(nibbles=P + 8), "weight planes"), (dict(w_scales=P + 2), "weight planes"),
    (dict(y=P), "in place"),
])
def test_q4_matmul_refuses(change, what):
    _refused("moe_q4_matmul", {**Q4, **change}, what)


def test_q4_matmul_refuses_a_small_workspace():
    for x_type in (moe.MOE_F32, moe.MOE_F16, moe.MOE_BF16, moe.MOE_Q8_32):
        for T in (200, 4096):
            need = moe.moe_q4_workspace_bytes(T, 4096, 4096, x_type)
            assert need > 0
            a = {**Q4, "n_tokens": T, "n_out": 4096, "y_stride": 4096, "k": 4096, "x_stride": 4096, "x_type": x_type}
            if x_type == moe.MOE_Q8_32:
                a.update(x_scales=6 * P, x_scales_stride=128)
            _refused("moe_q4_matmul", {**a, "workspace_bytes": need - 1}, "workspace")
            _refused("moe_q4_matmul", {**a, "workspace": None}, "workspace")
            _refused("moe_q4_matmul", {**a, "workspace": P + 64}, "workspace")


def test_workspace_sizes_refuse_bad_sizes():
    for bad in ((-1, 8, 64, 0), (1, 0, 64, 0), (1, 8, 63, 0), (1, 8, 0, 0), (1, 8, 64, 4), (1, 8, 64, -1)):
        assert moe.moe_q4_workspace_bytes(*bad) == -1
    assert moe.moe_q4_workspace_bytes(0, 8, 64, 0) == 0
    for bad in ((-1, 8), (1, 0), (1, 4097), ((1 << 24) + 1, 8)):
        assert moe.moe_router_balance_workspace_bytes(*bad) == -1
    assert moe.moe_router_balance_workspace_bytes(0, 8) > 0


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_tokens=(1 << 24) + 1), "out of range"),
    (dict(n_experts=4097), "out of range"), (dict(n_experts=0), "out of range"), (dict(top_k=0), "out of range"),
    (dict(top_k=9), "out of range"), (dict(n_experts=64, z_stride=64, top_k=33), "out of range"),
    (dict(z_type=moe.MOE_Q8_32), "type"), (dict(flags=4), "flags"), (dict(counts=None), "counts"),
    (dict(load=None), "counts"), (dict(stats=P + 2), "counts"), (dict(logits=None), "logits"),
    (dict(logits=P + 2), "logits"), (dict(z_stride=7), "logits"), (dict(lse=None), "lse"),
    (dict(workspace=None), "workspace"), (dict(workspace=P + 16), "workspace"), (dict(workspace_bytes=100), "workspace"),
])
def test_router_balance_refuses(change, what):
    _refused("moe_router_balance", {**BAL, **change}, what)


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_experts=4097), "out of range"), (dict(z_type=3), "type"),
    (dict(d_type=3), "type"), (dict(flags=4), "flags"), (dict(logits=None), "logits"), (dict(z_stride=7), "logits"),
    (dict(dlogits=None), "dlogits"), (dict(d_stride=7), "dlogits"), (dict(load=None), "load"), (dict(stats=None), "load"),
    (dict(lse=P + 1), "load"), (dict(dloss=P + 2), "load"), (dict(dlogits=P, d_stride=9), "in place"),
    (dict(dlogits=P, d_type=moe.MOE_F16), "in place"), (dict(dlogits=P, flags=moe.MOE_ACCUMULATE), "in place"),
])
def test_router_balance_grad_refuses(change, what):
    _refused("moe_router_balance_grad", {**GRAD, **change}, what)


def test_q4_split_is_the_canonical_format():
    blocks = q4_matrix(np.random.default_rng(3), 5, 96)
    nib, scl = moe.moe_q4_split(blocks)
    assert nib.shape == (5, 3, 16) and scl.shape == (5, 3) and scl.dtype == np.float16
    assert np.array_equal(nib, blocks[:, :, 2:])
    assert np.array_equal(scl.view(np.uint16), np.ascontiguousarray(blocks[:, :, :2]).view(np.uint16)[:, :, 0])
    L = moe.lib()
    assert L.moe_q4_split(1, 48, P, P, P) == moe.MOE_E_INVAL
    assert L.moe_q4_split(-1, 64, P, P, P) == moe.MOE_E_INVAL
    assert L.moe_q4_split(1, 64, None, P, P) == moe.MOE_E_INVAL
    assert L.moe_q4_split(0, 64, None, None, None) == moe.MOE_OK
    with pytest.raises(ValueError):
        moe.moe_q4_split(blocks[..., :17])


def test_binding_refuses_tensors_off_the_gpu():
    x, y = torch.zeros(2, 64), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="cuda"):
        moe.moe_add_rmsnorm(x, None, x)
    with pytest.raises(ValueError, match="cuda"):
        moe.moe_q4_matmul(x, torch.zeros(8, 2, 16, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.float16), y)
    z = torch.zeros(8)
    with pytest.raises(ValueError, match="cuda"):
        moe.moe_router_balance(y, 2, z.int(), z, z[:4], z[:2])
    with pytest.raises(ValueError, match="cuda"):
        moe.moe_router_balance_grad(y, z, z[:4], z[:2], y)

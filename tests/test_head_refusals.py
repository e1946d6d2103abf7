"""What the norm and rotation of heads, the product with an epilogue and the log probabilities refuse, before any device
call (CPU only), and what the binding does."""
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_dense_binding import Rows, planes  # noqa: E402
from tests.test_dense_refusals import P, _refused  # noqa: E402

F32, BF16 = moe.MOE_F32, moe.MOE_BF16

LINEAR = dict(device=0, stream=None, n_tokens=2, n_out=8, k=64, x_type=F32, x=P, x_stride=64, x_scales=None, x_scales_stride=0,
              nibbles=2 * P, w_scales=3 * P, bias=4 * P, act=moe.MOE_ACT_SILU, mul_type=BF16, mul=5 * P, mul_stride=8,
              res_type=BF16, residual=6 * P, res_stride=8, y_type=BF16, y=7 * P, y_stride=8, workspace=8 * P,
              workspace_bytes=1 << 30)
HEADS = dict(device=0, stream=None, n_tokens=5, q_heads=4, k_heads=2, head_dim=16, x_type=BF16, q=P, q_stride=96, q_head_stride=16,
             k=2 * P, k_stride=96, k_head_stride=16, q_weight=3 * P, k_weight=4 * P, eps=1e-6, rotary_dim=8, inv_freq=5 * P,
             positions=6 * P, pos_stride=5, n_axes=1, pair_axis=None)
OUTS = dict(out_type=BF16, q_out=7 * P, q_out_stride=64, q_out_head_stride=16, k_out=8 * P, k_out_stride=32, k_out_head_stride=16,
            flags=0)
GRADS = dict(g_type=BF16, gq=7 * P, gq_stride=64, gq_head_stride=16, gk=8 * P, gk_stride=32, gk_head_stride=16, d_type=BF16, dq=9 * P,
             dq_stride=64, dq_head_stride=16, dk=10 * P, dk_stride=32, dk_head_stride=16, dq_weight=11 * P, dk_weight=12 * P,
             workspace=13 * P, workspace_bytes=1 << 30, flags=0)
LOGP = dict(device=0, stream=None, n_tokens=2, n_vocab=50000, z_type=BF16, logits=P, z_stride=50000, targets=2 * P, scale=1.0, logp=3 * P,
            entropy=4 * P, lse=5 * P, top_n=3, top_ids=6 * P, top_logp=7 * P, workspace=8 * P, workspace_bytes=1 << 30)
LGRAD = dict(device=0, stream=None, n_tokens=2, n_vocab=50000, z_type=BF16, logits=P, z_stride=50000, targets=2 * P, scale=1.0, lse=3 * P,
             entropy=4 * P, dlogp=5 * P, dentropy=6 * P, d_type=F32, dlogits=7 * P, d_stride=50000, flags=0)


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_out=0), "out of range"), (dict(k=48), "out of range"), (dict(x_type=4), "out of range"),
    (dict(y_type=moe.MOE_Q8_32), "type of y"), (dict(act=-1), "act"), (dict(act=5), "act"), (dict(mul_type=3), "type of mul"),
    (dict(res_type=9), "type of mul or the residual"), (dict(x=None), "x null"), (dict(y=None), "y null"), (dict(y_stride=7), "stride"),
    (dict(y=7 * P + 1), "unaligned"), (dict(mul_stride=7), "mul"), (dict(mul=5 * P + 1), "mul"), (dict(res_stride=7), "residual"),
    (dict(residual=6 * P + 1), "residual"), (dict(bias=4 * P + 2), "bias"), (dict(y=P), "in place"),
    (dict(y=5 * P, y_type=F32), "in place"), (dict(y=5 * P, mul_stride=9), "in place"), (dict(y=6 * P, res_stride=9), "in place"),
    (dict(nibbles=None), "weight planes"), (dict(w_scales=3 * P + 2), "weight planes"), (dict(x_scales=9 * P, x_scales_stride=2), "x_scales"),
])
def test_q4_linear_refuses(change, what):
    _refused("moe_q4_linear", {**LINEAR, **change}, what)


def test_q4_linear_refuses_a_small_workspace():
    need = moe.moe_q4_workspace_bytes(4096, 4096, 4096, BF16)
    a = {**LINEAR, "n_tokens": 4096, "n_out": 4096, "k": 4096, "x_type": BF16, "x_stride": 4096, "y_stride": 4096, "mul_stride": 4096,
         "res_stride": 4096}
    _refused("moe_q4_linear", {**a, "workspace_bytes": need - 1}, "workspace")
    _refused("moe_q4_linear", {**a, "workspace": None}, "workspace")


COMMON = [
    (dict(n_tokens=-1), "out of range"), (dict(n_tokens=(1 << 24) + 1), "out of range"), (dict(q_heads=0), "out of range"),
    (dict(q_heads=1025), "out of range"), (dict(k_heads=-1), "out of range"), (dict(k_heads=1025), "out of range"),
    (dict(head_dim=15), "out of range"), (dict(head_dim=0), "out of range"), (dict(head_dim=514), "out of range"),
    (dict(rotary_dim=7), "rotary_dim"), (dict(rotary_dim=18), "rotary_dim"), (dict(rotary_dim=-2), "rotary_dim"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(rotary_dim=0), "without rotary_dim"),
    (dict(n_axes=0), "n_axes"), (dict(n_axes=9), "n_axes"), (dict(inv_freq=None), "inv_freq"), (dict(inv_freq=5 * P + 2), "inv_freq"),
    (dict(positions=None), "positions"), (dict(positions=6 * P + 2), "positions"), (dict(n_axes=2, pos_stride=-1), "positions"),
    (dict(n_axes=2, pos_stride=(1 << 36) + 1), "positions"),
    (dict(q_weight=3 * P + 2), "weights"), (dict(k_weight=4 * P + 1), "weights"), (dict(x_type=moe.MOE_Q8_32), "type of q"),
    (dict(q=None), "q "), (dict(q=P + 1), "q "), (dict(q_stride=15), "q "), (dict(q_head_stride=15), "q "), (dict(q_stride=63), "overlap"),
    (dict(k=None), "k "), (dict(k_stride=31), "overlap"), (dict(k_head_stride=8), "overlap"), (dict(flags=16), "flags"),
    (dict(flags=moe.MOE_NO_NORM), "weights without a norm"), (dict(q_stride=(1 << 36) + 1), "overlap"),
]


@pytest.mark.parametrize("change,what", COMMON + [
    (dict(flags=moe.MOE_ACCUMULATE), "flags"), (dict(out_type=3), "type of the outputs"), (dict(q_out=None), "q_out"),
    (dict(k_out=None), "k_out"), (dict(q_out_stride=63), "overlap"), (dict(q_out=P), "in place"),
    (dict(q_out=P, q_out_stride=96, out_type=F32), "in place"), (dict(k_out=2 * P), "in place"), (dict(k_out=7 * P), "outputs overlap"),
    (dict(q_out=2 * P), "outputs overlap"), (dict(k_out=P), "outputs overlap"),
    (dict(rotary_dim=0, inv_freq=None, positions=None, q_weight=None, k_weight=None, flags=moe.MOE_NO_NORM), "neither"),
])
def test_qk_norm_rope_refuses(change, what):
    _refused("moe_qk_norm_rope", {**HEADS, **OUTS, **change}, what)


@pytest.mark.parametrize("change,what", COMMON + [
    (dict(g_type=3), "type of the gradients"), (dict(d_type=-1), "type of the gradients"), (dict(gq=None), "gq"), (dict(dk=None), "dk"),
    (dict(gq_stride=63), "overlap"), (dict(dq=7 * P, d_type=F32), "in place"), (dict(dq=P), "in place"), (dict(dk=8 * P, dk_stride=48), "in place"),
    (dict(dk=9 * P), "outputs overlap"), (dict(dq=8 * P), "outputs overlap"), (dict(dq=2 * P), "outputs overlap"),
    (dict(dq_weight=11 * P + 2), "unaligned"), (dict(dk_weight=11 * P), "outputs overlap"), (dict(k_heads=0), "dk_weight"),
    (dict(workspace=None), "workspace"), (dict(workspace=13 * P + 128), "workspace"),
    (dict(flags=moe.MOE_NO_NORM, q_weight=None, k_weight=None), "gradients of weights"),
])
def test_qk_norm_rope_grad_refuses(change, what):
    _refused("moe_qk_norm_rope_grad", {**HEADS, **GRADS, **change}, what)


def test_qk_norm_rope_grad_refuses_a_small_workspace():
    need = moe.moe_qk_norm_rope_grad_workspace_bytes(5, 4, 2, 16)
    _refused("moe_qk_norm_rope_grad", {**HEADS, **GRADS, "workspace_bytes": need - 1}, "workspace")


def test_workspaces_of_larger_batches_serve_smaller_ones():
    for heads in ((1, 0, 2), (4, 2, 128), (33, 5, 80), (1024, 1024, 512)):
        need = [moe.moe_qk_norm_rope_grad_workspace_bytes(T, *heads) for T in list(range(0, 400)) + [1 << 24]]
        assert need == sorted(need)
    for V, n in ((100, 3), (5000, 0), (65537, 32), (1 << 22, 1)):
        need = [moe.moe_token_logprobs_workspace_bytes(T, V, n) for T in list(range(0, 1500)) + [1 << 24]]
        assert need == sorted(need)


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_tokens=(1 << 24) + 1), "out of range"), (dict(n_vocab=0), "out of range"),
    (dict(n_vocab=(1 << 22) + 1), "out of range"), (dict(top_n=-1), "out of range"), (dict(top_n=33), "out of range"),
    (dict(n_vocab=2, z_stride=2), "out of range"), (dict(z_type=3), "type"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"), (dict(scale=2.0 ** 65), "scale"), (dict(scale=2.0 ** -65), "scale"),
    (dict(logits=None), "logits null"),
    (dict(logits=P + 1), "unaligned"), (dict(z_stride=49999), "stride"), (dict(targets=None), "together"), (dict(logp=None), "together"),
    (dict(top_ids=None), "top_n"), (dict(top_logp=None), "top_n"), (dict(top_n=0), "top_n"), (dict(entropy=4 * P + 2), "unaligned"),
    (dict(lse=5 * P + 1), "unaligned"), (dict(workspace=None), "workspace"), (dict(workspace=8 * P + 64), "workspace"),
    (dict(workspace_bytes=100), "workspace"),
    (dict(targets=None, logp=None, entropy=None, lse=None, top_n=0, top_ids=None, top_logp=None), "nothing"),
])
def test_token_logprobs_refuses(change, what):
    _refused("moe_token_logprobs", {**LOGP, **change}, what)


@pytest.mark.parametrize("change,what", [
    (dict(n_tokens=-1), "out of range"), (dict(n_vocab=0), "out of range"), (dict(z_type=3), "type"), (dict(d_type=4), "type"),
    (dict(scale=0.0), "scale"), (dict(flags=2), "flags"), (dict(logits=None), "logits null"), (dict(z_stride=49999), "stride"),
    (dict(dlogits=None), "dlogits null"), (dict(d_stride=49999), "stride"), (dict(lse=None), "lse"), (dict(dlogp=None, dentropy=None), "neither"),
    (dict(targets=None), "needs targets"), (dict(entropy=None), "entropy"), (dict(dlogp=5 * P + 2), "unaligned"), (dict(dlogits=P), "in place"),
    (dict(dlogits=P, d_type=BF16, flags=moe.MOE_ACCUMULATE), "in place"),
])
def test_token_logprobs_grad_refuses(change, what):
    _refused("moe_token_logprobs_grad", {**LGRAD, **change}, what)


def test_sizes_past_32_bits_are_refused():
    many = (1 << 32) + 2
    with pytest.raises(ValueError, match="x: shape"):
        moe.moe_q4_linear(Rows(many, 64), *planes(8, 64), Rows(many, 8))
    with pytest.raises(ValueError, match="act"):
        moe.moe_q4_linear(Rows(2, 64), *planes(8, 64), Rows(2, 8), act=1 << 33, stream=0)
    with pytest.raises(ValueError, match="q: shape"):
        moe.moe_qk_norm_rope(Rows(many, 4, 16), None, Rows(many, 4, 16), None)
    with pytest.raises(ValueError, match="q: shape"):
        moe.moe_qk_norm_rope(Rows(2, many, 16), None, Rows(2, many, 16), None)
    with pytest.raises(ValueError, match="head_dim"):
        moe.moe_qk_norm_rope(Rows(2, 4, many), None, Rows(2, 4, many), None, stream=0)
    with pytest.raises(ValueError, match="flags"):
        moe.moe_qk_norm_rope(Rows(2, 4, 16), None, Rows(2, 4, 16), None, flags=1 << 32, stream=0)
    with pytest.raises(ValueError, match="flags"):
        moe.moe_qk_norm_rope_grad(*[Rows(2, 4, 16), None] * 3, flags=1 << 32, stream=0)
    with pytest.raises(ValueError, match="logits: shape"):
        moe.moe_token_logprobs(Rows(2, many), entropy=Rows(2))
    with pytest.raises(ValueError, match="flags"):
        moe.moe_token_logprobs_grad(Rows(2, 100), Rows(2, 2), Rows(2, 100), dlogp=Rows(2), targets=Rows(2, dtype=torch.int32),
                                    flags=(1 << 32) + 1, stream=0)
    assert moe.moe_qk_norm_rope_grad_workspace_bytes(many, 1, 1, 16) == -1
    assert moe.moe_token_logprobs_workspace_bytes(2, many) == -1

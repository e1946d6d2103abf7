"""Norm and rotation of query and key heads, and its gradient, on the GPU, against
their definitions in fp64.

Tolerances count roundings: E = 2^-24 of a result per fp32 operation, u(type) half a
step of the output's type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_gpu_dense_ops import TYPES, E, rng_of, smallest, u  # noqa: E402

pytestmark = pytest.mark.gpu

EPS = 1e-6


def turned(x, angle, R, pairs):
    """Heads [T][H][D] in fp64 with their first R values turned by angle [T][R / 2]."""
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    y = x.clone()
    ia = torch.arange(0, R, 2, device=x.device) if pairs else torch.arange(R // 2, device=x.device)
    ib = ia + 1 if pairs else ia + R // 2
    y[..., ia] = x[..., ia] * cos - x[..., ib] * sin
    y[..., ib] = x[..., ib] * cos + x[..., ia] * sin
    return y


def partner(x, R, pairs):
    """|a| + |b| of each value's pair (|a| alone where it has none)."""
    y = x.abs().clone()
    ia = torch.arange(0, R, 2, device=x.device) if pairs else torch.arange(R // 2, device=x.device)
    ib = ia + 1 if pairs else ia + R // 2
    both = y[..., ia] + y[..., ib]
    y[..., ia], y[..., ib] = both, both
    return y


class Rope:
    def __init__(self, T, D, R, axes=1, g=None, far=1 << 20):
        g = g or rng_of(31, T, D, R)
        self.R = R
        if R == 0:
            self.kw, self.angle = {}, torch.zeros((T, 0), dtype=torch.float64, device="cuda")
            return
        inv = torch.from_numpy(10000.0 ** (-np.arange(0, R, 2) / R)).float().cuda()
        pos = torch.from_numpy(g.integers(-far // 8, far, (axes, T))).int().cuda()
        if T > 1:
            pos[0, 0], pos[0, 1] = 0, far - 1
        axis = None
        which = torch.zeros(R // 2, dtype=torch.long)
        if axes > 1:
            which = torch.from_numpy(g.integers(0, axes, R // 2))
            axis = which.to(torch.uint8).cuda()
        self.angle = pos.double().t()[:, which.cuda()] * inv.double()
        self.kw = dict(inv_freq=inv, positions=pos if axes > 1 else pos[0], pair_axis=axis)


def normed(x, w, eps=EPS):
    r = 1 / torch.sqrt(x.square().mean(dim=2, keepdim=True) + eps)
    return x * r * (w if w is not None else 1.0), r


# Roundings of a normed value: the sum of squares (16 in a lane, 6 over lanes, half of them under the root), mean, eps, root,
# reciprocal, three products; of a turned one: cos and sin are within 5 E (the angle's last turn to 2^-26, its product with
# 2 pi, the series), a product and an FMA each
NORM = (22 / 2 + 2 + 2 + 3) * E
TURN = 8 * E


def head_tensor(g, T, H, D, dtype, layout, scale=1.0):
    """Heads of a layout: their own tensor; a part of a wider row, shifted; tokens of a head after each other."""
    a = torch.from_numpy(scale * g.standard_normal((T, H, D))).cuda()
    if layout == "row":
        wide = torch.full((T, (H + 2) * D + 3), 9.0, dtype=dtype, device="cuda")
        v = wide[:, 1:1 + H * D].view(T, H, D) if T == 1 else wide[:, 1:1 + H * D].unflatten(1, (H, D))
        v.copy_(a.to(dtype))
        return v, wide
    if layout == "heads":
        flat = torch.full((H, T + 1, D), 9.0, dtype=dtype, device="cuda")
        v = flat[:, :T].transpose(0, 1)
        v.copy_(a.to(dtype))
        return v, flat
    v = a.to(dtype).contiguous()
    return v, v


def rest(v, whole):
    """What of `whole` does not belong to the heads."""
    w = whole.clone()
    torch.as_strided(w, v.shape, v.stride(), v.storage_offset()).zero_()
    return w


SHAPES = [(1, 1, 0, 2, 2), (1, 16, 2, 128, 128), (3, 4, 4, 64, 64), (7, 5, 1, 80, 60), (5, 6, 2, 72, 54), (33, 8, 8, 96, 72),
          (2, 3, 1, 256, 64), (4, 2, 2, 512, 512), (9, 7, 3, 40, 40), (6, 1, 1, 64, 64), (300, 1, 0, 64, 32), (70, 2, 1, 512, 256),
          (11, 3, 2, 10, 6), (5, 2, 1, 194, 130), (257, 14, 2, 128, 128), (4, 3, 1, 100, 0), (40, 33, 5, 32, 24),
          (3, 2, 1, 510, 508)]


@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
@pytest.mark.parametrize("xt,ot", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("pairs,layout", [(False, "own"), (True, "row"), (False, "heads")])
def test_qk_norm_rope(T, Hq, Hk, D, R, xt, ot, pairs, layout):
    g = rng_of(32, T, Hq, D, R)
    rope = Rope(T, D, R, axes=1 + (T + D) % 3, g=g)
    flags = moe.MOE_ROPE_PAIRS if pairs else 0
    q, qf = head_tensor(g, T, Hq, D, TYPES[xt], layout)
    k, kf = head_tensor(g, T, Hk, D, TYPES[xt], layout, 3.0) if Hk else (None, None)
    qo, qof = head_tensor(g, T, Hq, D, TYPES[ot], layout)
    ko, kof = head_tensor(g, T, Hk, D, TYPES[ot], layout) if Hk else (None, None)
    qw = torch.from_numpy(1 + 0.2 * g.standard_normal(D)).float().cuda()
    kw = torch.from_numpy(1 + 0.2 * g.standard_normal(D)).float().cuda() if Hk and T % 2 else None
    before = [(t, f, rest(t, f), t.clone()) for t, f in ((q, qf), (k, kf), (qo, qof), (ko, kof)) if t is not None]
    moe.moe_qk_norm_rope(q, k, qo, ko, q_weight=qw, k_weight=kw, eps=EPS, flags=flags, **rope.kw)
    for t, f, r, v in before:
        assert torch.equal(rest(t, f), r)
        assert t is qo or t is ko or torch.equal(t, v)
    dt = TYPES[ot]
    outs = []
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        if x is None:
            continue
        v, _ = normed(x.double(), w.double() if w is not None else None)
        ref = turned(v, rope.angle, R, pairs)
        tol = (partner(v, R, pairs) * (NORM + TURN) + u(dt) * ref.abs()) * 1.01 + smallest(dt)
        off = (o.double() - ref).abs()
        assert (off <= tol).all(), float((off / tol).max())
        outs.append(o.clone())
    # in place
    if xt == ot:
        moe.moe_qk_norm_rope(q, k, q, k, q_weight=qw, k_weight=kw, eps=EPS, flags=flags, **rope.kw)
        assert torch.equal(q, outs[0]) and (k is None or torch.equal(k, outs[1]))


@pytest.mark.parametrize("T,H,D,R", [(5, 3, 64, 64), (2, 2, 80, 60), (9, 1, 54, 54)])
def test_rotation_alone_keeps_lengths_and_turns_back(T, H, D, R):
    g = rng_of(33, T, D)
    rope = Rope(T, D, R, g=g)
    for pairs in (0, moe.MOE_ROPE_PAIRS):
        x, _ = head_tensor(g, T, H, D, torch.float32, "own")
        y, back = torch.empty_like(x), torch.empty_like(x)
        moe.moe_qk_norm_rope(x, None, y, None, flags=moe.MOE_NO_NORM | pairs, **rope.kw)
        ref = turned(x.double(), rope.angle, R, bool(pairs))
        assert ((y.double() - ref).abs() <= partner(x.double(), R, bool(pairs)) * TURN * 1.01).all()
        # the gradient turns back; so do the negative positions
        moe.moe_qk_norm_rope_grad(x, None, y, None, back, None, flags=moe.MOE_NO_NORM | pairs, **rope.kw)
        assert ((back - x).abs() <= partner(x, R, bool(pairs)) * 3 * TURN).all()
        kw = dict(rope.kw, positions=-rope.kw["positions"])
        moe.moe_qk_norm_rope(y, None, back, None, flags=moe.MOE_NO_NORM | pairs, **kw)
        assert ((back - x).abs() <= partner(x, R, bool(pairs)) * 3 * TURN).all()


def test_far_positions():
    """Positions up to int32's limits: the angle in 64 bits is off by 2^31 * 2^-53 turns and less."""
    T, D = 9, 32
    x = torch.ones((T, 1, D), device="cuda")
    pos = torch.tensor([0, 1, -1, 1 << 20, 1 << 24, (1 << 24) + 1, 1 << 30, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda")
    inv = torch.from_numpy(1e6 ** (-np.arange(0, D, 2) / D)).float().cuda()
    y = torch.empty_like(x)
    moe.moe_qk_norm_rope(x, None, y, None, flags=moe.MOE_NO_NORM, inv_freq=inv, positions=pos)
    # the reference's own angle of 2^31 radians is rounded to 2^-23
    ref = turned(x.double(), pos.double()[:, None] * inv.double(), D, False)
    assert ((y.double() - ref).abs() <= 2 * (TURN + 2.0 ** -22 * (pos.double().abs() > 2 ** 25)[:, None, None])).all()


def test_one_row_of_positions_for_all_axes():
    """Positions of text in a model with several axes: one row, expanded (stride 0), or rows of a wider table."""
    T, D = 7, 24
    g = rng_of(50)
    x, _ = head_tensor(g, T, 2, D, torch.float32, "own")
    pos = torch.from_numpy(g.integers(0, 1000, T)).int().cuda()
    inv = torch.from_numpy(100.0 ** (-np.arange(0, D, 2) / D)).float().cuda()
    axis = torch.from_numpy(g.integers(0, 3, D // 2)).to(torch.uint8).cuda()
    want, y = torch.empty_like(x), torch.empty_like(x)
    moe.moe_qk_norm_rope(x, None, want, None, inv_freq=inv, positions=pos)
    wide = torch.full((3, 50), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, 5:5 + T] = pos
    for p in (pos.expand(3, T), wide[:, 5:5 + T], pos[None]):
        moe.moe_qk_norm_rope(x, None, y, None, inv_freq=inv, positions=p, pair_axis=axis if len(p) > 1 else None)
        assert torch.equal(y, want)


def test_axes_that_do_not_exist_are_not_turned():
    T, D = 4, 16
    g = rng_of(34)
    x, _ = head_tensor(g, T, 2, D, torch.float32, "own")
    pos = torch.from_numpy(g.integers(0, 100, (2, T))).int().cuda()
    inv = torch.ones(8, device="cuda")
    axis = torch.tensor([0, 1, 2, 255, 0, 1, 7, 0], dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    moe.moe_qk_norm_rope(x, None, y, None, flags=moe.MOE_NO_NORM, inv_freq=inv, positions=pos, pair_axis=axis)
    for i, a in enumerate(axis.tolist()):
        angle = pos[a].double() if a < 2 else torch.zeros(T, dtype=torch.float64, device="cuda")
        want = x[..., i].double() * angle.cos()[:, None] - x[..., i + 8].double() * angle.sin()[:, None]
        assert ((y[..., i].double() - want).abs() <= (x[..., i].abs() + x[..., i + 8].abs()) * TURN).all()
        if a >= 2:
            assert torch.equal(y[..., i], x[..., i]) and torch.equal(y[..., i + 8], x[..., i + 8])


@pytest.mark.parametrize("D", [2, 64, 80, 192, 512])
@pytest.mark.parametrize("size", [1e30, 1e-30, 1e-38])
def test_heads_far_from_unit_scale(D, size):
    g = rng_of(35, D)
    T, H = 3, 2
    x = torch.from_numpy(size * g.standard_normal((T, H, D))).float().cuda()
    x[1] = torch.from_numpy(g.standard_normal((H, D))).float().cuda()  # beside ordinary ones
    y = torch.empty_like(x)
    for eps in (0.0, 1e-6):
        moe.moe_qk_norm_rope(x, None, y, None, eps=eps)
        v, r = normed(x.double(), None, eps)
        assert ((y.double() - v).abs() <= NORM * 1.01 * v.abs() + smallest(torch.float32)).all()
        gr = torch.from_numpy(g.standard_normal((T, H, D))).float().cuda()
        dx = torch.empty_like(x)
        moe.moe_qk_norm_rope_grad(x, None, gr, None, dx, None, eps=eps)
        xh = v
        mag = r * (gr.double().abs() + xh.abs() * (gr.double() * xh).abs().mean(dim=2, keepdim=True))
        want = r * (gr.double() - xh * (gr.double() * xh).mean(dim=2, keepdim=True))
        fine = want.abs() < 1e38  # 1 / rms may leave fp32's range: inf there, as the formula has it
        tol = mag * 4 * (NORM + TURN) + smallest(torch.float32)
        assert ((dx.double() - want).abs() <= tol)[fine].all()


def test_heads_of_zeros_and_values_that_are_not_finite():
    x = torch.ones((4, 2, 64), device="cuda")
    x[0, 0] = 0
    x[1, 1, 5] = float("inf")
    x[2, 0, 7] = float("nan")
    y = torch.empty_like(x)
    moe.moe_qk_norm_rope(x, None, y, None, eps=1e-6)
    assert (y[0, 0] == 0).all() and torch.isnan(y[1, 1, 5]) and (y[1, 1, 6:] == 0).all() and torch.isnan(y[2, 0]).all()
    good = torch.ones((4, 2), dtype=torch.bool)
    good[0, 0] = good[1, 1] = good[2, 0] = False
    assert torch.isfinite(y[good]).all() and (y[good] == y[3, 0]).all()
    moe.moe_qk_norm_rope(x, None, y, None, eps=0.0)
    assert torch.isnan(y[0, 0]).all()


# ---------------------------------------------------------------------------
# gradient


def grad_ref(x, w, gr, angle, R, pairs, eps=EPS):
    """dx, dweight in fp64 and the magnitudes their roundings are relative to."""
    gb = turned(gr, -angle, R, pairs)
    mg = partner(gr, R, pairs)
    r = 1 / torch.sqrt(x.square().mean(dim=2, keepdim=True) + eps)
    xh = x * r
    wt = w if w is not None else torch.ones(x.shape[2], dtype=torch.float64, device=x.device)
    uu = gb * wt
    dx = r * (uu - xh * (uu * xh).mean(dim=2, keepdim=True))
    m = mg * wt.abs()
    mag = r * (m + xh.abs() * (m * xh.abs()).mean(dim=2, keepdim=True))
    return dx, (gb * xh).sum(dim=(0, 1)), mag, (mg * xh.abs()).sum(dim=(0, 1))


@pytest.mark.parametrize("T,Hq,Hk,D,R", SHAPES)
@pytest.mark.parametrize("xt,gt,dt", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f16", "f32", "f16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("pairs,layout", [(False, "own"), (True, "row"), (True, "heads")])
def test_qk_norm_rope_grad(T, Hq, Hk, D, R, xt, gt, dt, pairs, layout):
    g = rng_of(36, T, Hq, D, R)
    rope = Rope(T, D, R, axes=1 + (T + D) % 3, g=g)
    flags = moe.MOE_ROPE_PAIRS if pairs else 0
    one = lambda H, t, s=1.0: head_tensor(g, T, H, D, TYPES[t], layout, s) if H else (None, None)  # noqa: E731
    (q, qf), (k, kf), (gq, gqf), (gk, gkf) = one(Hq, xt), one(Hk, xt, 3.0), one(Hq, gt), one(Hk, gt)
    (dq, dqf), (dk, dkf) = one(Hq, dt), one(Hk, dt)
    qw = torch.from_numpy(1 + 0.2 * g.standard_normal(D)).float().cuda()
    kw = torch.from_numpy(1 + 0.2 * g.standard_normal(D)).float().cuda() if Hk and T % 2 else None
    dqw = torch.full((D,), 5.0, device="cuda")
    dkw = torch.full((D,), 5.0, device="cuda") if Hk else None
    before = [(t, f, rest(t, f), t.clone()) for t, f in ((q, qf), (k, kf), (gq, gqf), (gk, gkf), (dq, dqf), (dk, dkf))
              if t is not None]
    ws = moe.moe_qk_norm_rope_workspace(q, k)
    ws.fill_(255)
    args = dict(q_weight=qw, k_weight=kw, eps=EPS, flags=flags, **rope.kw)
    moe.moe_qk_norm_rope_grad(q, k, gq, gk, dq, dk, dq_weight=dqw, dk_weight=dkw, workspace=ws, **args)
    for t, f, r, v in before:
        assert torch.equal(rest(t, f), r)
        assert t is dq or t is dk or torch.equal(t, v)
    first = []
    for x, w, gr, d, dw in ((q, qw, gq, dq, dqw), (k, kw, gk, dk, dkw)):
        if x is None:
            continue
        H = x.shape[1]
        dx, dwr, mag, wmag = grad_ref(x.double(), w.double() if w is not None else None, gr.double(), rope.angle, R, pairs)
        # u, xh, their mean (22 additions and two roundings) and the last three products
        tol = (mag * (2 * NORM + TURN + 30 * E) + u(TYPES[dt]) * dx.abs()) * 1.01 + smallest(TYPES[dt])
        off = (d.double() - dx).abs()
        assert (off <= tol).all(), float((off / tol).max())
        # a lane's rows, the row groups of a work-group (256 at most), the shares (32 and 32)
        tol = wmag * (NORM + TURN + (T * H + 256 + 64) * E)
        assert ((dw.double() - dwr).abs() <= tol).all()
        # the additions' errors as independent ones of 0.58 E each beside partial sums of the size of the result
        assert torch.linalg.norm(dw.double() - dwr) <= 1e-6 * torch.linalg.norm(wmag)
        first += [d.clone(), dw.clone()]
    # again, without the weights' gradients; then in place of the gradients, the weights' added up
    moe.moe_qk_norm_rope_grad(q, k, gq, gk, dq, dk, **args)
    assert torch.equal(dq, first[0]) and (k is None or torch.equal(dk, first[2]))
    if gt == dt:
        args["flags"] |= moe.MOE_ACCUMULATE
        moe.moe_qk_norm_rope_grad(q, k, gq, gk, gq, gk, dq_weight=dqw, dk_weight=dkw, workspace=ws, **args)
        assert torch.equal(gq, first[0]) and (k is None or torch.equal(gk, first[2]))
        assert torch.equal(dqw, first[1] + first[1]) and (k is None or torch.equal(dkw, first[3] + first[3]))


def test_gradient_in_place_of_the_heads():
    g = rng_of(37)
    rope = Rope(5, 64, 64, g=g)
    q, _ = head_tensor(g, 5, 3, 64, torch.bfloat16, "own")
    gq, _ = head_tensor(g, 5, 3, 64, torch.float32, "own")
    dq = torch.empty_like(q)
    moe.moe_qk_norm_rope_grad(q, None, gq, None, dq, None, **rope.kw)
    moe.moe_qk_norm_rope_grad(q, None, gq, None, q, None, **rope.kw)
    assert torch.equal(q, dq)


def test_gradient_over_many_rows():
    """More rows than the work-groups take in one turn: every row counts once."""
    T, H, D = 9001, 9, 64
    q = torch.ones((T, H, D), dtype=torch.bfloat16, device="cuda")
    gq = torch.ones((T, H, D), dtype=torch.bfloat16, device="cuda")
    dq, dw = torch.empty_like(q), torch.empty(D, device="cuda")
    moe.moe_qk_norm_rope_grad(q, None, gq, None, dq, None, dq_weight=dw, eps=0.0)
    assert (dw == T * H).all()  # whole numbers below 2^24: exact in any order
    assert (dq.float().abs() <= 40 * E).all()


@pytest.mark.parametrize("D,R,pairs", [(16, 16, False), (20, 12, True), (72, 54, False)])
def test_gradient_against_differences(D, R, pairs):
    """Central differences of the forward call in fp32, step 2^-7: their own error is h^2 / 6 of a third derivative of size
    10 and a few roundings of the loss over the step."""
    g = rng_of(38, D)
    T, H = 3, 2
    rope = Rope(T, D, R, g=g, far=1 << 10)
    flags = moe.MOE_ROPE_PAIRS if pairs else 0
    x = torch.from_numpy(g.standard_normal((T, H, D))).float().cuda()
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(D)).float().cuda()
    c = torch.from_numpy(g.standard_normal((T, H, D))).float().cuda()
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(D, device="cuda")

    def loss(x, w):
        moe.moe_qk_norm_rope(x, None, y, None, q_weight=w, flags=flags, **rope.kw)
        return (y.double() * c.double()).sum()

    moe.moe_qk_norm_rope_grad(x, None, c, None, dx, None, q_weight=w, dq_weight=dw, flags=flags, **rope.kw)
    h = 2.0 ** -7
    for _ in range(6):
        d = torch.from_numpy(g.standard_normal((T, H, D))).float().cuda()
        d /= torch.linalg.norm(d)
        diff = (loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h)
        scale = torch.linalg.norm(c).double()
        assert abs(diff - (dx.double() * d.double()).sum()) <= (10 * h * h / 6 * 10 + 40 * E / h) * scale
        e = torch.from_numpy(g.standard_normal(D)).float().cuda()
        e /= torch.linalg.norm(e)
        diff = (loss(x, w + h * e) - loss(x, w - h * e)) / (2 * h)
        assert abs(diff - (dw.double() * e.double()).sum()) <= 40 * E / h * scale * 4


def test_of_no_tokens():
    q = torch.zeros((0, 4, 64), device="cuda")
    inv, pos = torch.ones(32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    moe.moe_qk_norm_rope(q, q.clone(), q.clone(), q.clone(), inv_freq=inv, positions=pos)
    dw = torch.full((64,), 3.0, device="cuda")
    moe.moe_qk_norm_rope_grad(q, None, q.clone(), None, q.clone(), None, dq_weight=dw, flags=moe.MOE_ACCUMULATE)
    assert (dw == 3).all()
    moe.moe_qk_norm_rope_grad(q, None, q.clone(), None, q.clone(), None, dq_weight=dw)
    assert (dw == 0).all()


def test_on_another_stream_captured_and_beside_eager_autograd():
    """Forward and gradient captured into a graph while autograd's own graph of the same tensors lives; replays with eager
    work in between."""
    T, Hq, Hk, D = 50, 6, 2, 128
    g = rng_of(39)
    rope = Rope(T, D, D, axes=2, g=g)
    q, _ = head_tensor(g, T, Hq, D, torch.float32, "own")
    k, _ = head_tensor(g, T, Hk, D, torch.float32, "own")
    gq, _ = head_tensor(g, T, Hq, D, torch.float32, "own")
    gk, _ = head_tensor(g, T, Hk, D, torch.float32, "own")
    w = torch.ones(D, device="cuda")
    leaf = q.requires_grad_()
    alive = (leaf * 2).sum()  # an eager graph of the same leaf
    q = leaf.detach()
    outs = [torch.empty_like(t) for t in (q, k, q, k)] + [torch.empty(D, device="cuda") for _ in range(2)]
    ws = moe.moe_qk_norm_rope_workspace(q, k)

    def step(stream=None):
        moe.moe_qk_norm_rope(q, k, outs[0], outs[1], q_weight=w, k_weight=w, stream=stream, **rope.kw)
        moe.moe_qk_norm_rope_grad(q, k, gq, gk, outs[2], outs[3], q_weight=w, k_weight=w, dq_weight=outs[4], dk_weight=outs[5],
                                  workspace=ws, stream=stream, **rope.kw)

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for i in range(4):
        q.copy_(torch.from_numpy(rng_of(40, i).standard_normal((T, Hq, D))).float())
        step()
        want = [o.clone() for o in outs]
        torch.cuda.synchronize()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for o in outs:
            o.zero_()
        side.wait_stream(torch.cuda.current_stream())
        step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    alive.backward()
    assert (leaf.grad == 2).all()


def test_binding_refusals():
    q, k = torch.ones((4, 3, 64), device="cuda"), torch.ones((4, 1, 64), device="cuda")
    inv, pos = torch.ones(32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    ok = dict(inv_freq=inv, positions=pos)
    o, ko = torch.empty_like(q), torch.empty_like(k)
    moe.moe_qk_norm_rope(q, k, o, ko, **ok)
    for a in ((q, k, o, None), (q, k, torch.empty((4, 3, 32), device="cuda"), ko), (q, k.half(), o, ko), (q.cpu(), k, o, ko),
              (q.transpose(1, 2), k, o, ko), (torch.ones((4, 64, 3), device="cuda").transpose(1, 2), k, o, ko)):
        with pytest.raises(ValueError):
            moe.moe_qk_norm_rope(*a, **ok)
    for bad in (dict(inv_freq=inv), dict(positions=pos), dict(inv_freq=inv, positions=pos.long()), dict(inv_freq=inv, positions=pos[:3]),
                dict(inv_freq=torch.ones(33, device="cuda"), positions=pos), dict(inv_freq=inv.half(), positions=pos),
                dict(inv_freq=inv, positions=torch.zeros((9, 4), dtype=torch.int32, device="cuda")),
                dict(ok, pair_axis=torch.zeros(31, dtype=torch.uint8, device="cuda")), dict(ok, q_weight=torch.ones(63, device="cuda"))):
        with pytest.raises(ValueError):
            moe.moe_qk_norm_rope(q, k, o, ko, **bad)
    for a, kw in (((q, k, o, ko), dict(ok, flags=8)), ((q, k, o, ko), dict(ok, flags=moe.MOE_ACCUMULATE)),
                  ((q, k, o, ko), dict(ok, eps=-1.0)), ((q, k, o, ko), dict(flags=moe.MOE_NO_NORM)),
                  ((q, k, o, ko), dict(ok, flags=moe.MOE_NO_NORM, q_weight=torch.ones(64, device="cuda"))),
                  ((q, k, q[:, :, :], q[:, :1]), ok), ((q, None, q.expand(4, 3, 64).as_strided((4, 3, 64), (192, 32, 1)), None), ok)):
        with pytest.raises(moe.MoeError):
            moe.moe_qk_norm_rope(*a, **kw)
    gq, gk, dq, dk = q.clone(), k.clone(), o, ko
    dw = torch.empty(64, device="cuda")
    ws = moe.moe_qk_norm_rope_workspace(q, k)
    moe.moe_qk_norm_rope_grad(q, k, gq, gk, dq, dk, dq_weight=dw, workspace=ws, **ok)
    with pytest.raises(ValueError):
        moe.moe_qk_norm_rope_grad(q, None, gq, None, dq, None, dk_weight=dw, **ok)
    with pytest.raises(ValueError, match="stream of its own"):
        moe.moe_qk_norm_rope_grad(q, k, gq, gk, dq, dk, dq_weight=dw, stream=torch.cuda.Stream(), **ok)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_qk_norm_rope_grad(q, k, gq, gk, dq, dk, dq_weight=dw, workspace=ws[:256], **ok)
    with pytest.raises(moe.MoeError, match="overlap"):
        moe.moe_qk_norm_rope_grad(q, k, gq, gk, dq, dk, dq_weight=dw, dk_weight=dw, workspace=ws, **ok)


def test_gradient_of_work_groups_that_take_several_turns():
    """One head of 512 per token: a work-group's angles are those of 16 tokens, and there are more sixteens than work-groups."""
    T, D = 40003, 512
    g = torch.Generator(device="cuda")
    g.manual_seed(51)
    x = torch.randn((T, 1, D), generator=g, device="cuda").bfloat16()
    gr = torch.randn((T, 1, D), generator=g, device="cuda").bfloat16()
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    rope = Rope(T, D, D, g=rng_of(51))
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(D, device="cuda")
    moe.moe_qk_norm_rope(x, None, y, None, q_weight=w, eps=EPS, **rope.kw)
    moe.moe_qk_norm_rope_grad(x, None, gr, None, dx, None, q_weight=w, dq_weight=dw, eps=EPS, **rope.kw)
    v, _ = normed(x.double(), w.double())
    ref = turned(v, rope.angle, D, False)
    assert ((y.double() - ref).abs() <= (partner(v, D, False) * (NORM + TURN) + u(torch.bfloat16) * ref.abs()) * 1.01 + 1e-40).all()
    want, wantw, mag, wmag = grad_ref(x.double(), w.double(), gr.double(), rope.angle, D, False)
    assert ((dx.double() - want).abs() <= (mag * (2 * NORM + TURN + 30 * E) + u(torch.bfloat16) * want.abs()) * 1.01 + 1e-40).all()
    assert ((dw.double() - wantw).abs() <= wmag * (NORM + TURN + (T / 1024 + 256 + 64) * E)).all()

"""The 4-bit product with bias, activation, factor and residual on the GPU,
against its definition in fp64.

Tolerances count roundings: E = 2^-24 of a result per fp32 operation, u(type) half a
step of the output's type; the product's own bound is test_gpu_dense_ops.Product's.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_gpu_dense_ops import TYPES, E, Product, rng_of, rows, smallest, u, untouched  # noqa: E402

pytestmark = pytest.mark.gpu

ACT = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
       "gelu_tanh": moe.MOE_ACT_GELU_TANH}


def act64(act, v):
    v = torch.as_tensor(v, dtype=torch.float64)
    if act == "relu":
        return torch.relu(v)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v * math.sqrt(0.5))  # ndtr loses the lower tail in torch
    if act == "gelu_tanh":
        return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))  # (1 + tanh a) / 2, which cancels
    return v


class Linear:
    """Operands of a call, its fp64 result and the bound of its error."""

    def __init__(self, T, N, K, xt, yt, act, bias, mt, rt, seed=0):
        g = rng_of(21, T, N, K, seed)
        self.p = Product(T, N, K, xt, seed)
        # a product of unit size, so that the activations' bends are met
        size = 2.0 ** -round(math.log2(max(np.std(self.p.ref), 1 / 16)))
        self.p.scl.mul_(size)
        bound = torch.from_numpy(self.p.bound * size)
        q = torch.cat([self.p.nib & 15, self.p.nib >> 4], dim=2).cpu().double() - 8
        x = self.p.x.cpu().double()
        if self.p.scales is not None:
            x = (x.view(T, K // 32, 32) * self.p.scales.cpu().double()[..., None]).view(T, K)
        self.pre = x @ (q * self.p.scl.cpu().double()[..., None]).reshape(N, K).t()
        self.bias = torch.from_numpy(0.5 * g.standard_normal(N)).float().cuda() if bias else None
        pad, lead = (0, 0) if (T + N) % 2 else (5, 3)
        self.mul = rows(g.standard_normal((T, N)), TYPES[mt], pad, lead)[0] if mt else None
        self.res = rows(2 * g.standard_normal((T, N)), TYPES[rt], pad, lead)[0] if rt else None
        self.pad, self.lead, self.dt = pad, lead, TYPES[yt]
        v = self.pre + (self.bias.cpu().double() if bias else 0)
        err = bound * 1.01 + E * v.abs()
        a = act64(act, v)
        # |act'| is at most 1.13; exponentials and erfc to 8 roundings, their arguments' roundings count v^2 times
        err = 1.13 * err + (8 + 4 * v * v) * E * a.abs() if act != "none" else err
        if mt:
            m = self.mul.cpu().double()
            a, err = a * m, err * m.abs() + E * (a * m).abs()
        if rt:
            a = a + self.res.cpu().double()
        self.ref, self.tol = a, (err + (E + u(self.dt)) * a.abs()) * 1.01 + smallest(self.dt)

    def call(self, y, act, ws):
        moe.moe_q4_linear(self.p.x, self.p.nib, self.p.scl, y, bias=self.bias, act=ACT[act], mul=self.mul, residual=self.res,
                          scales=self.p.scales, workspace=ws)

    def check(self, y):
        off = (y.cpu().double() - self.ref).abs()
        assert torch.isfinite(y).all()
        assert (off <= self.tol).all(), float((off / self.tol).max())


# dot products for a few tokens, of one wave and of four; tiles in one launch; split and whole wide tiles; two
# passes of tokens
SHAPES = [(1, 1, 32), (1, 2048, 2048), (3, 33, 96), (5, 100, 4096), (1, 37, 8224), (2, 2049, 6368), (16, 64, 256), (17, 65, 288),
          (64, 256, 512), (200, 512, 96), (257, 70, 1312), (130, 2050, 8224), (2100, 3900, 256), (4100, 4100, 160),
          (16500, 1100, 128)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("xt,yt,act,bias,mt,rt", [
    ("f32", "f32", "silu", False, "f32", None), ("bf16", "bf16", "gelu", True, None, "bf16"),
    ("f16", "f32", "gelu_tanh", True, "f16", "f32"), ("q8", "f16", "none", True, None, None),
    ("q8", "f32", "relu", False, "bf16", "f16"), ("f32", "bf16", "none", False, None, "f32")])
def test_q4_linear(T, N, K, xt, yt, act, bias, mt, rt):
    c = Linear(T, N, K, xt, yt, act, bias, mt, rt)
    y, yf = rows(np.full((T, N), 3.0), c.dt, c.pad, c.lead)
    ws = moe.moe_q4_workspace(c.p.x, c.p.nib)
    if ws is not None:
        ws.fill_(255)
    c.call(y, act, ws)
    c.check(y)
    assert untouched(yf, T, N, c.pad, c.lead)
    first = y.clone()
    c.call(y, act, None)
    assert torch.equal(first, y)  # equal calls, equal bits
    for name in ("mul", "res"):  # in place of either
        t = getattr(c, name)
        if t is not None and t.dtype == c.dt:
            keep = t.clone()
            c.call(t, act, ws)
            assert torch.equal(t, first)
            t.copy_(keep)


@pytest.mark.parametrize("T,N,K,xt", [(1, 300, 256, "f32"), (8, 90, 6400, "bf16"), (40, 50, 128, "q8"), (130, 2050, 8224, "f16"),
                                      (4100, 4100, 160, "bf16")])
def test_without_an_epilogue_it_is_the_product(T, N, K, xt):
    p = Product(T, N, K, xt)
    a, b = torch.empty((T, N), device="cuda"), torch.empty((T, N), device="cuda")
    moe.moe_q4_matmul(p.x, p.nib, p.scl, a, scales=p.scales)
    moe.moe_q4_linear(p.x, p.nib, p.scl, b, scales=p.scales)
    assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("T", [1, 40, 4100])
def test_activations_over_their_range(act, T):
    """bias alone (weights of scale 0) through every activation: far arguments, zeros, values that are not finite."""
    N = 4100 if T > 100 else 500
    nib = torch.zeros((N, 5, 16), dtype=torch.uint8, device="cuda")
    scl = torch.zeros((N, 5), dtype=torch.float16, device="cuda")
    g = torch.Generator().manual_seed(3)
    bias = torch.randn(N, generator=g) * 10 ** (4 * torch.rand(N, generator=g) - 2)
    bias[:8] = torch.tensor([0.0, -0.0, 1e30, -1e30, float("inf"), 3e38, -200.0, float("nan")])
    y = torch.empty((T, N), device="cuda")
    moe.moe_q4_linear(torch.ones((T, 160), device="cuda"), nib, scl, y, bias=bias.cuda(), act=ACT[act])
    ref = act64(act, bias.double())
    assert (y.cpu() == y[0].cpu()).logical_or(torch.isnan(y.cpu())).all()
    got = y[0].cpu().double()
    assert torch.isnan(got[7])
    assert got[4] == float("inf") and got[0] == 0 and got[1] == 0
    some = torch.ones(N, dtype=torch.bool)
    some[[4, 7]] = False
    v, r, o = bias.double()[some], ref[some], got[some]
    count = 8 + 4 * v * v
    if act == "gelu_tanh":
        # the exponential's argument a = 1.596 (v + 0.0447 v^3) has six roundings: v^2, 0.0447 and its product, the sum, 1.596
        # and its product. Each counts |a| times in the result, |a| = 87 at v = -10, the last that is not 0
        count = 8 + 6 * (1.596 * (v + 0.0447 * v ** 3)).abs()
    # 1 + e^-a passes fp32's range at 2^128: results below |v| 2^-128, or below fp32's normal range, may be 0
    least = v.abs() * 2.0 ** -127 + 2.0 ** -125
    assert ((o - r).abs() <= count.clamp(max=2.0 ** 23) * 1.01 * E * r.abs() + least).all()


@pytest.mark.parametrize("T", [1, 24, 300])
def test_swiglu_of_a_shared_expert_captured(T):
    """up, gate and down of a shared expert onto the stream, as three calls of a graph; replays against the eager result."""
    H, F = 512, 352
    g = rng_of(23, T)
    x = torch.from_numpy(g.standard_normal((T, H))).float().cuda()
    stream0 = torch.from_numpy(g.standard_normal((T, H))).float().cuda()
    w = []
    for n, k in ((F, H), (F, H), (H, F)):
        p = Product(1, n, k, "f32", seed=len(w))
        w.append((p.nib, p.scl))
    up, h, stream = torch.empty((T, F), device="cuda"), torch.empty((T, F), device="cuda"), torch.empty((T, H), device="cuda")
    ws = [moe.moe_q4_workspace(x, w[0][0]), moe.moe_q4_workspace(h, w[2][0])]

    def step():
        stream.copy_(stream0)
        moe.moe_q4_matmul(x, *w[0], up, workspace=ws[0])
        moe.moe_q4_linear(x, *w[1], h, act=moe.MOE_ACT_SILU, mul=up, workspace=ws[0])
        moe.moe_q4_linear(h, *w[2], stream, residual=stream, workspace=ws[1])

    step()
    want = stream.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    dense = [(torch.cat([n & 15, n >> 4], dim=2).double() - 8).mul(c.double()[..., None]).flatten(1) for n, c in w]
    for i in range(4):
        x.copy_(torch.from_numpy(rng_of(24, T, i).standard_normal((T, H))).float())
        step()
        want = stream.clone()
        torch.cuda.synchronize()
        stream.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(stream, want)
        v = x.double() @ dense[1].t()
        ref = stream0.double() + (v * torch.sigmoid(v) * (x.double() @ dense[0].t())) @ dense[2].t()
        assert torch.linalg.norm(stream.double() - ref) <= 2e-6 * torch.linalg.norm(ref)


def test_of_no_tokens():
    nib, scl = torch.zeros((8, 2, 16), dtype=torch.uint8, device="cuda"), torch.zeros((8, 2), dtype=torch.float16, device="cuda")
    moe.moe_q4_linear(torch.zeros((0, 64), device="cuda"), nib, scl, torch.zeros((0, 8), device="cuda"), act=ACT["gelu"])


def test_binding_refusals():
    p = Product(4, 40, 64, "f32")
    y = torch.empty((4, 40), device="cuda")
    good = dict(bias=torch.zeros(40, device="cuda"), mul=torch.ones((4, 40), device="cuda"))
    moe.moe_q4_linear(p.x, p.nib, p.scl, y, **good)
    for bad in (dict(bias=torch.zeros(39, device="cuda")), dict(bias=torch.zeros(40, device="cuda").half()),
                dict(mul=torch.ones((4, 39), device="cuda")), dict(residual=torch.ones((4, 40))),
                dict(residual=torch.ones((40, 4), device="cuda").t())):
        with pytest.raises(ValueError):
            moe.moe_q4_linear(p.x, p.nib, p.scl, y, **bad)
    for bad in (dict(act=5), dict(act=-1), dict(mul=torch.ones((4, 40), dtype=torch.int8, device="cuda"))):
        with pytest.raises(moe.MoeError):
            moe.moe_q4_linear(p.x, p.nib, p.scl, y, **bad)
    wide = torch.ones((4, 48), device="cuda")
    with pytest.raises(moe.MoeError, match="in place"):
        moe.moe_q4_linear(p.x, p.nib, p.scl, wide[:, :40].as_strided((4, 40), (40, 1)), residual=wide[:, :40])

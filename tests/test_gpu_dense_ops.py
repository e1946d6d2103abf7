"""The operators beside the experts on the GPU, each against its definition in
fp64, and a decode step made of them.

Tolerances count roundings. u(type) is half a step of the output type; every
fp32 operation is off by at most E = 2^-24 of its result.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
import oracle  # noqa: E402
from tests._gpu import TOL, Decode, token_rel_err  # noqa: E402
from workload import Workload, activations, q4_matrix, zipf_logits  # noqa: E402

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": moe.MOE_F32, "f16": moe.MOE_F16, "bf16": moe.MOE_BF16, "q8": moe.MOE_Q8_32}
GUARD = 77.0  # what lies between the rows


def u(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):  # a subnormal result is off by half the smallest subnormal step
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def rows(a, dtype, pad=0, lead=0):
    """a [T][n] on the GPU as rows of a wider array filled with GUARD; lead shifts the first value."""
    T, n = a.shape
    flat = torch.full((lead + T * (n + pad) + 8,), GUARD, dtype=dtype, device="cuda")
    v = torch.as_strided(flat, (T, n), (n + pad, 1), lead)
    v.copy_(torch.as_tensor(a).to(dtype).cuda())
    return v, flat


def untouched(flat, T, n, pad, lead):
    keep = torch.ones(flat.shape, dtype=torch.bool)
    for t in range(T):
        keep[lead + t * (n + pad): lead + t * (n + pad) + n] = False
    return bool((flat.cpu().float()[keep] == GUARD).all())


def rng_of(*key):
    return np.random.default_rng(list(key))


# ---------------------------------------------------------------------------
# residual add + RMS norm


def norm_ref(x, r, w, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    v = s / torch.sqrt(s.square().mean(dim=1, keepdim=True) + eps)
    return s, v * w.double() if w is not None else v


# roundings of v relative to it: the sum s, the sum of squares (at most 16 or,
# past 16384 values, hidden/1024 products in a thread, then 6 wave and 16
# work-group additions; half of them count, under the root), mean, eps, root,
# reciprocal, two products
def norm_tol(H):
    return (1 + (max(16, 8 * -(-H // 8192)) + 6 + 16 + 2 * 2) / 2 + 6) * E


NORM_SHAPES = [(1, 1), (1, 2048), (3, 7), (5, 64), (2, 513), (33, 96), (4, 2047), (2, 2049), (7, 4096), (3, 4100),
               (2, 8191), (2, 16384), (2, 16385), (1, 20000), (300, 32)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("xt,rt,ot", [("f32", "f32", "f32"), ("bf16", "bf16", "bf16"), ("f16", "f16", "f16"),
                                      ("f32", "bf16", "f16"), ("bf16", "f32", "f32"), ("f16", None, "bf16"),
                                      ("f32", None, "f32")])
def test_add_rmsnorm(T, H, xt, rt, ot):
    g = rng_of(1, T, H)
    pad, lead = (0, 0) if H % 2 == 0 and T % 2 == 1 else (3, 1)
    x, xf = rows(g.standard_normal((T, H)), TYPES[xt], pad, lead)
    r, rf = rows(2 * g.standard_normal((T, H)), TYPES[rt], pad, lead) if rt else (None, None)
    ro, rof = rows(np.zeros((T, H)), TYPES[rt], pad, lead) if rt else (None, None)
    out, of = rows(np.zeros((T, H)), TYPES[ot], pad, lead)
    w = torch.from_numpy(1 + 0.1 * g.standard_normal(H)).float().cuda() if (T + H) % 3 else None
    s, v = norm_ref(x, r, w, 1e-5)
    keep = [t.clone() for t in (xf, rf) if t is not None]
    moe.moe_add_rmsnorm(x, w, out, residual=r, residual_out=ro, eps=1e-5)
    dt = TYPES[ot]
    assert ((out.double() - v).abs() <= (norm_tol(H) + u(dt)) * 1.001 * v.abs() + smallest(dt)).all()
    if rt:
        assert ((ro.double() - s).abs() <= (E + u(TYPES[rt])) * 1.001 * s.abs() + smallest(TYPES[rt])).all()
        assert untouched(rof, T, H, pad, lead)
    assert untouched(of, T, H, pad, lead)
    for a, b in zip(keep, (t for t in (xf, rf) if t is not None)):
        assert torch.equal(a, b)
    # in place: the residual, and out in x's place where the types agree
    xo = x if xt == ot else out
    moe.moe_add_rmsnorm(x, w, xo, residual=r, eps=1e-5)
    if xt != ot:
        assert torch.equal(xo, out)
    assert ((xo.double() - v).abs() <= (norm_tol(H) + u(dt)) * 1.001 * v.abs() + smallest(dt)).all()
    if rt:
        assert torch.equal(r, ro)


@pytest.mark.parametrize("T,H,xt,pad", [(1, 32, "f32", 0), (3, 96, "bf16", 3), (5, 2048, "bf16", 0), (2, 4128, "f16", 1),
                                        (2, 8192, "f32", 4), (2, 16416, "f32", 0), (70, 512, "f16", 0)])
def test_add_rmsnorm_8_bit(T, H, xt, pad):
    g = rng_of(2, T, H)
    x, _ = rows(g.standard_normal((T, H)) * np.exp(g.standard_normal((T, 1)) * 3), TYPES[xt], pad, pad)
    x[0, :32] = 0.0  # a group of zeros
    r, _ = rows(np.zeros((T, H)), TYPES[xt])
    r[:, 32:] = torch.from_numpy(g.standard_normal((T, H - 32))).to(TYPES[xt]).cuda() if H > 32 else 0
    out = torch.full((T, H + pad), 55, dtype=torch.int8, device="cuda")
    scales = torch.full((T, H // 32 + pad), GUARD, device="cuda")
    w = torch.from_numpy(1 + 0.1 * g.standard_normal(H)).float().cuda()
    _, v = norm_ref(x, r, w, 1e-6)
    moe.moe_add_rmsnorm(x, w, out[:, :H], residual=r, scales=scales[:, :H // 32], eps=1e-6)
    step, v = scales[:, :H // 32].double(), v.view(T, H // 32, 32)
    top = v.abs().amax(dim=2)
    # v's roundings and the division by 127
    assert ((step * 127 - top).abs() <= (norm_tol(H) + 2 * E) * 1.001 * top).all()
    code = out[:, :H].view(T, H // 32, 32).double() if pad == 0 else out[:, :H].reshape(T, H // 32, 32).double()
    # half a code, and up to 127 codes times the roundings of v, 127 / a and their product
    off = (code * step.unsqueeze(2) - v).abs()
    assert (off <= (0.5 + 127 * (2 * norm_tol(H) + 3 * E)) * 1.001 * step.unsqueeze(2)).all()
    assert (code.abs().amax(dim=2)[top > 0] == 127).all()
    if (top[0, 0] == 0):
        assert scales[0, 0] == 0 and (out[0, :32] == 0).all()
    assert pad == 0 or ((out[:, H:] == 55).all() and (scales[:, H // 32:] == GUARD).all())


def test_add_rmsnorm_8_bit_extremes():
    x = torch.ones((4, 64), device="cuda")
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    x[3, 32:] = 2.0 ** -130
    out, scales = torch.full((4, 64), 9, dtype=torch.int8, device="cuda"), torch.zeros((4, 2), device="cuda")
    plain = torch.zeros((4, 64), device="cuda")
    moe.moe_add_rmsnorm(x, None, out, scales=scales, eps=0.0)
    moe.moe_add_rmsnorm(x, None, plain, eps=0.0)
    assert (out[0] == 127).all()
    # 1 / sqrt(inf) = 0: inf * 0 is NaN, the finite values become 0
    assert torch.isnan(plain[1, 3]) and (plain[1, 32:] == 0).all() and torch.isnan(plain[2]).all()
    assert torch.isnan(scales[1, 0]) and scales[1, 1] == 0 and torch.isnan(scales[2]).all()
    assert (out[1:3] == 0).all()
    # the small half: below 2^-100, stored as zeros
    assert scales[3, 1] == 0 and (out[3, 32:] == 0).all() and (out[3, :32] == 127).all()


def test_add_rmsnorm_of_no_tokens_and_of_many():
    x = torch.zeros((0, 64), device="cuda")
    moe.moe_add_rmsnorm(x, None, x.clone())
    # more rows than the grid has work-groups
    T = (1 << 16) + 5
    x = torch.randn((T, 40), device="cuda")
    out = torch.zeros_like(x)
    moe.moe_add_rmsnorm(x, None, out, eps=1e-6)
    _, v = norm_ref(x, None, None, 1e-6)
    assert ((out.double() - v).abs() <= (norm_tol(40) + E) * 1.001 * v.abs()).all()


# ---------------------------------------------------------------------------
# dense product with 4-bit weights


class Product:
    """y = x W^T of random 4-bit weights, its fp64 value and the bound of an fp32 sum."""

    def __init__(self, T, N, K, xt, seed=0, scale=1.0):
        g = rng_of(3, T, N, K, seed)
        blocks = q4_matrix(g, N, K)
        nib, scl = moe.moe_q4_split(blocks)
        scl = (scl * scale).astype(np.float16) if scale != 1.0 else scl
        scl[:, 0] *= np.float16(-1)  # scales may be negative
        self.nib, self.scl = torch.from_numpy(nib).cuda(), torch.from_numpy(scl).cuda()
        self.scales = None
        if xt == "q8":
            codes = g.integers(-127, 128, (T, K)).astype(np.int8)
            s = (0.02 * np.exp(g.standard_normal((T, K // 32)))).astype(np.float32)
            self.x, self.scales = torch.from_numpy(codes).cuda(), torch.from_numpy(s).cuda()
            x = codes.reshape(T, K // 32, 32).astype(np.float64) * s[..., None]
        else:
            self.x = torch.from_numpy(g.standard_normal((T, K))).to(TYPES[xt]).cuda()
            x = self.x.cpu().double().numpy().reshape(T, K // 32, 32)
        q = np.concatenate([nib & 15, nib >> 4], axis=2).astype(np.float64) - 8
        d = scl.astype(np.float64)
        self.ref = x.reshape(T, K) @ (q * d[..., None]).reshape(N, K).T
        # A block's product is an fp32 sum of up to 3 terms per activation and as many of the -24
        # offset, 32 each: at most 192 roundings of partial sums below 55 sum |x|. 8-bit x: one more,
        # of scale * code. Then at most K/32 roundings of the sum over blocks, each partial sum below
        # sum |d| |block|, and the waves' sums (8 more).
        A = np.abs(x).sum(axis=2)
        blocks_abs = np.einsum("tb,nb->tn", A, np.abs(d)) * 8
        self.bound = np.einsum("tb,nb->tn", A, np.abs(d)) * (192 * 55 + 8) * E + (K / 32 + 8) * E * blocks_abs
        # the same roundings as independent errors (0.29 of a step each, partial sums of about
        # 24 sqrt(32) against a block of 4.6 sqrt(32)): sqrt(192) * 0.29 * 2 E * 24 / 4.6
        self.rms = np.sqrt(192) * 0.29 * 2 * E * 24 / 4.6

    def check(self, y, dtype):
        y = y.cpu().double().numpy()
        off = np.abs(y - self.ref)
        assert np.isfinite(y).all()
        assert (off <= self.bound + u(dtype) * 1.01 * np.abs(self.ref) + self.bound * u(dtype) + smallest(dtype)).all()
        assert np.linalg.norm(off) <= (self.rms + u(dtype)) * np.linalg.norm(self.ref)


Q4_SHAPES = [(1, 1, 32), (1, 16, 32), (1, 2048, 2048), (1, 33, 96), (2, 17, 1056), (5, 100, 4096), (15, 48, 160),
             (16, 64, 256), (17, 65, 288), (32, 130, 1536), (33, 31, 64), (64, 256, 512), (65, 20, 2080), (100, 1001, 352),
             (128, 128, 128), (129, 127, 1024), (200, 512, 96), (256, 300, 640), (257, 70, 1312), (300, 260, 256),
             (515, 129, 416), (1030, 140, 128)]
# rows shared by four waves (some with nothing left for the last ones), and the longest of them and past it
Q4_LONG = [(1, 37, 8224), (1, 2100, 8224), (1, 19, 16384), (1, 20, 32768), (1, 9, 32800), (2, 33, 4128), (2, 50, 8192),
           (3, 40, 16384), (4, 70, 8128), (6, 30, 16352), (2, 2049, 6368), (8, 90, 6400), (8, 2100, 8160),
           (7, 33, 2080), (5, 2100, 2080), (4, 2100, 16000),
           (16, 4200, 1056), (31, 4000, 4128)]
# above 2e9 products: 64 x 64 tiles with the reduction split, 128 x 128 tiles, and those in two passes of tokens
Q4_LARGE = [(130, 2050, 8224), (2100, 3900, 256), (16500, 520, 256), (4100, 4100, 160), (16500, 1100, 128)]


@pytest.mark.parametrize("T,N,K,xt,yt", [s + (x, y) for s in Q4_SHAPES + Q4_LONG for x, y in
                                         (("f32", "f32"), ("bf16", "f32"), ("f16", "f32"), ("q8", "f32"),
                                          ("bf16", "bf16"), ("f16", "f16"), ("q8", "bf16"))]
                         + [s + (x, y) for s in Q4_LARGE for x, y in
                            (("f32", "f32"), ("bf16", "f32"), ("f16", "f16"), ("q8", "f32"))])
def test_q4_matmul(T, N, K, xt, yt):
    p = Product(T, N, K, xt)
    pad, lead = (0, 0) if (T + N) % 2 else (5, 3)
    x, xf = (p.x, None) if xt == "q8" and pad == 0 else rows(p.x, p.x.dtype, pad, lead)
    y, yf = rows(np.full((T, N), 3.0), TYPES[yt], pad, lead)
    ws = moe.moe_q4_workspace(x, p.nib)
    if ws is not None:
        ws.fill_(255)  # any content
    moe.moe_q4_matmul(x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    p.check(y, TYPES[yt])
    assert untouched(yf, T, N, pad, lead)
    first = y.clone()
    moe.moe_q4_matmul(x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    assert torch.equal(first, y)  # equal calls, equal bits
    # y += : one more rounding, of the sum
    y.fill_(1.0)
    moe.moe_q4_matmul(x, p.nib, p.scl, y, scales=p.scales, workspace=ws, flags=moe.MOE_ACCUMULATE)
    dt = TYPES[yt]
    off = np.abs(y.cpu().double().numpy() - (p.ref + 1.0))
    assert (off <= p.bound + (u(dt) + E) * 1.01 * (np.abs(p.ref + 1.0) + p.bound) + smallest(dt)).all()


@pytest.mark.parametrize("T,N,K", [(1, 40, 256), (20, 40, 256), (300, 40, 256), (40, 6000, 8704)])
@pytest.mark.parametrize("xt,scale", [("f32", 2.0 ** 100), ("f32", 2.0 ** -90), ("bf16", 2.0 ** 100), ("f16", 2.0 ** -12),
                                      ("f16", 2.0 ** 12)])
def test_q4_matmul_keeps_precision_far_from_unit_scale(T, N, K, xt, scale):
    # fp16 at 2^-12: most values of x are subnormal or near it; they enter unrounded like any other
    p = Product(T, N, K, xt, seed=1)
    g = rng_of(31, T)
    x = torch.from_numpy(g.standard_normal((T, K)) * scale).to(TYPES[xt]).cuda()
    y = torch.zeros((T, N), device="cuda")
    moe.moe_q4_matmul(x, p.nib, p.scl, y)
    q = torch.cat([p.nib & 15, p.nib >> 4], dim=2).cpu().double() - 8
    w = (q * p.scl.cpu().double().unsqueeze(2)).view(N, K)
    ref = x.cpu().double() @ w.t()
    assert torch.linalg.norm(y.cpu().double() - ref) <= (p.rms + u(torch.float32)) * torch.linalg.norm(ref)


@pytest.mark.parametrize("T,N,K", [(3, 50, 128), (40, 50, 128), (260, 50, 128), (260, 1000, 8000)])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_q4_matmul_values_that_are_not_finite_stay_in_their_token(T, N, K, xt):
    p = Product(T, N, K, xt)
    clean = torch.zeros((T, N), device="cuda")
    moe.moe_q4_matmul(p.x, p.nib, p.scl, clean)
    p.x[1, 5], p.x[2, 77] = float("nan"), float("inf")
    y = torch.zeros((T, N), device="cuda")
    moe.moe_q4_matmul(p.x, p.nib, p.scl, y)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    rest = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("T,N,K", [(3, 50, 6400), (8, 50, 4128)])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16"])
def test_q4_matmul_values_that_are_not_finite_in_split_rows(T, N, K, xt):
    test_q4_matmul_values_that_are_not_finite_stay_in_their_token(T, N, K, xt)


@pytest.mark.parametrize("T,N,K", [(3, 50, 128), (5, 50, 6400), (40, 50, 128), (260, 1000, 8000)])
def test_q4_matmul_scales_that_are_not_finite_stay_in_their_token(T, N, K):
    p = Product(T, N, K, "q8")
    clean = torch.zeros((T, N), device="cuda")
    moe.moe_q4_matmul(p.x, p.nib, p.scl, clean, scales=p.scales)
    p.scales[1, 1], p.scales[2, 3] = float("nan"), float("inf")
    y = torch.zeros((T, N), device="cuda")
    moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    rest = [t for t in range(T) if t not in (1, 2)]
    assert torch.equal(y[rest], clean[rest])


def test_q4_matmul_of_no_tokens():
    p = Product(1, 8, 64, "f32")
    moe.moe_q4_matmul(p.x[:0], p.nib, p.scl, torch.zeros((0, 8), device="cuda"))


def test_q4_matmul_binding_refusals():
    p = Product(2, 8, 64, "f32")
    y = torch.zeros((2, 8), device="cuda")
    with pytest.raises(ValueError):
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y[:1])
    with pytest.raises(ValueError):
        moe.moe_q4_matmul(p.x, p.nib[:, :1], p.scl, y)
    with pytest.raises(ValueError):
        moe.moe_q4_matmul(p.x, p.nib, p.scl.float(), y)
    with pytest.raises(ValueError):
        moe.moe_q4_matmul(p.x.t(), p.nib, p.scl, y)
    with pytest.raises(ValueError):
        moe.moe_q4_matmul(p.x.expand(2, 2, 64)[0].double(), p.nib, p.scl, y)
    with pytest.raises(moe.MoeError) as ei:
        moe.moe_q4_matmul(p.x.to(torch.int8), p.nib, p.scl, y)  # codes without scales
    assert ei.value.code == moe.MOE_E_INVAL


# ---------------------------------------------------------------------------
# router balance


def balance_ref(z, k, valid, a, b):
    """fp64: counts, load, (balance, z) terms, lse, dlogits of a batch (z fp64 numpy)."""
    T, n_e = z.shape
    with np.errstate(divide="ignore", invalid="ignore"):
        top = z.max(axis=1, initial=-np.inf, keepdims=True)
        e = np.exp(z - np.where(np.isinf(top), 0.0, top))
        lse = np.where(np.isinf(top[:, 0]), -np.inf, top[:, 0] + np.log(e.sum(axis=1)))
    use = valid.astype(bool) & (lse > -np.inf)
    lse = np.where(use, lse, -np.inf)
    counts = np.zeros(n_e, np.int64)
    picks = np.argsort(-z[use], axis=1, kind="stable")[:, :k]  # ties: lower id first
    np.add.at(counts, picks.ravel(), 1)
    n = int(use.sum())
    d = np.zeros_like(z)
    if n == 0:
        return counts, np.zeros(n_e), 0.0, 0.0, lse, d, 0
    p = e[use] / e[use].sum(axis=1, keepdims=True)
    load = n_e * counts / (k * n)
    bal, zt = a * load @ p.mean(axis=0), b * np.mean(lse[use] ** 2)
    d[use] = p * (a * (load - (p @ load)[:, None]) + 2 * b * lse[use][:, None]) / n
    return counts, load, bal, zt, lse, d, n


class Balance:
    def __init__(self, z, k, valid=None, a=0.02, b=0.003, pad=0, lead=0):
        T, n_e = z.shape
        self.z, self.zf = rows(z, z.dtype, pad, lead)
        self.k, self.a, self.b, self.pad, self.lead = k, a, b, pad, lead
        self.valid = None if valid is None else torch.as_tensor(valid, dtype=torch.uint8).cuda()
        self.counts = torch.zeros(n_e, dtype=torch.int32, device="cuda")
        self.load, self.stats = torch.full((n_e,), GUARD, device="cuda"), torch.full((4,), GUARD, device="cuda")
        self.lse = torch.full((T,), GUARD, device="cuda")
        self.ws = moe.moe_router_balance_workspace(self.z).fill_(255)

    def forward(self, **kw):
        moe.moe_router_balance(self.z, self.k, self.counts, self.load, self.stats, self.lse, valid=self.valid,
                               balance=self.a, z=self.b, workspace=self.ws, **kw)

    def backward(self, d, **kw):
        moe.moe_router_balance_grad(self.z, self.load, self.stats, self.lse, d, balance=self.a, z=self.b, **kw)

    def check(self):
        z = self.z.cpu().double().numpy()
        T = z.shape[0]
        valid = np.ones(T, np.uint8) if self.valid is None else self.valid.cpu().numpy()
        counts, load, bal, zt, lse, d, n = balance_ref(z, self.k, valid, self.a, self.b)
        self.forward()
        assert np.array_equal(self.counts.cpu().numpy(), counts)
        assert np.abs(self.load.cpu().numpy() - load).max(initial=0) <= 2 * E * load.max(initial=0)
        st = self.stats.cpu().double().numpy()
        assert st[3] == n
        # exp: argument x (|x| below 64) times log2 e rounded, 1 + 1.44 |x| steps of E at most;
        # lse adds its own roundings of values below 64. A sum over tokens rounds at most
        # T / 2048 + 40 times. Everything below 2^-15 of the terms, which are all positive.
        tol = 2.0 ** -15 + (T / 2048) * E
        assert abs(st[1] - bal) <= tol * abs(bal) and abs(st[2] - zt) <= tol * abs(zt) + 1e-30
        assert abs(st[0] - bal - zt) <= tol * (abs(bal) + abs(zt))
        got = self.lse.cpu().double().numpy()
        none = np.isinf(lse)
        assert np.array_equal(np.isinf(got), none)
        assert (np.abs(got[~none] - lse[~none]) <= 2.0 ** -17 * np.maximum(1, np.abs(lse[~none]))).all()
        # the gradient: p off by 2^-16 of itself, times the absolute terms of its factor, then a rounding
        p_abs = np.zeros_like(z)  # the softmax of the tokens that count
        e = np.exp(z[~none] - z[~none].max(axis=1, keepdims=True))
        p_abs[~none] = e / e.sum(axis=1, keepdims=True)
        inner = (p_abs @ load)[:, None]
        size = p_abs * (self.a * (load[None] + inner) + 2 * self.b * np.abs(np.where(none, 0, lse))[:, None]) / max(n, 1)
        for dt in {self.z.dtype, torch.float32}:
            g = 64.0 * max(n, 1)  # a loss scale keeps fp16 gradients normal
            out, of = rows(np.zeros(z.shape), dt, self.pad, self.lead)
            scale = torch.full((1,), g, device="cuda")
            self.backward(out, dloss=scale)
            off = np.abs(out.cpu().double().numpy() - g * d)
            assert (off <= 2.0 ** -15 * g * size + u(dt) * 1.01 * np.abs(g * d) + smallest(dt)).all()
            assert untouched(of, *z.shape, self.pad, self.lead)
            # added to another gradient
            out.fill_(0.5)
            self.backward(out, dloss=scale, flags=moe.MOE_ACCUMULATE)
            off = np.abs(out.cpu().double().numpy() - (0.5 + g * d))
            assert (off <= 2.0 ** -15 * g * size + (u(dt) + E) * 1.01 * np.abs(0.5 + g * d) + u(dt) * 2.0 ** -14 * g * size).all()
            assert (out.cpu().numpy() if dt == torch.float32 else out.cpu().float().numpy())[none].tolist() == \
                np.full(z[none].shape, 0.5).tolist()
        return d


BALANCE_SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 60, 4), (64, 64, 8), (65, 100, 6), (40, 128, 1), (33, 256, 8),
                  (50, 257, 9), (100, 512, 8), (19, 512, 17), (21, 700, 8), (9, 1024, 32), (11, 1500, 8), (5, 2048, 12),
                  (7, 4095, 8), (6, 4096, 32), (20000, 16, 2),
                  # 16 lanes a row, not a wave
                  (2100, 200, 8), (2049, 256, 12), (2500, 300, 8), (2049, 509, 32)]


@pytest.mark.parametrize("T,n_e,k", BALANCE_SHAPES)
@pytest.mark.parametrize("zt", ["f32", "f16", "bf16"])
def test_router_balance(T, n_e, k, zt):
    g = rng_of(4, T, n_e, k)
    z = torch.from_numpy(3 * g.standard_normal((T, n_e))).to(TYPES[zt])
    pad, lead = (0, 0) if T % 2 else (3, 1)
    Balance(z, k, None if T % 3 else g.integers(0, 2, T), pad=pad, lead=lead).check()


@pytest.mark.parametrize("n_e,k", [(8, 3), (60, 4), (512, 8), (300, 12), (1024, 8), (4096, 20)])
def test_router_balance_ties_go_to_the_lower_id(n_e, k):
    g = rng_of(5, n_e, k)
    z = torch.from_numpy(g.integers(0, 3, (37, n_e)).astype(np.float32))
    z[0] = 0.0
    z[1] = torch.where(torch.arange(n_e) % 2 == 0, 0.0, -0.0)  # equal, whatever the sign of zero
    Balance(z, k).check()


@pytest.mark.parametrize("n_e,k", [(130, 32), (256, 9), (300, 12), (512, 8), (511, 31)])
def test_router_balance_ties_in_many_rows(n_e, k):
    g = rng_of(15, n_e, k)
    z = torch.from_numpy(g.integers(0, 40, (2200, n_e)).astype(np.float32))
    z[:7] = 0.0
    z[7] = torch.arange(n_e) // 8  # eight of a kind
    z[8] = torch.arange(n_e) // 9
    Balance(z, k).check()


def test_router_balance_masked_logits_and_tokens():
    g = rng_of(6)
    z = torch.from_numpy(g.standard_normal((12, 64)).astype(np.float32))
    low = torch.finfo(torch.float32).min
    z[0, 10:] = float("-inf")    # most experts masked
    z[1] = float("-inf")         # all of them: left out
    z[2, :62] = low              # the type's lowest value as the mask
    z[3] = low                   # every logit the lowest value: a uniform row
    z[4] = -60.0
    z[4, 63] = 0.0
    valid = np.ones(12, np.uint8)
    valid[7] = 0
    for k in (2, 10):
        b = Balance(z, k, valid)
        b.b = 0.0  # the z loss of lse = -3.4e38 overflows fp32
        d = b.check()
        assert b.stats[3].item() == 10 and (d[[1, 7]] == 0).all()
    # fewer unmasked experts than picks: the picks go on to the lowest masked ids, as the routing's do
    b = Balance(z[:1], 20)
    b.b = 0.0
    b.check()
    assert (b.counts[:20] == 1).all() and (b.counts[20:] == 0).all()


def test_router_balance_without_tokens():
    z = torch.randn(5, 32)
    for zz, valid in ((z, np.zeros(5, np.uint8)), (z[:0], None), (torch.full((5, 32), float("-inf")), None)):
        b = Balance(zz, 4, valid)
        b.forward()
        assert (b.counts == 0).all() and (b.load == 0).all() and (b.stats == 0).all()
        d = torch.full(tuple(zz.shape), GUARD, device="cuda")
        b.backward(d)
        assert (d == 0).all() and (b.lse == float("-inf")).all()
    # nor is there a row to read: the address of an empty tensor is null
    none = torch.empty((0, 300), device="cuda")
    out = [torch.ones(300, dtype=torch.int32, device="cuda"), torch.ones(300, device="cuda"), torch.ones(4, device="cuda")]
    assert none.data_ptr() == 0
    moe.moe_router_balance(none, 8, *out, torch.empty(0, device="cuda"))
    moe.moe_router_balance_grad(none, out[1], out[2], torch.empty(0, device="cuda"), torch.empty((0, 300), device="cuda"))
    assert all((o == 0).all() for o in out)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_router_balance_values_that_are_not_finite_show(bad):
    z = torch.randn(6, 64)
    z[2, 5] = bad
    b = Balance(z, 4)
    b.forward()
    assert torch.isnan(b.stats[:3]).all() and b.stats[3] == 6 and int(b.counts.sum()) == 24
    d = torch.zeros((6, 64), device="cuda")
    b.backward(d)
    assert torch.isnan(d[2]).all() and torch.isfinite(d[[0, 1, 3, 4, 5]]).all()


def test_router_balance_gradient_against_differences():
    g = rng_of(7)
    z = g.standard_normal((5, 12))
    valid = np.array([1, 1, 0, 1, 1], np.uint8)
    a, b, k = 0.7, 0.3, 3

    bal = Balance(torch.from_numpy(z).float(), k, valid, a=a, b=b)
    z = bal.z.cpu().double().numpy()
    _, load, _, _, _, _, n = balance_ref(z, k, valid, a, b)

    def loss(z):  # the picks, so the loads, held
        use = valid.astype(bool)
        e = np.exp(z[use])
        lse = np.log(e.sum(axis=1))
        return a * load @ (e / e.sum(axis=1, keepdims=True)).mean(axis=0) + b * np.mean(lse ** 2)

    bal.forward()
    d = torch.zeros((5, 12), device="cuda")
    bal.backward(d)
    h = 1e-5
    for t in range(5):
        for e in range(12):
            hi, lo = z.copy(), z.copy()
            hi[t, e] += h
            lo[t, e] -= h
            # the difference is off by h^2 / 6 of the third derivative (below 1) and 1e-16 / h
            assert abs(d[t, e].item() - (loss(hi) - loss(lo)) / (2 * h)) <= 2.0 ** -15 * 0.3 / n + 1e-9
    # dlogits in the logits' place
    want = d.clone()
    moe.moe_router_balance_grad(bal.z, bal.load, bal.stats, bal.lse, bal.z, balance=a, z=b)
    assert torch.equal(bal.z, want)


def test_router_balance_counts_add_up_and_match_the_routing():
    """Counts over several batches are the frequency table of moe_seed, and the picks are moe_forward's."""
    wl = Workload("decode-e64k8-h256f512-t16-counts", 321, 1, 64, 8, 256, 512, tokens=16, steps=4, zipf_s=1.1, slots=24)
    d = Decode(wl, seed=False)
    try:
        z = zipf_logits(wl)
        counts = torch.zeros((1, 64), dtype=torch.int32, device="cuda")
        load, stats, lse = torch.zeros(64, device="cuda"), torch.zeros(4, device="cuda"), torch.zeros(16, device="cuda")
        for s in range(wl.steps):
            zl = torch.from_numpy(z[s, 0]).cuda()
            x = torch.from_numpy(activations(wl, s)).cuda()
            moe.moe_forward(d.ctx, 0, 16, x, zl, torch.empty_like(x))
            moe.moe_cache_step(d.ctx)
            moe.moe_router_balance(zl, 8, counts[0], load, stats, lse, balance=1.0, flags=moe.MOE_ACCUMULATE)
        want = moe.moe_get_counts(d.ctx, 1, 64)
        freq = counts.cpu().numpy().view(np.uint32)
        assert np.array_equal(freq, want)
        moe.moe_seed(d.ctx, freq)  # the 24 most used experts, ties to the lower id
        best = np.argsort(-freq[0].astype(np.int64), kind="stable")[:24]
        table = moe.moe_get_slot_table(d.ctx, 0, 64)
        assert np.array_equal(table[best], np.arange(24)) and (np.delete(table, best) == -1).all()
    finally:
        d.close()


# ---------------------------------------------------------------------------
# streams, graphs, and a step made of them


def test_calls_on_another_stream_and_two_at_once():
    ps = [Product(40, 300, 512, "f32", seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in ps]
    ys = [torch.zeros((40, 300), device="cuda") for _ in ps]
    wss = [moe.moe_q4_workspace(p.x, p.nib) for p in ps]
    zs = [Balance(torch.randn(500, 96), 6) for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, y, ws, b, s in zip(ps, ys, wss, zs, streams):
            moe.moe_q4_matmul(p.x, p.nib, p.scl, y, workspace=ws, stream=s)
            b.forward(stream=s)
    torch.cuda.synchronize()
    for p, y, b in zip(ps, ys, zs):
        p.check(y, torch.float32)
        b.check()
    # torch's current stream is taken when none is given
    with torch.cuda.stream(streams[0]):
        ys[0].zero_()
        moe.moe_q4_matmul(ps[0].x, ps[0].nib, ps[0].scl, ys[0])
    streams[0].synchronize()
    ps[0].check(ys[0], torch.float32)
    if moe.moe_q4_workspace(ps[0].x, ps[0].nib) is not None:
        with pytest.raises(ValueError):
            moe.moe_q4_matmul(ps[0].x, ps[0].nib, ps[0].scl, ys[0], stream=streams[0])
    with pytest.raises(ValueError):
        moe.moe_router_balance(zs[0].z, 6, zs[0].counts, zs[0].load, zs[0].stats, zs[0].lse, stream=streams[0])


@pytest.mark.parametrize("T,N,K,xt", [(260, 1000, 8000, "f32"), (260, 1000, 8000, "q8"), (4100, 4100, 160, "bf16"),
                                      (4, 300, 8192, "bf16")])
def test_large_and_split_products_at_once_and_captured(T, N, K, xt):
    ps = [Product(T, N, K, xt, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in ps]
    ys = [torch.zeros((T, N), device="cuda") for _ in ps]
    wss = [moe.moe_q4_workspace(p.x, p.nib) for p in ps]
    for p, y, ws in zip(ps, ys, wss):
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    torch.cuda.synchronize()
    want = [y.clone() for y in ys]
    for _ in range(5):
        for p, y, ws, s in zip(ps, ys, wss, streams):
            moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))
    # both in one graph, one after the other through the same workspace; another's eager calls between the replays
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for p, y in zip(ps, ys):
            moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=wss[0])
    for _ in range(3):
        for y in ys:
            y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ys, want))
        moe.moe_q4_matmul(ps[1].x, ps[1].nib, ps[1].scl, ys[0], scales=ps[1].scales, workspace=wss[0])
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 24, 300])
def test_captured_and_replayed(T):
    """One graph of norm (8-bit) -> product -> norm -> product, and the router's losses, replayed on changing inputs."""
    g = rng_of(8, T)
    H, N = 256, 320
    x, r = (torch.from_numpy(g.standard_normal((T, H))).float().cuda() for _ in range(2))
    p, p2 = Product(1, N, H, "f32", seed=T), Product(1, 64, N, "f32", seed=T + 1)
    codes, scales = torch.zeros((T, H), dtype=torch.int8, device="cuda"), torch.zeros((T, H // 32), device="cuda")
    y, yn, z = (torch.zeros((T, n), device="cuda") for n in (N, N, 64))
    ro = torch.zeros_like(r)
    ws = [moe.moe_q4_workspace(codes, p.nib), moe.moe_q4_workspace(yn, p2.nib)]
    counts, load = torch.zeros(64, dtype=torch.int32, device="cuda"), torch.zeros(64, device="cuda")
    stats, lse, d = torch.zeros(4, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros((T, 64), device="cuda")
    bws = moe.moe_router_balance_workspace(z)
    outs = [ro, codes, scales, y, yn, z, counts, load, stats, lse, d]

    def step():
        moe.moe_add_rmsnorm(x, None, codes, residual=r, residual_out=ro, scales=scales)
        moe.moe_q4_matmul(codes, p.nib, p.scl, y, scales=scales, workspace=ws[0])
        moe.moe_add_rmsnorm(y, None, yn)
        moe.moe_q4_matmul(yn, p2.nib, p2.scl, z, workspace=ws[1])
        moe.moe_router_balance(z, 8, counts, load, stats, lse, balance=0.1, z=0.01, workspace=bws)
        moe.moe_router_balance_grad(z, load, stats, lse, d, balance=0.1, z=0.01)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(5):
        x.copy_(torch.from_numpy(g.standard_normal((T, H))).float())
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i
        (x.sum() + r.sum()).item()  # the program's own work between the replays


def test_decode_step_of_norms_products_and_experts():
    """A layer as a user of the library decodes it: residual add + norm, router logits and a shared expert's
    up projection through 4-bit weights, the routed experts, everything added to the residual stream."""
    wl = Workload("decode-e64k8-h256f512-t5-layer", 322, 1, 64, 8, 256, 512, tokens=5, steps=3, zipf_s=1.1, slots=24)
    d = Decode(wl)
    try:
        T, H = wl.tokens, wl.hidden
        g = rng_of(9)
        shared, head = Product(1, H, H, "f32", seed=5), Product(1, 64, H, "f32", seed=6)
        dense = [(torch.cat([q.nib & 15, q.nib >> 4], dim=2).cpu().double() - 8) * q.scl.cpu().double().unsqueeze(2)
                 for q in (shared, head)]
        weight = torch.from_numpy(1 + 0.1 * g.standard_normal(H)).float().cuda()
        stream = torch.from_numpy(g.standard_normal((T, H))).float().cuda()
        y, xn = torch.zeros((T, H), device="cuda"), torch.zeros((T, H), device="cuda")
        logits, ids = torch.zeros((T, 64), device="cuda"), torch.zeros((T, 8), dtype=torch.int32, device="cuda")
        for s in range(wl.steps):
            before = stream.cpu().double() + y.cpu().double()
            moe.moe_add_rmsnorm(y, weight, xn, residual=stream, eps=1e-6)  # stream += y of the step before
            moe.moe_q4_matmul(xn, head.nib, head.scl, logits)
            moe.moe_forward(d.ctx, 0, T, xn, logits, y, ids)
            moe.moe_q4_matmul(xn, shared.nib, shared.scl, y, flags=moe.MOE_ACCUMULATE)
            moe.moe_cache_step(d.ctx)
            _, v = norm_ref(before, None, weight.cpu(), 1e-6)
            z = logits.cpu().double()
            assert (z - v @ dense[1].view(64, H).t()).abs().max() <= 1e-5 * z.abs().max()
            ref, ids_ref, _ = oracle.moe_layer(64, 8, H, wl.ffn, d.experts(0, ids.cpu().numpy()), v.numpy(),
                                               logits=logits.cpu().numpy())
            assert np.array_equal(ids.cpu().numpy(), ids_ref)
            ref = ref + (v @ dense[0].view(H, H).t()).numpy()
            assert token_rel_err(y.cpu().numpy(), ref) < TOL
            assert ((stream.cpu().double() - before).abs() <= E * 1.001 * before.abs()).all()
    finally:
        d.close()

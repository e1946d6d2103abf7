"""The operators beside the experts at the limits of their types: rows whose
squares leave fp32's range, values that are not finite, and calls after
somebody else's error.

Tolerances count roundings as in test_gpu_dense_ops.py.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests._gpu import Decode  # noqa: E402
from tests.test_gpu_dense_ops import (  # noqa: E402
    E, TYPES, Balance, Product, norm_ref, norm_tol, rng_of, smallest, u)
from workload import Workload, activations, zipf_logits  # noqa: E402

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# residual add + RMS norm: finite rows whose squares overflow or underflow

# one wave, four, sixteen, and rows that are read twice
NORM_WIDTHS = [1, 64, 100, 2048, 2051, 4096, 8200, 16384, 16400]


@pytest.mark.parametrize("H", NORM_WIDTHS)
@pytest.mark.parametrize("xt,rt,ot", [("f32", None, "f32"), ("f32", "f32", "f32"), ("bf16", "bf16", "bf16"),
                                      ("f32", "bf16", "f16"), ("bf16", None, "f32")])
def test_add_rmsnorm_far_from_unit_scale(H, xt, rt, ot):
    for size, eps in ((1e17, 1e-6), (1e19, 1e-6), (1e25, 1e-6), (5e37, 1e-6), (1e25, 1e35), (1e-14, 0.0), (1e-17, 0.0),
                      (1e-17, 1e-34), (1e-24, 0.0), (1e-30, 0.0), (1e-30, 1e-38), (1e-37, 0.0), (1e-30, 1e-6)):
        far_from_unit_scale(H, xt, rt, ot, size, eps)


def far_from_unit_scale(H, xt, rt, ot, size, eps):
    T = 3
    g = rng_of(40, H)
    x = torch.from_numpy(g.standard_normal((T, H)) * size).to(TYPES[xt]).cuda()
    x[1] = torch.from_numpy(g.standard_normal(H)).to(TYPES[xt]).cuda() * (1.0 if eps else 1e-3)  # a row of ordinary size
    r = torch.from_numpy(g.standard_normal((T, H)) * size / 4).to(TYPES[rt]).cuda() if rt else None
    w = torch.from_numpy(1 + 0.1 * g.standard_normal(H)).float().cuda() if H % 3 else None
    out = torch.zeros((T, H), dtype=TYPES[ot], device="cuda")
    ro = torch.zeros_like(r) if rt else None
    s, v = norm_ref(x, r, w, eps)
    moe.moe_add_rmsnorm(x, w, out, residual=r, residual_out=ro, eps=eps)
    dt = TYPES[ot]
    # one rounding more than an ordinary row: of s off its power of two
    assert ((out.double() - v).abs() <= (norm_tol(H) + E + u(dt)) * 1.001 * v.abs() + smallest(dt)).all(), (size, eps)
    if rt:
        assert ((ro.double() - s).abs() <= (E + u(TYPES[rt])) * 1.001 * s.abs() + smallest(TYPES[rt])).all()
        moe.moe_add_rmsnorm(x, w, out.clone(), residual=r, eps=eps)  # in place
        assert torch.equal(r, ro)


@pytest.mark.parametrize("H", [64, 2048, 8192, 16416])
@pytest.mark.parametrize("size", [1e24, 1e-28])
def test_add_rmsnorm_8_bit_far_from_unit_scale(H, size):
    g = rng_of(41, H)
    x = torch.from_numpy(g.standard_normal((2, H)) * size).float().cuda()
    out, scales = torch.zeros((2, H), dtype=torch.int8, device="cuda"), torch.zeros((2, H // 32), device="cuda")
    moe.moe_add_rmsnorm(x, None, out, scales=scales, eps=0.0)
    v = norm_ref(x, None, None, 0.0)[1].view(2, H // 32, 32)
    step = scales.double()
    top = v.abs().amax(dim=2)
    tol = norm_tol(H) + E
    assert ((step * 127 - top).abs() <= (tol + 2 * E) * 1.001 * top).all()
    off = (out.view(2, H // 32, 32).double() * step.unsqueeze(2) - v).abs()
    assert (off <= (0.5 + 127 * (2 * tol + 3 * E)) * 1.001 * step.unsqueeze(2)).all()


@pytest.mark.parametrize("H", [64, 2048, 8192, 16400])
def test_add_rmsnorm_rows_of_zeros_and_of_one_value(H):
    x = torch.zeros((5, H), device="cuda")
    x[1, 3] = 1e-45  # fp32's smallest
    x[2, 5] = 3e38
    x[3] = 3e38
    out = torch.zeros_like(x)
    moe.moe_add_rmsnorm(x, None, out, eps=0.0)
    v = norm_ref(x[1:4], None, None, 0.0)[1]
    assert ((out[1:4].double() - v).abs() <= (norm_tol(H) + 2 * E) * 1.001 * v.abs()).all()
    assert torch.isnan(out[[0, 4]]).all()  # 0 / 0
    moe.moe_add_rmsnorm(x, None, out, eps=1e-6)
    assert (out[[0, 4]] == 0).all()


# ---------------------------------------------------------------------------
# an error that another HIP call left with the thread


class PendingError:
    """A host-side error of the thread, left unread: no such device."""

    def __enter__(self):
        torch.cuda.synchronize()
        assert moe.lib().hipSetDevice(9999) != 0

    def __exit__(self, *exc):
        moe.lib().hipGetLastError()  # or the next call of torch would raise it


def test_a_pending_error_of_another_call_is_not_a_launchs():
    p = Product(5, 33, 64, "f32")
    x, out, y = torch.ones((3, 64), device="cuda"), torch.zeros((3, 64), device="cuda"), torch.zeros((5, 33), device="cuda")
    residual = torch.ones((3, 64), device="cuda")
    with PendingError():
        moe.moe_add_rmsnorm(x, None, out, residual=residual)
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y)
    assert (residual == 2).all() and (out - 1).abs().max() < 1e-6
    p.check(y, torch.float32)
    # calls of several launches: the operand pass and the tiles; rows, finish and gradient
    p = Product(200, 4100, 4096, "bf16")
    y, ws = torch.zeros((200, 4100), device="cuda"), moe.moe_q4_workspace(p.x, p.nib)
    assert ws is not None
    b = Balance(torch.randn(50, 96), 6)
    d = torch.zeros((50, 96), device="cuda")
    with PendingError():
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y, workspace=ws)
        b.forward()
        b.backward(d)
    p.check(y, torch.float32)
    assert int(b.counts.sum()) == 300 and b.stats[3] == 50 and d.abs().max() > 0
    b.check()


def test_a_pending_error_of_another_call_is_not_the_experts():
    wl = Workload("decode-e64k8-h256f512-t5-pending", 323, 1, 64, 8, 256, 512, tokens=5, steps=2, zipf_s=1.1, slots=24)
    d = Decode(wl)
    try:
        x, z = torch.from_numpy(activations(wl, 0)).cuda(), torch.from_numpy(zipf_logits(wl)[0, 0]).cuda()
        y, want = torch.zeros_like(x), torch.zeros_like(x)
        moe.moe_forward(d.ctx, 0, 5, x, z, want)
        moe.moe_cache_step(d.ctx)
        with PendingError():
            moe.moe_forward(d.ctx, 0, 5, x, z, y)
            moe.moe_cache_step(d.ctx)
            gbps = moe.moe_measure_read_bandwidth(nbytes=1 << 20)
        assert gbps > 0 and (y - want).abs().max() <= 1e-5 * want.abs().max()
    finally:
        d.close()


# ---------------------------------------------------------------------------
# dense product: an infinite weight scale belongs to its feature and block alone


# the dot product's lane layouts with places past the row, tiles, and split tiles
@pytest.mark.parametrize("T,N,K", [(1, 9, 96), (1, 9, 544), (1, 40, 2080), (2, 40, 1056), (1, 40, 4128), (1, 40, 8224),
                                   (4, 40, 2080), (8, 33, 4128), (20, 33, 96), (40, 33, 2080), (200, 3001, 3744)])
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16", "q8"])
def test_q4_matmul_infinite_scale_of_the_last_block(T, N, K, xt):
    p = Product(T, N, K, xt, seed=2)
    y = torch.zeros((T, N), device="cuda")
    p.scl[3, -1], p.scl[5, -1], p.scl[7, -1] = float("inf"), float("-inf"), float("nan")
    p.nib[3, -1] = p.nib[5, -1] = 0x99  # q - 8 = 1: the block's sum is that of x
    p.x[:, -32:] = p.x[:, -32:].abs() + 1 if xt != "q8" else p.x[:, -32:].clamp(1)
    moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales)
    assert (y[:, 3] == float("inf")).all() and (y[:, 5] == float("-inf")).all() and torch.isnan(y[:, 7]).all()
    rest = [n for n in range(N) if n not in (3, 5, 7)]
    assert torch.isfinite(y[:, rest]).all()


# ---------------------------------------------------------------------------
# router balance: NaN of any bits


@pytest.mark.parametrize("T,n_e", [(5, 3), (40, 8), (40, 60), (40, 100), (40, 200), (40, 512), (2100, 200), (2100, 500), (9, 1000),
                                   (9, 1500), (9, 4093)])
@pytest.mark.parametrize("zt", ["f32", "f16", "bf16"])
def test_router_balance_counts_its_picks_beside_nan(T, n_e, zt):
    g = rng_of(42, T, n_e)
    for k in {min(3, n_e), min(8, n_e), min(9, n_e), min(32, n_e)}:
        z = torch.from_numpy(g.standard_normal((T, n_e))).to(TYPES[zt])
        ones = z.view(torch.int32 if zt == "f32" else torch.int16)
        ones[1] = -1                                     # the lowest NaN there is, in every place
        ones[2, n_e // 2:] = -1                          # fewer numbers than picks, for few experts
        ones[3, [0, n_e - 1]] = -1
        z[4, n_e // 3] = float("nan")
        want = np.zeros(n_e, np.int64)
        # the order of moe_forward's picks: a NaN with the sign bit below all numbers, one without above
        key = z.float().numpy().view(np.uint32).astype(np.int64)
        key = np.where(key >> 31, 0xFFFFFFFF - key, key | 0x80000000)
        np.add.at(want, np.argsort(-key, axis=1, kind="stable")[:, :k].ravel(), 1)
        b = Balance(z, k)
        b.forward()
        assert np.array_equal(b.counts.cpu().numpy(), want), k
        assert torch.isnan(b.stats[:3]).all() and b.stats[3] == T


# ---------------------------------------------------------------------------
# dense product: activations near the end of fp32's range


@pytest.mark.parametrize("T,N,K", [(1, 40, 256), (20, 40, 256), (200, 4100, 4096), (4100, 4100, 160)])
@pytest.mark.parametrize("xt", ["f32", "bf16"])
def test_q4_matmul_tiny_activations(T, N, K, xt):
    p = Product(T, N, K, xt, seed=3)
    p.scl *= 2048  # the smallest of them times x is then a normal fp32 number still
    g = rng_of(43, T, N, K)
    q = torch.cat([p.nib & 15, p.nib >> 4], dim=2).float() - 8
    w = (q * p.scl.float().unsqueeze(2)).view(N, K).double()
    base = torch.from_numpy(g.standard_normal((T, K))).cuda()
    y = torch.zeros((T, N), device="cuda")
    for e in (-100, -109, -112, -118, -124, -130, -140):
        x = (base * 2.0 ** e).to(TYPES[xt])
        moe.moe_q4_matmul(x, p.nib, p.scl, y)
        ref = x.double() @ w.t().contiguous()
        # p.rms as for ordinary values (sums in fp32: a block's from its start, the values below 2^-126 to
        # 2^-150 each); of an fp32 value the bits below 2^-133, all of one sign
        cut = (2.0 ** -133 if xt == "f32" else 0.0) * w.abs().sum(dim=1)
        ends = 2.0 ** -150 * (192 * p.scl.double().abs().sum(dim=1) + 2 * K)
        off = (y.double() - ref).abs()
        size = torch.linalg.norm(ref, dim=1, keepdim=True) / N ** 0.5
        # the largest of N T errors of size p.rms: eight of them
        assert (off <= 8 * (p.rms + E) * size + (cut + ends) * 1.01).all(), e


# ---------------------------------------------------------------------------
# dense product: which form a call takes


# (tokens, features, reduction, types with an operand pass): rows too long, tiles too few or features too few for it
# (one launch), split tiles, and whole tiles (fp32: from fewer of them on)
FORMS = [(64, 510, 65536, ""), (33, 2050, 31008, ""), (300, 1024, 7008, ""), (17000, 255, 512, ""), (33000, 70, 960, ""),
         (448, 1000, 4800, "f32 bf16 f16"), (200, 4001, 3936, "f32 bf16 f16 q8"), (260, 2100, 4000, "f32 bf16 f16 q8"),
         (8200, 257, 992, "f32 bf16 f16 q8"), (1030, 4200, 512, "f32 bf16 f16 q8"), (16500, 258, 512, "f32 bf16 f16 q8")]


@pytest.mark.parametrize("T,N,K,passes", FORMS)
@pytest.mark.parametrize("xt", ["f32", "bf16", "f16", "q8"])
def test_q4_matmul_forms(T, N, K, passes, xt):
    p = Product(T, N, K, xt, seed=4)
    y = torch.zeros((T, N), device="cuda")
    ws = moe.moe_q4_workspace(p.x, p.nib)
    assert (ws is not None) == (xt in passes.split())
    if ws is not None:
        ws.fill_(255)
    moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    p.check(y, torch.float32)
    first = y.clone()
    moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    assert torch.equal(first, y)
    # a token that is not finite shows in its row alone
    if xt == "q8":
        p.scales[3, 1] = float("nan")
    else:
        p.x[3, 40] = float("inf")
    moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    assert torch.isnan(y[3]).all()
    assert torch.equal(torch.cat([y[:3], y[4:]]), torch.cat([first[:3], first[4:]]))


@pytest.mark.parametrize("xt", ["f32", "bf16", "q8"])
def test_q4_matmul_split_tiles_at_once_and_captured(xt):
    T, N, K = 200, 4001, 3936
    ps = [Product(T, N, K, xt, seed=s) for s in (5, 6)]
    ys, wss = [torch.zeros((T, N), device="cuda") for _ in ps], [moe.moe_q4_workspace(p.x, p.nib) for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    assert all(ws is not None for ws in wss)
    for p, y, ws in zip(ps, ys, wss):
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws)
    torch.cuda.synchronize()
    want = [y.clone() for y in ys]
    for y in ys:
        y.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for p, y, ws, s in zip(ps, ys, wss, streams):
            moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ys, want))
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


# ---------------------------------------------------------------------------
# workspaces on other streams


@pytest.mark.parametrize("xt", ["f32", "bf16", "q8"])
def test_q4_matmul_workspace_of_the_binding_on_a_side_stream(xt):
    T, N, K = 200, 4001, 3936
    p = Product(T, N, K, xt, seed=7)
    need = moe.moe_q4_workspace(p.x, p.nib)
    assert need is not None
    y, side = torch.zeros((T, N), device="cuda"), torch.cuda.Stream()
    with pytest.raises(ValueError, match="workspace"):  # torch's memory would follow the current stream, the call another
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, stream=side)
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, stream=side.cuda_stream)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales, workspace=need[:-256])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(5):
            y.zero_()
            moe.moe_q4_matmul(p.x, p.nib, p.scl, y, scales=p.scales)
            torch.empty_like(need).fill_(255)  # the same memory again, for the stream's next work
    side.synchronize()
    p.check(y, torch.float32)


def test_router_balance_workspace_of_the_binding_on_a_side_stream():
    b, side = Balance(torch.randn(500, 96), 6), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(5):
            moe.moe_router_balance(b.z, 6, b.counts, b.load, b.stats, b.lse, balance=b.a, z=b.b)
            torch.empty_like(b.ws).fill_(255)
        d = torch.zeros((500, 96), device="cuda")
        b.backward(d)
    side.synchronize()
    counts, stats, got = b.counts.clone(), b.stats.clone(), d.clone()
    b.check()
    b.backward(d)
    assert torch.equal(counts, b.counts) and torch.equal(stats, b.stats) and torch.equal(got, d)


# ---------------------------------------------------------------------------
# offsets past 32 bits


def far_rows(a, dtype, stride):
    """a [T][n] as rows `stride` values apart, in memory that is otherwise as it comes."""
    T, n = a.shape
    v = torch.empty(T * stride, dtype=dtype, device="cuda").view(T, stride)[:, :n]
    v.copy_(a)
    return v


@pytest.fixture
def big_memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("100 GB of free device memory are needed")
    yield
    torch.cuda.empty_cache()


def test_rows_further_apart_than_32_bits(big_memory):
    T, stride = 37, (1 << 27) + 24  # 4.9e9 values
    g = rng_of(44)
    near = torch.from_numpy(g.standard_normal((T, 96))).to(torch.bfloat16).cuda()
    x, r = far_rows(near, torch.bfloat16, stride), near.clone()
    out, want, res = far_rows(torch.zeros_like(near), torch.bfloat16, stride), torch.zeros_like(near), near.clone()
    moe.moe_add_rmsnorm(near, None, want, residual=r)
    moe.moe_add_rmsnorm(x, None, out, residual=res)
    assert torch.equal(out, want) and torch.equal(res, r)
    del out
    for n in (1, 2, 37):  # dots, tiles
        p = Product(n, 70, 96, "bf16", seed=8)
        y = [torch.zeros((n, 70), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        moe.moe_q4_matmul(near[:n], p.nib, p.scl, y[0])
        moe.moe_q4_matmul(x[:n], p.nib, p.scl, y[1])
        assert torch.equal(*y)
        y[1] = far_rows(torch.zeros_like(y[0]), torch.bfloat16, stride)
        moe.moe_q4_matmul(near[:n], p.nib, p.scl, y[1])
        assert torch.equal(*y)
    b, far = Balance(near, 6), Balance(near, 6)
    far.z = x
    d, dfar = torch.zeros_like(near), far_rows(torch.zeros_like(near), torch.bfloat16, stride)
    b.forward(), far.forward()
    b.backward(d), far.backward(dfar)
    assert torch.equal(b.counts, far.counts) and torch.equal(b.stats, far.stats) and torch.equal(b.lse, far.lse)
    assert torch.equal(d, dfar)


@pytest.mark.parametrize("T", [1, 20, 40])
def test_weights_of_more_than_2_31_blocks(T, big_memory):
    N, K = 1 << 22, 16416  # the most features, 513 blocks each: dots of rows split over waves, tiles, whole tiles
    p = Product(T, 64, K, "bf16", seed=9)
    nib = torch.empty((N, K // 32, 16), dtype=torch.uint8, device="cuda")
    scl = torch.zeros((N, K // 32), dtype=torch.float16, device="cuda")
    y = torch.full((T, N), 3.0, device="cuda")
    at = torch.tensor([i + j for i in (0, 40, (1 << 31) // 513 - 8, N - 16) for j in range(16)], device="cuda")
    nib[at], scl[at] = p.nib, p.scl
    moe.moe_q4_matmul(p.x, nib, scl, y)
    p.check(y[:, at], torch.float32)
    y[:, at] = 0
    assert (y == 0).all()  # every other feature's scales are zero

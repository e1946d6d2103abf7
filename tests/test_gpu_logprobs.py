"""Log probabilities, entropies, alternatives and their gradient on the GPU, against
their definitions in fp64.

Tolerances count roundings: E = 2^-24 of a result per fp32 operation, u(type) half a
step of the output's type.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_gpu_dense_ops import TYPES, E, rng_of, rows, smallest, u, untouched  # noqa: E402

pytestmark = pytest.mark.gpu

INF = float("inf")


def reference(z, targets, scale, n):
    """logp, entropy, lse, ids, log p of them, log p; in fp64."""
    z = z.double() * scale
    T, V = z.shape
    top = z.amax(dim=1, keepdim=True)
    none = top == -INF
    d = z - torch.where(none, 0.0, top)
    s = d.exp().sum(dim=1, keepdim=True)
    lp = torch.where(none, -INF, d - s.log())
    p = lp.exp()
    H = -torch.where(p > 0, p * lp, 0.0).sum(dim=1)
    lse = torch.where(none, -INF, top + s.log()).squeeze(1)
    y = targets.long()
    ok = (y >= 0) & (y < V)
    logp = torch.where(ok, lp.gather(1, y.clamp(0, V - 1)[:, None]).squeeze(1), 0.0)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :n]
    alt = lp.gather(1, ids)
    return logp, H, lse, torch.where(alt == -INF, -1, ids).int(), alt, lp


def bounds(lp, V):
    """Errors of log p and of the entropy.

    A power's argument has three roundings relative to it, the power two, so the sum of them is off by E * (3 mean |log p -
    log p of the best| + 2); it is added up by a thread over its share (256 threads a row, or one wave for short rows, of 8
    values each in turn), then over 6 + 4 (waves) + 6 (slices) steps; its rescalings are as many again as runs of 32.
    The entropy's second sum has the same, times the mean, and one rounding more each."""
    depth = V / (256 if V > 2048 else 64) * 1.1 + 8 + 20
    p = lp.exp()
    best = lp.amax(dim=1, keepdim=True)
    d = torch.where(p > 0, p * (best - lp), 0.0).sum(dim=1)
    d2 = torch.where(p > 0, p * (best - lp) ** 2, 0.0).sum(dim=1)
    s = E * (3 * d + 2 + depth)
    return s, s * (1 + 2 * d) + E * (3 * d2 + 4 * d)


class Out:
    def __init__(self, T, V, n, z):
        f = lambda *d: torch.full(d, 7.0, device="cuda")  # noqa: E731
        self.logp, self.entropy, self.lse = f(T), f(T), f(T, 2)
        self.ids, self.alt = torch.full((T, n), 7, dtype=torch.int32, device="cuda"), f(T, n)
        self.ws = moe.moe_token_logprobs_workspace(z, n)
        if self.ws is not None:
            self.ws.fill_(255)

    def all(self):
        return [self.logp, self.entropy, self.lse, self.ids, self.alt]


def check(z, targets, scale, n, o):
    logp, H, lse, ids, alt, lp = reference(z, targets, scale, n)
    V = z.shape[1]
    s, h = bounds(lp, V)
    # log p itself: three roundings of z - max, the logarithm's, the result's
    at = lambda v: s + E * (4 * torch.where(v > -INF, v.abs(), 0.0) + 8)  # noqa: E731

    def near(got, want, tol):
        got, fin = got.double(), torch.isfinite(want)
        assert torch.equal(got[~fin], want[~fin])
        off = (got - want).abs()[fin]
        tol = tol.expand_as(want)[fin]
        assert (off <= tol).all(), float((off / tol).max())

    near(o.logp, logp, at(logp))
    near(o.entropy, H, h + 4 * E * H)
    near(o.lse.double().sum(dim=1), lse, s + 2.0 ** -45 * torch.where(lse > -INF, lse.abs(), 0.0))
    near(o.lse[:, 0], lse, s + E * torch.where(lse > -INF, lse.abs(), 0.0) * 1.01)
    if n:
        assert torch.equal(o.ids, ids)
        near(o.alt, alt, (s[:, None] + E * (4 * torch.where(alt > -INF, alt.abs(), 0.0) + 16)))
    return logp, H, lp


def logits_of(g, T, V, banned=0.0, size=3.0):
    z = size * g.standard_normal((T, V))
    if banned:
        z[g.random((T, V)) < banned] = -np.inf
    return z


SHAPES = [(1, 1, 1), (1, 5, 5), (3, 7, 2), (2, 64, 32), (5, 100, 0), (4, 511, 20), (3, 2048, 32), (2, 2049, 1), (1, 2055, 8),
          (9, 4097, 32), (1, 65537, 20), (33, 8200, 5), (2, 131072, 32), (300, 333, 7), (2100, 3000, 3), (2050, 20, 20),
          (1, 600001, 32), (300, 10000, 0), (2, 32768, 3), (1, 32769, 3), (9, 40000, 32), (33, 33000, 5), (300, 40000, 0),
          (520, 40000, 4), (257, 65537, 4), (256, 65536, 2)]


@pytest.mark.parametrize("T,V,n", SHAPES)
@pytest.mark.parametrize("zt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("banned,scale", [(0.0, 1.0), (0.6, 1.3)])
def test_token_logprobs(T, V, n, zt, banned, scale):
    g = rng_of(41, T, V)
    pad, lead = (0, 0) if (T + V) % 2 else (3, 1)
    z, zf = rows(logits_of(g, T, V, banned), TYPES[zt], pad, lead)
    targets = torch.from_numpy(g.integers(0, V, T)).int().cuda()
    targets[:: 7] = torch.tensor(-100 if T % 2 else V, dtype=torch.int32)
    o = Out(T, V, n, z)
    before = zf.clone()
    kw = dict(targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, scale=scale, workspace=o.ws)
    top = dict(top_ids=o.ids, top_logp=o.alt) if n else {}
    moe.moe_token_logprobs(z, **kw, **top)
    check(z, targets, float(np.float32(scale)), n, o)
    assert torch.equal(zf, before)
    first = [t.clone() for t in o.all()]
    moe.moe_token_logprobs(z, **kw, **top)
    assert all(torch.equal(a, b) for a, b in zip(first, o.all()))  # equal calls, equal bits
    # one output at a time
    e = torch.full((T,), 7.0, device="cuda")
    moe.moe_token_logprobs(z, entropy=e, scale=scale)
    assert torch.equal(e, first[1])
    if n:
        o.ids.fill_(7)
        moe.moe_token_logprobs(z, top_ids=o.ids, top_logp=o.alt, scale=scale, workspace=o.ws)
        assert torch.equal(o.ids, first[3]) and torch.equal(o.alt, first[4])


@pytest.mark.parametrize("T,V", [(1, 40), (3, 1500), (2, 5000), (1, 65537), (2100, 2500), (2, 300000)])
@pytest.mark.parametrize("kind", ["equal", "lowest", "few", "two values", "rising", "falling", "one run", "nothing"])
def test_alternatives_of_unusual_rows(T, V, kind):
    """Ties, masks of the type's lowest value, fewer words than alternatives, sorted rows: more values may reach the bound
    than there is room for."""
    g = rng_of(42, T, V)
    n = 32
    low = torch.finfo(torch.float32).min
    z = torch.from_numpy(logits_of(g, T, V)).float()
    if kind == "equal":
        z[:] = 1.5
    elif kind == "lowest":
        z[torch.from_numpy(g.random((T, V)) > 10 / V)] = low
    elif kind == "few":
        z[torch.from_numpy(g.random((T, V)) > 10 / V)] = -INF
        z[0] = -INF
        z[0, V // 2] = 0.25
    elif kind == "two values":
        z = torch.from_numpy(g.integers(0, 2, (T, V))).float()
    elif kind == "rising":
        z = (torch.arange(V).float() / V * 20).expand(T, V).contiguous()
    elif kind == "falling":
        z = (-torch.arange(V).float() / V * 20).expand(T, V).contiguous()
    elif kind == "one run":
        z[:] = -3.0
        z[:, V // 3:V // 3 + 40] = torch.arange(min(40, V - V // 3)).float()
    elif kind == "nothing":
        z[:] = -INF
    z = z.cuda()
    targets = torch.zeros(T, dtype=torch.int32, device="cuda")
    o = Out(T, V, n, z)
    moe.moe_token_logprobs(z, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, top_ids=o.ids, top_logp=o.alt, workspace=o.ws)
    check(z, targets, 1.0, n, o)


@pytest.mark.parametrize("V", [30, 3000, 65537])
def test_values_that_are_not_finite_stay_in_their_row(V):
    g = rng_of(43, V)
    T, n = 6, 4
    z = torch.from_numpy(logits_of(g, T, V)).float().cuda()
    z[1, V // 2], z[2, V - 1], z[3, 0], z[4] = float("nan"), INF, -float("nan"), -INF
    targets = torch.full((T,), 3, dtype=torch.int32, device="cuda")
    targets[2] = -1
    o = Out(T, V, n, z)
    moe.moe_token_logprobs(z, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, top_ids=o.ids, top_logp=o.alt, workspace=o.ws)
    for t in (1, 2, 3):
        assert torch.isnan(o.entropy[t]) and torch.isnan(o.lse[t, 0]) and torch.isnan(o.alt[t]).all() and (o.ids[t] == -1).all()
        assert torch.isnan(o.logp[t]) if t != 2 else o.logp[t] == 0
    assert o.entropy[4] == 0 and o.lse[4, 0] == -INF and o.logp[4] == -INF and (o.ids[4] == -1).all() and (o.alt[4] == -INF).all()
    good = torch.tensor([0, 5], device="cuda")
    for name in ("logp", "entropy", "lse", "ids", "alt"):
        setattr(o, name, getattr(o, name)[good])
    check(z[good], targets[good], 1.0, n, o)
    d = torch.full_like(z, 7.0)
    one = torch.ones(T, device="cuda")
    H = torch.zeros(T, device="cuda")
    lse = torch.zeros((T, 2), device="cuda")
    moe.moe_token_logprobs(z, entropy=H, lse=lse)
    moe.moe_token_logprobs_grad(z, lse, d, targets=targets, dlogp=one)
    assert torch.isnan(d[1]).all() and (d[4] == 0).all() and (d[2] == 0).all() and torch.isfinite(d[good]).all()
    # nothing asked of a row: zeros whatever its logits
    moe.moe_token_logprobs_grad(z, lse, d, targets=targets, dlogp=0 * one, entropy=H, dentropy=0 * one)
    assert (d == 0).all()


@pytest.mark.parametrize("scale", [1e-3, 1.0, 50.0])
def test_logits_far_from_zero(scale):
    """A common offset of the logits changes nothing but lse, whose two floats carry the gradient."""
    g = rng_of(44)
    z = torch.from_numpy(np.round(logits_of(g, 4, 3000) * 16) / 16).float().cuda()
    far = z + 4096.0  # exact
    targets = torch.tensor([0, 5, 2999, 100], dtype=torch.int32, device="cuda")
    a, b = Out(4, 3000, 8, z), Out(4, 3000, 8, z)
    one = torch.ones(4, device="cuda")
    ds = []
    for x, o in ((z, a), (far, b)):
        moe.moe_token_logprobs(x, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, top_ids=o.ids, top_logp=o.alt, scale=scale,
                               workspace=o.ws)
        check(x, targets, float(np.float32(scale)), 8, o)
        ds.append(torch.empty_like(z))
        moe.moe_token_logprobs_grad(x, o.lse, ds[-1], targets=targets, dlogp=one, scale=scale)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.logp, b.logp) and torch.equal(a.entropy, b.entropy)
    lp = torch.log_softmax(z.double() * float(np.float32(scale)), dim=1)
    # z's rounding stays out: fma(x, scale, -lse) rounds the difference alone
    assert ((ds[0] - ds[1]).abs() <= scale * lp.exp() * (8 + 4 * lp.abs()) * E + scale * 2 * E).all()


@pytest.mark.parametrize("power", [64, -64])
@pytest.mark.parametrize("T,V", [(3, 900), (2, 30000)])
def test_scales_at_their_limits(power, T, V):
    """Powers of two: exact, so logits times 2^-power say the same with a scale of 2^power."""
    g = rng_of(49, V)
    z = torch.from_numpy(logits_of(g, T, V)).float().cuda()
    far = z * 2.0 ** -power
    targets = torch.zeros(T, dtype=torch.int32, device="cuda")
    outs = []
    for x, scale in ((z, 1.0), (far, 2.0 ** power)):
        o = Out(T, V, 9, z)
        moe.moe_token_logprobs(x, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, top_ids=o.ids, top_logp=o.alt, scale=scale)
        d = torch.empty_like(z)
        moe.moe_token_logprobs_grad(x, o.lse, d, targets=targets, dlogp=o.logp, entropy=o.entropy, dentropy=o.logp, scale=scale)
        outs.append(o.all() + [d / scale])
    assert all(torch.equal(a, b) for a, b in zip(*outs))


# ---------------------------------------------------------------------------
# gradient


@pytest.mark.parametrize("T,V", [(1, 1), (1, 5), (3, 7), (5, 100), (4, 511), (3, 2048), (2, 2049), (9, 4097), (1, 65537), (300, 333),
                                 (2100, 300), (2, 131072)])
@pytest.mark.parametrize("zt,dt", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("parts,banned,scale", [("both", 0.0, 1.0), ("logp", 0.5, 0.7), ("entropy", 0.5, 1.0)])
def test_token_logprobs_grad(T, V, zt, dt, parts, banned, scale):
    g = rng_of(45, T, V)
    pad, lead = (0, 0) if (T + V) % 2 else (3, 1)
    z, zf = rows(logits_of(g, T, V, banned), TYPES[zt], pad, lead)
    z[:, 0] = 0.5  # at least one word
    targets = torch.from_numpy(g.integers(0, V, T)).int().cuda()
    targets[::5] = -1
    lse, H = torch.empty((T, 2), device="cuda"), torch.empty(T, device="cuda")
    moe.moe_token_logprobs(z, entropy=H, lse=lse, scale=scale)
    a = torch.from_numpy(g.standard_normal(T)).float().cuda()
    b = torch.from_numpy(g.standard_normal(T)).float().cuda()
    kw = dict(targets=targets, scale=scale)
    if parts != "entropy":
        kw.update(dlogp=a)
    if parts != "logp":
        kw.update(entropy=H, dentropy=b)
    d, df = rows(np.full((T, V), 3.0), TYPES[dt], pad, lead)
    before = zf.clone()
    moe.moe_token_logprobs_grad(z, lse, d, **kw)
    assert untouched(df, T, V, pad, lead) and torch.equal(zf, before)
    sc = float(np.float32(scale))
    _, H64, _, _, _, lp = reference(z, targets, sc, 0)
    p = lp.exp()
    a64 = torch.where(targets >= 0, a, 0.0).double()[:, None] if parts != "entropy" else 0.0 * a.double()[:, None]
    b64 = b.double()[:, None] if parts != "logp" else 0.0 * b.double()[:, None]
    lpf = torch.where(p > 0, lp, 0.0)
    want = -p * (a64 + b64 * (lpf + H64[:, None]))
    delta = torch.zeros_like(p).scatter_(1, targets.long().clamp(min=0)[:, None], 1.0)
    want = sc * (want + delta * a64)
    # p: the errors of lse, of z - lse (two roundings) and of its power; then of the sums and products around it
    s, h = bounds(lp, V)
    mag = p * (a64.abs() + b64.abs() * (lpf.abs() + H64[:, None]))
    tol = mag * (s[:, None] + E * (3 * lpf.abs() + 12)) + p * b64.abs() * (s + h + 4 * E * H64)[:, None] + 3 * E * (delta * a64).abs()
    tol = (sc * tol + u(TYPES[dt]) * want.abs()) * 1.01 + smallest(TYPES[dt])
    off = (d.double() - want).abs()
    assert (off <= tol).all(), float((off / tol).max())
    first = d.clone()
    # added to what is there: one more rounding
    d.fill_(1.0)
    moe.moe_token_logprobs_grad(z, lse, d, flags=moe.MOE_ACCUMULATE, **kw)
    assert ((d.double() - (want + 1.0)).abs() <= tol + (u(TYPES[dt]) + E) * 1.01 * ((want + 1.0).abs() + tol)).all()
    if zt == dt:  # in place
        moe.moe_token_logprobs_grad(z, lse, z, **kw)
        assert torch.equal(z, first)


@pytest.mark.parametrize("T,V,zt,dt", [(520, 65537, "bf16", "bf16"), (270, 65537, "f32", "f32"), (40, 500000, "f16", "f32")])
def test_gradient_larger_than_the_caches(T, V, zt, dt):
    """64 MB and more of dlogits, rows that begin anywhere: against the formula row by row, into its own memory, onto
    what is there, and in place."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    z = (3 * torch.randn((T, V), generator=g, device="cuda")).to(TYPES[zt])
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    targets[:3] = torch.tensor([0, V - 1, -1], dtype=torch.int32)
    a, b = torch.randn(T, generator=g, device="cuda"), torch.randn(T, generator=g, device="cuda")
    H, lse = torch.empty(T, device="cuda"), torch.empty((T, 2), device="cuda")
    moe.moe_token_logprobs(z, entropy=H, lse=lse)
    d = torch.full((T, V + 1), 7.0, dtype=TYPES[dt], device="cuda")[:, :V]
    kw = dict(targets=targets, dlogp=a, entropy=H, dentropy=b)
    moe.moe_token_logprobs_grad(z, lse, d, **kw)
    more = torch.ones((T, V), dtype=TYPES[dt], device="cuda")
    moe.moe_token_logprobs_grad(z, lse, more, flags=moe.MOE_ACCUMULATE, **kw)
    for t in range(0, T, 37):
        lp = torch.log_softmax(z[t].double(), dim=0)
        p, h = lp.exp(), -(lp.exp() * lp).sum()
        at = a[t].double() if targets[t] >= 0 else torch.zeros((), dtype=torch.float64, device="cuda")
        want = -p * (at + b[t].double() * (lp + h))
        if targets[t] >= 0:
            want[targets[t]] += at
        s, hb = bounds(lp[None], V)
        mag = p * (at.abs() + b[t].double().abs() * (lp.abs() + h))
        tol = mag * (s + E * (3 * lp.abs() + 12)) + p * b[t].double().abs() * (s + hb + 4 * E * h) + 3 * E * at.abs() * (want.abs() > 0)
        tol = (tol + u(TYPES[dt]) * want.abs()) * 1.01 + smallest(TYPES[dt])
        assert ((d[t].double() - want).abs() <= tol).all()
        assert ((more[t].double() - (want + 1)).abs() <= tol + (u(TYPES[dt]) + E) * 1.01 * ((want + 1).abs() + tol)).all()
    assert (d.as_strided((T,), (V + 1,), V) == 7).all()
    if zt == dt:
        moe.moe_token_logprobs_grad(z, lse, z, **kw)
        assert torch.equal(z, d)


def test_gradient_against_differences():
    """Central differences of the forward call, step 2^-6: h^2 / 6 times third derivatives below 1, roundings over the step."""
    g = rng_of(46)
    T, V = 4, 50
    z = torch.from_numpy(logits_of(g, T, V, size=1.0)).float().cuda()
    targets = torch.tensor([3, 49, -1, 0], dtype=torch.int32, device="cuda")
    a, b = torch.from_numpy(g.standard_normal(T)).float().cuda(), torch.from_numpy(g.standard_normal(T)).float().cuda()
    logp, H, lse, d = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty((T, 2), device="cuda"), torch.empty_like(z)

    def loss(z):
        moe.moe_token_logprobs(z, targets=targets, logp=logp, entropy=H, lse=lse, scale=0.8)
        return (a.double() * logp.double() + b.double() * H.double()).sum()

    loss(z)
    moe.moe_token_logprobs_grad(z, lse, d, targets=targets, dlogp=a, entropy=H.clone(), dentropy=b, scale=0.8)
    h = 2.0 ** -6
    size = float((a.abs() + b.abs()).sum())
    for _ in range(8):
        v = torch.from_numpy(g.standard_normal((T, V))).float().cuda()
        v /= v.abs().max()
        diff = (loss(z + h * v) - loss(z - h * v)) / (2 * h)
        assert abs(diff - (d.double() * v.double()).sum()) <= size * (h * h + 100 * E / h)


def test_more_rows_than_work_groups():
    T, V = (1 << 22) + 3, 3  # the sums' grid ends at 2^20, the gradient's at 2^22
    g = torch.Generator(device="cuda")
    g.manual_seed(52)
    z = torch.randn((T, V), generator=g, device="cuda")
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    logp, H, lse = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros((T, 2), device="cuda")
    ids, alt = torch.full((T, 2), 9, dtype=torch.int32, device="cuda"), torch.zeros((T, 2), device="cuda")
    moe.moe_token_logprobs(z, targets=targets, logp=logp, entropy=H, lse=lse, top_ids=ids, top_logp=alt)
    lp = torch.log_softmax(z.double(), dim=1)
    # three values: their powers' roundings (5 E of a result below 8 each) and those of the sums and logarithms
    tol = 60 * E
    assert (logp - lp.gather(1, targets.long()[:, None]).squeeze(1)).abs().max() <= tol
    assert (H + (lp.exp() * lp).sum(dim=1)).abs().max() <= tol
    assert torch.equal(ids.long(), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :2])
    assert (alt - lp.gather(1, ids.long())).abs().max() <= tol
    d = torch.full_like(z, 7.0)
    moe.moe_token_logprobs_grad(z, lse, d, targets=targets, dlogp=torch.ones(T, device="cuda"))
    want = torch.zeros_like(lp).scatter_(1, targets.long()[:, None], 1.0) - lp.exp()
    assert (d - want).abs().max() <= tol


def test_of_no_tokens():
    z = torch.zeros((0, 500), device="cuda")
    e = torch.zeros(0, device="cuda")
    moe.moe_token_logprobs(z, entropy=e)
    moe.moe_token_logprobs_grad(z, torch.zeros((0, 2), device="cuda"), z.clone(), targets=torch.zeros(0, dtype=torch.int32, device="cuda"),
                                dlogp=e)


@pytest.mark.parametrize("T,V", [(2, 20000), (2, 40000), (5, 700), (2100, 2500)])
def test_captured_two_at_once_and_on_another_stream(T, V):
    g = rng_of(47, T)
    zs = [torch.from_numpy(logits_of(g, T, V)).bfloat16().cuda() for _ in range(2)]
    targets = torch.from_numpy(g.integers(0, V, T)).int().cuda()
    a = torch.ones(T, device="cuda")
    os_ = [Out(T, V, 6, zs[0]) for _ in range(2)]
    ds = [torch.empty_like(z) for z in zs]

    def step(i, stream=None):
        z, o = zs[i], os_[i]
        moe.moe_token_logprobs(z, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, top_ids=o.ids, top_logp=o.alt,
                               workspace=o.ws if o.ws is not None else torch.empty(0, dtype=torch.uint8, device="cuda"), stream=stream)
        moe.moe_token_logprobs_grad(z, o.lse, ds[i], targets=targets, dlogp=a, entropy=o.entropy, dentropy=a, stream=stream)

    step(0), step(1)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=side):
            step(i)
    for r in range(3):
        for z in zs:
            z.copy_(torch.from_numpy(logits_of(rng_of(48, r, T), T, V)).bfloat16())
            zs[1].neg_()
        want = []
        for i in range(2):
            step(i)
            want.append([t.clone() for t in os_[i].all() + [ds[i]]])
            check(zs[i], targets, 1.0, 6, os_[i])
        torch.cuda.synchronize()
        for i in range(2):
            for t in os_[i].all() + [ds[i]]:
                t.zero_()
        with torch.cuda.stream(side):
            graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(x, y) for x, y in zip(os_[i].all() + [ds[i]], want[i]))
            for t in os_[i].all() + [ds[i]]:
                t.zero_()
        torch.cuda.synchronize()
        step(0, side), step(1, other)
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(x, y) for x, y in zip(os_[i].all() + [ds[i]], want[i]))


def test_binding_refusals():
    z = torch.zeros((3, 50000), device="cuda")
    y, f = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, device="cuda")
    lse = torch.zeros((3, 2), device="cuda")
    for bad in (dict(targets=y.long(), logp=f), dict(targets=y[:2], logp=f), dict(entropy=f.half()), dict(lse=f),
                dict(top_ids=torch.zeros((3, 2), dtype=torch.int32, device="cuda")), dict(entropy=f.cpu()),
                dict(entropy=f, stream=torch.cuda.Stream())):
        with pytest.raises(ValueError):
            moe.moe_token_logprobs(z, **bad)
    for bad in (dict(targets=y), dict(logp=f), dict(), dict(entropy=f, scale=0.0), dict(entropy=f, scale=-1.0), dict(entropy=f, scale=INF),
                dict(entropy=f, scale=float("nan")), dict(entropy=f, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(moe.MoeError):
            moe.moe_token_logprobs(z, **bad)
    with pytest.raises((ValueError, moe.MoeError)):
        moe.moe_token_logprobs(z, top_ids=torch.zeros((3, 33), dtype=torch.int32, device="cuda"), top_logp=torch.zeros((3, 33), device="cuda"))
    d = torch.zeros_like(z)
    for bad in (dict(), dict(dlogp=f), dict(dentropy=f), dict(targets=y, dlogp=f, flags=2), dict(targets=y, dlogp=f, scale=0.0)):
        with pytest.raises(moe.MoeError):
            moe.moe_token_logprobs_grad(z, lse, d, **bad)
    with pytest.raises(moe.MoeError, match="in place"):
        moe.moe_token_logprobs_grad(z, lse, z, targets=y, dlogp=f, flags=moe.MOE_ACCUMULATE)
    with pytest.raises(ValueError):
        moe.moe_token_logprobs_grad(z, None, d[:2], targets=y, dlogp=f)

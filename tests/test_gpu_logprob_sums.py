"""Sums behind the log probabilities on the GPU: rows of one confident word, whose log probability is the
mass of all the others together.

Tolerances count roundings: E = 2^-24 of a result per fp32 operation. They do not grow with the row.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
from tests.test_gpu_dense_ops import TYPES, E, rng_of  # noqa: E402
from tests.test_gpu_logprobs import INF, Out, check  # noqa: E402

pytestmark = pytest.mark.gpu

# Every word but one is 16, 17 or 18 below it (exact in every type). Of a word's power, relative to it: the argument, at most 18
# nats in all however it is reached over rising maxima, with a rounding of its product with log2 e and 0.3 for that
# constant, 1.3 * 18; the power 2; its sum with the 15 beside it 8; rising maxima, two of a thread, then lanes, waves, slices,
# each with a power of 2 and a product, 5 * 3.
WORD = 1.3 * 18 + 2 + 8 + 15
# Beside the confident word, which is 1: the 15 words added to it in fp32, 8 roundings of 1 and a bit.
PEAK = 8.1


# uncut rows by one wave and by four; cut; many rows, uncut; long, cut and uncut (from 384 rows on nothing is)
@pytest.mark.parametrize("T,V", [(3, 2000), (3, 32768), (2, 65537), (260, 65536), (1, 1 << 22), (520, 1 << 20)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("zt", ["f32", "bf16"])
def test_one_confident_word(T, V, where, zt):
    g = rng_of(61, T, V)
    at = {"first": 0, "middle": V // 2 + 1, "last": V - 1}[where]
    rest = torch.from_numpy(g.integers(-18, -15, V)).to(TYPES[zt]).cuda()
    rest[at] = 0
    z = torch.empty((T, V), dtype=TYPES[zt], device="cuda")
    z[:] = rest
    targets = torch.full((T,), at, dtype=torch.int32, device="cuda")
    targets[1:] = (at + 5) % V
    n = 2
    o = Out(T, V, n, z)
    kw = dict(targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, workspace=o.ws)
    moe.moe_token_logprobs(z, **kw, **({"top_ids": o.ids, "top_logp": o.alt} if T < 100 else {}))
    x = rest.double().cpu().numpy()
    p = np.exp(x)
    others = p.sum() - 1.0  # beside 1: 53 bits are plenty for what is asked below
    log_s = np.log1p(others)
    s = PEAK * E + others * WORD * E
    assert abs(float(o.logp[0]) + log_s) <= s + 1.01 * E * log_s
    assert abs(o.lse.double().sum(dim=1).cpu().numpy() - log_s).max() <= s
    H = float(log_s - (p * x).sum() / p.sum())
    assert abs(o.entropy.double().cpu().numpy() - H).max() <= s + (WORD + 12) * E * H
    if T > 1:
        far = float(x[(at + 5) % V]) - log_s
        assert abs(o.logp[1:].double().cpu().numpy() - far).max() <= s + 1.01 * E * abs(far)
    if T < 100:
        assert (o.ids[:, 0] == at).all() and abs(o.alt[:, 0].double().cpu().numpy() + log_s).max() <= s + 3 * E * log_s
    if T * V > 1 << 26:
        return
    # 1 - p of the confident word, and a gradient that sums to nothing: each p has its own power's roundings besides
    d = torch.empty((T, V), dtype=torch.float32, device="cuda")
    moe.moe_token_logprobs_grad(z, o.lse, d, targets=torch.full_like(targets, at), dlogp=torch.ones(T, device="cuda"))
    d = d.double().cpu().numpy()
    assert abs(d[:, at] - others / (1 + others)).max() <= s + 4 * E
    assert abs(d.sum(axis=1)).max() <= s + 4 * E + others * (3.3 * 18 + 4) * E


@pytest.mark.parametrize("V", [5, 3000, 65537])
@pytest.mark.parametrize("scale", [0.5, 2.0 ** -64])
def test_alternatives_far_below_the_best(V, scale):
    """The difference of two fp32 logits may pass fp32's range where scale times it does not."""
    z = torch.full((2, V), -3e38, device="cuda")
    z[:, 1], z[1, 2] = 3e38, 2.9e38
    n = 4
    targets = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    o = Out(2, V, n, z)
    moe.moe_token_logprobs(z, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, top_ids=o.ids, top_logp=o.alt, scale=scale,
                           workspace=o.ws)
    lp = scale * (z.double() - 3e38)
    lp = lp - torch.logsumexp(lp, dim=1, keepdim=True)
    assert (o.ids == torch.tensor([[1, 0, 2, 3], [1, 2, 0, 3]], device="cuda")).all()
    want = lp.gather(1, o.ids.long())
    # the float nearest 3e38 is within E of it, the difference and the product are rounded
    assert ((o.alt.double() - want).abs() <= 4 * E * want.abs() + 1e-6).all()
    assert ((o.logp.double() - lp[:, 3]).abs() <= 3 * E * lp[:, 3].abs() + 1e-6).all()


def test_a_row_that_is_not_cut_needs_no_workspace():
    """The workspace of fewer rows serves more of them, and more that are not cut use none: nothing to allocate on a stream of
    the caller's own."""
    side = torch.cuda.Stream()
    for T, V in ((300, 40000), (600, 70000)):
        assert moe.moe_token_logprobs_workspace_bytes(T, V, 3) > 0
        z = torch.randn((T, V), device="cuda")
        want, got = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_token_logprobs(z, entropy=want, workspace=moe.moe_token_logprobs_workspace(z))
        side.wait_stream(torch.cuda.current_stream())
        moe.moe_token_logprobs(z, entropy=got, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        moe.moe_token_logprobs(z, entropy=got.zero_())
        assert torch.equal(got, want)
    with pytest.raises(ValueError, match="workspace"):
        moe.moe_token_logprobs(z[:5], entropy=got[:5].clone(), stream=side)


@pytest.mark.parametrize("T,n,V", [(1, 0, 33068), (2, 32, 33368), (60, 9, 50768), (255, 0, 109268), (256, 2, 109568), (383, 0, 147668),
                                   (384, 1, 147968)])
def test_rows_about_as_long_as_are_not_cut(T, n, V):
    """One logit more is another form of the same row, to its roundings; so is a workspace of more rows and alternatives."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T + V)
    ws = torch.full((moe.moe_token_logprobs_workspace_bytes(400, V + 1, 32),), 255, dtype=torch.uint8, device="cuda")
    assert len(ws) >= moe.moe_token_logprobs_workspace_bytes(T, V + 1, n)
    whole = (3 * torch.randn((T, V + 1), generator=g, device="cuda")).bfloat16()
    whole[:, V] = -INF  # the word more
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    outs = []
    for z in (whole[:, :V], whole):
        o = Out(T, z.shape[1], n, z)
        moe.moe_token_logprobs(z, targets=targets, logp=o.logp, entropy=o.entropy, lse=o.lse, workspace=ws,
                               **({"top_ids": o.ids, "top_logp": o.alt} if n else {}))
        check(z[:8], targets[:8], 1.0, n, _first(o, 8))
        outs.append(o)
    assert torch.equal(outs[0].ids, outs[1].ids)
    assert (outs[0].lse.double().sum(dim=1) - outs[1].lse.double().sum(dim=1)).abs().max() <= 2 * (1.3 * 18 + 2 + 8 + 3 * 24) * E


def _first(o, rows):
    f = Out.__new__(Out)
    f.logp, f.entropy, f.lse, f.ids, f.alt = (t[:rows] for t in o.all())
    return f


@pytest.mark.parametrize("T,V,step", [(1, 131072, 2048), (4, 70000, 2048), (3, 20000, 20000)])
def test_many_candidates_close_together(T, V, step):
    """More than 256 values within the 16 bits of a bound, distinct, in every other slice (or anywhere in a row that is not cut)."""
    g = rng_of(62, T, V)
    n = 32
    z = torch.from_numpy(g.standard_normal((T, V)) - 5).float().cuda()
    for t in range(T):
        for at in range(0, V - step + 1, 2 * step):
            many = 32 if step < V else 700
            z[t, at + torch.from_numpy(g.permutation(step)[:many]).cuda()] = torch.from_numpy(10 + 0.06 * g.random(many)).float().cuda()
    o = Out(T, V, n, z)
    moe.moe_token_logprobs(z, top_ids=o.ids, top_logp=o.alt, workspace=o.ws)
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :n]
    assert torch.equal(o.ids.long(), ids)
    lp = torch.log_softmax(z.double(), dim=1).gather(1, ids)
    # the best lie within 0.06 of each other: their own differences are nearly exact, the sum's roundings as in any row
    assert ((o.alt.double() - lp).abs() <= 100 * E).all()

"""The operators around attention and behind the output head together, as a layer of a model uses them: prompt and decode
steps through norm, fused query/key/value product, head norms and rotation, attention (torch, fp64), output projection, routed and
shared experts, and the head's log probabilities; and their limits: offsets past 32 bits, calls at once."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import moe_expert_offload_gemv_amd as moe  # noqa: E402
import oracle  # noqa: E402
from tests._gpu import TOL, Decode, token_rel_err  # noqa: E402
from tests.test_gpu_dense_limits import big_memory, far_rows  # noqa: E402,F401
from tests.test_gpu_dense_ops import Product, norm_ref, rng_of  # noqa: E402
from tests.test_gpu_heads import Rope, normed, turned  # noqa: E402
from workload import Workload  # noqa: E402

pytestmark = pytest.mark.gpu


def dense_of(p):
    """The weights of a product in fp64."""
    return ((torch.cat([p.nib & 15, p.nib >> 4], dim=2).double() - 8) * p.scl.double()[..., None]).flatten(1)


def attention(q, k, v, first):
    """Causal attention of queries at positions first .. over all keys, heads in groups; fp64 on the CPU."""
    q, k, v = (t.cpu().double() for t in (q, k, v))
    T, H, D = q.shape
    group = H // k.shape[1]
    k, v = k.repeat_interleave(group, dim=1).transpose(0, 1), v.repeat_interleave(group, dim=1).transpose(0, 1)
    z = torch.matmul(q.transpose(0, 1), k.transpose(1, 2).contiguous()) / D ** 0.5
    z = z.masked_fill(torch.arange(k.shape[1]) > torch.arange(T)[:, None] + first, -torch.inf)
    return torch.matmul(torch.softmax(z, dim=2), v).transpose(0, 1).reshape(T, H * D)


def test_prompt_and_decode_through_a_layer_and_the_head():
    wl = Workload("decode-e64k8-h256f512-t5-attention", 323, 1, 64, 8, 256, 512, tokens=5, steps=3, zipf_s=1.1, slots=24)
    H, Hq, Hk, D, F, V = 256, 8, 2, 32, 512, 4099
    d = Decode(wl)
    try:
        g = rng_of(61)
        make = lambda n, k, seed: Product(1, n, k, "f32", seed=seed)  # noqa: E731
        qkv, proj, router, up, gate, down, head = (make(n, k, i) for i, (n, k) in enumerate(
            [((Hq + 2 * Hk) * D, H), (H, Hq * D), (64, H), (F, H), (F, H), (H, F), (V, H)]))
        for p in (proj, down):
            p.scl.mul_(0.25)
        W = [dense_of(p).cpu() for p in (qkv, proj, router, up, gate, down, head)]
        bias = torch.from_numpy(0.1 * g.standard_normal((Hq + 2 * Hk) * D)).float().cuda()
        w1, w2, qw, kw = (torch.from_numpy(1 + 0.1 * g.standard_normal(n)).float().cuda() for n in (H, H, D, D))
        inv = torch.from_numpy(10000.0 ** (-np.arange(0, D, 2) / D)).float().cuda()
        cache_k, cache_v = torch.zeros((64, Hk, D), device="cuda"), torch.zeros((64, Hk, D), device="cuda")
        at = 0
        for T in (5, 1, 3):  # a prompt, one token, a speculative check
            x0 = torch.from_numpy(g.standard_normal((T, H))).float().cuda()
            stream, xn = x0.clone(), torch.empty((T, H), device="cuda")
            fused = torch.empty((T, (Hq + 2 * Hk) * D), device="cuda")
            q = fused[:, :Hq * D].unflatten(1, (Hq, D))
            k = fused[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
            pos = torch.arange(at, at + T, device="cuda", dtype=torch.int32)
            moe.moe_add_rmsnorm(stream, w1, xn, eps=1e-6)
            moe.moe_q4_linear(xn, qkv.nib, qkv.scl, fused, bias=bias)
            # queries in place, keys into the cache
            moe.moe_qk_norm_rope(q, k, q, cache_k[at:at + T], q_weight=qw, k_weight=kw, inv_freq=inv, positions=pos)
            cache_v[at:at + T] = fused[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
            o = attention(q, cache_k[:at + T], cache_v[:at + T], at).float().cuda()
            moe.moe_q4_linear(o, proj.nib, proj.scl, stream, residual=stream)
            moe.moe_add_rmsnorm(stream, w2, xn, eps=1e-6)
            logits, ids = torch.empty((T, 64), device="cuda"), torch.empty((T, 8), dtype=torch.int32, device="cuda")
            moe.moe_q4_matmul(xn, router.nib, router.scl, logits)
            y, u, h = torch.empty((T, H), device="cuda"), torch.empty((T, F), device="cuda"), torch.empty((T, F), device="cuda")
            moe.moe_forward(d.ctx, 0, T, xn, logits, y, ids)
            moe.moe_q4_matmul(xn, up.nib, up.scl, u)
            moe.moe_q4_linear(xn, gate.nib, gate.scl, h, act=moe.MOE_ACT_SILU, mul=u)
            moe.moe_q4_linear(h, down.nib, down.scl, y, residual=y)
            words = torch.empty((T, V), device="cuda")
            moe.moe_q4_linear(y, head.nib, head.scl, words)
            targets = torch.from_numpy(g.integers(0, V, T)).int().cuda()
            logp, entropy = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
            top, alt = torch.empty((T, 5), dtype=torch.int32, device="cuda"), torch.empty((T, 5), device="cuda")
            moe.moe_token_logprobs(words, targets=targets, logp=logp, entropy=entropy, top_ids=top, top_logp=alt)
            moe.moe_cache_step(d.ctx)

            # the same in fp64, step by step from what the step before gave
            x = x0.cpu().double()
            _, v1 = norm_ref(x, None, w1.cpu(), 1e-6)
            f = v1 @ W[0].t() + bias.cpu().double()
            angle = (pos.cpu().double()[:, None] * inv.cpu().double())
            part = lambda a, b: f[:, a * D:b * D].unflatten(1, (b - a, D))  # noqa: E731
            qr = turned(normed(part(0, Hq), qw.cpu().double())[0], angle, D, False)
            kr = turned(normed(part(Hq, Hq + Hk), kw.cpu().double())[0], angle, D, False)
            near = lambda a, b, tol=2e-5: torch.linalg.norm(a.cpu().double() - b) <= tol * torch.linalg.norm(b)  # noqa: E731
            assert near(q, qr) and near(cache_k[at:at + T], kr) and near(cache_v[at:at + T], part(Hq + Hk, Hq + 2 * Hk))
            s64 = x + o.cpu().double() @ W[1].t()
            assert near(stream, s64)
            _, v2 = norm_ref(s64, None, w2.cpu(), 1e-6)
            assert near(logits, v2 @ W[2].t())
            ref, ids_ref, _ = oracle.moe_layer(64, 8, H, wl.ffn, d.experts(0, ids.cpu().numpy()), v2.numpy(), logits=logits.cpu().numpy())
            assert np.array_equal(ids.cpu().numpy(), ids_ref)
            a = v2 @ W[4].t()
            ref = ref + ((a * torch.sigmoid(a) * (v2 @ W[3].t())) @ W[5].t()).numpy()
            assert token_rel_err(y.cpu().numpy(), ref) < TOL
            assert near(words, y.cpu().double() @ W[6].t())
            lp = torch.log_softmax(words.cpu().double(), dim=1)
            assert (logp.cpu() - lp[torch.arange(T), targets.cpu().long()]).abs().max() <= 1e-5 * lp.abs().max()
            assert (entropy.cpu() + (lp.exp() * lp).sum(dim=1)).abs().max() <= 1e-5
            assert torch.equal(top.cpu().long(), torch.sort(words.cpu(), dim=1, descending=True, stable=True).indices[:, :5])
            assert (alt.cpu() - lp.gather(1, top.cpu().long())).abs().max() <= 1e-5 * lp.abs().max()
            at += T
    finally:
        d.close()


def test_training_step_of_heads_and_loss():
    """Cross entropy of a linear map of normed, turned queries: the gradients chained by hand against autograd in fp64."""
    T, Hq, D, V = 70, 4, 32, 333
    g = rng_of(62)
    rope = Rope(T, D, D, g=g, far=1 << 12)
    x = torch.from_numpy(g.standard_normal((T, Hq, D))).float().cuda()
    w = torch.from_numpy(1 + 0.1 * g.standard_normal(D)).float().cuda()
    M = torch.from_numpy(g.standard_normal((V, Hq * D)) / 8).float().cuda()
    targets = torch.from_numpy(g.integers(0, V, T)).int().cuda()
    targets[::9] = -100
    n = int((targets >= 0).sum())
    q, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    logp, entropy, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty((T, 2), device="cuda")
    moe.moe_qk_norm_rope(x, None, q, None, q_weight=w, **rope.kw)
    z = q.flatten(1) @ M.t()
    moe.moe_token_logprobs(z, targets=targets, logp=logp, entropy=entropy, lse=lse)
    loss = -logp.sum() / n - 0.01 * entropy.mean()
    dlogp, dent = torch.full((T,), -1.0 / n, device="cuda"), torch.full((T,), -0.01 / T, device="cuda")
    moe.moe_token_logprobs_grad(z, lse, z, targets=targets, dlogp=dlogp, entropy=entropy, dentropy=dent)  # in the logits' place
    gq = (z @ M).unflatten(1, (Hq, D))
    moe.moe_qk_norm_rope_grad(x, None, gq, None, dx, None, q_weight=w, dq_weight=dw, **rope.kw)

    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    v = x64 / torch.sqrt(x64.square().mean(dim=2, keepdim=True) + 1e-6) * w64
    a, b = v[..., :D // 2], v[..., D // 2:]
    c, s = rope.angle.cos()[:, None], rope.angle.sin()[:, None]
    z64 = torch.cat([a * c - b * s, b * c + a * s], dim=2).flatten(1) @ M.double().t()
    lp = torch.log_softmax(z64, dim=1)
    ok = targets >= 0
    want = -lp[ok, targets[ok].long()].sum() / n + 0.01 * (lp.exp() * lp).sum(dim=1).mean()
    gx, gw = torch.autograd.grad(want, (x64, w64))
    assert abs(loss.double() - want) <= 1e-6 * abs(want)
    assert torch.linalg.norm(dx.double() - gx) <= 3e-6 * torch.linalg.norm(gx)
    assert torch.linalg.norm(dw.double() - gw) <= 3e-6 * torch.linalg.norm(gw)


def test_rows_further_apart_than_32_bits(big_memory):  # noqa: F811
    T, stride = 37, (1 << 27) + 24  # 4.9e9 values
    g = rng_of(63)
    near = torch.from_numpy(g.standard_normal((T, 96))).to(torch.bfloat16).cuda()
    far = far_rows(near, torch.bfloat16, stride)
    heads = lambda t: t.unflatten(1, (3, 32))  # noqa: E731
    rope = Rope(T, 32, 32, g=g)
    out, want = torch.zeros_like(near), torch.zeros_like(near)
    moe.moe_qk_norm_rope(heads(near), None, heads(want), None, **rope.kw)
    moe.moe_qk_norm_rope(heads(far), None, heads(out), None, **rope.kw)
    assert torch.equal(out, want)
    dw = [torch.zeros(32, device="cuda") for _ in range(2)]
    moe.moe_qk_norm_rope_grad(heads(near), None, heads(near), None, heads(want), None, dq_weight=dw[0], **rope.kw)
    moe.moe_qk_norm_rope_grad(heads(far), None, heads(far), None, heads(out), None, dq_weight=dw[1], **rope.kw)
    assert torch.equal(out, want) and torch.equal(*dw)
    a, b, lse = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"), torch.zeros((T, 2), device="cuda")
    moe.moe_token_logprobs(near, entropy=a, lse=lse)
    moe.moe_token_logprobs(far, entropy=b)
    assert torch.equal(a, b)
    for n in (1, 20, 37):
        p = Product(n, 96, 96, "bf16", seed=8)
        y = [torch.zeros((n, 96), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        moe.moe_q4_linear(near[:n], p.nib, p.scl, y[0], mul=near[:n], residual=near[:n])
        moe.moe_q4_linear(far[:n], p.nib, p.scl, y[1], mul=far[:n], residual=far[:n])
        assert torch.equal(*y)
    moe.moe_token_logprobs_grad(near, lse, want, entropy=a, dentropy=a)
    moe.moe_token_logprobs_grad(far, lse, far, entropy=a, dentropy=a)
    assert torch.equal(far, want)
    # last: outputs that far apart, in place
    far.copy_(near)
    moe.moe_qk_norm_rope(heads(near), None, heads(want), None, **rope.kw)
    moe.moe_qk_norm_rope(heads(far), None, heads(far), None, **rope.kw)
    assert torch.equal(far, want)


@pytest.mark.parametrize("T,N,K,xt", [(300, 1600, 8000, "f32"), (4100, 4100, 160, "bf16"), (300, 2300, 4096, "q8")])
def test_products_with_an_epilogue_at_once_and_captured(T, N, K, xt):
    ps = [Product(T, N, K, xt, seed=s) for s in (1, 2)]
    bias = torch.from_numpy(rng_of(64).standard_normal(N)).float().cuda()
    ys, wants = [torch.empty((T, N), device="cuda") for _ in range(2)], []
    wss = [moe.moe_q4_workspace(p.x, p.nib) for p in ps]
    assert wss[0] is not None

    def call(i, stream=None):
        p = ps[i]
        moe.moe_q4_linear(p.x, p.nib, p.scl, ys[i], bias=bias, act=moe.MOE_ACT_GELU_TANH, residual=p.x[:, :1].float().expand(T, N).contiguous()
                          if stream is None else res[i], scales=p.scales, workspace=wss[i], stream=stream)

    res = [p.x[:, :1].float().expand(T, N).contiguous() for p in ps]
    for i in range(2):
        call(i)
        wants.append(ys[i].clone())
        v = torch.from_numpy(ps[i].ref).cuda() + bias.double()
        ref = v * torch.sigmoid(2 * 0.7978845608028654 * (v + 0.044715 * v ** 3)) + res[i].double()
        assert torch.linalg.norm(ys[i].double() - ref) <= (1.2 * ps[i].rms + 1e-6) * torch.linalg.norm(ref)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            call(i, streams[i])
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, wants))
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            call(i, streams[i].cuda_stream)
    for _ in range(3):
        for y in ys:
            y.zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, wants))

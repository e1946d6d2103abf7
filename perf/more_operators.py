"""Measured cases of the operators behind the dense products: the norm and
rotation of queries and keys (moe_qk_norm_rope, moe_qk_norm_rope_grad), the
4-bit product with bias, activation, factor and residual (moe_q4_linear), and
the log probabilities of tokens (moe_token_logprobs, moe_token_logprobs_grad).

own = False: `run` computes the operator in elementary torch operations, in
fp32 (rotation angles in fp64), rounded once at the end. own = True: `run`
calls the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2, "q8": 1 + 4 / 32}  # q8: a byte and a 32nd of an fp32 scale
EPS = 1e-6
MAX_POS = 1 << 18

# the largest listed work of each operator bounds what is drawn
MAX_HEADS = 12287 * 36 * 128
MAX_HEADS_GRAD = 4096 * 36 * 128
MAX_WEIGHTS = 20481 * 4096
MAX_PRODUCTS = 4096 * 4096 * 4096
MAX_LOGITS = 4096 * 65537
MAX_SORTED = 301 * 131072  # with alternatives


def listed():
    return [
        # one decode token of the hidden-2048 model: 16 query and 2 key heads out of the fused projection
        {"name": "qk-t1-q16k2-d128-f32", "op": "qk", "T": 1, "Hq": 16, "Hk": 2, "D": 128, "R": 128, "axes": 1, "pairs": False, "x": "f32", "out": "f32"},
        # the hidden-4096 model's prompt: 32 + 4 heads, rows of a fused 5120-wide projection
        {"name": "qk-t4096-q32k4-d128-bf16", "op": "qk", "T": 4096, "Hq": 32, "Hk": 4, "D": 128, "R": 128, "axes": 1, "pairs": False, "x": "bf16", "out": "bf16"},
        # frames of a video: time, height and width, a quarter of the head not rotated, ragged
        {"name": "qk-t12287-q14k2-d80-axes3-f16", "op": "qk", "T": 12287, "Hq": 14, "Hk": 2, "D": 80, "R": 60, "axes": 3, "pairs": True, "x": "f16", "out": "f16"},
        # the training step of the second: gradients of queries, keys and both norms' weights
        {"name": "qkgrad-t4096-q32k4-d128-bf16", "op": "qkgrad", "T": 4096, "Hq": 32, "Hk": 4, "D": 128, "R": 128, "axes": 1, "pairs": False, "x": "bf16", "out": "bf16"},
        # one decode token through the gate of a shared expert: silu, times the up product
        {"name": "linear-t1-n1024-k2048-f32", "op": "linear", "T": 1, "N": 1024, "K": 2048, "x": "f32", "y": "f32", "bias": False, "act": "silu", "mul": True, "res": False, "pad": 0},
        # five tokens (a speculative check) through fused query/key/value weights with a bias, 8-bit activations
        {"name": "linear-t5-n5120-k4096-q8", "op": "linear", "T": 5, "N": 5120, "K": 4096, "x": "q8", "y": "f32", "bias": True, "act": "none", "mul": False, "res": False, "pad": 0},
        # the batch-32 decode through the down projection of a shared expert, onto the residual stream
        {"name": "linear-t32-n4096-k1536-f32", "op": "linear", "T": 32, "N": 4096, "K": 1536, "x": "f32", "y": "f32", "bias": False, "act": "none", "mul": False, "res": True, "pad": 0},
        # a prompt through a square projection with all of it
        {"name": "linear-t4096-n4096-k4096-bf16", "op": "linear", "T": 4096, "N": 4096, "K": 4096, "x": "bf16", "y": "bf16", "bias": True, "act": "gelu_tanh", "mul": True, "res": True, "pad": 0},
        # one sampled token of a 65537-word head, with 20 alternatives
        {"name": "logp-t1-v65537-n20-f32", "op": "logp", "T": 1, "V": 65537, "n": 20, "z": "f32", "banned": 0.0, "scale": 1.0, "grad": False},
        # a batch-32 decode, words left out by a grammar, a temperature
        {"name": "logp-t32-v32001-n5-f16", "op": "logp", "T": 32, "V": 32001, "n": 5, "z": "f16", "banned": 0.5, "scale": 1.25, "grad": False},
        # scoring a prompt, 8 alternatives each
        {"name": "logp-t301-v131072-n8-bf16", "op": "logp", "T": 301, "V": 131072, "n": 8, "z": "bf16", "banned": 0.0, "scale": 1.0, "grad": False},
        # a training step over 4096 positions: log probabilities, entropies and the gradient
        {"name": "logpgrad-t4096-v65537-bf16", "op": "logp", "T": 4096, "V": 65537, "n": 0, "z": "bf16", "banned": 0.0, "scale": 1.0, "grad": True},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "qk", "qkgrad", "linear", "linear", "linear", "logp", "logp", "logp"])
    if op in ("qk", "qkgrad"):
        D = rng.choice([32, 64, 64, 72, 80, 96, 128, 128, 192, 256])
        Hk = _log_uniform(rng, 1, 16)
        Hq = Hk * rng.choice([1, 2, 4, 7, 8])
        R = rng.choice([D, D, D // 2, D // 8 * 6])
        T = _log_uniform(rng, 1, max(1, min(12287, (MAX_HEADS if op == "qk" else MAX_HEADS_GRAD) // ((Hq + Hk) * D))))
        x = rng.choice(["f32", "f16", "bf16"])
        return {"op": op, "T": T, "Hq": Hq, "Hk": Hk, "D": D, "R": R, "axes": rng.choice([1, 1, 2, 3]),
                "pairs": rng.random() < 0.3, "x": x, "out": rng.choice([x, x, "bf16"])}
    if op == "linear":
        K = _log_uniform(rng, 2, 128) * 32
        N = _log_uniform(rng, 16, min(20481, MAX_WEIGHTS // K))
        T = _log_uniform(rng, 1, max(1, min(4096, MAX_PRODUCTS // (N * K))))
        return {"op": op, "T": T, "N": N, "K": K, "x": rng.choice(["f32", "f16", "bf16", "q8"]),
                "y": rng.choice(["f32", "f16", "bf16"]), "bias": rng.random() < 0.5,
                "act": rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), "mul": rng.random() < 0.4,
                "res": rng.random() < 0.4, "pad": rng.choice([0, 0, 8, 3])}
    V = _log_uniform(rng, 500, 131072)
    grad = rng.random() < 0.4
    n = 0 if grad else rng.randint(0, 32)
    T = _log_uniform(rng, 1, max(1, min(4096, (MAX_SORTED if n else MAX_LOGITS) // V)))
    return {"op": op, "T": T, "V": V, "n": n, "z": rng.choice(["f32", "f16", "bf16"]), "banned": rng.choice([0.0, 0.5, 0.9]),
            "scale": rng.choice([1.0, 1.0, 0.7, 1.25]), "grad": grad}


# ---------------------------------------------------------------------------
# inputs


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _rows(gen, T, n, pad, dtype):
    """T rows of n values, N(0, 1) with a few large channels as activations have, row stride n + pad."""
    a = _normal(gen, T, n) * torch.where(torch.rand(n, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    wide = torch.zeros((T, n + pad), dtype=dtype, device="cuda")
    wide[:, :n] = a.to(dtype)
    return wide[:, :n]


def _empty(T, n, pad, dtype):
    return torch.zeros((T, n + pad), dtype=dtype, device="cuda")[:, :n]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    T = case["T"]
    if case["op"] in ("qk", "qkgrad"):
        Hq, Hk, D, R, A = case["Hq"], case["Hk"], case["D"], case["R"], case["axes"]
        qkv = _rows(gen, T, (Hq + 2 * Hk) * D, 0, TYPES[case["x"]])  # a row of the fused projection
        s["q"], s["k"] = qkv[:, :Hq * D].view(T, Hq, D), qkv[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D)
        s["qw"], s["kw"] = 1 + 0.1 * _normal(gen, D), 1 + 0.1 * _normal(gen, D)
        s["inv_freq"] = (1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)).float()
        # sequences of up to some thousand tokens, some of them far into their context
        start = torch.randint(0, MAX_POS, (1 + T // 2000,), generator=gen, device="cuda")
        at = torch.arange(T, device="cuda")
        first = (start[at // 2000] + at % 2000).int()
        s["pos"] = torch.cat([first[None], torch.randint(0, 512, (A - 1, T), generator=gen, device="cuda", dtype=torch.int32)])
        s["axis"] = None if A == 1 else (torch.arange(R // 2, device="cuda") * A // (R // 2)).to(torch.uint8)
        to = TYPES[case["out"]]
        if case["op"] == "qk":
            s["q_out"], s["k_out"] = (torch.zeros((T, h, D), dtype=to, device="cuda") for h in (Hq, Hk))
        else:
            s["gq"], s["gk"] = (_normal(gen, T, h, D).to(to) for h in (Hq, Hk))
            s["dq"], s["dk"] = (torch.zeros((T, h, D), dtype=TYPES[case["x"]], device="cuda") for h in (Hq, Hk))
            s["dqw"], s["dkw"] = torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")
    elif case["op"] == "linear":
        N, K, pad = case["N"], case["K"], case["pad"]
        s["nib"] = torch.randint(0, 256, (N, K // 32, 16), generator=gen, device="cuda", dtype=torch.uint8)
        s["scl"] = ((0.2 + 1.8 * torch.rand((N, K // 32), generator=gen, device="cuda")) / (5 * math.sqrt(K))).half()
        s["scales"] = None
        if case["x"] == "q8":
            v = _rows(gen, T, K, 0, torch.float32).view(T, K // 32, 32)
            top = v.abs().amax(dim=2, keepdim=True)
            s["scales"] = (top / 127).view(T, K // 32).contiguous()
            s["x"] = torch.round(v * (127 / top)).to(torch.int8).view(T, K)
        else:
            s["x"] = _rows(gen, T, K, pad, TYPES[case["x"]])
        yt = TYPES[case["y"]]
        s["bias"] = 0.3 * _normal(gen, N) if case["bias"] else None
        s["mul"] = _normal(gen, T, N).to(yt) if case["mul"] else None
        s["res"] = _rows(gen, T, N, pad, yt) if case["res"] else None
        s["y"] = _empty(T, N, pad, yt)
    else:
        V, n = case["V"], case["n"]
        # popular and rare words, and each position's own preference
        z = -1.1 * torch.log1p(torch.randperm(V, generator=gen, device="cuda").float()) + 3 * _normal(gen, T, V)
        if case["banned"]:
            z[:, 1:].masked_fill_(torch.rand((T, V - 1), generator=gen, device="cuda") < case["banned"], -math.inf)
        s["logits"] = z.to(TYPES[case["z"]])
        # the most likely of a few random words and word 0, which no grammar leaves out; none in a tenth of a
        # training step's positions
        some = torch.randint(0, V, (T, 8), generator=gen, device="cuda")
        some[:, 0] = 0
        s["targets"] = some.gather(1, z.gather(1, some).argmax(dim=1, keepdim=True)).squeeze(1).int()
        s["logp"], s["entropy"], s["lse"] = (torch.zeros(d, device="cuda") for d in ((T,), (T,), (T, 2)))
        if n:
            s["ids"], s["alt"] = torch.zeros((T, n), dtype=torch.int32, device="cuda"), torch.zeros((T, n), device="cuda")
        if case["grad"]:
            s["targets"].masked_fill_(torch.rand(T, generator=gen, device="cuda") < 0.1, -1)
            s["dlogp"], s["dentropy"] = _normal(gen, T), -0.01 * torch.rand(T, generator=gen, device="cuda")
            s["dlogits"] = torch.zeros_like(s["logits"])
    return s


# ---------------------------------------------------------------------------
# plain forms


def _angles(s):
    R = s["case"]["R"]
    pos = s["pos"].double()
    pos = pos[0][:, None] if s["axis"] is None else pos[s["axis"].long()].t()
    a = pos * s["inv_freq"].double()
    return a.cos().float().view(-1, 1, R // 2), a.sin().float().view(-1, 1, R // 2)


def _turned(x, cos, sin, R, pairs):
    """Head values with their pairs turned: (a, b) -> (a cos - b sin, b cos + a sin)."""
    if pairs:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., R:]], dim=-1)


def _plain_qk(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w):
        v = x.float()
        v = v * torch.rsqrt((v * v).mean(dim=2, keepdim=True) + EPS) * w
        return _turned(v, cos, sin, c["R"], c["pairs"]).to(TYPES[c["out"]])

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _plain_qk_grad(s):
    c = s["case"]
    cos, sin = _angles(s)

    def one(x, w, g):
        v = x.float()
        r = torch.rsqrt((v * v).mean(dim=2, keepdim=True) + EPS)
        v = v * r
        g = _turned(g.float(), cos, -sin, c["R"], c["pairs"])
        u = g * w
        dx = r * (u - v * (u * v).mean(dim=2, keepdim=True))
        return dx.to(x.dtype), (g * v).sum(dim=(0, 1))

    (dq, dqw), (dk, dkw) = one(s["q"], s["qw"], s["gq"]), one(s["k"], s["kw"], s["gk"])
    return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def _plain_linear(s):
    c = s["case"]
    T, N, K = c["T"], c["N"], c["K"]
    q = torch.cat([s["nib"] & 15, s["nib"] >> 4], dim=2).float() - 8.0
    w = (q * s["scl"].float().unsqueeze(2)).view(N, K)
    x = s["x"].float()
    if s["scales"] is not None:
        x = (x.view(T, K // 32, 32) * s["scales"].unsqueeze(2)).view(T, K)
    v = x @ w.t()
    if s["bias"] is not None:
        v = v + s["bias"]
    if c["act"] == "relu":
        v = v.clamp(min=0)
    elif c["act"] == "silu":
        v = v / (1 + torch.exp(-v))
    elif c["act"] == "gelu":
        v = 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        v = v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(s["y"].dtype)


def _plain_logp(s):
    c = s["case"]
    n, scale = c["n"], c["scale"]
    z = s["logits"].float() * scale
    top = z.amax(dim=1, keepdim=True)
    d = z - top
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total - torch.where(e > 0, e * d, 0.0).sum(dim=1, keepdim=True) / total
    ok = (s["targets"] >= 0).unsqueeze(1)
    at = s["targets"].long().clamp(min=0).unsqueeze(1)
    logp = torch.where(ok, d.gather(1, at) - log_total, 0.0)
    out = {"logp": logp.squeeze(1), "entropy": entropy.squeeze(1)}
    if n:
        ids = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :n]
        out["alt"] = d.gather(1, ids) - log_total
        out["ids"] = torch.where(out["alt"] > -math.inf, ids, -1).int()  # fewer words than alternatives
    if c["grad"]:
        a, b = torch.where(ok, s["dlogp"].unsqueeze(1), 0.0), s["dentropy"].unsqueeze(1)
        p = e / total
        g = torch.where(p > 0, -p * (a + b * (d - log_total + entropy)), 0.0)
        g.scatter_add_(1, at, a)
        out["dlogits"] = (scale * g).to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"qk": _plain_qk, "qkgrad": _plain_qk_grad, "linear": _plain_linear, "logp": _plain_logp}[op](s)
    import moe_expert_offload_gemv_amd as moe

    if op in ("qk", "qkgrad"):
        rope = dict(eps=EPS, inv_freq=s["inv_freq"], positions=s["pos"], pair_axis=s["axis"],
                    flags=moe.MOE_ROPE_PAIRS if s["case"]["pairs"] else 0)
        if op == "qk":
            moe.moe_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], q_weight=s["qw"], k_weight=s["kw"], **rope)
            return {"q": s["q_out"], "k": s["k_out"]}
        if "work" not in s:  # the workspace a program keeps for its calls
            s["work"] = moe.moe_qk_norm_rope_workspace(s["q"], s["k"])
        moe.moe_qk_norm_rope_grad(s["q"], s["k"], s["gq"], s["gk"], s["dq"], s["dk"], q_weight=s["qw"], k_weight=s["kw"],
                                  dq_weight=s["dqw"], dk_weight=s["dkw"], workspace=s["work"], **rope)
        return {"dq": s["dq"], "dk": s["dk"], "dqw": s["dqw"], "dkw": s["dkw"]}
    if op == "linear":
        if "work" not in s:
            s["work"] = moe.moe_q4_workspace(s["x"], s["nib"])
        act = {"none": moe.MOE_ACT_NONE, "relu": moe.MOE_ACT_RELU, "silu": moe.MOE_ACT_SILU, "gelu": moe.MOE_ACT_GELU,
               "gelu_tanh": moe.MOE_ACT_GELU_TANH}[s["case"]["act"]]
        moe.moe_q4_linear(s["x"], s["nib"], s["scl"], s["y"], bias=s["bias"], act=act, mul=s["mul"], residual=s["res"],
                          scales=s["scales"], workspace=s["work"])
        return s["y"]
    if "work" not in s:
        s["work"] = moe.moe_token_logprobs_workspace(s["logits"], s["case"]["n"])
    moe.moe_token_logprobs(s["logits"], targets=s["targets"], logp=s["logp"], entropy=s["entropy"], lse=s["lse"],
                           top_ids=s.get("ids"), top_logp=s.get("alt"), scale=s["case"]["scale"], workspace=s["work"])
    out = {"logp": s["logp"], "entropy": s["entropy"]}
    if s["case"]["n"]:
        out["ids"], out["alt"] = s["ids"], s["alt"]
    if s["case"]["grad"]:
        moe.moe_token_logprobs_grad(s["logits"], s["lse"], s["dlogits"], targets=s["targets"], dlogp=s["dlogp"],
                                    entropy=s["entropy"], dentropy=s["dentropy"], scale=s["case"]["scale"])
        out["dlogits"] = s["dlogits"]
    return out


def work(case):
    T = case["T"]
    if case["op"] in ("qk", "qkgrad"):
        n = T * (case["Hq"] + case["Hk"]) * case["D"]
        if case["op"] == "qk":
            return {"bytes": n * (WIDTH[case["x"]] + WIDTH[case["out"]]) + 4 * T * case["axes"], "flops": 8 * n}
        return {"bytes": n * (2 * WIDTH[case["x"]] + WIDTH[case["out"]]) + 4 * T * case["axes"], "flops": 16 * n}
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        outs = WIDTH[case["y"]] * (1 + case["mul"] + case["res"])
        return {"bytes": N * K * 18 / 32 + T * K * WIDTH[case["x"]] + T * N * outs + 4 * N * case["bias"], "flops": 2 * T * N * K}
    n = T * case["V"]
    # one read of the logits for the sums, one for the gradient, which is written
    return {"bytes": n * WIDTH[case["z"]] * (3 if case["grad"] else 1) + T * (12 + 8 * case["n"]),
            "flops": n * (12 if case["grad"] else 6)}


# ---------------------------------------------------------------------------
# the definitions in fp64


def _exact_heads(x, w, s):
    """Norm and rotation of heads [T][H][D] in fp64, each pair a complex number."""
    c = s["case"]
    R, half = c["R"], c["R"] // 2
    y = x / x.square().mean(dim=2, keepdim=True).add(EPS).sqrt() * w
    which = torch.zeros(half, dtype=torch.long, device="cuda") if s["axis"] is None else s["axis"].long()
    angle = s["pos"].double().t()[:, which] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    lead = y[..., :R].reshape(*y.shape[:2], half, 2) if c["pairs"] else y[..., :R].reshape(*y.shape[:2], 2, half).transpose(2, 3)
    t = torch.view_as_real(torch.view_as_complex(lead.contiguous()) * turn)
    if not c["pairs"]:
        t = t.transpose(2, 3)
    return torch.cat([t.reshape(*y.shape[:2], R), y[..., R:]], dim=2)


def exact(case, seed):
    s = prepare(case, seed)
    T = case["T"]
    if case["op"] == "qk":
        return {"q": _exact_heads(s["q"].double(), s["qw"].double(), s), "k": _exact_heads(s["k"].double(), s["kw"].double(), s)}
    if case["op"] == "qkgrad":
        leaves = [s[n].double().requires_grad_() for n in ("q", "k", "qw", "kw")]
        outs = [_exact_heads(leaves[0], leaves[2], s), _exact_heads(leaves[1], leaves[3], s)]
        return dict(zip(("dq", "dk", "dqw", "dkw"), torch.autograd.grad(outs, leaves, [s["gq"].double(), s["gk"].double()])))
    if case["op"] == "linear":
        N, K = case["N"], case["K"]
        x = s["x"].double()
        if s["scales"] is not None:
            x = x * s["scales"].double().repeat_interleave(32, dim=1)
        level = torch.arange(-8, 8, dtype=torch.float64, device="cuda")
        y = torch.empty((T, N), dtype=torch.float64, device="cuda")
        for n in range(0, N, 4096):  # some weight rows at a time
            byte = s["nib"][n:n + 4096].int()
            w = torch.stack([level[byte % 16], level[byte // 16]], dim=2)  # [rows][blocks][half][16]
            w = w * s["scl"][n:n + 4096, :, None, None].double()
            y[:, n:n + 4096] = torch.mm(x, w.reshape(-1, K).t().contiguous())
        if case["bias"]:
            y += s["bias"].double()
        if case["act"] == "relu":
            y = torch.relu(y)
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "gelu":
            y = y * torch.special.ndtr(y)
        elif case["act"] == "gelu_tanh":
            y = y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))) / 2
        if case["mul"]:
            y *= s["mul"].double()
        return y + s["res"].double() if case["res"] else y
    out = {"logp": torch.zeros(T, dtype=torch.float64, device="cuda"), "entropy": torch.zeros(T, dtype=torch.float64, device="cuda")}
    if case["n"]:
        out["ids"] = torch.zeros((T, case["n"]), dtype=torch.int32, device="cuda")
        out["alt"] = torch.zeros((T, case["n"]), dtype=torch.float64, device="cuda")
    if case["grad"]:
        out["dlogits"] = torch.zeros((T, case["V"]), dtype=torch.float64, device="cuda")
    for t in range(0, T, 256):  # some positions at a time
        some = slice(t, t + 256)
        z = s["logits"][some].double() * case["scale"]
        lp = torch.log_softmax(z, dim=1)
        p = lp.exp()
        H = torch.special.entr(p).sum(dim=1)
        y = s["targets"][some].long()
        row = torch.arange(len(y), device="cuda")
        out["logp"][some] = torch.where(y >= 0, lp[row, y.clamp(min=0)], 0.0)
        out["entropy"][some] = H
        if case["n"]:
            # rounds of taking the largest, the first of equal ones
            left = s["logits"][some].double()
            for j in range(case["n"]):
                best = (left == left.amax(dim=1, keepdim=True)).int().argmax(dim=1)
                out["alt"][some, j] = torch.where(left[row, best] > -math.inf, lp[row, best], -math.inf)
                out["ids"][some, j] = torch.where(left[row, best] > -math.inf, best, -1).int()
                left[row, best] = -math.inf
        if case["grad"]:
            a, b = torch.where(y >= 0, s["dlogp"][some].double(), 0.0), s["dentropy"][some].double()
            g = -p * a[:, None] - torch.where(p > 0, p * (lp + H[:, None]), 0.0) * b[:, None]
            g[row, y.clamp(min=0)] += a
            out["dlogits"][some] = g * case["scale"]
    return out

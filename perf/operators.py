"""Measured cases of the operators beside the routed experts: the residual
add with RMS norm (moe_add_rmsnorm), the dense product with 4-bit weights
(moe_q4_matmul) and the router's balance loss with its gradient
(moe_router_balance, moe_router_balance_grad).

own = False: `run` computes the operator in elementary torch operations, in
fp32, rounded once at the end. own = True: `run` calls the library.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDTH = {"f32": 4, "f16": 2, "bf16": 2, "q8": 1 + 4 / 32}  # q8: a byte and a 32nd of an fp32 scale
EPS = 1e-6
ALPHA, BETA = 1e-2, 1e-3  # weights of the balance and z terms

# the largest listed work of each operator bounds what is drawn
MAX_NORM = 12287 * 4096
MAX_Q4_WEIGHTS = 65537 * 4096
MAX_Q4_PRODUCTS = 4096 * 5120 * 4096
MAX_LOGITS = 32768 * 512


def listed():
    return [
        # one decode token of the hidden-2048 model: fp32 residual stream, fp32 input of the experts
        {"name": "norm-t1-h2048-f32", "op": "norm", "T": 1, "H": 2048, "x": "f32", "res": "f32", "out": "f32", "pad": 0},
        # its 4096-token prompt pass: bf16 stream, 8-bit input of the dense products
        {"name": "norm-t4096-h2048-q8", "op": "norm", "T": 4096, "H": 2048, "x": "bf16", "res": "bf16", "out": "q8", "pad": 0},
        # the hidden-4096 model's long prompt, ragged: the experts' fp32 output joins a bf16 stream
        {"name": "norm-t12287-h4096-bf16", "op": "norm", "T": 12287, "H": 4096, "x": "f32", "res": "bf16", "out": "bf16", "pad": 0},
        # one decode token through a square projection
        {"name": "q4-t1-n2048-k2048-f32", "op": "q4", "T": 1, "N": 2048, "K": 2048, "x": "f32", "y": "f32", "pad": 0},
        # one decode token through the output head of a 65537-word vocabulary
        {"name": "q4-t1-n65537-k4096-bf16", "op": "q4", "T": 1, "N": 65537, "K": 4096, "x": "bf16", "y": "f32", "pad": 0},
        # five tokens (a speculative check) through fused query/key/value weights, 8-bit activations
        {"name": "q4-t5-n5120-k4096-q8", "op": "q4", "T": 5, "N": 5120, "K": 4096, "x": "q8", "y": "f32", "pad": 0},
        # the batch-32 decode through the down projection of a shared expert
        {"name": "q4-t32-n4096-k1536-f32", "op": "q4", "T": 32, "N": 4096, "K": 1536, "x": "f32", "y": "f32", "pad": 0},
        # a short prompt, odd sizes, rows cut from wider arrays
        {"name": "q4-t201-n1001-k1056-f16", "op": "q4", "T": 201, "N": 1001, "K": 1056, "x": "f16", "y": "f16", "pad": 8},
        # a 4096-token prompt through fused query/key/value weights
        {"name": "q4-t4096-n5120-k4096-bf16", "op": "q4", "T": 4096, "N": 5120, "K": 4096, "x": "bf16", "y": "bf16", "pad": 0},
        # a small router's micro-batch, odd sizes, padded tokens
        {"name": "balance-t999-e60k4-f16", "op": "balance", "T": 999, "E": 60, "k": 4, "z": "f16", "masked": True},
        # the 256-expert model's 12288-token micro-batch, padded tokens
        {"name": "balance-t12288-e256k8-bf16", "op": "balance", "T": 12288, "E": 256, "k": 8, "z": "bf16", "masked": True},
        # the 512-expert model, calibration over a large batch
        {"name": "balance-t32768-e512k8-f32", "op": "balance", "T": 32768, "E": 512, "k": 8, "z": "f32", "masked": False},
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "q4", "q4", "balance"])
    if op == "norm":
        out = rng.choice(["f32", "f16", "bf16", "q8"])
        H = _log_uniform(rng, 64, 8192)
        H = max(32, H // 32 * 32) if out == "q8" or rng.random() < 0.6 else H
        T = _log_uniform(rng, 1, max(1, min(12287, MAX_NORM // H)))
        res = rng.choice(["f32", "f16", "bf16"])
        return {"op": op, "T": T, "H": H, "x": rng.choice([res, "f32"]), "res": res, "out": out,
                "pad": rng.choice([0, 0, 8, 3])}
    if op == "q4":
        K = _log_uniform(rng, 2, 256) * 32
        N = _log_uniform(rng, 16, min(65537, MAX_Q4_WEIGHTS // K))
        T = _log_uniform(rng, 1, max(1, min(4096, MAX_Q4_PRODUCTS // (N * K))))
        return {"op": op, "T": T, "N": N, "K": K, "x": rng.choice(["f32", "f16", "bf16", "q8"]),
                "y": rng.choice(["f32", "f16", "bf16"]), "pad": rng.choice([0, 0, 8, 3])}
    E = _log_uniform(rng, 8, 512)
    return {"op": op, "T": _log_uniform(rng, 1, max(1, min(32768, MAX_LOGITS // E))), "E": E,
            "k": rng.randint(1, min(E, 16)), "z": rng.choice(["f32", "f16", "bf16"]), "masked": rng.random() < 0.5}


# ---------------------------------------------------------------------------
# inputs


def _rows(gen, T, n, pad, dtype):
    """T rows of n values, N(0, 1) with a few large channels as activations have, row stride n + pad."""
    a = torch.randn((T, n), generator=gen, device="cuda")
    a *= torch.where(torch.rand(n, generator=gen, device="cuda") < 0.01, 8.0, 1.0)
    wide = torch.zeros((T, n + pad), dtype=dtype, device="cuda")
    wide[:, :n] = a.to(dtype)
    return wide[:, :n]


def _empty(T, n, pad, dtype):
    return torch.zeros((T, n + pad), dtype=dtype, device="cuda")[:, :n]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, H, pad, out = case["T"], case["H"], case["pad"], case["out"]
        s["x"] = _rows(gen, T, H, pad, TYPES[case["x"]])
        s["residual"] = _rows(gen, T, H, pad, TYPES[case["res"]])
        s["residual_out"] = _empty(T, H, pad, TYPES[case["res"]])
        s["weight"] = 1.0 + 0.1 * torch.randn(H, generator=gen, device="cuda")
        if out == "q8":
            s["out"] = torch.zeros((T, H), dtype=torch.int8, device="cuda")
            s["scales"] = torch.zeros((T, H // 32), device="cuda")
            s["values"] = torch.zeros((T, H // 32, 32), dtype=torch.float16, device="cuda")
        else:
            s["out"], s["scales"] = _empty(T, H, pad, TYPES[out]), None
    elif case["op"] == "q4":
        T, N, K, pad = case["T"], case["N"], case["K"], case["pad"]
        s["nib"] = torch.randint(0, 256, (N, K // 32, 16), generator=gen, device="cuda", dtype=torch.uint8)
        s["scl"] = (0.001 + 0.009 * torch.rand((N, K // 32), generator=gen, device="cuda")).half()
        s["scales"] = None
        if case["x"] == "q8":
            v = _rows(gen, T, K, 0, torch.float32).view(T, K // 32, 32)
            top = v.abs().amax(dim=2, keepdim=True)
            s["scales"] = (top / 127).view(T, K // 32).contiguous()
            s["x"] = torch.round(v * (127 / top)).to(torch.int8).view(T, K)
        else:
            s["x"] = _rows(gen, T, K, pad, TYPES[case["x"]])
        s["y"] = _empty(T, N, pad, TYPES[case["y"]])
    else:
        T, E = case["T"], case["E"]
        # ln of a Zipf popularity plus Gumbel noise: top-k of it picks experts by that popularity
        pop = -1.1 * torch.log1p(torch.randperm(E, generator=gen, device="cuda").float())
        u = torch.rand((T, E), generator=gen, device="cuda").clamp_(1e-7, 1 - 1e-7)
        s["logits"] = (pop - torch.log(-torch.log(u))).to(TYPES[case["z"]])
        s["valid"] = (torch.rand(T, generator=gen, device="cuda") < 0.9).to(torch.uint8) if case["masked"] else None
        s["counts"] = torch.zeros(E, dtype=torch.int32, device="cuda")
        s["load"] = torch.zeros(E, device="cuda")
        s["stats"] = torch.zeros(4, device="cuda")
        s["lse"] = torch.zeros(T, device="cuda")
        s["dlogits"] = torch.zeros_like(s["logits"])
        # gradient of the whole loss to this one: fp16 training scales it
        s["dloss"] = torch.full((1,), 65536.0 if case["z"] == "f16" else 1.0, device="cuda")
    return s


# ---------------------------------------------------------------------------
# plain forms


def _plain_norm(s):
    H = s["case"]["H"]
    v = s["x"].float() + s["residual"].float()
    stream = v.to(s["residual"].dtype)
    v = v * (torch.rsqrt((v * v).sum(dim=1, keepdim=True) / H + EPS)) * s["weight"]
    if s["case"]["out"] != "q8":
        return {"residual": stream, "out": v.to(s["out"].dtype)}
    v = v.view(v.shape[0], H // 32, 32)
    top = v.abs().amax(dim=2, keepdim=True)
    code = torch.where(top > 0, torch.round(v * (127 / top)), 0.0)
    return {"residual": stream, "out": (code * (top / 127)).half()}


def _plain_q4(s):
    T, N, K = s["case"]["T"], s["case"]["N"], s["case"]["K"]
    q = torch.cat([s["nib"] & 15, s["nib"] >> 4], dim=2).float() - 8.0
    w = (q * s["scl"].float().unsqueeze(2)).view(N, K)
    x = s["x"].float()
    if s["scales"] is not None:
        x = (x.view(T, K // 32, 32) * s["scales"].unsqueeze(2)).view(T, K)
    return (x @ w.t()).to(s["y"].dtype)


def _plain_balance(s):
    E, k = s["case"]["E"], s["case"]["k"]
    z = s["logits"].float()
    ok = torch.ones(z.shape[0], device=z.device) if s["valid"] is None else s["valid"].float()
    ids = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
    counts = (torch.zeros_like(z).scatter_(1, ids, 1.0) * ok.unsqueeze(1)).sum(dim=0)
    top = z.amax(dim=1, keepdim=True)
    ex = torch.exp(z - top)
    total = ex.sum(dim=1, keepdim=True)
    p, lse = ex / total, (top + torch.log(total)).squeeze(1)
    n = ok.sum()
    each = torch.where(n > 0, 1 / n, 0.0)
    load = counts * (E / k) * each
    balance = ALPHA * (load * (p * ok.unsqueeze(1)).sum(dim=0)).sum() * each
    zterm = BETA * (lse * lse * ok).sum() * each
    inner = (p * load).sum(dim=1, keepdim=True)
    grad = s["dloss"] * ok.unsqueeze(1) * each * p * (ALPHA * (load - inner) + 2 * BETA * lse.unsqueeze(1))
    return {"counts": counts.to(torch.int32), "load": load, "losses": torch.stack([balance + zterm, balance, zterm]),
            "dlogits": grad.to(s["logits"].dtype)}


# ---------------------------------------------------------------------------


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_norm(s) if op == "norm" else _plain_q4(s) if op == "q4" else _plain_balance(s)
    import moe_expert_offload_gemv_amd as moe

    if op == "norm":
        moe.moe_add_rmsnorm(s["x"], s["weight"], s["out"], residual=s["residual"], residual_out=s["residual_out"],
                            scales=s["scales"], eps=EPS)
        if s["scales"] is None:
            return {"residual": s["residual_out"], "out": s["out"]}
        # the codes as the values they stand for
        return {"residual": s["residual_out"],
                "out": torch.mul(s["out"].view_as(s["values"]), s["scales"].unsqueeze(2), out=s["values"])}
    if op == "q4":
        if "work" not in s:  # the workspace a program keeps for its calls
            s["work"] = moe.moe_q4_workspace(s["x"], s["nib"])
        moe.moe_q4_matmul(s["x"], s["nib"], s["scl"], s["y"], scales=s["scales"], workspace=s["work"])
        return s["y"]
    if "work" not in s:
        s["work"] = moe.moe_router_balance_workspace(s["logits"])
    moe.moe_router_balance(s["logits"], s["case"]["k"], s["counts"], s["load"], s["stats"], s["lse"], valid=s["valid"],
                           balance=ALPHA, z=BETA, workspace=s["work"])
    moe.moe_router_balance_grad(s["logits"], s["load"], s["stats"], s["lse"], s["dlogits"], dloss=s["dloss"], balance=ALPHA,
                                z=BETA)
    return {"counts": s["counts"], "load": s["load"], "losses": s["stats"][:3], "dlogits": s["dlogits"]}


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"]
        stream = WIDTH[case["x"]] + 2 * WIDTH[case["res"]]
        return {"bytes": n * (stream + WIDTH[case["out"]]) + 4 * case["H"], "flops": 5 * n}
    if case["op"] == "q4":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K * 18 / 32 + T * K * WIDTH[case["x"]] + T * N * WIDTH[case["y"]], "flops": 2 * T * N * K}
    n = case["T"] * case["E"]
    # one read of the logits for the loss and counts, one for the gradient, which is written
    return {"bytes": 3 * n * WIDTH[case["z"]], "flops": 15 * n}


# ---------------------------------------------------------------------------
# the definitions in fp64


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        stream = s["x"].double().add_(s["residual"].double())
        rms = torch.sqrt(stream.square().mean(dim=1) + EPS)
        v = (stream / rms[:, None]).mul_(s["weight"].double())
        if case["out"] == "q8":
            v = v.reshape(T, -1, 32)
            step = v.abs().max(dim=2).values / 127
            v = torch.round(v / step[..., None]).nan_to_num_(0.0).mul_(step[..., None])
        return {"residual": stream, "out": v}
    if case["op"] == "q4":
        T, N, K = case["T"], case["N"], case["K"]
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
        return y
    T, E, k = case["T"], case["E"], case["k"]
    z = s["logits"].double()
    ok = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"].bool()
    n = int(ok.sum())
    out = torch.zeros_like(z)
    if n == 0:
        none = torch.zeros(E, dtype=torch.float64, device="cuda")
        return {"counts": none.int(), "load": none, "losses": none[:3].clone(), "dlogits": out}
    zv = z[ok]
    p, lse = torch.softmax(zv, dim=1), torch.logsumexp(zv, dim=1)
    # the k best: k rounds of taking the largest, the first of equal ones
    left, counts = zv.clone(), torch.zeros(E, dtype=torch.int64, device="cuda")
    for _ in range(k):
        best = (left == left.max(dim=1, keepdim=True).values).int().argmax(dim=1)
        left[torch.arange(n, device="cuda"), best] = -math.inf
        counts += torch.bincount(best, minlength=E)
    load = counts.double() * E / (k * n)
    balance, zterm = ALPHA * torch.dot(load, p.mean(dim=0)), BETA * lse.square().mean()
    out[ok] = s["dloss"].double() * (p * (ALPHA * (load - (p @ load)[:, None]) + 2 * BETA * lse[:, None])) / n
    return {"counts": counts.int(), "load": load, "losses": torch.stack([balance + zterm, balance, zterm]), "dlogits": out}

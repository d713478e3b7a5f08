"""The operators around a quantized linear that learn and adapt, as measured cases.

Three operators, each in its plain form (elementary torch operations in 32
bits) and through the package's own entry points:

  * low-rank adapters of many requests beside one shared projection, forward
    (Y = base + scale_a (X A_a^T) B_a^T, optionally with the classifier-free-
    guidance combine) and backward (dX, dA, dB);
  * group normalisation with an activation over channels-last images, forward
    and backward (dX, dgamma, dbeta);
  * the global norm of many gradients and their clipping.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

# (name, K, N) of the four linears of a transformer block of hidden size 1152.
_BLOCK = (("qkv", 1152, 3456), ("proj", 1152, 1152), ("fc1", 1152, 4608), ("fc2", 4608, 1152))
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # One conditioning vector per image through the modulation linear (six
        # vectors of the hidden size): single-row requests, an adapter each.
        dict(name="lora_rows", op="lora", rows=8, requests=8, adapters=8, K=1152, N=6912, rank=16,
             x="bf16", w="bf16", ragged=False, bare=0, mixed_ranks=False, cfg=False),
        # fc1 of a block in a guided step: 8 images of 256 tokens, conditional and
        # unconditional halves, 4 adapters, 2 images without one.
        dict(name="lora_guided", op="lora", rows=4096, requests=8, adapters=4, K=1152, N=4608,
             rank=16, x="f32", w="f32", ragged=False, bare=2, mixed_ranks=False, cfg=True),
        # Requests of unlike lengths, ranks and an odd output width.
        dict(name="lora_ragged", op="lora", rows=1003, requests=23, adapters=9, K=1152, N=1001,
             rank=12, x="f32", w="bf16", ragged=True, bare=0, mixed_ranks=True, cfg=False),
        # Large images: 4 requests of 4096 tokens on a wide projection.
        dict(name="lora_wide", op="lora", rows=16384, requests=4, adapters=4, K=2048, N=8192,
             rank=64, x="bf16", w="bf16", ragged=False, bare=0, mixed_ranks=False, cfg=False),
        # One adapter trained on a batch of 8 images beside fc1.
        dict(name="lora_grad_fc1", op="lora_grad", rows=2048, requests=8, adapters=1, K=1152,
             N=4608, rank=16, x="f32", w="f32", ragged=False, bare=0, mixed_ranks=False,
             cfg=False),
        # Three adapters trained at once beside fc2 on 64 images' tokens, unlike lengths.
        dict(name="lora_grad_fc2", op="lora_grad", rows=16384, requests=7, adapters=3, K=4608,
             N=1152, rank=64, x="bf16", w="bf16", ragged=True, bare=0, mixed_ranks=False,
             cfg=False),
        # The lowest resolution of a latent denoiser, one guided image: latency.
        dict(name="norm_small", op="norm", batch=2, positions=256, channels=1280, groups=32,
             x="bf16", w="f32", act="silu", stats=False),
        # The widest images of a decoder.
        dict(name="norm_large", op="norm", batch=8, positions=16384, channels=320, groups=32,
             x="bf16", w="f32", act="silu", stats=True),
        # Training at a middle resolution, 32 bits.
        dict(name="norm_grad_mid", op="norm_grad", batch=4, positions=1024, channels=640,
             groups=32, x="f32", w="f32", act="silu", stats=True),
        # Training on large crops with an odd number of positions (127 x 129).
        dict(name="norm_grad_large", op="norm_grad", batch=4, positions=16383, channels=256,
             groups=32, x="bf16", w="bf16", act="silu", stats=True),
        # The gradients of rank-16 adapters of all 112 linears of 28 blocks, f32.
        dict(name="clip_adapters", op="clip", kind="adapters", blocks=28, rank=16, count=224,
             size_seed=0, x="f32", out="f32"),
        # The bf16 gradients of the 28 blocks' weights, clipped into the f32
        # buffers that the optimizer reads.
        dict(name="clip_model", op="clip", kind="blocks", blocks=28, rank=0, count=112,
             size_seed=0, x="bf16", out="f32"),
    ]


# ------------------------------------------------------------------ sizes ----

def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e14)


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["lora", "lora", "lora_grad", "norm", "norm_grad", "clip"])
    while True:
        x = rng.choice(["f32", "bf16"])
        if op in ("lora", "lora_grad"):
            fwd = op == "lora"
            cfg = fwd and rng.random() < 0.3
            rows = _log(rng, 4, 16384) if fwd else _log(rng, 64, 16384)
            rows += rows % 2 if cfg else 0
            requests = min(_log(rng, 1, 48), rows // 2 if cfg else rows)
            case = dict(op=op, rows=rows, requests=requests,
                        adapters=rng.randint(1, min(requests, 12)),
                        K=16 * _log(rng, 16, 288), N=_log(rng, 200, 8192),
                        rank=rng.choice([4, 8, 16, 16, 31, 32, 64]), x=x,
                        w=rng.choice(["f32", "bf16"]), ragged=rng.random() < 0.5, bare=0,
                        mixed_ranks=rng.random() < 0.3, cfg=cfg)
        elif op in ("norm", "norm_grad"):
            groups = rng.choice([8, 16, 32, 32])
            case = dict(op=op, batch=rng.randint(1, 16), positions=_log(rng, 64, 16384),
                        channels=groups * rng.randint(1, 1280 // groups), groups=groups, x=x,
                        w=rng.choice(["f32", "bf16"]), act=rng.choice(["silu", "silu", "none"]),
                        stats=op == "norm_grad" or rng.random() < 0.5)
        else:
            case = dict(op=op, kind="mixed", blocks=0, rank=0, count=_log(rng, 3, 400),
                        size_seed=rng.randrange(1 << 30), x=x, out=rng.choice([x, "f32"]))
        if _cost(case) <= top[op]:
            return case


def _grad_sizes(case):
    if case["kind"] == "adapters":
        return [n for _ in range(case["blocks"]) for _, k, m in _BLOCK
                for n in (case["rank"] * k, m * case["rank"])]
    if case["kind"] == "blocks":
        return [k * m for _ in range(case["blocks"]) for _, k, m in _BLOCK]
    r = np.random.RandomState(case["size_seed"])
    return [int(v) for v in np.exp(r.uniform(0.0, math.log(2e6), case["count"]))]


def _lengths(case, seed):
    """Rows of each request: even, or cut at random (some may be empty)."""
    rows = case["rows"] // 2 if case["cfg"] else case["rows"]
    n = case["requests"]
    if case["ragged"]:
        cuts = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, rows + 1, n - 1))
        off = np.concatenate([[0], cuts, [rows]])
    else:
        off = np.arange(n + 1) * rows // n
    return [int(v) for v in off]


def _adapter_ids(case):
    ids = [i % case["adapters"] for i in range(case["requests"])]
    for i in range(case["bare"]):
        ids[-1 - i] = -1
    return ids


def _ranks(case):
    r = case["rank"]
    return [max(1, r >> (a % 3)) if case["mixed_ranks"] else r for a in range(case["adapters"])]


def work(case):
    op = case["op"]
    if op in ("lora", "lora_grad"):
        M, K, N, r = case["rows"], case["K"], case["N"], case["rank"]
        off, ids = _lengths(case, 0), _adapter_ids(case)
        with_adapter = sum(b - a for a, b, i in zip(off, off[1:], ids) if i >= 0)
        halves = 2 if case["cfg"] else 1
        if case["ragged"]:
            with_adapter = off[-1]
        xs, ws = _SIZE[case["x"]], _SIZE[case["w"]]
        weights = sum(_ranks(case)) * (K + N) * ws
        if op == "lora":
            return {"bytes": with_adapter * halves * K * xs + weights + off[-1] * N * 4 * 2,
                    "flops": 2 * with_adapter * r * (halves * K + N)}
        return {"bytes": 2 * M * K * xs + M * N * 4 + M * r * 4 + 2 * weights,
                "flops": 4 * M * r * (K + N)}
    if op in ("norm", "norm_grad"):
        n = case["batch"] * case["positions"] * case["channels"]
        b, per = (2, 10) if op == "norm" else (3, 25)
        return {"bytes": b * n * _SIZE[case["x"]] + 4 * case["channels"] * _SIZE[case["w"]],
                "flops": per * n}
    n = sum(_grad_sizes(case))
    # Clipping needs the norm of all of them first: two readings and one writing.
    return {"bytes": n * (2 * _SIZE[case["x"]] + _SIZE[case["out"]]), "flops": 3 * n}


# ----------------------------------------------------------------- inputs ----

def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed & ((1 << 62) - 1))

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g)
        return t.to(dtype)

    op = case["op"]
    if op in ("lora", "lora_grad"):
        M, K, N, r, n = case["rows"], case["K"], case["N"], case["rank"], case["adapters"]
        wt = _DT[case["w"]]
        off, ids, ranks = _lengths(case, seed), _adapter_ids(case), _ranks(case)
        X = normal(M, K)
        X[:, :: 97] *= 8.0  # outlier channels
        s = dict(X=X.to(_DT[case["x"]]), A=normal(n, r, K, dtype=wt, std=K ** -0.5),
                 B=normal(n, N, r, dtype=wt, std=0.02),
                 scales=torch.tensor([2.0 / (1 + a % 3) for a in range(n)], device="cuda"),
                 off=off, ids=ids, ranks=ranks,
                 d_off=torch.tensor(off, dtype=torch.int32, device="cuda"),
                 d_ids=torch.tensor(ids, dtype=torch.int32, device="cuda"),
                 d_ranks=torch.tensor(ranks, dtype=torch.int32, device="cuda")
                 if case["mixed_ranks"] else None)
        for a, k in enumerate(ranks):  # past an adapter's rank its storage is unused
            s["A"][a, k:] = 0
            s["B"][a, :, k:] = 0
        if op == "lora":
            s["base"] = normal(off[-1], N)
            s["guidance"] = 4.0
        else:
            s["dY"] = normal(M, N, std=1e-2)
            s["S"] = torch.zeros(M, r, device="cuda")  # X A^T, as the forward call saved it
            for i, a in enumerate(ids):
                lo, hi = off[i], off[i + 1]
                if a >= 0 and hi > lo:
                    s["S"][lo:hi] = s["X"][lo:hi].float() @ s["A"][a].float().t()
        return s
    if op in ("norm", "norm_grad"):
        B, L, C, G = case["batch"], case["positions"], case["channels"], case["groups"]
        wt = _DT[case["w"]]
        x = normal(B, L, C) * (0.5 + normal(C).abs()) + normal(C)  # channels of unlike size
        s = dict(x=x.to(_DT[case["x"]]), gamma=normal(C, dtype=wt, std=0.2, mean=1.0),
                 beta=normal(C, dtype=wt, std=0.2), groups=G, eps=1e-5, act=case["act"])
        if op == "norm_grad":
            s["dy"] = normal(B, L, C, dtype=_DT[case["x"]], std=1e-2)
            xg = s["x"].float().view(B, L, G, C // G)
            s["mean"] = xg.mean((1, 3))  # as the forward call saved them
            var = (xg - s["mean"].view(B, 1, G, 1)).square().mean((1, 3))
            s["rstd"] = torch.rsqrt(var + s["eps"])
        return s
    sizes = _grad_sizes(case)
    flat = normal(sum(sizes), std=1e-2, dtype=_DT[case["x"]])
    return dict(grads=[t.clone() for t in flat.split(sizes)], max_norm=1.0)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "clip":
        # one long buffer that the optimizer reads, a view of it for each gradient
        sizes = [t.numel() for t in s["grads"]]
        s["flat"] = torch.empty(sum(sizes), dtype=_DT[case["out"]], device="cuda")
        s["out"] = list(s["flat"].split(sizes))
    if own:
        import bit_post_quantization_amd as q
        if case["op"] in ("lora", "lora_grad"):
            s["layer"] = q.LoraAdapters(s["A"], s["B"], scales=s["scales"], ranks=s["d_ranks"],
                                        x_dtype=case["x"])
        elif case["op"] in ("norm", "norm_grad"):
            s["layer"] = q.GroupNormAct(s["gamma"], s["beta"], s["groups"], eps=s["eps"],
                                        act=s["act"])
        else:
            s["layer"] = q.GradSet(s["grads"], out=s["out"])
    return s


# -------------------------------------------------------------- one pass ----

def run(state):
    case = state["case"]
    return (_run_own if own else _PLAIN[case["op"]])(case, state)


def _run_own(case, s):
    op = case["op"]
    if op == "lora":
        return s["layer"].apply(s["X"], s["d_off"], s["d_ids"], s["base"],
                                cfg=int(case["cfg"]), w=s["guidance"])
    if op == "lora_grad":
        return s["layer"].grad(s["X"], s["d_off"], s["d_ids"], s["S"], s["dY"])
    if op == "norm":
        return s["layer"].forward(s["x"], stats=case["stats"])
    if op == "norm_grad":
        return s["layer"].grad(s["dy"], s["x"], s["mean"], s["rstd"])
    return s["layer"].clip(s["max_norm"]), s["flat"]


def _plain_lora(case, s):
    out = s["base"].clone()
    h, w = out.shape[0], s["guidance"]
    for i, a in enumerate(s["ids"]):
        lo, hi = s["off"][i], s["off"][i + 1]
        if a < 0 or hi == lo:
            continue
        At, Bt = s["A"][a].float().t(), s["B"][a].float().t()
        t = s["X"][lo:hi].float() @ At
        if case["cfg"]:
            u = s["X"][h + lo:h + hi].float() @ At
            t = u + w * (t - u)
        out[lo:hi] += (t * s["scales"][a]) @ Bt
    return out


def _plain_lora_grad(case, s):
    X, dY, S = s["X"], s["dY"], s["S"]
    dX = torch.zeros(X.shape, device="cuda")
    dA = torch.zeros(s["A"].shape, device="cuda")
    dB = torch.zeros(s["B"].shape, device="cuda")
    for i, a in enumerate(s["ids"]):
        lo, hi = s["off"][i], s["off"][i + 1]
        if a < 0 or hi == lo:
            continue
        k = s["ranks"][a]
        dS = (dY[lo:hi] @ s["B"][a, :, :k].float()) * s["scales"][a]
        dX[lo:hi] = dS @ s["A"][a, :k].float()
        dA[a, :k] += dS.t() @ X[lo:hi].float()
        dB[a, :, :k] += dY[lo:hi].t() @ (S[lo:hi, :k] * s["scales"][a])
    return dX.to(X.dtype), dA.to(s["A"].dtype), dB.to(s["B"].dtype)


def _plain_norm(case, s):
    x = s["x"].float()
    B, L, C = x.shape
    G = s["groups"]
    xg = x.view(B, L, G, C // G)
    mean = xg.mean((1, 3), keepdim=True)
    rstd = torch.rsqrt((xg - mean).square().mean((1, 3), keepdim=True) + s["eps"])
    z = ((xg - mean) * rstd).view(B, L, C) * s["gamma"].float() + s["beta"].float()
    if s["act"] == "silu":
        z = z / (1.0 + torch.exp(-z))
    y = z.to(s["x"].dtype)
    return (y, mean.view(B, G), rstd.view(B, G)) if case["stats"] else y


def _plain_norm_grad(case, s):
    x, dy = s["x"].float(), s["dy"].float()
    B, L, C = x.shape
    G = s["groups"]
    n = L * (C // G)
    gamma = s["gamma"].float()
    rstd = s["rstd"].view(B, 1, G, 1)
    xhat = ((x.view(B, L, G, C // G) - s["mean"].view(B, 1, G, 1)) * rstd).view(B, L, C)
    dz = dy
    if s["act"] == "silu":
        z = xhat * gamma + s["beta"].float()
        sig = 1.0 / (1.0 + torch.exp(-z))
        dz = dy * (sig * (1.0 + z * (1.0 - sig)))
    dgamma = (dz * xhat).sum((0, 1))
    dbeta = dz.sum((0, 1))
    t = (dz * gamma).view(B, L, G, C // G)
    xh = xhat.view(B, L, G, C // G)
    s1 = t.sum((1, 3), keepdim=True) / n
    s2 = (t * xh).sum((1, 3), keepdim=True) / n
    dx = (rstd * (t - s1 - xh * s2)).view(B, L, C)
    return dx.to(s["x"].dtype), dgamma.to(s["gamma"].dtype), dbeta.to(s["beta"].dtype)


def _plain_clip(case, s):
    total = torch.stack([t.float().square().sum() for t in s["grads"]]).sum()
    norm = torch.sqrt(total)
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    for t, o in zip(s["grads"], s["out"]):
        o.copy_(t.float() * coef)
    return norm, s["flat"]


_PLAIN = {"lora": _plain_lora, "lora_grad": _plain_lora_grad, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad, "clip": _plain_clip}


# ---------------------------------------------------------------- 64 bits ----

def exact(case, seed):
    """The definitions in 64 bits, by other routes than the plain forms: the
    adapters through the full-width weight change scale B A, the norm's
    gradients by differentiating its definition, the norm of one long vector."""
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("lora", "lora_grad"):
        X = s["X"].double()
        delta = [float(s["scales"][a]) * (s["B"][a, :, :k].double() @ s["A"][a, :k].double())
                 for a, k in enumerate(s["ranks"])]
        spans = [(s["off"][i], s["off"][i + 1], a) for i, a in enumerate(s["ids"]) if a >= 0]
        if op == "lora":
            Y = s["base"].double()
            h, w = Y.shape[0], s["guidance"]
            if case["cfg"]:
                X = w * X[:h] + (1.0 - w) * X[h:]
            for lo, hi, a in spans:
                Y[lo:hi] += X[lo:hi] @ delta[a].t()
            return Y
        dY = s["dY"].double()
        dX, dA, dB = (torch.zeros(s[k].shape, dtype=torch.float64, device="cuda")
                      for k in ("X", "A", "B"))
        for lo, hi, a in spans:
            k, c = s["ranks"][a], float(s["scales"][a])
            dX[lo:hi] = dY[lo:hi] @ delta[a]
            dA[a, :k] += c * ((dY[lo:hi] @ s["B"][a, :, :k].double()).t() @ X[lo:hi])
            # the saved product is an input here, with the rounding it was saved with
            dB[a, :, :k] += c * (dY[lo:hi].t() @ s["S"][lo:hi, :k].double())
        return dX, dA, dB
    if op in ("norm", "norm_grad"):
        B, L, C = s["x"].shape
        G = s["groups"]
        train = op == "norm_grad"
        x = s["x"].double().requires_grad_(train)
        gamma = s["gamma"].double().requires_grad_(train)
        beta = s["beta"].double().requires_grad_(train)
        xg = x.reshape(B, L, G, C // G).permute(0, 2, 1, 3).reshape(B, G, -1)
        var, mean = torch.var_mean(xg, 2, correction=0)
        rstd = 1.0 / torch.sqrt(var + s["eps"])
        xh = (xg - mean[..., None]) * rstd[..., None]
        z = xh.reshape(B, G, L, C // G).permute(0, 2, 1, 3).reshape(B, L, C) * gamma + beta
        y = z * torch.sigmoid(z) if s["act"] == "silu" else z
        if not train:
            return (y, mean, rstd) if case["stats"] else y
        return torch.autograd.grad(y, (x, gamma, beta), s["dy"].double())
    flat = torch.cat([t.reshape(-1) for t in s["grads"]]).double()
    norm = torch.linalg.vector_norm(flat)
    coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return norm, flat * coef

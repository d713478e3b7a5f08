"""What a conditioned transformer block computes between its quantized linears,
as measured cases.

Three operators, each in its plain form (elementary torch operations in 32
bits) and through the package's own entry points:

  * the modulation linear on few rows: 4-bit weight codes with a scale for each
    group of input channels, SiLU on the input, a bias on the output;
  * norms of queries and keys for each head with the rotation by positions of
    several axes (time, height, width) in the same pass, forward and backward;
  * attention to an encoder's states of another length, forward and backward.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}


def listed():
    return [
        # One guided image: its two conditioning vectors through the modulation
        # linear of a block of hidden size 1152 (six vectors): latency.
        dict(name="rows4_pair", op="rows4", rows=2, K=1152, N=6912, group=128, x="f32", s="f32",
             act="silu", bias=True),
        # Eight images at once through a wide modulation linear, small groups.
        dict(name="rows4_wide", op="rows4", rows=8, K=4096, N=24576, group=64, x="bf16", s="bf16",
             act="silu", bias=True),
        # A short prompt's 77 states through a projection with an odd output width.
        dict(name="rows4_text", op="rows4", rows=77, K=4608, N=1151, group=32, x="f32", s="f32",
             act="none", bias=False),
        # A guided image's tokens behind the qkv linear: 16 x 16 positions of two axes,
        # 16 heads of 72, from the linear's 32 bits to bf16.
        dict(name="heads_image", op="heads", batch=2, positions=256, q_heads=16, kv_heads=16,
             dim=72, axes="36 36", grid="16 16", shared=True, pairs="adjacent", x="f32",
             y="bf16", norm=True),
        # One clip: 13 frames of 30 x 45 positions, three axes, an eighth of the keys' heads.
        dict(name="heads_video", op="heads", batch=1, positions=17550, q_heads=32, kv_heads=4,
             dim=128, axes="16 56 56", grid="13 30 45", shared=True, pairs="halves",
             x="bf16", y="bf16", norm=True),
        # Training at the block's own sizes, 32 bits.
        dict(name="heads_grad_image", op="heads_grad", batch=8, positions=256, q_heads=16,
             kv_heads=16, dim=72, axes="36 36", grid="16 16", shared=True, pairs="adjacent",
             x="f32", y="f32", norm=True),
        # Training on large images, each packed with positions of its own.
        dict(name="heads_grad_large", op="heads_grad", batch=4, positions=4608, q_heads=16,
             kv_heads=16, dim=128, axes="16 56 56", grid="2 48 48", shared=False,
             pairs="adjacent", x="bf16", y="bf16", norm=True),
        # One pooling token an image that looks over 4608 states: single-token latency.
        dict(name="attn_token", op="attn", batch=4, q_len=1, k_len=4608, heads=16, kv_heads=16,
             dim=64, x="bf16", mask="none", size_seed=0, save=False),
        # An image's tokens look at padded prompts of unlike lengths.
        dict(name="attn_text", op="attn", batch=16, q_len=1024, k_len=120, heads=16, kv_heads=16,
             dim=72, x="bf16", mask="lens", size_seed=1, save=False),
        # Image tokens look at the image's and the prompt's states together.
        dict(name="attn_joint", op="attn", batch=2, q_len=4096, k_len=4608, heads=16, kv_heads=16,
             dim=128, x="bf16", mask="none", size_seed=0, save=True),
        # Training on prompts at the block's own sizes, 32 bits, prompts with holes.
        dict(name="attn_grad_text", op="attn_grad", batch=8, q_len=256, k_len=77, heads=16,
             kv_heads=16, dim=72, x="f32", mask="holes", size_seed=2, save=True),
        # Training on a clip's tokens against a long prompt, heads shared by two.
        dict(name="attn_grad_large", op="attn_grad", batch=2, q_len=8190, k_len=512, heads=16,
             kv_heads=8, dim=128, x="bf16", mask="lens", size_seed=3, save=True),
    ]


# ------------------------------------------------------------------ sizes ----

def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _ints(text):
    return [int(v) for v in text.split()]


def _text(ints):
    return " ".join(str(v) for v in ints)


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e14)


def _shape_of_heads(rng):
    dim = rng.choice([40, 64, 64, 72, 72, 80, 96, 128, 128, 160])
    kv = rng.choice([1, 2, 4, 8, 16])
    return dim, kv, kv * rng.choice([1, 1, 1, 2, 4])


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    op = rng.choice(["rows4", "heads", "heads_grad", "attn", "attn", "attn_grad"])
    while True:
        x = rng.choice(["f32", "bf16"])
        if op == "rows4":
            case = dict(op=op, rows=_log(rng, 1, 80), K=16 * _log(rng, 8, 512),
                        N=_log(rng, 64, 24576), group=rng.choice([32, 64, 128]), x=x,
                        s=rng.choice(["f32", "bf16"]), act=rng.choice(["silu", "none"]),
                        bias=rng.random() < 0.7)
        elif op in ("heads", "heads_grad"):
            dim, kv, q = _shape_of_heads(rng)
            left, axes = dim // 2, []
            for _ in range(rng.randint(1, 3)):
                axes.append(2 * rng.randint(1, max(1, left - 2)))
                left -= axes[-1] // 2
                if left < 3:
                    break
            grid = [_log(rng, 1, 48) for _ in axes]
            case = dict(op=op, batch=rng.randint(1, 16), positions=math.prod(grid), q_heads=q,
                        kv_heads=kv, dim=dim, axes=_text(axes), grid=_text(grid),
                        shared=rng.random() < 0.5,
                        pairs=rng.choice(["adjacent", "halves"]), x=x,
                        y=rng.choice([x, "bf16"]), norm=rng.random() < 0.8)
        else:
            dim, kv, q = _shape_of_heads(rng)
            case = dict(op=op, batch=rng.randint(1, 16), q_len=_log(rng, 1, 8192),
                        k_len=_log(rng, 1, 8192), heads=q, kv_heads=kv, dim=dim, x=x,
                        mask=rng.choice(["none", "lens", "holes"]),
                        size_seed=rng.randrange(1 << 30), save=op == "attn_grad" or
                        rng.random() < 0.3)
        if _cost(case) <= top[op]:
            return case


def _lens(case):
    """Keys of each sequence: all, or at random from one to all (one has all)."""
    n = case["k_len"]
    if case["mask"] != "lens":
        return [n] * case["batch"]
    lens = np.random.RandomState(case["size_seed"]).randint(1, n + 1, case["batch"])
    lens[0] = n
    return [int(v) for v in lens]


def work(case):
    op = case["op"]
    if op == "rows4":
        M, K, N = case["rows"], case["K"], case["N"]
        groups = -(-K // case["group"])
        return {"bytes": N * K // 2 + N * groups * _SIZE[case["s"]] + M * K * _SIZE[case["x"]]
                + M * N * 4 + (N * 4 if case["bias"] else 0), "flops": 2 * M * N * K}
    if op in ("heads", "heads_grad"):
        tokens = case["batch"] * case["positions"]
        n = tokens * case["dim"] * (case["q_heads"] + 2 * case["kv_heads"])
        pos = (1 if case["shared"] else case["batch"]) * case["positions"] * len(_ints(case["axes"])) * 4
        x, y = _SIZE[case["x"]], _SIZE[case["y"]]
        back = op == "heads_grad"
        return {"bytes": n * ((2 * x + y) if back else (x + y)) + pos, "flops": n * (16 if back else 8)}
    B, H, G, D, size = case["batch"], case["heads"], case["kv_heads"], case["dim"], _SIZE[case["x"]]
    q, keys = B * case["q_len"] * H * D, sum(_lens(case))
    products = case["q_len"] * H * keys * D
    lse = 4 * B * case["q_len"] * H if case["save"] else 0
    if op == "attn":
        return {"bytes": (2 * q + 2 * keys * G * D) * size + lse, "flops": 4 * products}
    return {"bytes": (4 * q + 2 * keys * G * D + 2 * B * case["k_len"] * G * D) * size + lse,
            "flops": 10 * products}


# ----------------------------------------------------------------- inputs ----

def _positions(case):
    """int32 [positions, axes]: the grid's points in order, an offset for each batch
    entry where it has positions of its own."""
    mesh = torch.meshgrid(*[torch.arange(n) for n in _ints(case["grid"])], indexing="ij")
    pos = torch.stack([m.reshape(-1) for m in mesh], 1).to(torch.int32)
    if not case["shared"]:
        first = torch.arange(case["batch"], dtype=torch.int32).view(-1, 1, 1) * 1009
        pos = pos + first
    return pos.contiguous().cuda()


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed & ((1 << 62) - 1))

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g)
        return t.to(dtype)

    op = case["op"]
    if op == "rows4":
        M, K, N = case["rows"], case["K"], case["N"]
        groups = -(-K // case["group"])
        # codes of normal weights, whose largest of a group is near 7
        codes = torch.clamp(torch.round(normal(N, K, std=2.6)), -7, 7).to(torch.int8)
        scales = (normal(N, groups).abs() * 0.3 + 0.7) * (0.02 / 2.6)
        return dict(codes=codes, scales=scales.to(_DT[case["s"]]), X=normal(M, K, dtype=_DT[case["x"]]),
                    bias=normal(N, std=0.1) if case["bias"] else None)
    if op in ("heads", "heads_grad"):
        B, L, D = case["batch"], case["positions"], case["dim"]
        Hq, Hk = case["q_heads"], case["kv_heads"]
        x = normal(B, L, Hq + 2 * Hk, D) * (0.3 + normal(Hq + 2 * Hk, 1).abs())  # unlike heads
        s = dict(x=x.to(_DT[case["x"]]).view(B, L, -1), pos=_positions(case), gamma_q=None,
                 gamma_k=None)
        if case["norm"]:
            s["gamma_q"] = normal(D, mean=1.0, std=0.2)
            s["gamma_k"] = normal(D, mean=1.0, std=0.2)
        if op == "heads_grad":
            y = _DT[case["y"]]
            s["dy"] = [normal(B, L, h, D, dtype=y, std=1e-2) for h in (Hq, Hk, Hk)]
        return s
    B, H, G, D, t = case["batch"], case["heads"], case["kv_heads"], case["dim"], _DT[case["x"]]
    s = dict(q=normal(B, case["q_len"], H, D, dtype=t, std=1.5), lens=None, mask=None,
             k=normal(B, case["k_len"], G, D, dtype=t, std=1.5),
             v=normal(B, case["k_len"], G, D, dtype=t))
    if case["mask"] == "lens":
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device="cuda")
    if case["mask"] == "holes":
        s["mask"] = torch.rand(B, case["k_len"], generator=g, device="cuda") < 0.8
        s["mask"][:, 0] = True
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op in ("heads", "heads_grad"):
        s["pairs"] = [torch.tensor(p, device="cuda") for p in _pairs(case)]
    if op == "attn_grad":
        s["out"], s["lse"] = _attend(case, s)  # as the forward call saved them
        s["dout"] = torch.randn(s["q"].shape, device="cuda", generator=torch.Generator(
            device="cuda").manual_seed(1 + (seed & ((1 << 62) - 1)))).mul_(1e-2).to(s["q"].dtype)
    if own:
        import bit_post_quantization_amd as q
        if op == "rows4":
            s["layer"] = q.GroupLinear4.from_codes(s["codes"], s["scales"], case["group"],
                                                   bias=s["bias"], act=case["act"])
        elif op in ("heads", "heads_grad"):
            s["layer"] = q.HeadNormRope(
                (case["q_heads"], case["kv_heads"], case["kv_heads"]), case["dim"],
                gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], norm="rms" if case["norm"] else "none",
                axes=_ints(case["axes"]), pairs=case["pairs"], y_dtype=case["y"])
        else:
            s["layer"] = q.CrossAttention(case["heads"], case["dim"], kv_heads=case["kv_heads"])
    return s


# -------------------------------------------------------------- one pass ----

def run(state):
    case = state["case"]
    return (_run_own if own else _PLAIN[case["op"]])(case, state)


def _run_own(case, s):
    op = case["op"]
    if op == "rows4":
        return s["layer"].apply(s["X"])
    if op == "heads":
        return s["layer"].forward(s["x"], s["pos"])
    if op == "heads_grad":
        dx, *dgammas = s["layer"].grad(s["dy"], s["x"], s["pos"])
        return (dx, *dgammas) if case["norm"] else (dx,)
    if op == "attn":
        return s["layer"].forward(s["q"], s["k"], s["v"], lens=s["lens"], mask=s["mask"],
                                  save=case["save"])
    return s["layer"].grad(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], lens=s["lens"],
                           mask=s["mask"])


def _plain_rows4(case, s):
    x = s["X"].float()
    if case["act"] == "silu":
        x = x / (1.0 + torch.exp(-x))
    K = case["K"]
    scales = s["scales"].float().repeat_interleave(case["group"], 1)[:, :K]
    y = x @ (s["codes"].float() * scales).t()
    return y if s["bias"] is None else y + s["bias"]


def _pairs(case):
    """Channels of the first and second members of all pairs: a plan, made once."""
    first, second, at = [], [], 0
    for d in _ints(case["axes"]):
        h = d // 2
        for i in range(h):
            first.append(at + (2 * i if case["pairs"] == "adjacent" else i))
            second.append(at + (2 * i + 1 if case["pairs"] == "adjacent" else h + i))
        at += d
    return first, second


def _angles(case, pos):
    """Radians [..., positions, pairs], in 64 bits: position times 10000^(-2 i / d)."""
    parts = []
    for a, d in enumerate(_ints(case["axes"])):
        f = 10000.0 ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device="cuda") / d)
        parts.append(pos[..., a:a + 1].double() * f)
    return torch.cat(parts, -1)


def _rotate(pairs, t, cos, sin):
    first, second = pairs
    out = t.clone()
    a, b = t[..., first], t[..., second]
    out[..., first] = a * cos - b * sin
    out[..., second] = a * sin + b * cos
    return out


def _plain_heads(case, s):
    B, L, D = case["batch"], case["positions"], case["dim"]
    Hq, Hk, y = case["q_heads"], case["kv_heads"], _DT[case["y"]]
    x = s["x"].view(B, L, -1, D).float()
    angle = _angles(case, s["pos"])
    cos, sin = (f(angle).float().unsqueeze(-2) for f in (torch.cos, torch.sin))
    outs = []
    for t, gamma in ((x[:, :, :Hq], s["gamma_q"]), (x[:, :, Hq:Hq + Hk], s["gamma_k"])):
        if case["norm"]:
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * gamma
        outs.append(_rotate(s["pairs"], t, cos, sin).to(y))
    return (*outs, x[:, :, Hq + Hk:].to(y))


def _plain_heads_grad(case, s):
    B, L, D = case["batch"], case["positions"], case["dim"]
    Hq, Hk = case["q_heads"], case["kv_heads"]
    x = s["x"].view(B, L, -1, D).float()
    angle = _angles(case, s["pos"])
    cos, sin = (f(angle).float().unsqueeze(-2) for f in (torch.cos, torch.sin))
    dx, dgammas = [], []
    for t, gamma, dy in ((x[:, :, :Hq], s["gamma_q"], s["dy"][0]),
                         (x[:, :, Hq:Hq + Hk], s["gamma_k"], s["dy"][1])):
        dn = _rotate(s["pairs"], dy.float(), cos, -sin)
        if case["norm"]:
            rstd = torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)
            hat = t * rstd
            dgammas.append((dn * hat).sum((0, 1, 2)))
            dn = dn * gamma
            dn = rstd * (dn - hat * (dn * hat).mean(-1, keepdim=True))
        dx.append(dn)
    dx.append(s["dy"][2].float())
    return (torch.cat(dx, 2).view(B, L, -1).to(s["x"].dtype), *dgammas)


def _allowed(case, s):
    """Truth values [B, 1, 1, k_len] of the keys that count, or None."""
    if s["lens"] is not None:
        keys = torch.arange(case["k_len"], device="cuda")
        return (keys < s["lens"][:, None])[:, None, None]
    return None if s["mask"] is None else s["mask"][:, None, None]


def _by_head(t, heads):
    """[B, L, G, D] in 32 bits by head, [B, heads, L, D]: shared heads repeated."""
    return t.float().repeat_interleave(heads // t.shape[2], 2).transpose(1, 2).contiguous()


def _attend(case, s):
    H, D = case["heads"], case["dim"]
    q, k, v = (_by_head(s[n], H) for n in "qkv")
    score = (q @ k.transpose(2, 3).contiguous()).mul_(D ** -0.5)
    ok = _allowed(case, s)
    if ok is not None:
        score.masked_fill_(~ok, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p @ v).div_(total).transpose(1, 2).contiguous().to(s["q"].dtype)
    return out, (top + torch.log(total)).squeeze(-1)


def _plain_attn(case, s):
    out, lse = _attend(case, s)
    return (out, lse) if case["save"] else out


def _plain_attn_grad(case, s):
    B, H, G, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    q, k, v, do, out = (_by_head(s[n], H) for n in ("q", "k", "v", "dout", "out"))
    p = (q @ k.transpose(2, 3).contiguous()).mul_(D ** -0.5)
    ok = _allowed(case, s)
    if ok is not None:
        p.masked_fill_(~ok, float("-inf"))
    p = p.sub_(s["lse"].unsqueeze(-1)).exp_()
    dv = p.transpose(2, 3).contiguous() @ do
    ds = do @ v.transpose(2, 3).contiguous()
    ds = ds.sub_((do * out).sum(-1, keepdim=True)).mul_(p).mul_(D ** -0.5)
    dq = (ds @ k).transpose(1, 2).contiguous()
    dk = ds.transpose(2, 3).contiguous() @ q
    dk, dv = (t.view(B, G, H // G, -1, D).sum(2).transpose(1, 2).contiguous() for t in (dk, dv))
    return tuple(t.to(s["q"].dtype) for t in (dq, dk, dv))


_PLAIN = {"rows4": _plain_rows4, "heads": _plain_heads, "heads_grad": _plain_heads_grad,
          "attn": _plain_attn, "attn_grad": _plain_attn_grad}


# ---------------------------------------------------------------- 64 bits ----

def exact(case, seed):
    """The definitions in 64 bits, by other routes than the plain forms: the 4-bit
    product group by group, the rotation as a complex product and its gradients
    by differentiation, attention and its gradients one sequence and head at a time."""
    op = case["op"]
    if op == "rows4":
        s = _inputs(case, seed)
        x = s["X"].double()
        if case["act"] == "silu":
            x = x * torch.sigmoid(x)
        y = torch.zeros(case["rows"], case["N"], dtype=torch.float64, device="cuda")
        if s["bias"] is not None:
            y += s["bias"].double()
        g = case["group"]
        for i in range(s["scales"].shape[1]):
            part = x[:, i * g:(i + 1) * g] @ s["codes"][:, i * g:(i + 1) * g].double().t()
            y += part * s["scales"][:, i].double()
        return y
    if op in ("heads", "heads_grad"):
        s = _inputs(case, seed)
        return _exact_heads(case, s)
    s = prepare(case, seed)
    B, H, G, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    names = ("q", "k", "v", "out", "dout") if op == "attn_grad" else ("q", "k", "v")
    d = {n: s[n].double() for n in names}
    if op == "attn":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        lse = torch.zeros(B, H, case["q_len"], dtype=torch.float64, device="cuda")
    else:
        grads = [torch.zeros(s[n].shape, dtype=torch.float64, device="cuda") for n in "qkv"]
    lens = _lens(case)
    for b in range(B):
        keys = torch.arange(lens[b], device="cuda")
        if s["mask"] is not None:
            keys = keys[s["mask"][b]]
        for h in range(H):
            g = h * G // H
            q, k, v = d["q"][b, :, h], d["k"][b, keys, g], d["v"][b, keys, g]
            score = (q @ k.t()) / math.sqrt(D)
            if op == "attn":
                out[b, :, h] = torch.softmax(score, 1) @ v
                lse[b, h] = torch.logsumexp(score, 1)
                continue
            p = torch.softmax(score, 1)
            do = d["dout"][b, :, h]
            # the saved output is an input here, with the rounding it was saved with
            back = p * (do @ v.t() - (do * d["out"][b, :, h]).sum(1, keepdim=True)) / math.sqrt(D)
            grads[0][b, :, h] = back @ k
            grads[1][b, :, g].index_add_(0, keys, back.t() @ q)
            grads[2][b, :, g].index_add_(0, keys, p.t() @ do)
    if op == "attn":
        return (out, lse) if case["save"] else out
    return tuple(grads)


def _exact_heads(case, s):
    B, L, D = case["batch"], case["positions"], case["dim"]
    Hq, Hk = case["q_heads"], case["kv_heads"]
    train = case["op"] == "heads_grad"
    x = s["x"].double().requires_grad_(train)
    gammas = [s[n].double().requires_grad_(train) if case["norm"] else None
              for n in ("gamma_q", "gamma_k")]
    which = [(a, -2.0 * i / d) for a, d in enumerate(_ints(case["axes"])) for i in range(d // 2)]
    freqs = np.exp(math.log(10000.0) * np.array([power for _, power in which]))
    angle = s["pos"].cpu().numpy()[..., [a for a, _ in which]].astype(np.float64) * freqs
    turn = torch.from_numpy(np.cos(angle) + 1j * np.sin(angle)).cuda().unsqueeze(-2)
    first, second = _pairs(case)
    rest = [c for c in range(D) if c not in set(first + second)]
    place = torch.argsort(torch.tensor(first + second + rest, device="cuda"))
    q, k, v = x.view(B, L, -1, D).split([Hq, Hk, Hk], 2)
    outs = []
    for t, gamma in zip((q, k), gammas):
        if gamma is not None:
            t = t / torch.sqrt((t * t).sum(-1, keepdim=True) / D + 1e-6) * gamma
        z = torch.complex(t[..., first], t[..., second]) * turn
        outs.append(torch.cat([z.real, z.imag, t[..., rest]], -1)[..., place])
    outs.append(v)
    if not train:
        return tuple(outs)
    wrt = [x] + [g for g in gammas if g is not None]
    return torch.autograd.grad(outs, wrt, [t.double() for t in s["dy"]])

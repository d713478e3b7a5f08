"""The operators of a conditioned block on the GPU against their formulas in 64 bits.

Tolerances (EPS = 2^-24, half a unit in the last place of fp32; a bf16 result is
off by up to 2^-8 of itself): a sum of n products is allowed (16 + 4 sqrt(n)) EPS times
the sum of the products' magnitudes, as in the tests of the operators beside the layer.

Attention: a score's error moves its weight by as much of itself. With d_j the sum of
 - the score's own error, (16 + 4 sqrt(D)) EPS scale sum |q k_j|,
 - the rounding of the exponent's argument and of lse, 4 EPS (|s_j| + |lse|), and of exp, 8 EPS,
 - with bf16 tensors the rounding of the weight, 2^-8,
the result sum p v is off by at most sum p_j d_j |v_j| + sum p_j d_j sum p_j |v_j| (its
norm) + the sum's own (16 + 4 sqrt(Lk)) EPS sum p |v|, and the rounding of the result.
The gradients follow the same way from dS = p (dP - delta).
"""
from __future__ import annotations

import math

import numpy as np
import pytest

from tests.parity import say

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a ROCm device"
    import bit_post_quantization_amd  # noqa: F401  (fails loudly if the library is missing)
    return _t


def _dt(t, name):
    return {"f32": t.float32, "bf16": t.bfloat16}[name]


def _within(got, ref, tol, what):
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(((got - ref).abs() / tol)[bad].max()):.3g} of it")


def _round(t, ref, dtype):
    return ref.abs() * (2.0 ** -8 if dtype == t.bfloat16 else 2 * EPS)


def _sum(n):
    return (16 + 4 * math.sqrt(n)) * EPS


def _gen(t, seed):
    return t.Generator(device="cuda").manual_seed(seed)


# ----------------------------------------------------------------- 4-bit rows ----

ROWS4 = [
    # M, K, N, group, x, s, act, bias
    (1, 16, 1, 32, "f32", "f32", "none", False),
    (1, 1152, 6912, 128, "bf16", "f32", "silu", True),
    (2, 1168, 100, 64, "f32", "bf16", "silu", True),
    (3, 8192, 17, 32, "f32", "f32", "none", True),
    (16, 48, 333, 32, "bf16", "bf16", "none", False),
    (17, 272, 31, 128, "f32", "f32", "silu", False),
    (8, 1024, 16400, 64, "bf16", "bf16", "silu", True),
    (33, 2048, 96, 128, "bf16", "f32", "none", True),
    (48, 80, 160, 64, "f32", "f32", "silu", False),
    (100, 4608, 50, 32, "f32", "bf16", "none", True),
    (257, 160, 47, 128, "bf16", "bf16", "silu", False),
]


class Rows4:
    def __init__(self, t, M, K, N, group, x, s, act, bias, seed=0):
        g = _gen(t, seed)
        self.t, self.K, self.group, self.act = t, K, group, act
        self.codes = t.randint(-8, 8, (N, K), generator=g, device="cuda", dtype=t.int8)
        self.scales = (t.rand(N, -(-K // group), generator=g, device="cuda") + 0.1).to(_dt(t, s))
        self.X = t.empty(M, K, device="cuda").normal_(0, 2, generator=g).to(_dt(t, x))
        self.bias = t.empty(N, device="cuda").normal_(generator=g) if bias else None

    def layer(self):
        from bit_post_quantization_amd import GroupLinear4
        return GroupLinear4.from_codes(self.codes, self.scales, self.group, bias=self.bias,
                                       act=self.act)

    def formula(self, X=None):
        x = (self.X if X is None else X).double()
        if self.act == "silu":
            x = x / (1 + self.t.exp(-x))
        W = self.codes.double() * self.scales.double().repeat_interleave(self.group, 1)[:, :self.K]
        y, mag = x @ W.t(), x.abs() @ W.abs().t()
        if self.bias is not None:
            y, mag = y + self.bias.double(), mag + self.bias.double().abs()
        # products with exact codes; SiLU within 8 EPS of itself
        return y, (8 * EPS + _sum(self.K)) * mag


@pytest.mark.parametrize("case", ROWS4, ids=str)
def test_rows4(torch, case):
    say(f"[rows4] {case}")
    c = Rows4(torch, *case)
    layer = c.layer()
    ref, tol = c.formula()
    _within(layer.apply(c.X), ref, tol, "Y")
    codes, scales = layer.weights()
    assert torch.equal(codes, c.codes) and torch.equal(scales, c.scales)


def test_rows4_strided_rows(torch):
    c = Rows4(torch, 6, 96, 40, 32, "f32", "f32", "silu", True)
    wide = torch.full((6, 200), float("nan"), device="cuda")
    wide[:, 7:103] = c.X
    out = torch.full((9, 64), 3.0, device="cuda")
    y = c.layer().apply(wide[:, 7:103], out=out[:6, :40])
    ref, tol = c.formula()
    _within(y, ref, tol, "Y")
    assert bool((out[6:] == 3).all()) and bool((out[:, 40:] == 3).all())
    assert c.layer().apply(c.X[:0]).shape == (0, 40)


@pytest.mark.parametrize("w,s,group,K", [("f32", "f32", 128, 1152), ("bf16", "bf16", 32, 80),
                                         ("f32", "bf16", 64, 16), ("bf16", "f32", 128, 144)])
def test_rows4_quantized(torch, w, s, group, K):
    """Codes and scales of the rule: absmax / 7, half to even, ties and a group of zeros
    among them (whole numbers: equal)."""
    from bit_post_quantization_amd import GroupLinear4
    g = _gen(torch, 3)
    N = 37
    W = torch.empty(N, K, device="cuda").normal_(generator=g)
    W[3] = 0.0
    W[5, :8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -3.5, 6.5, -7.0], device="cuda")
    W[5, 8:] = 0.0
    W = W.to(_dt(torch, w))
    codes, scales = GroupLinear4(W, group=group, s_dtype=s).weights()
    groups = -(-K // group)
    pad = torch.zeros(N, groups * group, device="cuda")
    pad[:, :K] = W.float()
    pad = pad.view(N, groups, group)
    # fp32 quotients rounded correctly, as the rule says
    ref_s = (pad.abs().amax(2).cpu().numpy() / np.float32(7)).astype(np.float32)
    ref_s = torch.from_numpy(ref_s).cuda().to(_dt(torch, s))
    assert torch.equal(scales, ref_s)
    d = ref_s.float().unsqueeze(2).cpu().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(d > 0, np.rint(pad.cpu().numpy() / d), 0)
    ref = torch.from_numpy(np.clip(q, -7, 7).astype(np.int8)).view(N, -1)[:, :K]
    assert torch.equal(codes.cpu(), ref)


def test_rows4_values_not_finite(torch):
    """A row of X with an infinity or a NaN spoils its own outputs and no other row's; SiLU
    has its limits at both ends."""
    c = Rows4(torch, 5, 64, 33, 32, "f32", "f32", "silu", False)
    c.codes[:, 3] = 5
    X = c.X.clone()
    X[1, 3], X[2, 3] = float("nan"), float("inf")
    X[4, :4] = torch.tensor([-1e30, -200.0, 200.0, 90.0], device="cuda")
    y = c.layer().apply(X)
    assert not bool(torch.isfinite(y[1:3]).any())
    ref, tol = c.formula(X)
    for r in (0, 3, 4):
        _within(y[r], ref[r], tol[r], f"row {r}")


# --------------------------------------------------------------- norms, turns ----

HEADS = [
    # B, L, (q, k, v heads), dim, axes, pairs, x, y, w, norm, pos
    (2, 9, (3, 3, 3), 72, (36, 36), "adjacent", "f32", "bf16", "f32", "rms", "shared"),
    (1, 1, (1, 0, 0), 8, (), "adjacent", "f32", "f32", "f32", "rms", "shared"),
    (3, 65, (4, 2, 2), 128, (16, 56, 56), "halves", "bf16", "bf16", "bf16", "rms", "own"),
    (2, 33, (2, 1, 1), 40, (10, 6, 14), "halves", "bf16", "f32", "f32", "rms", "float"),
    (2, 33, (2, 1, 1), 40, (10, 6, 14), "adjacent", "bf16", "f32", "f32", "none", "own"),
    (1, 130, (16, 16, 16), 64, (64,), "halves", "f32", "f32", "bf16", "none", "shared"),
    (2, 17, (0, 5, 5), 96, (2, 2, 2, 90), "adjacent", "bf16", "bf16", "f32", "rms", "own"),
    (4, 7, (0, 0, 3), 160, (), "adjacent", "f32", "bf16", "f32", "rms", "shared"),
    (1, 600, (8, 1, 1), 160, (40, 60, 60), "halves", "f32", "bf16", "f32", "rms", "shared"),
    (2, 50, (1, 1, 0), 80, (24, 16), "halves", "f32", "f32", "f32", "rms", "float"),
    (1, 3000, (1, 1, 1), 24, (8, 8), "adjacent", "bf16", "bf16", "f32", "rms", "shared"),
]


class Heads:
    """Inputs, the formula by pairs in 64 bits, and error bounds."""

    def __init__(self, t, B, L, heads, dim, axes, pairs, x, y, w, norm, pos, seed=0):
        g = _gen(t, seed)
        self.t, self.B, self.L, self.heads, self.dim, self.axes = t, B, L, heads, dim, axes
        self.norm, self.y, self.pairs = norm, y, pairs
        self.x = t.empty(B, L, sum(heads) * dim, device="cuda").normal_(0, 1.5, generator=g)
        self.x = self.x.to(_dt(t, x))
        self.gq = self.gk = None
        if norm == "rms":
            self.gq, self.gk = (t.empty(dim, device="cuda").normal_(1, 0.3, generator=g)
                                .to(_dt(t, w)) for _ in range(2))
        shape = (B, L, len(axes)) if pos == "own" else (L, len(axes))
        self.pos = t.randint(-50, 100000, shape, generator=g, device="cuda", dtype=t.int32)
        if pos == "float":
            self.pos = self.pos.float() / 8
        if not axes:
            self.pos = None
        self.dy = [t.empty(B, L, h, dim, device="cuda").normal_(generator=g).to(_dt(t, y))
                   if h else None for h in heads]
        first, second, angle, at = [], [], [], 0
        for a, d in enumerate(axes):
            for i in range(d // 2):
                first.append(at + (2 * i if pairs == "adjacent" else i))
                second.append(at + (2 * i + 1 if pairs == "adjacent" else d // 2 + i))
                angle.append(self.pos[..., a].double() * 10000.0 ** (-2.0 * i / d))
            at += d
        self.first, self.second = first, second
        if axes:
            angle = t.stack(angle, -1)
            angle = (angle if pos == "own" else angle.expand(B, *angle.shape)).unsqueeze(2)
            self.cos, self.sin = t.cos(angle), t.sin(angle)

    def layer(self):
        from bit_post_quantization_amd import HeadNormRope
        return HeadNormRope(self.heads, self.dim, gamma_q=self.gq, gamma_k=self.gk, norm=self.norm,
                            axes=self.axes, pairs=self.pairs, y_dtype=self.y)

    def split(self, x):
        return x.view(self.B, self.L, -1, self.dim).split(list(self.heads), 2)

    def turn(self, n, back=False, size=False):
        if not self.axes:
            return n
        out = n.clone()
        a, b = n[..., self.first], n[..., self.second]
        if size:  # of both products
            out[..., self.first] = out[..., self.second] = a.abs() + b.abs()
            return out
        s = -self.sin if back else self.sin
        out[..., self.first] = a * self.cos - b * s
        out[..., self.second] = a * s + b * self.cos
        return out

    def formula(self, x):
        outs = []
        for i, n in enumerate(self.split(x)):
            if self.norm == "rms" and i < 2:
                n = n / self.t.sqrt((n * n).mean(-1, keepdim=True) + 1e-6)
                n = n * (self.gq, self.gk)[i].double()
            outs.append(n if i == 2 else self.turn(n))
        return outs

    def bounds(self):
        """Each factor of a result (norm, turn, product) within a few EPS of itself: 32
        EPS of the pair's size."""
        outs = []
        for i, n in enumerate(self.split(self.x.double())):
            if self.norm == "rms" and i < 2:
                n = n / self.t.sqrt((n * n).mean(-1, keepdim=True) + 1e-6)
                n = n * (self.gq, self.gk)[i].double()
            outs.append(n.abs() * 0 if i == 2 else 32 * EPS * self.turn(n.abs(), size=True))
        return outs

    def grads(self):
        """((dx, dgamma_q, dgamma_k), bounds) by the formula."""
        t = self.t
        dxs, tols, dg, dgt = [], [], [], []
        for i, x in enumerate(self.split(self.x.double())):
            if not self.heads[i]:
                if i < 2:
                    dg.append(t.zeros(self.dim, device="cuda", dtype=t.float64))
                    dgt.append(dg[-1])
                continue
            dy = self.dy[i].double()
            if i == 2:
                dxs.append(dy)
                tols.append(dy * 0)
                continue
            dn, size = self.turn(dy, back=True), self.turn(dy.abs(), size=True).abs()
            if self.norm != "rms":
                dxs.append(dn)
                tols.append(32 * EPS * size)
                continue
            gamma = (self.gq, self.gk)[i].double()
            r = 1 / t.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            hat = x * r
            dg.append((dn * hat).sum((0, 1, 2)))
            dgt.append((32 * EPS + _sum(hat.numel() / self.dim)) * (size * hat.abs()).sum((0, 1, 2)))
            u, us = dn * gamma, size * gamma.abs()
            dxs.append(r * (u - hat * (u * hat).mean(-1, keepdim=True)))
            tols.append((48 * EPS + _sum(self.dim)) * r *
                        (us + hat.abs() * (us * hat.abs()).mean(-1, keepdim=True)))
        cat = lambda v: t.cat(v, 2).view(self.B, self.L, -1)  # noqa: E731
        return [cat(dxs)] + dg, [cat(tols)] + dgt


@pytest.mark.parametrize("case", HEADS, ids=str)
def test_heads(torch, case):
    say(f"[heads] {case}")
    c = Heads(torch, *case)
    outs = c.layer().forward(c.x, c.pos)
    for got, ref, tol, h in zip(outs, c.formula(c.x.double()), c.bounds(), c.heads):
        if h == 0:
            assert got is None
            continue
        assert got.dtype == _dt(torch, c.y)
        _within(got, ref, tol + _round(torch, ref, got.dtype), "y")


@pytest.mark.parametrize("case", HEADS, ids=str)
def test_heads_grad(torch, case):
    say(f"[heads grad] {case}")
    c = Heads(torch, *case)
    dx, dgq, dgk = c.layer().grad(c.dy, c.x, c.pos)
    ref, tol = c.grads()
    _within(dx, ref[0], tol[0] + _round(torch, ref[0], dx.dtype), "dx")
    if c.norm == "rms":
        for got, r, e, name in zip((dgq, dgk), ref[1:], tol[1:], ("dgamma_q", "dgamma_k")):
            _within(got, r, e + _round(torch, r, got.dtype), name)
    else:
        assert dgq is None and dgk is None


def test_heads_grad_differences(torch):
    """The gradient along a direction against the formula's central difference."""
    c = Heads(torch, 2, 9, (3, 2, 2), 72, (36, 20), "halves", "f32", "f32", "f32", "rms", "own")
    dx, dgq, dgk = c.layer().grad(c.dy, c.x, c.pos)
    g = _gen(torch, 9)
    u = torch.empty_like(c.x).normal_(generator=g).double()
    v = torch.empty_like(c.gq).normal_(generator=g).double()
    h, x, gq, gk = 1e-5, c.x.double(), c.gq, c.gk

    def loss(s):
        c.gq, c.gk = gq.double() + s * v, gk.double() + s * v
        return sum(float((o * d.double()).sum()) for o, d in zip(c.formula(x + s * u), c.dy))

    slope = (loss(h) - loss(-h)) / (2 * h)
    c.gq, c.gk = gq, gk
    got = float((dx.double() * u).sum() + ((dgq + dgk).double() * v).sum())
    _, tol = c.grads()
    size = float((dx.double() * u).abs().sum())
    bound = float((tol[0] * u.abs()).sum() + ((tol[1] + tol[2]) * v.abs()).sum()) + 1e-7 * size
    assert abs(got - slope) <= bound, (got, slope, bound)


def test_heads_into_slices(torch):
    """Into a joint sequence's slice by head-major strides, from a slice of a wider row, and
    from rows that no vector load is aligned to."""
    c = Heads(torch, 2, 21, (3, 2, 2), 64, (32, 16), "halves", "f32", "bf16", "f32", "rms", "own")
    ref, tol = c.formula(c.x.double()), c.bounds()
    joint = [torch.full((2, h, 40, 64), 7.0, dtype=torch.bfloat16, device="cuda") for h in c.heads]
    parts = [j.transpose(1, 2)[:, 11:32] for j in joint]
    outs = c.layer().forward(c.x, c.pos, out=parts)
    for o, r, e, j in zip(outs, ref, tol, joint):
        _within(o, r, e + _round(torch, r, torch.bfloat16), "joint")
        assert bool((j[:, :, :11] == 7).all()) and bool((j[:, :, 32:] == 7).all())
    wide = torch.full((2, 21, 3 + 7 * 64 + 5), float("nan"), device="cuda")
    wide[:, :, 3:-5] = c.x
    for o, r, e in zip(c.layer().forward(wide[:, :, 3:-5], c.pos), ref, tol):
        _within(o, r, e + _round(torch, r, torch.bfloat16), "unaligned")
    dx, _, _ = c.layer().grad(c.dy, wide[:, :, 3:-5], c.pos)
    assert torch.equal(dx, c.layer().grad(c.dy, c.x, c.pos)[0])
    empty = c.layer().forward(c.x[:, :0], c.pos[:, :0])
    assert empty[0].shape == (2, 0, 3, 64)


def test_heads_far_positions_and_own_freqs(torch):
    """Positions near 2^31 keep their angle to the accuracy of a turn's 53 bits."""
    from bit_post_quantization_amd import HeadNormRope
    f = [1.0, 0.37, 2.0 ** -20]
    pos = torch.tensor([[2 ** 31 - 1], [-2 ** 31], [123456789]], dtype=torch.int32, device="cuda")
    x = torch.zeros(1, 3, 8, device="cuda")
    x[..., 0:6:2] = 1.0
    q, _, _ = HeadNormRope((1, 0, 0), 8, norm="none", axes=(6,), freqs=f, y_dtype="f32").forward(x, pos)
    angle = (pos.cpu().double() * torch.tensor(f, dtype=torch.float64)).unsqueeze(0)
    got = q[0, :, 0].cpu().double().view(1, 3, 4, 2)
    # 2^31 turns have 2^-22 of a unit in the last of 53 bits; three roundings of that
    tol = 8 * EPS + 3 * 2 * math.pi * 2.0 ** 29 * 2.0 ** -53
    assert bool(((got[..., :3, 0] - angle.cos()).abs() <= tol).all())
    assert bool(((got[..., :3, 1] - angle.sin()).abs() <= tol).all())
    assert bool((got[..., 3, :] == 0).all())


# ------------------------------------------------------------------ attention ----

ATTN = [
    # B, Lq, Lk, heads, kv, dim, type, mask
    (1, 1, 1, 1, 1, 8, "f32", "none"),
    (2, 1, 700, 4, 4, 64, "bf16", "none"),
    (2, 1, 300, 8, 2, 128, "bf16", "lens"),
    (3, 5, 77, 3, 3, 40, "bf16", "holes"),
    (2, 33, 65, 2, 1, 72, "bf16", "both"),
    (2, 200, 129, 2, 2, 72, "f32", "lens"),
    (1, 129, 64, 4, 2, 96, "bf16", "none"),
    (1, 70, 511, 2, 2, 160, "bf16", "holes"),
    (1, 64, 200, 2, 1, 160, "f32", "both"),
    (2, 300, 77, 6, 3, 80, "f32", "holes"),
    (1, 260, 1000, 2, 2, 128, "f32", "none"),
    (2, 513, 333, 4, 1, 64, "bf16", "lens"),
    (1, 1500, 33, 1, 1, 24, "bf16", "none"),
    (2, 31, 2050, 2, 2, 80, "f32", "lens"),
]


class Attn:
    def __init__(self, t, B, Lq, Lk, H, G, D, dt, mask, seed=0, std=1.5):
        g = _gen(t, seed)
        dtype = _dt(t, dt)

        def normal(*s, std=1.0):
            return t.empty(s, device="cuda").normal_(0, std, generator=g).to(dtype)

        self.t, self.H, self.G, self.D, self.dtype = t, H, G, D, dtype
        self.q, self.k = normal(B, Lq, H, D, std=std), normal(B, Lk, G, D, std=std)
        self.v, self.dout = normal(B, Lk, G, D), normal(B, Lq, H, D)
        self.lens = self.mask = None
        self.ok = t.ones(B, Lk, dtype=t.bool, device="cuda")
        if mask in ("lens", "both"):  # one of no key, one of all
            lens = t.randint(0, Lk + 1, (B,), generator=g, device="cuda", dtype=t.int32)
            lens[0] = Lk
            lens[-1] = 0 if B > 1 else lens[-1]
            self.lens = lens
            self.ok &= t.arange(Lk, device="cuda") < lens[:, None]
        if mask in ("holes", "both"):
            self.mask = t.rand(B, Lk, generator=g, device="cuda") < 0.6
            self.ok &= self.mask
        for x in (self.k, self.v):  # what does not count is not used, whatever it holds
            x[~self.ok] = float("nan")
            x.view(-1, G, D)[~self.ok.reshape(-1)] = float("inf") if x is self.v else float("nan")

    def layer(self):
        from bit_post_quantization_amd import CrossAttention
        return CrossAttention(self.H, self.D, kv_heads=self.G)

    def by_head(self, x, keys=False):
        x = x.double()
        if keys:
            x = self.t.where(self.ok[:, :, None, None], x, self.t.zeros_like(x))
            x = x.repeat_interleave(self.H // self.G, 2)
        return x.transpose(1, 2).contiguous()

    def weights(self):
        """(p, lse, d): the weights, their log sums and their relative errors (above)."""
        t, D = self.t, self.D
        q, k = self.by_head(self.q), self.by_head(self.k, True)
        s = (q @ k.transpose(2, 3)) * D ** -0.5
        size = (q.abs() @ k.abs().transpose(2, 3)) * D ** -0.5
        s = s.masked_fill(~self.ok[:, None, None], -math.inf)
        lse = t.logsumexp(s, -1)
        p = t.exp(s - lse[..., None])
        p = t.where(p.isfinite(), p, t.zeros_like(p))
        fin = lambda x: t.where(x.isfinite(), x, t.zeros_like(x))  # noqa: E731
        d = _sum(D) * size + 4 * EPS * (fin(s).abs() + fin(lse).abs()[..., None]) + 8 * EPS
        return p, lse, d

    def p_rounding(self):
        return 2.0 ** -8 if self.dtype == self.t.bfloat16 else 0.0

    def forward(self):
        p, lse, d = self.weights()
        v = self.by_head(self.v, True)
        out, size = p @ v, p @ v.abs()
        dd = d + self.p_rounding()
        tol = (p * dd) @ v.abs() + (p * d).sum(-1, keepdim=True) * size + _sum(p.shape[-1]) * size
        lse_tol = (p * d).sum(-1) + 8 * EPS + 4 * EPS * lse.abs() + _sum(p.shape[-1])
        return out.transpose(1, 2), tol.transpose(1, 2), lse, lse_tol

    def grads(self, out, lse_in):
        """By the formula, from the saved out and lse."""
        t, D, sc = self.t, self.D, self.D ** -0.5
        p, lse, d = self.weights()
        q, k, v = self.by_head(self.q), self.by_head(self.k, True), self.by_head(self.v, True)
        do, o = self.by_head(self.dout), self.by_head(out)
        # the saved lse's own error moves p too
        fin = lambda x: t.where(x.isfinite(), x, t.zeros_like(x))  # noqa: E731
        d = d + fin(lse_in.double() - lse).abs()[..., None]
        r = self.p_rounding()
        R, Lk = q.shape[2] * self.H // self.G, k.shape[2]
        dv = p.transpose(2, 3) @ do
        dv_tol = (p * (d + r + _sum(R))).transpose(2, 3) @ do.abs()
        dp, dps = do @ v.transpose(2, 3), do.abs() @ v.abs().transpose(2, 3)
        delta, deltas = (do * o).sum(-1, keepdim=True), (do * o).abs().sum(-1, keepdim=True)
        ds = p * (dp - delta)
        e = p * (d * (dp - delta).abs() + _sum(D) * (dps + deltas)) + (r + 4 * EPS) * ds.abs()
        dq, dk = (ds @ k) * sc, (ds.transpose(2, 3) @ q) * sc
        dq_tol = ((e + _sum(Lk) * ds.abs()) @ k.abs()) * sc
        dk_tol = ((e + _sum(R) * ds.abs()).transpose(2, 3) @ q.abs()) * sc

        def keys(x):
            B, _, n, _ = x.shape
            return x.view(B, self.G, -1, n, D).sum(2).transpose(1, 2)

        return ((dq.transpose(1, 2), keys(dk), keys(dv)),
                (dq_tol.transpose(1, 2), keys(dk_tol), keys(dv_tol)))


def _same_lse(t, got, ref, tol):
    empty = ref == -math.inf
    assert bool((got[empty] == -math.inf).all())
    _within(got[~empty], ref[~empty], tol[~empty], "lse")


@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention(torch, case):
    say(f"[attention] {case}")
    c = Attn(torch, *case)
    out, lse = c.layer().forward(c.q, c.k, c.v, lens=c.lens, mask=c.mask, save=True)
    ref, tol, ref_lse, lse_tol = c.forward()
    _within(out, ref, tol + _round(torch, ref, out.dtype), "out")
    _same_lse(torch, lse, ref_lse, lse_tol)
    assert torch.equal(out, c.layer().forward(c.q, c.k, c.v, lens=c.lens, mask=c.mask))


@pytest.mark.parametrize("case", ATTN, ids=str)
def test_attention_grad(torch, case):
    say(f"[attention grad] {case}")
    c = Attn(torch, *case)
    out, lse = c.layer().forward(c.q, c.k, c.v, lens=c.lens, mask=c.mask, save=True)
    got = c.layer().grad(c.dout, c.q, c.k, c.v, out, lse, lens=c.lens, mask=c.mask)
    ref, tol = c.grads(out, lse)
    for g, r, e, name in zip(got, ref, tol, ("dq", "dk", "dv")):
        _within(g, r, e + _round(torch, r, g.dtype), name)
    off = ~c.ok
    assert bool((got[1][off] == 0).all()) and bool((got[2][off] == 0).all())


def test_attention_grad_differences(torch):
    """The gradients along a direction against the formula's central difference."""
    c = Attn(torch, 2, 20, 37, 4, 2, 24, "f32", "holes")
    out, lse = c.layer().forward(c.q, c.k, c.v, mask=c.mask, save=True)
    got = c.layer().grad(c.dout, c.q, c.k, c.v, out, lse, mask=c.mask)
    _, tol = c.grads(out, lse)
    g = _gen(torch, 5)
    base = [torch.where(c.ok[:, :, None, None], x, torch.zeros_like(x)).double() if i else x.double()
            for i, x in enumerate((c.q, c.k, c.v))]
    us = [torch.empty_like(x).normal_(generator=g) for x in base]

    def loss(s):
        c.q, c.k, c.v = (x + s * u for x, u in zip(base, us))
        p, _, _ = c.weights()
        return float(((p @ c.by_head(c.v, True)) * c.by_head(c.dout)).sum())

    h = 1e-5
    slope = (loss(h) - loss(-h)) / (2 * h)
    along = sum(float((a.double() * u).sum()) for a, u in zip(got, us))
    size = sum(float((a.double() * u).abs().sum()) for a, u in zip(got, us))
    bound = sum(float((e * u.abs()).sum()) for e, u in zip(tol, us)) + 1e-7 * size
    assert abs(along - slope) <= bound, (along, slope, bound)


def test_attention_layouts(torch):
    """[B, heads, L, dim] storage, slices of a fused row, one batch entry of keys for all,
    outputs and gradients into slices: the same bits as from packed tensors."""
    c = Attn(torch, 3, 50, 90, 4, 4, 72, "bf16", "none")
    c.k[:], c.v[:] = c.k[:1], c.v[:1]
    layer = c.layer()
    out, lse = layer.forward(c.q, c.k, c.v, save=True)
    dq, dk, dv = layer.grad(c.dout, c.q, c.k, c.v, out, lse)
    q = c.q.transpose(1, 2).contiguous().transpose(1, 2)
    kv = torch.cat([c.k[:1], c.v[:1]], 2)
    k, v = kv[:, :, :4].expand(3, -1, -1, -1), kv[:, :, 4:].expand(3, -1, -1, -1)
    wide = torch.full((3, 60, 4, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    o = layer.forward(q, k, v, out=wide[:, 4:54])
    assert torch.equal(o, out) and bool((wide[:, :4] == 5).all()) and bool((wide[:, 54:] == 5).all())
    fused = torch.full((3, 90, 10, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    into = (torch.empty_like(q), fused[:, :, 1:5], fused[:, :, 5:9])
    got = layer.grad(c.dout, q, k, v, o, lse, into=into)
    for a, b in zip(got, (dq, dk, dv)):
        assert torch.equal(a, b)
    assert bool((fused[:, :, 0] == 5).all()) and bool((fused[:, :, 9] == 5).all())


def test_attention_without_keys_or_queries(torch):
    layer = Attn(torch, 2, 3, 4, 2, 1, 32, "f32", "none").layer()
    e = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    out, lse = layer.forward(e(2, 3, 2, 32), e(2, 0, 1, 32), e(2, 0, 1, 32), save=True)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    dq, dk, dv = layer.grad(e(2, 3, 2, 32), e(2, 3, 2, 32), e(2, 0, 1, 32), e(2, 0, 1, 32), out, lse)
    assert bool((dq == 0).all()) and dk.shape == (2, 0, 1, 32)
    none = e(2, 0, 2, 32)
    out, lse = layer.forward(none, e(2, 4, 1, 32), e(2, 4, 1, 32), save=True)
    assert out.shape == (2, 0, 2, 32)
    dq, dk, dv = layer.grad(none, none, e(2, 4, 1, 32), e(2, 4, 1, 32), out, lse)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


@pytest.mark.parametrize("Lq,dt", [(3, "bf16"), (200, "bf16"), (40, "f32"), (200, "f32")])
def test_attention_values_not_finite(torch, Lq, dt):
    """A query with a NaN spoils its own output and no other; scores of -infinity weigh
    nothing; large scores do not overflow."""
    c = Attn(torch, 1, Lq, 150, 2, 2, 64, dt, "none")
    clean = c.layer().forward(c.q, c.k, c.v)
    c.q[0, 1, 0, 5] = float("nan")
    out = c.layer().forward(c.q, c.k, c.v)
    bad = torch.isnan(out)
    assert bool(bad[0, 1, 0].all()) and int(bad.sum()) == 64
    keep = ~bad
    assert torch.equal(out[keep], clean[keep])
    big = Attn(torch, 1, Lq, 150, 2, 2, 64, dt, "none", std=30.0)
    out, lse = big.layer().forward(big.q, big.k, big.v, save=True)
    ref, tol, ref_lse, lse_tol = big.forward()
    _within(out, ref, tol + _round(torch, ref, out.dtype), "large scores")
    _same_lse(torch, lse, ref_lse, lse_tol)
    low = Attn(torch, 1, Lq, 150, 2, 2, 64, dt, "none")
    low.q[:] = low.q.abs() + 0.1
    low.k[:, 70:90] = -math.inf
    out = low.layer().forward(low.q, low.k, low.v)
    low.ok[:, 70:90] = False
    ref, tol, _, _ = low.forward()
    _within(out, ref, tol + _round(torch, ref, out.dtype), "scores of -infinity")


def test_attention_far_offsets(torch):
    """Offsets past 2^31 elements in a long cache: a batch entry and rows far apart."""
    c = Attn(torch, 2, 40, 70, 2, 2, 64, "bf16", "lens")
    row = 1 << 25  # 70 rows of it pass 2^31
    store = torch.empty(71 * row, dtype=torch.bfloat16, device="cuda")
    far = [store.as_strided(c.k.shape, (1 << 20, row, 64, 1), at) for at in (0, 256)]
    for f, x in zip(far, (c.k, c.v)):
        f.copy_(x)
    layer = c.layer()
    out, lse = layer.forward(c.q, c.k, c.v, lens=c.lens, save=True)
    assert torch.equal(layer.forward(c.q, *far, lens=c.lens), out)
    grads = layer.grad(c.dout, c.q, c.k, c.v, out, lse, lens=c.lens)
    into = [torch.empty_like(c.q)] + [store.as_strided(c.k.shape, (1 << 20, row, 64, 1), at)
                                      for at in (512, 768)]
    for a, b in zip(layer.grad(c.dout, c.q, *far, out, lse, lens=c.lens, into=into), grads):
        assert torch.equal(a, b)
    say(f"  cache of {store.numel()} elements, offsets up to {69 * row + (1 << 20)}")


# ------------------------------------------------------------ streams, graphs ----

def _calls(t, seed):
    """A call of each operator on inputs of a seed: a function that returns all outputs,
    and the inputs it reads."""
    r = Rows4(t, 3, 2048, 64, 64, "f32", "f32", "silu", True, seed)
    h = Heads(t, 2, 40, (4, 2, 2), 64, (32, 32), "adjacent", "f32", "bf16", "f32", "rms", "own", seed)
    a = Attn(t, 2, 40, 300, 4, 2, 64, "bf16", "lens", seed)
    for x in (a.k, a.v):
        x[~a.ok] = 0
    few = Attn(t, 2, 2, 3000, 4, 2, 64, "bf16", "none", seed)
    rows, heads, attn = r.layer(), h.layer(), a.layer()

    def run():
        y = rows.apply(r.X)
        q, k, v = heads.forward(h.x, h.pos)
        dx, dgq, dgk = heads.grad(h.dy, h.x, h.pos)
        o, lse = attn.forward(a.q, a.k, a.v, lens=a.lens, save=True)
        g = attn.grad(a.dout, a.q, a.k, a.v, o, lse, lens=a.lens)
        one = attn.forward(few.q, few.k, few.v)
        return [y, q, k, v, dx, dgq, dgk, o, lse, *g, one]

    return run, [r.X, h.x, *h.dy, a.q, a.k, a.v, a.dout, few.q, few.k, few.v]


def test_same_bits_every_time(torch):
    run, _ = _calls(torch, 0)
    first = run()
    for _ in range(3):
        for a, b in zip(run(), first):
            assert torch.equal(a, b)


def test_captured_graphs(torch):
    """Two captured graphs with the operators in turn, replayed on changed inputs with
    eager work between, give what eager calls give."""
    graphs = []
    for seed in (1, 2):
        run, inputs = _calls(torch, seed)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            run()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = run()
        graphs.append((run, inputs, g, outs))
    for i in range(3):
        for run, inputs, g, outs in graphs:
            for x in inputs:
                x.mul_(0.9).add_(0.01 * i)
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, run()):
                assert torch.equal(a, b)


def test_other_stream(torch):
    """Calls on a stream behind work that makes their inputs."""
    run, inputs = _calls(torch, 4)
    ref = run()
    keep = [x.clone() for x in inputs]
    for x in inputs:
        x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        for x, k in zip(inputs, keep):
            x.copy_(k)
        outs = run()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(outs, ref):
        assert torch.equal(a, b)


def test_refusals(torch):
    """What the classes refuse before anything runs."""
    from bit_post_quantization_amd import CrossAttention, GroupLinear4, HeadNormRope, QLError
    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)  # noqa: E731
    bad = []

    def no(f):
        with pytest.raises(QLError):
            f()
        bad.append(f)

    codes, scales = z(8, 64, dtype=torch.int8), z(8, 2)
    lin = GroupLinear4.from_codes(codes, scales, 32)
    no(lambda: GroupLinear4.from_codes(codes, scales, 48))
    no(lambda: GroupLinear4.from_codes(codes, scales, 64))
    no(lambda: GroupLinear4.from_codes(codes.cpu(), scales, 32))
    no(lambda: GroupLinear4.from_codes(codes, scales, 32, bias=z(9)))
    no(lambda: GroupLinear4.from_codes(codes, scales, 32, act="gelu"))
    no(lambda: GroupLinear4(z(8, 72)))
    no(lambda: GroupLinear4(z(8, 64, dtype=torch.float16)))
    no(lambda: lin.apply(z(2, 63)))
    no(lambda: lin.apply(z(2, 64, dtype=torch.float16)))
    no(lambda: lin.apply(z(2, 64), out=z(2, 9)))
    no(lambda: lin.apply(z(2, 128)[:, ::2]))
    h = HeadNormRope((2, 1, 1), 64, gamma_q=z(64), axes=(32,))
    pos = z(5, 1, dtype=torch.int32)
    no(lambda: HeadNormRope((2, 1, 1), 60))
    no(lambda: HeadNormRope((2, 1, 1), 168))
    no(lambda: HeadNormRope((0, 0, 0), 64))
    no(lambda: HeadNormRope((2, 1, 1), 64, axes=(33,)))
    no(lambda: HeadNormRope((2, 1, 1), 64, axes=(32, 34)))
    no(lambda: HeadNormRope((2, 1, 1), 64, axes=(2,) * 5))
    no(lambda: HeadNormRope((2, 1, 1), 64, gamma_q=z(63)))
    no(lambda: HeadNormRope((2, 1, 1), 64, gamma_q=z(64), norm="none"))
    no(lambda: HeadNormRope((2, 1, 1), 64, axes=(32,), freqs=[1.0]))
    no(lambda: h.forward(z(2, 5, 255), pos))
    no(lambda: h.forward(z(2, 5, 256)))
    no(lambda: h.forward(z(2, 5, 256), z(4, 1, dtype=torch.int32)))
    no(lambda: h.forward(z(2, 5, 256), pos.long()))
    no(lambda: h.forward(z(2, 5, 256), pos, out=(z(2, 5, 2, 64),) * 3))
    a = CrossAttention(4, 64, kv_heads=2)
    q, k = z(2, 3, 4, 64), z(2, 6, 2, 64)
    no(lambda: CrossAttention(4, 64, kv_heads=3))
    no(lambda: CrossAttention(4, 60))
    no(lambda: CrossAttention(4, 64, scale=0.0))
    no(lambda: CrossAttention(4, 64, scale=float("inf")))
    no(lambda: a.forward(q, k, z(2, 7, 2, 64)))
    no(lambda: a.forward(q, k, k.bfloat16()))
    no(lambda: a.forward(q.half(), k.half(), k.half()))
    no(lambda: a.forward(q, k.cpu(), k))
    no(lambda: a.forward(q, k, k, lens=z(3, dtype=torch.int32)))
    no(lambda: a.forward(q, k, k, lens=z(2)))
    no(lambda: a.forward(q, k, k, mask=z(2, 5, dtype=torch.bool)))
    no(lambda: a.forward(q, k, k, mask=z(2, 6)))
    no(lambda: a.forward(z(2, 3, 4, 66)[..., 1:65], k, k))       # start is not 16-byte aligned
    no(lambda: a.forward(q, k, k, out=q))
    no(lambda: a.forward(q, k, k, out=z(1, 3, 4, 64).expand(2, -1, -1, -1)))
    no(lambda: a.grad(q, q, k, k, q, z(2, 4, 4)))
    no(lambda: a.grad(q, q, k, k, q, z(2, 4, 3), into=(z(2, 3, 4, 64), k, z(2, 6, 2, 64))))
    same = z(2, 6, 2, 64)
    no(lambda: a.grad(q, q, k, k, q, z(2, 4, 3), into=(z(2, 3, 4, 64), same, same)))
    say(f"  {len(bad)} calls refused")

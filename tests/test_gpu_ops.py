"""The operators beside the layer on the GPU against their formulas in 64 bits.

Tolerances (EPS = 2^-24, half a unit in the last place of fp32): a sum of n
products is allowed (16 + 4 sqrt(n)) EPS times the sum of the products'
magnitudes, four standard deviations of n independent roundings and a margin
for the order of the sum; a result rounded to bf16 gets 2^-8 of itself more.
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
    assert got.shape == ref.shape, what
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                           f"{float(((got - ref).abs() / tol)[bad].max()):.3g} of it")


def _round(t, ref, dtype):
    """What rounding to the output's type may add."""
    return ref.abs() * (2.0 ** -8 if dtype == t.bfloat16 else 2 * EPS)


# ---------------------------------------------------------------- adapters ----

class Case:
    """Inputs of one adapter call and the 64-bit values and error bounds."""

    def __init__(self, t, lens, ids, K, N, rank, x="f32", w="f32", ranks=None, cfg=False, seed=0):
        g = t.Generator(device="cuda")
        g.manual_seed(seed)

        def normal(*s, std=1.0):
            return t.empty(s, device="cuda").normal_(0, std, generator=g)

        self.t, self.lens, self.ids, self.cfg = t, lens, ids, cfg
        rows = sum(lens)
        self.M, self.K, self.N, self.rank = rows * (2 if cfg else 1), K, N, rank
        n = max([3] + [i + 1 for i in ids])
        self.n = n
        self.X = normal(self.M, K).to(_dt(t, x))
        self.A = normal(n, rank, K, std=K ** -0.5).to(_dt(t, w))
        self.B = normal(n, N, rank, std=0.5).to(_dt(t, w))
        self.scales = t.tensor([0.5 + a for a in range(n)], device="cuda")
        self.base = normal(rows, N)
        self.dY = normal(self.M, N)
        self.w = 3.5
        self.r = [rank] * n if ranks is None else [ranks[a % len(ranks)] for a in range(n)]
        self.d_ranks = None if ranks is None else t.tensor(self.r, dtype=t.int32, device="cuda")
        self.off = t.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=t.int32, device="cuda")
        self.d_ids = t.tensor(ids, dtype=t.int32, device="cuda")
        for a, k in enumerate(self.r):  # unused storage is not used, whatever it holds
            self.A[a, k:] = float("nan")
            self.B[a, :, k:] = float("inf")
        self.x_name = x

    def spans(self):
        lo = 0
        for n, i in zip(self.lens, self.ids):
            if n and 0 <= i < self.n:
                yield lo, lo + n, i, min(max(self.r[i], 0), self.rank), float(self.scales[i])
            lo += n

    def layer(self):
        from bit_post_quantization_amd import LoraAdapters
        return LoraAdapters(self.A, self.B, scales=self.scales, ranks=self.d_ranks,
                            x_dtype=self.x_name)

    def forward(self, base=True):
        """(Y, bound, S) in 64 bits."""
        t, h = self.t, sum(self.lens)
        Y = self.base.double() if base else t.zeros(h, self.N, device="cuda", dtype=t.float64)
        mag = Y.abs()
        S = t.zeros(self.M, self.rank, device="cuda", dtype=t.float64)
        X = self.X.double()
        for lo, hi, a, k, c in self.spans():
            A, B = self.A[a, :k].double(), self.B[a, :, :k].double()
            s, sm = X[lo:hi] @ A.t(), X[lo:hi].abs() @ A.abs().t()
            S[lo:hi, :k] = s
            if self.cfg:
                u, um = X[h + lo:h + hi] @ A.t(), X[h + lo:h + hi].abs() @ A.abs().t()
                S[h + lo:h + hi, :k] = u
                s, sm = u + self.w * (s - u), um + self.w * (sm + um)
            Y[lo:hi] += c * (s @ B.t())
            mag[lo:hi] += c * (sm @ B.abs().t())
        return Y, (16 + 4 * math.sqrt(self.K + self.rank)) * EPS * mag, S

    def grads(self, S):
        """((dX, dA, dB), bounds) in 64 bits, from the saved S."""
        t = self.t
        z = lambda *s: t.zeros(s, device="cuda", dtype=t.float64)  # noqa: E731
        out = [z(self.M, self.K), z(*self.A.shape), z(*self.B.shape)]
        mag = [z(*o.shape) for o in out]
        X, dY, S = self.X.double(), self.dY.double(), S.double()
        for lo, hi, a, k, c in self.spans():
            A, B = self.A[a, :k].double(), self.B[a, :, :k].double()
            dS, dm = c * (dY[lo:hi] @ B), c * (dY[lo:hi].abs() @ B.abs())
            out[0][lo:hi], mag[0][lo:hi] = dS @ A, dm @ A.abs()
            out[1][a, :k] += dS.t() @ X[lo:hi]
            mag[1][a, :k] += dm.t() @ X[lo:hi].abs()
            out[2][a, :, :k] += c * (dY[lo:hi].t() @ S[lo:hi, :k])
            mag[2][a, :, :k] += c * (dY[lo:hi].abs().t() @ S[lo:hi, :k].abs())
        n = (self.N + self.rank, self.N + self.M, self.M)
        return out, [(16 + 4 * math.sqrt(v)) * EPS * m for v, m in zip(n, mag)]


LORA = [
    # lens, ids, K, N, rank, x, w, ranks, cfg
    ([1], [0], 16, 1, 1, "f32", "f32", None, False),
    ([1, 1, 1, 1, 1], [0, 2, -1, 1, 2], 1152, 96, 16, "bf16", "bf16", None, False),
    ([5, 0, 17, 1, 40], [1, 0, -1, 2, 1], 64, 37, 5, "f32", "bf16", None, False),
    ([16, 15, 33, 64], [0, 1, 2, 0], 48, 130, 31, "bf16", "f32", (31, 7, 16), False),
    ([0, 0, 70, 0], [5, 1, 2, 0], 144, 68, 64, "bf16", "bf16", (64, 1, 33), False),
    ([65, 127], [1, 0], 2320, 257, 128, "f32", "f32", (128, 100), False),
    ([130, 2], [0, 1], 512, 100, 72, "bf16", "bf16", None, False),
    ([20, 1, 0, 44], [0, -1, 1, 2], 80, 52, 12, "f32", "f32", (12, 0, 4), True),
    ([3, 90], [2, 1], 1040, 33, 33, "bf16", "bf16", None, True),
    ([300], [0], 176, 200, 16, "f32", "bf16", None, False),
    ([1] * 70 + [9] * 70, list(range(5)) * 28, 32, 20, 8, "bf16", "bf16", (8, 3), False),
    ([7] * 3, [99, -7, 1], 32, 20, 8, "f32", "f32", None, False),
    ([1] * 300 + [0] * 250 + [2, 40] * 60, list(range(-1, 4)) * 134, 32, 24, 8, "f32", "bf16", None, False),
    ([2049], [1], 64, 4112, 16, "bf16", "f32", (7, 16), False),          # two launches, an odd tail
    ([700, 0, 1500], [0, 1, -1], 96, 4100, 40, "f32", "bf16", None, True),
    ([600, 1537, 1], [2, 0, 1], 80, 4099, 70, "bf16", "bf16", (70, 3), False),
]


@pytest.mark.parametrize("case", LORA, ids=range(len(LORA)))
def test_lora_forward(torch, case):
    say(f"[lora] {case}")
    c = Case(torch, *case)
    L = c.layer()
    args = (c.X, c.off, c.d_ids)
    kw = dict(cfg=int(c.cfg), w=c.w)
    ref, tol, S_ref = c.forward()
    got, S = L.apply(*args, c.base, save=True, **kw)
    torch.cuda.synchronize()
    _within(got, ref, tol + 2 * EPS * ref.abs(), "Y")
    mag = c.X.double().abs().sum(1, keepdim=True) * float(c.A.nan_to_num(0.0).abs().max())
    _within(S, S_ref, (16 + 4 * math.sqrt(c.K)) * EPS * mag.expand_as(S_ref), "S")
    # the same bits again, in place, on another stream; and without a base
    Y = c.base.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    assert L.apply(*args, Y, out=Y, stream=st, **kw) is Y
    st.synchronize()
    assert torch.equal(Y, got)
    ref, tol, _ = c.forward(base=False)
    _within(L.apply(*args, **kw), ref, tol + 2 * EPS * ref.abs(), "Y without base")


@pytest.mark.parametrize("case", [c for c in LORA if not c[-1]],
                         ids=[i for i, c in enumerate(LORA) if not c[-1]])
def test_lora_gradient(torch, case):
    say(f"[lora grad] {case}")
    c = Case(torch, *case, seed=1)
    L = c.layer()
    _, S = L.apply(c.X, c.off, c.d_ids, c.base, save=True)
    got = L.grad(c.X, c.off, c.d_ids, S, c.dY)
    torch.cuda.synchronize()
    ref, tol = c.grads(S)
    for name, g, r, b in zip(("dX", "dA", "dB"), got, ref, tol):
        _within(g, r, b + _round(torch, r, g.dtype), name)
    again = L.grad(c.X, c.off, c.d_ids, S, c.dY)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    none, dA, dB = L.grad(c.X, c.off, c.d_ids, S, c.dY, need_dx=False)
    assert none is None and torch.equal(dA, got[1]) and torch.equal(dB, got[2])


def test_lora_gradient_by_differences(torch):
    # <dY, Y> is linear in X, in A and in B each: a difference of step 1 has no
    # truncation error, only the roundings of two forward calls.
    c = Case(torch, [33, 4, 50], [0, 1, 0], 96, 72, 12, seed=2)
    L = c.layer()
    Y, S = L.apply(c.X, c.off, c.d_ids, save=True)
    grads = L.grad(c.X, c.off, c.d_ids, S, c.dY)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    for name, grad in zip(("X", "A", "B"), grads):
        p = getattr(c, name)
        d = torch.empty(p.shape, device="cuda").normal_(generator=g) * p.abs().mean()
        vals = []
        for sign in (0.5, -0.5):
            q = {k: getattr(c, k) for k in ("X", "A", "B")}
            q[name] = p + sign * d
            from bit_post_quantization_amd import LoraAdapters
            y = LoraAdapters(q["A"], q["B"], c.scales).apply(q["X"], c.off, c.d_ids).double()
            vals.append(y)
        want = float((c.dY.double() * (vals[0] - vals[1])).sum())
        have = float((grad.double() * d.double()).sum())
        # each of the M N values carries 2^-24-sized roundings of about its own size
        noise = 40 * EPS * float((c.dY.double().abs() * Y.double().abs()).sum())
        assert abs(want - have) <= noise + 1e-6 * abs(want), (name, want, have, noise)


def test_lora_strides_and_alignment(torch):
    # X, base and dY as slices of wider tensors, at odd offsets and row strides
    for x, off in (("f32", 4), ("f32", 1), ("bf16", 8), ("bf16", 3)):
        c = Case(torch, [18, 31], [1, 0], 112, 45, 10, x, "f32", seed=4)
        L = c.layer()
        wide = torch.zeros(c.M, c.K + off + 3, dtype=c.X.dtype, device="cuda")
        Xs = wide[:, off:off + c.K]
        Xs.copy_(c.X)
        out = torch.full((c.M, 3 * c.N), 7.0, device="cuda")
        Ys = out[:, c.N:2 * c.N]  # the middle third of a fused projection
        Ys.copy_(c.base)
        want, S = L.apply(c.X, c.off, c.d_ids, c.base, save=True)
        L.apply(Xs, c.off, c.d_ids, Ys, out=Ys)
        assert torch.equal(Ys, want)
        assert bool((out[:, :c.N] == 7).all()) and bool((out[:, 2 * c.N:] == 7).all())
        dwide = torch.zeros(c.M, c.N + 5, device="cuda")
        dYs = dwide[:, 2:2 + c.N]
        dYs.copy_(c.dY)
        ref, tol = c.grads(S)
        for name, g, r, b in zip(("dX", "dA", "dB"), L.grad(Xs, c.off, c.d_ids, S, dYs), ref, tol):
            _within(g, r, b + _round(torch, r, g.dtype), name)


def test_lora_non_finite_rows_stay_alone(torch):
    c = Case(torch, [20, 21, 9], [0, 1, -1], 64, 40, 8, seed=5)
    c.X[3, 5], c.X[25, 0], c.X[45] = float("nan"), float("inf"), float("nan")
    got, S = c.layer().apply(c.X, c.off, c.d_ids, c.base, save=True)
    bad = ~torch.isfinite(got).all(1)
    assert bad.nonzero().flatten().tolist() == [3, 25]  # row 45 has no adapter
    assert torch.equal(got[41:], c.base[41:]) and not bool(S[41:].any())
    dY = c.dY.clone()
    dY[4, 1] = float("inf")
    dX, dA, dB = c.layer().grad(c.X.nan_to_num(0, 1, 1), c.off, c.d_ids, S.nan_to_num(0, 1, 1), dY)
    assert (~torch.isfinite(dX).all(1)).nonzero().flatten().tolist() == [4]
    assert bool(torch.isfinite(dA[1]).all()) and not bool(torch.isfinite(dA[0]).all())


def test_lora_empty_batches(torch):
    c = Case(torch, [0, 0], [0, 1], 32, 24, 4, ranks=(4,))
    c.A.nan_to_num_(0)
    got, S = c.layer().apply(c.X, c.off, c.d_ids, c.base, save=True)
    assert got.shape == (0, 24) and S.shape == (0, 4)
    dX, dA, dB = c.layer().grad(c.X, c.off, c.d_ids, S, c.dY)
    assert dX.shape == (0, 32) and not bool(dA.any()) and not bool(dB.any())


def test_lora_offsets_past_32_bits(torch):
    # rows far enough apart that element offsets pass 2^32
    M, ld = 70000, 65536
    wide = torch.empty(M * ld, dtype=torch.bfloat16, device="cuda")
    X = wide.view(M, ld)[:, :32]
    c = Case(torch, [M - 5, 5], [0, 1], 32, 8, 4, "bf16", "bf16", seed=6)
    X.copy_(c.X)
    L = c.layer()
    want, S = L.apply(c.X, c.off, c.d_ids, c.base, save=True)
    assert torch.equal(L.apply(X, c.off, c.d_ids, c.base), want)
    a, b = (L.grad(x, c.off, c.d_ids, S, c.dY) for x in (c.X, X))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_lora_replayed_in_a_graph(torch):
    c = Case(torch, [40, 9, 30], [0, 1, 2], 96, 50, 8, "bf16", "bf16", seed=7)
    L = c.layer()
    out = torch.empty_like(c.base)
    L.apply(c.X, c.off, c.d_ids, c.base, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.apply(c.X, c.off, c.d_ids, c.base, out=out)
    for k in range(3):  # other rows and other requests each time
        c.X.copy_(torch.roll(c.X, k + 1, 0))
        c.off[1], c.off[2] = 10 + k, 60 + k
        eager = L.apply(c.X, c.off, c.d_ids, c.base)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k


def test_lora_refuses_bad_tensors(torch):
    from bit_post_quantization_amd import LoraAdapters, QLError
    c = Case(torch, [8], [0], 32, 24, 4)
    L = c.layer()
    bad = [
        lambda: L.apply(c.X.half(), c.off, c.d_ids, c.base),
        lambda: L.apply(c.X.cpu(), c.off, c.d_ids, c.base),
        lambda: L.apply(c.X[:, :16], c.off, c.d_ids, c.base),
        lambda: L.apply(c.X.t().contiguous().t(), c.off, c.d_ids, c.base),
        lambda: L.apply(c.X, c.off[:1], c.d_ids, c.base),
        lambda: L.apply(c.X, c.off.long(), c.d_ids, c.base),
        lambda: L.apply(c.X, c.off, c.d_ids, c.base[:7]),
        lambda: L.apply(c.X, c.off, c.d_ids, c.base, cfg=2),
        lambda: L.apply(c.X[:7], c.off, c.d_ids, c.base[:3], cfg=1),
        lambda: LoraAdapters(c.A.half(), c.B.half()),
        lambda: LoraAdapters(c.A, c.B.bfloat16()),
        lambda: LoraAdapters(c.A[:2], c.B),
        lambda: LoraAdapters(c.A, c.B, x_dtype="f64"),
        lambda: LoraAdapters(torch.zeros(1, 129, 32, device="cuda"),
                             torch.zeros(1, 24, 129, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(QLError):
            f()
            pytest.fail(f"case {i} was accepted")


# -------------------------------------------------------------- group norm ----

def _norm_ref(t, x, gamma, beta, G, eps, act):
    """(y, bound, mean, rstd) in 64 bits over [B, L, C]."""
    B, L, C = x.shape
    x = x.double()
    xg = x.view(B, L, G, C // G)
    m = xg.mean((1, 3), keepdim=True)
    var = (xg - m).square().mean((1, 3), keepdim=True)
    r = 1 / (var + eps).sqrt()
    ga = t.ones(C, device="cuda", dtype=t.float64) if gamma is None else gamma.double()
    be = t.zeros(C, device="cuda", dtype=t.float64) if beta is None else beta.double()
    xh = ((xg - m) * r).view(B, L, C)
    z = xh * ga + be
    y = z * t.sigmoid(z) if act == "silu" else z
    # fp32 roundings of x - mean, of rstd and gamma, of the sum; statistics a few EPS
    dz = EPS * (16 * (1 + xh.abs()) * ga.abs() + 4 * be.abs()
                + 4 * ((xg.abs() + m.abs()) * r).reshape(B, L, C) * ga.abs())
    tol = 1.1 * dz + y.abs() * (z.abs() + 4) * 2 * EPS if act == "silu" else dz
    return y, tol, m.view(B, G), r.view(B, G)


def _norm_grad_ref(t, dy, x, gamma, beta, G, eps, act):
    x = x.double().requires_grad_()
    ga = gamma.double().requires_grad_()
    be = beta.double().requires_grad_()
    B, L, C = x.shape
    xg = x.view(B, L, G, C // G)
    m = xg.mean((1, 3), keepdim=True)
    r = 1 / ((xg - m).square().mean((1, 3), keepdim=True) + eps).sqrt()
    xh = ((xg - m) * r).reshape(B, L, C)
    z = xh * ga + be
    y = z * t.sigmoid(z) if act == "silu" else z
    dx, dg, db = t.autograd.grad(y, (x, ga, be), dy.double())
    with t.no_grad():
        xh, z, r = xh.detach(), z.detach(), r.detach().expand(B, L, G, C // G).reshape(B, L, C)
        ga, d = ga.detach().abs(), dy.double().abs()
        if act == "silu":
            s = t.sigmoid(z)
            dz = d * (s * (1 + z * (1 - s))).abs()
            # derivative's slope is at most 1/2; its own roundings a few EPS of |z| + 1
            ez = d * EPS * (16 * (1 + xh.abs()) * ga + 8 * (z.abs() + 1) + 4 * beta.double().abs()
                            + 4 * (x.abs() + x.abs().mean()) * r * ga)
        else:
            dz, ez = d, 0 * d
        mean = lambda v: (v.view(B, L, G, C // G).mean((1, 3), keepdim=True)  # noqa: E731
                          .expand(B, L, G, C // G).reshape(B, L, C))
        e = ez + 16 * EPS * dz * (1 + xh.abs())
        tol = r * (ga * e + mean(ga * e) + xh.abs() * mean(ga * e * (1 + xh.abs()))
                   + 16 * EPS * (1 + xh.abs()) * (mean(ga * dz) + xh.abs() * mean(ga * dz * xh.abs())))
        n = 16 + 4 * math.sqrt(B * L)
        tg = (e * (1 + xh.abs()) + n * EPS * dz * xh.abs()).sum((0, 1))
        tb = (e + n * EPS * dz).sum((0, 1))
    return (dx, dg, db), (tol, tg, tb)


NORM = [
    # B, L, C, G, x, w, act, mean of x, gamma/beta
    (1, 1, 1, 1, "f32", "f32", "none", 0.0, True),
    (1, 1, 8, 8, "f32", "f32", "silu", 0.0, True),
    (2, 256, 1280, 32, "bf16", "f32", "silu", 0.5, True),
    (3, 77, 40, 8, "f32", "bf16", "silu", 2.0, True),
    (1, 1000, 30, 5, "bf16", "bf16", "none", 0.0, False),
    (2, 65, 21, 7, "f32", "f32", "silu", 100.0, True),
    (5, 9, 8192, 32, "f32", "f32", "none", 0.0, True),
    (1, 4099, 64, 2, "bf16", "f32", "silu", -3.0, True),
    (2, 50, 96, 1, "f32", "f32", "silu", 0.0, False),
    (1, 3, 2048, 2048, "bf16", "f32", "none", 0.0, True),
    (16, 1023, 320, 32, "bf16", "bf16", "silu", 0.0, True),
    (2, 4096, 640, 32, "f32", "f32", "silu", 0.1, True),
]


def _norm_inputs(t, case, seed=0):
    B, L, C, G, x, w, act, mean, affine = case
    g = t.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*s):
        return t.empty(s, device="cuda").normal_(generator=g)

    X = (normal(B, L, C) * (0.5 + normal(C).abs()) + mean).to(_dt(t, x))
    ga = (1 + 0.3 * normal(C)).to(_dt(t, w)) if affine else None
    be = (0.3 * normal(C)).to(_dt(t, w)) if affine else None
    return X, ga, be, normal(B, L, C).to(_dt(t, x))


def _group_norm(ga, be, G, act, C):
    from bit_post_quantization_amd import GroupNormAct
    return GroupNormAct(ga, be, G, act=act, channels=C)


@pytest.mark.parametrize("case", NORM, ids=range(len(NORM)))
def test_group_norm(torch, case):
    say(f"[norm] {case}")
    B, L, C, G, _, _, act, _, _ = case
    x, ga, be, _ = _norm_inputs(torch, case)
    op = _group_norm(ga, be, G, act, C)
    y, mean, rstd = op.forward(x, stats=True)
    torch.cuda.synchronize()
    ref, tol, m, r = _norm_ref(torch, x, ga, be, G, 1e-5, act)
    _within(y, ref, tol + _round(torch, ref, x.dtype), "y")
    sd = 1 / r
    _within(mean, m, 2 * EPS * m.abs() + 16 * EPS * sd, "mean")
    # a variance far below eps or the mean's square keeps an absolute error of that size
    _within(rstd, r, r * (16 * EPS + 4 * (EPS * (m.abs() + 1) * r) ** 2), "rstd")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    z = x.clone()
    st.wait_stream(torch.cuda.current_stream())
    assert op.forward(z, out=z, stream=st) is z
    st.synchronize()
    assert torch.equal(z, y)


@pytest.mark.parametrize("case", [c for c in NORM if c[8] and c[7] < 10], ids=str)
def test_group_norm_gradient(torch, case):
    say(f"[norm grad] {case}")
    B, L, C, G, _, _, act, _, _ = case
    x, ga, be, dy = _norm_inputs(torch, case, seed=1)
    op = _group_norm(ga, be, G, act, C)
    _, mean, rstd = op.forward(x, stats=True)
    got = op.grad(dy, x, mean, rstd)
    torch.cuda.synchronize()
    ref, tol = _norm_grad_ref(torch, dy, x, ga, be, G, 1e-5, act)
    for name, a, r, b in zip(("dx", "dgamma", "dbeta"), got, ref, tol):
        _within(a, r, b + _round(torch, r, a.dtype) + 1e-30, name)
    assert all(torch.equal(a, b) for a, b in zip(got, op.grad(dy, x, mean, rstd)))


def test_group_norm_gradient_by_differences(torch):
    # central differences of <dy, y> of the 32-bit forward call with step 2^-6:
    # truncation h^2 times a third derivative of order 1, roundings EPS / h
    case = (2, 60, 24, 4, "f32", "f32", "silu", 0.0, True)
    x, ga, be, dy = _norm_inputs(torch, case, seed=2)
    op = _group_norm(ga, be, 4, "silu", 24)
    y, mean, rstd = op.forward(x, stats=True)
    grads = op.grad(dy, x, mean, rstd)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    h = 2.0 ** -6
    for i, grad in enumerate(grads):
        p = [x, ga, be]
        d = torch.empty(p[i].shape, device="cuda").normal_(generator=g)
        vals = []
        for s in (h, -h):
            q = list(p)
            q[i] = p[i] + s * d
            vals.append(_group_norm(q[1], q[2], 4, "silu", 24).forward(q[0]).double())
        want = float((dy.double() * (vals[0] - vals[1])).sum()) / (2 * h)
        have = float((grad.double() * d.double()).sum())
        size = float(dy.double().norm()) * float(vals[0].norm()) / math.sqrt(vals[0].numel())
        tol = 10 * h * h * size + 40 * EPS / h * size
        assert abs(want - have) <= tol, (i, want, have, tol)


def test_group_norm_images_and_slices(torch):
    # NHWC images, and channel slices of a wider (concatenated) image
    for dt, C, extra, start in (("f32", 24, 12, 4), ("bf16", 32, 16, 8), ("bf16", 32, 5, 3)):
        case = (2, 35, C, 4, dt, "f32", "silu", 0.0, True)
        x, ga, be, dy = _norm_inputs(torch, case, seed=3)
        op = _group_norm(ga, be, 4, "silu", C)
        want, mean, rstd = op.forward(x, stats=True)
        img = x.view(2, 5, 7, C).permute(0, 3, 1, 2)
        assert img.is_contiguous(memory_format=torch.channels_last)
        y = op.forward(img)
        assert y.is_contiguous(memory_format=torch.channels_last)
        assert torch.equal(y.permute(0, 2, 3, 1).reshape(2, 35, C), want)
        wide = torch.full((2, 35, C + extra), 9.0, dtype=x.dtype, device="cuda")
        part = wide[:, :, start:start + C]
        part.copy_(x)
        ref, tol, _, _ = _norm_ref(torch, x, ga, be, 4, 1e-5, "silu")
        _within(op.forward(part), ref, tol + _round(torch, ref, x.dtype), "slice")
        gref, gtol = _norm_grad_ref(torch, dy, x, ga, be, 4, 1e-5, "silu")
        dx, dg, db = op.grad(dy, part, mean, rstd)
        for name, a, r, b in zip(("dx", "dgamma", "dbeta"), (dx, dg, db), gref, gtol):
            _within(a, r, b + _round(torch, r, a.dtype), name)
        op.forward(part, out=part)
        _within(part, ref, tol + _round(torch, ref, x.dtype), "slice in place")
        assert bool((wide[:, :, :start] == 9).all() and (wide[:, :, start + C:] == 9).all())


def test_group_norm_extreme_values(torch):
    # constant groups, a mean far from zero, non-finite values in one group only
    x = torch.zeros(2, 300, 16, device="cuda")
    x[0] += 5.0
    x[1, :, :4] = 1e4 + torch.randn(300, 4, device="cuda")
    x[1, 7, 9] = float("nan")
    x[1, 8, 13] = float("inf")
    op = _group_norm(None, None, 4, "silu", 16)
    y, mean, rstd = op.forward(x, stats=True)
    assert not bool(y[0].any()) and bool((mean[0] == 5).all())
    ref, tol, _, _ = _norm_ref(torch, x[1:, :, :4], None, None, 1, 1e-5, "silu")
    _within(y[1:, :, :4], ref, tol, "far mean")
    assert bool(torch.isnan(y[1, :, 8:12]).all()) and bool(torch.isnan(y[1, :, 12:16]).all())
    assert not bool(torch.isnan(y[1, :, :8]).any())


def test_group_norm_empty(torch):
    ga = torch.ones(8, device="cuda")
    op = _group_norm(ga, ga, 2, "silu", 8)
    for shape in ((0, 5, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = op.forward(x, stats=True)
        assert y.shape == x.shape
        dx, dg, db = op.grad(x, x, mean, rstd)
        torch.cuda.synchronize()
        assert dx.shape == x.shape and not bool(dg.any()) and not bool(db.any())


def test_group_norm_offsets_past_32_bits(torch):
    L, ld = 70000, 65536
    wide = torch.empty(L * ld, dtype=torch.bfloat16, device="cuda").view(1, L, ld)
    case = (1, L, 32, 4, "bf16", "f32", "silu", 0.0, True)
    x, ga, be, dy = _norm_inputs(torch, case, seed=4)
    part = wide[:, :, :32]
    part.copy_(x)
    op = _group_norm(ga, be, 4, "silu", 32)
    y, mean, rstd = op.forward(x, stats=True)
    assert torch.equal(op.forward(part), y)
    a, b = (op.grad(dy, v, mean, rstd) for v in (x, part))
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_group_norm_replayed_in_a_graph(torch):
    case = (2, 500, 64, 8, "f32", "f32", "silu", 0.0, True)
    x, ga, be, dy = _norm_inputs(torch, case, seed=5)
    op = _group_norm(ga, be, 8, "silu", 64)
    out = torch.empty_like(x)
    op.forward(x, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op.forward(x, out=out)
    for k in range(3):
        x.mul_(1.5).add_(0.1)
        eager = op.forward(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), k


def test_group_norm_refuses_bad_tensors(torch):
    from bit_post_quantization_amd import GroupNormAct, QLError
    ga = torch.ones(16, device="cuda")
    op = GroupNormAct(ga, ga, 4)
    x = torch.zeros(2, 9, 16, device="cuda")
    st = torch.zeros(2, 4, device="cuda")
    bad = [
        lambda: op.forward(x.half()),
        lambda: op.forward(x.cpu()),
        lambda: op.forward(x[:, :, :8]),
        lambda: op.forward(torch.zeros(2, 16, 3, 3, device="cuda")),  # channels first
        lambda: op.forward(x, out=torch.zeros(2, 8, 16, device="cuda")),
        lambda: op.forward(x, out=x.bfloat16()),
        lambda: op.grad(x[:1], x, st, st),
        lambda: op.grad(x, x, st[:1], st),
        lambda: GroupNormAct(ga, ga, 3),
        lambda: GroupNormAct(ga, ga, 4, act="relu"),
        lambda: GroupNormAct(ga, ga.bfloat16(), 4),
        lambda: GroupNormAct(ga, ga, 4, eps=0.0),
        lambda: GroupNormAct(None, None, 4),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(QLError):
            f()
            pytest.fail(f"case {i} was accepted")


# ---------------------------------------------------------------- clipping ----

CLIP = [
    # sizes, gradient type, out (None: in place), max_norm
    ([1], "f32", None, 1.0),
    ([1, 0, 3, 4096, 4097, 0], "f32", None, 0.5),
    ([4096 * 3, 5, 100000], "bf16", "f32", 2.0),
    ([8192] * 300, "f32", "bf16", 10.0),
    ([1000003, 17, 4095], "bf16", None, 1e9),
    ([7] * 5000, "f32", "f32", 3.0),
    ([], "f32", None, 1.0),
]


@pytest.mark.parametrize("case", CLIP, ids=range(len(CLIP)))
def test_clip(torch, case):
    from bit_post_quantization_amd import GradSet
    sizes, x, out, max_norm = case
    say(f"[clip] {len(sizes)} tensors {x} -> {out or 'in place'}")
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    flat = torch.empty(sum(sizes), device="cuda").normal_(0, 0.1, generator=g).to(_dt(torch, x))
    grads = [t.clone() for t in flat.split(sizes)] if sizes else []
    outs = None
    if out:  # views of one buffer: odd offsets
        buf = torch.zeros(sum(sizes) + 1, dtype=_dt(torch, out), device="cuda")
        outs = list(buf[1:].split(sizes))
    s = GradSet(grads, out=outs)
    norm = s.clip(max_norm)
    torch.cuda.synchronize()
    ref = flat.double().norm()
    assert abs(float(norm) - float(ref)) <= 2 * EPS * float(ref)
    coef = min(1.0, max_norm / (float(ref) + 1e-6))
    got = outs if outs else s.grads
    for a, b in zip(got, flat.split(sizes) if sizes else []):
        r = b.double() * coef
        _within(a, r, 4 * EPS * r.abs() + _round(torch, r, a.dtype), "clipped")
    if not outs and coef == 1.0:
        assert all(torch.equal(a, b) for a, b in zip(got, flat.split(sizes)))


def test_clip_extreme_values(torch):
    from bit_post_quantization_amd import GradSet
    big = torch.full((5000,), 3e38, device="cuda")  # squares beyond fp32
    big[1:] = 1e30
    ref = big.double().norm()
    norm = GradSet([big]).clip(1.0)
    assert abs(float(norm) / float(ref) - 1) < 1e-6 and abs(float(big.double().norm()) - 1) < 1e-5
    tiny = torch.full((5000,), 1e-30, device="cuda")  # squares below fp32
    assert abs(float(GradSet([tiny]).clip(1.0)) / (1e-30 * math.sqrt(5000)) - 1) < 1e-6
    a, b = torch.ones(10, device="cuda"), torch.ones(6000, device="cuda")
    b[7] = float("inf")
    assert math.isinf(float(GradSet([a, b]).clip(1.0)))
    assert not bool(a.any()) and bool(torch.isnan(b[7])) and not bool(b[8:].any())
    b[7] = float("nan")
    a.fill_(1.0)
    assert math.isnan(float(GradSet([a, b]).clip(1.0))) and bool(torch.isnan(a).all())
    assert float(GradSet([torch.zeros(9, device="cuda")]).clip(0.0)) == 0.0


def test_clip_partials_add_over_ranks(torch):
    # two shards' partials added, as an all-reduce does, clip by the whole norm
    from bit_post_quantization_amd import GradSet
    a, b = torch.randn(30000, device="cuda"), torch.randn(50, device="cuda")
    whole = torch.cat([a, b]).double().norm()
    s, u = GradSet([a.clone()]), GradSet([b])
    norm = s.clip(1.0, partials=s.partials() + u.partials())
    assert abs(float(norm) - float(whole)) <= 2 * EPS * float(whole)
    _within(s.grads[0], a.double() / (whole + 1e-6), 4 * EPS * a.abs().double(), "shard")


def test_clip_past_32_bits_and_again(torch):
    from bit_post_quantization_amd import GradSet
    n = (1 << 32) + 4099
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    g[-1] = 2.0
    s = GradSet([g, torch.ones(3, device="cuda")])
    want = math.sqrt(n + 3 + 3)
    first = s.partials()
    assert torch.equal(first, s.partials())
    assert abs(float(s.clip(want * 1.5)) - want) <= 2 * EPS * want
    assert float(g[-1]) == 2.0 and float(g[0]) == 1.0
    s.clip(want / 4)
    assert float(g[0]) == 0.25 and float(g[-1]) == 0.5 and float(g[1 << 32]) == 0.25


def test_clip_on_another_stream_and_in_a_graph(torch):
    from bit_post_quantization_amd import GradSet
    src = [torch.randn(n, device="cuda") for n in (5, 40000, 4096)]
    out = [torch.empty_like(t) for t in src]
    s = GradSet(src, out=out)
    want = float(s.clip(1.0))
    ref = [t.clone() for t in out]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for t in out:
        t.zero_()
    st.wait_stream(torch.cuda.current_stream())
    n = s.clip(1.0, stream=st)
    st.synchronize()
    assert float(n) == want and all(torch.equal(a, b) for a, b in zip(out, ref))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        norm = s.clip(1.0)
    for k in range(3):
        for t in src:
            t.mul_(1.25)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = s.clip(1.0)
        torch.cuda.synchronize()
        assert float(norm) == float(eager) and all(torch.equal(a, b) for a, b in zip(got, out)), k


def test_clip_refuses_bad_tensors(torch):
    from bit_post_quantization_amd import GradSet, QLError
    a = torch.ones(8, device="cuda")
    bad = [
        lambda: GradSet([a.half()]),
        lambda: GradSet([a.cpu()]),
        lambda: GradSet([torch.ones(8, 2, device="cuda")[:, 0]]),
        lambda: GradSet([a], out=[a[:7]]),
        lambda: GradSet([a], out=[]),
        lambda: GradSet([a], out=[a.view(torch.bfloat16)[:8]]),
        lambda: GradSet([a]).clip(-1.0),
        lambda: GradSet([a]).clip(1.0, partials=torch.zeros(3, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(QLError):
            f()
            pytest.fail(f"case {i} was accepted")

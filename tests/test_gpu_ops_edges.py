"""The operators beside the layer where they can go wrong: sums that cancel,
values that are not finite, the forms that only large calls take, lifetimes.

Bounds as in test_gpu_ops: (16 + 4 sqrt(n)) EPS times the sum of the products'
magnitudes for a sum of n products, 2^-8 of itself for a result rounded to bf16.
"""
from __future__ import annotations

import math

import pytest

from tests.parity import say
from tests.test_gpu_ops import EPS, _dt, _norm_ref, _round, _within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    assert _t.cuda.is_available(), "GPU tests need a ROCm device"
    import bit_post_quantization_amd  # noqa: F401  (fails loudly if the library is missing)
    return _t


# ---------------------------------------------------------------- adapters ----

@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("rank", [4, 16, 31, 64, 128])
def test_lora_gradient_sums_that_cancel(torch, x, rank):
    # Three rows a request whose products cancel up to their roundings: what is
    # left shows how many bits of dS, S and dY the sums saw. 16 bits of an operand
    # would miss the bound, which is relative to the products and not to the sum.
    from bit_post_quantization_amd import LoraAdapters
    say(f"[lora grad cancel] x {x} rank {rank}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rank)
    n, N, K = 24, 1, 48

    def normal(*s):
        return torch.empty(s, device="cuda").normal_(generator=g)

    def cancelling(*s):  # [n, 3, ...]: the third row is minus the sum of the others
        v = normal(n, 2, *s)
        return torch.cat([v, -v.sum(1, keepdim=True)], 1).reshape(3 * n, *s)

    off = torch.arange(n + 1, dtype=torch.int32, device="cuda") * 3
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    A, B = normal(n, rank, K).bfloat16(), normal(n, N, rank).bfloat16()
    L = LoraAdapters(A, B, x_dtype=x)
    same = lambda *s: normal(n, 1, *s).expand(n, 3, *s).reshape(3 * n, *s)  # noqa: E731
    # dA = sum of dS^T X with dS = dY B: n = N + 3 products
    X, dY, S = same(K).to(_dt(torch, x)), cancelling(N), normal(3 * n, rank)
    _, dA, _ = L.grad(X, off, ids, S, dY)
    v = lambda t: t.double().view(n, 3, -1)  # noqa: E731
    ref = ((v(dY) @ B.double()).transpose(1, 2) @ v(X))
    mag = ((v(dY).abs() @ B.double().abs()).transpose(1, 2) @ v(X).abs())
    _within(dA, ref, (16 + 4 * math.sqrt(N + 3)) * EPS * mag + _round(torch, ref, dA.dtype), "dA")
    # dB = sum of dY^T S: n = 3 products
    N = 70
    L = LoraAdapters(A, normal(n, N, rank).bfloat16(), x_dtype=x)
    dY, S = same(N), cancelling(rank)
    _, _, dB = L.grad(X, off, ids, S, dY)
    ref = v(dY).transpose(1, 2) @ v(S)
    mag = v(dY).abs().transpose(1, 2) @ v(S).abs()
    _within(dB, ref, (16 + 4 * math.sqrt(3)) * EPS * mag + _round(torch, ref, dB.dtype), "dB")


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("rank", [3, 33, 66])
def test_lora_gradient_ranks_that_cancel(torch, x, rank):
    # dX = dS A where the ranks cancel in threes: B's third column is minus the
    # sum of the other two (exactly: their values are small whole numbers) and
    # A's three rows are one. n = N + 3 products.
    from bit_post_quantization_amd import LoraAdapters
    say(f"[lora grad cancel] dX x {x} rank {rank}")
    g = torch.Generator(device="cuda")
    g.manual_seed(rank)
    M, N, K, t = 200, 1, 48, rank // 3
    b = torch.randint(1, 60, (1, N, t, 2), generator=g, device="cuda").float()
    B = torch.cat([b, -b.sum(-1, keepdim=True)], -1).reshape(1, N, rank).bfloat16()
    A = torch.empty((1, t, 1, K), device="cuda").normal_(generator=g).expand(1, t, 3, K)
    A = A.reshape(1, rank, K).bfloat16()
    keep = torch.zeros(t, 3, dtype=torch.bool, device="cuda")
    keep[0] = True  # one triple at a time: the others' storage holds zeros
    X = torch.empty((M, K), device="cuda").normal_(generator=g).to(_dt(torch, x))
    dY = torch.empty((M, N), device="cuda").normal_(generator=g)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    ids = torch.zeros(1, dtype=torch.int32, device="cuda")
    for k in {0, t // 2, t - 1}:
        keep.zero_()
        keep[k] = True
        Bk = B * keep.view(1, 1, rank)
        L = LoraAdapters(A, Bk, x_dtype=x)
        dX, _, _ = L.grad(X, off, ids, torch.zeros(M, rank, device="cuda"), dY)
        dS = dY.double() @ Bk[0].double()
        ref, mag = dS @ A[0].double(), dS.abs() @ A[0].double().abs()
        _within(dX, ref, (16 + 4 * math.sqrt(N + 3)) * EPS * mag + _round(torch, ref, dX.dtype),
                f"dX, ranks {3 * k}..")


def test_lora_batch_without_requests(torch):
    from bit_post_quantization_amd import LoraAdapters
    A, B = torch.randn(2, 4, 32, device="cuda"), torch.randn(2, 24, 4, device="cuda")
    L = LoraAdapters(A, B)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    off = torch.zeros(1, dtype=torch.int32, device="cuda")
    X, dY = torch.empty(0, 32, device="cuda"), torch.empty(0, 24, device="cuda")
    for cfg in (0, 1):
        Y, S = L.apply(X, off, none, cfg=cfg, save=True)
        assert Y.shape == (0, 24) and S.shape == (0, 4)
    dX, dA, dB = L.grad(X, off, none, S, dY)
    assert dX.shape == (0, 32) and not bool(dA.any()) and not bool(dB.any())


@pytest.mark.parametrize("x,w", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rank", [1, 16, 30, 70])
def test_lora_non_finite_values_reach_their_products_only(torch, rank, x, w):
    # one infinity or NaN in one operand at a time: what the formula has non-finite
    # is non-finite, everything else is what it is without it, to the last bit
    from tests.test_gpu_ops import Case
    say(f"[lora non-finite] rank {rank} x {x} w {w}")
    for v in (float("inf"), float("-inf"), float("nan")):
        for what, at in (("X", (9, 17)), ("A", (1, rank - 1, 40)), ("B", (1, 33, rank // 2)),
                         ("dY", (70, 5)), ("S", (44, 0))):
            c = Case(torch, [40, 41, 7], [0, 1, 0], 80, 50, rank, x, w, seed=8)
            L = c.layer()
            want, S = L.apply(c.X, c.off, c.d_ids, c.base, save=True)
            grads = L.grad(c.X, c.off, c.d_ids, S, c.dY)
            if what == "S":
                S[at] = v
            else:
                getattr(c, what)[at] = v
            if what not in ("S", "dY"):
                got = L.apply(c.X, c.off, c.d_ids, c.base)
                hit = ~torch.isfinite(c.forward()[0])
                assert torch.equal(~torch.isfinite(got), hit), (what, v)
                assert torch.equal(got[~hit], want[~hit]), (what, v)
            for name, g, r, u in zip(("dX", "dA", "dB"), L.grad(c.X, c.off, c.d_ids, S, c.dY),
                                     c.grads(S)[0], grads):
                hit = ~torch.isfinite(r)
                assert torch.equal(~torch.isfinite(g), hit), (what, v, name)
                assert torch.equal(g[~hit], u[~hit]), (what, v, name)


# Large outputs, S of 32 rows a workgroup (512 tiles of 32 rows or more, and rank 64 at
# most, guided 32), and what is next to it: rank above, rows just short of it.
TALL = [
    ([16001, 0, 403], [0, 1, 2], 48, 521, 12, "f32", "f32", (12, 5), False),
    ([5000, 1, 11399], [2, -1, 0], 80, 520, 30, "bf16", "bf16", None, False),
    ([16395, 7], [1, 0], 64, 516, 64, "f32", "bf16", (64, 33), False),
    ([9, 16400], [0, 2], 144, 513, 64, "bf16", "f32", None, False),
    ([300] * 55, list(range(-1, 4)) * 11, 48, 512, 16, "bf16", "bf16", (16, 3), False),
    ([16400], [0], 32, 513, 100, "bf16", "bf16", None, False),
    ([16401, 30], [1, 0], 48, 512, 16, "f32", "f32", None, True),
    ([8200, 8205], [0, 2], 48, 520, 32, "bf16", "bf16", (32, 9), True),
    ([16300, 101], [1, -1], 32, 519, 48, "f32", "bf16", None, True),
    ([16300], [0], 48, 520, 16, "f32", "f32", None, False),
]


@pytest.mark.parametrize("case", TALL, ids=range(len(TALL)))
def test_lora_forward_of_many_rows(torch, case):
    from tests.test_gpu_ops import Case
    say(f"[lora tall] {case}")
    assert sum(case[0]) * case[3] >= 1 << 23
    c = Case(torch, *case, seed=10)
    kw = dict(cfg=int(c.cfg), w=c.w)
    ref, tol, S_ref = c.forward()
    got, S = c.layer().apply(c.X, c.off, c.d_ids, c.base, save=True, **kw)
    torch.cuda.synchronize()
    _within(got, ref, tol + 2 * EPS * ref.abs(), "Y")
    mag = c.X.double().abs().sum(1, keepdim=True) * float(c.A.nan_to_num(0.0).abs().max())
    _within(S, S_ref, (16 + 4 * math.sqrt(c.K)) * EPS * mag.expand_as(S_ref), "S")
    Y = c.base.clone()
    assert c.layer().apply(c.X, c.off, c.d_ids, Y, out=Y, **kw) is Y and torch.equal(Y, got)
    ref, tol, _ = c.forward(base=False)
    _within(c.layer().apply(c.X, c.off, c.d_ids, **kw), ref, tol + 2 * EPS * ref.abs(), "no base")


# dS by 32 rows (rows / 32 + requests of 256 and more), and dS split over the columns
# (few rows beside a wide output; two, three, seven and eight parts).
TALL_GRAD = [
    ([8000, 0, 333], [0, 1, 2], 48, 75, 30, "f32", "f32", None, False),
    ([4100, 1, 4203], [2, -1, 0], 80, 45, 30, "bf16", "bf16", (30, 7), False),
    ([8300, 9], [1, 1], 48, 101, 64, "f32", "bf16", None, False),
    ([17, 8250], [0, 2], 272, 33, 64, "bf16", "f32", (64, 40), False),
    ([8291], [0], 32, 70, 12, "f32", "f32", None, False),
    ([8200], [1], 32, 70, 100, "bf16", "bf16", None, False),
    ([31] * 270, list(range(-1, 4)) * 54, 32, 50, 64, "bf16", "bf16", (64, 1), False),
]
SPLIT_GRAD = [
    ([40], [0], 48, 4099, 4, "f32", "f32", None, False),
    ([33, 1, 62], [1, -1, 0], 64, 1100, 31, "bf16", "bf16", (31, 7), False),
    ([17, 0, 19], [0, 1, 2], 48, 3599, 64, "f32", "bf16", None, False),
    ([5], [2], 48, 1633, 128, "bf16", "f32", (128, 3), False),
    ([300, 300], [0, 1], 32, 4097, 16, "f32", "bf16", None, False),
    ([1], [0], 32, 1024, 1, "bf16", "bf16", None, False),
]


@pytest.mark.parametrize("case", TALL_GRAD + SPLIT_GRAD,
                         ids=range(len(TALL_GRAD) + len(SPLIT_GRAD)))
def test_lora_gradient_tall_and_split(torch, case):
    from tests.test_gpu_ops import Case
    say(f"[lora grad tall / split] {case}")
    lens, N = case[0], case[3]
    if case in TALL_GRAD:
        assert sum(lens) // 32 + len(lens) >= 256
    else:
        assert 256 // (sum(lens) // 16 + len(lens)) >= 2 and N >= 1024
    c = Case(torch, *case, seed=11)
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


# -------------------------------------------------------------- group norm ----

def _affine(t, C, w="f32", seed=0):
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda: t.empty(C, device="cuda").normal_(generator=g)  # noqa: E731
    return (1 + 0.3 * n()).to(_dt(t, w)), (0.3 * n()).to(_dt(t, w))


# B, L, C, G: one workgroup a group; two readings; two readings element by element
# (the rows of 65 channels lie at odd multiples of 4 bytes)
FORMS = [(2, 300, 16, 4), (2, 9001, 64, 4), (2, 60001, 65, 5)]


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_group_norm_statistics_of_non_finite_groups(torch, shape, dtype, act):
    # A NaN or an infinity anywhere in a group leaves it no variance: rstd is NaN
    # and with it every output of that group; the others are what they are alone.
    from bit_post_quantization_amd import GroupNormAct
    say(f"[norm non-finite] {shape} {dtype} {act}")
    B, L, C, G = shape
    cpg = C // G
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.empty(shape[:3], device="cuda").normal_(generator=g).to(_dt(torch, dtype))
    ga, be = _affine(torch, C)
    ga[1] = -ga[1].abs()
    op = GroupNormAct(ga, be, G, act=act)
    want = op.forward(x, stats=True)
    bad = x.clone()
    inf = float("inf")
    for b, l, grp, c, v in ((0, 7, 0, 1, float("nan")), (0, 5, 1, 0, inf), (1, 0, 2, 0, -inf),
                            (1, L - 1, 3, cpg - 1, inf), (1, 0, 0, 0, float("nan"))):
        bad[b, l, grp * cpg + c] = v
    y, mean, rstd = op.forward(bad, stats=True)
    hit = torch.zeros(B, G, dtype=torch.bool, device="cuda")
    for b, grp in ((0, 0), (0, 1), (1, 2), (1, 3), (1, 0)):
        hit[b, grp] = True
    assert bool(torch.isnan(rstd[hit]).all()) and not bool(torch.isfinite(mean[hit]).any())
    yg, wg = (t.view(B, L, G, cpg).transpose(1, 2) for t in (y, want[0]))
    assert bool(torch.isnan(yg[hit]).all())
    assert torch.equal(yg[~hit], wg[~hit])
    assert torch.equal(mean[~hit], want[1][~hit]) and torch.equal(rstd[~hit], want[2][~hit])


@pytest.mark.parametrize("shape", FORMS, ids=str)
def test_group_norm_squares_past_fp32(torch, shape):
    # deviations whose squares pass fp32: an infinite variance in every form, so
    # rstd is 0 and y = beta (not the quotient by sqrt(eps) of a variance lost)
    from bit_post_quantization_amd import GroupNormAct
    B, L, C, G = shape
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.empty((B, L, C), device="cuda").normal_(generator=g) * 3e19
    ga, be = _affine(torch, C)
    y, mean, rstd = GroupNormAct(ga, be, G, act="none").forward(x, stats=True)
    assert not bool(rstd.any()) and bool(torch.isfinite(mean).all())
    assert torch.equal(y, be.expand(B, L, C))


def test_group_norm_output_strides(torch):
    # outputs whose images do not overlap are taken in any order: positions first,
    # images between one another's rows, gaps; repeated images as input
    from bit_post_quantization_amd import GroupNormAct, QLError
    B, L, C, G = 3, 41, 24, 4
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.empty((B, L, C), device="cuda").normal_(generator=g)
    ga, be = _affine(torch, C)
    op = GroupNormAct(ga, be, G)
    ref, tol, _, _ = _norm_ref(torch, x, ga, be, G, 1e-5, "silu")
    tol = tol + _round(torch, ref, x.dtype)
    for yb, yr in ((C, B * C), (C + 1, 4 * C), (L * C, C), (L * (C + 4), C + 4), (3 * C, 2 * C * L),
                   (5 * C, 4 * C)):
        buf = torch.full((B * yb + L * yr,), 7.0, device="cuda")
        out = buf.as_strided((B, L, C), (yb, yr, 1))
        op.forward(x, out=out)
        _within(out, ref, tol, f"strides {yb}, {yr}")
        out.fill_(7.0)
        assert bool((buf == 7.0).all())
    one = x[:1].expand(B, L, C)
    _within(op.forward(one), ref[:1].expand(B, L, C), tol[:1].expand(B, L, C), "one image repeated")
    for out in (torch.empty((1, L, C), device="cuda").expand(B, L, C),
                torch.empty(B * L * C, device="cuda").as_strided((B, L, C), (L * C - 1, C, 1))):
        with pytest.raises(QLError):
            op.forward(x, out=out)


def test_group_norm_statistics_without_positions(torch):
    # 0 / 0: written as NaN, not left as they were
    from bit_post_quantization_amd import GroupNormAct, ops
    op = GroupNormAct(None, None, 2, channels=8)
    d, nb = op._of(torch.float32, 3, 0, 8, 0)
    assert nb == 0
    for which in ((True, True), (True, False), (False, True)):
        st = torch.full((2, 3, 2), 7.0, device="cuda")
        at = [t.data_ptr() if w else None for t, w in zip(st, which)]
        ops.qlinear_group_norm(d, None, 0, 8, None, 0, 8, *at, None, 0,
                               torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        for t, w in zip(st, which):
            assert bool(torch.isnan(t).all()) if w else bool((t == 7.0).all())
    y, mean, rstd = op.forward(torch.empty((3, 0, 8), device="cuda"), stats=True)
    assert y.shape == (3, 0, 8) and bool(torch.isnan(mean).all()) and bool(torch.isnan(rstd).all())


# B, L, C, G, x, w, act, columns of a wider image before and after
TWO_READINGS = [
    (1, 9001, 64, 2, "f32", "f32", "silu", (3, 2)),      # odd offset: element by element
    (2, 9001, 64, 2, "bf16", "bf16", "none", (1, 0)),
    (1, 5001, 525, 1, "f32", "bf16", "silu", (0, 0)),    # odd rows, more channels than threads
    (2, 3001, 525, 1, "bf16", "f32", "silu", (0, 0)),
    (1, 2000, 8192, 8, "f32", "f32", "silu", (0, 0)),    # more vectors a row than threads
    (1, 1500, 8192, 4, "bf16", "f32", "none", (0, 0)),
    (3, 4099, 1040, 2, "bf16", "f32", "silu", (8, 8)),   # a slice whose vectors are aligned
    (2, 4099, 260, 4, "f32", "f32", "none", (0, 0)),
    (1, 30011, 24, 3, "bf16", "f32", "silu", (0, 0)),
]


def _image_case(torch, case):
    B, L, C, G, dt, w, act, (before, after) = case
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    normal = lambda *s: torch.empty(s, device="cuda").normal_(generator=g)  # noqa: E731
    wide = torch.zeros((B, L, before + C + after), device="cuda").to(_dt(torch, dt))
    x = wide[:, :, before:before + C]
    x.copy_(normal(B, L, C) * (0.5 + normal(C).abs()) + 0.3)
    return x, *_affine(torch, C, w, seed=13), normal(B, L, C).to(_dt(torch, dt))


@pytest.mark.parametrize("case", TWO_READINGS, ids=str)
def test_group_norm_in_two_readings(torch, case):
    from bit_post_quantization_amd import GroupNormAct
    from tests.test_gpu_ops import _norm_grad_ref
    say(f"[norm two readings] {case}")
    B, L, C, G, _, _, act, _ = case
    x, ga, be, dy = _image_case(torch, case)
    op = GroupNormAct(ga, be, G, act=act)
    y, mean, rstd = op.forward(x, stats=True)
    torch.cuda.synchronize()
    xc = x.contiguous()
    ref, tol, m, r = _norm_ref(torch, xc, ga, be, G, 1e-5, act)
    _within(y, ref, tol + _round(torch, ref, x.dtype), "y")
    _within(mean, m, 2 * EPS * m.abs() + 16 * EPS / r, "mean")
    _within(rstd, r, r * (16 * EPS + 4 * (EPS * (m.abs() + 1) * r) ** 2), "rstd")
    got = op.grad(dy, x, mean, rstd)
    ref, tol = _norm_grad_ref(torch, dy, xc, ga, be, G, 1e-5, act)
    for name, a, r, b in zip(("dx", "dgamma", "dbeta"), got, ref, tol):
        _within(a, r, b + _round(torch, r, a.dtype) + 1e-30, name)
    assert all(torch.equal(a, b) for a, b in zip(got, op.grad(dy, x, mean, rstd)))
    want = y.clone()
    assert torch.equal(op.forward(x, out=x), want)


@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("given", [(True, False), (False, True), (False, False)], ids=str)
@pytest.mark.parametrize("shape", [(2, 300, 16, 4), (1, 77, 40, 8), (2, 9001, 64, 4),
                                   (2, 60001, 65, 5)], ids=str)
def test_group_norm_gradient_without_parameters(torch, shape, given, act):
    # gamma or beta or both absent: 1 and 0, and no gradient of them
    from bit_post_quantization_amd import GroupNormAct
    from tests.test_gpu_ops import _norm_grad_ref
    say(f"[norm grad] {shape} gamma, beta {given} {act}")
    B, L, C, G = shape
    x, ga, be, dy = _image_case(torch, (*shape, "f32", "f32", act, (0, 0)))
    ga, be = (t if k else None for t, k in zip((ga, be), given))
    op = GroupNormAct(ga, be, G, act=act, channels=C)
    y, mean, rstd = op.forward(x, stats=True)
    ref, tol, _, _ = _norm_ref(torch, x, ga, be, G, 1e-5, act)
    _within(y, ref, tol + _round(torch, ref, x.dtype), "y")
    got = op.grad(dy, x, mean, rstd)
    ref, tol = _norm_grad_ref(torch, dy, x, torch.ones(C, device="cuda") if ga is None else ga,
                              torch.zeros(C, device="cuda") if be is None else be, G, 1e-5, act)
    for name, a, r, b, k in zip(("dx", "dgamma", "dbeta"), got, ref, tol, (True, *given)):
        assert (a is not None) == k
        if k:
            _within(a, r, b + _round(torch, r, a.dtype) + 1e-30, name)


# ---------------------------------------------------------------- clipping ----

def test_clip_table_outlives_its_set_on_another_stream(torch):
    from bit_post_quantization_amd import GradSet
    a = torch.full((5000,), 2.0, device="cuda")
    st = torch.cuda.Stream()
    s = GradSet([a])
    at = s.table.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)  # some milliseconds of work ahead of the call
    norm = s.clip(1.0, stream=st)
    del s
    taken = [torch.empty((1, 5), dtype=torch.int64, device="cuda") for _ in range(4)]
    assert st.query() or at not in [t.data_ptr() for t in taken]
    st.synchronize()
    want = 2.0 * math.sqrt(5000)
    assert abs(float(norm) - want) <= 2 * EPS * want
    _within(a, torch.full((5000,), 2.0 / (want + 1e-6), dtype=torch.float64, device="cuda"),
            2.0 / want * 4 * EPS, "clipped")


def test_clip_of_dense_gradients_in_any_order(torch):
    # the norm and the scaling need no order: channels-last images' and transposed
    # gradients go as they are, an out in the same order
    from bit_post_quantization_amd import GradSet, QLError
    g = torch.Generator(device="cuda")
    g.manual_seed(4)

    def make():
        a = torch.empty((48, 33, 3, 5), device="cuda").normal_(generator=g)
        return [a.to(memory_format=torch.channels_last),
                torch.empty((70, 131), device="cuda").normal_(generator=g).bfloat16().t(),
                torch.empty((6, 1, 9, 4), device="cuda").normal_(generator=g).permute(3, 1, 0, 2),
                torch.empty((5, 7), device="cuda").normal_(generator=g)]

    grads = make()
    was = [t.double() for t in grads]
    assert not any(t.is_contiguous() for t in grads[:3])
    norm = math.sqrt(sum(float(t.square().sum()) for t in was))
    outs = [torch.empty_like(t, dtype=torch.float32) for t in grads]
    assert [o.stride() for o in outs] == [t.stride() for t in grads]
    assert abs(float(GradSet(grads, out=outs).clip(2.0)) - norm) <= 2 * EPS * norm
    GradSet(grads).clip(2.0)
    for got in (outs, grads):
        for a, b in zip(got, was):
            r = b * (2.0 / (norm + 1e-6))
            _within(a, r, 4 * EPS * r.abs() + _round(torch, r, a.dtype), "clipped")
    for bad in (lambda: GradSet([grads[0]], out=[grads[0].contiguous()]),
                lambda: GradSet([grads[1].contiguous()], out=[grads[1]]),
                lambda: GradSet([grads[3].expand(2, 5, 7)]),
                lambda: GradSet([grads[3][:, ::2]]),
                lambda: GradSet([grads[0][:, 1:]])):
        with pytest.raises(QLError):
            bad()


def test_clip_refuses_overlapping_outputs(torch):
    from bit_post_quantization_amd import GradSet, QLError
    buf = torch.zeros(9000, device="cuda")
    a, b, c = buf[:4000], buf[3999:6000], buf[6000:]
    bad = [
        lambda: GradSet([a, a]),                              # would be scaled twice, or once
        lambda: GradSet([a, b]),
        lambda: GradSet([c, a], out=[b, torch.empty_like(a)]),  # an out over another's gradient
        lambda: GradSet([a.clone(), c.clone()], out=[buf[:4000], buf[1000:4000]]),
        lambda: GradSet([a], out=[buf[1:4001]]),              # over its own, shifted
    ]
    for i, f in enumerate(bad):
        with pytest.raises(QLError):
            f()
            pytest.fail(f"case {i} was accepted")
    e = torch.empty(0, device="cuda")
    out = torch.empty(8000, device="cuda")
    a.fill_(3.0)
    # neighbours, empty ones, and one gradient read twice into two places are fine
    s = GradSet([a, a, e, e], out=[out[:4000], out[4000:], e, e])
    want = 3.0 * math.sqrt(8000)
    assert abs(float(s.clip(1e9)) - want) <= 2 * EPS * want and bool((out == 3.0).all())
    GradSet([buf[:4000], buf[4000:]]).clip(1.0)


# ---------------------------------------------------------- kept gradients ----

def test_gradients_into_given_tensors(torch):
    # parameters' gradients that stay where they are, so that a set of them is made
    # once: the same bits as in new tensors, every element written
    from bit_post_quantization_amd import GradSet, GroupNormAct, QLError
    from tests.test_gpu_ops import Case
    c = Case(torch, [20, 0, 31], [0, 1, 2], 64, 40, 8, "f32", "bf16", ranks=(8, 3), seed=9)
    L = c.layer()
    _, S = L.apply(c.X, c.off, c.d_ids, c.base, save=True)
    want = L.grad(c.X, c.off, c.d_ids, S, c.dY)
    x = torch.randn(2, 50, 16, device="cuda")
    ga, be = _affine(torch, 16)
    op = GroupNormAct(ga, be, 4)
    _, mean, rstd = op.forward(x, stats=True)
    nwant = op.grad(x, x, mean, rstd)
    kept = [torch.full_like(t, float("nan")) for t in (*want[1:], *nwant[1:])]
    s = GradSet(kept)
    st = torch.cuda.Stream()
    for k in range(3):
        stream = st if k == 2 else None
        st.wait_stream(torch.cuda.current_stream())
        dX, dA, dB = L.grad(c.X, c.off, c.d_ids, S, c.dY, out=kept[:2], stream=stream)
        dx, dg, db = op.grad(x, x, mean, rstd, out=kept[2:], stream=stream)
        torch.cuda.synchronize()
        assert dA is kept[0] and dB is kept[1] and dg is kept[2] and db is kept[3]
        assert torch.equal(dX, want[0]) and torch.equal(dx, nwant[0])
        assert all(torch.equal(a, b) for a, b in zip(kept, (*want[1:], *nwant[1:])))
        norm = math.sqrt(sum(float(t.double().square().sum()) for t in kept))
        assert abs(float(s.clip(0.5 * norm)) - norm) <= 2 * EPS * norm
    for bad in (lambda: L.grad(c.X, c.off, c.d_ids, S, c.dY, out=(kept[1], kept[0])),
                lambda: L.grad(c.X, c.off, c.d_ids, S, c.dY, out=(kept[0].float(), kept[1])),
                lambda: L.grad(c.X, c.off, c.d_ids, S, c.dY, out=(kept[0].cpu(), kept[1])),
                lambda: op.grad(x, x, mean, rstd, out=(kept[2], None)),
                lambda: op.grad(x, x, mean, rstd, out=(kept[2][:8], kept[3])),
                lambda: GroupNormAct(ga, None, 4).grad(x, x, mean, rstd, out=(kept[2], kept[3]))):
        with pytest.raises(QLError):
            bad()

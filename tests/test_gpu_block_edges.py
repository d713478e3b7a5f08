"""Edges of a conditioned block's operators: every head size, every way a call is cut, long
and odd sizes, masks that leave parts of a split empty, two calls at once, captured calls
with much LDS. Formulas, bounds and inputs are those of test_gpu_block.py."""
from __future__ import annotations

import math

import pytest

from tests.parity import say
from tests.test_gpu_block import EPS, Attn, Heads, Rows4, _round, _same_lse, _within, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def _attention(t, c):
    """Forward and backward of a case against the formula."""
    layer = c.layer()
    out, lse = layer.forward(c.q, c.k, c.v, lens=c.lens, mask=c.mask, save=True)
    ref, tol, ref_lse, lse_tol = c.forward()
    _within(out, ref, tol + _round(t, ref, out.dtype), "out")
    _same_lse(t, lse, ref_lse, lse_tol)
    got = layer.grad(c.dout, c.q, c.k, c.v, out, lse, lens=c.lens, mask=c.mask)
    ref, tol = c.grads(out, lse)
    for g, r, e, name in zip(got, ref, tol, ("dq", "dk", "dv")):
        _within(g, r, e + _round(t, r, g.dtype), name)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", list(range(8, 168, 8)))
def test_attention_every_head_size(torch, D, dt):  # noqa: F811
    say(f"[attention] dim {D} {dt}")
    _attention(torch, Attn(torch, 1, 45, 70, 2, 2, D, dt, "holes"))
    _attention(torch, Attn(torch, 1, 140, 200, 2, 1, D, dt, "lens"))
    c = Attn(torch, 2, 3, 400, 2, 2, D, dt, "both")  # few rows, keys shared out
    out = c.layer().forward(c.q, c.k, c.v, lens=c.lens, mask=c.mask)
    ref, tol, _, _ = c.forward()
    _within(out, ref, tol + _round(torch, ref, out.dtype), "few rows")


CUTS = [
    # B, Lq, Lk, heads, kv, dim, type, mask: how the call is cut
    (1, 1, 33000, 1, 1, 64, "bf16", "holes"),     # keys shared out 64 ways
    (3, 1, 5000, 6, 2, 72, "bf16", "lens"),       # splits without any key that counts
    (1, 11, 3000, 9, 3, 40, "bf16", "both"),      # 33 rows of a key head: more than one tile
    (2, 40, 1500, 3, 1, 128, "f32", "lens"),      # 3 heads a key head, 120 rows
    (1, 700, 96, 7, 1, 64, "bf16", "holes"),      # rows that 32 does not divide into heads
    (5, 257, 128, 3, 3, 80, "bf16", "lens"),      # few keys, exactly two tiles
    (5, 257, 129, 3, 3, 80, "bf16", "none"),      # one more
    (32, 130, 64, 8, 8, 64, "bf16", "lens"),      # many heads: runs of them share an L2
    (17, 129, 65, 5, 5, 72, "f32", "holes"),      # numbers of heads that 8 does not divide
    (1, 4100, 40, 2, 2, 128, "bf16", "lens"),     # rows of the gradient shared out
    (1, 2049, 100, 2, 1, 96, "f32", "both"),
    (600, 1, 1, 1, 1, 32, "bf16", "none"),
    (2, 128, 512, 16, 16, 64, "bf16", "none"),
    (3, 1100, 300, 8, 8, 64, "bf16", "lens"),     # tiles of unlike sequences shared out alike
    (5, 1300, 130, 3, 3, 40, "f32", "lens"),
    (90, 300, 20, 2, 2, 32, "bf16", "both"),
]


@pytest.mark.parametrize("case", CUTS, ids=str)
def test_attention_every_cut(torch, case):  # noqa: F811
    say(f"[attention cut] {case}")
    _attention(torch, Attn(torch, *case))


SHARED_OUT = [
    # B, Lq, Lk, heads, kv, dim, type, mask: tiles of keys of many sequences, rows shared out
    (65, 600, 30, 1, 1, 32, "bf16", "lens"),      # one sequence past the first 64
    (100, 600, 20, 1, 1, 32, "bf16", "both"),
    (128, 130, 40, 1, 1, 64, "f32", "both"),
    (120, 600, 200, 1, 1, 24, "bf16", "lens"),    # one or two tiles, or none
    (256, 520, 33, 1, 1, 32, "bf16", "lens"),     # as many as are shared out
    (257, 520, 33, 1, 1, 32, "bf16", "lens"),     # one more: they are not
    (16, 520, 33, 16, 8, 32, "bf16", "holes"),    # heads by eight
]


@pytest.mark.parametrize("case", SHARED_OUT, ids=str)
def test_attention_many_sequences(torch, case):  # noqa: F811
    say(f"[attention, many sequences] {case}")
    _attention(torch, Attn(torch, *case))


@pytest.mark.parametrize("where", [None, 0, 63, 64, 199])
def test_attention_keys_of_one_sequence_only(torch, where):  # noqa: F811
    """All workgroups of a head go to one tile, or to none: more sharers than tiles of rows."""
    c = Attn(torch, 200, 520, 20, 1, 1, 32, "bf16", "none")
    c.lens = torch.zeros(200, dtype=torch.int32, device="cuda")
    if where is not None:
        c.lens[where] = 13
    c.ok = torch.arange(20, device="cuda") < c.lens[:, None]
    c.k[~c.ok], c.v[~c.ok] = float("nan"), float("inf")
    _attention(torch, c)


ONE_TOKEN = [
    # B, Lq, Lk, heads, kv, dim, type, mask: rows that fill a part of one tile only
    (8, 1, 77, 4, 4, 72, "bf16", "lens"),         # keys in LDS
    (8, 1, 77, 8, 2, 160, "bf16", "both"),
    (2, 1, 4096, 32, 8, 128, "bf16", "lens"),     # keys shared out
    (3, 8, 2000, 8, 8, 160, "bf16", "holes"),
    (2, 33, 1000, 2, 1, 64, "bf16", "both"),      # three waves with rows, one without
    (2, 97, 1000, 2, 2, 64, "bf16", "none"),
    (2, 1, 1000, 8, 4, 96, "f32", "lens"),
    (2, 65, 1000, 2, 2, 72, "f32", "both"),
]


@pytest.mark.parametrize("case", ONE_TOKEN, ids=str)
def test_attention_few_rows(torch, case):  # noqa: F811
    say(f"[attention, few rows] {case}")
    _attention(torch, Attn(torch, *case))


def test_attention_first_keys_do_not_count(torch):  # noqa: F811
    """Whole tiles without a key before the first one that counts, for rows of any number."""
    for Lq, dt in ((2, "bf16"), (200, "bf16"), (200, "f32")):
        c = Attn(torch, 1, Lq, 700, 2, 2, 64, dt, "none")
        c.mask = torch.zeros(1, 700, dtype=torch.bool, device="cuda")
        c.mask[0, 641] = True
        c.ok = c.mask.clone()
        c.k[:, :641] = float("nan")
        c.v[:, :641] = float("inf")
        _attention(torch, c)


def test_attention_scores_that_rise(torch):  # noqa: F811
    """Every tile's largest score well above all before it: the running maximum, and what is
    held by an older one, keep up; and falling ones, where it never moves again."""
    for sign in (1.0, -1.0):
        for Lq in (3, 150):
            c = Attn(torch, 1, Lq, 640, 2, 2, 64, "f32", "none")
            c.q.fill_(0.25)
            ramp = torch.linspace(0, 60, 640, device="cuda") * sign
            c.k[:] = ramp[None, :, None, None] * 0.25 + torch.randn_like(c.k) * 0.02
            _attention(torch, c)


def test_attention_scale(torch):  # noqa: F811
    from bit_post_quantization_amd import CrossAttention
    c = Attn(torch, 2, 50, 90, 2, 2, 64, "f32", "none")
    out = CrossAttention(2, 64, scale=0.5).forward(c.q * 0.25, c.k, c.v)
    assert torch.equal(out, c.layer().forward(c.q, c.k, c.v))  # powers of two


ROWS4_CUTS = [
    # M, K, N, group, x, s, act, bias
    (16, 2304, 25600, 32, "f32", "bf16", "silu", True),    # groups of 32: four tiles
    (4, 1152, 25601, 64, "f32", "f32", "none", False),     # six tiles, an odd width
    (16, 2320, 24600, 128, "bf16", "bf16", "silu", True),  # digits past LDS: read
    (9, 16384, 40, 64, "f32", "f32", "silu", True),        # inputs shared out
    (1, 65536, 20, 128, "bf16", "f32", "none", True),
    (50, 4096, 3300, 64, "f32", "bf16", "none", True),
    (31, 144, 8000, 32, "bf16", "f32", "silu", False),
    (1000, 64, 500, 64, "f32", "f32", "silu", True),
]


@pytest.mark.parametrize("case", ROWS4_CUTS, ids=str)
def test_rows4_every_cut(torch, case):  # noqa: F811
    say(f"[rows4 cut] {case}")
    c = Rows4(torch, *case)
    ref, tol = c.formula()
    _within(c.layer().apply(c.X), ref, tol, "Y")


def test_rows4_values_of_unlike_size(torch):  # noqa: F811
    """Fixed point drops up to 2^-31 of the largest of 128 inputs: a row with one value of
    2^20 keeps the others to 2^-11 each, and rows near the ends of the range come out."""
    c = Rows4(torch, 4, 512, 65, 128, "f32", "f32", "none", False)
    c.X[0, 5] = 2.0 ** 20
    c.X[1] *= 2.0 ** -100
    c.X[2] *= 2.0 ** 90
    c.X[3, ::2] = 0
    ref, tol = c.formula()
    unit = c.X.double().abs().view(4, 4, 128).amax(2, keepdim=True).expand(-1, -1, 128).reshape(4, 512)
    W = c.codes.double() * c.scales.double().repeat_interleave(128, 1)
    drop = 2.0 ** -31 * (unit @ W.abs().t())
    _within(c.layer().apply(c.X), ref, tol + drop, "Y")


HEADS_CUTS = [
    (1, 5, (40, 1, 1), 160, (100, 2), "halves", "bf16", "f32", "f32", "rms", "own"),
    (1, 2000, (1, 0, 0), 8, (8,), "halves", "f32", "f32", "f32", "rms", "shared"),
    (70, 3, (2, 2, 2), 56, (18, 10, 6), "halves", "f32", "bf16", "f32", "rms", "own"),
    (1, 4000, (3, 2, 1), 128, (2, 126), "halves", "bf16", "bf16", "f32", "rms", "float"),
    (3, 77, (0, 4, 4), 104, (), "adjacent", "bf16", "bf16", "bf16", "rms", "shared"),
    (1, 1, (500, 100, 100), 32, (16, 16), "adjacent", "f32", "bf16", "f32", "none", "shared"),
]


@pytest.mark.parametrize("case", HEADS_CUTS, ids=str)
def test_heads_every_cut(torch, case):  # noqa: F811
    say(f"[heads cut] {case}")
    c = Heads(torch, *case)
    outs = c.layer().forward(c.x, c.pos)
    for got, ref, tol, h in zip(outs, c.formula(c.x.double()), c.bounds(), c.heads):
        if h:
            _within(got, ref, tol + _round(torch, ref, got.dtype), "y")
    dx, dgq, dgk = c.layer().grad(c.dy, c.x, c.pos)
    ref, tol = c.grads()
    _within(dx, ref[0], tol[0] + _round(torch, ref[0], dx.dtype), "dx")
    if c.norm == "rms":
        for got, r, e in zip((dgq, dgk), ref[1:], tol[1:]):
            _within(got, r, e + _round(torch, r, got.dtype), "dgamma")


def test_heads_values_not_finite(torch):  # noqa: F811
    """A head with a NaN spoils itself only; a head of zeros stays zero; large values whose
    squares fit fp32 are normed."""
    c = Heads(torch, 1, 6, (2, 1, 1), 64, (32, 32), "halves", "f32", "f32", "f32", "rms", "shared")
    x = c.x.clone().view(1, 6, 4, 64)
    x[0, 1, 0, 3] = float("nan")
    x[0, 2, 1] = 0
    x[0, 3] *= 1e17
    q, k, v = c.layer().forward(x.view(1, 6, 256), c.pos)
    assert bool(torch.isnan(q[0, 1, 0]).all()) and int(torch.isnan(q).sum()) == 64
    assert bool((q[0, 2, 1] == 0).all()) and bool(torch.isfinite(k).all())
    ref = c.formula(x.double().view(1, 6, 256))
    bound = 32 * EPS * 8.0 * 1.9 * 2  # of a pair: norms of at most sqrt(64), gammas below 1.9
    assert bool(((q[0, 3].double() - ref[0][0, 3]).abs() <= bound).all())


# ------------------------------------------------------------ streams, graphs ----

def test_two_calls_at_once(torch):  # noqa: F811
    """The same layers on two streams at the same time, other inputs on each."""
    r = [Rows4(torch, 8, 4096, 300, 64, "f32", "f32", "silu", True, s) for s in (0, 1)]
    r[1].codes, r[1].scales, r[1].bias = r[0].codes, r[0].scales, r[0].bias
    h = [Heads(torch, 2, 300, (4, 4, 4), 72, (36, 36), "adjacent", "f32", "bf16", "f32", "rms",
               "shared", s) for s in (0, 1)]
    a = [Attn(torch, 2, 300, 400, 4, 2, 64, "bf16", "none", s) for s in (0, 1)]
    rows, heads, attn = r[0].layer(), h[0].layer(), a[0].layer()

    def run(i):
        o, lse = attn.forward(a[i].q, a[i].k, a[i].v, save=True)
        return [rows.apply(r[i].X), *heads.forward(h[i].x, h[i].pos),
                *heads.grad(h[i].dy, h[i].x, h[i].pos), o, lse,
                *attn.grad(a[i].dout, a[i].q, a[i].k, a[i].v, o, lse)]

    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        for outs in got[i]:
            for x, y in zip(outs, want[i]):
                assert torch.equal(x, y)


def test_given_stream(torch):  # noqa: F811
    c = Attn(torch, 1, 50, 60, 2, 2, 64, "f32", "none")
    h = Heads(torch, 1, 9, (2, 2, 2), 64, (64,), "adjacent", "f32", "f32", "f32", "rms", "shared")
    r = Rows4(torch, 2, 64, 20, 32, "f32", "f32", "none", False)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    layer, heads, rows = c.layer(), h.layer(), r.layer()
    for s in (side, side.cuda_stream):
        got = [layer.forward(c.q, c.k, c.v, stream=s), *heads.forward(h.x, h.pos, stream=s),
               rows.apply(r.X, stream=s)]
        side.synchronize()
        want = [layer.forward(c.q, c.k, c.v), *heads.forward(h.x, h.pos), rows.apply(r.X)]
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_captured_calls_with_much_lds(torch):  # noqa: F811
    """Rows whose digits fill LDS, the kinds of attention that use most of it: replayed with
    eager work between, against eager calls."""
    r = Rows4(torch, 8, 4096, 400, 64, "bf16", "bf16", "silu", True)
    wide = Rows4(torch, 40, 1024, 400, 32, "f32", "f32", "none", True)
    a = [Attn(torch, 1, 140, 200, 2, 2, 160, dt, "none") for dt in ("f32", "bf16")]
    few = Attn(torch, 1, 2, 900, 2, 2, 160, "bf16", "none")
    rows, wider, attn = r.layer(), wide.layer(), a[0].layer()

    def run():
        outs = [rows.apply(r.X), wider.apply(wide.X), attn.forward(few.q, few.k, few.v)]
        for c in a:
            o, lse = attn.forward(c.q, c.k, c.v, save=True)
            outs += [o, lse, *attn.grad(c.dout, c.q, c.k, c.v, o, lse)]
        return outs

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run()
    for i in range(3):
        r.X.mul_(0.9)
        a[0].q.add_(0.01)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, run()):
            assert torch.equal(x, y)


def test_rows_behind_are_left_alone(torch):  # noqa: F811
    """Outputs into the middle of larger buffers: nothing before, behind or between changes."""
    c = Attn(torch, 2, 33, 47, 3, 3, 72, "bf16", "lens")
    layer = c.layer()
    out, lse = layer.forward(c.q, c.k, c.v, lens=c.lens, save=True)

    def room(t):
        big = torch.full((t.shape[0] + 2, t.shape[1] + 3, t.shape[2] + 1, 80), 9.0, dtype=t.dtype,
                         device="cuda")
        return big, big[1:-1, 2:-1, :-1, :72]

    bigs, into = zip(*(room(t) for t in (c.q, c.k, c.v)))
    big, o = room(c.q)
    assert torch.equal(layer.forward(c.q, c.k, c.v, lens=c.lens, out=o), out)
    grads = layer.grad(c.dout, c.q, c.k, c.v, out, lse, lens=c.lens)
    for x, y in zip(layer.grad(c.dout, c.q, c.k, c.v, out, lse, lens=c.lens, into=into), grads):
        assert torch.equal(x, y)
    for b, t in ((big, c.q), *zip(bigs, (c.q, c.k, c.v))):
        assert int((b != 9).sum()) <= t.numel()
        b[1:-1, 2:-1, :-1, :72] = 9.0
        assert bool((b == 9).all())


def test_math_of_the_bounds():
    """The bound's own ingredients: half a step of each type."""
    import torch as t
    assert EPS == t.finfo(t.float32).eps / 2 and 2.0 ** -8 == t.finfo(t.bfloat16).eps / 2
    assert math.isclose(1 / math.log(2), 1.4426950408889634)

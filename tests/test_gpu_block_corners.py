"""Corners of a conditioned block's operators, infinities first. Formulas, bounds and inputs
are those of test_gpu_block.py."""
from __future__ import annotations

import math

import pytest

from tests.parity import say
from tests.test_gpu_block import (EPS, Attn, Heads, Rows4, _gen, _round, _same_lse,  # noqa: F401
                                  _sum, _within, torch)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention ----

ALL_LOW = [
    # Lq, Lk, heads, kv, dim, type: every way the forward pass ends
    (40, 100, 2, 2, 64, "bf16"),     # keys in LDS
    (100, 100, 2, 2, 72, "f32"),
    (200, 200, 2, 1, 64, "bf16"),    # tiles of keys
    (70, 100, 2, 2, 160, "f32"),
    (3, 100, 4, 2, 64, "f32"),       # waves that share the keys
    (3, 1500, 4, 2, 64, "f32"),      # parts joined
    (5, 1500, 2, 2, 128, "bf16"),
]


@pytest.mark.parametrize("case", ALL_LOW, ids=str)
def test_attention_every_score_minus_infinity(torch, case):  # noqa: F811
    """A query whose keys count and all score -infinity has no softmax: NaN, as the formula
    says, and so have its gradients. One without keys still gets 0, and neither touches
    another sequence."""
    say(f"[attention, all scores -inf] {case}")
    Lq, Lk, H, G, D, dt = case
    c = Attn(torch, 4, Lq, Lk, H, G, D, dt, "holes")
    c.lens = torch.tensor([Lk, Lk, 0, Lk // 2], dtype=torch.int32, device="cuda")
    c.mask[:, 0] = True
    c.ok = c.mask & (torch.arange(Lk, device="cuda") < c.lens[:, None])
    c.q[:] = c.q.abs() + 0.1
    c.k[1], c.v[1] = c.k[1].nan_to_num(), c.v[1].nan_to_num(posinf=0.0)
    for b in (0, 3):
        c.k[b] = torch.where(c.ok[b, :, None, None], -math.inf, 1.0).to(c.k.dtype)
        c.v[b] = 1.0
    layer = c.layer()
    out, lse = layer.forward(c.q, c.k, c.v, lens=c.lens, mask=c.mask, save=True)
    grads = layer.grad(c.dout, c.q, c.k, c.v, out, lse, lens=c.lens, mask=c.mask)
    dq, dk, dv = grads
    for b in (0, 3):
        assert bool(out[b].isnan().all()) and bool(lse[b].isnan().all())
        assert bool(dq[b].isnan().all())
        for d in (dk, dv):
            assert bool(d[b, c.ok[b]].isnan().all()) and bool((d[b, ~c.ok[b]] == 0).all())
    assert bool((out[2] == 0).all()) and bool((lse[2] == -math.inf).all())
    assert all(bool((d[2] == 0).all()) for d in grads)
    one = Attn(torch, 1, Lq, Lk, H, G, D, dt, "none")
    one.q, one.k, one.v, one.dout, one.ok = (x[1:2] for x in (c.q, c.k, c.v, c.dout, c.ok))
    ref, tol, ref_lse, lse_tol = one.forward()
    _within(out[1:2], ref, tol + _round(torch, ref, out.dtype), "out")
    _same_lse(torch, lse[1:2], ref_lse, lse_tol)
    ref, tol = one.grads(out[1:2], lse[1:2])
    for g, r, e, name in zip(grads, ref, tol, ("dq", "dk", "dv")):
        _within(g[1:2], r, e + _round(torch, r, g.dtype), name)


LOW_KEY = [
    # Lq, Lk, heads, kv, dim, type: rows that do not fill their last tile
    (40, 70, 2, 2, 64, "bf16"),
    (45, 70, 4, 2, 72, "f32"),
    (33, 200, 6, 2, 128, "bf16"),
    (1301, 40, 2, 2, 64, "bf16"),    # rows shared out
    (301, 77, 2, 2, 96, "f32"),
]


@pytest.mark.parametrize("case", LOW_KEY, ids=str)
def test_attention_grad_of_a_key_that_scores_minus_infinity(torch, case):  # noqa: F811
    """A key of -infinity that counts weighs nothing: its gradients are sums of zeros. (Those
    of the queries hold 0 times the key, NaN.)"""
    say(f"[attention grad, a key of -inf] {case}")
    c = Attn(torch, 2, *case, "none")
    c.q[:] = c.q.abs() + 0.1
    c.k[:, 7] = -math.inf
    out, lse = c.layer().forward(c.q, c.k, c.v, save=True)
    dq, dk, dv = c.layer().grad(c.dout, c.q, c.k, c.v, out, lse)
    c.ok[:, 7] = False
    ref, tol = c.grads(out, lse)
    assert bool(dq.isnan().all())
    _within(dk, ref[1], tol[1] + _round(torch, ref[1], dk.dtype), "dk")
    _within(dv, ref[2], tol[2] + _round(torch, ref[2], dv.dtype), "dv")


# --------------------------------------------------------------- norms, turns ----

def _same(torch, got, ref, tol, what):  # noqa: F811
    """Within the bound where the formula is finite, and infinite or NaN where it is."""
    got, fin = got.double(), ref.isfinite()
    assert torch.equal(got.isnan(), ref.isnan()), what
    assert torch.equal(got.isinf(), ref.isinf()), what
    assert bool(((got - ref).abs() <= tol)[fin].all()), what


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("x,norm", [("f32", "none"), ("f32", "rms"), ("bf16", "none")])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_heads_infinite_channel_that_does_not_turn(torch, pairs, x, norm, shift):  # noqa: F811
    """Channels past the axes' do not turn: an infinity in one stays there. ``shift``: rows
    that no vector load is aligned to."""
    c = Heads(torch, 1, 12, (2, 1, 1), 40, (10, 6), pairs, x, "f32", "f32", norm, "own")
    v = c.x.view(1, 12, 4, 40)
    v[0, 1, 0, 20], v[0, 2, 1, 39], v[0, 3, 2, 16] = math.inf, -math.inf, math.inf
    wide = torch.zeros(1, 12, 160 + shift, device="cuda", dtype=c.x.dtype)
    wide[:, :, shift:] = c.x
    ref = c.formula(c.x.double())
    tol = [t.nan_to_num(0.0, 0.0) for t in c.bounds()]
    for got, r, e in zip(c.layer().forward(wide[:, :, shift:], c.pos), ref, tol):
        _same(torch, got, r, e + _round(torch, r, got.dtype).nan_to_num(0.0, 0.0), "y")
    if norm == "none":
        c.dy[0][0, 4, 1, 17], c.dy[1][0, 5, 0, 30] = math.inf, math.nan
        dx, _, _ = c.layer().grad(c.dy, wide[:, :, shift:], c.pos)
        ref, tol = c.grads()
        _same(torch, dx, ref[0], tol[0].nan_to_num(0.0, 0.0)
              + _round(torch, ref[0], dx.dtype).nan_to_num(0.0, 0.0), "dx")


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_heads_at_position_zero(torch, pairs):  # noqa: F811
    """Not turned yet: every channel is what it was, infinities beside others and NaN."""
    c = Heads(torch, 1, 12, (2, 1, 1), 40, (10, 6), pairs, "f32", "f32", "f32", "none", "own")
    c.x[0, 3, 0:90:7], c.x[0, 4, 1:90:9] = math.inf, math.nan
    c.pos.zero_()
    for got, ref in zip(c.layer().forward(c.x, c.pos), c.split(c.x)):
        assert torch.equal(got.nan_to_num(9e9), ref.nan_to_num(9e9))
        assert torch.equal(got.isnan(), ref.isnan())


HEADS_LDS = [
    # heads long and few, positions many: a workgroup's tokens and rooms fill LDS
    (1, 3000, (1, 1, 1), 160, (40, 60, 60), "halves", "bf16", "bf16", "f32", "rms", "shared"),
    (1, 3000, (1, 1, 1), 136, (40, 40, 40), "halves", "bf16", "f32", "f32", "rms", "own"),
    (2, 1500, (2, 1, 1), 120, (120,), "halves", "bf16", "bf16", "bf16", "rms", "shared"),
    (1, 3000, (1, 1, 1), 112, (40, 40), "halves", "bf16", "bf16", "f32", "none", "shared"),
    (1, 3000, (1, 1, 1), 160, (160,), "halves", "f32", "f32", "f32", "rms", "shared"),
    (1, 40000, (1, 0, 0), 160, (80, 80), "halves", "bf16", "bf16", "f32", "rms", "shared"),
]


@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("case", HEADS_LDS, ids=str)
def test_heads_with_much_lds(torch, case, shift):  # noqa: F811
    say(f"[heads, much LDS] {case} {shift}")
    c = Heads(torch, *case)
    wide = torch.zeros(*c.x.shape[:2], c.x.shape[2] + shift, device="cuda", dtype=c.x.dtype)
    wide[:, :, shift:] = c.x
    for got, ref, tol, h in zip(c.layer().forward(wide[:, :, shift:], c.pos),
                                c.formula(c.x.double()), c.bounds(), c.heads):
        if h:
            _within(got, ref, tol + _round(torch, ref, got.dtype), "y")
    dx, dgq, dgk = c.layer().grad(c.dy, wide[:, :, shift:], c.pos)
    ref, tol = c.grads()
    _within(dx, ref[0], tol[0] + _round(torch, ref[0], dx.dtype), "dx")
    if c.norm == "rms":
        for got, r, e in zip((dgq, dgk), ref[1:], tol[1:]):
            _within(got, r, e + _round(torch, r, got.dtype), "dgamma")


@pytest.mark.parametrize("x,y", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_heads_neighbours_in_unaligned_rows(torch, x, y):  # noqa: F811
    c = Heads(torch, 2, 33, (3, 2, 2), 72, (36, 20), "adjacent", x, y, "f32", "rms", "own")
    wide = torch.full((2, 33, 3 + 7 * 72 + 4), math.nan, device="cuda", dtype=c.x.dtype)
    wide[:, :, 3:-4] = c.x
    for got, ref, tol in zip(c.layer().forward(wide[:, :, 3:-4], c.pos), c.formula(c.x.double()),
                             c.bounds()):
        _within(got, ref, tol + _round(torch, ref, got.dtype), "y")
    dx, dgq, dgk = c.layer().grad(c.dy, wide[:, :, 3:-4], c.pos)
    ref, tol = c.grads()
    for got, r, e in zip((dx, dgq, dgk), ref, tol):
        _within(got, r, e + _round(torch, r, got.dtype), "gradient")


@pytest.mark.parametrize("shift", [0, 8, 3])
def test_heads_grad_into_strided_rows(torch, shift):  # noqa: F811
    """dx with strides of its own, as the C ABI takes them: a slice of wider rows of a longer
    sequence, with and without room for vectors."""
    from bit_post_quantization_amd import block
    c = Heads(torch, 2, 21, (3, 2, 2), 64, (32, 16), "halves", "bf16", "bf16", "f32", "rms", "own")
    layer = c.layer()
    want = layer.grad(c.dy, c.x, c.pos)
    width = c.x.shape[2]
    room = torch.full((2, 30, width + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = room[:, 4:25, shift:shift + width]
    dev, s, size, xb, xr, at, pb = layer._call(c.x, c.pos)
    dq, dk, dv = layer._views(c.dy, ("dq", "dk", "dv"), dev, size)
    dgq, dgk = torch.empty_like(c.gq), torch.empty_like(c.gk)
    ws = torch.empty(size[1], dtype=torch.uint8, device="cuda")
    block.qlinear_heads_grad(size[0], dq, dk, dv, c.x.data_ptr(), xb, xr, at, pb, dx.data_ptr(),
                             dx.stride(0), dx.stride(1), dgq.data_ptr(), dgk.data_ptr(),
                             ws.data_ptr(), size[1], s)
    for a, b in zip((dx, dgq, dgk), want):
        assert torch.equal(a, b)
    dx.fill_(7.0)
    assert bool((room == 7).all())


# ----------------------------------------------------------------- 4-bit rows ----

def test_rows4_bound_of_one_input(torch):  # noqa: F811
    """Each output reads one small input behind a code of 7, and none the unit's large one:
    off by no more than 1.004 * 2^-31 of that large one (half a step of the fixed point, which
    lies 31 bits below its power of two; 30 where it is within 0.4 % of the next), times 7,
    and two roundings."""
    from bit_post_quantization_amd import GroupLinear4
    K, N, M = 128, 127, 64
    codes = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    codes[torch.arange(N), torch.arange(1, K)] = 7
    layer = GroupLinear4.from_codes(codes, torch.ones(N, 1, device="cuda"), 128)
    X = torch.empty(M, K, device="cuda").normal_(generator=_gen(torch, 1))
    large = 2.0 ** 10 * torch.linspace(1.0, 2.0, M, device="cuda")
    large[1], large[2] = 2047.9999, -2.0 ** 10 * 1.9922  # next to the border
    X[:, 0] = large
    got = layer.apply(X).double()
    ref = 7 * X[:, 1:].double()
    step = 1.004 * 2.0 ** -31 * large.double().abs()[:, None]
    bound = 7 * step + 2 * EPS * (ref.abs() + 7 * step)
    worst = float(((got - ref).abs() / bound).max())
    say(f"  worst {worst:.3f} of the bound")
    assert worst <= 1.0


@pytest.mark.parametrize("power", [-112, -105, -95, 60, 96])
def test_rows4_rows_of_any_size(torch, power):  # noqa: F811
    """The fixed point follows a row's size: down to 2^-114, where it stays, and up to where
    the sums themselves leave fp32 (codes and scales of up to 9 and 512 inputs of up to 8
    make 2^16)."""
    c = Rows4(torch, 3, 512, 65, 64, "f32", "f32", "none", False)
    c.X *= 2.0 ** power
    ref, tol = c.formula()
    _within(c.layer().apply(c.X), ref, tol, "Y")


def test_rows4_from_two_host_threads(torch):  # noqa: F811
    """Calls of one kernel with unlike needs of LDS, from two threads at once."""
    import threading
    from bit_post_quantization_amd import GroupLinear4
    c = Rows4(torch, 8, 4096, 400, 64, "f32", "f32", "silu", True)
    layer = c.layer()
    assert isinstance(layer, GroupLinear4)
    want = {m: layer.apply(c.X[:m]) for m in (8, 5)}
    torch.cuda.synchronize()
    failed = []

    def calls(m):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                outs = [layer.apply(c.X[:m]) for _ in range(300)]
                torch.cuda.current_stream().synchronize()
            failed.extend(m for o in outs if not torch.equal(o, want[m]))
        except Exception as e:  # noqa: BLE001  (a thread's failure is reported by the test)
            failed.append(e)

    threads = [threading.Thread(target=calls, args=(m,)) for m in (8, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:3]


ROWS4_TILES = [
    # M, K, N, group, x, s, act, bias: six tiles, four and two of every form that takes them, and
    # widths next to where a round of workgroups ends
    (8, 2304, 24576, 32, "bf16", "bf16", "silu", True),
    (4, 1152, 24600, 32, "f32", "bf16", "none", True),
    (8, 2304, 24600, 32, "f32", "f32", "none", False),
    (16, 4096, 12288, 32, "bf16", "bf16", "none", True),
    (16, 4096, 12300, 64, "bf16", "f32", "silu", True),
    (16, 4096, 24576, 64, "f32", "bf16", "none", False),
    (2, 128, 4096, 128, "f32", "f32", "none", True),
    (2, 128, 4097, 128, "f32", "f32", "none", True),
    (1, 128, 8208, 64, "bf16", "f32", "silu", True),
    (3, 256, 24592, 64, "f32", "bf16", "none", True),
    (20, 256, 8200, 32, "bf16", "f32", "none", True),
    (40, 256, 4500, 32, "f32", "bf16", "none", True),
]


@pytest.mark.parametrize("case", ROWS4_TILES, ids=str)
def test_rows4_tiles_of_a_workgroup(torch, case):  # noqa: F811
    say(f"[rows4 tiles] {case}")
    c = Rows4(torch, *case)
    ref, tol = c.formula()
    _within(c.layer().apply(c.X), ref, tol, "Y")


def test_rows4_largest_weights(torch):  # noqa: F811
    """One code short of 2^34: packed, multiplied and unpacked, with the last rows of the
    weights as the first."""
    from bit_post_quantization_amd import GroupLinear4
    N, K, group = 1649373, 10416, 128
    g = _gen(torch, 7)
    codes = torch.empty(N, K, dtype=torch.int8, device="cuda")
    for part in codes.split(1 << 17):
        part.random_(-8, 8, generator=g)
    scales = torch.rand(N, -(-K // group), generator=g, device="cuda") + 0.5
    layer = GroupLinear4.from_codes(codes, scales, group)
    X = torch.empty(2, K, device="cuda").normal_(generator=g)
    y = layer.apply(X)
    some = torch.cat([torch.arange(64), torch.arange(N - 64, N),
                      torch.randint(0, N, (128,), generator=torch.Generator().manual_seed(1))])
    some = some.cuda()
    W = codes[some].double() * scales[some].double().repeat_interleave(group, 1)[:, :K]
    x = X.double()
    _within(y[:, some], x @ W.t(), (8 * EPS + _sum(K)) * (x.abs() @ W.abs().t()), "Y")
    got, got_scales = layer.weights()
    assert torch.equal(got_scales, scales)
    assert all(torch.equal(a, b) for a, b in zip(got.split(1 << 17), codes.split(1 << 17)))

"""The streaming operators against plain 64-bit forms (_stream_ref), at the sizes,
strides, masks and lengths where they can go wrong."""
import math

import pytest
import torch

import _stream_ref as ref
import cluster_routed_sparse_b200 as crs
from cluster_routed_sparse_b200 import _lib

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# ------------------------------------------------------------------ rotary embedding
ROPE_TOL = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def assert_rotated(y, x, pos, pairs, fr, interleaved, inverse=False):
    # one rounding of the output; sine and cosine are off by 2^-23 (half a step of the fp32
    # half turns, pi 2^-25, and 2 ulp of sincospi), two products and a sum by 3 * 2^-24 more
    want = ref.rotate(x, pos, pairs, fr, interleaved, inverse)
    pair = 2 * x.double().abs().amax(-1, keepdim=True)
    tol = ROPE_TOL[x.dtype] * want.abs() + 2.0 ** -21 * pair
    # fp16 has subnormals: half a step of 2^-24 there
    tol = tol + (2.0 ** -25 if x.dtype == torch.float16 else 0)
    assert bool(((y.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("B,L,Hq,Hk,d,pairs", [
    (1, 1, 1, 1, 64, (32,)),
    (2, 129, 5, 5, 128, (22, 21, 21)),
    (1, 77, 6, 2, 64, (8, 12, 8)),       # 4 pairs stay as they are
    (1, 33, 3, 1, 64, (7, 5, 11)),       # an odd number of pairs: rows that do not split on 16 bytes
    (3, 260, 17, 4, 128, (16, 24, 24)),
    (1, 5, 2, 2, 256, (64, 32, 16, 16)),
    (1, 9, 2, 2, 10, (1, 0, 2)),
])
def test_rope(dtype, interleaved, B, L, Hq, Hk, d, pairs):
    g = gen(L + d)
    q, k = normal(g, B, L, Hq, d, dtype=dtype).transpose(1, 2), normal(g, B, Hk, L, d, dtype=dtype)
    pos = torch.randint(-50, 3000, (B, L, len(pairs)), generator=g, device="cuda", dtype=torch.int32)
    fr = ref.freqs(pairs)
    oq, ok = crs.rope_axes(q, k, pos, pairs, interleaved=interleaved)
    assert oq.is_contiguous() and oq.shape == q.shape
    assert_rotated(oq, q, pos, pairs, fr, interleaved)
    assert_rotated(ok, k, pos, pairs, fr, interleaved)
    # one tensor alone, positions shared by the sequences, backwards, in place
    y = q.clone()
    alone = crs.rope_axes(y, None, pos[0].contiguous(), pairs, interleaved=interleaved, inverse=True, out=(y, None))
    assert alone is y
    assert_rotated(y, q, pos[:1].expand(B, L, -1), pairs, fr, interleaved, inverse=True)


def test_rope_far_positions_given_frequencies_and_odd_views():
    g = gen(3)
    pos = torch.tensor([[2**31 - 1, 1000000], [-2**31, 999999937], [0, 1]], device="cuda", dtype=torch.int32)
    pairs = (13, 9)
    fr = [2.0 ** -i for i in range(13)] + [3.0, 1.25, 0.5, 0.0, -0.25, 1e-3, 7.5, 2.0 ** -20, 1.0]
    base = normal(g, 1, 3, 4 * 64 + 1, dtype=torch.float32)
    x = base[..., 1:].unflatten(-1, (4, 64)).transpose(1, 2)  # rows on 4-byte boundaries only
    y = crs.rope_axes(x, None, pos, pairs, freqs=fr)
    # 64-bit floats keep pos * freq to 2^-52 of up to 2^34: too little, so the reference takes exact fractions
    from fractions import Fraction
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021")
    ax = [0] * 13 + [1] * 9
    want = x.double().clone()
    for l in range(3):
        for p, f in enumerate(fr):
            turn = (int(pos[l, ax[p]]) * Fraction(f) / two_pi) % 1
            c, s = math.cos(2 * math.pi * float(turn)), math.sin(2 * math.pi * float(turn))
            a, b = x[0, :, l, 2 * p].double(), x[0, :, l, 2 * p + 1].double()
            want[0, :, l, 2 * p], want[0, :, l, 2 * p + 1] = a * c - b * s, a * s + b * c
    tol = 2.0 ** -24 * want.abs() + 2.0 ** -21 * 2 * x.double().abs().amax(-1, keepdim=True)
    assert bool(((y.double() - want).abs() <= tol).all())


def test_rope_gradient_against_differences_and_formula():
    """sum(w * rope(x)) has the gradient rope^-1(w); fp32, both by the formula and by central differences."""
    g = gen(9)
    x, w = normal(g, 1, 1, 3, 16, dtype=torch.float32), normal(g, 1, 1, 3, 16, dtype=torch.float32)
    pos = torch.tensor([[0, 5], [7, 1], [100, 30]], device="cuda", dtype=torch.int32)
    grad = crs.rope_axes(w, None, pos, (3, 4), interleaved=False, inverse=True)
    h = 0.25  # the map is linear: a large step has no truncation error
    for l in range(3):
        for e in range(16):
            up, dn = x.clone(), x.clone()
            up[0, 0, l, e] += h
            dn[0, 0, l, e] -= h
            f = [float((w.double() * crs.rope_axes(t, None, pos, (3, 4), interleaved=False).double()).sum()) for t in (up, dn)]
            # each f: 48 terms |w y| < 10 with y off by 2^-21 * 8
            assert abs((f[0] - f[1]) / (2 * h) - float(grad[0, 0, l, e])) < 48 * 10 * 8 * 2.0 ** -21 / h


def test_rope_empty_and_passed_values():
    pos = torch.zeros(4, 1, device="cuda", dtype=torch.int32)
    assert crs.rope_axes(torch.empty(1, 2, 0, 64, device="cuda", dtype=torch.bfloat16), None,
                         pos[:0], (32,)).shape == (1, 2, 0, 64)
    x = torch.full((1, 1, 4, 64), math.inf, device="cuda", dtype=torch.bfloat16)
    x[..., :16] = 1
    y = crs.rope_axes(x, None, pos, (8,))  # what does not turn is copied, infinities too
    assert torch.equal(y, x)


# ------------------------------------------------------------------ window attention
CASES = [
    # B, Hq, Hk, Lq, Lk, d, left, right, sinks, block
    (1, 1, 1, 1, 1, 64, -1, 0, 0, 1),
    (1, 2, 2, 128, 128, 128, -1, -1, 0, 1),
    (1, 1, 1, 300, 300, 64, -1, 0, 0, 1),
    (2, 3, 3, 257, 257, 128, 31, 0, 4, 1),
    (1, 2, 1, 129, 513, 128, 63, 63, 200, 1),
    (1, 4, 2, 384, 384, 64, 1, 0, 48, 48),      # frames
    (1, 2, 2, 500, 500, 128, 2, 1, 50, 50),
    (2, 6, 2, 190, 333, 64, 40, 7, 3, 1),       # three query heads share a key head
    (1, 5, 1, 100, 700, 128, 100, 0, 1, 1),
    (1, 8, 1, 37, 1000, 128, -1, 0, 0, 1),
    (1, 16, 1, 3, 1500, 64, 600, 0, 20, 1),
    (1, 2, 2, 400, 150, 128, -1, 0, 0, 1),      # more queries than keys: the first rows see nothing
    (1, 2, 2, 400, 150, 64, 3, 2, 9, 7),
    (1, 1, 1, 256, 1024, 128, 0, 0, 0, 1),      # a row sees one key
    (3, 2, 2, 1, 777, 128, 300, 0, 16, 1),      # single tokens
    (2, 40, 8, 1, 2049, 128, -1, 0, 0, 1),
    (2, 16, 1, 1, 131, 64, -1, -1, 0, 1),
    (1, 4, 4, 5, 4097, 128, 1000, 0, 64, 1),
    (1, 2, 2, 640, 640, 128, 0, 0, 700, 64),    # first tokens past the diagonal: only those not ahead
    (1, 128, 1, 2, 200, 64, -1, 0, 0, 1),
    (2, 40, 40, 300, 1100, 64, -1, 0, 0, 1),    # many tiles to a block, with padding in the last
    (1, 40, 40, 1000, 1300, 128, -1, 200, 0, 1),
    (1, 2, 1, 3, 40000, 64, -1, 0, 0, 1),       # one head, many keys: many parts to join
    (1, 1, 1, 1, 70001, 128, 65000, 0, 100, 1),
    (1, 16, 1, 2, 9000, 128, -1, 0, 0, 1),
]


def tensors(case, seed=0):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    g = gen(1000 + seed)
    q, k, v = normal(g, B, Hq, Lq, d), normal(g, B, Hk, Lk, d), normal(g, B, Hk, Lk, d)
    return q, k * 1.5 + 0.5, v, normal(g, B, Hq, Lq, d)


def rule(case):
    return dict(left=case[6], right=case[7], sinks=case[8], block=case[9])


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("ragged", [False, True])
def test_window_attn(case, ragged):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    q, k, v, _ = tensors(case)
    q_lens = k_lens = None
    if ragged:  # lengths down to zero, garbage behind them
        q_lens = torch.tensor([(Lq * (3 - b)) // 3 for b in range(B)], device="cuda", dtype=torch.int32)
        k_lens = torch.tensor([(Lk * (b + 1)) // (B + 1) for b in range(B)], device="cuda", dtype=torch.int32)
        for b in range(B):
            k[b, :, int(k_lens[b]):] = math.nan
            v[b, :, int(k_lens[b]):] = math.inf
            q[b, :, int(q_lens[b]):] = math.nan
    o, lse = crs.window_attn(q, k, v, return_lse=True, q_lens=q_lens, k_lens=k_lens, **rule(case))
    crs.ops_status()
    mask = ref.visible(B, Lq, Lk, *case[6:], q_lens, k_lens)
    r = ref.attention(q, k, v, mask)
    ref.check("o", o, r)
    ref.check("lse", lse, r)
    again = crs.window_attn(q, k, v, q_lens=q_lens, k_lens=k_lens, **rule(case))
    assert torch.equal(again, o)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("ragged", [False, True])
def test_window_attn_backward(case, ragged):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    q, k, v, g = tensors(case, 1)
    q_lens = k_lens = None
    if ragged:
        q_lens = torch.tensor([(Lq * (b + 1)) // (B + 1) for b in range(B)], device="cuda", dtype=torch.int32)
        k_lens = torch.tensor([(Lk * (3 - b)) // 3 for b in range(B)], device="cuda", dtype=torch.int32)
        for b in range(B):
            for x, n in ((k, k_lens), (v, k_lens), (q, q_lens), (g, q_lens)):
                x[b, :, int(n[b]):] = math.nan
    kw = dict(q_lens=q_lens, k_lens=k_lens, **rule(case))
    o, lse = crs.window_attn(q, k, v, return_lse=True, **kw)
    dq, dk, dv = crs.window_attn_backward(g, q, k, v, o, lse, **kw)
    crs.ops_status()
    r = ref.attention(q, k, v, ref.visible(B, Lq, Lk, *case[6:], q_lens, k_lens), d_out=g)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        ref.check(name, x, r)
    for a, b in zip((dq, dk, dv), crs.window_attn_backward(g, q, k, v, o, lse, **kw)):
        assert torch.equal(a, b)  # the same bits every time


@pytest.mark.parametrize("cached", [False, True])
@pytest.mark.parametrize("case", [
    (4, 1, 1, 200, 2000, 128, -1, 0, 0, 1),
    (4, 2, 2, 200, 900, 64, 300, 0, 130, 1),
    (3, 5, 1, 13, 5000, 128, -1, -1, 0, 1),
    (4, 8, 1, 20, 1300, 128, 200, 0, 40, 1),
    (2, 1, 1, 30, 130, 64, 3, 3, 1, 1),
    (40, 4, 4, 140, 700, 64, 500, 0, 100, 1),   # enough heads that no key is split off
    (40, 4, 4, 100, 200, 128, -1, 50, 0, 1),
])
def test_one_tile_of_queries(case, cached):
    """Sequences whose queries fill at most one row tile of two, and lengths that leave the other one,
    or both, behind the sequence: those rows get zeros whatever the output held."""
    B, Hq, Hk, Lq, Lk, d = case[:6]
    q, k, v, _ = tensors(case, 3)
    ints = dict(device="cuda", dtype=torch.int32)
    q_lens = torch.tensor([(Lq, 5, 0, min(130, Lq))[b % 4] for b in range(B)], **ints)
    k_lens = torch.tensor([(Lk, Lk - 7, 60, 129, 0)[b % 5] for b in range(B)], **ints)
    out = torch.full_like(q, math.nan)
    kw = dict(q_lens=q_lens, out=out, return_lse=True, **rule(case))
    if cached:
        T = 32
        per = (Lk + T - 1) // T
        c = crs.Cache8.empty(B * per, Hk, T, d)
        table = torch.randperm(B * per, generator=gen(1), device="cuda").view(B, per).to(torch.int32)
        crs.cache8_append(k, v, c, table, torch.zeros(B, **ints), k_lens)
        o, lse = crs.cache8_attn(q, c, table, k_lens, **kw)
        k, v = dense(c, table, Lk)
        keep = torch.arange(Lk, device="cuda").view(1, 1, Lk, 1) < k_lens.view(B, 1, 1, 1)
        k, v = torch.where(keep, k, 0.0), torch.where(keep, v, 0.0)
    else:
        for b in range(B):
            k[b, :, int(k_lens[b]):] = math.nan
            v[b, :, int(k_lens[b]):] = math.nan
        o, lse = crs.window_attn(q, k, v, k_lens=k_lens, **kw)
    crs.ops_status()
    r = ref.attention(q, k, v, ref.visible(B, Lq, Lk, *case[6:], q_lens, k_lens))
    ref.check("o", o, r)
    ref.check("lse", lse, r)


def test_window_attn_strided_views_and_scale():
    """[B, L, H, d] projections and one fused tensor for q, k and v; outputs written into views."""
    B, H, L, d = 2, 3, 210, 64
    g = gen(5)
    qkv = normal(g, B, L, 3, H, d)
    q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
    go = normal(g, B, L, H, d).transpose(1, 2)
    buf = torch.full((B, L, 4, H, d), 7.0, device="cuda", dtype=torch.bfloat16)
    views = [buf[:, :, i].transpose(1, 2) for i in range(4)]
    w = dict(left=33, right=5, sinks=2, scale=0.07)
    o, lse = crs.window_attn(q, k, v, return_lse=True, out=views[0], **w)
    assert o is views[0]
    crs.window_attn_backward(go, q, k, v, o, lse, out=tuple(views[1:]), **w)
    r = ref.attention(q, k, v, ref.visible(B, L, L, 33, 5, 2, 1), scale=0.07, d_out=go)
    for name, x in zip(("o", "dq", "dk", "dv"), views):
        ref.check(name, x, r)


def test_window_attn_empty():
    e = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    assert crs.window_attn(e(1, 2, 0, 64), e(1, 2, 5, 64), e(1, 2, 5, 64)).shape == (1, 2, 0, 64)
    q = normal(gen(1), 1, 2, 5, 64)
    o, lse = crs.window_attn(q, e(1, 2, 0, 64), e(1, 2, 0, 64), return_lse=True)
    assert not o.any() and bool((lse == -math.inf).all())
    dq, dk, dv = crs.window_attn_backward(q, q, e(1, 2, 0, 64), e(1, 2, 0, 64), o, lse)
    assert not dq.any() and dk.numel() == 0
    k = normal(gen(2), 1, 2, 5, 64)
    _, dk, dv = crs.window_attn_backward(e(1, 2, 0, 64), e(1, 2, 0, 64), k, k, e(1, 2, 0, 64),
                                         torch.empty(1, 2, 0, device="cuda"))
    assert dk.shape == k.shape and not dk.any() and not dv.any()


def test_window_attn_large_scores():
    """Scores of thousands: the softmax has one weight of 1 and nothing overflows."""
    g = gen(8)
    q, k, v = normal(g, 1, 1, 200, 64) * 40, normal(g, 1, 1, 200, 64) * 40, normal(g, 1, 1, 200, 64)
    o, lse = crs.window_attn(q, k, v, right=-1, return_lse=True)
    r = ref.attention(q, k, v, ref.visible(1, 200, 200, -1, -1, 0, 1))
    ref.check("o", o, r)
    ref.check("lse", lse, r)


def test_gradient_against_differences():
    """d/dt of sum(g * attention) along random directions, by central differences of the 64-bit form."""
    B, Hq, Hk, Lq, Lk, d = 1, 4, 2, 40, 90, 64
    w = dict(left=20, right=3, sinks=5)
    g = gen(17)
    q, k, v, go = normal(g, B, Hq, Lq, d), normal(g, B, Hk, Lk, d), normal(g, B, Hk, Lk, d), normal(g, B, Hq, Lq, d)
    o, lse = crs.window_attn(q, k, v, return_lse=True, **w)
    grads = crs.window_attn_backward(go, q, k, v, o, lse, **w)
    mask = ref.visible(B, Lq, Lk, 20, 3, 5, 1)
    tol = ref.attention(q, k, v, mask, d_out=go)["tol"]

    def f(args):
        q, k, v = args
        kk, vv = (x.repeat_interleave(Hq // Hk, 1) for x in (k, v))
        s = (q @ kk.transpose(2, 3) / math.sqrt(d)).masked_fill(~mask[:, None], -math.inf)
        return float((go.double() * (torch.softmax(s, 3) @ vv)).sum())

    base = [x.double() for x in (q, k, v)]
    for n, (name, grad) in enumerate(zip(("dq", "dk", "dv"), grads)):
        u = torch.randn(base[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, dn = list(base), list(base)
        up[n], dn[n] = base[n] + h * u, base[n] - h * u
        diff = (f(up) - f(dn)) / (2 * h)
        assert abs(diff - float((grad.double() * u).sum())) <= float((tol[name] * u.abs()).sum()) + 1e-5 * abs(diff) + 1e-5


# ------------------------------------------------------------------ 8-bit cache
def random_cache(g, pages, H, T, d):
    c = crs.Cache8.empty(pages, H, T, d)
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x.copy_((torch.randn(pages, H, T, d, generator=g, device="cuda") * 60).clamp(-448, 448))
        s.copy_(torch.exp2(torch.randint(-8, -4, (pages, H), generator=g, device="cuda").float()))
    return c


def copy_cache(c):
    return crs.Cache8(*(t.clone() for t in c))


@pytest.mark.parametrize("B,H,n,d,T,starts,counts", [
    (1, 1, 1, 64, 16, (0,), None),
    (3, 2, 1, 128, 64, (0, 63, 64), None),
    (2, 3, 37, 64, 16, (5, 31), None),
    (2, 1, 300, 128, 128, (1, 128), None),
    (3, 2, 70, 128, 32, (0, 33, 7), (70, 0, 13)),
    (1, 2, 129, 64, 128, (127,), (100,)),
])
def test_cache8_append(B, H, n, d, T, starts, counts):
    g = gen(n + T)
    per = (max(starts) + n + T - 1) // T
    c = random_cache(g, B * per + 3, H, T, d)
    table = torch.randperm(B * per + 3, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32)
    # token sizes over many powers of two, so that pages grow, and one head of zeros
    size = torch.exp2(torch.randint(-12, 12, (B, 1, n, 1), generator=g, device="cuda").float())
    k = (torch.randn(B, n, H, d, generator=g, device="cuda").transpose(1, 2) * size).to(torch.bfloat16)
    v = normal(g, B, H, n, d)
    v[:, 0] = 0
    start = torch.tensor(starts, device="cuda", dtype=torch.int32)
    cnt = None if counts is None else torch.tensor(counts, device="cuda", dtype=torch.int32)
    old = copy_cache(c)
    crs.cache8_append(k, v, c, table, start, cnt)
    crs.ops_status()
    for x8, sc, o8, osc, x in ((c.k, c.k_scale, old.k, old.k_scale, k), (c.v, c.v_scale, old.v, old.v_scale, v)):
        val, want = ref.append(o8.float().double().cpu(), osc.double().cpu(), x.cpu(), table.cpu(), start.cpu(),
                               None if counts is None else list(counts), T)
        assert torch.equal(sc.double().cpu(), want)
        assert torch.equal(x8.float().double().cpu(), val)  # other pages and slots as they were
    # once more: nothing changes
    twice = copy_cache(c)
    crs.cache8_append(k, v, twice, table, start, cnt)
    for a, b in zip(c, twice):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_cache8_append_special_values():
    c = crs.Cache8.empty(3, 1, 16, 64)
    table = torch.tensor([[1, 2]], device="cuda", dtype=torch.int32)
    k = torch.zeros(1, 1, 5, 64, device="cuda", dtype=torch.bfloat16)
    k[0, 0, 0, 0], k[0, 0, 1, 1], k[0, 0, 2, 2] = math.nan, 3.3895e38, 2.0 ** -130
    v = torch.zeros_like(k)
    v[0, 0, 0, 0], v[0, 0, 1, 0] = math.inf, -math.inf
    zero = torch.zeros(1, device="cuda", dtype=torch.int32)
    crs.cache8_append(k, v, c, table, zero)
    crs.ops_status()
    kk, vv = c.k[1].float() * c.k_scale[1], c.v[1].float() * c.v_scale[1]
    assert math.isnan(float(kk[0, 0, 0])) and float(c.k_scale[1]) == 2.0 ** 119
    assert float(kk[0, 1, 1]) == 448 * 2.0 ** 119 and float(kk[0, 2, 2]) == 0
    assert float(vv[0, 0, 0]) == 448 * 2.0 ** 119 and float(vv[0, 1, 0]) == -448 * 2.0 ** 119
    assert not c.k[0].float().any() and not c.k[2].float().any()


def test_bad_pages_and_lengths_are_reported():
    g = gen(4)
    c = random_cache(g, 4, 2, 16, 64)
    before = copy_cache(c)
    k = normal(g, 1, 2, 20, 64)
    start = torch.zeros(1, device="cuda", dtype=torch.int32)
    for bad in (-1, 4, 2**31 - 1):
        table = torch.tensor([[bad, 2]], device="cuda", dtype=torch.int32)
        crs.cache8_append(k, k, c, table, start)
        with pytest.raises(_lib.ACError) as e:
            crs.ops_status()
        assert e.value.status == _lib.AC_ERR_BOUNDS
        crs.ops_status()  # reported once
        assert torch.equal(c.k[[0, 1, 3]].view(torch.uint8), before.k[[0, 1, 3]].view(torch.uint8))
        # a visible bad page reads as zeros, one that no query sees is never looked at
        q = normal(g, 1, 2, 1, 64)
        lens = torch.tensor([20], device="cuda", dtype=torch.int32)
        o = crs.cache8_attn(q, c, table, lens)
        with pytest.raises(_lib.ACError):
            crs.ops_status()
        kk, vv = (torch.nn.functional.pad((x[2, :, :4].float() * s[2, :, None, None]).unsqueeze(0), (0, 0, 16, 0))
                  for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)))
        ref.check("o", o, ref.attention(q, kk, vv, torch.ones(1, 1, 20, dtype=torch.bool, device="cuda")))
        o = crs.cache8_attn(q, c, table, lens, left=3)
        ref.check("o", o, ref.attention(q, kk[:, :, 16:], vv[:, :, 16:], torch.ones(1, 1, 4, dtype=torch.bool, device="cuda")))
        crs.ops_status()
    # a table that is too short, a negative start, a length beyond the table
    crs.cache8_append(k, k, c, torch.tensor([[2]], device="cuda", dtype=torch.int32), start)
    with pytest.raises(_lib.ACError):
        crs.ops_status()
    crs.cache8_append(k, k, c, torch.tensor([[0, 1]], device="cuda", dtype=torch.int32), start - 1)
    with pytest.raises(_lib.ACError):
        crs.ops_status()
    crs.window_attn(k, k, k, k_lens=start + 21)
    with pytest.raises(_lib.ACError):
        crs.ops_status()


def dense(c, table, Lk):
    """The cached keys and values as [B, H, Lk, d], exact in bf16."""
    T = c.k.shape[2]
    out = []
    for x, s in ((c.k, c.k_scale), (c.v, c.v_scale)):
        val = x.view(torch.uint8)[table.long()].view(torch.float8_e4m3fn).float() * s[table.long()][..., None, None]
        val = val.transpose(1, 2).flatten(2, 3)
        out.append(torch.nn.functional.pad(val, (0, 0, 0, max(0, Lk - val.shape[2])))[:, :, :Lk])
    return out


@pytest.mark.parametrize("T", [16, 32, 64, 128])
@pytest.mark.parametrize("case", [c for c in CASES if c[4] > 1])
def test_cache8_attn(case, T):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    g = gen(T + Lk)
    per = (Lk + T - 1) // T + 1
    c = random_cache(g, B * per + 1, Hk, T, d)
    c.k.view(torch.uint8)[B * per] = 0x7F  # a page of NaN, used by nobody
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    lens = torch.tensor([max(1, Lk - 5 * b) for b in range(B)], device="cuda", dtype=torch.int32)
    for b in range(B):  # codes behind the sequence are NaN, the table behind it is junk
        n = int(lens[b])
        last = int(table[b, (n - 1) // T])
        if n % T:
            c.k.view(torch.uint8)[last, :, n % T:] = 0x7F
            c.v.view(torch.uint8)[last, :, n % T:] = 0xFF
        table[b, (n - 1) // T + 1:] = -7
    q = normal(g, B, Hq, Lq, d)
    o, lse = crs.cache8_attn(q, c, table, lens, return_lse=True, **rule(case))
    crs.ops_status()
    k, v = dense(c, table.clamp(min=0), Lk)
    mask = ref.visible(B, Lq, Lk, *case[6:], None, lens)
    keep = torch.arange(Lk, device="cuda").view(1, 1, Lk, 1) < lens.view(B, 1, 1, 1)
    r = ref.attention(q, torch.where(keep, k, 0.0), torch.where(keep, v, 0.0), mask)
    ref.check("o", o, r)
    ref.check("lse", lse, r)


@pytest.mark.parametrize("T", [16, 64, 128])
@pytest.mark.parametrize("case", [
    (2, 4, 2, 500, 4200, 128, 900, 0, 100, 1),
    (1, 8, 8, 800, 2100, 64, 1, 0, 250, 300),
    (1, 2, 1, 700, 17000, 128, 300, 20, 0, 1),
    (3, 6, 3, 450, 1900, 128, -1, -1, 0, 1),
])
def test_cache8_attn_of_many_rows(case, T):
    """More rows than a few tiles: ragged sequences, NaN codes behind them, junk in the table wherever
    no query sees the page, and one page that is visible and bad, which reads as zeros."""
    B, Hq, Hk, Lq, Lk, d = case[:6]
    g = gen(2 * T + Lk)
    per = (Lk + T - 1) // T
    c = random_cache(g, B * per + 1, Hk, T, d)
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    lens = torch.tensor([max(1, Lk - 77 * b) for b in range(B)], device="cuda", dtype=torch.int32)
    q_lens = torch.tensor([Lq - 40 * b for b in range(B)], device="cuda", dtype=torch.int32)
    for b in range(B):
        n = int(lens[b])
        last = int(table[b, (n - 1) // T])
        if n % T:
            c.k.view(torch.uint8)[last, :, n % T:] = 0x7F
            c.v.view(torch.uint8)[last, :, n % T:] = 0xFF
    k, v = dense(c, table, Lk)
    mask = ref.visible(B, Lq, Lk, *case[6:], q_lens, lens)
    seen = mask.reshape(B, -1, mask.shape[-2], Lk).any(2).any(1)  # [B, Lk]
    pages = torch.nn.functional.pad(seen, (0, per * T - Lk)).view(B, per, T).any(2)
    table = torch.where(pages, table, -9)
    bad = int(pages[0].nonzero()[-2])
    keep = (torch.arange(Lk, device="cuda") < lens.view(B, 1)).view(B, 1, Lk, 1)
    q = normal(g, B, Hq, Lq, d)
    for broken in (False, True):
        if broken:
            table[0, bad] = B * per + 1
            keep = keep.clone()
            keep[0, :, bad * T:(bad + 1) * T] = False
        out = torch.full_like(q, math.nan)
        o, lse = crs.cache8_attn(q, c, table, lens, q_lens=q_lens, return_lse=True, out=out, **rule(case))
        if broken:
            with pytest.raises(Exception, match="out of range"):
                crs.ops_status()
        crs.ops_status()
        r = ref.attention(q, torch.where(keep, k, 0.0), torch.where(keep, v, 0.0), mask)
        ref.check("o", o, r)
        ref.check("lse", lse, r)


@pytest.mark.parametrize("Lq", [1, 40])
def test_cache8_attn_scales_of_very_different_size(Lq):
    """Pages of zeros (the smallest scale), pages 2^40 apart, and queries of any size."""
    B, H, T, d, n = 1, 2, 16, 64, 200
    g = gen(61)
    c = random_cache(g, 13, H, T, d)
    e = torch.randint(-20, 20, (13, H), generator=g, device="cuda").float()
    c.v_scale.copy_(torch.exp2(e))
    c.k_scale.copy_(torch.exp2(torch.randint(-12, -6, (13, H), generator=g, device="cuda").float()))
    c.v[3] = 0
    c.v_scale[3] = 2.0 ** -120
    c.v.view(torch.uint8)[:, 1] = 0  # a whole head of zeros
    c.v_scale[:, 1] = 2.0 ** -120
    table = torch.arange(13, device="cuda", dtype=torch.int32).view(1, 13)
    lens = torch.tensor([n], device="cuda", dtype=torch.int32)
    for size in (2.0 ** -20, 1.0, 2.0 ** 4):
        q = normal(g, B, H, Lq, d) * size
        o, lse = crs.cache8_attn(q, c, table, lens, return_lse=True)
        k, v = dense(c, table, n)
        r = ref.attention(q, k, v, ref.visible(B, Lq, n, -1, 0, 0, 1))
        ref.check("lse", lse, r)
        ref.check("o", o, r)
        assert not o[:, 1].any()


@pytest.mark.parametrize("T", [16, 64])
@pytest.mark.parametrize("Lq", [2, 40])
def test_cache8_attn_of_zeros(T, Lq):
    """Queries of zeros over pages of zeros, with masked keys: the plain mean of the values, no NaN."""
    g = gen(71)
    c = crs.Cache8.empty(20, 1, T, 64)
    table = torch.arange(20, device="cuda", dtype=torch.int32).view(1, 20)
    lens = torch.tensor([T * 5 + 3], device="cuda", dtype=torch.int32)
    v = normal(g, 1, 1, T * 5 + 3, 64)
    crs.cache8_append(torch.zeros_like(v), v, c, table, torch.zeros_like(lens))
    q = torch.zeros(1, 1, Lq, 64, device="cuda", dtype=torch.bfloat16)
    q[:, :, 1::2] = 2.0 ** -126
    w = dict(left=T + 5, sinks=3)
    o, lse = crs.cache8_attn(q, c, table, lens, return_lse=True, **w)
    kk, vv = dense(c, table, T * 5 + 3)
    r = ref.attention(q, kk, vv, ref.visible(1, Lq, T * 5 + 3, T + 5, 0, 3, 1))
    ref.check("o", o, r)
    ref.check("lse", lse, r)


def test_counts_out_of_range_are_reported():
    c = crs.Cache8.empty(4, 1, 16, 64)
    k = normal(gen(72), 1, 1, 5, 64)
    table = torch.arange(4, device="cuda", dtype=torch.int32).view(1, 4)
    zero = torch.zeros(1, device="cuda", dtype=torch.int32)
    for n, held in ((6, 5), (-1, 0)):
        c.k.zero_()
        crs.cache8_append(k, k, c, table, zero, zero + n)
        with pytest.raises(_lib.ACError):
            crs.ops_status()
        assert int((c.k[0, 0].float().abs().sum(1) > 0).sum()) == held


def test_offsets_beyond_32_bits():
    """A cache of more than 2^31 codes, and keys of more than 2^31 elements: the far end is read and written."""
    g = gen(73)
    pages, H, T, d = 17000, 8, 128, 128
    c = crs.Cache8.empty(pages, H, T, d)
    far = torch.tensor([[pages - 1, 3, pages - 2]], device="cuda", dtype=torch.int32)
    k, v = normal(g, 1, H, 300, d), normal(g, 1, H, 300, d)
    zero = torch.zeros(1, device="cuda", dtype=torch.int32)
    crs.cache8_append(k, v, c, far, zero)
    kk, vv = dense(c, far, 300)
    for Lq in (1, 40):
        q = normal(g, 1, H, Lq, d)
        o = crs.cache8_attn(q, c, far, zero + 300)
        ref.check("o", o, ref.attention(q, kk, vv, ref.visible(1, Lq, 300, -1, 0, 0, 1)))
    assert float((kk - k.float()).norm() / k.float().norm()) < 2.0 ** -4
    crs.ops_status()
    del c, kk, vv
    L = 2**31 // (H * d) + 1000
    k = torch.zeros(1, H, L, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    k[:, :, -500:], v[:, :, -500:] = normal(g, 1, H, 500, d), normal(g, 1, H, 500, d)
    for Lq in (1, 300):
        q = normal(g, 1, H, Lq, d)
        o, lse = crs.window_attn(q, k, v, left=150, return_lse=True)
        r = ref.attention(q, k[:, :, -500:], v[:, :, -500:], ref.visible(1, Lq, 500, 150, 0, 0, 1), d_out=q)
        ref.check("o", o, r)
    dq, dk, dv = crs.window_attn_backward(q, q, k, v, o, lse, left=150)
    for name, x in (("dq", dq), ("dk", dk[:, :, -500:]), ("dv", dv[:, :, -500:])):
        ref.check(name, x, r)
    assert not dk[:, :, :-500].any() and not dv[:, :, :-500].any()


# ------------------------------------------------------------------ together
def test_streaming_generation_and_training_step():
    """Frame after frame: rotate, attend within the window over the cache, append; the rotation and the window
    attention of the whole clip give the same outputs within what 8 bits cost, and its gradients pass through."""
    B, H, d, hw, frames, T = 1, 4, 64, 60, 5, 32
    L = hw * frames
    g = gen(21)
    q0, k0, v0 = (normal(g, B, L, H, d).transpose(1, 2) for _ in range(3))
    t = torch.arange(L, device="cuda")
    pos = torch.stack([t // hw, t % hw // 10, t % 10], 1).to(torch.int32).contiguous()
    pairs = (12, 10, 10)
    w = dict(left=1, right=0, sinks=hw, block=hw)
    q, k = crs.rope_axes(q0, k0, pos, pairs)
    whole, lse = crs.window_attn(q, k, v0, return_lse=True, **w)
    cache = crs.Cache8.empty(12, H, T, d)
    table = torch.arange(11, -1, -1, device="cuda", dtype=torch.int32).view(1, 12)
    for f in range(frames):
        part = slice(f * hw, (f + 1) * hw)
        qf, kf = crs.rope_axes(q0[:, :, part], k0[:, :, part], pos[part], pairs)
        n = torch.tensor([f * hw], device="cuda", dtype=torch.int32)
        crs.cache8_append(kf, v0[:, :, part], cache, table, n)
        o = crs.cache8_attn(qf, cache, table, n + hw, **w)
        kk, vv = dense(cache, table, (f + 1) * hw)
        r = ref.attention(qf, kk, vv, ref.visible(B, hw, (f + 1) * hw, 1, 0, hw, hw))
        ref.check("o", o, r)
        # keys and values in 8 bits: off by half a step of e4m3, 2^-4 relative, each
        assert float((o.double() - whole[:, :, part].double()).norm() / whole[:, :, part].double().norm()) < 2 * 2.0 ** -4
    crs.ops_status()
    go = normal(g, B, H, L, d)
    dq, dk, dv = crs.window_attn_backward(go, q, k, v0, whole, lse, **w)
    gq, gk = crs.rope_axes(dq, dk, pos, pairs, inverse=True)
    want = ref.attention(q, k, v0, ref.visible(B, L, L, 1, 0, hw, hw), d_out=go)
    for name, got in (("dq", gq), ("dk", gk)):
        back = ref.rotate(want[name], pos.unsqueeze(0), pairs, ref.freqs(pairs), True, inverse=True)
        # the rotation mixes two entries, each off by its tolerance, and rounds once
        tol = want["tol"][name]
        pair = tol.unflatten(-1, (-1, 2)).sum(-1, keepdim=True).expand(*tol.shape[:-1], d // 2, 2).flatten(-2)
        assert bool(((got.double() - back).abs() <= pair + ref.U * back.abs() + 2.0 ** -20).all())


def test_sparse_layer_takes_positions():
    """SparseLayer.forward(rope=...) is rope_axes and then the layer."""
    from cluster_routed_sparse_b200.api import SparseLayer
    B, H, L, d = 1, 2, 700, 64
    g = gen(30)
    q, k, v = (normal(g, B, H, L, d) for _ in range(3))
    t = torch.arange(L, device="cuda")
    pos = torch.stack([t // 100, t % 100 // 10, t % 10], 1).to(torch.int32).contiguous()
    kw = dict(Cq=8, m0=8, n_max=32, tau_mode=1, tau_value=1.0, topk=4, iters_q=3, iters_k=3)
    a, b = SparseLayer(B, H, L, d, **kw), SparseLayer(B, H, L, d, **kw)
    qr, kr = crs.rope_axes(q, k, pos, (12, 10, 10), theta=256.0)
    want = a.forward(qr, kr, v)
    got = b.forward(q, k, v, rope=(pos, (12, 10, 10), 256.0))
    strided = b.forward(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, rope=(pos, (12, 10, 10), 256.0))
    a.synchronize(), b.synchronize()
    assert torch.equal(got, want) and torch.equal(strided, want)
    a.close(), b.close()


# ------------------------------------------------------------------ streams, graphs, overlap
def all_ops(seed):
    """A run of every operator; returns the outputs."""
    case = (2, 6, 2, 190, 333, 64, 40, 7, 3, 1)
    q, k, v, go = tensors(case, seed)
    g = gen(seed)
    c = random_cache(g, 14, 2, 64, 64)
    table = torch.arange(14, device="cuda", dtype=torch.int32).view(2, 7)
    start = torch.tensor([70, 3], device="cuda", dtype=torch.int32)
    pos = torch.arange(190, device="cuda", dtype=torch.int32).view(190, 1)

    def run():
        qr = crs.rope_axes(q, None, pos, (32,))
        o, lse = crs.window_attn(qr, k, v, return_lse=True, **rule(case))
        grads = crs.window_attn_backward(go, qr, k, v, o, lse, **rule(case))
        crs.cache8_append(k[:, :, :100], v[:, :, :100], c, table, start)
        few = crs.cache8_attn(qr[:, :, :1], c, table, start + 100)
        many = crs.cache8_attn(qr, c, table, start + 100, left=64)
        step = crs.window_attn(qr[:, :, :2], k, v)
        return [qr, o, lse, *grads, few, many, step, c.k.view(torch.uint8).clone(), c.k_scale.clone()]
    return run


def test_another_stream_and_two_at_once():
    runs = [all_ops(s) for s in (1, 2)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    got = [None, None]
    for _ in range(3):
        for i, (s, r) in enumerate(zip(streams, runs)):
            with torch.cuda.stream(s):
                got[i] = r()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_captured_and_replayed():
    runs = [all_ops(s) for s in (3, 4)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(r())
        graphs.append(graph)
    for o in outs:
        for t in o:
            t.zero_()
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(2):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    crs.ops_status()


def test_query_gradient_over_many_keys_with_a_common_part():
    """Thousands of keys and values with a large common part: what rounding o costs sum(dO o) must not
    reach dq along the mean key.  Left are roundings of single entries (bf16, half a step 2^-8): the norm of
    their error is below half a step of the whole."""
    B, H, L, d = 1, 2, 6000, 128
    g = gen(41)
    q, go = normal(g, B, H, 300, d), normal(g, B, H, 300, d)
    k, v = normal(g, B, H, L, d) + 2, normal(g, B, H, L, d) + 2
    o, lse = crs.window_attn(q, k, v, right=-1, return_lse=True)
    dq, dk, dv = crs.window_attn_backward(go, q, k, v, o, lse, right=-1)
    r = ref.attention(q, k, v, ref.visible(B, 300, L, -1, -1, 0, 1), d_out=go)
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert float((x.double() - r[name]).norm() / r[name].norm()) < 2.0 ** -8, name

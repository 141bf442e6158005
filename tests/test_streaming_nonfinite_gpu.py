"""What is not finite inside a sequence stays visible: a row whose scores hold a NaN or overflow is NaN, in
every kernel that the sizes select, with the keys in one part and in several."""
import math

import pytest
import torch

import _stream_ref as ref
import cluster_routed_sparse_b200 as crs
from test_streaming_gpu import dense, gen, normal, random_cache

pytestmark = pytest.mark.gpu

WINDOW = [
    # B, Hq, Hk, Lq, Lk, d, left, right, sinks, block
    (1, 2, 2, 1, 100, 64, -1, 0, 0, 1),          # few rows, one part
    (2, 4, 2, 3, 100, 128, 40, 0, 8, 1),
    (1, 1, 1, 1, 20000, 128, -1, 0, 0, 1),       # few rows, several parts
    (1, 40, 40, 300, 300, 64, 50, 0, 3, 1),      # tiles, one part
    (1, 2, 2, 300, 8192, 128, -1, 0, 0, 1),      # tiles, several parts
    (1, 2, 2, 40, 4000, 64, -1, 0, 0, 1),        # one row tile alone, several parts
    (1, 160, 160, 40, 700, 64, -1, -1, 0, 1),    # one row tile alone, one part
]
CACHE = WINDOW + [
    (1, 160, 160, 70, 400, 64, -1, 0, 0, 1),     # tiles over the codes, one part
    (1, 2, 1, 900, 17000, 128, 3000, 0, 40, 1),  # many rows: the cache as bf16 rows
]


def inputs(case, seed):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    g = gen(seed)
    return normal(g, B, Hq, Lq, d), normal(g, B, Hk, Lk, d), normal(g, B, Hk, Lk, d)


def rule(case):
    return dict(left=case[6], right=case[7], sinks=case[8], block=case[9])


def check_rows(o, lse, want, bad, lse_too=True):
    """Rows [B, Hq, Lq] of `bad` are NaN as a whole, all others as in `want`."""
    assert bool(bad.any())
    assert bool(torch.isnan(o[bad]).all()), "an output that hides a NaN"
    if lse_too:
        assert bool(torch.isnan(lse[bad]).all()), "a log-sum-exp that hides a NaN"
        lse = torch.where(bad, want["lse"], lse.double())
    ref.check("o", torch.where(bad.unsqueeze(3), want["o"], o.double()), want)
    ref.check("lse", lse, want)


@pytest.mark.parametrize("case", WINDOW)
@pytest.mark.parametrize("what", [math.nan, "overflow"])
def test_query_rows(case, what):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    q, k, v = inputs(case, 1)
    k[:, :, :, 0] = k[:, :, :, 0].abs() + 1
    clean = q.clone()
    bad = torch.zeros(B, Hq, Lq, dtype=torch.bool, device="cuda")
    for b, h, i in ((0, 0, 0), (B - 1, Hq - 1, Lq - 1), (0, Hq // 2, Lq // 2)):
        bad[b, h, i] = True
        clean[b, h, i] = 0
        q[b, h, i, 0] = 3e38 if what == "overflow" else what  # 3e38 times 128 keys' sizes: past fp32
    if what == "overflow":
        k[:, :, :, 0] *= 8
    want = ref.attention(clean, k, v, ref.visible(B, Lq, Lk, *case[6:]))
    o, lse = crs.window_attn(q, k, v, return_lse=True, **rule(case))
    crs.ops_status()
    check_rows(o, lse, want, bad)


@pytest.mark.parametrize("case", CACHE)
@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_cache(case, what):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    T, g = 32, gen(5)
    per = (Lk + T - 1) // T
    c = random_cache(g, B * per, Hk, T, d)
    table = torch.randperm(B * per, generator=g, device="cuda").view(B, per).to(torch.int32)
    lens = torch.full((B,), Lk, device="cuda", dtype=torch.int32)
    q = normal(g, B, Hq, Lq, d)
    k, v = dense(c, table, Lk)
    mask = ref.visible(B, Lq, Lk, *case[6:])
    if what == "query":
        bad = torch.zeros(B, Hq, Lq, dtype=torch.bool, device="cuda")
        bad[0, Hq - 1, Lq // 2] = True
        clean = q.clone()
        clean[0, Hq - 1, Lq // 2] = 0
        q[0, Hq - 1, Lq // 2, d - 1] = math.nan
    else:
        clean = q
        # a key that some rows see; a value goes to rows that do not see it too where the product covers it, so
        # there all rows of the head see it
        at = Lk - 1 - Lq // 2 if what == "key" else Lk - Lq
        if what == "value":
            mask = ref.visible(B, Lq, Lk, -1, -1, 0, 1)
        x = c.k if what == "key" else c.v
        x.view(torch.uint8)[int(table[0, at // T]), Hk - 1, at % T, 7] = 0x7F
        k[0, Hk - 1, at], v[0, Hk - 1, at] = 0, 0
        bad = torch.zeros(B, Hq, Lq, dtype=torch.bool, device="cuda")
        bad[0, (Hk - 1) * (Hq // Hk):] = mask[0, :, at]
    w = rule(case) if what != "value" else dict(left=-1, right=-1)
    want = ref.attention(clean, k, v, mask)
    o, lse = crs.cache8_attn(q, c, table, lens, return_lse=True, **w)
    crs.ops_status()
    if what == "value":  # one element of the output
        assert bool(torch.isnan(o[bad][:, 7]).all())
    else:
        check_rows(o, lse, want, bad)


@pytest.mark.parametrize("case", [(1, 4, 2, 300, 500, 64, 60, 0, 5, 1), (2, 2, 2, 130, 130, 128, -1, 0, 0, 1)])
def test_gradients(case):
    B, Hq, Hk, Lq, Lk, d = case[:6]
    q, k, v = inputs(case, 3)
    g = normal(gen(4), B, Hq, Lq, d)
    clean, i, h = q.clone(), Lq // 2, Hq - 1
    clean[0, h, i] = 0
    q[0, h, i, 3] = math.nan
    o, lse = crs.window_attn(q, k, v, return_lse=True, **rule(case))
    dq, dk, dv = crs.window_attn_backward(g, q, k, v, o, lse, **rule(case))
    crs.ops_status()
    mask = ref.visible(B, Lq, Lk, *case[6:])
    want = ref.attention(clean, k, v, mask, d_out=g)
    assert bool(torch.isnan(dq[0, h, i]).all())
    dq[0, h, i] = want["dq"][0, h, i].to(dq.dtype)
    ref.check("dq", dq, want)
    seen = mask[0, i]
    assert bool(torch.isnan(dk[0, Hk - 1, seen]).all()) and bool(torch.isnan(dv[0, Hk - 1, seen]).all())
    for name, x in (("dk", dk), ("dv", dv)):  # other heads and sequences know nothing of it
        x, keep = x.double(), torch.ones(B, Hk, dtype=torch.bool, device="cuda")
        keep[0, Hk - 1] = False
        ref.check(name, torch.where(keep[:, :, None, None], x, want[name]), want)

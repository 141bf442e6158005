"""Small weights of the attention over the 8-bit cache keep their bits: whatever scale the values of other
pages have, and however many keys share the small weights, each channel is right element by element."""
import pytest
import torch

import _stream_ref as ref
import cluster_routed_sparse_b200 as crs
from test_streaming_gpu import dense, gen, random_cache

pytestmark = pytest.mark.gpu

ROUTES = [
    # Lq, keys, heads
    (1, 4096, 1),       # few rows
    (1, 200, 4),        # few rows, one part
    (40, 4096, 2),      # tiles over the codes
    (70, 300, 160),     # the same, one part
    (800, 16384, 1),    # the cache as bf16 rows
]


def one_ahead(Lq, n, H, T, d, bits, seed):
    """A cache in which the keys score 0 but for one, in the middle, that is `bits` powers of two ahead of them
    for a query of ones; values everywhere but in channel 0."""
    g = gen(seed)
    c = random_cache(g, -(-n // T), H, T, d)
    c.k.view(torch.uint8).zero_()
    c.k_scale.fill_(1.0)
    c.v_scale.fill_(1.0)
    at = n // 2
    x = c.v.float()
    x[..., 0] = 0
    x[at // T, :, at % T] = 0
    c.v.copy_(x)
    c.k.view(torch.float8_e4m3fn)[at // T, :, at % T, 0] = 1.0
    table = torch.arange(c.k.shape[0], device="cuda", dtype=torch.int32).view(1, -1)
    q = torch.zeros(1, H, Lq, d, device="cuda", dtype=torch.bfloat16)
    q[..., 0] = float(bits)
    scale = 0.6931471805599453  # scores count powers of two
    return c, table, q, scale, at


@pytest.mark.parametrize("Lq,n,H", ROUTES)
@pytest.mark.parametrize("ratio", [0, 10, 22, 60])
def test_a_page_of_large_values(Lq, n, H, ratio):
    """One page's values are 2^ratio times the others', in one channel only: the rest of the softmax still
    reaches the other channels."""
    T, d = 16, 64
    c, table, q, scale, at = one_ahead(Lq, n, H, T, d, 12, ratio)
    page = at // T
    x = c.v[page].float()
    x[..., 1:] = 0
    x[:, at % T, 0] = 448
    c.v[page] = x.to(torch.float8_e4m3fn)
    c.v_scale[page] = 2.0 ** ratio
    o, lse = crs.cache8_attn(q, c, table, torch.tensor([n], device="cuda", dtype=torch.int32), right=-1, scale=scale,
                             return_lse=True)
    crs.ops_status()
    k, v = dense(c, table, n)
    r = ref.attention(q, k, v, ref.visible(1, Lq, n, -1, -1, 0, 1), scale=scale)
    ref.check("o", o, r)
    ref.check("lse", lse, r)


@pytest.mark.parametrize("Lq,n,H", [(1, 65536, 1), (40, 65536, 1), (3, 2000, 1), (200, 2000, 2)])
@pytest.mark.parametrize("bits", [16, 26, 60])
def test_many_small_weights(Lq, n, H, bits):
    """Keys 2^-bits below the first in weight, which has no values in their channels."""
    T, d = 64, 128
    c, table, q, scale, at = one_ahead(Lq, n, H, T, d, bits, bits)
    o, lse = crs.cache8_attn(q, c, table, torch.tensor([n], device="cuda", dtype=torch.int32), right=-1, scale=scale,
                             return_lse=True)
    crs.ops_status()
    k, v = dense(c, table, n)
    r = ref.attention(q, k, v, ref.visible(1, Lq, n, -1, -1, 0, 1), scale=scale)
    ref.check("o", o, r)
    ref.check("lse", lse, r)


@pytest.mark.parametrize("Lq,n,H", [(1, 200, 4), (40, 400, 2), (800, 16384, 1)])
def test_pages_of_small_values(Lq, n, H):
    """Scales down to the smallest: values are those that bf16 holds, not zeros."""
    T, d = 16, 64
    g = gen(7)
    c = random_cache(g, -(-n // T), H, T, d)
    c.v_scale.copy_(torch.exp2(torch.randint(-118, -92, c.v_scale.shape, generator=g, device="cuda").float()))
    table = torch.arange(c.k.shape[0], device="cuda", dtype=torch.int32).view(1, -1)
    q = torch.randn(1, H, Lq, d, generator=g, device="cuda").to(torch.bfloat16)
    o = crs.cache8_attn(q, c, table, torch.tensor([n], device="cuda", dtype=torch.int32), right=-1)
    crs.ops_status()
    k, v = dense(c, table, n)
    r = ref.attention(q, k, v, ref.visible(1, Lq, n, -1, -1, 0, 1))
    # instead of the reference's 1e-30, which is more than these values: a weight times a scale is held in bf16,
    # whose smallest step is 2^-133; half of it, times a code of 448 at most, for each key
    r["tol"]["o"] = r["tol"]["o"] - 1e-30 + n * 2.0 ** -125
    ref.check("o", o, r)


@pytest.mark.parametrize("Lq,n,H", ROUTES)
def test_scales_that_are_no_powers_of_two(Lq, n, H):
    """A cache filled elsewhere may have any scales: the code times the scale then rounds to nearest, once, in bf16."""
    T, d = 16, 64
    g = gen(13)
    c = random_cache(g, -(-n // T), H, T, d)
    for s in (c.k_scale, c.v_scale):
        s.copy_((torch.rand(s.shape, generator=g, device="cuda") + 1.0) * 2.0 ** -7)
    c.v.copy_(c.v.float().abs())  # no sign to hide a bias in
    table = torch.arange(c.k.shape[0], device="cuda", dtype=torch.int32).view(1, -1)
    q = torch.randn(1, H, Lq, d, generator=g, device="cuda").to(torch.bfloat16)
    o = crs.cache8_attn(q, c, table, torch.tensor([n], device="cuda", dtype=torch.int32), right=-1)
    crs.ops_status()
    # (the plain form on the products in fp32: dense() and its reader keep them)
    k, v = dense(c, table, n)
    s = (q.double() @ k.double().transpose(2, 3)) / 8.0
    p = torch.softmax(s, 3)
    want = p @ v.double()
    # a key off by half a step of bf16 in each element moves its score by 2^-9 |q| |k| at most, and the weight as much
    # again; random over 64 elements, an eighth of it: the norms tell a bias (2^-9 and more, of one sign) from that
    off = (o.double() - want)
    assert abs(float(off.sum() / want.sum())) < 2.0 ** -10
    assert float(off.norm() / want.norm()) < 2.0 ** -6


@pytest.mark.parametrize("Lq,n,H", ROUTES)
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 100])
def test_queries_with_one_large_channel(Lq, n, H, size):
    """A channel of the queries `size` times the others, of which the keys hold nothing: the scores are the others'."""
    T, d = 16, 64
    g = gen(19)
    c = random_cache(g, -(-n // T), H, T, d)
    x = c.k.float()
    x[..., 0] = 0
    c.k.copy_(x)
    table = torch.arange(c.k.shape[0], device="cuda", dtype=torch.int32).view(1, -1)
    q = torch.randn(1, H, Lq, d, generator=g, device="cuda").to(torch.bfloat16)
    q[..., 0] = size
    if Lq > 1:
        q[:, :, 1::3, 0] = 0  # (and rows without it)
    o, lse = crs.cache8_attn(q, c, table, torch.tensor([n], device="cuda", dtype=torch.int32), right=-1, return_lse=True)
    crs.ops_status()
    k, v = dense(c, table, n)
    r = ref.attention(q, k, v, ref.visible(1, Lq, n, -1, -1, 0, 1))
    ref.check("o", o, r)
    ref.check("lse", lse, r)

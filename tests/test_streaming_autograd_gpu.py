"""Gradients reach what requires them: rope_axes and window_attn record themselves where torch records, give the
gradients of their own backward calls, and refuse what would be lost."""
import pytest
import torch
import torch.autograd.forward_ad as fwd

import cluster_routed_sparse_b200 as crs
from cluster_routed_sparse_b200 import streaming
from test_streaming_gpu import gen, normal

pytestmark = pytest.mark.gpu

W = dict(left=60, right=3, sinks=5)


@pytest.fixture(params=["compiled", "ctypes"])
def way(request, monkeypatch):
    if request.param == "ctypes":
        monkeypatch.setattr(streaming, "_fast", None)


def leaves(*shapes, seed=1, dtype=torch.bfloat16):
    g = gen(seed)
    return [normal(g, *s, dtype=dtype).requires_grad_() for s in shapes]


def test_window_attn(way):
    q, k, v = leaves((2, 6, 70, 64), (2, 2, 90, 64), (2, 2, 90, 64))
    lens = torch.tensor([70, 31], device="cuda", dtype=torch.int32)
    o, lse = crs.window_attn(q, k, v, q_lens=lens, k_lens=lens + 20, return_lse=True, **W)
    assert o.requires_grad
    g = normal(gen(2), *o.shape)
    o.backward(g)
    with torch.no_grad():
        o2, lse2 = crs.window_attn(q, k, v, q_lens=lens, k_lens=lens + 20, return_lse=True, **W)
        want = crs.window_attn_backward(g, q, k, v, o2, lse2, q_lens=lens, k_lens=lens + 20, **W)
    assert not o2.requires_grad and torch.equal(o, o2) and torch.equal(lse, lse2)
    for t, w in zip((q, k, v), want):
        assert torch.equal(t.grad, w)
    alone = crs.window_attn(q, k.detach(), v.detach(), q_lens=lens, k_lens=lens + 20, **W)
    dq, = torch.autograd.grad(alone, q, g)
    assert torch.equal(dq, want[0])


def test_a_gradient_of_any_strides(way):
    """sum() hands back one broadcast value, a transpose what the next layer's strides are."""
    q, k, v = leaves((1, 2, 40, 64), (1, 2, 40, 64), (1, 2, 40, 64))
    crs.window_attn(q, k, v).float().sum().backward()
    want = [t.grad.clone() for t in (q, k, v)]
    with torch.no_grad():
        o, lse = crs.window_attn(q, k, v, return_lse=True)
        for a, b in zip(want, crs.window_attn_backward(torch.ones_like(o), q, k, v, o, lse)):
            assert torch.equal(a, b)
    o = crs.window_attn(q, k, v)
    dq, = torch.autograd.grad(o.sum(), q)  # stride 0 in every dimension
    assert torch.equal(dq, want[0])
    dq, = torch.autograd.grad(o2 := crs.window_attn(q, k, v), q, torch.ones(1, 2, 64, 40, device="cuda", dtype=o2.dtype).transpose(2, 3))
    assert torch.equal(dq, want[0])


@pytest.mark.parametrize("inverse", [False, True])
def test_rope_axes(way, inverse):
    q, k = leaves((2, 3, 20, 64), (2, 1, 20, 64), dtype=torch.float32)
    pos = torch.randint(0, 500, (2, 20, 2), generator=gen(3), device="cuda", dtype=torch.int32)
    a, b = crs.rope_axes(q, k, pos, (10, 20), interleaved=False, inverse=inverse)
    ga, gb = normal(gen(4), *a.shape, dtype=torch.float32), normal(gen(5), *b.shape, dtype=torch.float32)
    (a * ga).sum().backward(retain_graph=True)
    with torch.no_grad():
        wa, wb = crs.rope_axes(ga, gb, pos, (10, 20), interleaved=False, inverse=not inverse)
    assert torch.equal(q.grad, wa) and k.grad is None or not k.grad.any()
    dk, = torch.autograd.grad(b, k, gb)
    assert torch.equal(dk, wb)
    one = crs.rope_axes(q, None, pos, (10, 20), interleaved=False, inverse=inverse)
    dq, = torch.autograd.grad(one, q, ga)
    assert torch.equal(dq, wa)
    # a second derivative of a linear map: the gradient's gradient is the rotation again
    z = ga.clone().requires_grad_()
    dq, = torch.autograd.grad(crs.rope_axes(q, None, pos, (10, 20), interleaved=False, inverse=inverse), q, z, create_graph=True)
    dz, = torch.autograd.grad(dq, z, wa)
    with torch.no_grad():
        assert torch.equal(dz, crs.rope_axes(wa, None, pos, (10, 20), interleaved=False, inverse=inverse))


def test_a_module_around_them(way):
    """The gradients of projections in front of the rotation and the attention, against a plain form."""
    torch.manual_seed(0)
    B, L, H, d = 1, 48, 2, 64
    x = normal(gen(6), B, L, 32)
    lin = torch.nn.Linear(32, 3 * H * d, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(L, device="cuda", dtype=torch.int32).view(L, 1)

    def run(rope, attn):
        q, k, v = lin(x).unflatten(-1, (3, H, d)).permute(2, 0, 3, 1, 4)
        return attn(*rope(q, k), v)

    def plain_rope(*xs):
        i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
        ang = pos.double() * 10000.0 ** (-i / (d // 2))
        z = torch.polar(torch.ones_like(ang), ang)
        return [torch.view_as_real(torch.view_as_complex(t.double().unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
                for t in xs]

    def plain_attn(q, k, v):
        s = (q @ k.transpose(2, 3) / d ** 0.5).masked_fill(torch.ones(L, L, device="cuda").triu(1).bool(), -torch.inf)
        return torch.softmax(s, 3) @ v.double()

    g = normal(gen(7), B, H, L, d)
    got = torch.autograd.grad(run(lambda q, k: crs.rope_axes(q, k, pos, (d // 2,)), crs.window_attn), list(lin.parameters()), g)
    want = torch.autograd.grad(run(plain_rope, plain_attn), list(lin.parameters()), g.double())
    for a, b in zip(got, want):  # every step rounds to bf16, five of them: 2^-8 each
        assert float((a.double() - b.double()).norm() / b.double().norm()) < 5 * 2.0 ** -8


def test_what_would_be_lost_is_refused(way):
    q, k, v = leaves((1, 2, 40, 64), (1, 2, 40, 64), (1, 2, 40, 64))
    o, lse = crs.window_attn(q, k, v, return_lse=True)
    with pytest.raises(RuntimeError, match="lse"):  # no gradient through the log-sum-exp
        (o.float().sum() + lse.sum()).backward()
    o = crs.window_attn(q, k, v)
    dq, = torch.autograd.grad(o, q, torch.ones_like(o), create_graph=True)
    with pytest.raises(RuntimeError):  # no second derivative
        dq.float().sum().backward()
    with fwd.dual_level():
        d = fwd.make_dual(q.detach(), torch.ones_like(q))
        with pytest.raises(RuntimeError):
            crs.window_attn(d, k.detach(), v.detach())
        with pytest.raises(RuntimeError):
            crs.rope_axes(d, None, torch.zeros(40, 1, device="cuda", dtype=torch.int32), (32,))


def test_what_is_not_recorded_says_so(way):
    """Outputs written into given tensors, and the cache, carry no gradients: a warning, and the values as before."""
    q, k, v = leaves((1, 2, 16, 64), (1, 2, 16, 64), (1, 2, 16, 64))
    pos = torch.arange(16, device="cuda", dtype=torch.int32).view(16, 1)
    cache = crs.Cache8.empty(1, 2, 16, 64)
    ints = torch.zeros(1, 1, device="cuda", dtype=torch.int32)
    calls = [lambda: crs.window_attn(q, k, v, out=torch.empty_like(q)),
             lambda: crs.rope_axes(q, None, pos, (32,), out=(torch.empty_like(q), None)),
             lambda: crs.cache8_append(k, v, cache, ints, ints[0]),
             lambda: crs.cache8_attn(q, cache, ints, ints[0] + 16)]
    for call in calls:
        with pytest.warns(UserWarning, match="not recorded"):
            r = call()
        assert r is None or not r.requires_grad
    with torch.no_grad():
        import warnings
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            for call in calls:
                call()
    crs.ops_status()


def test_captured_backward_while_an_eager_graph_lives(way):
    """The gradients of the same leaves, captured into a CUDA graph while an eager graph of theirs is alive."""
    q, k, v = leaves((1, 2, 40, 64), (1, 2, 40, 64), (1, 2, 40, 64))
    pos = torch.arange(40, device="cuda", dtype=torch.int32).view(40, 1)
    g = normal(gen(8), 1, 2, 40, 64)

    def step():
        o = crs.window_attn(*crs.rope_axes(q, k, pos, (32,)), v, **W)
        return torch.autograd.grad(o, (q, k, v), g)

    want = step()
    # (on the stream of the capture: torch lets the gradients of a leaf meet on the stream that its first graph ran on)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        held = crs.window_attn(*crs.rope_axes(q, k, pos, (32,)), v, **W)
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    for a, b in zip(torch.autograd.grad(held, (q, k, v), g), want):
        assert torch.equal(a, b)
    crs.ops_status()

"""Plain 64-bit forms of the streaming operators, and how far a kernel that rounds
its products' operands to bf16 may be from them.

U is half a step of bf16, 2^-8 relative.  A tiled kernel rounds the softmax
weights p and (backward) ds to bf16 before the second product, and every output
once; its scores come from fp32 sums of d products, off by at most
d 2^-23 sum|q k|, and so are the exponents, which a relative error of p follows.
"""
import math

import torch

U = 2.0 ** -8


def visible(B, Lq, Lk, left, right, sinks, block, q_lens=None, k_lens=None, device="cuda"):
    """[B, Lq, Lk]: query i of sequence b sees key j."""
    i = torch.arange(Lq, device=device).view(1, Lq, 1)
    j = torch.arange(Lk, device=device).view(1, 1, Lk)
    ql = torch.full((B,), Lq, device=device) if q_lens is None else q_lens.long()
    kl = torch.full((B,), Lk, device=device) if k_lens is None else k_lens.long()
    ql, kl = ql.view(B, 1, 1), kl.view(B, 1, 1)
    bp = torch.div(i + kl - ql, block, rounding_mode="floor")
    bj = torch.div(j, block, rounding_mode="floor")
    m = (j < kl) & (i < ql)
    if right >= 0:
        m = m & (bj <= bp + right)
    if left >= 0:
        m = m & ((bj >= bp - left) | (j < sinks))
    return m.expand(B, Lq, Lk)


def attention(q, k, v, mask, scale=None, d_out=None):
    """64-bit attention, its gradients where d_out is given, and the bounds of both.
    Returns a dict of tensors and, under "tol", their tolerances."""
    B, Hq, Lq, d = q.shape
    G = Hq // k.shape[1]
    qd = q.double()
    kd, vd = (x.double().nan_to_num(0, 0, 0).repeat_interleave(G, 1) for x in (k, v))
    scale = 1 / math.sqrt(d) if not scale else scale
    m = mask.unsqueeze(1)
    any_key = m.any(2, keepdim=True).transpose(2, 3)  # keys that some row sees
    kd, vd = kd * any_key, vd * any_key
    live_row = m.any(3, keepdim=True)
    qd = torch.where(live_row, qd, torch.zeros_like(qd))
    s = (qd @ kd.transpose(2, 3) * scale).masked_fill(~m, -math.inf)
    mag = (qd.abs() @ kd.abs().transpose(2, 3) * abs(scale)).masked_fill(~m, 0).amax(3, keepdim=True)
    lse = torch.logsumexp(s, 3, keepdim=True)
    p = torch.exp(s - lse.clamp(min=-1e300))
    o = p @ vd
    delta = d * 2.0 ** -23 * mag + 2.0 ** -18  # of an exponent, and of one exponential
    out = {"o": o, "lse": lse.squeeze(3)}
    tol = {"o": U * o.abs() + (U + 2 * delta) * (p @ vd.abs()) * (1 + U) + 1e-30,
           "lse": (delta + q.shape[2] * 0 + mask.shape[2] * 2.0 ** -24 + 2.0 ** -22 * lse.abs().clamp(max=1e30)).squeeze(3)}
    if d_out is not None:
        g = torch.where(live_row, d_out.double(), torch.zeros_like(qd))
        big_d = (g * o).sum(3, keepdim=True)
        dp = g @ vd.transpose(2, 3)
        ds = p * (dp - big_d)
        dsum = (g.abs() @ vd.abs().transpose(2, 3) + (g * o).abs().sum(3, keepdim=True)) * p
        # o enters the gradient as the forward rounded it: U |g o| in all, and its own error
        err = ds.abs() * (U + 2 * delta) + dsum * d * 2.0 ** -23 + p * (g.abs() * tol["o"]).sum(3, keepdim=True)

        def heads(x):  # sum over the query heads of a key head
            return x.view(B, Hq // G, G, *x.shape[2:]).sum(2)

        out["dq"] = scale * (ds @ kd)
        tol["dq"] = U * out["dq"].abs() + abs(scale) * (err @ kd.abs()) * (1 + U) + 1e-30
        out["dk"] = heads(scale * (ds.transpose(2, 3) @ qd))
        tol["dk"] = U * out["dk"].abs() + heads(abs(scale) * (err.transpose(2, 3) @ qd.abs())) * (1 + U) + 1e-30
        out["dv"] = heads(p.transpose(2, 3) @ g)
        tol["dv"] = U * out["dv"].abs() + heads((p * (U + 2 * delta)).transpose(2, 3) @ g.abs()) * (1 + U) + 1e-30
    out["tol"] = tol
    return out


def check(name, got, ref):
    want, tol = ref[name], ref["tol"][name]
    got = got.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf]), f"{name}: infinities differ"
    assert not torch.isnan(got).any(), f"{name}: NaN"
    bad = ((got - want).abs() > tol) & ~inf
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((got - want).abs() / tol)[~inf].max()):.2f} of the tolerance")


def freqs(pairs, theta=10000.0):
    return [theta ** (-i / n) for n in pairs for i in range(n)]


def rotate(x, pos, pairs, fr, interleaved, inverse=False):
    """64-bit rotary embedding of x [B, H, L, d] with pos [B, L, axes]."""
    P = sum(pairs)
    ax = torch.tensor([a for a, n in enumerate(pairs) for _ in range(n)], dtype=torch.long)
    # whole turns leave the angle before its sine: the positions are integers
    f = torch.tensor(fr, dtype=torch.float64)
    ang = (pos.double().cpu()[..., ax] * f).to(x.device).unsqueeze(1)
    c, s = ang.cos(), ang.sin() * (-1 if inverse else 1)
    y = x.double().clone()
    i = torch.arange(P, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, P + i)
    u, w = y[..., a].clone(), y[..., b].clone()
    y[..., a] = u * c - w * s
    y[..., b] = u * s + w * c
    return y


def exponent(amax):
    """Least e with amax <= 448 * 2^e, from -120 to 119."""
    e = -120
    while e < 119 and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(k8, scale, x, table, start, counts, T):
    """One of K, V: codes (as values) and scale exponents after the append, token by token.
    k8: float values of the codes [pages, H, T, d] (fp64, CPU), scale [pages, H]."""
    B, H, n, d = x.shape
    val, sc = k8.clone(), scale.clone()
    e4m3 = lambda t: t.float().to(torch.float8_e4m3fn).double()  # noqa: E731  (the values fit: no overflow)
    for b in range(B):
        st, cnt = int(start[b]), n if counts is None else int(counts[b])
        for p in range(st // T, (st + cnt - 1) // T + 1 if cnt else 0):
            page = int(table[b, p])
            i0, i1 = max(st, p * T), min(st + cnt, p * T + T)
            for h in range(H):
                tok = x[b, h, i0 - st:i1 - st].double()
                e = exponent(float(tok.abs().max()))
                if st > p * T:
                    old = int(math.log2(float(sc[page, h])))
                    if e > old:
                        val[page, h, :st - p * T] = e4m3(val[page, h, :st - p * T] * 2.0 ** (old - e))
                    e = max(e, old)
                val[page, h, i0 - p * T:i1 - p * T] = e4m3(tok * 2.0 ** -e)
                sc[page, h] = 2.0 ** e
    return val, sc

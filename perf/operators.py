"""Workloads of the operators around the attention layer of a streaming video generator: the rotary embedding over
(time, height, width), attention within a window of frames and a few first tokens, its gradients, and the 8-bit cache
of earlier frames with the attention that reads it.

`run` computes each operator in its plain form (torch operations in 32 bits), or, where `own` is set, with the
package's kernels; `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -120, 119  # range of a cache page's scale exponent


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One new token of a 40-head layer: latency of the smallest call.
        dict(name="rope-token", op="rope", B=1, L=1, Hq=40, Hk=40, d=128, s0=22, s1=21, s2=21, dtype="bfloat16",
             interleaved=True, inverse=False, grid_h=45, grid_w=80, t0=100000),
        # Q and K of the 14B-class layer, straight from the projections ([B, L, H, d]) to the layer's [B, H, L, d].
        dict(name="rope-layer", op="rope", B=1, L=75600, Hq=40, Hk=40, d=128, s0=22, s1=21, s2=21, dtype="bfloat16",
             interleaved=True, inverse=False, grid_h=45, grid_w=80, t0=0),
        # Gradients through the embedding of a 30-head, d = 64 layer, pairs split half by half, fp32 gradients.
        dict(name="rope-grad", op="rope", B=1, L=17550, Hq=30, Hk=30, d=64, s0=8, s1=12, s2=12, dtype="float32",
             interleaved=False, inverse=True, grid_h=30, grid_w=45, t0=0),
        # A short odd clip with shared heads, in a padded batch: small launches.
        dict(name="window-clip", op="window", B=2, Hq=4, Hk=2, Lq=257, Lk=301, d=64, left=48, right=16, sinks=5, g=1,
             ragged=True),
        # Frame-causal attention of the 1.3B-class layer: 21 frames of 1,560 tokens, two earlier frames and the first.
        dict(name="window-frames", op="window", B=1, Hq=12, Hk=12, Lq=32760, Lk=32760, d=128, left=2, right=0,
             sinks=1560, g=1560, ragged=False),
        # One new token per sequence over bf16 keys: a window of 16,384 tokens and 128 first ones.
        dict(name="window-step", op="window", B=4, Hq=40, Hk=40, Lq=1, Lk=32760, d=128, left=16384, right=0, sinks=128,
             g=1, ragged=False),
        # Training on a clip with shared heads: odd length, causal.
        dict(name="grad-clip", op="grad", B=2, Hq=12, Hk=4, Lq=2049, Lk=2049, d=64, left=511, right=0, sinks=64, g=1,
             ragged=False),
        # Training at the 1.3B-class layer's length with the frame-causal window.
        dict(name="grad-frames", op="grad", B=1, Hq=12, Hk=12, Lq=32760, Lk=32760, d=128, left=2, right=0, sinks=1560,
             g=1560, ragged=False),
        # One token of eight sequences goes into the cache.
        dict(name="append-token", op="append", B=8, Hk=8, n=1, start=5000, d=128, T=64),
        # Four frames of the 14B-class layer (45 x 80 tokens each) go into the cache at once.
        dict(name="append-frames", op="append", B=1, Hk=40, n=14400, start=3601, d=128, T=128),
        # One new token of eight sequences reads a cache of 32,760 tokens, shared heads.
        dict(name="cache-step", op="cache", B=8, Hq=40, Hk=8, Lq=1, Lk=32760, d=128, T=64, left=-1, right=0, sinks=0,
             g=1),
        # A frame of 1,560 tokens reads the cached frames of the window and the first one.
        dict(name="cache-frame", op="cache", B=1, Hq=12, Hk=12, Lq=1560, Lk=32760, d=128, T=128, left=10, right=0,
             sinks=1560, g=1560),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope", "window", "window", "window", "grad", "grad", "append", "cache", "cache"])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        half = d // 2
        s0 = rng.randint(1, half // 2)
        s1 = rng.randint(1, (half - s0) // 2 + 1)
        s2 = half - s0 - s1 - rng.choice([0, 0, 4])  # a few pairs may stay unrotated
        Hk = _log(rng, 1, 40)
        c = dict(op=op, B=rng.choice([1, 1, 2]), L=_log(rng, 1, 12000), Hq=Hk * rng.choice([1, 1, 2]), Hk=Hk, d=d, s0=s0,
                 s1=s1, s2=max(1, s2), dtype=rng.choice(["bfloat16", "bfloat16", "float16", "float32"]),
                 interleaved=rng.random() < 0.5, inverse=rng.random() < 0.4, grid_h=_log(rng, 1, 60),
                 grid_w=_log(rng, 1, 90), t0=rng.choice([0, 1000, 1000000]))
        return c
    if op == "append":
        return dict(op=op, B=_log(rng, 1, 16), Hk=_log(rng, 1, 40), n=_log(rng, 1, 800), start=rng.randint(0, 3000), d=d,
                    T=rng.choice([16, 32, 64, 128]))
    Hk = _log(rng, 1, 12)
    B = rng.choice([1, 1, 2, 3])
    gq = rng.choice([1, 1, 2, 3, 5, 8])
    Lk = _log(rng, 1, 9000)
    if op == "grad":
        Lk = min(Lk, 4000)
        Lq = Lk if rng.random() < 0.7 else _log(rng, 1, Lk)
    elif op == "window":
        Lq = Lk if rng.random() < 0.6 else _log(rng, 1, Lk)
    else:
        Lq = rng.choice([1, 1, _log(rng, 1, 40), _log(rng, 1, 1600)])
        Lq = min(Lq, Lk)
    g = rng.choice([1, 1, _log(rng, 2, 600)])
    left = rng.choice([-1, _log(rng, 1, 3000) // g, rng.randint(0, 3)])
    right = rng.choice([0, 0, 0, rng.randint(0, 40) // g, -1])
    sinks = rng.choice([0, rng.randint(1, 200), g])
    c = dict(op=op, B=B, Hq=Hk * gq, Hk=Hk, Lq=Lq, Lk=Lk, d=d, left=left, right=right, sinks=sinks, g=g)
    while c["Hq"] * c["B"] * Lq * Lk > 1_200_000_000 and c["Hk"] > 1:  # no more than the listed ones cost
        c["Hk"] -= 1
        c["Hq"] = c["Hk"] * gq
    if op == "cache":
        c["T"] = rng.choice([16, 32, 64, 128])
    else:
        c["ragged"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _keys(gen, B, H, L, d):
    """Keys gather around a few directions, as those of a layer do, and their size differs from head to head."""
    out = _normal(gen, B, H, L, d)
    out.add_(_normal(gen, B, H, 1, d), alpha=0.5)
    return out.mul_(torch.exp2(_normal(gen, B, H, 1, 1).mul_(0.5))).to(torch.bfloat16)


def _pages(gen, B, L, T):
    """Pages of B sequences of up to L tokens, in no order, two more than are used; the table and the pool's size."""
    per = -(-L // T)
    table = torch.randperm(B * per + 2, generator=gen, device="cuda")[:B * per].to(torch.int32).view(B, per).contiguous()
    return table, B * per + 2


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c = dict(case)
    op, d = c["op"], c["d"]
    s = {"c": c}
    if op == "rope":
        B, L = c["B"], c["L"]
        t = torch.arange(L, device="cuda")
        hw = c["grid_h"] * c["grid_w"]
        pos = torch.stack([c["t0"] + t // hw, t % hw // c["grid_w"], t % c["grid_w"]], 1)
        s["pos"] = (pos + int(seed) % 7).to(torch.int32).contiguous()
        dt = getattr(torch, c["dtype"])
        # [B, L, H, d] as the projections leave it, seen as [B, H, L, d]
        s["q"] = torch.randn(B, L, c["Hq"], d, generator=gen, device="cuda", dtype=dt).transpose(1, 2)
        s["k"] = torch.randn(B, L, c["Hk"], d, generator=gen, device="cuda", dtype=dt).transpose(1, 2)
        return s
    if op == "append":
        B, Hk, T = c["B"], c["Hk"], c["T"]
        s["table"], pages = _pages(gen, B, c["start"] + c["n"], T)
        lens = c["start"] - torch.randint(0, min(c["start"], T) + 1, (B,), generator=gen, device="cuda")
        s["start"] = lens.to(torch.int32)
        s["k"] = _keys(gen, B, Hk, c["n"], d)
        s["v"] = _keys(gen, B, Hk, c["n"], d)
        for x in ("k", "v"):
            s[x + "8"] = (_normal(gen, pages, Hk, T, d) * 60).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            s[x + "s"] = torch.exp2(torch.randint(-9, -4, (pages, Hk), generator=gen, device="cuda").float())
        return s
    B, Hq, Hk, Lq, Lk = c["B"], c["Hq"], c["Hk"], c["Lq"], c["Lk"]
    s["q"] = _normal(gen, B, Hq, Lq, d).to(torch.bfloat16)
    if op == "cache":
        T = c["T"]
        s["table"], pages = _pages(gen, B, Lk, T)
        lens = Lk - torch.randint(0, max(1, (Lk - Lq) // 4 + 1), (B,), generator=gen, device="cuda")
        s["k_lens"] = lens.to(torch.int32)
        for x in ("k", "v"):
            s[x + "s"] = torch.exp2(torch.randint(-7, -5, (pages, Hk), generator=gen, device="cuda").float())
            s[x + "8"] = (_normal(gen, pages, Hk, T, d) * 80).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return s
    s["k"] = _keys(gen, B, Hk, Lk, d)
    s["v"] = _keys(gen, B, Hk, Lk, d)
    s["q_lens"] = s["k_lens"] = None
    if c["ragged"]:
        cut = torch.randint(0, max(1, Lq // 3), (B,), generator=gen, device="cuda")
        s["q_lens"] = (Lq - cut).to(torch.int32)
        s["k_lens"] = (Lk - cut).to(torch.int32)
    if op == "grad":
        s["do"] = _normal(gen, B, Hq, Lq, d).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ plain forms
def _freqs(c, device="cuda"):
    """Angle per step of each pair, 64 bits, and its axis: every axis has a geometric series of its own."""
    f = [10000.0 ** (-i / n) for n in (c["s0"], c["s1"], c["s2"]) for i in range(n)]
    ax = [a for a, n in enumerate((c["s0"], c["s1"], c["s2"])) for _ in range(n)]
    return torch.tensor(f, dtype=torch.float64, device=device), torch.tensor(ax, device=device)


def _rotate(x, cos, sin, P, interleaved):
    x32 = x.float()
    rot, rest = x32[..., :2 * P], x32[..., 2 * P:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = rot[..., :P], rot[..., P:]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([y, rest], -1).to(x.dtype)


def _plain_rope(s):
    c = s["c"]
    f, ax = _freqs(c)
    ang = s["pos"].double()[:, ax] * f  # positions far out need their angles in 64 bits
    cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
    if c["inverse"]:
        sin = -sin
    return [_rotate(s[x], cos, sin, f.numel(), c["interleaved"]) for x in ("q", "k")]


def _bands(c, q_lens, k_lens, device):
    """The rows in chunks of `n`: per chunk the key columns that any of its rows may see, and which of them each row
    sees.  Returns rows [m, n], columns [B, m, C] and the mask [B, m, n, C]."""
    Lq, Lk, g, left, right, sinks = c["Lq"], c["Lk"], c["g"], c["left"], c["right"], c["sinks"]
    whole = left < 0 or right < 0
    n = Lq if whole else min(Lq, max(256, (left + right + 1) * g // 3))
    m = -(-Lq // n)
    span = Lk if whole else min(Lk, (-(-(n - 1) // g) + 1 + left + right) * g)
    rows = torch.arange(m * n, device=device).view(m, n)
    off = (k_lens - q_lens).long().view(-1, 1, 1)
    blk = torch.div(rows + off, g, rounding_mode="floor")  # [B, m, n]
    lo = torch.zeros_like(blk) if left < 0 else (blk - left) * g
    hi = torch.full_like(blk, Lk) if right < 0 else (blk + right + 1) * g
    hi = torch.minimum(hi, k_lens.long().view(-1, 1, 1)).clamp_(min=0)
    hi = torch.where(rows < q_lens.long().view(-1, 1, 1), hi, torch.zeros_like(hi))
    first = lo[:, :, :1].clamp(min=0)  # [B, m, 1]
    if whole:
        first = torch.zeros_like(first)
    near = first + torch.arange(span, device=device)  # [B, m, span]
    cols, own_part = near, (near < 0)
    if sinks > 0 and not whole:
        far = torch.arange(min(sinks, Lk), device=device).expand(first.shape[0], m, -1)
        cols = torch.cat([far, near], -1)
        own_part = torch.cat([far >= first, near < 0], -1)  # a first token inside the window counts once
    j = cols.unsqueeze(2)
    mask = (j < hi.unsqueeze(3)) & ((j >= lo.unsqueeze(3)) | (j < sinks)) & ~own_part.unsqueeze(2)
    return rows, cols.clamp(max=Lk - 1), mask


def _chunks(x, rows):
    """[B, H, Lq, d] -> [B, H, m, n, d] in 32 bits, rows past the end as zeros."""
    B, H, L, d = x.shape
    m, n = rows.shape
    x = x.float()
    if m * n != L:
        x = torch.cat([x, x.new_zeros(B, H, m * n - L, d)], 2)
    return x.view(B, H, m, n, d)


def _columns(x, cols):
    """[B, Hk, Lk, d] -> [B, Hk, 1, m, C, d] in 32 bits."""
    b = torch.arange(x.shape[0], device=x.device).view(-1, 1, 1)
    return x.transpose(1, 2)[b, cols].float().permute(0, 3, 1, 2, 4).unsqueeze(2)


def _scores(s, c, q_lens, k_lens, k, v):
    rows, cols, mask = _bands(c, q_lens, k_lens, s["q"].device)
    B, Hq, Hk, d = c["B"], c["Hq"], c["Hk"], c["d"]
    q = _chunks(s["q"], rows).view(B, Hk, Hq // Hk, *rows.shape, d)
    kc, vc = _columns(k, cols), _columns(v, cols)
    sc = (q @ kc.transpose(-1, -2)).mul_(1.0 / math.sqrt(d))
    sc.masked_fill_(~mask[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = sc.sub_(top.clamp(min=-3e38)).exp_()
    tot = p.sum(-1, keepdim=True)
    lse = torch.where(tot > 0, top + tot.log(), torch.full_like(tot, -math.inf))
    p.div_(tot.clamp(min=1e-37))
    return rows, cols, mask, q, kc, vc, p, lse


def _rows_back(x, c):
    """[B, Hk, G, m, n, e] -> [B, Hq, Lq, e]."""
    return x.reshape(c["B"], c["Hq"], -1, x.shape[-1])[:, :, :c["Lq"]]


def _lens(s, c):
    q = s.get("q_lens")
    k = s.get("k_lens")
    full = lambda n: torch.full((c["B"],), n, device="cuda", dtype=torch.int32)  # noqa: E731
    return full(c["Lq"]) if q is None else q, full(c["Lk"]) if k is None else k


def _plain_window(s, k=None, v=None):
    c = s["c"]
    q_lens, k_lens = _lens(s, c)
    _, _, _, _, _, vc, p, lse = _scores(s, c, q_lens, k_lens, s["k"] if k is None else k, s["v"] if v is None else v)
    return [_rows_back(p @ vc, c).to(torch.bfloat16), _rows_back(lse, c)[..., 0].contiguous()]


def _plain_grad(s):
    c = s["c"]
    B, Hk, d, scale = c["B"], c["Hk"], c["d"], 1.0 / math.sqrt(c["d"])
    q_lens, k_lens = _lens(s, c)
    rows, cols, mask, q, kc, vc, p, lse = _scores(s, c, q_lens, k_lens, s["k"], s["v"])
    o = p @ vc
    do = _chunks(s["do"], rows).view_as(q)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    dp = do @ vc.transpose(-1, -2)
    ds = dp.sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = ds @ kc
    dk = (ds.transpose(-1, -2) @ q).sum(2)
    at = (torch.arange(B, device="cuda").view(-1, 1, 1) * c["Lk"] + cols).reshape(-1)

    def back(g):  # the columns of the chunks add up over the keys
        g = g.permute(0, 2, 3, 1, 4).reshape(-1, Hk * d)
        return torch.zeros(B * c["Lk"], Hk * d, device="cuda").index_add_(0, at, g).view(B, c["Lk"], Hk, d).transpose(1, 2)

    return [_rows_back(o, c).to(torch.bfloat16), _rows_back(dq, c).to(torch.bfloat16),
            back(dk).to(torch.bfloat16), back(dv).to(torch.bfloat16)]


def _plain_exponent(amax):
    """The least e with amax <= 448 * 2^e, within its range (frexp: amax = m * 2^x, 1/2 <= m < 1; 448 = 0.875 * 2^9)."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)


def _plain_append(s):
    c = s["c"]
    B, Hk, n, d, T = c["B"], c["Hk"], c["n"], c["d"], c["T"]
    start = s["start"].long()
    touched = -(-n // T) + 1  # pages that a sequence's new tokens can meet
    blk = (start // T).view(B, 1) + torch.arange(touched, device="cuda")
    at = blk.view(B, touched, 1) * T + torch.arange(T, device="cuda") - start.view(B, 1, 1)  # index of the new token
    new = (at >= 0) & (at < n)
    real = new.any(-1)
    page = s["table"].long().gather(1, blk.clamp(max=s["table"].shape[1] - 1))[real]  # [R]
    is_new, is_old = new[real][:, None, :, None], (at < 0)[real][:, None, :, None]
    grows = is_old.any(2)[:, :, 0]  # pages with earlier tokens keep their scale, or a larger one
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    out = []
    for x in ("k", "v"):
        tok = s[x].transpose(1, 2)[b, at.clamp(0, n - 1)][real].transpose(1, 2).float()  # [R, Hk, T, d]
        amax = (tok * is_new).abs().amax((2, 3))
        e = _plain_exponent(amax)
        e_old = torch.frexp(s[x + "s"][page])[1] - 1
        e = torch.where(grows, torch.maximum(e, e_old), e)
        keep = s[x + "8"].view(torch.uint8)[page]
        old = keep.view(torch.float8_e4m3fn).float() * torch.exp2((e_old - e).float())[:, :, None, None]
        val = torch.where(is_new, tok * torch.exp2(-e.float())[:, :, None, None], old).to(torch.float8_e4m3fn)
        codes = torch.where(is_new | is_old, val.view(torch.uint8), keep)
        s[x + "8"].view(torch.uint8)[page] = codes
        s[x + "s"][page] = torch.exp2(e.float())
        out += [s[x + "8"], s[x + "s"]]
    return out


def _plain_cache(s):
    c = s["c"]
    page = s["table"].long()
    kv = []
    for x in ("k", "v"):
        codes = s[x + "8"].view(torch.uint8)[page].view(torch.float8_e4m3fn)
        val = codes.float() * s[x + "s"][page][..., None, None]  # [B, pages, Hk, T, d]
        kv.append(val.transpose(1, 2).reshape(c["B"], c["Hk"], -1, c["d"])[:, :, :c["Lk"]])
    return _plain_window(s, *kv)


# ------------------------------------------------------------------ one pass
def run(state):
    c = state["c"]
    op = c["op"]
    if own:
        import cluster_routed_sparse_b200 as crs
        if op == "rope":
            return list(crs.rope_axes(state["q"], state["k"], state["pos"], (c["s0"], c["s1"], c["s2"]), theta=10000.0,
                                      interleaved=c["interleaved"], inverse=c["inverse"]))
        if op == "append":
            cache = crs.Cache8(state["k8"], state["v8"], state["ks"], state["vs"])
            crs.cache8_append(state["k"], state["v"], cache, state["table"], state["start"])
            return [state["k8"], state["ks"], state["v8"], state["vs"]]
        window = dict(left=c["left"], right=c["right"], sinks=c["sinks"], block=c["g"])
        if op == "cache":
            cache = crs.Cache8(state["k8"], state["v8"], state["ks"], state["vs"])
            return list(crs.cache8_attn(state["q"], cache, state["table"], state["k_lens"], return_lse=True, **window))
        window.update(q_lens=state["q_lens"], k_lens=state["k_lens"])
        o, lse = crs.window_attn(state["q"], state["k"], state["v"], return_lse=True, **window)
        if op == "window":
            return [o, lse]
        return [o] + list(crs.window_attn_backward(state["do"], state["q"], state["k"], state["v"], o, lse, **window))
    return {"rope": _plain_rope, "window": _plain_window, "grad": _plain_grad, "append": _plain_append,
            "cache": _plain_cache}[op](state)


# ------------------------------------------------------------------ work
def _pairs(c):
    """(visible (query, key) pairs, keys that any query sees) of one head, for sequences of the full length."""
    Lq, Lk, g = c["Lq"], c["Lk"], c["g"]
    pairs, low = 0, Lk
    top = 0
    for i in range(Lq):
        b = (i + Lk - Lq) // g
        lo = 0 if c["left"] < 0 else max(0, (b - c["left"]) * g)
        hi = Lk if c["right"] < 0 else max(0, min(Lk, (b + c["right"] + 1) * g))
        pairs += max(0, hi - lo) + min(max(0, min(c["sinks"], hi)), lo)
        low, top = min(low, lo), max(top, hi)
    keys = max(0, top - low) + min(c["sinks"], low)
    return pairs, min(keys, Lk)


def work(case):
    c = case
    op, d, B = c["op"], c["d"], c["B"]
    if op == "rope":
        e = {"bfloat16": 2, "float16": 2, "float32": 4}[c["dtype"]]
        n = B * c["L"] * (c["Hq"] + c["Hk"]) * d
        return {"bytes": 2 * n * e + 12 * c["L"], "flops": 3 * n}
    if op == "append":
        n = B * c["n"] * c["Hk"] * d * 2
        return {"bytes": 3 * n, "flops": 3 * n}
    pairs, keys = _pairs(c)
    q = B * c["Hq"] * c["Lq"] * d
    k = B * c["Hk"] * keys * d
    if op == "grad":  # forward and backward: q, k, v, do in; o, dq, dk, dv out
        return {"bytes": 2 * (4 * q + 4 * k) + 4 * q // d, "flops": 14.0 * B * c["Hq"] * pairs * d}
    kv = 2 * k * (1 if op == "cache" else 2)
    return {"bytes": 4 * q + kv + 4 * q // d, "flops": 4.0 * B * c["Hq"] * pairs * d}


# ------------------------------------------------------------------ 64 bits
def _exact_rope(s):
    c = s["c"]
    f, ax = _freqs(c, "cpu")
    ang = s["pos"].cpu().double().index_select(1, ax) * f
    z = torch.polar(torch.ones_like(ang), -ang if c["inverse"] else ang).cuda()
    P, out = f.numel(), []
    for x in ("q", "k"):
        y = s[x].double()
        i = torch.arange(P, device="cuda")
        a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, P + i)
        w = torch.complex(y[..., a], y[..., b]) * z
        y[..., a], y[..., b] = w.real, w.imag
        out.append(y)
    return out


def _exact_attention(s, k, v):
    """Row blocks against all keys, the mask written out from its definition."""
    c = s["c"]
    B, Hq, Hk, Lq, Lk, d, g = (c[x] for x in ("B", "Hq", "Hk", "Lq", "Lk", "d", "g"))
    o = torch.zeros(B, Hq, Lq, d, device="cuda", dtype=torch.float64)
    lse = torch.full((B, Hq, Lq), -math.inf, device="cuda", dtype=torch.float64)
    grad = c["op"] == "grad"
    dq, dk, dv = torch.zeros_like(o), torch.zeros(k.shape, device="cuda", dtype=torch.float64), \
        torch.zeros(k.shape, device="cuda", dtype=torch.float64)
    j = torch.arange(Lk, device="cuda")
    bj = torch.div(j, g, rounding_mode="floor")
    for b in range(B):
        ql = Lq if s.get("q_lens") is None else int(s["q_lens"][b])
        kl = Lk if s.get("k_lens") is None else int(s["k_lens"][b])
        step = max(1, min(ql, 60_000_000 // Lk))
        for i0 in range(0, ql, step):
            i = torch.arange(i0, min(ql, i0 + step), device="cuda")
            bi = torch.div(i + kl - ql, g, rounding_mode="floor")[:, None]
            see = (j < kl)[None].expand(len(i), Lk)
            if c["right"] >= 0:
                see = see & (bj[None] <= bi + c["right"])
            if c["left"] >= 0:
                see = see & ((bj[None] >= bi - c["left"]) | (j < c["sinks"])[None])
            for h in range(Hq):
                kk, vv, qq = k[b, h * Hk // Hq].double(), v[b, h * Hk // Hq].double(), s["q"][b, h, i].double()
                a = (qq @ kk.T / math.sqrt(d)).masked_fill_(~see, -math.inf)
                z = torch.logsumexp(a, 1)
                lse[b, h, i] = z
                p = torch.exp(a - z.clamp(min=-1e300)[:, None])
                o[b, h, i] = p @ vv
                if grad:
                    go = s["do"][b, h, i].double()
                    dv[b, h * Hk // Hq] += p.T @ go
                    ds = p * (go @ vv.T - (go * o[b, h, i]).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[b, h, i] = ds @ kk
                    dk[b, h * Hk // Hq] += ds.T @ qq
    return [o, dq, dk, dv] if grad else [o, lse]


def _exact_cache(s):
    c = s["c"]
    T = c["T"]
    kv = []
    t = torch.arange(c["Lk"], device="cuda")
    for x in ("k", "v"):
        page = s["table"][:, t // T].long()
        val = s[x + "8"].double()[page, :, t % T] * s[x + "s"].double()[page][..., None]
        kv.append(val.transpose(1, 2))
    return _exact_attention(s, *kv)


def _exact_append(s):
    """Sequence by sequence and page by page: what each code of a page stands for, in units of the page's scale and
    before its rounding to 8 bits, and the scales."""
    c = s["c"]
    n, T, out = c["n"], c["T"], []
    units = torch.tensor([2.0 ** e for e in range(MIN_EXP, MAX_EXP + 1)], dtype=torch.float64, device="cuda")
    for x in ("k", "v"):
        val, scale = s[x + "8"].double(), s[x + "s"].double()
        for b in range(c["B"]):
            start = int(s["start"][b])
            for p in range(start // T, (start + n - 1) // T + 1):
                page = int(s["table"][b, p])
                i0, i1 = max(start, p * T), min(start + n, p * T + T)
                tok = s[x][b, :, i0 - start:i1 - start].double()
                amax = tok.abs().amax((1, 2))
                unit = units[(E4M3_MAX * units[:-1] < amax[:, None]).sum(1)]
                if start > p * T:
                    unit = torch.maximum(unit, scale[page])
                    val[page, :, :start - p * T] *= (scale[page] / unit)[:, None, None]
                val[page, :, i0 - p * T:i1 - p * T] = tok / unit[:, None, None]
                scale[page] = unit
        out += [val, scale]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["c"]["op"]
    if op == "rope":
        return _exact_rope(s)
    if op == "append":
        return _exact_append(s)
    return _exact_cache(s) if op == "cache" else _exact_attention(s, s["k"], s["v"])

"""Measured cases of the cache operators: appending rows to a KV cache with the
position rotation applied on the way, and attention of the last tokens over the
cache, with a sliding window and sinks, over 16/32-bit rows and over e4m3 codes
with one scale per block of tokens and KV head.

With ``own`` false, ``run`` computes each operator in elementary torch
operations in fp32; with ``own`` true it calls the framework."""
import math

import torch

own = False

ROPE_BASE = 5e5
E_MIN, E_MAX = -24, 60          # exponents of an e4m3 block's power-of-two scale


def listed():
    c = []
    # -- appending with rotation
    # one token of one sequence into a bf16 page pool: the smallest call, all latency
    c.append(_append("append_one", "bf16", True, B=1, n=1, H=32, Hkv=8, dh=128, T=4096, block=16, lo=1000, hi=1000))
    # a decode step of 64 sequences into e4m3 pages, most of them partly filled
    c.append(_append("append_e4m3_step", "e4m3", True, B=64, n=1, H=32, Hkv=8, dh=128, T=2048, block=32, lo=300,
                     hi=2001))
    # ragged prompt chunks of the 32/8-head block into bf16 pages: memory rate
    c.append(_append("append_chunk", "bf16", True, B=4, n=4096, H=32, Hkv=8, dh=128, T=8192, block=64, lo=17, hi=4001,
                     ragged=True))
    # odd chunk of a 12-head block with 64-wide heads into contiguous e4m3 rows
    c.append(_append("append_e4m3_chunk", "e4m3", False, B=3, n=1371, H=12, Hkv=12, dh=64, T=4096, block=64, lo=5,
                     hi=2000, ragged=True))
    # -- window and sinks
    # one sequence, one token, a short window: latency
    c.append(_attn("window_one", "window", "bf16", True, B=1, n=1, H=32, Hkv=8, dh=128, T=8192, block=16, lo=8001,
                   hi=8001, window=1024, sinks=4))
    # a decode step of 32 sequences over contiguous rows, window 4096
    c.append(_attn("window_step", "window", "bf16", False, B=32, n=1, H=32, Hkv=8, dh=128, T=16384, block=0, lo=1024,
                   hi=16384, window=4096, sinks=4))
    # a few drafted tokens on the fp32 path
    c.append(_attn("window_draft_f32", "window", "f32", False, B=2, n=3, H=8, Hkv=2, dh=64, T=2048, block=0, lo=700,
                   hi=1999, window=500, sinks=7, ragged=True))
    # a prompt of 8192 tokens with a window: matrix instructions
    c.append(_attn("window_chunk", "window", "bf16", True, B=2, n=8192, H=32, Hkv=8, dh=128, T=8192, block=64, lo=8192,
                   hi=8192, window=4096, sinks=128))
    # -- e4m3 blocks
    # one token over one long cache: split over the keys
    c.append(_attn("e4m3_one_long", "e4m3", "e4m3", True, B=1, n=1, H=32, Hkv=8, dh=128, T=65536, block=64, lo=64003,
                   hi=64003))
    # a decode step of 32 ragged sequences
    c.append(_attn("e4m3_step", "e4m3", "e4m3", False, B=32, n=1, H=32, Hkv=8, dh=128, T=16384, block=32, lo=1024,
                   hi=16384))
    # drafted tokens of eight sequences: more rows than a decode step, fewer than a chunk
    c.append(_attn("e4m3_draft", "e4m3", "e4m3", True, B=8, n=7, H=32, Hkv=8, dh=128, T=8192, block=16, lo=2000,
                   hi=8001, window=2048, sinks=16, ragged=True))
    # a chunk of 2048 tokens at the end of a 16k cache
    c.append(_attn("e4m3_chunk", "e4m3", "e4m3", True, B=1, n=2048, H=32, Hkv=8, dh=128, T=16384, block=128, lo=16000,
                   hi=16000))
    return c


def _append(name, cache, paged, B, n, H, Hkv, dh, T, block, lo, hi, ragged=False):
    # lo, hi: the sequences' lengths before the append
    return dict(name=name, op="append", cache=cache, paged=paged, B=B, n=n, H=H, Hkv=Hkv, dh=dh, T=T, block=block,
                lo=lo, hi=hi, ragged=ragged, window=0, sinks=0)


def _attn(name, op, cache, paged, B, n, H, Hkv, dh, T, block, lo, hi, window=0, sinks=0, ragged=False):
    # lo, hi: the sequences' lengths with the call's own tokens in them
    return dict(name=name, op=op, cache=cache, paged=paged, B=B, n=n, H=H, Hkv=Hkv, dh=dh, T=T, block=block, lo=lo,
                hi=hi, ragged=ragged, window=window, sinks=sinks)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "window", "e4m3"])
    cache = "e4m3" if op == "e4m3" else rng.choice(["bf16", "bf16", "f32"] + (["e4m3"] if op == "append" else []))
    paged = rng.random() < 0.6
    dh = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 4, 8])
    block = rng.choice([16, 32, 48, 64, 128]) if paged or cache == "e4m3" else 0
    unit = block or 1
    ragged = rng.random() < 0.5
    if op == "append":
        n = _log(rng, 1, 4096)
        B = max(1, min(_log(rng, 1, 64), 16384 // n))
        hi = _log(rng, 1, 4096)
        lo = rng.randint(0, hi)
        T = -(-(hi + n + rng.randint(0, 100)) // unit) * unit
        c = _append("drawn", cache, paged, B, n, H, Hkv, dh, T, block, lo, hi, ragged)
    else:
        n = _log(rng, 1, 64 if cache == "f32" else 4096)
        if rng.random() < 0.35:
            n = rng.randint(1, 8)
        hi = n + _log(rng, 1, 4096 if cache == "f32" else 16384)
        lo = rng.randint(n, hi)
        B = max(1, min(_log(rng, 1, 32), 131072 // hi, 8192 // n))
        if cache == "f32":
            B = min(B, 4)
        T = -(-(hi + rng.randint(0, 500)) // unit) * unit
        window = rng.choice([0, _log(rng, 1, 8192)]) if op == "e4m3" else _log(rng, 1, 8192)
        sinks = rng.choice([0, 1, 4, 16, rng.randint(1, 300)]) if window else 0
        c = _attn("drawn", op, cache, paged, B, n, H, Hkv, dh, T, block, lo, hi, window, sinks, ragged)
    del c["name"]
    return c


# ---- sizes of a case -------------------------------------------------------

def _n_new(c):
    """Tokens of each sequence: all n, or ragged from n down to about n/2."""
    return [c["n"] - (b * c["n"] // (2 * c["B"]) if c["ragged"] else 0) for b in range(c["B"])]


def _lens(c):
    step = max(c["B"] - 1, 1)
    return [c["hi"] - b * (c["hi"] - c["lo"]) // step for b in range(c["B"])]


def _esize(c):
    return {"bf16": 2, "f32": 4, "e4m3": 1}[c["cache"]]


def work(case):
    c = case
    dh, H, Hkv = c["dh"], c["H"], c["Hkv"]
    es = 4 if c["cache"] == "f32" else 2                 # bytes of q, k, v and o
    nn = _n_new(c)
    tokens = sum(nn)
    if c["op"] == "append":
        rows = tokens * ((H * 2 * es) + 2 * Hkv * (es + _esize(c)))
        return {"bytes": rows * dh + tokens * dh * 4, "flops": 3 * tokens * (H + Hkv) * dh}
    keys = pairs = 0
    W, S = c["window"], c["sinks"]
    for L, m in zip(_lens(c), nn):
        first = L - m
        if W == 0:
            keys += L
            pairs += sum(range(first + 1, L + 1))
        else:
            lo = max(0, first - W + 1)
            keys += L - lo + min(S, lo)
            pairs += sum(min(p + 1, W) + min(S, max(0, p + 1 - W)) for p in range(first, L))
    scales = keys // c["block"] * Hkv * 8 if c["cache"] == "e4m3" else 0
    return {"bytes": keys * Hkv * 2 * dh * _esize(c) + scales + 2 * tokens * H * dh * es, "flops": 4 * dh * H * pairs}


# ---- inputs ----------------------------------------------------------------

def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    B, n, H, Hkv, dh, T = (c[k] for k in ("B", "n", "H", "Hkv", "dh", "T"))
    row = torch.float32 if c["cache"] == "f32" else torch.bfloat16

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    s = {"case": c}
    table = None
    if c["paged"]:
        per = T // c["block"]
        pages = B * per + 3                               # scattered over a pool with pages of others in it
        table = torch.randperm(pages, generator=g, device=dev)[:B * per].reshape(B, per).to(torch.int32)
        shape = (pages, Hkv, c["block"], dh)
        scale_shape = (pages, Hkv)
    else:
        shape = (B, Hkv, T, dh)
        scale_shape = (B, Hkv, T // c["block"]) if c["cache"] == "e4m3" else None
    for name in ("k", "v"):
        if c["cache"] == "e4m3":
            s[name] = (randn(*shape) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
            e = torch.randint(-8, -5, scale_shape, generator=g, device=dev)
            s[name + "_scale"] = torch.exp2(e.to(torch.float32))
        else:
            s[name] = randn(*shape).to(row)
            s[name + "_scale"] = None
    s["table"] = table
    lens = torch.tensor(_lens(c), dtype=torch.int32, device=dev)
    order = torch.randperm(B, generator=g, device=dev)
    s["lens"] = lens[order].contiguous()
    s["n_new"] = torch.tensor(_n_new(c), dtype=torch.int32, device=dev)[order].contiguous()
    if c["op"] == "append":
        s["start"] = s["lens"].clone()
        # the rows of a fused projection: q, k and v side by side
        qkv = randn(B, n, (H + 2 * Hkv) * dh).to(row)
        s["q"] = qkv[..., :H * dh].unflatten(-1, (H, dh))
        s["new_k"] = qkv[..., H * dh:(H + Hkv) * dh].unflatten(-1, (Hkv, dh))
        s["new_v"] = qkv[..., (H + Hkv) * dh:].unflatten(-1, (Hkv, dh))
        s["q_out"] = torch.zeros(B, n, H, dh, dtype=row, device=dev)
        phi = (torch.arange(T, dtype=torch.float64, device=dev)[:, None]
               * ROPE_BASE ** (torch.arange(dh // 2, dtype=torch.float64, device=dev) * (-2.0 / dh)))
        s["rope"] = torch.stack([phi.cos(), phi.sin()], -1).to(torch.float32)
    else:
        s["q"] = randn(B, n, H, dh).to(row)
        s["o"] = torch.zeros(B, n, H, dh, dtype=row, device=dev)
    if own:
        import causal_gqa_attention_rmsnorm_gb300 as tb
        s["kv"] = tb.KVCache(s["k"], s["v"], s["lens"], table, s["k_scale"], s["v_scale"])
        if c["op"] != "append":
            s["cfg"] = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=c["window"], sinks=c["sinks"],
                                     dtype=tb.TB_F32 if c["cache"] == "f32" else tb.TB_BF16)
            s["ws"] = tb.tb_kvcache_attn_workspace(s["cfg"], s["kv"], n)
    return s


# ---- the operators ---------------------------------------------------------

def run(state):
    s = state
    if s["case"]["op"] == "append":
        if own:
            import causal_gqa_attention_rmsnorm_gb300 as tb
            tb.tb_kvcache_append_rope(s["kv"], s["new_k"], s["new_v"], s["rope"], q=s["q"], q_out=s["q_out"],
                                      start=s["start"], n_new=s["n_new"])
        else:
            _plain_append(s)
        out = {"q": s["q_out"], "k": s["k"], "v": s["v"], "lens": s["lens"]}
        if s["k_scale"] is not None:
            out["k_scale"], out["v_scale"] = s["k_scale"], s["v_scale"]
        return out
    if own:
        import causal_gqa_attention_rmsnorm_gb300 as tb
        tb.tb_kvcache_attn(s["cfg"], s["q"], s["kv"], n_new=s["n_new"], o=s["o"], ws=s["ws"])
    else:
        _plain_attn(s)
    return s["o"]


def _rotate(x, cos, sin):
    a, b = x.float().unflatten(-1, (-1, 2)).unbind(-1)
    return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)


def _planes(s, pos, unit):
    """Index of (sequence, KV head, pos // unit) among the cache's planes of
    `unit` rows, [B, Hkv, *pos.shape[1:]]: pages, or runs of contiguous rows."""
    c = s["case"]
    B, Hkv = c["B"], c["Hkv"]
    h = torch.arange(Hkv, device=pos.device)[None, :, None]
    if s["table"] is not None:
        page = s["table"].long().gather(1, pos // c["block"])[:, None, :]
        return (page * Hkv + h) * (c["block"] // unit) + (pos % c["block"] // unit)[:, None, :]
    b = torch.arange(B, device=pos.device)[:, None, None]
    return (b * Hkv + h) * (c["T"] // unit) + (pos // unit)[:, None, :]


def _plain_append(s):
    c = s["case"]
    n, dh, T = c["n"], c["dh"], c["T"]
    start, n_new = s["start"].long()[:, None], s["n_new"].long()[:, None]
    i = torch.arange(n, device=start.device)[None, :]
    pos, live = start + i, i < n_new
    cos, sin = s["rope"][pos][:, :, None].unbind(-1)
    q = _rotate(s["q"], cos, sin)
    s["q_out"].copy_(torch.where(live[..., None, None], q, s["q_out"].float()))
    rows = {"k": _rotate(s["new_k"], cos, sin).transpose(1, 2), "v": s["new_v"].float().transpose(1, 2)}
    s["lens"].copy_((start + n_new)[:, 0])
    if c["cache"] != "e4m3":
        at = _planes(s, pos, 1)
        k, v = s["k"].view(-1, dh), s["v"].view(-1, dh)
        k[at] = torch.where(live[:, None, :, None], rows["k"].to(k.dtype), k[at])
        v[at] = torch.where(live[:, None, :, None], rows["v"].to(v.dtype), v[at])
        return
    # the blocks that the rows reach: old rows, then the new ones, then rows of no one
    bs = c["block"]
    nb = (n + bs - 2) // bs + 1
    blk = start // bs + torch.arange(nb, device=start.device)[None, :]
    used = blk * bs < start + n_new
    # (entries past the last block stand for the first one once more, with the same values)
    at = _planes(s, torch.where(used, blk, blk[:, :1]) * bs, bs)              # [B, Hkv, nb]
    r = (start // bs * bs + torch.arange(nb * bs, device=start.device)[None, :])
    old, new = r < start, (r >= start) & (r < start + n_new)
    src = (r - start).clamp(0, n - 1)[:, None, :, None].expand(-1, c["Hkv"], -1, dh)
    head = (start % bs != 0)[:, :, None] & (torch.arange(nb, device=start.device) == 0)
    k, v = s["k"].view(torch.uint8).view(-1, bs, dh), s["v"].view(torch.uint8).view(-1, bs, dh)
    _write_blocks(k, s["k_scale"].view(-1), at, rows["k"].gather(2, src), old, new, head, used)
    _write_blocks(v, s["v_scale"].view(-1), at, rows["v"].gather(2, src), old, new, head, used)


def _write_blocks(codes, scales, at, x, old, new, head, used):
    B, Hkv, nb = at.shape
    bs, dh = codes.shape[1:]
    x = x.unflatten(2, (nb, bs))
    new, old = (m.unflatten(1, (nb, bs))[:, None, :, :, None] for m in (new, old))
    top = torch.where(new, x.abs(), 0).amax((-1, -2))
    m, e = torch.frexp(top)                                                    # top = m 2^e, m in [1/2, 1)
    e = torch.where(top > 0, e - 9 + (m > 0.875), E_MIN).clamp(E_MIN, E_MAX)   # 448 = 0.875 * 2^9
    was = scales[at]
    scale = torch.where(head, torch.maximum(was, torch.exp2(e.float())), torch.exp2(e.float()))
    scale = torch.where(used[:, None], scale, scale[..., :1])
    had = codes[at]
    recoded = had.view(torch.float8_e4m3fn).float() * (was / scale)[..., None, None]
    put = torch.where(new, (x / scale[..., None, None]).clamp(-448, 448), recoded).to(torch.float8_e4m3fn)
    put = torch.where(new | old, put.view(torch.uint8), had)
    codes[at] = torch.where(used[:, None, :, None, None], put, put[:, :, :1])
    scales[at] = scale


def _rows32(s, name):
    """The cache's rows as fp32 [B, Hkv, T, dh]."""
    c = s["case"]
    x = s[name]
    if s["table"] is not None:
        x = x.view(torch.uint8)[s["table"].long()].view(x.dtype)               # [B, pages, Hkv, block, dh]
        x = x.float()
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][s["table"].long()][..., None, None]
        return x.transpose(1, 2).reshape(c["B"], c["Hkv"], c["T"], c["dh"])
    x = x.float()
    if s[name + "_scale"] is not None:
        x = (x.unflatten(2, (-1, c["block"])) * s[name + "_scale"][..., None, None]).flatten(2, 3)
    return x


def _plain_attn(s):
    c = s["case"]
    B, n, H, Hkv, dh, T = (c[k] for k in ("B", "n", "H", "Hkv", "dh", "T"))
    G = H // Hkv
    q = s["q"].float().reshape(B, n, Hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, dh)
    p = torch.matmul(q, _rows32(s, "k").transpose(-1, -2)).mul_(1 / math.sqrt(dh)).view(B, Hkv, G, n, T)
    i = torch.arange(n, device=q.device)[None, :, None]
    at = s["lens"][:, None, None] - s["n_new"][:, None, None] + i
    j = torch.arange(T, device=q.device)[None, None, :]
    hidden = j > at
    if c["window"]:
        hidden |= (j <= at - c["window"]) & (j >= c["sinks"])
    p.masked_fill_(hidden[:, None, None], -math.inf)
    p.sub_(p.amax(-1, keepdim=True).clamp_(min=-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * n, T), _rows32(s, "v")).view(B, Hkv, G, n, dh)
    o = (o / total.clamp_(min=1e-30)).permute(0, 3, 1, 2, 4).reshape(B, n, H, dh)
    live = (i < s["n_new"][:, None, None])[..., None]
    s["o"].copy_(torch.where(live, o, s["o"].float()))


# ---- the same in 64 bits, one sequence at a time ---------------------------

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    f64 = torch.float64
    B, n, H, Hkv, dh, T, bs = (c[k] for k in ("B", "n", "H", "Hkv", "dh", "T", "block"))
    lens, n_new = s["lens"].tolist(), s["n_new"].tolist()
    e4m3 = c["cache"] == "e4m3"
    pages = s["table"].tolist() if c["paged"] else None

    def where(b, t):
        """(plane, row) of token t of sequence b in a [planes, Hkv, rows, dh] cache."""
        return (pages[b][t // bs], t % bs) if c["paged"] else (b, t)

    if c["op"] != "append":
        out = torch.zeros(B, n, H, dh, dtype=f64, device=s["q"].device)
        for b in range(B):
            L, m = lens[b], n_new[b]
            first = L - m
            keep = 0 if c["window"] == 0 else max(0, first - c["window"] + 1)  # oldest key of any window
            js = torch.arange(L, device=out.device)
            js = torch.cat([js[:min(c["sinks"], keep)], js[keep:]])
            for h in range(Hkv):
                kv = []
                for name in ("k", "v"):
                    x, sc = s[name], s[name + "_scale"]
                    if c["paged"]:
                        pg = s["table"][b].long()[js // bs]
                        y = x.view(torch.uint8)[pg, h, js % bs] if e4m3 else x[pg, h, js % bs]
                        f = sc[pg, h].to(f64) if e4m3 else None
                    else:
                        y = (x.view(torch.uint8) if e4m3 else x)[b, h][js]
                        f = sc[b, h, js // bs].to(f64) if e4m3 else None
                    y = y.view(torch.float8_e4m3fn).float().to(f64) * f[:, None] if e4m3 else y.to(f64)
                    kv.append(y)
                at = torch.arange(first, L, device=out.device)[:, None]
                seen = js[None, :] <= at
                if c["window"]:
                    seen &= (at - js[None, :] < c["window"]) | (js[None, :] < c["sinks"])
                for r in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                    z = s["q"][b, :m, r].to(f64) @ kv[0].T / math.sqrt(dh)
                    out[b, :m, r] = torch.softmax(z.masked_fill_(~seen, -math.inf), -1) @ kv[1]
        return out

    phi = (torch.arange(T, dtype=f64, device=s["q"].device)[:, None]
           * torch.pow(torch.tensor(ROPE_BASE, dtype=f64, device=s["q"].device),
                       -2.0 * torch.arange(dh // 2, device=s["q"].device) / dh))
    turn = torch.polar(torch.ones_like(phi), phi)

    def turned(x, t0):
        z = torch.view_as_complex(x.to(f64).unflatten(-1, (-1, 2)).contiguous())
        return torch.view_as_real(z * turn[t0:t0 + len(x), None]).flatten(-2)

    out = {"q": s["q_out"].to(f64), "lens": None,
           **{name: s[name].to(torch.float32).to(f64) for name in ("k", "v")}}
    if e4m3:
        out.update({name: s[name].to(f64) for name in ("k_scale", "v_scale")})
    for b in range(B):
        t0, m = lens[b], n_new[b]
        out["q"][b, :m] = turned(s["q"][b, :m], t0)
        for name in ("k", "v"):
            x = s["new_" + name][b, :m]
            x = turned(x, t0) if name == "k" else x.to(f64)
            step = bs if c["paged"] or e4m3 else T
            t = t0
            while t < t0 + m:                              # one page, block or run of rows at a time
                end = min((t // step + 1) * step, t0 + m)
                plane, r = where(b, t)
                rows = x[t - t0:end - t0].transpose(0, 1)  # [Hkv, rows, dh]
                cache = out[name][plane]
                if not e4m3:
                    cache[:, r:r + end - t] = rows
                else:
                    scales = out[name + "_scale"]
                    slot = scales[plane] if c["paged"] else scales[b, :, t // bs]
                    top = rows.abs().amax((-1, -2))
                    e = torch.ceil(torch.log2(top / 448)).clamp_(E_MIN, E_MAX)
                    new = torch.exp2(e)
                    if t % bs:
                        new = torch.maximum(new, slot)
                        past = cache[:, r - t % bs:r]
                        past.copy_((past * (slot / new)[:, None, None]).float().to(torch.float8_e4m3fn).float())
                    cache[:, r:r + end - t] = (rows / new[:, None, None]).float().clamp(-448, 448).to(
                        torch.float8_e4m3fn).float().to(f64)
                    slot.copy_(new)
                t = end
    return out

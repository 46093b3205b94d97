"""Shared plumbing of the cache-operator tests: caches of every layout filled
from per-sequence rows, and reading them back."""
from __future__ import annotations

import numpy as np
import torch

import causal_gqa_attention_rmsnorm_gb300 as tb

ROW = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}       # half a rounding step, relative


def make_cache(kind, paged, B, Hkv, T, dh, block, seed=0, spare=3, fill=float("nan")):
    """A cache whose every row holds `fill` (e4m3: NaN codes), scales 1."""
    g = torch.Generator().manual_seed(seed)
    bt, pages = None, 0
    if paged:
        per = T // block
        pages = B * per + spare
        bt = torch.randperm(pages, generator=g)[:B * per].reshape(B, per).to(torch.int32).cuda()
    if kind == "e4m3":
        kv = tb.KVCache.empty_e4m3(B, Hkv, T, dh, block, block_table=bt, num_pages=pages)
        for t in (kv.k, kv.v):
            t.view(torch.uint8).fill_(0x7F if fill != 0 else 0)
        return kv
    if paged:
        return tb.KVCache.empty_paged(B, Hkv, T, dh, block, pages, bt, dtype=ROW[kind], fill=fill)
    return tb.KVCache.empty(B, Hkv, T, dh, dtype=ROW[kind], fill=fill)


def block_of(kv):
    """Rows per page or scale block (0: neither)."""
    if kv.block_table is not None:
        return kv.k.shape[2]
    return kv.k.shape[2] // kv.k_scale.shape[2] if kv.k_scale is not None else 0


def raw_rows(kv, name, b):
    """Stored rows of sequence b, [Hkv, T, dh], in the stored type (e4m3: uint8)."""
    x = getattr(kv, name)
    x = x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    if kv.block_table is None:
        return x[b]
    y = x[kv.block_table[b].long()]                       # [pages, Hkv, ps, dh]
    return y.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])


def scales(kv, name, b):
    """Scales of sequence b's blocks [Hkv, blocks] (e4m3)."""
    s = getattr(kv, name + "_scale")
    return s[b] if kv.block_table is None else s[kv.block_table[b].long()].T


def values(kv, name, b):
    """The values sequence b's rows stand for, [Hkv, T, dh] float64 numpy."""
    x = raw_rows(kv, name, b)
    if x.dtype == torch.uint8:
        x = x.contiguous().view(torch.float8_e4m3fn).float().double()
        return (x * scales(kv, name, b).double().repeat_interleave(block_of(kv), 1)[..., None]).cpu().numpy()
    return x.double().cpu().numpy()


def put_rows(kv, b, k, v):
    """Fill rows [0, L) of sequence b with k, v [Hkv, L, dh] (CPU fp32 tensors);
    e4m3: codes of the rows over scales of 2^-7."""
    for name, x in (("k", k), ("v", v)):
        buf, L = getattr(kv, name), x.shape[1]
        e4m3 = buf.dtype == torch.float8_e4m3fn
        x = (x * 128).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x.to(buf.dtype)
        x = x.cuda()
        buf = buf.view(torch.uint8) if e4m3 else buf
        if e4m3:
            s = getattr(kv, name + "_scale")
            if kv.block_table is None:
                s[b] = 2.0 ** -7
            else:
                s[kv.block_table[b].long()] = 2.0 ** -7
        if kv.block_table is None:
            buf[b, :, :L] = x
        else:
            ps = buf.shape[2]
            for p in range(-(-L // ps)):
                part = x[:, p * ps:(p + 1) * ps]
                buf[int(kv.block_table[b, p]), :, :part.shape[1]] = part


def rows(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def bits(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def attn_tolerance(kind, out, mag, top, dh, nkeys):
    """How far an output may be off its 64-bit value.  A score is an fp32 sum of
    dh products: off by at most (dh + 2) 2^-24 sum|q k|; with the rounding of the
    exponent's argument (|z| <= top, one unit of 2^-24 each for the product and
    the subtraction of the maximum) and 2^-22 of the exponential, a weight is off
    by e = (dh + 6) 2^-24 top + 2^-22, and a normalised one by 2e.  fp32 sums over
    the keys add (nkeys + 4) 2^-24, doubled for numerator and denominator.  The
    weights are rounded once more for their product with v (bf16 2^-8; over e4m3
    fp16 2^-11; fp32 not), and the output once to its type."""
    e = 2 * ((dh + 6) * 2.0 ** -24 * top[..., None] + 2.0 ** -22) + 2 * (nkeys + 4) * 2.0 ** -24
    p = {"f32": 0.0, "bf16": 2.0 ** -8, "e4m3": 2.0 ** -11}[kind]
    o = 2.0 ** -24 if kind == "f32" else 2.0 ** -8
    tol = (e + p) * mag * (1 + o)
    return tol + o * np.abs(out) + 1e-30


def check_attention(kind, got, out, mag, top, dh, nkeys, what=""):
    err = np.abs(got - out)
    tol = attn_tolerance(kind, out, mag, top, dh, nkeys)
    assert np.isfinite(got).all(), what
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst {float((err / tol).max()):.2f} of its bound"

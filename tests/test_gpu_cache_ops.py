"""tb_kvcache_append_rope and tb_kvcache_attn against the fp64 oracle: every
cache layout and type, head layouts, lengths from nothing to many key tiles,
windows and sinks, ragged batches, and what must stay untouched."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.cache as ref
from cache_helpers import (ROW, U, attn_tolerance, bits, block_of, check_attention, make_cache, put_rows, raw_rows,
                           rows, scales, values)

pytestmark = pytest.mark.gpu
BASE = 1e4


def tbm():
    import causal_gqa_attention_rmsnorm_gb300 as tb
    return tb


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def fused_rows(seed, B, n, H, Hkv, dh, dtype, pad=16):
    """q, k, v as column blocks of one padded projection."""
    x = rows(seed, B, n, (H + 2 * Hkv) * dh + pad, dtype=dtype).cuda()
    return (x[..., :H * dh].unflatten(-1, (H, dh)), x[..., H * dh:(H + Hkv) * dh].unflatten(-1, (Hkv, dh)),
            x[..., (H + Hkv) * dh:(H + 2 * Hkv) * dh].unflatten(-1, (Hkv, dh)))


# ---- append -----------------------------------------------------------------

def _check_block(kv, name, b, h, t_lo, t_hi, want, old_raw, old_scale, t0):
    """One e4m3 block's rows [t_lo, t_hi) against fp64 rows `want`, its older rows against what they were."""
    bs = block_of(kv)
    blk = t_lo // bs
    s = float(scales(kv, name, b)[h, blk])
    got = values(kv, name, b)[h, t_lo:t_hi]
    top = np.abs(want).max() if want.size else 0.0
    eps = 2.0 ** -20                                     # the fp32 rotation may move a maximum across a border
    need_lo, need_hi = ref.e4m3_scale(top * (1 - eps)), ref.e4m3_scale(top * (1 + eps))
    partial = t0 > blk * bs
    keep = float(old_scale[h, blk]) if partial else 0.0
    assert max(need_lo, keep) <= s <= max(need_hi, keep), (name, b, h, blk, s, top)
    # half a step of a code: 2^-4 relative, or half the smallest subnormal 2^-9
    rot = 4 * 2.0 ** -24 * 2 * max(top, 1e-30)
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * s + rot).all(), (name, b, h, blk)
    if partial:
        was = (old_raw[h, blk * bs:t0].contiguous().view(torch.float8_e4m3fn).float().double()
               * float(old_scale[h, blk])).cpu().numpy()
        now = values(kv, name, b)[h, blk * bs:t0]
        # a power-of-two change of scale moves nothing but subnormal codes
        assert (np.abs(now - was) <= 2.0 ** -10 * s)[~np.isnan(was)].all()


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("B,n,H,Hkv,dh,T,block,start,n_new", [
    (1, 1, 4, 1, 64, 64, 16, (0,), None),
    (3, 1, 8, 2, 128, 96, 32, (31, 0, 95), None),                     # last row, first row
    (4, 5, 8, 8, 64, 192, 48, (46, 0, 187, 60), (5, 0, 5, 3)),        # none at all; ends on the last row
    (2, 70, 32, 8, 128, 256, 16, (3, 186), (70, 70)),
    (3, 33, 2, 2, 16, 64, 64, (0, 31, 15), (33, 33, 17)),
    (2, 130, 12, 12, 64, 384, 128, (127, 250), (129, 130)),
])
def test_append(kind, paged, B, n, H, Hkv, dh, T, block, start, n_new):
    tb = tbm()
    if dh == 16 and kind == "e4m3":
        dh = 32
    kv = make_cache(kind, paged, B, Hkv, T, dh, block, seed=n, fill=0.0)
    for b in range(B):
        put_rows(kv, b, rows(100 + b, Hkv, T, dh, scale=0.2), rows(200 + b, Hkv, T, dh, scale=0.2))
    before = [(raw_rows(kv, "k", b).clone(), raw_rows(kv, "v", b).clone()) for b in range(B)]
    old_s = [(scales(kv, "k", b).clone(), scales(kv, "v", b).clone()) for b in range(B)] if kind == "e4m3" else None
    spare = bits(kv.k), bits(kv.v)
    q, k, v = fused_rows(n, B, n, H, Hkv, dh, ROW[kind])
    q_out = torch.full((B, n, H, dh), 7.0, dtype=ROW[kind], device="cuda")
    table = tb.tb_rope_table(dh, T + 3, BASE)
    got = tb.tb_kvcache_append_rope(kv, k, v, table, q=q, q_out=q_out, start=i32(*start),
                                    n_new=None if n_new is None else i32(*n_new))
    assert got is q_out
    assert tb.tb_get_device_error(clear=True) == 0
    nn = n_new or (n,) * B
    assert kv.lens.tolist() == [s + m for s, m in zip(start, nn)]
    rel = U["f32" if kind == "f32" else "bf16"]
    for b in range(B):
        t0, m = start[b], nn[b]
        q64, k64, v64 = (x[b, :m].double().cpu().numpy() for x in (q, k, v))
        def near(x, raw, turned):
            # two products and their sum, each rounded to fp32, of a table rounded to fp32: 4 * 2^-24 (|a| + |b|)
            pair = np.abs(raw).reshape(*raw.shape[:-1], dh // 2, 2).sum(-1).repeat(2, -1)
            assert (np.abs(x - turned) <= rel * np.abs(turned) * (1 + 2.0 ** -8) + 4 * 2.0 ** -24 * pair).all()
        near(q_out[b, :m].double().cpu().numpy(), q64, ref.rotated(q64, t0, BASE))
        assert (q_out[b, m:] == 7.0).all()
        k_rot = ref.rotated(k64, t0, BASE).transpose(1, 0, 2) if m else np.zeros((Hkv, 0, dh))
        v_row = v64.transpose(1, 0, 2)
        for idx, (name, want) in enumerate((("k", k_rot), ("v", v_row))):
            now = raw_rows(kv, name, b)
            if kind != "e4m3":
                x = now[:, t0:t0 + m].double().cpu().numpy()
                if name == "v":
                    assert np.array_equal(x, want)
                else:
                    near(x.transpose(1, 0, 2), k64, want.transpose(1, 0, 2))
                keep = torch.ones(T, dtype=torch.bool, device="cuda")
                keep[t0:t0 + m] = False
                assert np.array_equal(bits(now[:, keep]), bits(before[b][idx][:, keep]))
                continue
            bs = block_of(kv)
            for blk in range(T // bs):
                lo, hi = max(t0, blk * bs), min(t0 + m, (blk + 1) * bs)
                if lo >= hi:                              # a block that the call does not reach
                    assert np.array_equal(bits(now[:, blk * bs:(blk + 1) * bs]),
                                          bits(before[b][idx][:, blk * bs:(blk + 1) * bs]))
                    assert torch.equal(scales(kv, name, b)[:, blk], old_s[b][idx][:, blk])
                    continue
                assert np.array_equal(bits(now[:, hi:(blk + 1) * bs]), bits(before[b][idx][:, hi:(blk + 1) * bs]))
                for h in range(Hkv):
                    _check_block(kv, name, b, h, lo, hi, want[h, lo - t0:hi - t0], before[b][idx], old_s[b][idx], t0)
    if paged:                                             # pages of no sequence
        mine = set(kv.block_table.flatten().tolist())
        other = [p for p in range(kv.k.shape[0]) if p not in mine]
        for x, was in ((kv.k, spare[0]), (kv.v, spare[1])):
            assert np.array_equal(bits(x)[other], was[other])


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("block,dh", [(128, 128), (512, 128), (144, 256), (1536, 48)])
def test_append_into_large_blocks(paged, block, dh):
    """e4m3 blocks of more rows than a CTA's threads hold at once, and sizes that are no power of two."""
    T = 3 * block if block < 1536 else block
    test_append("e4m3", paged, 2, T // 2 + 5, 6, 3, dh, T, block, (T // 2 - 7, 3), (T // 2 + 5, T // 2 - 40))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_append_at_lens_equals_append_at_start(kind):
    """start=None reads the positions from lens; q may be rotated in place."""
    tb = tbm()
    B, n, H, Hkv, dh, T, block = 3, 7, 4, 2, 64, 128, 32
    a, b = (make_cache(kind, True, B, Hkv, T, dh, block, fill=0.0) for _ in range(2))
    lens = i32(0, 30, 121)
    a.lens.copy_(lens)
    b.lens.fill_(99)
    q = rows(1, B, n, H, dh, dtype=torch.bfloat16).cuda()
    k, v = rows(2, B, n, Hkv, dh, dtype=torch.bfloat16).cuda(), rows(3, B, n, Hkv, dh, dtype=torch.bfloat16).cuda()
    table = tb.tb_rope_table(dh, T, BASE)
    qa = q.clone()
    tb.tb_kvcache_append_rope(a, k, v, table, q=qa, q_out=qa)
    qb = tb.tb_kvcache_append_rope(b, k, v, table, q=q, start=lens)
    assert tb.tb_get_device_error(clear=True) == 0
    assert torch.equal(qa, qb) and torch.equal(a.lens, b.lens) and a.lens.tolist() == [7, 37, 128]
    assert np.array_equal(bits(a.k), bits(b.k)) and np.array_equal(bits(a.v), bits(b.v))


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_append_that_does_not_fit_leaves_the_sequence(kind):
    tb = tbm()
    B, n, H, Hkv, dh, T, block = 4, 6, 2, 1, 64, 64, 16
    kv = make_cache(kind, True, B, Hkv, T, dh, block, fill=0.0)
    kv.lens.copy_(i32(1, 2, 3, 4))
    bad = int(kv.block_table[3, 0])
    kv.block_table[3, 0] = kv.k.shape[0]                  # a page outside the pool
    k0, v0 = bits(kv.k).copy(), bits(kv.v).copy()
    q, k, v = fused_rows(5, B, n, H, Hkv, dh, ROW[kind])
    q_out = torch.full((B, n, H, dh), 7.0, dtype=ROW[kind], device="cuda")
    table = tb.tb_rope_table(dh, T, BASE)
    tb.tb_kvcache_append_rope(kv, k, v, table, q=q, q_out=q_out, start=i32(59, -1, 2147483647, 12))
    assert tb.tb_get_device_error(clear=True) == tb.TB_DEVERR_CACHE_FULL | tb.TB_DEVERR_BAD_PAGE
    assert kv.lens.tolist() == [1, 2, 3, 18]
    assert (q_out[:3] == 7.0).all() and (q_out[3] != 7.0).any()
    k1 = bits(kv.k)
    second = int(kv.block_table[3, 1])
    same = [p for p in range(kv.k.shape[0]) if p != second]
    assert np.array_equal(k1[same], k0[same]) and np.array_equal(bits(kv.v)[same], v0[same]) and bad != second
    assert not np.array_equal(k1[second], k0[second])     # the rows of its good page are stored


def test_append_e4m3_extremes():
    """Zero blocks, the smallest and largest magnitudes, infinities and NaN, a
    scale that grows, and a start taken back."""
    tb = tbm()
    dh, T, bs = 64, 64, 16
    kv = make_cache("e4m3", False, 1, 1, T, dh, bs, fill=0.0)
    table = tb.tb_rope_table(dh, T, BASE)
    v = torch.zeros(1, T, 1, dh, dtype=torch.bfloat16)
    v[0, 16:32] = rows(1, 16, 1, dh) * 1e-9
    v[0, 32:48] = 3e38
    v[0, 48:64] = rows(2, 16, 1, dh)
    v[0, 50, 0, 3], v[0, 51, 0, 4], v[0, 52, 0, 5] = math.inf, -math.inf, math.nan
    k = torch.zeros_like(v)
    tb.tb_kvcache_append_rope(kv, k.cuda(), v.cuda(), table, start=i32(0))
    s = kv.v_scale[0, 0].tolist()
    assert s[0] == 2.0 ** -24 and s[2] == 2.0 ** 60
    got = torch.from_numpy(values(kv, "v", 0))[0]
    assert (got[:16] == 0).all() and (got[32:48] == 448 * 2.0 ** 60).all()
    x = v[0, 16:32, 0].double()
    assert ((got[16:32] - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * s[1]).all()
    y = v[0, 48:64, 0].double()
    odd = ~torch.isfinite(y)
    assert torch.isnan(got[48:64][odd]).all() and int(odd.sum()) == 3
    assert ((got[48:64] - y).abs() <= 2.0 ** -4 * y.abs() + 2.0 ** -10 * s[3])[~odd].all()
    # small rows, then a large one in the same block: the older codes follow the larger scale
    small = rows(3, 1, 5, 1, dh, dtype=torch.bfloat16).cuda()
    big = (rows(4, 1, 2, 1, dh) * 300).to(torch.bfloat16).cuda()
    tb.tb_kvcache_append_rope(kv, small, small, table, start=i32(16))
    first = values(kv, "v", 0)[0, 16:21].copy()
    s0 = float(kv.v_scale[0, 0, 1])
    tb.tb_kvcache_append_rope(kv, big, big, table)
    s1 = float(kv.v_scale[0, 0, 1])
    assert s1 > s0 and kv.lens.tolist() == [23]
    assert (np.abs(values(kv, "v", 0)[0, 16:21] - first) <= 2.0 ** -10 * s1).all()
    # taken back to the block's start, its scale is that of the new rows again
    tb.tb_kvcache_append_rope(kv, small, small, table, start=i32(16))
    assert float(kv.v_scale[0, 0, 1]) == s0 and np.array_equal(values(kv, "v", 0)[0, 16:21], first)
    assert tb.tb_get_device_error(clear=True) == 0


# ---- attention --------------------------------------------------------------

def run_attention(kind, paged, lens, n, H, Hkv, dh, T, block, window=0, sinks=0, n_new=None, seed=0, scale=0.0,
                  fill=float("nan"), mutate=None):
    """One call against the oracle; rows of padding must keep their 7s."""
    tb = tbm()
    B = len(lens)
    kv = make_cache(kind, paged, B, Hkv, T, dh, block, seed=seed, fill=fill)
    for b, L in enumerate(lens):
        put_rows(kv, b, rows(seed + 10 * b + 1, Hkv, L, dh), rows(seed + 10 * b + 2, Hkv, L, dh))
    kv.lens.copy_(i32(*lens))
    vals = [(values(kv, "k", b)[:, :L], values(kv, "v", b)[:, :L]) for b, L in enumerate(lens)]
    if mutate:
        mutate(kv)
    q = rows(seed + 5, B, n, H, dh, dtype=ROW[kind]).cuda()
    o = torch.full((B, n, H, dh), 7.0, dtype=ROW[kind], device="cuda")
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=window, sinks=sinks, scale=scale,
                        dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    got = tb.tb_kvcache_attn(cfg, q, kv, n_new=None if n_new is None else i32(*n_new), o=o)
    assert got is o and tb.tb_get_device_error(clear=True) == 0
    for b, L in enumerate(lens):
        m = n if n_new is None else n_new[b]
        out, mag, top = ref.attend(q[b, :m].double().cpu().numpy(), *vals[b], L - m, window, sinks, scale or None)
        check_attention(kind, o[b, :m].double().cpu().numpy(), out, mag, top, dh, L, f"sequence {b}")
        assert (o[b, m:] == 7.0).all()
    return o


SHAPES = [  # H, Hkv, dh
    (4, 1, 64), (8, 8, 64), (8, 1, 128), (8, 4, 128), (8, 2, 128),
]


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,dh", SHAPES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 0), (100, 7)])
def test_one_token(kind, H, Hkv, dh, window, sinks):
    run_attention(kind, True, (1, 15, 16, 17, 49, 50, 51, 200, 333), 1, H, Hkv, dh, 352, 16, window, sinks, seed=3)
    run_attention(kind, False, (1, 33, 106, 107, 108, 240), 1, H, Hkv, dh, 240, 48, window, sinks, seed=4)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,dh", SHAPES)
@pytest.mark.parametrize("n,window,sinks", [(2, 0, 0), (4, 30, 3), (5, 0, 0), (9, 40, 20), (17, 0, 0), (33, 25, 130)])
def test_few_tokens(kind, H, Hkv, dh, n, window, sinks):
    lens, nn = (n, n + 1, 129, 300, 161), (n, n, 1, n, n - 1)
    run_attention(kind, True, lens, n, H, Hkv, dh, 320, 32, window, sinks, nn, seed=n)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,dh", SHAPES)
@pytest.mark.parametrize("n,lens,window,sinks", [
    (64, (64, 700), 0, 0),
    (128, (128, 129, 641), 0, 0),
    (200, (200, 1000), 130, 0),
    (257, (257, 600), 64, 140),
    (300, (300, 900), 128, 1),
])
def test_chunks(kind, H, Hkv, dh, n, lens, window, sinks):
    nn = [n - 3 * i for i in range(len(lens))]
    run_attention(kind, n % 2 == 0, lens, n, H, Hkv, dh, 1024, 64, window, sinks, nn, seed=n)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("block", [16, 48, 64, 128, 256])
def test_page_sizes(kind, block):
    T = 768
    run_attention(kind, True, (768, 500), 1, 8, 2, 128, T, block, 0, 0, seed=1)
    run_attention(kind, True, (768, 431), 40, 8, 2, 128, T, block, 200, 5, seed=2)
    if kind == "e4m3":
        run_attention(kind, False, (768, 431), 140, 8, 2, 64, T, block, 0, 0, seed=2)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 40, 150])
def test_rows_without_keys_and_empty_sequences(kind, n):
    """Sequences shorter than their queries (negative positions), of no rows, of no queries."""
    run_attention(kind, True, (0, n // 2, n, 96), n, 8, 2, 64, 160, 32, 0, 0, (n, n, n, 0), seed=n)
    run_attention(kind, True, (0, n // 2, n, 96), n, 8, 2, 64, 160, 32, 11, 2, (0, n, n, min(n, 96)), seed=n)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_window_of_one_and_wide_sinks(kind):
    run_attention(kind, True, (130, 260), 20, 4, 2, 64, 288, 32, 1, 0, seed=1)
    run_attention(kind, True, (130, 260), 20, 4, 2, 64, 288, 32, 1, 200, seed=2)
    run_attention(kind, True, (130, 260), 20, 4, 2, 64, 288, 32, 2 ** 31 - 1, 2 ** 31 - 1, seed=3)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_scale_argument(kind):
    run_attention(kind, True, (150,), 3, 4, 2, 64, 160, 32, scale=0.03125, seed=1)
    run_attention(kind, True, (150,), 60, 4, 2, 64, 160, 32, scale=-0.05, seed=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_pages_nobody_sees_are_not_read(kind, n):
    """Entries of the block table before every window and behind the sinks may be anything."""
    def mutate(kv):
        # first position of the sequence 700 - n; window 64, sinks 5: rows 5 .. 700 - n - 64 are hidden
        last = (700 - n - 64) // 16 - 1
        kv.block_table[0, 1:max(last, 1)] = -5
    run_attention(kind, True, (700,), n, 8, 2, 128, 704, 16, 64, 5, seed=n, mutate=mutate)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_visible_bad_page_counts_as_zeros(kind, n):
    tb = tbm()
    kv = make_cache(kind, True, 1, 2, 512, 64, 32, fill=0.0)
    put_rows(kv, 0, rows(1, 2, 512, 64), rows(2, 2, 512, 64))
    kv.lens.fill_(500)
    k, v = values(kv, "k", 0)[:, :500], values(kv, "v", 0)[:, :500]
    for p in (2, 9):
        k[:, p * 32:(p + 1) * 32], v[:, p * 32:(p + 1) * 32] = 0, 0
    kv.block_table[0, 2], kv.block_table[0, 9] = kv.k.shape[0], -1
    q = rows(5, 1, n, 8, 64, dtype=ROW[kind]).cuda()
    cfg = tb.AttnConfig(H=8, Hkv=2, dh=64, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    o = tb.tb_kvcache_attn(cfg, q, kv)
    assert tb.tb_get_device_error(clear=True) == tb.TB_DEVERR_BAD_PAGE
    out, mag, top = ref.attend(q[0].double().cpu().numpy(), k, v, 500 - n)
    check_attention(kind, o[0].double().cpu().numpy(), out, mag, top, 64, 500)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 40, 200])
def test_non_finite_rows_reach_only_queries_that_see_them(kind, n):
    """NaN in the v and k of single rows: the last row (seen by the last query
    only), one that leaves the window inside the call, and one before it."""
    tb = tbm()
    L, W, S, dh = 400, 64, 3, 64
    kv = make_cache(kind, True, 1, 2, 416, dh, 16, fill=float("nan"))
    put_rows(kv, 0, rows(1, 2, L, dh), rows(2, 2, L, dh))
    kv.lens.fill_(L)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    rows_bad = {L - 1: "v", L - n - W + 1 + n // 2: "v", max(S, L - n - W - 3): "k"}
    page = lambda t: int(kv.block_table[0, t // 16])
    for t, name in rows_bad.items():
        x = getattr(kv, name)
        (x.view(torch.uint8) if kind == "e4m3" else x)[page(t), 1, t % 16, 5] = 0x7F if kind == "e4m3" else math.nan
    q = rows(5, 1, n, 4, dh, dtype=ROW[kind]).cuda()
    cfg = tb.AttnConfig(H=4, Hkv=2, dh=dh, window=W, sinks=S, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    o = tb.tb_kvcache_attn(cfg, q, kv)[0].double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    out, mag, top = ref.attend(q[0].double().cpu().numpy(), k, v, L - n, W, S)
    tol = attn_tolerance(kind, out, mag, top, dh, L)
    for i in range(n):
        see = ref.visible(L - n + i, L, W, S)
        for h in range(4):
            bad_v = h >= 2 and any(see[t] for t, name in rows_bad.items() if name == "v")
            bad_k = h >= 2 and any(see[t] for t, name in rows_bad.items() if name == "k")
            nan = np.isnan(o[i, h])
            if bad_k:
                assert nan.all()
            else:
                assert nan[5] == bad_v and not np.delete(nan, 5).any(), (i, h)
                good = ~nan
                assert (np.abs(o[i, h] - out[i, h]) <= tol[i, h])[good].all(), (i, h)


@pytest.mark.parametrize("n", [1, 30, 200])
def test_e4m3_scales_that_differ_widely(n):
    """V scales 2^40 apart and an all-zero block keep their weights."""
    tb = tbm()
    L, dh, bs = 320, 64, 16
    kv = make_cache("e4m3", False, 1, 2, L, dh, bs, fill=0.0)
    put_rows(kv, 0, rows(1, 2, L, dh), rows(2, 2, L, dh))
    e = torch.randint(-24, 17, (1, 2, L // bs), generator=torch.Generator().manual_seed(1)).float()
    kv.v_scale.copy_(torch.exp2(e))
    kv.v.view(torch.uint8)[0, :, 64:80] = 0
    kv.v_scale[0, :, 4] = 2.0 ** -24
    kv.lens.fill_(L)
    q = rows(5, 1, n, 4, dh, dtype=torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=4, Hkv=2, dh=dh), q, kv)[0].double().cpu().numpy()
    out, mag, top = ref.attend(q[0].double().cpu().numpy(), values(kv, "k", 0), values(kv, "v", 0), L - n)
    check_attention("e4m3", o, out, mag, top, dh, L)


@pytest.mark.parametrize("n", [1, 40, 200])
def test_large_and_tiny_queries_over_e4m3(n):
    """Queries of very different sizes: one far above fp16's largest value (its
    softmax is a choice of one key), one far below its smallest."""
    tb = tbm()
    L, dh = 300, 64
    kv = make_cache("e4m3", False, 1, 2, 320, dh, 32, fill=0.0)
    put_rows(kv, 0, rows(1, 2, L, dh), rows(2, 2, L, dh))
    kv.lens.fill_(L)
    q = rows(5, 1, n, 4, dh)
    q[:, :, 0] *= 1e6
    q[:, :, 1] *= 1e-9
    q[:, :, 2] = 0
    q = q.to(torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=4, Hkv=2, dh=dh), q, kv)[0].double().cpu().numpy()
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    out, mag, top = ref.attend(q[0].double().cpu().numpy(), k, v, L - n)
    check_attention("e4m3", o[:, 1:], out[:, 1:], mag[:, 1:], top[:, 1:], dh, L)
    assert np.isfinite(o[:, 0]).all()


@pytest.mark.parametrize("n", [1, 5, 12, 40, 200])
def test_queries_with_one_large_element_over_e4m3(n):
    """An element of a query row 1000 times the others.  Chunks multiply queries
    as two 8-bit terms, which leaves an element off by at most 2^-17 of its row's
    largest: a score by 2^-17 max|q| sum|k| scale, counted on top."""
    tb = tbm()
    L, dh = 300, 64
    kv = make_cache("e4m3", False, 1, 2, 320, dh, 32, fill=0.0)
    put_rows(kv, 0, rows(1, 2, L, dh), rows(2, 2, L, dh))
    kv.k.view(torch.uint8)[..., 7] = 0                        # its dim is zero in the keys
    kv.lens.fill_(L)
    q = rows(5, 1, n, 4, dh)
    q[..., 7] = 1000
    q = q.to(torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=4, Hkv=2, dh=dh), q, kv)[0].double().cpu().numpy()
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    out, mag, top = ref.attend(q[0].double().cpu().numpy(), k, v, L - n)
    off = 2.0 ** -17 * 1000 * np.abs(k).sum(-1).max() / math.sqrt(dh)
    check_attention("e4m3", o, out, mag, top + off / ((dh + 6) * 2.0 ** -24), dh, L)


def test_lens_above_capacity_counts_as_capacity():
    tb = tbm()
    kv = make_cache("bf16", False, 1, 2, 160, 64, 0, fill=0.0)
    put_rows(kv, 0, rows(1, 2, 160, 64), rows(2, 2, 160, 64))
    q = rows(5, 1, 2, 4, 64, dtype=torch.bfloat16).cuda()
    cfg = tb.AttnConfig(H=4, Hkv=2, dh=64)
    kv.lens.fill_(160)
    want = tb.tb_kvcache_attn(cfg, q, kv)
    assert tb.tb_get_device_error(clear=True) == 0
    kv.lens.fill_(2 ** 31 - 1)
    got = tb.tb_kvcache_attn(cfg, q, kv)
    assert tb.tb_get_device_error(clear=True) == tb.TB_DEVERR_CACHE_FULL
    assert torch.equal(got, want)
    kv.lens.fill_(-3)
    assert (tb.tb_kvcache_attn(cfg, q, kv) == 0).all()
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_offsets_beyond_32_bits(kind):
    """A pool of more than 2^31 elements: pages at its far end."""
    tb = tbm()
    Hkv, dh, ps = 8, 128, 128
    pages = 2 ** 31 // (Hkv * dh * ps) + 40
    shape = (pages, Hkv, ps, dh)
    mk = lambda: torch.zeros(shape, dtype=torch.uint8 if kind == "e4m3" else torch.bfloat16, device="cuda")
    k, v = mk(), mk()
    T = 384
    bt = torch.tensor([[pages - 1, 3, pages - 7]], dtype=torch.int32, device="cuda")
    sc = lambda: torch.ones(pages, Hkv, device="cuda") if kind == "e4m3" else None
    if kind == "e4m3":
        k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
    kv = tb.KVCache(k, v, i32(0), bt, sc(), sc())
    table = tb.tb_rope_table(dh, T, BASE)
    n, H = 300, 16
    kn, vn = rows(1, 1, n, Hkv, dh, dtype=torch.bfloat16).cuda(), rows(2, 1, n, Hkv, dh, dtype=torch.bfloat16).cuda()
    qn = rows(3, 1, n, H, dh, dtype=torch.bfloat16).cuda()
    q = tb.tb_kvcache_append_rope(kv, kn, vn, table, q=qn)
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh)
    kk, vv = values(kv, "k", 0)[:, :n], values(kv, "v", 0)[:, :n]
    assert np.abs(vv).max() > 1
    for m in (1, n):
        o = tb.tb_kvcache_attn(cfg, q[:, n - m:].contiguous(), kv)[0].double().cpu().numpy()
        pick = [0, m - 1]
        for i in pick:
            out, mag, top = ref.attend(q[0, n - m + i:n - m + i + 1].double().cpu().numpy(), kk, vv, n - m + i)
            check_attention(kind, o[i:i + 1], out, mag, top, dh, n)
    assert tb.tb_get_device_error(clear=True) == 0


# ---- together ---------------------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 4)])
def test_chunks_drafts_and_steps_together(kind, window, sinks):
    """A prompt in two chunks, drafted tokens of which some are taken back, and
    single tokens, each appended and attended over, against attention of the
    whole sequence over the rows the cache ends up with at each point."""
    tb = tbm()
    B, H, Hkv, dh, T, bs = 2, 8, 2, 64, 384, 32
    kv = make_cache(kind, True, B, Hkv, T, dh, bs)
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=window, sinks=sinks,
                        dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    table = tb.tb_rope_table(dh, T, BASE)
    lens = [0, 0]
    steps = [(150, None, (150, 131)), (60, None, (37, 60)), (5, None, (5, 5)), (4, "back 3", (4, 4)),
             (1, None, (1, 1)), (1, None, (1, 1))]
    for s, (n, what, nn) in enumerate(steps):
        q, k, v = fused_rows(50 + s, B, n, H, Hkv, dh, ROW[kind])
        start = [x - 3 for x in lens] if what else lens
        o = torch.full((B, n, H, dh), 7.0, dtype=ROW[kind], device="cuda")
        qr = tb.tb_kvcache_append_rope(kv, k, v, table, q=q, start=i32(*start) if what else None, n_new=i32(*nn))
        tb.tb_kvcache_attn(cfg, qr, kv, n_new=i32(*nn), o=o)
        lens = [a + m for a, m in zip(start, nn)]
        assert kv.lens.tolist() == lens and tb.tb_get_device_error(clear=True) == 0
        for b in range(B):
            L, m = lens[b], nn[b]
            want_q = ref.rotated(q[b, :m].double().cpu().numpy(), L - m, BASE)
            assert np.abs(qr[b, :m].double().cpu().numpy() - want_q).max() <= 2.0 ** -7 * np.abs(want_q).max()
            out, mag, top = ref.attend(qr[b, :m].double().cpu().numpy(), values(kv, "k", b)[:, :L],
                                       values(kv, "v", b)[:, :L], L - m, window, sinks)
            check_attention(kind, o[b, :m].double().cpu().numpy(), out, mag, top, dh, L, f"step {s} sequence {b}")
            assert (o[b, m:] == 7.0).all()


def test_cache_of_the_block_goes_on():
    """A cache filled by the block's prefill is continued by these calls: the
    same rows as the block's decode step stores, and its attention."""
    import workloads
    from helpers import block_config, to_device
    tb = tbm()
    s = workloads.BlockShape("goes_on", "prefill", "bf16", B=2, T=70, d=512, H=8, Hkv=2, dh=64, f=1024,
                             rope_base=BASE, eps=1e-6, gains="ones")
    cfg = block_config(s, max_pos=128)
    inp = to_device(workloads.make_block_inputs(s, seed=3))
    packed = tb.tb_pack_weights(cfg, inp)
    kv = tb.KVCache.empty(s.B, s.Hkv, 128, s.dh, fill=float("nan"))
    tb.tb_block_prefill(cfg, packed, inp["x"], kv=kv)
    mine = tb.KVCache(kv.k.clone(), kv.v.clone(), kv.lens.clone())
    x = workloads.make_block_inputs(s, seed=4, x_tokens=1)["x"].cuda()
    tb.tb_block_decode(cfg, packed, x, kv)
    # the block's own projection, in fp64
    xf = x.double()
    xn = xf / torch.sqrt((xf * xf).mean(-1, keepdim=True) + s.eps)
    k = (xn @ inp["wk"].double()).unflatten(-1, (s.Hkv, s.dh)).to(torch.bfloat16)
    v = (xn @ inp["wv"].double()).unflatten(-1, (s.Hkv, s.dh)).to(torch.bfloat16)
    tb.tb_kvcache_append_rope(mine, k, v, tb.tb_rope_table(s.dh, 128, BASE))
    assert torch.equal(mine.lens, kv.lens)
    # rounded twice (projection, rotation) against once: two bf16 half steps of the pair
    a, b = mine.k[:, :, 70].double(), kv.k[:, :, 70].double()
    pair = (a.abs().unflatten(-1, (-1, 2)).sum(-1).repeat_interleave(2, -1))
    assert ((a - b).abs() <= 2.0 ** -8 * 3 * pair).all()
    assert ((mine.v[:, :, 70].double() - kv.v[:, :, 70].double()).abs() <= 2.0 ** -8 * 2 * v.double()[:, 0].abs() + 1e-6).all()
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 6, 150])
def test_graph_capture_streams_and_repeats(kind, n):
    """Captured and replayed with other contents, on a stream of its own, twice
    with the same inputs: the same bits."""
    tb = tbm()
    B, H, Hkv, dh, T, bs = 3, 8, 2, 128, 512, 64
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=200, sinks=4)
    table = tb.tb_rope_table(dh, T, BASE)
    start, nn = i32(0, 100, 512 - n), i32(n, max(n - 1, 1), n)

    def state():
        kv = make_cache(kind, True, B, Hkv, T, dh, bs, seed=1, fill=0.0)
        for b in range(B):
            put_rows(kv, b, rows(b, Hkv, T, dh), rows(b + 9, Hkv, T, dh))
        return kv, torch.zeros(B, n, H, dh, dtype=torch.bfloat16, device="cuda"), tb.tb_kvcache_attn_workspace(cfg, kv, n)

    def step(kv, o, ws, x, stream=None):
        qr = tb.tb_kvcache_append_rope(kv, x[1], x[2], table, q=x[0], start=start, n_new=nn, stream=stream)
        return tb.tb_kvcache_attn(cfg, qr, kv, n_new=nn, o=o, ws=ws, stream=stream)

    xa, xb = fused_rows(1, B, n, H, Hkv, dh, torch.bfloat16), fused_rows(2, B, n, H, Hkv, dh, torch.bfloat16)
    want = []
    for x in (xa, xb):
        kv, o, ws = state()
        step(kv, o, ws, x)
        want.append((o.clone(), bits(kv.k)))
    kv, o, ws = state()
    buf = [t.clone() for t in xa]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(kv, o, ws, buf)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want[0][0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(kv, o, ws, buf)
    for x, (w, kw) in zip((xb, xa, xb), (want[1], want[0], want[1])):
        for dst, src in zip(buf, x):
            dst.copy_(src)
        ws.fill_(255)                                     # nothing is expected in a workspace
        fresh, _, _ = state()
        kv.k.view(torch.uint8).copy_(fresh.k.view(torch.uint8))
        kv.v.view(torch.uint8).copy_(fresh.v.view(torch.uint8))
        if kind == "e4m3":
            kv.k_scale.copy_(fresh.k_scale)
            kv.v_scale.copy_(fresh.v_scale)
        g.replay()
        assert torch.equal(o, w) and np.array_equal(bits(kv.k), kw)
    # the stream argument, with buffers that the call allocates itself
    kv, o, _ = state()
    side.wait_stream(torch.cuda.current_stream())
    got = step(kv, None, None, xa, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for b in range(B):
        m = int(nn[b])
        assert torch.equal(got[b, :m], want[0][0][b, :m])
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 8, 700])
def test_a_value_row_of_nan_in_every_head(kind, n):
    """The first row's v is NaN and every query sees it: all NaN, in time."""
    tb = tbm()
    L, dh, Hkv, H = 1500, 128, 4, 16
    kv = make_cache(kind, True, 2, Hkv, 1536, dh, 64, fill=0.0)
    for b in range(2):
        put_rows(kv, b, rows(1 + b, Hkv, L, dh), rows(2 + b, Hkv, L, dh))
        (kv.v.view(torch.uint8) if kind == "e4m3" else kv.v)[int(kv.block_table[b, 0]), :, 0] = (
            0x7F if kind == "e4m3" else math.nan)
    kv.lens.fill_(L)
    q = rows(5, 2, n, H, dh, dtype=torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=H, Hkv=Hkv, dh=dh), q, kv)
    assert torch.isnan(o).all() and tb.tb_get_device_error(clear=True) == 0


def test_more_sequences_than_one_launch_takes():
    """1500 sequences of one token: two launches of the streaming kernel."""
    tb = tbm()
    B, Hkv, H, dh, T = 1500, 1, 2, 64, 32
    kv = tb.KVCache.empty(B, Hkv, T, dh)
    kv.k.copy_(rows(1, B, Hkv, T, dh))
    kv.v.copy_(rows(2, B, Hkv, T, dh))
    kv.lens.copy_(torch.arange(B, dtype=torch.int32) % (T + 1))
    q = rows(3, B, 1, H, dh, dtype=torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=H, Hkv=Hkv, dh=dh), q, kv).double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    for b in list(range(0, 40)) + list(range(1000, 1060)) + list(range(1480, 1500)):
        L = b % (T + 1)
        out, mag, top = ref.attend(q[b].double().cpu().numpy(), kv.k[b, :, :L].double().cpu().numpy(),
                                   kv.v[b, :, :L].double().cpu().numpy(), L - 1)
        check_attention("bf16", o[b], out, mag, top, dh, max(L, 1), f"sequence {b}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dh", [48, 256])
def test_append_of_other_widths(kind, dh):
    """Widths that the attention has no kernel for can be appended all the same."""
    tb = tbm()
    B, n, H, Hkv, T, bs = 2, 21, 3, 1, 64, 16
    kv = make_cache(kind, False, B, Hkv, T, dh, bs, fill=0.0)
    q, k, v = fused_rows(7, B, n, H, Hkv, dh, torch.bfloat16)
    qr = tb.tb_kvcache_append_rope(kv, k, v, tb.tb_rope_table(dh, T, BASE), q=q, start=i32(0, 40))
    assert kv.lens.tolist() == [21, 61] and tb.tb_get_device_error(clear=True) == 0
    for b, t0 in enumerate((0, 40)):
        want = ref.rotated(q[b].double().cpu().numpy(), t0, BASE)
        assert np.abs(qr[b].double().cpu().numpy() - want).max() <= 2.0 ** -8 * np.abs(want).max() * 1.01
        for name, x in (("k", ref.rotated(k[b].double().cpu().numpy(), t0, BASE)), ("v", v[b].double().cpu().numpy())):
            got = values(kv, name, b)[:, t0:t0 + n]
            rel = 2.0 ** -4 if kind == "e4m3" else 2.0 ** -8
            assert (np.abs(got - x.transpose(1, 0, 2)) <= rel * np.abs(x).max()).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv", [(8, 8), (8, 1), (4, 2)])
@pytest.mark.parametrize("n", [18, 40, 70, 129])
def test_one_and_two_row_tiles_over_long_caches(kind, H, Hkv, n):
    """Few row tiles and many key tiles: the slots share the tile, cuts go through every item."""
    run_attention(kind, True, (1500, 700), n, H, Hkv, 128, 1536, 64, 0, 0, (n, n - 1), seed=n)
    run_attention(kind, True, (1500, 131), n, H, Hkv, 64, 1536, 32, 300, 140, seed=n + 1)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("lens", [(9001,), (9001, 1, 0, 5000)])
@pytest.mark.parametrize("n", [1, 2, 4, 60])
def test_one_head_over_long_caches(kind, lens, n):
    """Many parts of one row's keys to join, and sequences with next to none beside it."""
    run_attention(kind, True, lens, n, 8, 1, 128, 9216, 64, seed=n)


@pytest.mark.parametrize("n", [1, 40, 300])
def test_small_addends_survive_large_ones(n):
    """A score whose products cancel but for one 2^-17 of them: sums are fp32."""
    tb = tbm()
    dh = 128
    for kind in ("e4m3", "bf16"):
        kv = make_cache(kind, False, 1, 1, 320, dh, 16, fill=0.0)
        if kind == "e4m3":
            kv.k_scale.fill_(1.0)
            kv.v_scale.fill_(1.0)
        k, v = torch.zeros(2, dh), torch.zeros(2, dh)
        k[:, 0:30:2], k[:, 1:30:2] = 256.0, -256.0
        k[0, 30] = 2.0 ** -9
        v[0] = 1
        for name, x in (("k", k), ("v", v)):
            buf = getattr(kv, name)
            if kind == "e4m3":
                buf.view(torch.uint8)[0, 0, :2] = x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            else:
                buf[0, 0, :2] = x.to(buf.dtype).cuda()
        kv.lens.fill_(2)
        q = torch.ones(1, n, 2, dh, dtype=torch.bfloat16, device="cuda")
        o = tb.tb_kvcache_attn(tb.AttnConfig(H=2, Hkv=1, dh=dh, scale=2.0 ** 9), q, kv, n_new=i32(1))
        # weights e / (1 + e) and 1 / (1 + e); one rounding of the weight, one of the output
        assert abs(float(o[0, 0, 0, 0]) - math.e / (1 + math.e)) <= 2 * 2.0 ** -8, kind
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_two_calls_at_once(kind):
    """Steps of two caches on two streams, each with a workspace of its own."""
    tb = tbm()
    B, H, Hkv, dh, T, bs = 2, 8, 2, 64, 1024, 32
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=300, sinks=4, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    table = tb.tb_rope_table(dh, T, BASE)
    sizes = (1, 150, 6, 40)

    def fresh(seed):
        kv = make_cache(kind, True, B, Hkv, T, dh, bs, seed=seed, fill=0.0)
        for b in range(B):
            put_rows(kv, b, rows(seed + b, Hkv, T, dh), rows(seed + b + 9, Hkv, T, dh))
        kv.lens.copy_(i32(500, 700))
        return kv, tb.tb_kvcache_attn_workspace(cfg, kv, max(sizes))

    xs = [[fused_rows(7 * s + n, B, n, H, Hkv, dh, ROW[kind]) for n in sizes] for s in range(2)]

    def steps(kv, ws, x):
        return [tb.tb_kvcache_attn(cfg, tb.tb_kvcache_append_rope(kv, k, v, table, q=q), kv, ws=ws) for q, k, v in x]

    want = [steps(*fresh(s), xs[s]) for s in range(2)]
    states = [fresh(s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in range(2):
        with torch.cuda.stream(streams[s]):
            got.append(steps(*states[s], xs[s]))
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[s], want[s]))
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_one_workspace_for_fewer_tokens(kind):
    tb = tbm()
    H, Hkv, dh, T = 8, 4, 64, 512
    kv = make_cache(kind, True, 3, Hkv, T, dh, 16, fill=0.0)
    for b in range(3):
        put_rows(kv, b, rows(b, Hkv, T, dh), rows(b + 5, Hkv, T, dh))
    kv.lens.copy_(i32(512, 300, 77))
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    ws = tb.tb_kvcache_attn_workspace(cfg, kv, 70)
    for n in (70, 1, 4, 5, 8, 9, 16, 17, 64, 65):
        q = rows(n, 3, n, H, dh, dtype=ROW[kind]).cuda()
        ws.fill_(255)
        assert torch.equal(tb.tb_kvcache_attn(cfg, q, kv, ws=ws), tb.tb_kvcache_attn(cfg, q, kv))
    assert tb.tb_get_device_error(clear=True) == 0


FIRST_CALL = """
import sys, torch
sys.path[:0] = [%r, %r]
import causal_gqa_attention_rmsnorm_gb300 as tb
from cache_helpers import make_cache, put_rows, rows
kind, n = %r, %d
kv = make_cache(kind, True, 2, 2, 512, 64, 32, fill=0.0)
for b in range(2):
    put_rows(kv, b, rows(b, 2, 512, 64), rows(b + 5, 2, 512, 64))
f32 = kind == "f32"
q, k, v = (rows(s, 2, n, h, 64, dtype=torch.float32 if f32 else torch.bfloat16).cuda() for s, h in ((1, 4), (2, 2), (3, 2)))
start = torch.tensor([100, 300], dtype=torch.int32, device="cuda")
cfg = tb.AttnConfig(H=4, Hkv=2, dh=64, dtype=tb.TB_F32 if f32 else tb.TB_BF16)
ws = tb.tb_kvcache_attn_workspace(cfg, kv, n)
o, qr = torch.zeros_like(q), torch.zeros_like(q)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    table = tb.tb_rope_table(64, 512, 1e4)
    tb.tb_kvcache_append_rope(kv, k, v, table, q=q, q_out=qr, start=start)
    tb.tb_kvcache_attn(cfg, qr, kv, o=o, ws=ws)
g.replay()
got = o.clone()
tb.tb_kvcache_append_rope(kv, k, v, tb.tb_rope_table(64, 512, 1e4), q=q, q_out=qr, start=start)
tb.tb_kvcache_attn(cfg, qr, kv, o=o, ws=ws)
assert torch.equal(o, got) and o.abs().max() > 0 and tb.tb_get_device_error() == 0
print("same")
"""


@pytest.mark.parametrize("kind,n", [("f32", 3), ("bf16", 1), ("bf16", 60), ("e4m3", 12), ("e4m3", 130)])
def test_first_calls_of_a_process_may_be_captured(kind, n):
    here = os.path.dirname(os.path.abspath(__file__))
    out = subprocess.run([sys.executable, "-c", FIRST_CALL % (os.path.dirname(here), here, kind, n)], cwd=here, timeout=300,
                         capture_output=True, text=True)
    assert out.stdout.split()[-1:] == ["same"], out.stderr[-2000:]


def test_the_binding_refuses_tensors_that_do_not_fit():
    tb = tbm()
    kv = make_cache("bf16", True, 2, 2, 128, 64, 16, fill=0.0)
    table = tb.tb_rope_table(64, 128, BASE)
    x = lambda *s, dtype=torch.bfloat16, device="cuda": torch.zeros(*s, dtype=dtype, device=device)
    q, k, v = x(2, 3, 4, 64), x(2, 3, 2, 64), x(2, 3, 2, 64)
    bad_rows = [x(2, 3, 2, 32), x(1, 3, 2, 64), x(2, 4, 2, 64), x(2, 3, 4, 64), x(2, 3, 2, 64, dtype=torch.float32),
                x(2, 3, 2, 64, device="cpu"), x(2, 3, 64, 2).transpose(2, 3), x(2, 2, 3, 64).transpose(1, 2), x(2, 3, 64)]
    for r in bad_rows:
        with pytest.raises(ValueError):
            tb.tb_kvcache_append_rope(kv, k, r, table)
    for kw in (dict(q_out=q), dict(q=q, q_out=x(2, 3, 4, 32)), dict(q=q, q_out=x(2, 3, 4, 64, dtype=torch.float32)),
               dict(start=i32(0)), dict(start=torch.zeros(2, dtype=torch.int64, device="cuda")),
               dict(n_new=torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError):
            tb.tb_kvcache_append_rope(kv, k, v, table, **kw)
    for t in (table.half(), table[:, :16].contiguous(), table.cpu(), table.reshape(-1)):
        with pytest.raises(ValueError):
            tb.tb_kvcache_append_rope(kv, k, v, t)
    with pytest.raises(tb.TbError):
        tb.tb_kvcache_append_rope(kv, k, v, table[:64])                       # shorter than the cache
    assert kv.lens.tolist() == [0, 0]
    cfg = tb.AttnConfig(H=4, Hkv=2, dh=64)
    for bad in (x(2, 3, 2, 64), x(2, 3, 4, 64, dtype=torch.float32), x(2, 3, 4, 64, device="cpu"), x(6, 4, 64),
                x(2, 4, 3, 64).transpose(1, 2)):
        with pytest.raises(ValueError):
            tb.tb_kvcache_attn(cfg, bad, kv)
        with pytest.raises(ValueError):
            tb.tb_kvcache_attn(cfg, q, kv, o=bad)
    for kw in (dict(n_new=i32(1)), dict(ws=torch.empty(1 << 24, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            tb.tb_kvcache_attn(cfg, q, kv, **kw)
    for kw in (dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda")), dict(o=q)):
        with pytest.raises(tb.TbError):
            tb.tb_kvcache_attn(cfg, q, kv, **kw)
    assert tb.tb_get_device_error(clear=True) == 0

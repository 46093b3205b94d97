"""Forms of the cache operators that a size, a width or a capacity selects: two row
tiles per warp of the streaming kernel, narrow fp32 heads, e4m3 rows of 16 elements,
queries of one key; and the attention beside the block's own."""
import math

import numpy as np
import pytest
import torch

import oracle.cache as ref
from cache_helpers import ROW, check_attention, make_cache, put_rows, rows, values
from test_gpu_cache_ops import BASE, i32, run_attention

pytestmark = pytest.mark.gpu


def tbm():
    import causal_gqa_attention_rmsnorm_gb300 as tb
    return tb


# ---- 17 to 32 rows of a KV head over much cache: two row tiles per warp -----------

# (H, Hkv, dh), n: 17, 24, 28 and 32 rows
TWO_TILES = [((8, 8, 64), 17), ((64, 8, 128), 3), ((32, 8, 128), 7), ((16, 8, 128), 14), ((16, 8, 64), 16),
             ((64, 8, 64), 4)]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape,n", TWO_TILES)
def test_two_row_tiles_per_warp(kind, shape, n):
    """More than 2^18 keys of capacity in all; ragged lengths, rows without keys,
    padding, pieces of many warps and of one."""
    H, Hkv, dh = shape
    T, lens = 8704, (3001, n, 0, 130, 1000)
    assert 16 < n * H // Hkv <= 32 and T * len(lens) * Hkv > 1 << 18
    run_attention(kind, False, lens, n, H, Hkv, dh, T, 32, 0, 0, (n, n, n, n - 1, 0), seed=n)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape,n", TWO_TILES[:4])
@pytest.mark.parametrize("window,sinks", [(2100, 37), (2048, 0), (2090, 5)])
def test_two_row_tiles_per_warp_with_a_window(kind, shape, n, window, sinks):
    """A window wide enough for the form, many sequences, scattered pages."""
    H, Hkv, dh = shape
    T, lens = 2304, (2300, 2150, 2048, 40) + (n + 1, ) * 12
    assert min(T, window + sinks + n) * len(lens) * Hkv > 1 << 18
    run_attention(kind, True, lens, n, H, Hkv, dh, T, 48, window, sinks, seed=n)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_two_row_tiles_repeat_and_agree_with_one_token_calls(kind):
    """The same bits in every call, with the workspace full of ones; each token's
    output is within two roundings of that of a call of its own."""
    tb = tbm()
    H, Hkv, dh, T, n, L = 32, 8, 128, 40960, 7, 5003
    kv = make_cache(kind, False, 1, Hkv, T, dh, 64, fill=0.0)
    put_rows(kv, 0, rows(1, Hkv, L, dh), rows(2, Hkv, L, dh))
    kv.lens.fill_(L)
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh)
    q = rows(3, 1, n, H, dh, dtype=torch.bfloat16).cuda()
    ws = tb.tb_kvcache_attn_workspace(cfg, kv, n)
    want = tb.tb_kvcache_attn(cfg, q, kv)
    for _ in range(20):
        ws.fill_(255)
        assert torch.equal(tb.tb_kvcache_attn(cfg, q, kv, ws=ws), want)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    for i in range(n):
        kv.lens.fill_(L - n + 1 + i)
        one = tb.tb_kvcache_attn(cfg, q[:, i:i + 1].contiguous(), kv)
        out, mag, _ = ref.attend(q[0, i:i + 1].double().cpu().numpy(), k, v, L - n + i)
        # both sides: a weight and an output rounded (2^-8 each over bf16, 2^-11 and 2^-8 over e4m3), and 2^-10 for the sums
        p = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
        tol = 2 * ((p + 2.0 ** -10) * mag + 2.0 ** -8 * (np.abs(out) + mag * p))
        assert (np.abs((one - want[:, i:i + 1])[0].double().cpu().numpy()) <= tol).all()
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_two_row_tiles_and_nan(kind):
    """A NaN that leaves the window inside the call reaches the queries that see it, and no other."""
    tb = tbm()
    H, Hkv, dh, B, T, n, W, S = 16, 8, 64, 16, 2304, 16, 2100, 20
    kv = make_cache(kind, True, B, Hkv, T, dh, 32)
    L = 2290
    for b in range(B):
        put_rows(kv, b, rows(b, Hkv, L, dh), rows(b + 9, Hkv, L, dh))
    kv.lens.fill_(L)
    t = L - n - W + 8                                      # seen by queries 0 .. 7
    page = int(kv.block_table[3, t // 32])
    x = kv.v.view(torch.uint8) if kind == "e4m3" else kv.v
    x[page, 5, t % 32, 9] = 0x7F if kind == "e4m3" else math.nan
    q = rows(3, B, n, H, dh, dtype=torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=W, sinks=S), q, kv)
    bad = torch.zeros(B, n, H, dh, dtype=torch.bool, device="cuda")
    see = [bool(ref.visible(L - n + i, L, W, S)[t]) for i in range(n)]
    assert see == [i < 8 for i in range(n)]
    bad[3, :8, 10:12, 9] = True
    assert torch.equal(torch.isnan(o), bad) and tb.tb_get_device_error(clear=True) == 0
    # queries on both sides of the row against the oracle
    k, v = values(kv, "k", 3)[:, :L], values(kv, "v", 3)[:, :L]
    for i in (8, 15):
        out, mag, top = ref.attend(q[3, i:i + 1].double().cpu().numpy(), k, np.nan_to_num(v), L - n + i, W, S)
        check_attention(kind, o[3, i:i + 1].double().cpu().numpy(), out, mag, top, dh, L)


# ---- fp32 heads of 16 and 32 ----------------------------------------------------

@pytest.mark.parametrize("dh", [16, 32])
@pytest.mark.parametrize("H,Hkv", [(4, 1), (8, 8), (8, 1), (8, 4)])
@pytest.mark.parametrize("n,window,sinks", [(1, 0, 0), (1, 50, 3), (5, 0, 0), (9, 40, 20), (150, 0, 0), (150, 33, 70)])
def test_narrow_fp32_heads(dh, H, Hkv, n, window, sinks):
    lens = (n, n + 1, max(n, 129), 300, max(n // 2, 1), 0)
    nn = (n, n, n, n - 1, n, n)
    run_attention("f32", True, lens, n, H, Hkv, dh, 320, 16, window, sinks, nn, seed=n)
    run_attention("f32", False, lens, n, H, Hkv, dh, 301, 0, window, sinks, seed=n + 1)


@pytest.mark.parametrize("dh", [16, 32])
@pytest.mark.parametrize("n", [1, 3, 60])
def test_narrow_fp32_heads_over_long_caches(dh, n):
    """Key ranges of a row joined."""
    run_attention("f32", True, (9001, 1, 0, 5000), n, 8, 1, dh, 9216, 64, seed=n)
    run_attention("f32", False, (7003, ), n, 4, 2, dh, 7003, 0, 3000, 9, seed=n)


def test_a_workspace_of_the_fp32_kernel_that_does_not_do_is_refused():
    tb = tbm()
    kv = make_cache("f32", False, 1, 8, 4096, 64, 0, fill=0.0)
    kv.lens.fill_(4000)
    cfg = tb.AttnConfig(H=8, Hkv=8, dh=64, dtype=tb.TB_F32)
    q = rows(1, 1, 1, 8, 64).cuda()
    need = tb.tb_kvcache_attn_workspace_bytes(cfg, kv, 1)
    assert need > 256
    for ws in (torch.empty(need // 2, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 128, dtype=torch.uint8, device="cuda")[128:]):
        with pytest.raises(tb.TbError, match="ws must be"):
            tb.tb_kvcache_attn(cfg, q, kv, ws=ws)


# ---- append ---------------------------------------------------------------------

@pytest.mark.parametrize("paged", [False, True])
def test_append_e4m3_rows_of_16(paged):
    tb = tbm()
    B, n, Hkv, dh, T, bs = 2, 37, 3, 16, 96, 16
    kv = make_cache("e4m3", paged, B, Hkv, T, dh, bs, fill=0.0)
    k, v = rows(1, B, n, Hkv, dh, dtype=torch.bfloat16).cuda(), rows(2, B, n, Hkv, dh, dtype=torch.bfloat16).cuda()
    tb.tb_kvcache_append_rope(kv, k, v, tb.tb_rope_table(dh, T, BASE), start=i32(5, 59))
    assert kv.lens.tolist() == [42, 96] and tb.tb_get_device_error(clear=True) == 0
    for b, t0 in enumerate((5, 59)):
        for name, x in (("k", ref.rotated(k[b].double().cpu().numpy(), t0, BASE)), ("v", v[b].double().cpu().numpy())):
            got, want = values(kv, name, b)[:, t0:t0 + n], x.transpose(1, 0, 2)
            for h in range(Hkv):
                for blk in range(t0 // bs, (t0 + n - 1) // bs + 1):
                    lo, hi = max(blk * bs, t0) - t0, min((blk + 1) * bs, t0 + n) - t0
                    # half a step of a code, or of the smallest of the block's scale; the first block keeps a scale of 1
                    s = max(ref.e4m3_scale(np.abs(want[h, lo:hi]).max()), 1.0 if blk * bs < t0 else 0.0)
                    err = np.abs(got[h, lo:hi] - want[h, lo:hi])
                    assert (err <= 2.0 ** -4 * np.abs(want[h, lo:hi]) + 2.0 ** -10 * s + 2.0 ** -20).all(), (name, b, h, blk)


def test_a_lens_that_is_not_dense_is_refused():
    tb = tbm()
    state = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    kv = make_cache("bf16", True, 2, 2, 128, 64, 16, fill=0.0)
    x = lambda h: torch.zeros(2, 3, h, 64, dtype=torch.bfloat16, device="cuda")
    for lens in (state[:, 0], torch.zeros(1, dtype=torch.int32, device="cuda").expand(2)):
        bad = tb.KVCache(kv.k, kv.v, lens, kv.block_table)
        with pytest.raises(ValueError, match="lens"):
            tb.tb_kvcache_append_rope(bad, x(2), x(2), tb.tb_rope_table(64, 128, BASE))
        with pytest.raises(ValueError, match="lens"):
            tb.tb_kvcache_attn(tb.AttnConfig(H=4, Hkv=2, dh=64), x(4), bad)
    assert (state == 0).all()


# ---- queries that choose one key -------------------------------------------------

@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 9, 40, 200])
def test_large_queries_choose_one_key(kind, n):
    """Queries 10^6 times the usual: where the two largest scores lie far enough
    apart, the output is one row of v."""
    tb = tbm()
    L, dh, H = 300, 64, 4
    kv = make_cache(kind, False, 1, 2, 320, dh, 32, fill=0.0)
    put_rows(kv, 0, rows(1, 2, L, dh), rows(2, 2, L, dh))
    kv.lens.fill_(L)
    q = (rows(5, 1, n, H, dh) * 1e6).to(ROW[kind]).cuda()
    cfg = tb.AttnConfig(H=H, Hkv=2, dh=dh, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    o = tb.tb_kvcache_attn(cfg, q, kv)[0].double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    k, v, q = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L], q[0].double().cpu().numpy()
    sure = 0
    for i in range(n):
        for h in range(H):
            m = L - n + i + 1
            z = k[h // 2, :m] @ q[i, h] / math.sqrt(dh)
            # fp32 sums of dh products; over e4m3 an element of q off by 2^-17 of the largest
            off = (dh + 6) * 2.0 ** -24 * (np.abs(k[h // 2, :m]) @ np.abs(q[i, h])).max() / math.sqrt(dh)
            if kind == "e4m3":
                off += 2.0 ** -17 * np.abs(q[i, h]).max() * np.abs(k[h // 2, :m]).sum(-1).max() / math.sqrt(dh)
            best, second = np.argsort(z)[::-1][:2]
            if z[best] - z[second] <= 2 * off + 40:
                continue
            sure += 1
            # all other weights together below 300 e^-40; one rounding of the weight, one of the output
            want = v[h // 2, best]
            tol = {"f32": 2.0 ** -22, "bf16": 2.0 ** -7, "e4m3": 2.0 ** -8 + 2.0 ** -10}[kind]
            assert (np.abs(o[i, h] - want) <= tol * np.abs(want) + 1e-12).all(), (i, h)
    assert sure >= n * H // 2


# ---- beside the block --------------------------------------------------------------

@pytest.mark.parametrize("H,Hkv,dh", [(8, 2, 64), (8, 8, 64), (4, 1, 128)])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_beside_the_blocks_decode_step(H, Hkv, dh, window):
    """A block whose output projection is the identity and whose feed-forward part
    is zero returns x plus its attention: the same step through these calls over
    the cache that it left."""
    import workloads
    from helpers import block_config, to_device
    tb = tbm()
    d = H * dh
    s = workloads.BlockShape("beside", "prefill", "bf16", B=2, T=70, d=d, H=H, Hkv=Hkv, dh=dh, f=1024, rope_base=BASE,
                             eps=1e-6, gains="ones")
    inp = workloads.make_block_inputs(s, seed=3)
    inp["wo"] = torch.eye(d, dtype=inp["wo"].dtype)
    inp["w2"] = torch.zeros_like(inp["w2"])
    inp = to_device(inp)
    cfg = block_config(s, max_pos=128)
    if window:
        cfg = tb.BlockConfig(**{**cfg.__dict__, "window": window})
    packed = tb.tb_pack_weights(cfg, inp)
    kv = tb.KVCache.empty(s.B, Hkv, 128, dh, fill=float("nan"))
    tb.tb_block_prefill(cfg, packed, inp["x"], kv=kv)
    x = workloads.make_block_inputs(s, seed=4, x_tokens=1)["x"].cuda()
    y = tb.tb_block_decode(cfg, packed, x, kv)
    assert kv.lens.tolist() == [71, 71]
    theirs = (y.double() - x.double())[:, 0].unflatten(-1, (H, dh)).cpu().numpy()
    # the query of the block's own projection, rotated, in fp64
    xf = x.double()
    xn = xf / torch.sqrt((xf * xf).mean(-1, keepdim=True) + s.eps)
    q64 = (xn @ inp["wq"].double()).unflatten(-1, (H, dh))
    pos = torch.full((s.B, ), 70, dtype=torch.int32, device="cuda")
    scratch = tb.KVCache.empty(s.B, Hkv, 128, dh)
    zero = torch.zeros(s.B, 1, Hkv, dh, dtype=torch.bfloat16, device="cuda")
    q = tb.tb_kvcache_append_rope(scratch, zero, zero, tb.tb_rope_table(dh, 128, BASE), q=q64.to(torch.bfloat16), start=pos)
    mine = tb.tb_kvcache_attn(tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, window=window), q, kv)[:, 0].double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    for b in range(s.B):
        qe = ref.rotated(q64[b].cpu().numpy(), 70, BASE)
        out, mag, _ = ref.attend(qe, values(kv, "k", b)[:, :71], values(kv, "v", b)[:, :71], 70, window)
        # Both against the formula.  A query is rounded to bf16 twice here and once or
        # twice in the block (the projection's fp32 sums below that): an element of a
        # pair by 2^-8 twice of its length, at most, so a score by e = 2 2^-8 sum_pairs
        # |q||k| scale and a weight by e^(2e) - 1; weight and output are rounded to bf16.
        pair = lambda a: np.sqrt((a.reshape(*a.shape[:-1], -1, 2) ** 2).sum(-1))
        see = ref.visible(70, 71, window)
        for h in range(H):
            ks = pair(values(kv, "k", b)[h // (H // Hkv), :71][see])
            e = 2 * 2.0 ** -8 * (ks @ pair(qe[0, h])).max() / math.sqrt(dh)
            tol = (math.expm1(2 * e) + 2.0 ** -8) * mag[0, h] * (1 + 2.0 ** -7) + 2.0 ** -8 * np.abs(out[0, h])
            assert (np.abs(mine[b, h] - out[0, h]) <= tol).all()
            # (x + attention in fp32)
            assert (np.abs(theirs[b, h] - out[0, h]) <= tol + 2.0 ** -22 * (np.abs(out[0, h]) + 8)).all()


# ---- calls that are allowed and unusual ------------------------------------------

@pytest.mark.parametrize("kind,T,block", [("bf16", 1, 0), ("bf16", 5, 0), ("bf16", 77, 0), ("bf16", 333, 0),
                                          ("e4m3", 16, 16), ("e4m3", 48, 48), ("e4m3", 80, 16), ("e4m3", 336, 112),
                                          ("f32", 1, 0), ("f32", 77, 0)])
@pytest.mark.parametrize("H,Hkv,dh", [(4, 4, 64), (8, 1, 128)])
def test_short_and_odd_contiguous_caches(kind, T, block, H, Hkv, dh):
    """Capacities below a tile and no multiple of anything: the last rows of a plane
    lie before the first of the next one, which no query sees."""
    for n in sorted({1, min(T, 3), min(T, 7), min(T, 40), min(T, 140)}):
        run_attention(kind, False, (T, max(T - 1, n), n, n // 2, 0), n, H, Hkv, dh, T, block, seed=n + T)
        run_attention(kind, False, (T, max(T - 1, n)), n, H, Hkv, dh, T, block, 9, 2, seed=n + T + 1)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 3, 12, 20, 60])
def test_negative_and_small_scales(kind, n):
    for scale in (-0.05, 1e-30, -1e-30):
        run_attention(kind, True, (150, 20), n, 4, 2, 64, 160, 32, 30, 5, (n, min(n, 20)), scale=scale, seed=n)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 12, 60, 200])
def test_zero_queries_over_zero_keys(kind, n):
    """All weights equal: the mean of what is seen.  e4m3: the smallest block scale."""
    tb = tbm()
    L, dh = 300, 64
    kv = make_cache(kind, False, 1, 2, 304, dh, 16)
    put_rows(kv, 0, torch.zeros(2, L, dh), rows(2, 2, L, dh))
    if kind == "e4m3":
        kv.k_scale.fill_(2.0 ** -24)
    kv.lens.fill_(L)
    q = torch.zeros(1, n, 4, dh, dtype=ROW[kind], device="cuda")
    cfg = tb.AttnConfig(H=4, Hkv=2, dh=dh, window=100, sinks=3, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    o = tb.tb_kvcache_attn(cfg, q, kv)[0].double().cpu().numpy()
    out, mag, top = ref.attend(q[0].double().cpu().numpy(), values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L], L - n, 100, 3)
    check_attention(kind, o, out, mag, top, dh, L)
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_many_sequences_of_many_rows(kind):
    """1300 short sequences of 20 tokens on the tensor-core kernel, lengths from nothing on."""
    tb = tbm()
    B, Hkv, H, dh, T, n = 1300, 1, 2, 64, 48, 20
    kv = make_cache(kind, False, B, Hkv, T, dh, 16, fill=0.0)
    g = torch.Generator().manual_seed(1)
    for x in (kv.k, kv.v):
        if kind == "e4m3":
            x.view(torch.uint8).copy_((torch.randn(x.shape, generator=g) * 100).to(torch.float8_e4m3fn).view(torch.uint8))
        else:
            x.copy_(torch.randn(x.shape, generator=g))
    if kind == "e4m3":
        kv.k_scale.fill_(2.0 ** -7)
        kv.v_scale.fill_(2.0 ** -7)
    kv.lens.copy_(torch.arange(B, dtype=torch.int32) % (T + 1))
    q = rows(3, B, n, H, dh, dtype=torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=H, Hkv=Hkv, dh=dh), q, kv).double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    for b in list(range(0, 52)) + list(range(700, 730)) + list(range(1270, 1300)):
        L = b % (T + 1)
        out, mag, top = ref.attend(q[b].double().cpu().numpy(), values(kv, "k", b)[:, :L], values(kv, "v", b)[:, :L], L - n)
        check_attention(kind, o[b], out, mag, top, dh, max(L, 1), f"sequence {b}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 7, 60])
def test_sequences_that_share_pages(kind, n):
    """A common prefix lies once in the pool and stands in both tables, a page even
    twice in one of them."""
    tb = tbm()
    H, Hkv, dh, ps, L = 8, 2, 128, 32, 256
    kv = make_cache(kind, True, 2, Hkv, L, dh, ps, fill=0.0)
    kv.block_table[1, :4] = kv.block_table[0, :4]
    kv.block_table[1, 5] = kv.block_table[1, 1]
    for b in (1, 0):
        put_rows(kv, b, rows(b, Hkv, L, dh), rows(b + 9, Hkv, L, dh))
    kv.lens.fill_(L)
    q = rows(3, 2, n, H, dh, dtype=torch.bfloat16).cuda()
    o = tb.tb_kvcache_attn(tb.AttnConfig(H=H, Hkv=Hkv, dh=dh), q, kv).double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    for b in range(2):
        out, mag, top = ref.attend(q[b].double().cpu().numpy(), values(kv, "k", b), values(kv, "v", b), L - n)
        check_attention(kind, o[b], out, mag, top, dh, L)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
def test_append_of_rows_that_repeat(kind):
    """Strides of 0: one row for all tokens, or one sequence's rows for all sequences."""
    tb = tbm()
    B, n, Hkv, dh, T, bs = 3, 9, 2, 64, 64, 16
    table = tb.tb_rope_table(dh, T, BASE)
    one = rows(1, 1, 1, Hkv, dh, dtype=ROW[kind]).cuda()
    seq = rows(2, 1, n, Hkv, dh, dtype=ROW[kind]).cuda()
    a, b = (make_cache(kind, True, B, Hkv, T, dh, bs, fill=0.0) for _ in range(2))
    tb.tb_kvcache_append_rope(a, one.expand(B, n, Hkv, dh), seq.expand(B, n, Hkv, dh), table, start=i32(0, 5, 55))
    tb.tb_kvcache_append_rope(b, one.expand(B, n, Hkv, dh).contiguous(), seq.expand(B, n, Hkv, dh).contiguous(), table,
                              start=i32(0, 5, 55))
    assert a.lens.tolist() == b.lens.tolist() == [9, 14, 64] and tb.tb_get_device_error(clear=True) == 0
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_calls_with_nothing_to_do():
    tb = tbm()
    kv = make_cache("bf16", False, 2, 2, 64, 64, 0, fill=0.0)
    kv.lens.fill_(5)
    e = lambda B, n, h: torch.empty(B, n, h, 64, dtype=torch.bfloat16, device="cuda")
    cfg = tb.AttnConfig(H=4, Hkv=2, dh=64)
    table = tb.tb_rope_table(64, 64, BASE)
    assert tb.tb_kvcache_append_rope(kv, e(2, 0, 2), e(2, 0, 2), table, q=e(2, 0, 4)).shape == (2, 0, 4, 64)
    assert tb.tb_kvcache_attn(cfg, e(2, 0, 4), kv).shape == (2, 0, 4, 64)
    none = tb.KVCache.empty(0, 2, 64, 64)
    assert tb.tb_kvcache_append_rope(none, e(0, 3, 2), e(0, 3, 2), table) is None
    assert tb.tb_kvcache_attn(cfg, e(0, 3, 4), none).shape == (0, 3, 4, 64)
    assert kv.lens.tolist() == [5, 5] and tb.tb_get_device_error(clear=True) == 0


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [8, 512])
def test_zero_rows_cost_what_others_do(kind, n):
    """Rows of zeros at the end of a cache, as a padded batch has them, are not
    computed key by key (which takes some hundred times as long; ten is the bound
    here, for the noise of a clock)."""
    tb = tbm()
    H, Hkv, dh, T = 16, 4, 128, 2048
    row = ROW[kind]
    kv = make_cache(kind, False, 1, Hkv, T, dh, 64, fill=0.0)
    table = tb.tb_rope_table(dh, T, BASE)
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh, dtype=tb.TB_F32 if kind == "f32" else tb.TB_BF16)
    took = []
    for zeros in (False, True):
        x, q = rows(1, 1, T, Hkv, dh, dtype=row).cuda(), rows(2, 1, n, H, dh, dtype=row).cuda()
        if zeros:
            x[:, -n:] = 0
            q.zero_()
        tb.tb_kvcache_append_rope(kv, x, x, table, start=i32(0))
        best = math.inf
        for _ in range(6):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            o = tb.tb_kvcache_attn(cfg, q, kv)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        took.append(best)
    assert torch.isfinite(o).all() and tb.tb_get_device_error(clear=True) == 0
    assert took[1] <= 10 * took[0], took

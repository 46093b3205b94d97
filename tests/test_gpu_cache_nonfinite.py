"""tb_kvcache_attn over caches and queries that hold infinities and NaN: what a
query sees reaches it as IEEE arithmetic says, what it does not see never does."""
import math

import numpy as np
import pytest
import torch

import oracle.cache as ref
from cache_helpers import ROW, attn_tolerance, make_cache, put_rows, rows, values

pytestmark = pytest.mark.gpu


def tbm():
    import causal_gqa_attention_rmsnorm_gb300 as tb
    return tb


def filled(kind, L, Hkv, dh, T, block=16, paged=True):
    kv = make_cache(kind, paged, 1, Hkv, T, dh, block, fill=float("nan"))
    put_rows(kv, 0, rows(1, Hkv, L, dh), rows(2, Hkv, L, dh))
    kv.lens.fill_(L)
    return kv


def poke(kv, name, h, t, d, x):
    """Element (KV head h, token t, dim d) of a one-sequence cache becomes x (e4m3: a code)."""
    buf = getattr(kv, name)
    e4m3 = buf.dtype == torch.float8_e4m3fn
    buf = buf.view(torch.uint8) if e4m3 else buf
    at = (0, h, t, d) if kv.block_table is None else (int(kv.block_table[0, t // buf.shape[2]]), h, t % buf.shape[2], d)
    buf[at] = x


def attend(kv, q, window=0, sinks=0):
    tb = tbm()
    H, dh = q.shape[2:]
    cfg = tb.AttnConfig(H=H, Hkv=kv.k.shape[1], dh=dh, window=window, sinks=sinks,
                        dtype=tb.TB_F32 if q.dtype == torch.float32 else tb.TB_BF16)
    o = tb.tb_kvcache_attn(cfg, q, kv)[0].double().cpu().numpy()
    assert tb.tb_get_device_error(clear=True) == 0
    return o


def expect(q, k, v, first, window=0, sinks=0):
    """The formula in 64 bits with the infinities and NaN of its inputs, and the
    same with the keys of an infinite or NaN score left out, for tolerances.  q [m,
    H, dh], k and v [Hkv, L, dh]."""
    m, H, dh = q.shape
    Hkv, L, _ = k.shape
    out, mag, top = np.zeros((m, H, dh)), np.zeros((m, H, dh)), np.zeros((m, H))
    with np.errstate(all="ignore"):
        for i in range(m):
            see = ref.visible(first + i, L, window, sinks)
            for h in range(H):
                kk, vv = k[h // (H // Hkv)][see], v[h // (H // Hkv)][see]
                if not see.any():
                    continue
                z = kk @ q[i, h] / np.sqrt(dh)
                w = np.exp(z - z.max())
                w /= w.sum()
                out[i, h] = w @ vv
                ok = np.isfinite(z)
                mag[i, h] = w[ok] @ np.abs(vv[ok]) if ok.any() else 0
                top[i, h] = (np.abs(kk[ok]) @ np.abs(q[i, h])).max() / np.sqrt(dh) if ok.any() else 0
    return out, mag, top


def same(kind, got, out, mag, top, dh, nkeys):
    """NaN and infinities in the same places, the rest within its bound."""
    wrong = int((np.isnan(got) != np.isnan(out)).sum())
    assert wrong == 0, f"{wrong} of {out.size} NaN where no NaN belongs, or none where one does"
    inf = np.isinf(out)
    wrong = int((np.isinf(got) != inf).sum() + (got[inf] != out[inf]).sum())
    assert wrong == 0, f"{wrong} infinities"
    fine = np.isfinite(out)
    with np.errstate(all="ignore"):
        tol = attn_tolerance(kind, out, mag, top, dh, nkeys)
        off = int((np.abs(got - out) > tol)[fine].sum())
    assert off == 0, f"{off} of {int(fine.sum())} finite outputs off"


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n,L", [(40, 129), (40, 257), (129, 129)])
def test_a_piece_of_one_nan_score_is_joined(kind, dh, n, L):
    """The last key is alone in its key tile and its score is NaN: the piece of
    that tile has no finite score, but the last query sees it."""
    kv = filled(kind, L, 1, dh, 272)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    poke(kv, "k", 0, L - 1, 5, 0x7F if kind == "e4m3" else math.nan)
    k[0, L - 1, 5] = math.nan
    q = rows(5, 1, n, 1, dh, dtype=torch.bfloat16).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n)
    assert np.isnan(want[0][-1]).all() and np.isfinite(want[0][:-1]).all()
    same(kind, attend(kv, q), *want, dh, L)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n,L", [(40, 129), (40, 257), (129, 129)])
def test_a_piece_of_one_weightless_infinity_is_joined(dh, n, L):
    """The last key is alone in its key tile, its score is -inf and its value
    infinite: 0 times infinity is NaN for the query that sees it."""
    kv = filled("bf16", L, 1, dh, 272)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    poke(kv, "k", 0, L - 1, 5, -math.inf)
    poke(kv, "v", 0, L - 1, 7, math.inf)
    k[0, L - 1, 5], v[0, L - 1, 7] = -math.inf, math.inf
    q = rows(5, 1, n, 1, dh)
    q[..., 5] = 1
    q = q.to(torch.bfloat16).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n)
    assert np.isnan(want[0][-1, 0, 7]) and np.isfinite(np.delete(want[0][-1, 0], 7)).all()
    same("bf16", attend(kv, q), *want, dh, L)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n,L,H,Hkv", [(1, 1, 4, 1), (3, 3, 2, 2), (8, 8, 8, 2), (12, 12, 4, 2), (40, 40, 2, 2),
                                      (200, 200, 4, 2), (3, 2, 4, 2), (40, 38, 2, 1), (6, 700, 4, 2), (150, 700, 4, 2)])
def test_scores_that_are_all_minus_infinity_give_nan(kind, dh, n, L, H, Hkv):
    """Key 0 of KV head 0 scores -inf, and so do all keys of KV head 1 (where there
    is one): NaN where a query sees nothing else, a weight of 0 beside other keys,
    zeros at negative positions all the same."""
    T = -(-L // 16) * 16
    kv = filled(kind, L, Hkv, dh, T)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    poke(kv, "k", 0, 0, 5, -math.inf)
    k[0, 0, 5] = -math.inf
    if Hkv > 1:
        for t in range(L):
            poke(kv, "k", 1, t, 5, -math.inf)
        k[1, :, 5] = -math.inf
    q = rows(5, 1, n, H, dh)
    q[..., 5] = 1
    q = q.to(ROW[kind]).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n)
    at0 = n - L                                           # the query at position 0
    if at0 >= 0:
        assert np.isnan(want[0][at0]).all() and (want[0][:at0] == 0).all()
    assert np.isfinite(want[0][max(at0 + 1, 0):, :H // Hkv]).all()
    same(kind, attend(kv, q), *want, dh, L)


@pytest.mark.parametrize("n,L", [(1, 1), (1, 300), (8, 300), (40, 300), (200, 300), (3, 2)])
def test_an_infinite_query_over_e4m3_gives_nan(n, L):
    """A query with an infinite element against keys whose element is negative:
    every score -inf."""
    kv = filled("e4m3", L, 2, 64, 304)
    for t in range(L):
        for h in range(2):
            poke(kv, "k", h, t, 5, 0xB8)                  # -1
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    assert (k[:, :, 5] < 0).all()
    q = rows(5, 1, n, 4, 64)
    q[:, -1, 1, 5] = math.inf
    q[:, -1, 2, 5] = -math.inf
    q = q.to(torch.bfloat16).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n)
    assert np.isnan(want[0][-1, 1:3]).all() and np.isfinite(want[0][-1, ::3]).all()
    same("e4m3", attend(kv, q), *want, 64, L)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 4, 12, 40, 200])
@pytest.mark.parametrize("dh", [64, 128])
def test_a_nan_key_reaches_the_queries_that_see_it(kind, n, dh):
    """NaN in the K of a row that leaves the window inside the call, of the last row
    and of a sink: each seen by some queries, or heads, and not by others."""
    L, W, S, H, Hkv = 400, 64, 3, 8, 4
    kv = filled(kind, L, Hkv, dh, 416)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    leaves = L - n - W + 1 + n // 2
    for h, t in ((0, leaves), (1, L - 1), (2, 1)):
        poke(kv, "k", h, t, 5, 0x7F if kind == "e4m3" else math.nan)
        k[h, t, 5] = math.nan
    q = rows(5, 1, n, H, dh, dtype=ROW[kind]).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n, W, S)
    nan = np.isnan(want[0]).all(-1)
    assert np.array_equal(nan, np.isnan(want[0]).any(-1))
    assert nan[:, 4:6].all() and not nan[:, 6:].any() and nan[:, :2].any() and (n == 1 or not nan[:, :2].all())
    assert nan[-1, 2:4].all() and not nan[:-1, 2:4].any()
    same(kind, attend(kv, q, W, S), *want, dh, L)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 4, 12, 40, 200])
@pytest.mark.parametrize("window", [0, 64])
def test_infinities_in_the_cache(kind, n, window):
    """In K: a score of +inf is NaN for its query, one of -inf a weight of 0.  In V:
    an infinity for the queries that give the row a weight, NaN beside a second one
    of the other sign."""
    L, S, H, Hkv, dh = 400, 0, 8, 4, 64
    kv = filled(kind, L, Hkv, dh, 416)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    t = L - n - 5                                          # inside the window of the first queries
    for name, x, h, at, d, val in (("k", k, 0, t, 5, math.inf), ("k", k, 1, t, 5, -math.inf),
                                   ("v", v, 2, t, 6, math.inf), ("v", v, 2, t + 1, 7, -math.inf),
                                   ("v", v, 3, t, 8, math.inf), ("v", v, 3, t + 2, 8, -math.inf)):
        poke(kv, name, h, at, d, val)
        x[h, at, d] = val
    q = rows(5, 1, n, H, dh)
    q[..., 5] = 1
    q = q.to(ROW[kind]).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n, window, S)
    assert np.isnan(want[0][0, :2]).all() and np.isfinite(want[0][:, 2:4]).all()
    assert np.isinf(want[0][0, 4:6, 6:8]).all() and np.isnan(want[0][0, 6:, 8]).all()
    same(kind, attend(kv, q, window, S), *want, dh, L)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 12, 40])
def test_infinite_and_nan_queries_stay_alone(kind, n):
    """A query row of infinities or NaN is NaN itself; the rows beside it are not."""
    L, H, Hkv, dh = 300, 8, 2, 64
    kv = filled(kind, L, Hkv, dh, 304)
    k, v = values(kv, "k", 0)[:, :L], values(kv, "v", 0)[:, :L]
    q = rows(5, 1, n, H, dh)
    q[0, -1, 1, 5], q[0, -1, 6, 9], q[0, 0, 3, :] = math.inf, math.nan, -math.inf
    q = q.to(ROW[kind]).cuda()
    want = expect(q[0].double().cpu().numpy(), k, v, L - n)
    bad = np.zeros((n, H), dtype=bool)
    bad[-1, 1] = bad[-1, 6] = bad[0, 3] = True
    assert np.array_equal(np.isnan(want[0]).all(-1), bad)
    same(kind, attend(kv, q), *want, dh, L)

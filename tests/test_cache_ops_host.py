"""Host side of the cache operators, without a GPU: what their C entry points
refuse before they launch anything, empty calls, and the oracle's own pins."""
import ctypes

import numpy as np
import pytest

import causal_gqa_attention_rmsnorm_gb300 as tb
import oracle
import oracle.cache as ref
from causal_gqa_attention_rmsnorm_gb300 import binding

FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def cache(**k):
    d = dict(k=FAKE, v=FAKE, lens=FAKE, B=2, Hkv=2, T=256, dh=64, dtype=tb.TB_BF16, bt=None, ps=0, pages=0, ks=None,
             vs=None)
    d.update(k)
    return binding.tb_kvcache(d["k"], d["v"], d["lens"], d["B"], d["Hkv"], d["T"], d["dh"], d["dtype"], d["bt"],
                              d["ps"], d["pages"], d["ks"], d["vs"])


def e4m3(**k):
    return cache(**{**dict(dtype=tb.TB_E4M3, ps=32, ks=FAKE, vs=FAKE), **k})


def append(lib, kv, rope=FAKE, max_pos=256, **k):
    d = dict(q=FAKE, k=FAKE + (1 << 20), v=FAKE + (1 << 21), q_out=FAKE + (1 << 22), q_tok=256, q_seq=256, k_tok=128, k_seq=128, v_tok=128,
             v_seq=128, H=4, n=1, start=None, n_new=None)
    d.update(k)
    rows = binding.tb_append_rows(*[d[n] for n, _ in binding.tb_append_rows._fields_])
    return lib.tb_kvcache_append_rope(None if kv is None else ctypes.byref(kv), ctypes.byref(rows), rope, max_pos, None)


BAD_CACHES = [
    (dict(dtype=tb.TB_I8), 2), (dict(dtype=9), 1), (dict(dh=24), 2), (dict(dh=512), 2), (dict(T=0), 1), (dict(Hkv=0), 1),
    (dict(B=-1), 1), (dict(B=40000), 2), (dict(k=None), 1), (dict(lens=None), 1), (dict(v=FAKE + 8), 1),
    (dict(bt=FAKE, ps=24, pages=9), 1), (dict(bt=FAKE, ps=96, pages=9), 1), (dict(bt=FAKE, ps=32, pages=0), 1),
    (dict(bt=FAKE + 2, ps=32, pages=9), 1),
    (dict(dtype=tb.TB_E4M3, ps=32, ks=FAKE), 1), (dict(dtype=tb.TB_E4M3, ps=8, ks=FAKE, vs=FAKE), 1),
    (dict(dtype=tb.TB_E4M3, ps=0, ks=FAKE, vs=FAKE), 1), (dict(dtype=tb.TB_E4M3, ps=32, ks=FAKE + 2, vs=FAKE), 1),
]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_both_calls_refuse_the_cache(lib, bad, status):
    kv = cache(**bad)
    assert append(lib, kv) == status, lib.tb_last_error_message()
    cfg = binding.tb_attn_cfg(4, kv.Hkv or 2, kv.dh, tb.TB_BF16, 0, 0, 0.0)
    got = lib.tb_kvcache_attn(ctypes.byref(cfg), FAKE, ctypes.byref(kv), None, 1, FAKE, FAKE, 1 << 40, None)
    assert got != 0, lib.tb_last_error_message()


def test_append_refusals(lib):
    assert append(lib, None) == 1
    assert append(lib, cache(), n=-1) == 1
    assert append(lib, cache(), n=257) == 1                      # more rows than T_max
    assert append(lib, cache(), max_pos=255) == 1                # table shorter than the cache
    assert append(lib, cache(), rope=None) == 1
    assert append(lib, cache(), rope=FAKE + 8) == 1
    assert append(lib, cache(), k=None) == 1
    assert append(lib, cache(), q=None) == 1                     # q_out without q
    assert append(lib, cache(), q_out=None) == 1
    assert append(lib, cache(), H=0) == 1
    assert append(lib, cache(), H=65536, q_tok=65536 * 64, q_seq=65536 * 64 * 4) == 2
    assert append(lib, cache(), v=FAKE + 2) == 1
    assert append(lib, cache(), k_tok=132) == 1                  # stride not a multiple of 8
    assert append(lib, cache(), v_seq=-128) == 1
    assert append(lib, cache(), q_out=FAKE, q_seq=512) == 1      # in place, but q not dense
    assert append(lib, cache(), q_out=FAKE + 16) == 1            # overlapping q
    assert append(lib, cache(), q_out=FAKE + (1 << 20) + 16) == 1 and b"overlaps k" in lib.tb_last_error_message()
    assert append(lib, cache(), n_new=FAKE + 4) == 1             # overlapping lens
    assert append(lib, cache(), start=FAKE) == 1                 # start is lens
    assert append(lib, cache(), start=FAKE + 4) == 1             # and overlapping it
    assert b"overlap" in lib.tb_last_error_message()
    assert append(lib, cache(), n_new=FAKE + 1) == 1
    # nothing to do
    assert append(lib, cache(), n=0) == 0
    assert append(lib, cache(B=0, k=None, v=None, lens=None)) == 0


def test_attention_refusals(lib):
    def call(cfg=None, kv=None, n=1, q=FAKE, o=FAKE + (1 << 40), ws=FAKE, wsb=1 << 40, n_new=None):
        d = dict(H=4, Hkv=2, dh=64, dtype=tb.TB_BF16, window=0, sinks=0, scale=0.0)
        d.update(cfg or {})
        c = binding.tb_attn_cfg(*[d[n] for n, _ in binding.tb_attn_cfg._fields_])
        kv = kv or cache()
        return lib.tb_kvcache_attn(ctypes.byref(c), q, ctypes.byref(kv), n_new, n, o, ws, wsb, None)
    assert lib.tb_kvcache_attn(None, FAKE, ctypes.byref(cache()), None, 1, FAKE, FAKE, 1 << 40, None) == 1
    assert call(dict(H=5)) == 1
    assert call(dict(H=6)) == 2                                  # three query heads per KV head
    assert call(dict(Hkv=4)) == 1                                # not the cache's
    assert call(dict(dh=128)) == 1
    assert call(dict(dtype=tb.TB_F32)) == 1                      # fp32 queries over a bf16 cache
    assert call(dict(dtype=7)) == 1
    assert call(dict(window=-1)) == 1 and call(dict(sinks=-1)) == 1
    assert call(dict(scale=float("nan"))) == 1
    assert call(dict(dh=32), cache(dh=32)) == 2                  # bf16 of a width without a kernel
    assert call(dict(dtype=tb.TB_F32), cache(dtype=tb.TB_BF16)) == 1
    assert call(kv=e4m3(), cfg=dict(dtype=tb.TB_F32)) == 1
    assert call(n=-1) == 1 and call(n=257) == 1
    assert call(q=None) == 1 and call(o=None) == 1 and call(q=FAKE + 8) == 1 and call(n_new=FAKE + 2) == 1
    assert call(dict(H=4, Hkv=2), cache(B=32767, T=1 << 20), n=1 << 20) == 2   # too many rows
    assert call(o=FAKE) == 1 and call(o=FAKE + 16) == 1 and b"overlap" in lib.tb_last_error_message()
    assert call(n=0) == 0 and call(kv=cache(B=0, k=None, v=None, lens=None)) == 0


def test_attention_workspace_is_checked(lib):
    c = binding.tb_attn_cfg(32, 8, 128, tb.TB_BF16, 0, 0, 0.0)
    kv = cache(B=1, Hkv=8, T=65536, dh=128)
    need = lib.tb_kvcache_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(kv), 1)
    bad = binding.tb_attn_cfg(32, 8, 128, tb.TB_BF16, -1, 0, 0.0)
    assert lib.tb_kvcache_attn_workspace_bytes(ctypes.byref(bad), ctypes.byref(kv), 1) == 0
    if need:
        for ws, wsb in ((None, need), (FAKE, need - 1), (FAKE + 128, need)):
            assert lib.tb_kvcache_attn(ctypes.byref(c), FAKE, ctypes.byref(kv), None, 1, FAKE, ws, wsb, None) == 1


def test_the_blocks_calls_take_no_e4m3_cache(lib):
    kv = e4m3()
    assert lib.tb_kvcache_append(ctypes.byref(kv), FAKE, FAKE, 1, None) == 1
    c = binding.BlockConfig(d=128, H=2, Hkv=2, dh=64, f=256, max_pos=256, rope_base=1e4, eps=1e-6, dtype=tb.TB_BF16).c()
    y = FAKE + (1 << 30)
    assert lib.tb_block_decode(ctypes.byref(c), FAKE, FAKE, y, tb.TB_F32, ctypes.byref(kv), FAKE, 1 << 40, None) == 1
    assert lib.tb_block_prefill(ctypes.byref(c), FAKE, FAKE, y, tb.TB_F32, 2, 16, ctypes.byref(kv), FAKE, 1 << 40, None) == 1


@pytest.mark.parametrize("dtype", [tb.TB_F32, tb.TB_BF16, tb.TB_E4M3])
@pytest.mark.parametrize("H,Hkv,B,T,window", [(32, 8, 1, 65536, 0), (8, 8, 40, 4096, 0), (16, 2, 3, 2048, 300), (4, 4, 900, 512, 0)])
def test_a_workspace_holds_for_fewer_tokens(lib, dtype, H, Hkv, B, T, window):
    c = binding.tb_attn_cfg(H, Hkv, 128, tb.TB_F32 if dtype == tb.TB_F32 else tb.TB_BF16, window, 4, 0.0)
    kv = cache(B=B, Hkv=Hkv, T=T, dh=128, dtype=dtype, ps=32, ks=FAKE, vs=FAKE)
    need = [lib.tb_kvcache_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(kv), n) for n in range(0, 200)]
    assert need == sorted(need) and need[0] == 0


def test_rope_table_refusals(lib):
    assert lib.tb_rope_table(63, 8, 1e4, FAKE, None) == 1
    assert lib.tb_rope_table(64, -1, 1e4, FAKE, None) == 1
    assert lib.tb_rope_table(64, 8, 0.0, FAKE, None) == 1
    assert lib.tb_rope_table(64, 8, 1e4, None, None) == 1
    assert lib.tb_rope_table(64, 8, 1e4, FAKE + 4, None) == 1
    assert lib.tb_rope_table(64, 0, 1e4, None, None) == 0


# ---- the oracle ---------------------------------------------------------------

def test_oracle_attention_of_all_rows_is_the_blocks():
    """Every row of a sequence at once, without and with a window, against the block oracle's attention."""
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(9, 4, 16)), r.normal(size=(2, 9, 16)), r.normal(size=(2, 9, 16))
    for w in (0, 3):
        got, mag, top = ref.attend(q, k, v, 0, w)
        for h in range(4):
            for i in range(9):
                see = [j for j in range(9) if j <= i and (w == 0 or j > i - w)]
                z = np.array([q[i, h] @ k[h // 2][j] / 4 for j in see])
                p = np.exp(z - z.max()) / np.exp(z - z.max()).sum()
                want = sum(a * v[h // 2][j] for a, j in zip(p, see))
                assert np.allclose(got[i, h], want, rtol=1e-12)
        assert (mag >= np.abs(got) - 1e-12).all() and (top > 0).all()


def test_oracle_sinks_and_empty_rows():
    assert ref.visible(10, 12, 3, 2).nonzero()[0].tolist() == [0, 1, 8, 9, 10]
    assert ref.visible(1, 12, 3, 5).nonzero()[0].tolist() == [0, 1]       # a sink ahead of the query stays hidden
    assert not ref.visible(-1, 12, 3, 5).any()
    out, _, _ = ref.attend(np.ones((2, 1, 4)), np.ones((1, 3, 4)), np.ones((1, 3, 4)), -1)
    assert (out[0] == 0).all() and np.allclose(out[1], 1)


def test_oracle_scale_is_the_smallest_that_holds():
    for top in (448.0, 448.0001, 1.0, 3.5, 7e-5, 5e18):
        s = ref.e4m3_scale(top)
        assert top <= 448 * s and top > 224 * s
    assert ref.e4m3_scale(0.0) == 2.0 ** -24 and ref.e4m3_scale(1e38) == 2.0 ** 60 and ref.e4m3_scale(1e-30) == 2.0 ** -24


def test_oracle_rotation_is_the_blocks():
    x = np.random.default_rng(2).normal(size=(3, 2, 8))
    assert np.array_equal(ref.rotated(x, 5, 1e4), oracle.rope(x, [5, 6, 7], 1e4))

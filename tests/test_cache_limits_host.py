"""Refusals of the cache operators, on the host and before anything is launched: sizes
at which their 32-bit counts would run over, caches and workspaces that do not do."""
import ctypes

import pytest

import causal_gqa_attention_rmsnorm_gb300 as tb
from causal_gqa_attention_rmsnorm_gb300 import binding
from test_cache_ops_host import BAD_CACHES, FAKE, append, cache, e4m3


@pytest.fixture(scope="module")
def lib():
    return binding.lib()


def attn(lib, kv, n=1, G=1, **k):
    """Status of a call that has nothing wrong beside its sizes."""
    c = binding.tb_attn_cfg(kv.Hkv * G, kv.Hkv, kv.dh, tb.TB_F32 if kv.dtype == tb.TB_F32 else tb.TB_BF16,
                            k.get("window", 0), k.get("sinks", 0), k.get("scale", 0.0))
    return lib.tb_kvcache_attn(ctypes.byref(c), FAKE, ctypes.byref(kv), None, n, FAKE + (1 << 45), None, 0, None)


def need(lib, kv, n=1, G=1, window=0, sinks=0):
    c = binding.tb_attn_cfg(kv.Hkv * G, kv.Hkv, kv.dh, tb.TB_F32 if kv.dtype == tb.TB_F32 else tb.TB_BF16, window,
                            sinks, 0.0)
    return lib.tb_kvcache_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(kv), n)


def many_pages(Hkv, T, dtype=tb.TB_BF16, dh=128):
    """A page may stand in the table more than once, so long sequences of many heads need no memory."""
    return cache(B=1, Hkv=Hkv, T=T, dh=dh, dtype=dtype, bt=FAKE, ps=32, pages=9, ks=FAKE, vs=FAKE)


@pytest.mark.parametrize("dtype", [tb.TB_BF16, tb.TB_E4M3])
def test_stages_of_one_sequence_are_counted_in_32_bits(lib, dtype):
    big = many_pages(65535, 600000, dtype)                # 65535 heads x 37501 runs: above 2^31
    assert attn(lib, big) == 2 and b"2^30" in lib.tb_last_error_message()
    assert need(lib, big) == 0
    assert attn(lib, many_pages(32768, 32 * 20000, dtype), G=8, n=4) == 2
    # what can be counted is not refused: fewer heads, a window, and the tensor-core kernel's 64-bit line
    assert need(lib, many_pages(1024, 600000, dtype)) > 0
    assert need(lib, big, window=1000, sinks=4) > 0
    assert need(lib, many_pages(1024, 600000, dtype), n=64) > 0


@pytest.mark.parametrize("dtype", [tb.TB_F32, tb.TB_BF16, tb.TB_E4M3])
@pytest.mark.parametrize("n", [1, 64])
def test_positions_leave_room_for_a_whole_tile(lib, dtype, n):
    """A position rounded up to a tile of keys stays a 32-bit number."""
    for T in (2 ** 31 - 32, 2 ** 31 - 256 + 32):
        assert attn(lib, many_pages(1, T, dtype), n=n) == 2 and b"T_max" in lib.tb_last_error_message()
    assert need(lib, many_pages(1, 2 ** 31 - 512, dtype), n=n) > 0


def test_pieces_of_an_e4m3_block_are_counted_in_32_bits(lib):
    """2^24 tokens of 256 elements are 2^29 pieces; far larger blocks ran over, and
    their older codes were not rewritten for a new scale."""
    for block in (1 << 25, 1 << 27, (1 << 31) - 16):
        kv = e4m3(B=1, Hkv=1, T=block, dh=128, ps=block)
        assert append(lib, kv, max_pos=block) == 2 and b"2^24" in lib.tb_last_error_message()
        # reading such a block has no such count
        assert need(lib, e4m3(B=1, Hkv=1, T=1 << 27, dh=128, ps=1 << 27)) > 0
    # (a block of 2^24 gets as far as the next check)
    assert append(lib, e4m3(B=1, Hkv=1, T=1 << 24, dh=128, ps=1 << 24), max_pos=16) == 1


@pytest.mark.parametrize("dtype", [tb.TB_F32, tb.TB_BF16, tb.TB_E4M3])
def test_the_scale_times_log2_e_is_finite(lib, dtype):
    kv = e4m3(dtype=dtype)
    for scale in (3e38, -3e38, float("inf")):
        assert attn(lib, kv, scale=scale) == 1 and b"scale" in lib.tb_last_error_message()
    for scale in (2.0 ** 127, -2.0 ** 127, 1e-45):
        c = binding.tb_attn_cfg(2, 2, 64, tb.TB_F32 if dtype == tb.TB_F32 else tb.TB_BF16, 0, 0, scale)
        assert lib.tb_kvcache_attn(ctypes.byref(c), FAKE, ctypes.byref(kv), None, 0, FAKE, None, 0, None) == 0


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_the_attention_refuses_the_cache_for_the_reason_the_append_gives(lib, bad, status):
    """q, o, ws and cfg are right, so that only the cache can be refused."""
    kv = cache(**bad)
    assert append(lib, kv) == status
    why = lib.tb_last_error_message()
    c = binding.tb_attn_cfg(4, kv.Hkv or 2, kv.dh, tb.TB_BF16, 0, 0, 0.0)
    assert lib.tb_kvcache_attn(ctypes.byref(c), FAKE, ctypes.byref(kv), None, 1, FAKE + (1 << 40), FAKE, 1 << 40, None) == status
    assert lib.tb_last_error_message() == why


@pytest.mark.parametrize("kv,n,H", [
    (cache(B=1, Hkv=8, T=65536, dh=128), 1, 32),                               # streaming kernel
    (cache(B=1, Hkv=8, T=65536, dh=128), 64, 32),                              # tensor-core kernel
    (e4m3(B=3, Hkv=8, T=4096, dh=64), 7, 32),
])
def test_a_workspace_that_does_not_do_is_named(lib, kv, n, H):
    dtype = tb.TB_F32 if kv.dtype == tb.TB_F32 else tb.TB_BF16
    c = binding.tb_attn_cfg(H, kv.Hkv, kv.dh, dtype, 0, 0, 0.0)
    bytes_ = lib.tb_kvcache_attn_workspace_bytes(ctypes.byref(c), ctypes.byref(kv), n)
    assert bytes_ > 0
    for ws, have in ((None, bytes_), (FAKE, bytes_ // 2), (FAKE + 128, bytes_), (FAKE, 0)):
        status = lib.tb_kvcache_attn(ctypes.byref(c), FAKE, ctypes.byref(kv), None, n, FAKE + (1 << 45), ws, have, None)
        assert status == 1 and b"ws must be" in lib.tb_last_error_message()

"""The 8-bit projections without a GPU: what the C entry points and the binding refuse,
and the oracle's own pins."""
import ctypes
import os

import numpy as np
import pytest
import torch

import causal_gqa_attention_rmsnorm_gb300 as tb
from causal_gqa_attention_rmsnorm_gb300 import binding
from oracle import e4m3 as ref

BASE = 0x7F0000000000        # never dereferenced: every call below fails validation first
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libtb.so not built")
    return binding.lib()


def at(i):
    """Places far apart."""
    return BASE + i * (1 << 30)


def mat(rows, cols, codes=at(20), scale=at(21)):
    return ctypes.byref(binding.tb_e4m3(codes, scale, rows, cols))


def refused(lib, status, text, want=1):
    msg = lib.tb_last_error_message().decode()
    assert status == want and text in msg, (status, msg)


def norm(lib, x=at(1), dtype=1, r=None, r_dtype=1, h=None, g=at(4), eps=1e-5, out=None):
    return lib.tb_rmsnorm_e4m3(x, dtype, r, r_dtype, h, g, eps, mat(4, 256) if out is None else out, None)


@pytest.mark.parametrize("kw,text,status", [
    (dict(x=None), "x must be", 1), (dict(x=at(1) + 8), "x must be", 1), (dict(g=at(4) + 2), "g must be", 1),
    (dict(g=None), "g must be", 1), (dict(dtype=2), "unknown dtype", 1), (dict(dtype=3), "unknown dtype", 1),
    (dict(eps=-1e-5), "eps", 1), (dict(eps=float("nan")), "eps", 1), (dict(eps=float("inf")), "eps", 1),
    (dict(r=at(2)), "r and h go together", 1), (dict(h=at(3)), "r and h go together", 1),
    (dict(r=at(2), h=at(3), r_dtype=7), "unknown r_dtype", 1),
    (dict(r=at(2) + 4, h=at(3)), "r must be", 1), (dict(r=at(2), h=at(3) + 2), "h must be", 1),
    (dict(r=at(2), h=at(1) + 16), "h overlaps", 1), (dict(r=at(2), h=at(2), r_dtype=0), "h overlaps", 1),
    (dict(r=at(2), h=at(2) + 32), "h overlaps", 1), (dict(r=at(2), h=at(4)), "h overlaps", 1),
    (dict(x=at(20)), "an output overlaps", 1), (dict(g=at(21)), "an output overlaps", 1),
    (dict(r=at(2), h=at(20) + 16), "an output overlaps", 1), (dict(r=at(21), h=at(3)), "an output overlaps", 1),
])
def test_norm_refusals(lib, kw, text, status):
    refused(lib, norm(lib, **kw), text, status)


@pytest.mark.parametrize("m,text,status", [
    ((4, 0), "cols must be positive", 1), ((-1, 16), "rows non-negative", 1), ((4, 24), "multiple of 16", 2),
    ((4, 32784), "at most 32768", 2), ((2 ** 30, 1024), "2^39", 2), ((2 ** 31 - 1, 16), "2^31 - 1024", 2),
    ((2, 2 ** 31 - 16), "2^31 - 1024", 2), ((4, 256, None), "non-NULL", 1),
    ((4, 256, at(20), None), "non-NULL", 1), ((4, 256, at(20) + 8), "codes must be 16-byte", 1),
    ((4, 256, at(20), at(20) + 100), "two outputs overlap", 1),
])
def test_out_refusals(lib, m, text, status):
    refused(lib, norm(lib, out=mat(*m)), text, status)
    if "32768" not in text:
        refused(lib, lib.tb_quant_e4m3(at(1), 1, mat(*m), None), text, status)
        refused(lib, lib.tb_pack_e4m3(at(1), 1, mat(*m), None), text, status)


def test_quant_of_too_wide_rows(lib):
    refused(lib, lib.tb_quant_e4m3(at(1), 1, mat(1, 2 ** 26 + 16), None), "2^26 columns", 2)


def test_null_structs(lib):
    refused(lib, lib.tb_quant_e4m3(at(1), 1, None, None), "out is NULL")
    refused(lib, lib.tb_gemm_e4m3(None, mat(16, 16), None, at(1), 1, None), "x is NULL")
    refused(lib, lib.tb_gemm_e4m3(mat(16, 16), None, None, at(1), 1, None), "w is NULL")
    refused(lib, lib.tb_gated_e4m3(mat(16, 16), mat(16, 16), None, at(1), 1, None, None), "w3 is NULL")


W = dict(codes=at(10), scale=at(11))


@pytest.mark.parametrize("x,w,res,y,dtype,text,status", [
    (mat(4, 256), mat(32, 272, **W), None, at(1), 1, "columns", 1),
    (mat(4, 256), mat(0, 256, **W), None, at(1), 1, "rows must be positive", 1),
    (mat(4, 256), mat(40, 256, **W), None, at(1), 1, "multiple of 16", 2),
    (mat(4, 256), mat(2 ** 28 + 16, 256, **W), None, at(1), 1, "2^28 rows", 2),
    (mat(4, 256), mat(32, 256, **W), None, at(1), 3, "unknown y_dtype", 1),
    (mat(4, 256), mat(32, 256, **W), None, None, 1, "y must be", 1),
    (mat(4, 256), mat(32, 256, **W), None, at(1) + 8, 1, "y must be", 1),
    (mat(4, 256), mat(32, 256, **W), at(2) + 8, at(1), 1, "res must be", 1),
    (mat(4, 256), mat(32, 256, **W), at(1) + 16, at(1), 1, "y overlaps res", 1),
    (mat(4, 256), mat(32, 256, **W), None, at(20) + 1008, 1, "an output overlaps", 1),
    (mat(4, 256), mat(32, 256, **W), None, at(21), 1, "an output overlaps", 1),
    (mat(4, 256), mat(32, 256, **W), None, at(10), 0, "an output overlaps", 1),
    (mat(4, 256), mat(32, 256, **W), None, at(11), 0, "an output overlaps", 1),
    (mat(4, 256, None), mat(32, 256, **W), None, at(1), 1, "x: codes", 1),
    (mat(4, 256), mat(32, 256, None), None, at(1), 1, "w: codes", 1),
])
def test_gemm_refusals(lib, x, w, res, y, dtype, text, status):
    refused(lib, lib.tb_gemm_e4m3(x, w, res, y, dtype, None), text, status)


@pytest.mark.parametrize("w3,y,dtype,ys,text", [
    (mat(48, 256, at(12), at(13)), at(1), 1, None, "w1 has 32 rows"),
    (mat(32, 128, at(12), at(13)), at(1), 1, None, "w3 has 128 columns"),
    (mat(32, 256, at(12), at(13)), at(1), 2, None, "unknown y_dtype"),
    (mat(32, 256, at(12), at(13)), at(1), 3, None, "y_scale goes with codes"),
    (mat(32, 256, at(12), at(13)), at(1), 1, at(2), "y_scale goes with codes"),
    (mat(32, 256, at(12), at(13)), at(1), 3, at(1) + 100, "two outputs overlap"),
    (mat(32, 256, at(12), at(13)), at(1), 3, at(13), "an output overlaps"),
    (mat(32, 256, at(12), at(13)), at(12) + 16, 3, at(2), "an output overlaps"),
    (mat(32, 256, at(12), at(13)), at(20), 3, at(2), "an output overlaps"),
])
def test_gated_refusals(lib, w3, y, dtype, ys, text):
    refused(lib, lib.tb_gated_e4m3(mat(4, 256), mat(32, 256, **W), w3, y, dtype, ys, None), text)


def test_empty_calls_need_no_pointers(lib):
    none = mat(0, 256, None, None)
    assert lib.tb_rmsnorm_e4m3(None, 1, None, 0, None, None, 1e-5, none, None) == 0
    assert lib.tb_quant_e4m3(None, 0, none, None) == 0
    assert lib.tb_pack_e4m3(None, 0, none, None) == 0
    assert lib.tb_gemm_e4m3(none, mat(32, 256), None, None, 1, None) == 0
    assert lib.tb_gated_e4m3(none, mat(32, 256), mat(32, 256), None, 3, None, None) == 0


# ---- the rule for the kernel --------------------------------------------------------

@pytest.mark.parametrize("M,N,K,mats,light,tile", [
    (1, 6144, 4096, 1, 0, 16), (16, 6144, 4096, 1, 0, 16), (17, 6144, 4096, 1, 0, 32), (33, 6144, 4096, 1, 0, 64),
    (512, 2304, 768, 1, 0, 32), (513, 2304, 768, 1, 0, 64), (1371, 2304, 768, 1, 1, 128), (1371, 2304, 768, 1, 0, 0), (128, 20000, 768, 1, 0, 128),
    (129, 20000, 768, 1, 0, 0), (1371, 2304, 1536, 1, 1, 128), (1371, 2304, 1536, 1, 0, 0),
    (2049, 2304, 768, 1, 1, 0), (256, 4096, 4096, 1, 0, 64), (257, 4096, 4096, 1, 0, 128), (512, 4096, 4096, 1, 0, 128),
    (513, 4096, 4096, 1, 0, 0), (64, 14336, 4096, 1, 0, 64), (128, 14336, 4096, 1, 0, 128), (129, 14336, 4096, 1, 0, 0),
    (32, 14336, 4096, 2, 0, 32), (64, 14336, 4096, 2, 0, -1), (128, 14336, 4096, 2, 0, -1), (129, 14336, 4096, 2, 0, 0),
    (64, 8192, 4096, 2, 0, 32), (65, 8192, 4096, 2, 0, 0), (128, 50304, 768, 1, 0, -1), (129, 50304, 768, 1, 0, 0), (64, 50304, 768, 1, 0, 64), (128, 2048, 768, 2, 0, 32), (129, 2048, 768, 2, 0, 0), (333, 2048, 768, 2, 1, 32), (96, 11008, 2048, 2, 0, 32),
    (1024, 2048, 768, 2, 0, 0), (128, 4096, 1536, 2, 0, 32), (192, 4096, 1536, 2, 0, 0), (256, 2048, 4096, 2, 0, 32), (333, 2048, 4096, 2, 0, 0),
    (2 ** 31 - 1024, 16, 16, 1, 0, 0), (2 ** 31 - 1024, 16, 16, 2, 1, 0), (64, 2 ** 28, 16, 1, 0, 64)])
def test_tile_rule(lib, M, N, K, mats, light, tile):
    assert lib.tbx_e4m3_few_tile(M, N, K, mats, light, 152) == tile


# ---- the binding ----------------------------------------------------------------

@pytest.fixture
def on_gpu(monkeypatch):
    """CPU tensors stand in for tensors of cuda:0, the current device."""
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: getattr(self, "_dev", 0))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)


def codes(*shape, dtype=CODE):
    return torch.zeros(*shape, dtype=torch.uint8).view(dtype)


def rows(M, K):
    return tb.E4M3Rows(codes(M, K), codes(M, -(-K // 128), dtype=SCALE))


def weight(N, K):
    return tb.E4M3Weight(codes(N, K), codes(-(-N // 128), -(-K // 128), dtype=SCALE))


def test_handles_take_dense_tensors_of_their_shapes(on_gpu):
    x = rows(5, 272)
    assert (x.rows, x.cols, x._struct.codes) == (5, 272, x.codes.data_ptr())
    w = weight(272, 144)
    assert (w.rows, w.cols, w._struct.scale) == (272, 144, w.scale.data_ptr())
    for bad in (lambda: tb.E4M3Rows(codes(5, 272), codes(5, 2, dtype=SCALE)),
                lambda: tb.E4M3Rows(codes(5, 272), codes(1, 3, dtype=SCALE)),
                lambda: tb.E4M3Rows(codes(272), codes(3, dtype=SCALE)),
                lambda: tb.E4M3Rows(codes(5, 544)[:, ::2], codes(5, 3, dtype=SCALE)),
                lambda: tb.E4M3Rows(codes(5, 272), codes(5, 6, dtype=SCALE)[:, :3]),
                lambda: tb.E4M3Rows(torch.zeros(5, 272), codes(5, 3, dtype=SCALE)),
                lambda: tb.E4M3Rows(codes(5, 272), torch.ones(5, 3)),
                lambda: tb.E4M3Weight(codes(272, 144), codes(272, 2, dtype=SCALE))):
        with pytest.raises(ValueError):
            bad()


def test_handles_refuse_cpu_tensors_and_counts_beyond_the_struct(monkeypatch):
    with pytest.raises(ValueError, match="CUDA tensor"):
        rows(4, 256)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)

    class Tall:
        """Stands in for a tensor of 2^32 + 4 rows."""
        shape = (2 ** 32 + 4, 16)

        def dim(self):
            return 2

        def get_device(self):
            return 0

    with pytest.raises(ValueError, match="2\\^31 - 1"):
        tb.E4M3Rows(Tall(), None)


def test_binding_refusals(on_gpu):
    x, w = rows(4, 256), weight(32, 256)
    f = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    other = f(4, 32)
    other._dev = 1
    calls = [
        (lambda: tb.tb_gemm_e4m3(w, w), "x must be E4M3Rows"),
        (lambda: tb.tb_gemm_e4m3(x, x), "w must be E4M3Weight"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=f(4, 33)), "y must"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=f(4, 64)[:, ::2]), "y must"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=f(4, 32, dtype=torch.float16)), "float32 or bfloat16"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=f(4, 32), y_dtype=tb.TB_F32), "another type"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=f(4, 32), res=f(4, 32, dtype=torch.float32)), "res must"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=f(4, 32), res=f(1, 32)), "res must"),
        (lambda: tb.tb_gemm_e4m3(x, w, y=other), "y must"),
        (lambda: tb.tb_gated_e4m3(x, w, x), "w3 must be E4M3Weight"),
        (lambda: tb.tb_gated_e4m3(x, w, w, out=rows(4, 48)), "out must have 4 rows of 32"),
        (lambda: tb.tb_gated_e4m3(x, w, w, out=rows(4, 32), out_dtype=tb.TB_BF16), "out must be a tensor"),
        (lambda: tb.tb_gated_e4m3(x, w, w, out=f(4, 32), out_dtype=tb.TB_E4M3), "out must be E4M3Rows"),
        (lambda: tb.tb_gated_e4m3(x, w, w, out=f(4, 32), out_dtype=tb.TB_F32), "another type"),
        (lambda: tb.tb_gated_e4m3(x, w, w, out_dtype=9), "out_dtype"),
        (lambda: tb.tb_quant_e4m3(f(4, 256, dtype=torch.float16)), "float32 or bfloat16"),
        (lambda: tb.tb_quant_e4m3(f(4, 256), out=rows(4, 128)), "out must have 4 rows of 256"),
        (lambda: tb.tb_quant_e4m3(f(256, 4).T, out=rows(4, 256)), "x must"),
        (lambda: tb.tb_rmsnorm_e4m3(f(4, 256), f(128), 1e-5), "g must"),
        (lambda: tb.tb_rmsnorm_e4m3(f(4, 256), f(256, dtype=torch.float32), 1e-5), "g must"),
        (lambda: tb.tb_rmsnorm_e4m3(f(4, 256), f(256), 1e-5, h=f(4, 256)), "h without r"),
        (lambda: tb.tb_rmsnorm_e4m3(f(4, 256), f(256), 1e-5, r=f(4, 128)), "r must"),
        (lambda: tb.tb_rmsnorm_e4m3(f(4, 256), f(256), 1e-5, r=f(4, 256), h=f(4, 256, dtype=torch.float32)), "h must"),
        (lambda: tb.tb_pack_e4m3(f(2, 4, 8)), "w must be"),
        (lambda: tb.tb_pack_e4m3(f(256, 32), out=weight(256, 32)), "out must have 32 rows of 256"),
    ]
    for call, text in calls:
        with pytest.raises(ValueError, match=text):
            call()


def test_another_device_than_the_current_one_is_refused(on_gpu, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 1)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    x, w = rows(4, 256), weight(32, 256)
    with pytest.raises(ValueError, match="cuda:1"):
        tb.tb_gemm_e4m3(x, w, y=torch.zeros(4, 32, dtype=torch.bfloat16))


# ---- the oracle -------------------------------------------------------------------

def test_code_values_are_torch_s():
    want = torch.arange(256, dtype=torch.uint8).view(CODE).double().numpy()
    assert np.array_equal(ref.VALUES, want, equal_nan=True)
    scales = torch.arange(256, dtype=torch.uint8).view(SCALE).double().numpy()
    assert np.array_equal(ref.scale_values(np.arange(256)), scales, equal_nan=True)


def test_exponents():
    for top, e in ((0.0, -100), (448.0, 0), (448.0 * (1 + 2 ** -50), 1), (224.0, -1), (1.0, -8), (2.0 ** -200, -100),
                   (3.4e38, 120)):
        assert ref.exponent(np.array([0.0, -top, np.nan, np.inf])) == e, top


def test_half_steps_are_half_the_distance_of_neighbours():
    v = np.sort(ref.VALUES[:0x7F])
    for lo, hi in zip(v, v[1:]):
        assert ref.half_step(np.array(lo)) == (hi - lo) / 2


def test_blocks_of_rows_and_weights():
    c = np.full((130, 144), 0x38, np.uint8)
    s = np.array([[127, 128], [129, 130]], np.uint8)
    w = ref.weight_values(c, s)
    assert w[0, 0] == 1 and w[127, 128] == 2 and w[128, 127] == 4 and w[129, 143] == 8
    x = ref.rows_values(c, np.tile(np.array([126, 129], np.uint8), (130, 1)))
    assert x[0, 127] == 0.5 and x[129, 128] == 4

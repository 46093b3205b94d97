"""Inputs and tolerances of the tests of the 8-bit projections.

A product's fp32 sum.  One tensor-core instruction adds 32 products of 4-bit mantissas
(exact in fp32) to the sum so far; alignment to the largest of them may cut what lies
below fp32's last place of the result, at most 2 steps of 2^-23 of the magnitudes summed
so far, S = sum |x w|.  64 instructions run in one accumulator, whose magnitudes are a
part of S; the parts are added with rounding (at most 15 of them, 2^-24 each):

    |sum - exact| <= (2·64 + 8)·2^-23·S          SUM·S below

The many-rows kernel keeps one accumulator for all of K: `accumulated(K)`."""
import numpy as np
import torch

from oracle import e4m3 as ref

BF16, F32 = torch.bfloat16, torch.float32
CODE, SCALE = torch.float8_e4m3fn, torch.float8_e8m0fnu
HALF = {BF16: 2.0 ** -9, F32: 2.0 ** -24}      # half a step, relative to the power of two below the value


def accumulated(K: int) -> float:
    return (2 * max(64, -(-K // 32)) + 8) * 2.0 ** -23


def rounding(ref_values, dtype):
    """Half a step of dtype at these values (2 HALF·|v| bounds it from above)."""
    return 2 * HALF[dtype] * np.abs(ref_values)


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def random_codes(rows, cols, g, lo=0, hi=256):
    """Code bytes without NaN."""
    b = torch.randint(lo, hi, (rows, cols), generator=g, dtype=torch.uint8)
    b[(b & 0x7F) == 0x7F] = 0x31
    return b


def random_scales(shape, g, lo=-5, hi=4):
    return torch.randint(127 + lo, 127 + hi, shape, generator=g, dtype=torch.uint8)


def normal_codes(rows, cols, g):
    """Codes of N(0, 1) values times 40: mostly of neighbouring exponents, as quantised rows are."""
    return (torch.randn(rows, cols, generator=g) * 40).clamp(-448, 448).to(CODE).view(torch.uint8)


def make_rows(tb, M, K, g, codes=normal_codes, device="cuda"):
    return tb.E4M3Rows(codes(M, K, g).view(CODE).to(device), random_scales((M, -(-K // 128)), g).view(SCALE).to(device))


def make_weight(tb, N, K, g, codes=normal_codes, device="cuda"):
    return tb.E4M3Weight(codes(N, K, g).view(CODE).to(device),
                         random_scales((-(-N // 128), -(-K // 128)), g).view(SCALE).to(device))


def rows_np(x):
    return ref.rows_values(bytes_of(x.codes), bytes_of(x.scale))


def weight_np(w):
    return ref.weight_values(bytes_of(w.codes), bytes_of(w.scale))


def product(x, w, res=None):
    """(exact, magnitudes summed) of x·wᵀ (+ res) from fp64 values."""
    y, s = x @ w.T, np.abs(x) @ np.abs(w).T
    return (y, s) if res is None else (y + res, s + np.abs(res))


def check_product(y, exact, mag, K, dtype):
    got = y.float().cpu().numpy().astype(np.float64)
    tol = accumulated(K) * mag
    bad = np.abs(got - exact) > tol + rounding(np.abs(exact) + tol, dtype)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), np.abs(got - exact)[bad][:4], tol[bad][:4])


def check_rows(codes, scale, exact, off):
    """Codes and scale bytes of rows against the values `exact` that they stand for,
    which the kernel knows to within `off` (of the same shape, absolute)."""
    M, n = exact.shape
    e = scale.astype(np.int64) - 127
    assert ((scale != 255) & (e >= ref.EXP[0]) & (e <= ref.EXP[1])).all()
    pad = (-n) % ref.BLOCK

    def tops(a):
        return np.pad(a, ((0, 0), (0, pad))).reshape(M, -1, ref.BLOCK).max(-1)

    fine = np.isfinite(exact)
    a = np.where(fine, np.abs(exact), 0)
    low, high = tops(np.where(fine, np.maximum(a - off, 0), 0)), tops(np.where(fine, a + off, 0))
    assert (low <= ref.TOP * np.ldexp(1.0, e)).all(), "a scale too small for its block"
    assert ((high > ref.TOP * np.ldexp(1.0, e - 1)) | (e == ref.EXP[0])).all(), "a scale too large for its block"
    s = np.repeat(np.ldexp(1.0, e), ref.BLOCK, 1)[:, :n]
    got = ref.VALUES[codes] * s
    assert (np.isnan(got) == ~fine).all()
    q = np.where(fine, np.abs(exact) + off, 0) / s
    bad = fine & (np.abs(got - np.where(fine, exact, 0)) > ref.half_step(np.minimum(q, ref.TOP)) * s + off)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], exact[bad][:4])


def gated_and_off(x, w1, w3, K):
    """(exact, error bound) of SiLU(x·w1ᵀ)·(x·w3ᵀ): SiLU's slope is below 1.1; its fp32
    evaluation (expf within 2 ulp, a sum, a quotient, a product) is within 8·2^-24.  To 16
    bits and codes it may be off by (0.28·2^-23 + 2^-21)·|g| more, which is less than
    2^-20·|g| and thus inside the first term, of which accumulated(K) leaves 8·2^-23·gs."""
    g, gs = product(x, w1)
    u, us = product(x, w3)
    with np.errstate(over="ignore"):
        a = ref.silu(g)
    eg, eu = accumulated(K) * gs, accumulated(K) * us
    exact = a * u
    return exact, 1.1 * eg * (np.abs(u) + eu) + np.abs(a) * eu + 8 * 2.0 ** -24 * np.abs(exact)

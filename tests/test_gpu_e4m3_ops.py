"""The 8-bit projections against fp64, element by element (e4m3_helpers derives the
tolerances)."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import causal_gqa_attention_rmsnorm_gb300 as tb
from causal_gqa_attention_rmsnorm_gb300.binding import tbx_e4m3_form
from e4m3_helpers import (BF16, CODE, F32, HALF, SCALE, bytes_of, check_product, check_rows, gated_and_off, make_rows,
                          make_weight, product, random_codes, rows_np, weight_np)
from oracle import e4m3 as ref

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def gen(seed):
    return torch.Generator().manual_seed(seed)


def f64(t):
    return t.double().cpu().numpy()


def no_error():
    assert tb.tb_get_device_error(clear=True) == 0


@pytest.fixture
def form():
    """Sets the form that the products of a test take."""
    yield tbx_e4m3_form
    tbx_e4m3_form(0)


# ---- rows ---------------------------------------------------------------------

def stream_rows(M, d, dtype, g):
    """Rows as a residual stream has them: a few large channels, rows of many sizes."""
    x = torch.randn(M, d, generator=g) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g).float())
    x[:, torch.randint(0, d, (2,), generator=g)] *= 30
    return x.to(dtype).cuda()


# A thread adds at most 64 squares one after another, then 5 + 15 levels; a square root,
# two quotients and two products follow, and the sum x + r before them: 100 roundings.
NORM_OFF = 100 * 2.0 ** -24


@pytest.mark.parametrize("M,d", [(1, 16), (1, 4096), (3, 128), (7, 144), (5, 768), (305, 1008), (306, 4096), (400, 784),
                                 (2, 11008), (310, 16384), (311, 16400), (3, 32768), (1, 14336), (700, 32)])
@pytest.mark.parametrize("dtype,r_dtype", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, None), (F32, BF16), (F32, F32)])
def test_norm(M, d, dtype, r_dtype):
    g = gen(M * 7 + d)
    x = stream_rows(M, d, dtype, g)
    gain = (1 + 0.1 * torch.randn(d, generator=g)).to(dtype).cuda()
    r = None if r_dtype is None else torch.randn(M, d, generator=g).to(r_dtype).cuda()
    out, h = tb.tb_rmsnorm_e4m3(x, gain, 1e-5, r=r)
    no_error()
    total = f64(x) + (0 if r is None else f64(r))
    if r is None:
        assert h is None
    else:
        one = np.abs(f64(h) - total) <= 2 * (HALF[dtype] + 2.0 ** -24) * np.abs(total)
        assert one.all()
    y = ref.norm(total, f64(gain), 1e-5)
    # (the sum's own rounding is relative to itself: x + r is one fp32 addition)
    check_rows(bytes_of(out.codes), bytes_of(out.scale), y, NORM_OFF * np.abs(y))


@pytest.mark.parametrize("M,d", [(1, 16), (1, 4096), (3, 128), (7, 144), (305, 784), (2, 11008), (309, 11008), (1, 65536),
                                 (3, 53248), (313, 8208)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quant(M, d, dtype):
    x = stream_rows(M, d, dtype, gen(M + d))
    out = tb.tb_quant_e4m3(x)
    no_error()
    # the quotients are exact: nothing but the codes' rounding
    check_rows(bytes_of(out.codes), bytes_of(out.scale), f64(x), np.zeros((M, d)))
    e = bytes_of(out.scale).astype(int) - 127
    assert (e == ref.rows_exponents(f64(x))).all()


def test_quant_ties_go_to_the_even_code_and_borders_keep_their_scale():
    x = torch.zeros(3, 256)
    x[0, :8] = torch.tensor([448.0, 17.0, 19.0, -17.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0625, 1.1875])
    x[1, :2] = torch.tensor([448.0 * (1 + 2.0 ** -23), 1.0])           # one step above: the next scale
    x[1, 128:130] = torch.tensor([448.0 * 2.0 ** -60, 2.0 ** -60])
    x[2, :2] = torch.tensor([2.0 ** -140, 3e38])
    x[2, 128:130] = torch.tensor([2.0 ** -149, 0.0])                    # below the smallest scale
    out = tb.tb_quant_e4m3(x.cuda())
    v = ref.VALUES[bytes_of(out.codes)]
    assert v[0, :8].tolist() == [448, 16, 20, -16, 0, 2.0 ** -8, 1.0, 1.25]
    e = bytes_of(out.scale).astype(int) - 127
    assert e.tolist() == [[0, -100], [1, -60], [120, -100]]
    assert (v[0, 128:] == 0).all() and v[1, 128] == 448 and v[2, 128] == 0


def test_rows_with_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    x = torch.randn(4, 400, generator=gen(2))
    x[0, 5], x[0, 200], x[1, 399], x[2, :128] = nan, inf, -inf, nan
    for dtype in (BF16, F32):
        y = x.to(dtype).cuda()
        out = tb.tb_quant_e4m3(y)
        check_rows(bytes_of(out.codes), bytes_of(out.scale), f64(y), np.zeros((4, 400)))
        assert bytes_of(out.scale)[2, 0] == 27                       # no finite value at all: as a block of zeros
        # the norm: a NaN or an infinity is in its row's mean; the others are as they were
        n, _ = tb.tb_rmsnorm_e4m3(y, torch.ones(400, dtype=dtype, device="cuda"), 1e-5)
        alone, _ = tb.tb_rmsnorm_e4m3(y[3:].clone(), torch.ones(400, dtype=dtype, device="cuda"), 1e-5)
        assert np.isnan(ref.VALUES[bytes_of(n.codes)[0]]).all() and np.isnan(ref.VALUES[bytes_of(n.codes)[2]]).all()
        v = ref.VALUES[bytes_of(n.codes)[1]]
        assert np.isnan(v[399]) and (v[:399] == 0).all()
        assert (bytes_of(n.codes)[3] == bytes_of(alone.codes)[0]).all()
        assert (bytes_of(n.scale)[3] == bytes_of(alone.scale)[0]).all()
    no_error()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_without_a_finite_result(dtype):
    """Rows of zeros without eps, results beyond fp32, an infinite gain: NaN codes where the
    value is none, the scale of what is finite, and nothing of it in the rows beside."""
    x = torch.randn(5, 272, generator=gen(3))
    x[1] = 0
    gain = torch.ones(272)
    gain[7], gain[130] = 3e38, float("inf")
    x[2, 7], x[3, 130] = 200.0, 0.0
    x, gain = x.to(dtype), gain.to(dtype)
    out, _ = tb.tb_rmsnorm_e4m3(x.cuda(), gain.cuda(), 0.0)
    no_error()
    with np.errstate(all="ignore"):
        y = ref.norm(f64(x), f64(gain), 0.0)
    y = np.where(np.abs(y) <= 3.4028234e38, y, np.nan)                # fp32's range
    assert np.isnan(y[1]).all() and np.isnan(y[3, 130]) and np.isnan(y[2, 7]) and np.isfinite(np.delete(y[0], [7, 130])).all()
    check_rows(bytes_of(out.codes), bytes_of(out.scale), y, NORM_OFF * np.abs(y))
    assert (bytes_of(out.scale)[1] == 27).all()


# one of each number of eights per thread that the rule takes for these types, with warps,
# a CTA's last block and its last eight partly filled
MANY_ROWS = [(401, 240, BF16, None), (401, 496, BF16, None), (401, 656, BF16, None), (403, 1008, BF16, None),
             (402, 2000, BF16, None), (2050, 1936, BF16, None), (401, 4112, BF16, None), (310, 5136, BF16, None),
             (401, 496, BF16, BF16), (401, 656, BF16, F32), (403, 1008, BF16, BF16), (310, 8176, BF16, F32), (310, 8208, BF16, BF16),
             (4099, 240, F32, None), (4099, 496, F32, None), (4099, 656, F32, None), (4099, 1008, F32, None),
             (401, 1040, F32, None), (305, 12304, F32, None), (401, 1008, F32, BF16), (401, 4080, F32, F32),
             (310, 4112, F32, F32), (401, 2064, F32, BF16), (310, 4112, F32, BF16), (305, 12304, F32, BF16)]


@pytest.mark.parametrize("M,d,dtype,r_dtype", MANY_ROWS)
def test_norm_of_many_rows(M, d, dtype, r_dtype):
    """With a NaN, an infinity, a row of zeros without eps and a result beyond fp32 among them."""
    g = gen(M + d)
    x = stream_rows(M, d, dtype, g)
    gain = (1 + 0.1 * torch.randn(d, generator=g)).to(dtype).cuda()
    r = None if r_dtype is None else torch.randn(M, d, generator=g).to(r_dtype).cuda()
    x[1, 7], x[3, d - 1], x[5] = float("nan"), float("inf"), 0
    gain[d // 2] = 3e38
    if r is not None:
        r[5] = 0
    out, h = tb.tb_rmsnorm_e4m3(x, gain, 0.0, r=r)
    no_error()
    total = f64(x) + (0 if r is None else f64(r))
    if r is not None:
        fine = np.isfinite(total)
        assert (np.abs(f64(h)[fine] - total[fine]) <= 2 * (HALF[dtype] + 2.0 ** -24) * np.abs(total)[fine]).all()
        assert (np.isnan(f64(h)) == np.isnan(total)).all() and (np.isinf(f64(h)) == np.isinf(total)).all()
    with np.errstate(all="ignore"):
        y = ref.norm(total, f64(gain), 0.0)
    assert np.isnan(y[1]).all() and np.isnan(y[5]).all() and (np.delete(y[3], d - 1) == 0).all()
    y = np.where(np.abs(y) <= 3.4028234e38, y, np.nan)                # fp32's range
    check_rows(bytes_of(out.codes), bytes_of(out.scale), y, NORM_OFF * np.abs(y))


@pytest.mark.parametrize("M,d,dtype", [(401, 240, BF16), (401, 496, BF16), (401, 1008, BF16), (310, 8208, BF16), (401, 240, F32), (401, 1008, F32),
                                       (310, 4112, F32)])
def test_quant_of_many_rows(M, d, dtype):
    x = stream_rows(M, d, dtype, gen(M + d))
    x[1, 7], x[3, d - 1], x[5] = float("nan"), float("inf"), 0
    x[7, :128] = float("-inf")
    out = tb.tb_quant_e4m3(x)
    no_error()
    check_rows(bytes_of(out.codes), bytes_of(out.scale), f64(x), np.zeros((M, d)))
    assert bytes_of(out.scale)[7, 0] == 27                           # no finite value at all


@pytest.mark.parametrize("M,d", [(2, 400), (400, 768)])
def test_norm_in_place_gives_the_same(M, d):
    g = gen(5)
    x, r = (torch.randn(M, d, generator=g).to(BF16).cuda() for _ in range(2))
    gain = torch.randn(d, generator=g).to(BF16).cuda()
    out, h = tb.tb_rmsnorm_e4m3(x, gain, 1e-6, r=r)
    for into in ("x", "r"):
        a, b = x.clone(), r.clone()
        mine, got = tb.tb_rmsnorm_e4m3(a, gain, 1e-6, r=b, h=a if into == "x" else b)
        assert torch.equal(got, h) and (bytes_of(mine.codes) == bytes_of(out.codes)).all()
    # rows of any leading shape
    again, h3 = tb.tb_rmsnorm_e4m3(x.view(2, M // 2, d), gain, 1e-6, r=r.view(2, M // 2, d))
    assert h3.shape == (2, M // 2, d) and (bytes_of(again.codes) == bytes_of(out.codes)).all()


@pytest.mark.parametrize("K,N", [(16, 16), (128, 128), (144, 272), (768, 2304), (400, 48)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pack(K, N, dtype):
    g = gen(K + N)
    w = (0.02 * torch.randn(K, N, generator=g) * torch.exp2(torch.randint(-8, 8, (K, 1), generator=g).float())).to(dtype)
    w[0, 0], w[K - 1, N - 1] = float("nan"), float("inf")
    got = tb.tb_pack_e4m3(w.cuda())
    no_error()
    x = f64(w).T
    e = bytes_of(got.scale).astype(int) - 127
    assert (e == ref.weight_exponents(x)).all()
    v = weight_np(got)
    fine = np.isfinite(x)
    assert (np.isnan(v) == ~fine).all()
    s = np.repeat(np.repeat(np.ldexp(1.0, e), 128, 0)[:N], 128, 1)[:, :K]
    assert (np.abs(v - np.where(fine, x, 0))[fine] <= (ref.half_step(np.where(fine, x, 0) / s) * s)[fine]).all()


# ---- the product ----------------------------------------------------------------

SIZES = [(1, 16, 16), (1, 128, 128), (1, 2304, 768), (3, 144, 400), (16, 256, 512), (17, 112, 2064), (33, 400, 640),
         (64, 128, 4096), (65, 272, 1168), (128, 768, 2176), (129, 144, 144), (200, 1040, 912), (300, 2304, 768),
         (7, 4096, 1024), (2, 128, 9216), (5, 32, 14336)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,with_res", [(F32, False), (BF16, True)])
def test_gemm(M, N, K, dtype, with_res):
    g = gen(M + N + K)
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    res = (torch.randn(M, N, generator=g) * 100).to(dtype).cuda() if with_res else None
    y = tb.tb_gemm_e4m3(x, w, res=res, y_dtype=tb.TB_F32 if dtype is F32 else tb.TB_BF16)
    no_error()
    assert y.dtype is dtype and y.shape == (M, N)
    check_product(y, *product(rows_np(x), weight_np(w), None if res is None else f64(res)), K, dtype)
    if with_res:                                    # in place
        z = tb.tb_gemm_e4m3(x, w, res=res, y=res)
        assert z is res and torch.equal(z, y)


def test_gemm_every_code_and_scale_counts():
    """Rows of one code each against weights of single ones: every code, at every scale
    byte that keeps the product an fp32 value, comes back exactly."""
    K = 256
    codes = torch.zeros(256, K, dtype=torch.uint8)
    codes[:, 130] = torch.arange(256, dtype=torch.uint8)
    scale = torch.full((256, 2), 127, dtype=torch.uint8)
    scale[:, 1] = 20 + (torch.arange(256) * 37 % 200).to(torch.uint8)
    w = torch.zeros(256, K, dtype=torch.uint8)
    w[:, 130] = 0x38                                # 1.0
    ws = torch.tensor([[127, 127], [127, 130]], dtype=torch.uint8)
    y = tb.tb_gemm_e4m3(tb.E4M3Rows(codes.view(CODE).cuda(), scale.view(SCALE).cuda()),
                        tb.E4M3Weight(w.view(CODE).cuda(), ws.view(SCALE).cuda()), y_dtype=tb.TB_F32)
    no_error()
    got = y.cpu().numpy().astype(np.float64)
    v = ref.VALUES[np.arange(256)] * np.ldexp(1.0, scale[:, 1].numpy().astype(int) - 127)
    for n, f in ((0, 1.0), (127, 1.0), (128, 8.0), (255, 8.0)):
        assert np.array_equal(got[:, n], v * f, equal_nan=True)


def test_gemm_nan_stays_in_its_row_and_its_column():
    g = gen(9)
    M, N, K = 70, 272, 528
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    clean = tb.tb_gemm_e4m3(x, w)
    x.codes.view(torch.uint8)[3, 100] = 0x7F
    x.scale.view(torch.uint8)[66, 4] = 255
    w.codes.view(torch.uint8)[5, 527] = 0xFF
    w.scale.view(torch.uint8)[2, 1] = 255           # rows 256 to 271
    y = tb.tb_gemm_e4m3(x, w)
    no_error()
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[3], hit[66], hit[:, 5], hit[:, 256:] = True, True, True, True
    assert torch.equal(torch.isnan(y), hit)
    assert torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("tile", [16, 64, 128, -1, -2])
def test_gemm_far_scales(form, tile):
    """Scales whose product leaves fp32: infinity above, 0 (or a subnormal) below, and
    zeros stay zeros under any scale."""
    form(tile)
    M, N, K = 20, 16, 256
    x = torch.zeros(M, K, dtype=torch.uint8)
    x[:, 5], x[:, 200] = 0x38, 0x38                    # 1 in each block
    x[1, 5] = x[2, 200] = 0
    xs = torch.full((M, 2), 127, dtype=torch.uint8)
    xs[0], xs[1], xs[2] = 247, torch.tensor([254, 127]), torch.tensor([127, 0])
    xs[3], xs[4] = torch.tensor([27, 127]), torch.tensor([0, 0])
    w = torch.zeros(N, K, dtype=torch.uint8)
    w[:, 5], w[:, 200] = 0x38, 0xB8                    # 1 and -1
    w[1, 5], w[1, 200] = 0, 0
    ws = torch.tensor([[247, 127]], dtype=torch.uint8)
    y = tb.tb_gemm_e4m3(tb.E4M3Rows(x.view(CODE).cuda(), xs.view(SCALE).cuda()),
                        tb.E4M3Weight(w.view(CODE).cuda(), ws.view(SCALE).cuda()), y_dtype=tb.TB_F32)
    no_error()
    got = f64(y)
    assert (got[:, 1] == 0).all()                      # a row of zero weights
    cols = [0] + list(range(2, N))
    want = {0: np.inf, 1: -1.0, 2: 2.0 ** 120, 3: 2.0 ** 20 - 1, 4: 2.0 ** -7, 5: 2.0 ** 120}
    for m, v in want.items():
        assert (got[m, cols] == v).all(), (m, v, got[m, :3])


@pytest.mark.parametrize("M", [1, 16, 40, 100, 130])
def test_gemm_writes_its_rows_only(M):
    g = gen(M)
    N, K = 144, 272
    buf = torch.full((M + 5, N), 7.0, dtype=BF16, device="cuda")
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    tb.tb_gemm_e4m3(x, w, y=buf[2:2 + M])
    no_error()
    assert (buf[:2] == 7).all() and (buf[2 + M:] == 7).all()
    check_product(buf[2:2 + M], *product(rows_np(x), weight_np(w)), K, BF16)


# ---- the gated half ---------------------------------------------------------------

@pytest.mark.parametrize("M,F,K", [(1, 16, 16), (1, 256, 128), (5, 144, 400), (16, 2048, 768), (17, 272, 2064), (32, 400, 1024),
                                   (33, 128, 640), (65, 144, 272), (130, 1040, 528), (333, 2048, 768), (2, 128, 9216)])
@pytest.mark.parametrize("out_dtype", ["codes", BF16, F32])
def test_gated(M, F, K, out_dtype):
    g = gen(M + F + K)
    x, w1, w3 = make_rows(tb, M, K, g), make_weight(tb, F, K, g), make_weight(tb, F, K, g)
    # gates of sizes where SiLU bends
    w1.scale.view(torch.uint8).sub_(int(np.log2(K) / 2) + 11)
    exact, off = gated_and_off(rows_np(x), weight_np(w1), weight_np(w3), K)
    if out_dtype == "codes":
        out = tb.tb_gated_e4m3(x, w1, w3)
        no_error()
        check_rows(bytes_of(out.codes), bytes_of(out.scale), exact, off)
    else:
        y = tb.tb_gated_e4m3(x, w1, w3, out_dtype=tb.TB_F32 if out_dtype is F32 else tb.TB_BF16)
        no_error()
        assert y.dtype is out_dtype
        assert (np.abs(f64(y) - exact) <= off + 2 * HALF[out_dtype] * (np.abs(exact) + off)).all()


@pytest.mark.parametrize("tile,M", [(16, 3), (32, 30), (64, 70), (-1, 200), (-2, 200)])
def test_gated_infinities_and_nan_become_nan_codes(form, tile, M):
    """Results beyond fp32 and NaN are NaN codes, and the scale is that of the others."""
    form(tile)
    g = gen(M)
    F, K = 272, 144
    x, w1, w3 = make_rows(tb, M, K, g), make_weight(tb, F, K, g), make_weight(tb, F, K, g)
    x.codes.view(torch.uint8)[1] = 0x7E                # 448 throughout: gates and values of thousands
    x.scale.view(torch.uint8)[1] = 200
    x.codes.view(torch.uint8)[0, 100] = 0x7F
    w3.codes.view(torch.uint8)[130] = 0xFF
    out = tb.tb_gated_e4m3(x, w1, w3)
    no_error()
    exact, off = gated_and_off(rows_np(x), weight_np(w1), weight_np(w3), K)
    sure = np.isfinite(exact) & (np.abs(exact) + off < 3.4e38)
    gone = ~np.isfinite(exact) | (np.abs(exact) - off > 3.41e38)
    assert gone[0].all() and gone[1].any() and gone[2:, 130].all() and (sure | gone)[[0] + list(range(2, M))].all()
    v = ref.VALUES[bytes_of(out.codes)]
    assert np.isnan(v[gone]).all() and np.isfinite(v[2:][sure[2:]]).all()
    check_rows(bytes_of(out.codes)[2:], bytes_of(out.scale)[2:], np.where(sure, exact, np.nan)[2:], np.where(sure, off, 0)[2:])


def test_gated_gates_far_below_zero():
    """SiLU of gates down to -448·2^4: below -87 it is under 1e-35 and may come back as 0."""
    M, F, K = 20, 128, 128
    x = torch.zeros(M, K, dtype=torch.uint8)
    x[:, 0] = 0x38
    w1, w3 = torch.zeros(F, K, dtype=torch.uint8), torch.zeros(F, K, dtype=torch.uint8)
    w1[:, 0], w3[:, 0] = 0x80 + torch.arange(F, dtype=torch.uint8).clamp(max=126), 0x38
    one = torch.full((M, 1), 127, dtype=torch.uint8).view(SCALE).cuda()
    big = torch.full((1, 1), 131, dtype=torch.uint8).view(SCALE).cuda()
    unit = torch.full((1, 1), 127, dtype=torch.uint8).view(SCALE).cuda()
    for form in (16, 64, -1, -2):
        tbx_e4m3_form(form)
        y = tb.tb_gated_e4m3(tb.E4M3Rows(x.view(CODE).cuda(), one), tb.E4M3Weight(w1.view(CODE).cuda(), big),
                             tb.E4M3Weight(w3.view(CODE).cuda(), unit), out_dtype=tb.TB_F32)
        tbx_e4m3_form(0)
        no_error()
        gates = ref.VALUES[w1[:, 0].numpy()] * 16
        with np.errstate(over="ignore"):
            want = ref.silu(gates)
        assert (np.abs(f64(y) - want[None]) <= 8 * 2.0 ** -24 * np.abs(want) + 1e-35).all()


def test_gated_far_gates():
    """Gates far below and above zero: SiLU gives 0 and the gate itself, not NaN."""
    M, F, K = 4, 128, 128
    x = torch.zeros(M, K, dtype=torch.uint8)
    x[:, 0] = 0x38
    w1, w3 = torch.zeros(F, K, dtype=torch.uint8), torch.zeros(F, K, dtype=torch.uint8)
    w1[:, 0], w3[:, 0] = torch.arange(F, dtype=torch.uint8).bitwise_xor(0x80), 0x38
    w1[64:, 0] = 0x78                                  # 256
    one = torch.full((M, 1), 127, dtype=torch.uint8).view(SCALE).cuda()
    big = torch.full((1, 1), 127, dtype=torch.uint8).view(SCALE).cuda()
    y = tb.tb_gated_e4m3(tb.E4M3Rows(x.view(CODE).cuda(), one), tb.E4M3Weight(w1.view(CODE).cuda(), big),
                         tb.E4M3Weight(w3.view(CODE).cuda(), big), out_dtype=tb.TB_F32)
    no_error()
    gates = ref.VALUES[w1[:, 0].numpy()]
    with np.errstate(over="ignore"):
        want = ref.silu(gates)
    assert (np.abs(f64(y) - want[None]) <= 8 * 2.0 ** -24 * np.abs(want) + 2.0 ** -126).all()


def test_empty_calls():
    w = make_weight(tb, 32, 64, gen(1))
    x = tb.E4M3Rows.empty(0, 64)
    assert tb.tb_gemm_e4m3(x, w).shape == (0, 32)
    assert tb.tb_gated_e4m3(x, w, w).rows == 0
    assert tb.tb_gated_e4m3(x, w, w, out_dtype=tb.TB_BF16).shape == (0, 32)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    assert tb.tb_quant_e4m3(e).rows == 0
    out, h = tb.tb_rmsnorm_e4m3(e, torch.ones(64, dtype=BF16, device="cuda"), 1e-5, r=e)
    assert out.rows == 0 and h.shape == (0, 64)
    no_error()


# ---- each width of tile, several tiles of rows ---------------------------------------

@pytest.mark.parametrize("tile", [16, 32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 272, 400), (131, 144, 2064), (300, 400, 640), (129, 128, 9216)])
def test_gemm_tiles(form, tile, M, N, K):
    form(tile)
    g = gen(M + N + K)
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    for dtype, with_res in ((F32, True), (BF16, False), (BF16, True)):
        res = (torch.randn(M, N, generator=g) * 100).to(dtype).cuda() if with_res else None
        buf = torch.full((M + 4, N), 7.0, dtype=dtype, device="cuda")
        y = tb.tb_gemm_e4m3(x, w, res=res, y=buf[2:2 + M])
        no_error()
        assert (buf[:2] == 7).all() and (buf[2 + M:] == 7).all()
        check_product(y, *product(rows_np(x), weight_np(w), None if res is None else f64(res)), K, dtype)


@pytest.mark.parametrize("tile", [16, 32, 64])
@pytest.mark.parametrize("M,F,K", [(1, 272, 400), (131, 144, 2064), (300, 400, 640), (70, 128, 9216)])
def test_gated_tiles(form, tile, M, F, K):
    form(tile)
    g = gen(M + F + K)
    x, w1, w3 = make_rows(tb, M, K, g), make_weight(tb, F, K, g), make_weight(tb, F, K, g)
    w1.scale.view(torch.uint8).sub_(int(np.log2(K) / 2) + 11)
    exact, off = gated_and_off(rows_np(x), weight_np(w1), weight_np(w3), K)
    buf = torch.full((M + 4, F), 9, dtype=torch.uint8, device="cuda")
    sc = torch.full((M + 4, -(-F // 128)), 9, dtype=torch.uint8, device="cuda")
    out = tb.tb_gated_e4m3(x, w1, w3, out=tb.E4M3Rows(buf[2:2 + M].view(CODE), sc[2:2 + M].view(SCALE)))
    no_error()
    for t in (buf, sc):
        assert (t[:2] == 9).all() and (t[2 + M:] == 9).all()
    check_rows(bytes_of(out.codes), bytes_of(out.scale), exact, off)
    y = tb.tb_gated_e4m3(x, w1, w3, out_dtype=tb.TB_F32)
    no_error()
    assert (np.abs(f64(y) - exact) <= off + 2 * HALF[F32] * (np.abs(exact) + off)).all()


# ---- many rows ----------------------------------------------------------------------
# One row to some tiles per cluster (both accumulators, more tiles than clusters), a row
# unit whose second half lies past M, K of one set and of an odd number of them.

MANY = [(1, 16, 16), (128, 256, 128), (129, 272, 144), (256, 512, 512), (300, 112, 2064), (400, 2304, 640), (511, 784, 1168),
        (1371, 2304, 768), (700, 8192, 400), (5000, 1040, 272), (260, 256, 9216)]


@pytest.mark.parametrize("tile", [-1, -2])
@pytest.mark.parametrize("M,N,K", MANY)
@pytest.mark.parametrize("dtype,with_res", [(F32, False), (BF16, False), (BF16, True), (F32, True)])
def test_gemm_many(form, tile, M, N, K, dtype, with_res):
    form(tile)
    g = gen(M + N + K)
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    res = (torch.randn(M, N, generator=g) * 100).to(dtype).cuda() if with_res else None
    buf = torch.full((M + 4, N), 7.0, dtype=dtype, device="cuda")
    y = tb.tb_gemm_e4m3(x, w, res=res, y=buf[2:2 + M])
    no_error()
    assert (buf[:2] == 7).all() and (buf[2 + M:] == 7).all()
    check_product(y, *product(rows_np(x), weight_np(w), None if res is None else f64(res)), K, dtype)
    if with_res:
        assert torch.equal(tb.tb_gemm_e4m3(x, w, res=res, y=res), y)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tile", [-1, -2])
def test_gemm_many_past_l2(form, tile, dtype):
    """Results too large to stay in L2 take their own cache hints."""
    form(tile)
    g = gen(6)
    M, N, K = 9001, 4112, 144
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    res = (torch.randn(M, N, generator=g) * 100).to(dtype).cuda()
    y = tb.tb_gemm_e4m3(x, w, res=res)
    no_error()
    check_product(y, *product(rows_np(x), weight_np(w), f64(res)), K, dtype)
    assert torch.equal(tb.tb_gemm_e4m3(x, w, res=res, y=res), y)


@pytest.mark.parametrize("M,F,K", [(1, 16, 16), (129, 144, 400), (333, 2048, 768), (300, 272, 2064), (1000, 1040, 528),
                                   (2100, 1296, 272)])
@pytest.mark.parametrize("out_dtype", ["codes", BF16, F32])
@pytest.mark.parametrize("tile", [-1, -2])
def test_gated_many(form, tile, M, F, K, out_dtype):
    form(tile)
    g = gen(M + F + K)
    x, w1, w3 = make_rows(tb, M, K, g), make_weight(tb, F, K, g), make_weight(tb, F, K, g)
    w1.scale.view(torch.uint8).sub_(int(np.log2(K) / 2) + 11)
    exact, off = gated_and_off(rows_np(x), weight_np(w1), weight_np(w3), K)
    if out_dtype == "codes":
        buf = torch.full((M + 4, F), 9, dtype=torch.uint8, device="cuda")
        sc = torch.full((M + 4, -(-F // 128)), 9, dtype=torch.uint8, device="cuda")
        out = tb.tb_gated_e4m3(x, w1, w3, out=tb.E4M3Rows(buf[2:2 + M].view(CODE), sc[2:2 + M].view(SCALE)))
        no_error()
        for t in (buf, sc):
            assert (t[:2] == 9).all() and (t[2 + M:] == 9).all()
        check_rows(bytes_of(out.codes), bytes_of(out.scale), exact, off)
    else:
        y = tb.tb_gated_e4m3(x, w1, w3, out_dtype=tb.TB_F32 if out_dtype is F32 else tb.TB_BF16)
        no_error()
        assert (np.abs(f64(y) - exact) <= off + 2 * HALF[out_dtype] * (np.abs(exact) + off)).all()


def test_both_kernels_agree_on_what_nan_reaches(form):
    g = gen(9)
    M, N, K = 300, 272, 528
    x, w = make_rows(tb, M, K, g), make_weight(tb, N, K, g)
    x.codes.view(torch.uint8)[3, 100] = 0x7F
    x.scale.view(torch.uint8)[266, 4] = 255
    w.codes.view(torch.uint8)[5, 527] = 0xFF
    w.scale.view(torch.uint8)[2, 1] = 255
    got = []
    for f in (16, 32, 64, 128, -1, -2):
        form(f)
        got.append(torch.isnan(tb.tb_gemm_e4m3(x, w)))
    no_error()
    hit = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    hit[3], hit[266], hit[:, 5], hit[:, 256:] = True, True, True, True
    assert all(torch.equal(t, hit) for t in got)


# ---- offsets beyond 32 bits -----------------------------------------------------------

def test_rows_beyond_2_31_values():
    M, d = 540_000, 4096                               # 2.2e9 values
    x = torch.ones(M, d, dtype=BF16, device="cuda")
    x[-3:] = torch.randn(3, d, generator=gen(1)).to(BF16)
    r = torch.zeros(M, d, dtype=BF16, device="cuda")
    r[-2] = 0.5
    out = tb.tb_quant_e4m3(x)
    no_error()
    check_rows(bytes_of(out.codes[-4:]), bytes_of(out.scale[-4:]), f64(x[-4:]), np.zeros((4, d)))
    tb.tb_rmsnorm_e4m3(x, torch.ones(d, dtype=BF16, device="cuda"), 1e-5, r=r, h=r, out=out)
    no_error()
    total = f64(x[-4:])
    total[2] += 0.5
    y = ref.norm(total, np.ones(d), 1e-5)
    check_rows(bytes_of(out.codes[-4:]), bytes_of(out.scale[-4:]), y, NORM_OFF * np.abs(y))
    assert (np.abs(f64(r[-4:]) - total) <= 2 * HALF[BF16] * np.abs(total) + 2.0 ** -23 * np.abs(total)).all()


@pytest.mark.parametrize("tile", [64, -1, -2])
def test_products_beyond_2_31_values(form, tile):
    form(tile)
    g = gen(4)
    M, N, K = 140_000, 16_000, 144                     # 2.24e9 results
    few = make_rows(tb, 1000, K, g)
    x = tb.E4M3Rows(few.codes.view(torch.uint8).repeat(140, 1).view(CODE), few.scale.view(torch.uint8).repeat(140, 1).view(SCALE))
    w = make_weight(tb, N, K, g)
    y = tb.tb_gemm_e4m3(x, w)
    no_error()
    want = y[:1000]
    check_product(want[:8], *product(rows_np(few)[:8], weight_np(w)), K, BF16)
    for i in (1, 70, 138, 139):
        assert torch.equal(y[1000 * i:1000 * (i + 1)], want)
    del y
    a = tb.tb_gated_e4m3(x, w, w)
    no_error()
    c, s = a.codes.view(torch.uint8), a.scale.view(torch.uint8)
    for i in (1, 70, 138, 139):
        assert torch.equal(c[1000 * i:1000 * (i + 1)], c[:1000]) and torch.equal(s[1000 * i:1000 * (i + 1)], s[:1000])
    exact, off = gated_and_off(rows_np(few)[:4], weight_np(w), weight_np(w), K)
    check_rows(bytes_of(a.codes[:4]), bytes_of(a.scale[:4]), exact, off)


# ---- together -----------------------------------------------------------------------

def test_repeated_calls_streams_and_graphs_give_the_same_bits():
    g = gen(11)
    M, d, f = 40, 512, 1040
    x = torch.randn(M, d, generator=g).to(BF16).cuda()
    gain = torch.ones(d, dtype=BF16, device="cuda")
    w1, w3, w2 = (tb.tb_pack_e4m3((0.05 * torch.randn(*s, generator=g)).to(BF16).cuda()) for s in ((d, f), (d, f), (f, d)))
    n, a, y = tb.E4M3Rows.empty(M, d), tb.E4M3Rows.empty(M, f), torch.empty_like(x)

    def mlp(stream=None):
        tb.tb_rmsnorm_e4m3(x, gain, 1e-5, out=n, stream=stream)
        tb.tb_gated_e4m3(n, w1, w3, out=a, stream=stream)
        return tb.tb_gemm_e4m3(a, w2, res=x, y=y, stream=stream)

    first = mlp().clone()
    for _ in range(3):
        assert torch.equal(mlp(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y.zero_()
    torch.cuda.synchronize()
    mlp(side)
    side.synchronize()
    assert torch.equal(y, first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mlp()
    x2 = x.flip(0).contiguous()
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first.flip(0))               # rows do not know each other
    no_error()


@pytest.mark.parametrize("M", [3, 700])
def test_two_streams_at_once(M):
    """No call leaves anything behind that another one uses."""
    g = gen(21)
    K, N = 1040, 2064
    w, w3 = make_weight(tb, N, K, g), make_weight(tb, N, K, g)
    xs = [make_rows(tb, M, K, g) for _ in range(2)]
    want = [(tb.tb_gemm_e4m3(x, w), tb.tb_gated_e4m3(x, w, w3, out_dtype=tb.TB_BF16)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            got[i].append((tb.tb_gemm_e4m3(xs[i], w, stream=s), tb.tb_gated_e4m3(xs[i], w, w3, out_dtype=tb.TB_BF16, stream=s)))
    torch.cuda.synchronize()
    no_error()
    for i in range(2):
        for a, b in got[i]:
            assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])


def test_first_calls_of_a_process_inside_a_capture():
    """Nothing of the launches' set-up is forbidden while a graph is captured."""
    code = """
import torch, causal_gqa_attention_rmsnorm_gb300 as tb
x = torch.randn(300, 512, device="cuda").to(torch.bfloat16)
g = torch.ones(512, dtype=torch.bfloat16, device="cuda")
w = torch.randn(512, 4112, device="cuda") * .05
def go():
    n, _ = tb.tb_rmsnorm_e4m3(x, g, 1e-5)
    p = tb.tb_pack_e4m3(w)
    return tb.tb_gemm_e4m3(n, p), tb.tb_gated_e4m3(n, p, p, out_dtype=tb.TB_BF16), tb.tb_gemm_e4m3(tb.tb_quant_e4m3(x[:3]), p)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = go()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, go()))
assert tb.tb_get_device_error() == 0
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.stdout.strip().endswith("fine"), r.stderr[-2000:]


@pytest.mark.parametrize("B,n", [(3, 1), (2, 37)])
def test_a_decoder_layer_in_8_bits(B, n):
    """Norm, projection, append with rotation, attention, quantisation, projection onto
    the stream, norm, gated half, projection onto the stream, over an e4m3 cache: each
    step against fp64 on the very inputs that it got."""
    H, Hkv, dh, f, T = 8, 2, 64, 1040, 256
    d, M = H * dh, B * n
    g = gen(B * n)
    x = torch.randn(M, d, generator=g).to(BF16).cuda()
    gains = [(1 + 0.1 * torch.randn(d, generator=g)).to(BF16).cuda() for _ in range(2)]
    shapes = dict(qkv=(d, (H + 2 * Hkv) * dh), o=(d, d), w1=(d, f), w3=(d, f), w2=(f, d))
    w = {k: tb.tb_pack_e4m3((0.05 * torch.randn(*s, generator=g)).to(BF16).cuda()) for k, s in shapes.items()}
    rope = tb.tb_rope_table(dh, T, 1e4)
    kv = tb.KVCache.empty_e4m3(B, Hkv, T, dh, 64)
    cfg = tb.AttnConfig(H=H, Hkv=Hkv, dh=dh)

    n1, _ = tb.tb_rmsnorm_e4m3(x, gains[0], 1e-5)
    qkv = tb.tb_gemm_e4m3(n1, w["qkv"])
    q, k, v = qkv.view(B, n, -1, dh).split([H, Hkv, Hkv], 2)
    qr = tb.tb_kvcache_append_rope(kv, k, v, rope, q=q)
    o = tb.tb_kvcache_attn(cfg, qr, kv)
    o8 = tb.tb_quant_e4m3(o.view(M, d))
    branch = tb.tb_gemm_e4m3(o8, w["o"])
    n2, h = tb.tb_rmsnorm_e4m3(x, gains[1], 1e-5, r=branch)
    a = tb.tb_gated_e4m3(n2, w["w1"], w["w3"])
    y = tb.tb_gemm_e4m3(a, w["w2"], res=h)
    no_error()

    z = ref.norm(f64(x), f64(gains[0]), 1e-5)
    check_rows(bytes_of(n1.codes), bytes_of(n1.scale), z, NORM_OFF * np.abs(z))
    check_product(qkv, *product(rows_np(n1), weight_np(w["qkv"])), d, BF16)
    check_rows(bytes_of(o8.codes), bytes_of(o8.scale), f64(o).reshape(M, d), np.zeros((M, d)))
    check_product(branch, *product(rows_np(o8), weight_np(w["o"])), d, BF16)
    total = f64(x) + f64(branch)
    assert (np.abs(f64(h) - total) <= 2 * HALF[BF16] * np.abs(total) + 2.0 ** -23 * np.abs(total)).all()
    z = ref.norm(total, f64(gains[1]), 1e-5)
    check_rows(bytes_of(n2.codes), bytes_of(n2.scale), z, NORM_OFF * np.abs(z))
    exact, off = gated_and_off(rows_np(n2), weight_np(w["w1"]), weight_np(w["w3"]), d)
    check_rows(bytes_of(a.codes), bytes_of(a.scale), exact, off)
    check_product(y, *product(rows_np(a), weight_np(w["w2"]), f64(h)), f, BF16)

"""The 8-bit projections at the ends of what they accept, against fp64 (e4m3_helpers
derives the tolerances)."""
import numpy as np
import pytest
import torch

import causal_gqa_attention_rmsnorm_gb300 as tb
from e4m3_helpers import (BF16, CODE, F32, HALF, SCALE, bytes_of, check_product, check_rows, gated_and_off, make_rows, make_weight,
                          product, rows_np, weight_np)
from oracle import e4m3 as ref
from test_gpu_e4m3_ops import MANY_ROWS, NORM_OFF, f64, form, gen, no_error  # noqa: F401 (form is a fixture)

pytestmark = pytest.mark.gpu


# ---- the norm of rows near zero -----------------------------------------------------

# The root mean squares of the rows, in turn: s = 1 / sqrt(mean square) is 2^28 at 3.7e-9.
SMALL = [1.0, 1e-10, 3.3e-9, 4.2e-9, 1e-15, 1e-12]


@pytest.mark.parametrize("M,d,dtype,r_dtype", [(6, 256, BF16, None), (6, 528, F32, None), (7, 4096, BF16, BF16), (6, 1040, F32, F32),
                                               (9, 4096, F32, BF16), (6, 11008, BF16, F32)] + MANY_ROWS)
@pytest.mark.parametrize("eps", [0.0, 1e-20])
def test_norm_of_rows_near_zero(M, d, dtype, r_dtype, eps):
    """Finite rows give finite codes: blocks of zeros, zeros among values, blocks whose gains
    are 0 or next to it, and whole rows of zeros where eps is positive."""
    g = gen(M + d)
    x = torch.randn(M, d, generator=g) * torch.tensor([SMALL[m % len(SMALL)] for m in range(M)])[:, None]
    gain = 1 + 0.1 * torch.randn(d, generator=g)
    last = (d - 1) // 128 * 128
    x[1::2, :128] = 0                                  # a block of zeros
    x[::2, 3:40] = 0                                   # zeros in a block
    if d > 512:
        gain[128:256] = 0
        gain[256:384] = 1e-28                          # times rows of 1e-15: v·g is subnormal, v·s·g is not
        x[:, 384:512] *= 2.0 ** -60
    if last >= 512:
        gain[last + 5:] = 0
    if eps > 0:
        x[2] = 0
    x = x.to(dtype).cuda()
    gain = gain.to(dtype).cuda()
    r = None
    if r_dtype is not None:
        r = (torch.randn(M, d, generator=g) * x.float().cpu().abs()).to(r_dtype).cuda()
    out, _ = tb.tb_rmsnorm_e4m3(x, gain, eps, r=r)
    no_error()
    total = f64(x) + (0 if r is None else f64(r))
    y = ref.norm(total, f64(gain), eps)
    assert np.isfinite(y).all()
    # v·g may round below fp32's normal numbers, by 2^-150, before an s of less than 2^28
    check_rows(bytes_of(out.codes), bytes_of(out.scale), y, NORM_OFF * np.abs(y) + 2.0 ** -122)


# ---- the largest counts -------------------------------------------------------------

def test_pack_of_the_most_columns():
    """Columns counted past 31 bits on the way: the first and the last of each step of the
    grid, and zeros everywhere else."""
    K, N = 16, 2 ** 31 - 1024
    w = torch.zeros(K, N, dtype=BF16, device="cuda")
    step = 65535 * 128
    places = sorted({0, 127, 128, step - 1, step, 100 * step + 3, 255 * step, 256 * step - 128, 256 * step, N - 129, N - 1})
    places = [p for p in places if p < N]
    v = torch.randn(K, len(places), generator=gen(1)).to(BF16).cuda()
    for i, p in enumerate(places):
        w[:, p] = v[:, i]
    codes = torch.full((N, K), 9, dtype=torch.uint8, device="cuda")
    scale = torch.full((-(-N // 128), 1), 9, dtype=torch.uint8, device="cuda")
    tb.tb_pack_e4m3(w, out=tb.E4M3Weight(codes.view(CODE), scale.view(SCALE)))
    no_error()
    e = np.array([ref.exponent(f64(w[:, p // 128 * 128:p // 128 * 128 + 128])) for p in places])
    assert (scale.cpu().numpy()[[p // 128 for p in places], 0].astype(int) - 127 == e).all()
    for i, p in enumerate(places):
        q = f64(v[:, i]) / 2.0 ** e[i]
        assert (np.abs(ref.VALUES[codes[p].cpu().numpy()] - q) <= ref.half_step(q)).all()
        codes[p] = 0
        scale[p // 128] = 27
    assert (scale == 27).all()
    for i in range(0, N, 2 ** 27):
        assert not codes[i:i + 2 ** 27].any()


# ---- long sums ----------------------------------------------------------------------
#
# The tensor core cuts its sums off.  In an accumulator of 64 instructions a sum of
# magnitudes S is off by at most (2·64 + 8)·2^-23·S (e4m3_helpers), and the parts are added
# with rounding, 2^-24 of what is summed up for each:

def in_parts(K):
    return (2 * 64 + 8) * 2.0 ** -23 + -(-K // 2048) * 2.0 ** -24


def one_sign(n, K, g, device="cuda"):
    """Codes of |N(0, 1)| times 40."""
    return (torch.randn(n, K, generator=g, device=device) * 40).abs().clamp(max=448).to(CODE)


def flat_scales(shape, e):
    return torch.full(shape, 127 + e, dtype=torch.uint8, device="cuda").view(SCALE)


def exact_product(x, w):
    """Of codes, in fp64 on the GPU, some columns of K at a time (for which every sum is exact
    but for fp64's own rounding)."""
    y = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for k in range(0, x.shape[1], 1 << 15):
        y += x[:, k:k + (1 << 15)].double() @ w[:, k:k + (1 << 15)].double().T
    return y


def check_between(got, exact, off):
    """got is a rounding, to its type, of a value within the factor 1 +- off of exact (> 0)."""
    low, high = (exact * (1 - off)).to(got.dtype), (exact * (1 + off)).to(got.dtype)
    bad = ~((got >= low) & (got <= high))
    assert not bad.any(), (int(bad.sum()), bad.numel(), ((got.double() - exact) / exact)[bad][:4].tolist())


def test_gemm_of_a_very_long_sum():
    """Values of one sign, whose cut-off sums are all off in the same direction: bf16 results
    are those of sums in parts (one accumulator comes out 2.5e-3 low, which is more than half
    a step)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    M, N, K = 1030, 2560, 1 << 20
    xc, wc = one_sign(M, K, g), one_sign(N, K, g)
    x = tb.E4M3Rows(xc, flat_scales((M, K // 128), -8))
    w = tb.E4M3Weight(wc, flat_scales((N // 128, K // 128), -8))
    y = tb.tb_gemm_e4m3(x, w)
    no_error()
    rows = [0, 1, 127, 128, 500, 1023, 1024, 1029]
    check_between(y[rows], exact_product(xc[rows], wc) * 2.0 ** -16, in_parts(K))


@pytest.mark.parametrize("out_dtype", [BF16, "codes"])
def test_gated_of_very_long_sums(out_dtype):
    """The same for gates of hundreds, where SiLU is the gate itself."""
    g = torch.Generator(device="cuda").manual_seed(4)
    M, F, K = 300, 2048, 1 << 20
    xc, wc, vc = one_sign(M, K, g), one_sign(F, K, g), one_sign(F, K, g)
    x = tb.E4M3Rows(xc, flat_scales((M, K // 128), -10))
    w1, w3 = (tb.E4M3Weight(c, flat_scales((F // 128, K // 128), -10)) for c in (wc, vc))
    out = tb.tb_gated_e4m3(x, w1, w3, out_dtype=tb.TB_BF16 if out_dtype is BF16 else None)
    no_error()
    rows = [0, 127, 128, 255, 256, 299]
    a, b = exact_product(xc[rows], wc) * 2.0 ** -20, exact_product(xc[rows], vc) * 2.0 ** -20
    assert a.min() > 200                              # SiLU(a) = a to 1e-80
    off = 2.01 * in_parts(K) + 8 * 2.0 ** -24
    if out_dtype is BF16:
        check_between(out[rows], a * b, off)
    else:
        y = (a * b).cpu().numpy()
        check_rows(bytes_of(out.codes[rows]), bytes_of(out.scale[rows]), y, off * y)


def off_by(y, exact):
    """The largest deviation of fp32 results (> 0), less half a step, relative to exact."""
    return (((y.double() - exact).abs() - 2 * HALF[F32] * exact) / exact).max().item()


@pytest.mark.parametrize("tile", [0, 16, 32, 64, 128])
@pytest.mark.parametrize("K", [14336, 65536])
def test_fp32_sums_are_formed_in_parts(form, tile, K):
    """Of one sign: the bound, 1.7e-5, is a quarter of what one of 14336 terms is worth, and a third
    of what one accumulator loses at 65536 (5.0e-5)."""
    g = torch.Generator(device="cuda").manual_seed(K)
    M, N = 1030, 2560
    xc, wc = one_sign(M, K, g), one_sign(N, K, g)
    x, w = tb.E4M3Rows(xc, flat_scales((M, K // 128), -8)), tb.E4M3Weight(wc, flat_scales((N // 128, K // 128), -8))
    exact = exact_product(xc, wc) * 2.0 ** -16
    form(tile)
    y = tb.tb_gemm_e4m3(x, w, y_dtype=tb.TB_F32)
    res = torch.zeros_like(y)
    with_res = tb.tb_gemm_e4m3(x, w, res=res)
    no_error()
    assert off_by(y, exact) <= in_parts(K) and off_by(with_res, exact) <= in_parts(K)


@pytest.mark.parametrize("tile", [0, 16, 32, 64])
@pytest.mark.parametrize("K", [14336, 65536])
def test_gated_fp32_sums_are_formed_in_parts(form, tile, K):
    g = torch.Generator(device="cuda").manual_seed(K + 1)
    M, F = 300, 2048
    xc, wc, vc = one_sign(M, K, g), one_sign(F, K, g), one_sign(F, K, g)
    x = tb.E4M3Rows(xc, flat_scales((M, K // 128), -7))
    w1, w3 = (tb.E4M3Weight(c, flat_scales((F // 128, K // 128), -8)) for c in (wc, vc))
    a, b = exact_product(xc, wc) * 2.0 ** -15, exact_product(xc, vc) * 2.0 ** -15
    assert a.min() > 200                              # SiLU(a) = a to 1e-80
    off = 2.01 * in_parts(K) + 8 * 2.0 ** -24
    form(tile)
    y = tb.tb_gated_e4m3(x, w1, w3, out_dtype=tb.TB_F32)
    no_error()
    assert off_by(y, a * b) <= off


# ---- weights that were written just ahead ---------------------------------------------

@pytest.mark.parametrize("M", [1, 20, 300])
def test_weights_packed_just_ahead_are_the_ones_used(M):
    """Set after set into the same tensors, by packing, and by copies outside the library,
    with nothing between them and the product, or other calls of the library."""
    g = torch.Generator(device="cuda").manual_seed(M)
    K, N, sets = 512, 2048, 12
    x = tb.tb_quant_e4m3(torch.randn(M, K, generator=g, device="cuda"))
    ws = [torch.randn(K, N, generator=g, device="cuda").to(BF16) for _ in range(sets)]
    packed = [tb.tb_pack_e4m3(w) for w in ws]
    torch.cuda.synchronize()
    want = [tb.tb_gemm_e4m3(x, p) for p in packed]
    gated = [tb.tb_gated_e4m3(x, p, p, out_dtype=tb.TB_BF16) for p in packed]
    torch.cuda.synchronize()
    w8 = tb.E4M3Weight.empty(N, K)
    other = torch.randn(64, K, generator=g, device="cuda")
    got = []
    for _ in range(4):
        for i in range(sets):
            tb.tb_pack_e4m3(ws[i], out=w8)
            if i % 3 == 1:
                tb.tb_quant_e4m3(other)
            got.append((tb.tb_gemm_e4m3(x, w8), want[i]))
            w8.codes.view(torch.uint8).copy_(packed[i - 1].codes.view(torch.uint8))
            w8.scale.view(torch.uint8).copy_(packed[i - 1].scale.view(torch.uint8))
            if i % 3 == 2:
                tb.tb_quant_e4m3(other)
            got.append((tb.tb_gated_e4m3(x, w8, w8, out_dtype=tb.TB_BF16), gated[i - 1]))
    torch.cuda.synchronize()
    no_error()
    assert all(torch.equal(a, b) for a, b in got)


# ---- weights beyond L2, whose tiles go in groups ----------------------------------------

def repeated_rows(M, P, K, g):
    """M rows of which P differ, P odd and no part of a tile: row m is row m % P."""
    few = make_rows(tb, P, K, g)
    n = -(-M // P)
    x = tb.E4M3Rows(few.codes.view(torch.uint8).repeat(n, 1)[:M].contiguous().view(CODE),
                    few.scale.view(torch.uint8).repeat(n, 1)[:M].contiguous().view(SCALE))
    return few, x


def all_repeat(t, P):
    u = t.view(torch.uint8) if t.element_size() == 1 else t
    for i in range(0, u.shape[0], P):
        if not torch.equal(u[i:i + P], u[:min(P, u.shape[0] - i)]):
            return False
    return True


@pytest.mark.parametrize("tile", [0, -1, -2])
@pytest.mark.parametrize("M", [257, 8453])
def test_gemm_of_large_weights(form, tile, M):
    """More than 48 MB of weights and K up to 8192: tiles in groups of 32 units of rows, the
    last group smaller, the last unit and the last column tile partly filled."""
    form(tile)
    g = gen(M)
    N, K, P = 24592, 2064, 97
    few, x = repeated_rows(M, P, K, g)
    w = make_weight(tb, N, K, g)
    for dtype in (BF16, F32):
        res = (torch.randn(P, N, generator=g) * 100).to(dtype).cuda()
        y = tb.tb_gemm_e4m3(x, w, res=res.repeat(-(-M // P), 1)[:M].contiguous())
        no_error()
        check_product(y[:P], *product(rows_np(few), weight_np(w), f64(res)), K, dtype)
        assert all_repeat(y, P)


@pytest.mark.parametrize("tile", [0, -1, -2])
@pytest.mark.parametrize("M,out_dtype", [(257, "codes"), (8453, "codes"), (8453, BF16)])
def test_gated_of_large_weights(form, tile, M, out_dtype):
    form(tile)
    g = gen(M + 1)
    F, K, P = 12400, 2064, 97
    few, x = repeated_rows(M, P, K, g)
    w1, w3 = make_weight(tb, F, K, g), make_weight(tb, F, K, g)
    w1.scale.view(torch.uint8).sub_(int(np.log2(K) / 2) + 11)
    exact, off = gated_and_off(rows_np(few), weight_np(w1), weight_np(w3), K)
    out = tb.tb_gated_e4m3(x, w1, w3, out_dtype=None if out_dtype == "codes" else tb.TB_BF16)
    no_error()
    if out_dtype == "codes":
        check_rows(bytes_of(out.codes[:P]), bytes_of(out.scale[:P]), exact, off)
        assert all_repeat(out.codes, P) and all_repeat(out.scale, P)
    else:
        assert (np.abs(f64(out[:P]) - exact) <= off + 2 * HALF[BF16] * (np.abs(exact) + off)).all()
        assert all_repeat(out, P)


# ---- gates far from zero, to bf16 and codes ----------------------------------------------

@pytest.mark.parametrize("tile", [16, 32, 64, -1, -2])
@pytest.mark.parametrize("out_dtype", [BF16, "codes"])
@pytest.mark.parametrize("up", [0, 40])
def test_far_gates_to_few_bits(form, tile, out_dtype, up):
    """Gates of every size a code has, of both signs, up to 7168, those below zero also in a
    block of their own from 0 to -112.  SiLU's short form has 2^x of an argument rounded by up to
    |g|·2^-23 of its effect and two functions within 2^-21 together; below -87, where it is
    under 1e-35, it may be 0."""
    form(tile)
    M, F, K = 140, 384, 128
    x = torch.zeros(M, K, dtype=torch.uint8)
    x[:, 0] = 0x38
    w1, w3 = torch.zeros(F, K, dtype=torch.uint8), torch.zeros(F, K, dtype=torch.uint8)
    size = torch.arange(128, dtype=torch.uint8).clamp(max=126)
    w1[:128, 0], w1[128:256, 0], w1[256:, 0], w3[:, 0] = size + 128, size + 128, size, 0x38
    s1 = torch.tensor([[125], [131], [131]], dtype=torch.uint8)
    out = tb.tb_gated_e4m3(tb.E4M3Rows(x.view(CODE).cuda(), flat_scales((M, 1), 0)), tb.E4M3Weight(w1.view(CODE).cuda(), s1.view(SCALE).cuda()),
                           tb.E4M3Weight(w3.view(CODE).cuda(), flat_scales((3, 1), up)), out_dtype=tb.TB_BF16 if out_dtype is BF16 else None)
    no_error()
    gates = ref.VALUES[w1[:, 0].numpy()] * np.repeat([0.25, 16.0, 16.0], 128)
    with np.errstate(over="ignore"):
        want = np.tile(ref.silu(gates) * 2.0 ** up, (M, 1))
    assert np.isfinite(want).all() and (gates == -112).any() and (gates == 7168).any()
    off = (np.abs(gates) * 2.0 ** -23 + 2.0 ** -21) * np.abs(want) + 1e-35 * 2.0 ** up
    if out_dtype is BF16:
        assert (np.abs(f64(out) - want) <= off + 2 * HALF[BF16] * (np.abs(want) + off)).all()
    else:
        check_rows(bytes_of(out.codes), bytes_of(out.scale), want, off)


# ---- beside other calls ---------------------------------------------------------------

def test_products_beside_a_decode_step():
    """On two streams at once: steps of the bf16 block over its cache, and 8-bit products of
    every form that takes tensor memory in another amount."""
    import workloads
    from helpers import block_config, to_device
    s = workloads.BlockShape("beside", "decode", "bf16", B=4, T=512, d=1024, H=8, Hkv=2, dh=128, f=4096, rope_base=5e5, eps=1e-5,
                             gains="normal")
    inp = workloads.make_block_inputs(s, seed=3)
    lens0 = torch.tensor([5, 100, 300, 500], dtype=torch.int32).cuda()
    kc, vc = workloads.make_decode_cache(s, 3, lens0.cpu(), fill=0.0, device="cuda")
    kv, cfg, dev = tb.KVCache(kc, vc, lens0.clone()), block_config(s, max_pos=512), to_device(inp)
    packed = tb.tb_pack_weights(cfg, dev)
    g = gen(8)
    calls = []
    for M, N, K, y in ((3, 2064, 4112, F32), (40, 4096, 4608, F32), (100, 2560, 1024, BF16), (300, 2304, 768, BF16)):
        x, w, w3 = make_rows(tb, M, K, g), make_weight(tb, N, K, g), make_weight(tb, N, K, g)
        dt = tb.TB_F32 if y is F32 else tb.TB_BF16
        calls.append(lambda x=x, w=w, dt=dt: tb.tb_gemm_e4m3(x, w, y_dtype=dt))
        calls.append(lambda x=x, w=w, w3=w3, dt=dt: tb.tb_gated_e4m3(x, w, w3, out_dtype=dt))

    def step():
        kv.lens.copy_(lens0)
        return tb.tb_block_decode(cfg, packed, dev["x"], kv)

    want_step, want = step(), [c() for c in calls]
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    steps, got = [], []
    for _ in range(8):
        with torch.cuda.stream(a):
            steps += [step() for _ in range(4)]
        with torch.cuda.stream(b):
            got += [(c(), w) for c, w in zip(calls, want)]
    torch.cuda.synchronize()
    no_error()
    assert all(torch.equal(y, want_step) for y in steps) and all(torch.equal(y, w) for y, w in got)

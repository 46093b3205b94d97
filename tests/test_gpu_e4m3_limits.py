"""The 8-bit projections at the ends of what they accept, against fp64 (e4m3_helpers
derives the tolerances)."""
import numpy as np
import pytest
import torch

import causal_gqa_attention_rmsnorm_gb300 as tb
from e4m3_helpers import BF16, CODE, F32, SCALE, bytes_of, check_rows
from oracle import e4m3 as ref
from test_gpu_e4m3_ops import MANY_ROWS, NORM_OFF, f64, gen, no_error

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

// C ABI of the 8-bit projections: argument checks and launches.  Declarations and
// contracts are in tb.h.
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "e4m3.cuh"
#include "gemm_tc.cuh"

namespace tb {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool is_float(int dtype) { return dtype == TB_F32 || dtype == TB_BF16; }
size_t esize(int dtype) { return dtype == TB_F32 ? 4 : dtype == TB_BF16 ? 2 : 1; }
long long blocks(long long n) { return (n + kBlk - 1) / kBlk; }

struct Range {
  const void* p;
  size_t n;
};
bool overlap(const Range& x, const Range& y) {
  const uintptr_t a = (uintptr_t)x.p, b = (uintptr_t)y.p;
  return x.p && y.p && a < b + y.n && b < a + x.n;
}
// Whether what is written overlaps anything read, or itself.
tb_status apart(const Range* w, int nw, const Range* r, int nr) {
  for (int i = 0; i < nw; ++i) {
    for (int j = 0; j < nr; ++j)
      if (overlap(w[i], r[j])) return report(TB_ERR_INVALID_ARG, "an output overlaps an input");
    for (int j = 0; j < i; ++j)
      if (overlap(w[i], w[j])) return report(TB_ERR_INVALID_ARG, "two outputs overlap");
  }
  return TB_OK;
}

// Shape of a matrix of codes; its pointers too with `tensors`.
tb_status check(const tb_e4m3* m, const char* name, bool tensors) {
  if (!m) return report(TB_ERR_INVALID_ARG, "%s is NULL", name);
  if (m->rows < 0 || m->cols <= 0) return report(TB_ERR_INVALID_ARG, "%s: cols must be positive, rows non-negative", name);
  if (m->cols % 16) return report(TB_ERR_UNSUPPORTED, "%s: cols (%d) must be a multiple of 16", name, m->cols);
  // (the kernels round both up to whole tiles, in 32 bits)
  if (m->rows > INT32_MAX - 1023 || m->cols > INT32_MAX - 1023)
    return report(TB_ERR_UNSUPPORTED, "%s: more than 2^31 - 1024 rows or cols", name);
  if ((long long)m->rows * m->cols > 1LL << 39) return report(TB_ERR_UNSUPPORTED, "%s: more than 2^39 codes", name);
  if (!tensors) return TB_OK;
  if (!m->codes || !m->scale) return report(TB_ERR_INVALID_ARG, "%s: codes and scale must be non-NULL", name);
  if (!aligned16(m->codes)) return report(TB_ERR_INVALID_ARG, "%s: codes must be 16-byte aligned", name);
  return TB_OK;
}
Range codes_of(const tb_e4m3* m) { return {m->codes, (size_t)m->rows * m->cols}; }
Range row_scales(const tb_e4m3* m) { return {m->scale, (size_t)m->rows * blocks(m->cols)}; }
Range weight_scales(const tb_e4m3* m) { return {m->scale, (size_t)(blocks(m->rows) * blocks(m->cols))}; }
Coded coded(const tb_e4m3* m) { return {static_cast<const uint8_t*>(m->codes), static_cast<const uint8_t*>(m->scale)}; }

tb_status check_in(const void* p, const char* name) {
  if (!p || !aligned16(p)) return report(TB_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", name);
  return TB_OK;
}

tb_status done(cudaError_t e, const char* fn) {
  return e == cudaSuccess ? TB_OK : report(TB_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
}

// Weights of a product with rows of K codes.
tb_status check_weights(const tb_e4m3* w, const char* name, const tb_e4m3* x, bool tensors) {
  const tb_status st = check(w, name, tensors);
  if (st != TB_OK) return st;
  if (w->rows <= 0) return report(TB_ERR_INVALID_ARG, "%s: rows must be positive", name);
  // (columns of the result are counted in bytes, in 32 bits)
  if (w->rows > 1 << 28) return report(TB_ERR_UNSUPPORTED, "%s: at most 2^28 rows (%d)", name, w->rows);
  if (w->rows % 16) return report(TB_ERR_UNSUPPORTED, "%s: rows (%d) must be a multiple of 16", name, w->rows);
  if (w->cols != x->cols)
    return report(TB_ERR_INVALID_ARG, "%s has %d columns, x has %d", name, w->cols, x->cols);
  return TB_OK;
}

// k_e4m3_many has one accumulator for all of K, k_e4m3_few one for each 2048 of it, added up
// with rounding.  The tensor core cuts its sums off, so that one accumulator is off the more
// the longer it is.  Measured against 64 bits, relative to the results' size, rows and weights
// of both signs / of one sign (there all of it in one direction):
//     K                  1024         2048         4096         14336        65536        2^20
//     one accumulator  5.4e-8/1.6e-7 1.0e-7/4.3e-7 2.1e-7/1.2e-6 9.8e-7/7.6e-6 7.6e-6/5.0e-5 3.0e-4/2.5e-3
//     parts of 2048    3.8e-8/7.3e-8 4.8e-8/7.3e-8 6.0e-8/7.5e-8 1.1e-7/3.6e-7 1.2e-7/4.1e-7 1.9e-7/4.1e-7
//     fp32 sums        3.9e-8/6.0e-8 5.7e-8/9.9e-8 5.8e-8/4.7e-8 8.2e-8/5.8e-8 1.7e-7/1.2e-7 3.0e-7/7.9e-7
// So an fp32 result is formed in parts beyond K = 4096, and one of bf16 or codes, half a step
// of which is 2e-3 or more, beyond K = 65536.
constexpr int kOneF32 = 4096, kOne16 = 65536;

// The rows per tile of k_e4m3_few, or 0 for k_e4m3_many, -1 with a CTA to a tile.
int rule(int M, int N, int K, int mats, int y_dtype, bool res, int sms) {
  const bool light = mats == 2 ? y_dtype != TB_E4M3 : y_dtype == TB_F32 && !res;
  const int tile = e4m3_few_tile(M, N, K, mats, light, sms);
  return tile > 0 || K <= (y_dtype == TB_F32 ? kOneF32 : kOne16) ? tile : mats == 2 ? 64 : 128;
}
std::atomic<int> g_form{0};            // test hook: 16 to 128 rows per tile, or -1 and -2 for many
int tile_of(const GemmArgs& a, int mats) {
  const int form = g_form.load(std::memory_order_relaxed);
  if (form) return form == -1 ? 0 : form == -2 ? -1 : mats == 2 && form > 64 ? 64 : form;
  return rule(a.M, a.N, a.K, mats, a.y_dtype, a.res != nullptr, sm_count());
}

RowsArgs rows_args(const void* x, const tb_e4m3* out) {
  RowsArgs a = {};
  a.x = x;
  a.M = out->rows;
  a.d = out->cols;
  a.codes = static_cast<uint8_t*>(out->codes);
  a.scale = static_cast<uint8_t*>(out->scale);
  return a;
}

}  // namespace
}  // namespace tb

using namespace tb;

#define TB_OR_RETURN(call)                 \
  do {                                     \
    const tb_status st_ = (call);          \
    if (st_ != TB_OK) return st_;          \
  } while (0)

extern "C" {

tb_status tb_rmsnorm_e4m3(const void* x, int32_t dtype, const void* r, int32_t r_dtype, void* h, const void* g,
                          float eps, const tb_e4m3* out, void* stream) {
  TB_OR_RETURN(check(out, "out", false));
  if (!is_float(dtype)) return report(TB_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (!(eps >= 0.f) || !isfinite(eps)) return report(TB_ERR_INVALID_ARG, "eps must be finite and non-negative");
  if (out->cols > kNormMax) return report(TB_ERR_UNSUPPORTED, "rows of at most %d columns (%d)", kNormMax, out->cols);
  if ((r == nullptr) != (h == nullptr)) return report(TB_ERR_INVALID_ARG, "r and h go together");
  if (r && !is_float(r_dtype)) return report(TB_ERR_INVALID_ARG, "unknown r_dtype %d", r_dtype);
  if (out->rows == 0) return TB_OK;
  TB_OR_RETURN(check(out, "out", true));
  TB_OR_RETURN(check_in(x, "x"));
  TB_OR_RETURN(check_in(g, "g"));
  const size_t n = (size_t)out->rows * out->cols;
  const Range rx = {x, n * esize(dtype)}, rg = {g, out->cols * esize(dtype)};
  const Range rr = {r, r ? n * esize(r_dtype) : 0}, rh = {h, n * esize(dtype)};
  if (r) {
    TB_OR_RETURN(check_in(r, "r"));
    TB_OR_RETURN(check_in(h, "h"));
    const bool on_x = h == x, on_r = h == r && dtype == r_dtype;
    if ((overlap(rh, rx) && !on_x) || (overlap(rh, rr) && !on_r) || overlap(rh, rg))
      return report(TB_ERR_INVALID_ARG, "h overlaps an input (it may be x itself, or r itself of the same type)");
  }
  const Range w[] = {codes_of(out), row_scales(out)}, in[] = {rx, rg, rr, rh};
  TB_OR_RETURN(apart(w, 2, in, 4));
  RowsArgs a = rows_args(x, out);
  a.r = r;
  a.h = h;
  a.g = g;
  a.eps = eps;
  return done(launch_norm_e4m3(a, dtype, r_dtype, (cudaStream_t)stream), "tb_rmsnorm_e4m3");
}

tb_status tb_quant_e4m3(const void* x, int32_t dtype, const tb_e4m3* out, void* stream) {
  TB_OR_RETURN(check(out, "out", false));
  if (!is_float(dtype)) return report(TB_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  // (pieces of at least 2048 columns are counted in the grid's second dimension)
  if (out->cols > 1 << 26) return report(TB_ERR_UNSUPPORTED, "rows of at most 2^26 columns (%d)", out->cols);
  if (out->rows == 0) return TB_OK;
  TB_OR_RETURN(check(out, "out", true));
  TB_OR_RETURN(check_in(x, "x"));
  const Range w[] = {codes_of(out), row_scales(out)}, in[] = {{x, (size_t)out->rows * out->cols * esize(dtype)}};
  TB_OR_RETURN(apart(w, 2, in, 1));
  return done(launch_quant_e4m3(rows_args(x, out), dtype, (cudaStream_t)stream), "tb_quant_e4m3");
}

tb_status tb_pack_e4m3(const void* w, int32_t dtype, const tb_e4m3* out, void* stream) {
  TB_OR_RETURN(check(out, "out", false));
  if (!is_float(dtype)) return report(TB_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (out->rows == 0) return TB_OK;
  TB_OR_RETURN(check(out, "out", true));
  TB_OR_RETURN(check_in(w, "w"));
  const Range o[] = {codes_of(out), weight_scales(out)}, in[] = {{w, (size_t)out->rows * out->cols * esize(dtype)}};
  TB_OR_RETURN(apart(o, 2, in, 1));
  return done(launch_pack_e4m3(w, dtype, out->cols, out->rows, static_cast<uint8_t*>(out->codes),
                               static_cast<uint8_t*>(out->scale), (cudaStream_t)stream),
              "tb_pack_e4m3");
}

tb_status tb_gemm_e4m3(const tb_e4m3* x, const tb_e4m3* w, const void* res, void* y, int32_t y_dtype, void* stream) {
  TB_OR_RETURN(check(x, "x", false));
  TB_OR_RETURN(check_weights(w, "w", x, false));
  if (!is_float(y_dtype)) return report(TB_ERR_INVALID_ARG, "unknown y_dtype %d", y_dtype);
  if (x->rows == 0) return TB_OK;
  TB_OR_RETURN(check(x, "x", true));
  TB_OR_RETURN(check(w, "w", true));
  TB_OR_RETURN(check_in(y, "y"));
  const size_t n = (size_t)x->rows * w->rows * esize(y_dtype);
  const Range ry = {y, n}, rres = {res, n};
  if (res) {
    TB_OR_RETURN(check_in(res, "res"));
    if (res != y && overlap(ry, rres)) return report(TB_ERR_INVALID_ARG, "y overlaps res (it may be res itself)");
  }
  const Range in[] = {codes_of(x), row_scales(x), codes_of(w), weight_scales(w)};
  TB_OR_RETURN(apart(&ry, 1, in, 4));
  GemmArgs a = {};
  a.x = coded(x);
  a.w = coded(w);
  a.M = x->rows;
  a.N = w->rows;
  a.K = x->cols;
  a.res = res;
  a.y = y;
  a.y_dtype = y_dtype;
  if (!device_error_word()) return report(TB_ERR_CUDA, "cannot resolve the device error word");
  const int tile = tile_of(a, 1);
  return done(tile > 0 ? launch_gemm_e4m3_few(a, tile, (cudaStream_t)stream) : launch_gemm_e4m3_many(a, tile < 0, (cudaStream_t)stream),
              "tb_gemm_e4m3");
}

tb_status tb_gated_e4m3(const tb_e4m3* x, const tb_e4m3* w1, const tb_e4m3* w3, void* y, int32_t y_dtype,
                        void* y_scale, void* stream) {
  TB_OR_RETURN(check(x, "x", false));
  TB_OR_RETURN(check_weights(w1, "w1", x, false));
  TB_OR_RETURN(check_weights(w3, "w3", x, false));
  if (w1->rows != w3->rows) return report(TB_ERR_INVALID_ARG, "w1 has %d rows, w3 has %d", w1->rows, w3->rows);
  if (!is_float(y_dtype) && y_dtype != TB_E4M3) return report(TB_ERR_INVALID_ARG, "unknown y_dtype %d", y_dtype);
  if ((y_dtype == TB_E4M3) != (y_scale != nullptr) && x->rows > 0)
    return report(TB_ERR_INVALID_ARG, "y_scale goes with codes (TB_E4M3)");
  if (x->rows == 0) return TB_OK;
  TB_OR_RETURN(check(x, "x", true));
  TB_OR_RETURN(check(w1, "w1", true));
  TB_OR_RETURN(check(w3, "w3", true));
  TB_OR_RETURN(check_in(y, "y"));
  const Range out[] = {{y, (size_t)x->rows * w1->rows * esize(y_dtype)},
                       {y_scale, (size_t)x->rows * blocks(w1->rows)}};
  const Range in[] = {codes_of(x), row_scales(x), codes_of(w1), weight_scales(w1), codes_of(w3), weight_scales(w3)};
  TB_OR_RETURN(apart(out, 2, in, 6));
  GemmArgs a = {};
  a.x = coded(x);
  a.w = coded(w1);
  a.w3 = coded(w3);
  a.M = x->rows;
  a.N = w1->rows;
  a.K = x->cols;
  a.y = y;
  a.y_dtype = y_dtype;
  a.y_scale = static_cast<uint8_t*>(y_scale);
  if (!device_error_word()) return report(TB_ERR_CUDA, "cannot resolve the device error word");
  const int tile = tile_of(a, 2);
  return done(tile > 0 ? launch_gated_e4m3_few(a, tile, (cudaStream_t)stream) : launch_gated_e4m3_many(a, tile < 0, (cudaStream_t)stream),
              "tb_gated_e4m3");
}

// Test hooks: the form that later products of this process take (0: by the rule; 16, 32,
// 64 or 128: k_e4m3_few with so many rows per tile; -1: k_e4m3_many; -2: the same with a
// CTA to a tile), returning the
// previous one; and the rule itself, for the tiles alone and with the type of the result.
TB_API int32_t tbx_e4m3_form(int32_t form) {
  return g_form.exchange(form == 16 || form == 32 || form == 64 || form == 128 || form == -1 || form == -2 ? form : 0);
}
TB_API int32_t tbx_e4m3_few_tile(int32_t M, int32_t N, int32_t K, int32_t mats, int32_t light, int32_t sms) {
  return e4m3_few_tile(M, N, K, mats, light != 0, sms);
}
TB_API int32_t tbx_e4m3_tile(int32_t M, int32_t N, int32_t K, int32_t mats, int32_t y_dtype, int32_t res, int32_t sms) {
  return rule(M, N, K, mats, y_dtype, res != 0, sms);
}

}  // extern "C"

// C ABI of the cache operators: argument checks and launches.  Declarations and
// contracts are in tb.h.
#include <math.h>
#include <stdint.h>

#include "cache.cuh"

namespace tb {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + nq && b < a + np;
}

// Layout rules of a cache these calls take; its tensors too with `tensors`.
tb_status check_cache(const tb_kvcache* kv, bool tensors) {
  if (!kv) return report(TB_ERR_INVALID_ARG, "kv is NULL");
  if (kv->dtype == TB_I8) return report(TB_ERR_UNSUPPORTED, "int8 caches: use tb_kvcache_append and tb_block_decode");
  if (kv->dtype != TB_F32 && kv->dtype != TB_BF16 && kv->dtype != TB_E4M3)
    return report(TB_ERR_INVALID_ARG, "unknown kv dtype %d", kv->dtype);
  if (kv->B < 0 || kv->Hkv <= 0 || kv->dh <= 0 || kv->T_max <= 0)
    return report(TB_ERR_INVALID_ARG, "kv shape must be positive (B may be 0)");
  if (kv->B > 32767 || kv->Hkv > 65535)
    return report(TB_ERR_UNSUPPORTED, "at most 32767 sequences and 65535 KV heads (%d, %d)", kv->B, kv->Hkv);
  if (kv->dh % 16 || kv->dh > 256)
    return report(TB_ERR_UNSUPPORTED, "dh (%d) must be a multiple of 16 of at most 256", kv->dh);
  if (kv->block_table || kv->dtype == TB_E4M3) {
    if (kv->page_size <= 0 || kv->page_size % 16)
      return report(TB_ERR_INVALID_ARG, "page_size (%d) must be a positive multiple of 16", kv->page_size);
    if (kv->T_max % kv->page_size)
      return report(TB_ERR_INVALID_ARG, "page_size (%d) must divide T_max (%d)", kv->page_size, kv->T_max);
  }
  if (kv->block_table) {
    if (kv->num_pages <= 0) return report(TB_ERR_INVALID_ARG, "num_pages must be positive");
    if ((long long)kv->num_pages * kv->Hkv >= (1LL << 31) - 1)
      return report(TB_ERR_UNSUPPORTED, "num_pages·Hkv above 2^31 - 2");
    if (!aligned4(kv->block_table)) return report(TB_ERR_INVALID_ARG, "block_table must be 4-byte aligned");
  }
  if (!tensors) return TB_OK;
  if (!kv->k || !kv->v || !kv->lens) return report(TB_ERR_INVALID_ARG, "kv cache pointers must be non-NULL");
  if (!aligned16(kv->k) || !aligned16(kv->v) || !aligned4(kv->lens))
    return report(TB_ERR_INVALID_ARG, "kv cache pointers must be 16-byte aligned (lens 4-byte)");
  if (kv->dtype == TB_E4M3 && (!kv->k_scale || !kv->v_scale || !aligned4(kv->k_scale) || !aligned4(kv->v_scale)))
    return report(TB_ERR_INVALID_ARG, "an e4m3 cache needs 4-byte aligned k_scale and v_scale");
  return TB_OK;
}

CacheView view_of(const tb_kvcache* kv, int* err) {
  CacheView c;
  c.k = kv->k;
  c.v = kv->v;
  c.ks = kv->k_scale;
  c.vs = kv->v_scale;
  c.bt = kv->block_table;
  c.lens = kv->lens;
  c.B = kv->B;
  c.Hkv = kv->Hkv;
  c.T = kv->T_max;
  c.dh = kv->dh;
  const bool blocks = kv->block_table || kv->dtype == TB_E4M3;
  c.ps = blocks ? kv->page_size : kv->T_max;
  c.ps_sh = shift_of(c.ps);
  c.per = blocks ? kv->T_max / kv->page_size : 1;
  c.num_pages = kv->num_pages;
  c.dtype = kv->dtype;
  c.err = err;
  return c;
}

AttnArgs attn_args(const tb_attn_cfg* cfg, const tb_kvcache* kv, int n, int* err) {
  AttnArgs a;
  a.c = view_of(kv, err);
  a.n = n;
  a.H = cfg->H;
  a.g_sh = shift_of(cfg->H / cfg->Hkv);
  a.window = cfg->window;
  a.sinks = cfg->window > 0 ? cfg->sinks : 0;
  const float scale = cfg->scale != 0.f ? cfg->scale : 1.0f / sqrtf((float)cfg->dh);
  a.scale_log2 = scale * 1.4426950408889634f;
  return a;
}

tb_status check_attn(const tb_attn_cfg* cfg, const tb_kvcache* kv, int n, bool tensors) {
  if (!cfg) return report(TB_ERR_INVALID_ARG, "cfg is NULL");
  const tb_status st = check_cache(kv, tensors);
  if (st != TB_OK) return st;
  if (n < 0) return report(TB_ERR_INVALID_ARG, "n must be non-negative");
  if (cfg->H <= 0 || cfg->Hkv <= 0 || cfg->H % cfg->Hkv)
    return report(TB_ERR_INVALID_ARG, "H (%d) must be a positive multiple of Hkv (%d)", cfg->H, cfg->Hkv);
  if (kv->Hkv != cfg->Hkv || kv->dh != cfg->dh)
    return report(TB_ERR_INVALID_ARG, "kv cache heads/width (%d, %d) differ from cfg (%d, %d)", kv->Hkv, kv->dh,
                  cfg->Hkv, cfg->dh);
  if (cfg->dtype != TB_F32 && cfg->dtype != TB_BF16)
    return report(TB_ERR_INVALID_ARG, "unknown dtype %d", cfg->dtype);
  if ((cfg->dtype == TB_F32) != (kv->dtype == TB_F32))
    return report(TB_ERR_INVALID_ARG, "fp32 queries go with an fp32 cache, bf16 queries with a bf16 or e4m3 one");
  if (cfg->window < 0 || cfg->sinks < 0)
    return report(TB_ERR_INVALID_ARG, "window (%d) and sinks (%d) must be non-negative", cfg->window, cfg->sinks);
  // (the kernels apply scale·log2 e, in fp32)
  if (!isfinite(cfg->scale * 1.4426950408889634f))
    return report(TB_ERR_INVALID_ARG, "scale must be finite, and its product with log2(e) too");
  const int G = cfg->H / cfg->Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8)
    return report(TB_ERR_UNSUPPORTED, "H/Hkv = %d: attention kernels exist for 1, 2, 4 and 8", G);
  const bool small = cfg->dh == 16 || cfg->dh == 32;
  if (cfg->dh != 64 && cfg->dh != 128 && !(small && cfg->dtype == TB_F32))
    return report(TB_ERR_UNSUPPORTED, "dh %d: attention kernels exist for 64 and 128 (fp32 also 16 and 32)", cfg->dh);
  if (n > kv->T_max) return report(TB_ERR_INVALID_ARG, "n (%d) exceeds kv->T_max (%d)", n, kv->T_max);
  // (the kernels round positions up to whole tiles of 128 keys, in 32 bits)
  if (kv->T_max > INT32_MAX - 256) return report(TB_ERR_UNSUPPORTED, "T_max (%d) above 2^31 - 257", kv->T_max);
  if ((long long)kv->B * n * cfg->H > (1LL << 31) - 1)
    return report(TB_ERR_UNSUPPORTED, "B·n·H above 2^31 - 1 query rows");
  if (!cache_attn_fits(attn_args(cfg, kv, n, nullptr)))
    return report(TB_ERR_UNSUPPORTED, "few rows over a sequence of more than 2^30 pieces (16 keys of a KV head each)");
  return TB_OK;
}

}  // namespace
}  // namespace tb

using namespace tb;

extern "C" {

tb_status tb_rope_table(int32_t dh, int32_t max_pos, float base, float* table, void* stream) {
  if (dh <= 0 || dh % 2 || max_pos < 0) return report(TB_ERR_INVALID_ARG, "dh must be even and positive, max_pos non-negative");
  if (!(base > 0.f)) return report(TB_ERR_INVALID_ARG, "base must be positive");
  if (max_pos == 0) return TB_OK;
  if ((long long)max_pos * (dh / 2) > (1LL << 38)) return report(TB_ERR_UNSUPPORTED, "rotation table above 2^38 pairs");
  if (!table || ((uintptr_t)table & 7u)) return report(TB_ERR_INVALID_ARG, "table must be non-NULL and 8-byte aligned");
  const cudaError_t e = launch_rope_table((float2*)table, max_pos, dh, base, (cudaStream_t)stream);
  return e == cudaSuccess ? TB_OK : report(TB_ERR_CUDA, "tb_rope_table: %s", cudaGetErrorString(e));
}

tb_status tb_kvcache_append_rope(const tb_kvcache* kv, const tb_append_rows* rows, const float* rope, int32_t max_pos,
                                 void* stream) {
  tb_status st = check_cache(kv, false);
  if (st != TB_OK) return st;
  if (!rows) return report(TB_ERR_INVALID_ARG, "rows is NULL");
  if (rows->n < 0) return report(TB_ERR_INVALID_ARG, "n must be non-negative");
  if (rows->n == 0 || kv->B == 0) return TB_OK;
  st = check_cache(kv, true);
  if (st != TB_OK) return st;
  if (rows->n > kv->T_max) return report(TB_ERR_INVALID_ARG, "n (%d) exceeds kv->T_max (%d)", rows->n, kv->T_max);
  // (the eight-element pieces of a block are counted in 32 bits)
  if (kv->dtype == TB_E4M3 && kv->page_size > 1 << 24)
    return report(TB_ERR_UNSUPPORTED, "appending to e4m3 blocks of at most 2^24 tokens (%d)", kv->page_size);
  if (max_pos < kv->T_max)
    return report(TB_ERR_INVALID_ARG, "the rotation table's max_pos (%d) is below kv->T_max (%d)", max_pos, kv->T_max);
  if (!rope || !aligned16(rope)) return report(TB_ERR_INVALID_ARG, "rope must be non-NULL and 16-byte aligned");
  if (!rows->k || !rows->v) return report(TB_ERR_INVALID_ARG, "k and v must be non-NULL");
  if ((rows->q == nullptr) != (rows->q_out == nullptr)) return report(TB_ERR_INVALID_ARG, "q and q_out go together");
  if (rows->q && rows->H <= 0) return report(TB_ERR_INVALID_ARG, "H must be positive");
  if (rows->q && rows->H > 65535) return report(TB_ERR_UNSUPPORTED, "at most 65535 query heads (%d)", rows->H);
  if (!aligned16(rows->q) || !aligned16(rows->q_out) || !aligned16(rows->k) || !aligned16(rows->v))
    return report(TB_ERR_INVALID_ARG, "q, q_out, k and v must be 16-byte aligned");
  const int64_t strides[6] = {rows->q_tok, rows->q_seq, rows->k_tok, rows->k_seq, rows->v_tok, rows->v_seq};
  for (int i = rows->q ? 0 : 2; i < 6; ++i)
    if (strides[i] % 8 || strides[i] < 0)
      return report(TB_ERR_INVALID_ARG, "row strides must be non-negative multiples of 8 elements");
  if (!aligned4(rows->start) || !aligned4(rows->n_new))
    return report(TB_ERR_INVALID_ARG, "start and n_new must be 4-byte aligned");
  const size_t lens_bytes = (size_t)kv->B * 4;
  if ((rows->start && overlap(rows->start, lens_bytes, kv->lens, lens_bytes)) ||
      (rows->n_new && overlap(rows->n_new, lens_bytes, kv->lens, lens_bytes)))
    return report(TB_ERR_INVALID_ARG, "start and n_new may not overlap lens (a NULL start stands for lens)");
  if (rows->q) {
    const size_t es = kv->dtype == TB_F32 ? 4 : 2;
    auto extent = [&](int64_t tok, int64_t seq, int heads) {
      return ((size_t)(kv->B - 1) * seq + (size_t)(rows->n - 1) * tok + (size_t)heads * kv->dh) * es;
    };
    const size_t out = (size_t)kv->B * rows->n * rows->H * kv->dh * es;
    const bool dense = (rows->n == 1 || rows->q_tok == (int64_t)rows->H * kv->dh) &&
                       (kv->B == 1 || rows->q_seq == (int64_t)rows->H * kv->dh * rows->n);
    if (rows->q == rows->q_out ? !dense : overlap(rows->q_out, out, rows->q, extent(rows->q_tok, rows->q_seq, rows->H)))
      return report(TB_ERR_INVALID_ARG, "q_out overlaps q, and is not a dense q itself");
    if (overlap(rows->q_out, out, rows->k, extent(rows->k_tok, rows->k_seq, kv->Hkv)) ||
        overlap(rows->q_out, out, rows->v, extent(rows->v_tok, rows->v_seq, kv->Hkv)))
      return report(TB_ERR_INVALID_ARG, "q_out overlaps k or v");
  }
  int* err = device_error_word();
  if (!err) return report(TB_ERR_CUDA, "cannot resolve the device error word");
  AppendArgs a;
  a.c = view_of(kv, err);
  a.q = rows->q;
  a.k = rows->k;
  a.v = rows->v;
  a.q_out = rows->q_out;
  a.q_tok = rows->q_tok;
  a.q_seq = rows->q_seq;
  a.k_tok = rows->k_tok;
  a.k_seq = rows->k_seq;
  a.v_tok = rows->v_tok;
  a.v_seq = rows->v_seq;
  a.H = rows->H;
  a.n = rows->n;
  a.start = rows->start;
  a.n_new = rows->n_new;
  a.pieces = kv->dh / 8;
  a.piece_sh = shift_of(a.pieces);
  a.hkv_sh = shift_of(kv->Hkv);
  a.rope = (const float2*)rope;
  const cudaError_t e = launch_append_rope(a, (cudaStream_t)stream);
  return e == cudaSuccess ? TB_OK : report(TB_ERR_CUDA, "tb_kvcache_append_rope: %s", cudaGetErrorString(e));
}

size_t tb_kvcache_attn_workspace_bytes(const tb_attn_cfg* cfg, const tb_kvcache* kv, int32_t n) {
  if (check_attn(cfg, kv, n, false) != TB_OK) return 0;
  return cache_attn_workspace_upto(attn_args(cfg, kv, n, nullptr));
}

tb_status tb_kvcache_attn(const tb_attn_cfg* cfg, const void* q, const tb_kvcache* kv, const int32_t* n_new, int32_t n,
                          void* o, void* ws, size_t ws_bytes, void* stream) {
  tb_status st = check_attn(cfg, kv, n, false);
  if (st != TB_OK) return st;
  if (n == 0 || kv->B == 0) return TB_OK;
  st = check_attn(cfg, kv, n, true);
  if (st != TB_OK) return st;
  if (!q || !o) return report(TB_ERR_INVALID_ARG, "q and o must be non-NULL");
  if (!aligned16(q) || !aligned16(o) || !aligned4(n_new))
    return report(TB_ERR_INVALID_ARG, "q and o must be 16-byte aligned, n_new 4-byte");
  const size_t rows = (size_t)kv->B * n * cfg->H * cfg->dh * (cfg->dtype == TB_F32 ? 4 : 2);
  if (overlap(q, rows, o, rows)) return report(TB_ERR_INVALID_ARG, "o may not overlap q");
  AttnArgs a = attn_args(cfg, kv, n, nullptr);
  a.q = q;
  a.o = o;
  a.n_new = n_new;
  const size_t need = cache_attn_workspace(a);
  if (need && (!ws || ((uintptr_t)ws & 255u) || ws_bytes < need))
    return report(TB_ERR_INVALID_ARG, "ws must be 256-byte aligned and hold %zu bytes (%zu)", need, ws_bytes);
  a.c.err = device_error_word();
  if (!a.c.err) return report(TB_ERR_CUDA, "cannot resolve the device error word");
  const cudaError_t e = launch_cache_attn(a, ws, (cudaStream_t)stream);
  return e == cudaSuccess ? TB_OK : report(TB_ERR_CUDA, "tb_kvcache_attn: %s", cudaGetErrorString(e));
}

}  // extern "C"

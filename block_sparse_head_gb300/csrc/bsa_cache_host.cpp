// bsa_cache_host.cpp -- entry points of the paged 8-bit cache: argument checks and launches.
// See include/bsa.h for the contract of every exported function.
#include "../../include/bsa.h"

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <limits>

#include "bsa_internal.h"

namespace {

constexpr int64_t kInt32Max = std::numeric_limits<int32_t>::max();

bool aligned(const void* p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// log2 of a supported page or block, or -1.
int shift_of(int n, int least) {
  for (int s = 4; s <= 7; ++s)
    if (n == (1 << s) && n >= least) return s;
  return -1;
}

int check_cache(const bsa_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr ||
      c->v_scale == nullptr)
    return BSA_ERR_NULL;
  if (shift_of(c->page, 16) < 0 || (c->d != 64 && c->d != 128)) return BSA_ERR_UNSUPPORTED;
  if (c->dtype != BSA_E4M3 && c->dtype != BSA_INT8) return BSA_ERR_DTYPE;
  if (c->n_pages < 1 || c->kv_heads < 1 || c->kv_heads > 65535 ||
      static_cast<int64_t>(c->n_pages) * c->page > kInt32Max ||
      static_cast<int64_t>(c->n_pages) * c->kv_heads > kInt32Max)
    return BSA_ERR_SHAPE;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return BSA_ERR_ALIGN;
  return BSA_OK;
}

int check_heads(int heads, int kv_heads) {
  return heads < 1 || kv_heads < 1 || heads > 65535 || heads % kv_heads != 0 ||
                 heads / kv_heads > 128
             ? BSA_ERR_SHAPE
             : BSA_OK;
}

// Rows of the decode kernel that a call takes, 0: too many for it.  A request's queries are then
// one tile, which reads the cache once, where they fill it to a power of two (bsa_cache_sched.cuh),
// and two else; with more rows each 8 or 16 of them would read it again.
int decode_rows(int group, int max_q) {
  const int64_t rows = static_cast<int64_t>(group) * max_q;
  return rows <= 8 ? 8 : rows <= bsa::kDecodeRows ? 16 : 0;
}

}  // namespace

extern "C" {

int bsa_cache_resize(int32_t* block_table, const int32_t* kv_len, const int32_t* new_len,
                     int32_t* free_pages, const int32_t* free_count, int32_t* kv_len_out,
                     int32_t* free_count_out, int32_t* cu_new, int32_t* slots, int32_t* status,
                     int B, int max_pages, int n_pages, int page, int tokens, void* stream) {
  if (block_table == nullptr || kv_len == nullptr || new_len == nullptr || free_pages == nullptr ||
      free_count == nullptr || kv_len_out == nullptr || free_count_out == nullptr ||
      cu_new == nullptr || status == nullptr || (slots == nullptr && tokens > 0))
    return BSA_ERR_NULL;
  const int shift = shift_of(page, 16);
  if (shift < 0) return BSA_ERR_UNSUPPORTED;
  if (B < 1 || B > bsa::kMaxResizeBatch || max_pages < 1 || n_pages < 1 || tokens < 0 ||
      tokens > bsa::kMaxPositions ||
      static_cast<int64_t>(max_pages) * page > kInt32Max ||
      static_cast<int64_t>(n_pages) * page > kInt32Max)
    return BSA_ERR_SHAPE;
  for (const void* ptr :
       {static_cast<const void*>(block_table), static_cast<const void*>(kv_len),
        static_cast<const void*>(new_len), static_cast<const void*>(free_pages),
        static_cast<const void*>(free_count), static_cast<const void*>(kv_len_out),
        static_cast<const void*>(free_count_out), static_cast<const void*>(cu_new),
        static_cast<const void*>(slots), static_cast<const void*>(status)})
    if (!aligned(ptr, 4)) return BSA_ERR_ALIGN;
  bsa::CacheResizeParams p{};
  p.table = block_table;
  p.kv_len = kv_len;
  p.new_len = new_len;
  p.free_pages = free_pages;
  p.free_count = free_count;
  p.kv_len_out = kv_len_out;
  p.free_count_out = free_count_out;
  p.cu_new = cu_new;
  p.slots = slots;
  p.status = status;
  p.B = B;
  p.max_pages = max_pages;
  p.n_pages = n_pages;
  p.tokens = tokens;
  p.page_shift = shift;
  return bsa::launch_cache_resize(p, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BSA_OK
             : BSA_ERR_CUDA;
}

int bsa_cache_append(const bsa_cache* cache, const void* k, const void* v, const int32_t* slots,
                     int T, int dtype, int64_t k_token_stride, int64_t k_head_stride,
                     int64_t v_token_stride, int64_t v_head_stride, void* stream) {
  const int bad = check_cache(cache);
  if (bad != BSA_OK) return bad;
  if (T < 0 || T > bsa::kMaxPositions) return BSA_ERR_SHAPE;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_DTYPE;
  if (T == 0) return BSA_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return BSA_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || k_token_stride % 8 != 0 ||
      k_head_stride % 8 != 0 || v_token_stride % 8 != 0 || v_head_stride % 8 != 0)
    return BSA_ERR_ALIGN;
  bsa::CacheAppendParams p{};
  p.x[0] = k;
  p.x[1] = v;
  p.token_stride[0] = k_token_stride;
  p.token_stride[1] = v_token_stride;
  p.head_stride[0] = k_head_stride;
  p.head_stride[1] = v_head_stride;
  p.cache[0] = cache->k;
  p.cache[1] = cache->v;
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.slots = slots;
  p.T = T;
  p.heads = cache->kv_heads;
  p.n_pages = cache->n_pages;
  p.page_shift = shift_of(cache->page, 16);
  return bsa::launch_cache_append(cache->d, dtype, cache->dtype, p,
                                  static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? BSA_OK
             : BSA_ERR_CUDA;
}

int bsa_cache_workspace(int heads, int kv_heads, int d, int max_q, int64_t* bytes) {
  if (bytes == nullptr) return BSA_ERR_NULL;
  *bytes = 0;
  if (d != 64 && d != 128) return BSA_ERR_UNSUPPORTED;
  if (check_heads(heads, kv_heads) != BSA_OK || max_q < 1) return BSA_ERR_SHAPE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  const int sms = bsa::sm_count(dev);
  if (sms <= 0) return BSA_ERR_CUDA;
  const int rows = decode_rows(heads / kv_heads, max_q);
  *bytes = bsa::cache_parts_bytes(sms, rows > 0 ? rows : bsa::kTileRows, d);
  return BSA_OK;
}

int bsa_cache_forward(const bsa_cache* cache, const void* q, const int32_t* block_table,
                      const int32_t* kv_len, const int32_t* cu_q, void* out, float* lse,
                      int32_t* status, void* workspace, int64_t workspace_bytes, int B,
                      int max_pages, int T, int heads, int max_q, int dtype,
                      int64_t q_token_stride, int64_t q_head_stride, float scale,
                      const bsa_cache_args* args, void* stream) {
  const int bad = check_cache(cache);
  if (bad != BSA_OK) return bad;
  bsa_cache_args x{-1, 0.f, nullptr, nullptr, 0};
  if (args != nullptr) x = *args;
  if (block_table == nullptr || kv_len == nullptr || cu_q == nullptr || workspace == nullptr ||
      (T > 0 && (q == nullptr || out == nullptr || lse == nullptr)))
    return BSA_ERR_NULL;
  if (dtype != BSA_BF16 && dtype != BSA_FP16) return BSA_ERR_DTYPE;
  if (B < 1 || T < 0 || T > bsa::kMaxPositions || max_pages < 1 || max_q < 1 ||
      check_heads(heads, cache->kv_heads) != BSA_OK ||
      static_cast<int64_t>(max_pages) * cache->page > bsa::kMaxPositions ||
      static_cast<int64_t>(B) * cache->kv_heads > kInt32Max)
    return BSA_ERR_SHAPE;
  if (!std::isfinite(scale) || !std::isfinite(x.softcap) || x.softcap < 0.f)
    return BSA_ERR_UNSUPPORTED;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(lse, 4) ||
      !aligned(status, 4) || !aligned(block_table, 4) || !aligned(kv_len, 4) ||
      !aligned(cu_q, 4) || !aligned(x.sinks, 4) || q_token_stride % 8 != 0 ||
      q_head_stride % 8 != 0)
    return BSA_ERR_ALIGN;
  bsa::CacheFwdParams p{};
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (x.softcap > 0.f) {
    p.softcap_log2 = static_cast<float>(static_cast<double>(x.softcap) * 1.4426950408889634);
    p.softcap_inv = static_cast<float>(static_cast<double>(scale) / x.softcap);
  }
  if (!std::isfinite(p.scale_log2) || !std::isfinite(p.softcap_log2) ||
      !std::isfinite(p.softcap_inv))
    return BSA_ERR_UNSUPPORTED;
  p.page_shift = shift_of(cache->page, 16);
  if (x.lut != nullptr) {
    p.block_shift = shift_of(x.block, 64);
    if (p.block_shift < 0) return BSA_ERR_UNSUPPORTED;
    const int64_t span = static_cast<int64_t>(max_pages) * cache->page;
    if (x.lut->H != cache->kv_heads || span > (static_cast<int64_t>(x.lut->nb) << p.block_shift) ||
        span > (static_cast<int64_t>(x.lut->nbk) << p.block_shift))
      return BSA_ERR_SHAPE;
    int dev = -1;
    if (x.lut->d_items == nullptr) return BSA_ERR_STATE;
    if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
    if (dev != x.lut->device) return BSA_ERR_STATE;
    p.row_ptr = x.lut->d_row_ptr;
    p.col_idx = x.lut->d_col_idx;
    p.nb = x.lut->nb;
    p.expire_site = x.lut->expire_site;
  }
  int64_t need = 0;
  const int rc = bsa_cache_workspace(heads, cache->kv_heads, cache->d, max_q, &need);
  if (rc != BSA_OK) return rc;
  if (workspace_bytes < need) return BSA_ERR_TOO_LARGE;
  p.q = q;
  p.q_token_stride = q_token_stride;
  p.q_head_stride = q_head_stride;
  p.k_cache = static_cast<const uint8_t*>(cache->k);
  p.v_cache = static_cast<const uint8_t*>(cache->v);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.table = block_table;
  p.kv_len = kv_len;
  p.cu_q = cu_q;
  p.out = out;
  p.lse = lse;
  p.status = status;
  p.sinks = x.sinks;
  p.B = B;
  p.T = T;
  p.Hq = heads;
  p.Hkv = cache->kv_heads;
  p.group = heads / cache->kv_heads;
  p.group_inv = (65536u + p.group - 1) / p.group;
  p.n_pages = cache->n_pages;
  p.max_pages = max_pages;
  p.window = x.window < 0 ? -1 : std::min(x.window, bsa::kMaxPositions);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return status == nullptr || cudaMemsetAsync(status, 0, 4, st) == cudaSuccess ? BSA_OK
                                                                                : BSA_ERR_CUDA;
  cudaError_t e;
  const int rows = decode_rows(p.group, max_q);
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  const int sms = bsa::sm_count(dev);
  const bool fp16 = dtype == BSA_FP16, int8 = cache->dtype == BSA_INT8;
  if (rows > 0) {
    const int64_t tiles = static_cast<int64_t>(cache->n_pages) * cache->kv_heads;
    p.box_shift = p.page_shift < 6 ? p.page_shift : 6;
    CUtensorMap k, v;
    if (!bsa::encode_cache(&k, cache->k, tiles, cache->page, cache->d, 1 << p.box_shift) ||
        !bsa::encode_cache(&v, cache->v, tiles, cache->page, cache->d, 1 << p.box_shift))
      return BSA_ERR_CUDA;
    e = cache->d == 128
            ? (int8 ? bsa::launch_cache_decode_int8_d128(fp16, rows, k, v, p, workspace, sms, st)
                    : bsa::launch_cache_decode_e4m3_d128(fp16, rows, k, v, p, workspace, sms, st))
            : (int8 ? bsa::launch_cache_decode_int8_d64(fp16, rows, k, v, p, workspace, sms, st)
                    : bsa::launch_cache_decode_e4m3_d64(fp16, rows, k, v, p, workspace, sms, st));
  } else {
    e = cache->d == 128 ? (int8 ? bsa::launch_cache_tile_int8_d128(fp16, p, workspace, sms, st)
                                : bsa::launch_cache_tile_e4m3_d128(fp16, p, workspace, sms, st))
                        : (int8 ? bsa::launch_cache_tile_int8_d64(fp16, p, workspace, sms, st)
                                : bsa::launch_cache_tile_e4m3_d64(fp16, p, workspace, sms, st));
  }
  return e == cudaSuccess ? BSA_OK : BSA_ERR_CUDA;
}

}  // extern "C"

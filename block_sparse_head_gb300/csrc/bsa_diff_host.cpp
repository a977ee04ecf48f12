// bsa_diff_host.cpp -- entry points of differential attention over a layout: argument checks
// and launches.  See include/bsa.h for the contract of every exported function.
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

// Sizes that the two calls share; 0 or an error.  On success the LUT is on the current device.
int check(const bsa_lut* lut, int B, int H, int kv_heads, int L, int d, int dq, float scale, int block,
          int* grid) {
  if ((block != 64 && block != 128) || (d != 64 && d != 128) || (dq != d && !(d == 128 && dq == 64)))
    return BSA_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !std::isfinite(static_cast<float>(scale * 1.4426950408889634)))
    return BSA_ERR_UNSUPPORTED;
  if (B < 1 || H < 1 || kv_heads < 1 || L < 1 || H % kv_heads != 0 || L > bsa::kMaxPositions ||
      B != lut->batch || kv_heads != lut->H || lut->nbk != lut->nb || lut->nb != (L + block - 1) / block)
    return BSA_ERR_SHAPE;
  // Rows of the queries, and sub-items of the work list with the steps that run ahead of it.
  if (2ll * B * H * L > kInt32Max - 128 ||
      static_cast<int64_t>(lut->n_items) * (H / kv_heads) * (block / 64) > kInt32Max - (1 << 16))
    return BSA_ERR_SHAPE;
  if (lut->d_list == nullptr) return BSA_ERR_STATE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  if (dev != lut->device) return BSA_ERR_STATE;
  const int sms = bsa::sm_count(dev);
  if (sms <= 0) return BSA_ERR_CUDA;
  *grid = sms;
  return BSA_OK;
}

void fill_list(bsa::DiffList& p, const bsa_lut* lut, int pairs, int block) {
  p.list = reinterpret_cast<const int4*>(lut->d_list);
  p.pairs = pairs;
  p.halves = block / 64;
  p.n = lut->n_items * pairs * p.halves;
  auto over = [](int by, uint32_t& mul, int& shift) {
    shift = 0;
    while ((1ll << shift) < by) ++shift;
    mul = static_cast<uint32_t>(((1ull << (31 + shift)) + by - 1) / by);
  };
  over(pairs * p.halves, p.each_mul, p.each_shift);
  over(pairs, p.pairs_mul, p.pairs_shift);
}

template <class F64_64, class F64_128, class F128_64, class F128_128>
auto pick(int block, int d, F64_64 a, F64_128 b, F128_64 c, F128_128 e) {
  return block == 64 ? (d == 64 ? a : b) : (d == 64 ? c : e);
}

// The workspace: row terms, the pieces of cut columns (two a CTA), sums of dlam, counts.
constexpr int kCounts = 8;  // of a CTA: one a warp

struct Parts {
  int64_t parts, sums, count, bytes;  // offsets
  Parts(int B, int H, int L, int d, int block, int sms) {
    const int64_t tiles = static_cast<int64_t>(B) * H * bsa::diff_vec_tiles((L + 63) / 64);
    parts = tiles * bsa::kDiffVecFloats * 4;
    sums = parts + static_cast<int64_t>(sms) * 2 * block * 2 * d * 4;
    count = sums + tiles * 16;
    bytes = count + static_cast<int64_t>(sms) * kCounts * 4;
  }
};

}  // namespace

extern "C" {

int bsa_diff_forward(const void* q, const void* k, const void* v, const float* lam,
                     const bsa_lut* lut, void* out, float* lse, void* out2, int B, int H,
                     int kv_heads, int L, int d, int dq, int lam_rows, float scale, int block,
                     int causal_diag, void* stream) {
  if (q == nullptr || k == nullptr || v == nullptr || lam == nullptr || lut == nullptr ||
      out == nullptr || lse == nullptr)
    return BSA_ERR_NULL;
  for (const void* ptr : {q, k, v, static_cast<const void*>(out), static_cast<const void*>(out2)})
    if (!aligned(ptr, 16)) return BSA_ERR_ALIGN;
  if (!aligned(lam, 4) || !aligned(lse, 4)) return BSA_ERR_ALIGN;
  int sms = 0;
  const int bad = check(lut, B, H, kv_heads, L, d, dq, scale, block, &sms);
  if (bad != BSA_OK) return bad;
  CUtensorMap tq, tk, tv;
  const int64_t heads = static_cast<int64_t>(B) * H, kv = static_cast<int64_t>(B) * kv_heads;
  if (!bsa::encode_heads(&tq, q, 2 * heads, L, dq, 16, 1) ||
      !bsa::encode_heads(&tk, k, kv, L, d, block, d / 64) ||
      !bsa::encode_heads(&tv, v, kv, L, d, block, d / 64))
    return BSA_ERR_CUDA;
  bsa::DiffFwdParams p{};
  fill_list(p, lut, H / kv_heads, block);
  p.col_idx = lut->d_col_idx;
  p.out = out;
  p.out2 = out2;
  p.lse = lse;
  p.lam = lam;
  p.status = lut->d_status;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.causal_diag = causal_diag != 0;
  p.lam_rows = lam_rows != 0;
  p.H = H;
  p.L = L;
  p.wait_limit_ns = lut->wait_limit_ns;
  p.expire_site = lut->expire_site;
  auto* launch = pick(block, d, bsa::launch_diff_fwd_b64_d64, bsa::launch_diff_fwd_b64_d128,
                      bsa::launch_diff_fwd_b128_d64, bsa::launch_diff_fwd_b128_d128);
  return launch(dq != d, p, tq, tk, tv, std::min(p.n, sms), static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? BSA_OK
             : BSA_ERR_CUDA;
}

int bsa_diff_workspace(int B, int H, int L, int d, int block, int64_t* bytes) {
  if (bytes == nullptr) return BSA_ERR_NULL;
  *bytes = 0;
  if ((block != 64 && block != 128) || (d != 64 && d != 128)) return BSA_ERR_UNSUPPORTED;
  if (B < 1 || H < 1 || L < 1 || L > bsa::kMaxPositions || 2ll * B * H > kInt32Max ||
      2ll * B * H * L > kInt32Max - 128)
    return BSA_ERR_SHAPE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return BSA_ERR_CUDA;
  const int sms = bsa::sm_count(dev);
  if (sms <= 0) return BSA_ERR_CUDA;
  *bytes = Parts(B, H, L, d, block, sms).bytes;
  return BSA_OK;
}

int bsa_diff_backward(const void* q, const void* k, const void* v, const float* lam,
                      const void* out, const void* out2, const float* lse, const void* dout,
                      const bsa_lut* lut, void* dq_out, void* dk, void* dv, float* dlam,
                      void* workspace, int64_t workspace_bytes, int B, int H, int kv_heads, int L,
                      int d, int dq, int lam_rows, float scale, int block, int causal_diag,
                      void* stream) {
  if (q == nullptr || k == nullptr || v == nullptr || lam == nullptr || out == nullptr ||
      out2 == nullptr || lse == nullptr || dout == nullptr || lut == nullptr || dq_out == nullptr ||
      dk == nullptr || dv == nullptr || dlam == nullptr || workspace == nullptr)
    return BSA_ERR_NULL;
  for (const void* ptr : {q, k, v, out, out2, dout, static_cast<const void*>(dq_out),
                          static_cast<const void*>(dk), static_cast<const void*>(dv),
                          static_cast<const void*>(workspace)})
    if (!aligned(ptr, 16)) return BSA_ERR_ALIGN;
  if (!aligned(lam, 4) || !aligned(lse, 4) || !aligned(dlam, 4)) return BSA_ERR_ALIGN;
  int sms = 0;
  const int bad = check(lut, B, H, kv_heads, L, d, dq, scale, block, &sms);
  if (bad != BSA_OK) return bad;
  const Parts parts(B, H, L, d, block, sms);
  if (workspace_bytes < parts.bytes) return BSA_ERR_TOO_LARGE;
  CUtensorMap tq, tk, tv, tdo32, tdo64;
  const int64_t heads = static_cast<int64_t>(B) * H, kv = static_cast<int64_t>(B) * kv_heads;
  if (!bsa::encode_heads(&tq, q, 2 * heads, L, dq, 32, 1) ||
      !bsa::encode_heads(&tk, k, kv, L, d, block, d / 64) ||
      !bsa::encode_heads(&tv, v, kv, L, d, block, d / 64) ||
      !bsa::encode_heads(&tdo32, dout, heads, L, d, 32, 1) ||
      !bsa::encode_heads(&tdo64, dout, heads, L, d, 64, d / 64))
    return BSA_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  bsa::DiffRowsParams r{};
  r.out = out;
  r.out2 = out2;
  r.dout = dout;
  r.lse = lse;
  r.lam = lam;
  r.vec = static_cast<float*>(workspace);
  r.pairs = heads;
  r.H = H;
  r.L = L;
  r.d = d;
  r.lam_rows = lam_rows != 0;
  char* ws = static_cast<char*>(workspace);
  bsa::DiffBwdParams p{};
  fill_list(p, lut, H / kv_heads, block);
  p.col_idx = lut->d_col_idx;
  p.col_ptr = lut->d_col_ptr;
  p.row_idx = lut->d_row_idx;
  p.diag_pos = lut->d_diag_t;
  p.B = B;
  p.nb = lut->nb;
  p.nnz = lut->nnz_total;
  p.cols = lut->H * lut->nb;
  p.steps = static_cast<int64_t>(B) * p.nnz * p.pairs * p.halves;
  p.share = std::max<int64_t>((p.steps + sms - 1) / sms, bsa::kDiffShare);
  p.vec = r.vec;
  p.parts = reinterpret_cast<float*>(ws + parts.parts);
  p.count = reinterpret_cast<int*>(ws + parts.count);
  p.dq = dq_out;
  p.dlam = dlam;
  p.lam_sums = reinterpret_cast<float*>(ws + parts.sums);
  p.lam_rows = lam_rows != 0;
  p.H = H;
  p.dk = dk;
  p.dv = dv;
  p.status = lut->d_status;
  p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  p.scale = scale;
  p.causal_diag = causal_diag != 0;
  p.L = L;
  p.block = block;
  p.d = d;
  p.wait_limit_ns = lut->wait_limit_ns;
  p.expire_site = lut->expire_site;
  auto* launch = pick(block, d, bsa::launch_diff_bwd_b64_d64, bsa::launch_diff_bwd_b64_d128,
                      bsa::launch_diff_bwd_b128_d64, bsa::launch_diff_bwd_b128_d128);
  if (bsa::launch_diff_rows(r, p, sms * kCounts, st) != cudaSuccess ||
      launch(dq != d, false, p, tq, tdo32, tk, tv, std::min(p.n, sms), st) != cudaSuccess ||
      launch(dq != d, true, p, tk, tv, tq, tdo64, sms, st) != cudaSuccess)
    return BSA_ERR_CUDA;
  return BSA_OK;
}

}  // extern "C"

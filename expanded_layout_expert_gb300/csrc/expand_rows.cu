// moe_expand_rows: the 16-bit row of each valid (token, expert) pair at its
// expanded row, the form moe_expand_scatter has for fp8 rows:
//   xe[src2dst[t, k], :] = x[t, :],   row_w[src2dst[t, k]] = topk_w[t, k]
// with the alignment gaps of every segment zeroed. It is the gather before
// the 16-bit grouped products, and, given dy, the gradient of moe_combine's
// unweighted sum; its own gradient is moe_combine.
// moe_collect_row_grads takes per-row values back to their pairs:
//   out[t, k] = src2dst[t, k] >= 0 ? row[src2dst[t, k]] : 0.
//
// Bytes: 2H read per token, 2H written per pair; nothing is computed.
#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kMaxK = 32;
constexpr int kThreads = 256;
constexpr int kPadRowsPerBlock = 8;

// Blocks [0, pad_blocks) zero the alignment gaps (first in the grid, so they
// are never its tail); the warps of the others take pieces of tokens' rows, a
// piece being 1 KB: two 16-byte vectors per lane, both read before the K pairs
// of stores. Small pieces spread a batch of few tokens over the GPU.
constexpr int kPieceVec = 64;

__global__ void __launch_bounds__(kThreads) expand_rows_kernel(
    const uint16_t* __restrict__ x, int64_t ld_x, const float* __restrict__ topk_w,
    const int32_t* __restrict__ src2dst, const int32_t* __restrict__ psum,
    const int32_t* __restrict__ d_n_valid, int64_t T, int nvec, int K, int align, int64_t M_cap,
    uint16_t* __restrict__ xe, int64_t ld_xe, float* __restrict__ row_w, int pad_blocks_per_expert,
    int pad_blocks, int32_t* __restrict__ status) {
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) < pad_blocks) {
    const int e = blockIdx.x / pad_blocks_per_expert;
    const int sub = blockIdx.x % pad_blocks_per_expert;
    const int64_t end = max(psum[e], 0);   // clamped into the buffer, as the products' segments are
    int64_t seg_end = (end + align - 1) / align * align;
    if (seg_end > M_cap) seg_end = M_cap;
    const int64_t r0 = end + static_cast<int64_t>(sub) * kPadRowsPerBlock;
    const int64_t r1 = r0 + kPadRowsPerBlock < seg_end ? r0 + kPadRowsPerBlock : seg_end;
    for (int64_t r = r0; r < r1; ++r) {
      for (int v = tid; v < nvec; v += kThreads)
        reinterpret_cast<uint4*>(xe + r * ld_xe)[v] = make_uint4(0, 0, 0, 0);
      if (row_w != nullptr && tid == 0) row_w[r] = 0.0f;
    }
    return;
  }
  int64_t nv = T;
  if (d_n_valid != nullptr) {
    nv = *d_n_valid;
    nv = nv < 0 ? 0 : (nv > T ? T : nv);
  }
  const int pieces = (nvec + kPieceVec - 1) / kPieceVec;
  const int64_t items = nv * pieces;
  const int lane = tid & 31;
  const int64_t step = static_cast<int64_t>(gridDim.x - pad_blocks) * (kThreads / 32);
  for (int64_t it = static_cast<int64_t>(blockIdx.x - pad_blocks) * (kThreads / 32) + (tid >> 5);
       it < items; it += step) {
    const int64_t t = it <= UINT32_MAX ? static_cast<uint32_t>(it) / static_cast<uint32_t>(pieces)
                                       : it / pieces;
    const int piece = static_cast<int>(it - t * pieces);
    const int v = piece * kPieceVec + lane;
    const uint4* src = reinterpret_cast<const uint4*>(x + t * ld_x) + v;
    const bool act0 = v < nvec, act1 = v + 32 < nvec;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (act0) a = __ldcs(src);
    if (act1) b = __ldcs(src + 32);
    // lane k < K holds pair k's row
    int my = -1;
    if (lane < K) {
      my = src2dst[t * K + lane];
      if (my >= M_cap) {
        set_status(status, MOE_ERR_DEVICE_CHECK);
        my = -1;
      }
      if (row_w != nullptr && piece == 0 && my >= 0) row_w[my] = topk_w[t * K + lane];
    }
    for (int k = 0; k < K; ++k) {
      const int r = __shfl_sync(0xffffffffu, my, k);
      if (r < 0) continue;
      uint4* dst = reinterpret_cast<uint4*>(xe + static_cast<int64_t>(r) * ld_xe) + v;
      if (act0) dst[0] = a;
      if (act1) dst[32] = b;
    }
  }
}

__global__ void __launch_bounds__(kThreads) collect_row_grads_kernel(
    const float* __restrict__ rows, const int32_t* __restrict__ src2dst,
    const int32_t* __restrict__ d_n_valid, int64_t T, int K, int64_t M_cap,
    float* __restrict__ out) {
  int64_t nv = T;
  if (d_n_valid != nullptr) {
    nv = *d_n_valid;
    nv = nv < 0 ? 0 : (nv > T ? T : nv);
  }
  const int64_t n = nv * K, step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step) {
    const int r = src2dst[i];
    out[i] = r >= 0 && r < M_cap ? rows[r] : 0.0f;
  }
}

}  // namespace
}  // namespace moe

extern "C" int moe_expand_rows(const uint16_t* x, int64_t ld_x, const float* topk_w,
                               const int32_t* src2dst, const int32_t* psum,
                               const int32_t* d_n_valid, int64_t T, int H, int K, int E, int align,
                               int64_t M_cap, uint16_t* xe, int64_t ld_xe, float* row_w,
                               int32_t* d_status, moe_stream_t stream) {
  MOE_REQUIRE(psum && (M_cap == 0 || xe), "moe_expand_rows: null psum or output");
  MOE_REQUIRE(T == 0 || (x && src2dst), "moe_expand_rows: null input");
  MOE_REQUIRE(row_w == nullptr || T == 0 || topk_w, "moe_expand_rows: row_w needs topk_w");
  MOE_REQUIRE(T >= 0 && K > 0 && K <= moe::kMaxK && E > 0 && align > 0 && M_cap >= 0 &&
                  M_cap <= INT32_MAX,
              "moe_expand_rows: bad sizes (K <= 32)");
  MOE_REQUIRE(H > 0 && H % 8 == 0, "moe_expand_rows: H must be a positive multiple of 8");
  MOE_REQUIRE(ld_x >= H && ld_xe >= H && ld_x % 8 == 0 && ld_xe % 8 == 0,
              "moe_expand_rows: row strides must be multiples of 8, >= H");
  MOE_REQUIRE(moe::aligned(x, 16) && moe::aligned(xe, 16),
              "moe_expand_rows: x and xe must be 16-byte aligned");
  MOE_REQUIRE_DEVICE();
  if (M_cap == 0) return MOE_OK;
  const int nvec = H / 8;
  const int64_t pad_per_expert =
      (align - 1 + moe::kPadRowsPerBlock - 1) / moe::kPadRowsPerBlock;
  const int64_t pad = pad_per_expert * E;
  // up to eight times the blocks that fit at once, so that the hardware evens
  // out what they have to do
  const int64_t items = T * ((nvec + moe::kPieceVec - 1) / moe::kPieceVec);
  const int64_t need = (items + moe::kThreads / 32 - 1) / (moe::kThreads / 32);
  int64_t blocks = static_cast<int64_t>(moe::device_sm_count()) * (2048 / moe::kThreads) * 8;
  if (blocks > need) blocks = need;
  if (pad + blocks == 0) return MOE_OK;
  MOE_REQUIRE(pad + blocks < (1ll << 31), "moe_expand_rows: grid too large");
  moe::expand_rows_kernel<<<static_cast<unsigned>(pad + blocks), moe::kThreads, 0,
                            reinterpret_cast<cudaStream_t>(stream)>>>(
      x, ld_x, topk_w, src2dst, psum, d_n_valid, T, nvec, K, align, M_cap, xe, ld_xe, row_w,
      static_cast<int>(pad_per_expert), static_cast<int>(pad), d_status);
  return moe::check_launch("expand_rows_kernel");
}

extern "C" int moe_collect_row_grads(const float* rows, const int32_t* src2dst,
                                     const int32_t* d_n_valid, int64_t T, int K, int64_t M_cap,
                                     float* out, moe_stream_t stream) {
  MOE_REQUIRE(T >= 0 && K > 0 && K <= moe::kMaxK && M_cap >= 0, "moe_collect_row_grads: bad sizes (K <= 32)");
  MOE_REQUIRE(T == 0 || (src2dst && out && (rows || M_cap == 0)), "moe_collect_row_grads: null pointer");
  MOE_REQUIRE_DEVICE();
  if (T == 0) return MOE_OK;
  int64_t blocks = static_cast<int64_t>(moe::device_sm_count()) * 8;
  const int64_t need = (T * K + moe::kThreads - 1) / moe::kThreads;
  if (blocks > need) blocks = need;
  moe::collect_row_grads_kernel<<<static_cast<unsigned>(blocks), moe::kThreads, 0,
                                  reinterpret_cast<cudaStream_t>(stream)>>>(
      rows, src2dst, d_n_valid, T, K, M_cap, out);
  return moe::check_launch("collect_row_grads_kernel");
}

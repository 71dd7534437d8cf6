// moe_combine_rows: the experts' rows back to their tokens, weighted,
//   y[t] = res[t] + sum_k w[t, k] rows[src2dst[t, k]]
// and its gradient, moe_combine_rows_backward,
//   drows[src2dst[t, k]] = w[t, k] dy[t],  dw[t, k] = sum_h dy[t, h] rows[src2dst[t, k], h].
// Sums in fp32 in a fixed order, each 16-bit result rounded once.
//
// Bytes: a row's 2H per pair, read (and, in the gradient, written), and 2H per
// token: both are bound by HBM. 16384 tokens of H = 7168 with 8 pairs by Zipf: 364 us
// (6.2 TB/s), the gradient 555 us (6.9 TB/s, what a copy reaches). 256 tokens: 8 us,
// a chain of three reads of which each waits for the one before.
#include <algorithm>
#include <type_traits>

#include "dtype16.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kMaxK = 32;
constexpr int kThreads = 256;
constexpr int kPadRowsPerBlock = 8;
constexpr uint32_t kAll = 0xffffffffu;

MOE_DEV int64_t valid_rows(const int32_t* d_n_valid, int64_t T) {
  if (d_n_valid == nullptr) return T;
  const int64_t nv = *d_n_valid;
  return nv < 0 ? 0 : (nv > T ? T : nv);
}

// `parts` warps take a token, each a share of its columns, a 16-byte vector a lane
// at a time; lane k holds pair k's row and weight, and the vectors of kDeep rows
// are asked for before their sum. (The Zipf case with a branch at each gather 608 us,
// gathers predicated and no branch in the sum 389, four at a time instead of eight
// 366, blocks of 128 threads instead of 256 364.)
constexpr int kDeep = 4;
constexpr int kCombineThreads = 128;

template <bool Half>
__global__ void __launch_bounds__(kCombineThreads) combine_rows_kernel(
    const uint16_t* __restrict__ rows, int64_t ld_rows, const float* __restrict__ topk_w,
    const int32_t* __restrict__ src2dst, const int32_t* __restrict__ d_n_valid, int64_t T, int nvec,
    int K, int64_t M_cap, const uint16_t* residual, int64_t ld_res, uint16_t* y, int64_t ld_y,
    int parts, int32_t* __restrict__ status) {
  const int lane = threadIdx.x & 31;
  const int64_t tasks = valid_rows(d_n_valid, T) * parts;
  const int64_t nwarps = (static_cast<int64_t>(gridDim.x) * kCombineThreads) >> 5;
  for (int64_t task = (static_cast<int64_t>(blockIdx.x) * kCombineThreads + threadIdx.x) >> 5; task < tasks;
       task += nwarps) {
    const int64_t t = task <= UINT32_MAX ? static_cast<uint32_t>(task) / static_cast<uint32_t>(parts)
                                         : task / parts;
    const int part = static_cast<int>(task - t * parts);
    int my = -1;
    float my_w = 1.0f;
    if (lane < K) {
      my = src2dst[t * K + lane];
      if (my >= M_cap) {
        set_status(status, MOE_ERR_DEVICE_CHECK);
        my = -1;
      }
      if (topk_w != nullptr) my_w = topk_w[t * K + lane];
    }
    // warp-uniform (the shuffles need every lane); lanes past the row idle
    for (int v0 = part * 32; v0 < nvec; v0 += parts * 32) {
      const int v = v0 + lane;
      const bool act = v < nvec;
      float a[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = 0.0f;
      if (residual != nullptr && act) unpack8<Half>(reinterpret_cast<const uint4*>(residual + t * ld_res)[v], a);
      for (int k0 = 0; k0 < K; k0 += kDeep) {
        uint4 d[kDeep];
        int r[kDeep];
        float w[kDeep];
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
          r[j] = __shfl_sync(kAll, my, (k0 + j) & 31);
          w[j] = __shfl_sync(kAll, my_w, (k0 + j) & 31);
          if (k0 + j >= K || !act) r[j] = -1;
          d[j] = make_uint4(0, 0, 0, 0);
          if (r[j] >= 0) d[j] = __ldcs(reinterpret_cast<const uint4*>(rows + r[j] * ld_rows) + v);
        }
#pragma unroll
        for (int j = 0; j < kDeep; ++j) {
          if (r[j] < 0) w[j] = 0.0f;   // zeros times this; a branch would wait for each row apart
          float f[8];
          unpack8<Half>(d[j], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = fmaf(f[i], w[j], a[i]);
        }
      }
      if (act) reinterpret_cast<uint4*>(y + t * ld_y)[v] = pack8<Half>(a);
    }
  }
}

// Blocks [0, pad_blocks) zero the alignment gaps; of the others kWarps warps
// take a token, each a share of its columns: dy's vector, then each of eight
// pairs' rows. drows may be rows: a lane reads a place before it writes it.
template <bool Half, int kWarps>
__global__ void __launch_bounds__(kThreads) combine_rows_backward_kernel(
    const uint16_t* __restrict__ dy, int64_t ld_dy, const uint16_t* rows, int64_t ld_rows,
    const float* __restrict__ topk_w, const int32_t* __restrict__ src2dst,
    const int32_t* __restrict__ psum, const int32_t* __restrict__ d_n_valid, int64_t T, int nvec, int K,
    int align, int64_t M_cap, uint16_t* drows, int64_t ld_drows, float* __restrict__ dtopk_w,
    int pad_blocks_per_expert, int pad_blocks, int32_t* __restrict__ status) {
  const int tid = threadIdx.x;
  if (static_cast<int>(blockIdx.x) < pad_blocks) {
    const int e = blockIdx.x / pad_blocks_per_expert;
    const int sub = blockIdx.x % pad_blocks_per_expert;
    const int64_t end = max(psum[e], 0);
    int64_t seg_end = (end + align - 1) / align * align;
    if (seg_end > M_cap) seg_end = M_cap;
    const int64_t r0 = end + static_cast<int64_t>(sub) * kPadRowsPerBlock;
    const int64_t r1 = r0 + kPadRowsPerBlock < seg_end ? r0 + kPadRowsPerBlock : seg_end;
    for (int64_t r = r0; r < r1; ++r)
      for (int v = tid; v < nvec; v += kThreads)
        reinterpret_cast<uint4*>(drows + r * ld_drows)[v] = make_uint4(0, 0, 0, 0);
    return;
  }
  __shared__ float s_part[kThreads / 32][8];
  const int lane = tid & 31, warp = tid >> 5;
  constexpr int kTokens = kThreads / 32 / kWarps;   // of a block at a time
  const int64_t nv = valid_rows(d_n_valid, T);
  const int64_t step = static_cast<int64_t>(gridDim.x - pad_blocks) * kTokens;
  // the block's warps go round together: they meet at a barrier
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x - pad_blocks) * kTokens; t0 < nv; t0 += step) {
    const int64_t t = t0 + warp / kWarps;
    const bool live = t < nv;
    int my = -1;
    float my_w = 1.0f;
    if (live && lane < K) {
      my = src2dst[t * K + lane];
      if (my >= M_cap) {
        set_status(status, MOE_ERR_DEVICE_CHECK);
        my = -1;
      }
      if (topk_w != nullptr) my_w = topk_w[t * K + lane];
    }
    const uint4* dy4 = reinterpret_cast<const uint4*>(dy + t * ld_dy);
    for (int k0 = 0; k0 < K; k0 += 8) {
      int64_t r[8];
      float w[8], dot[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r[j] = __shfl_sync(kAll, my, (k0 + j) & 31);
        w[j] = __shfl_sync(kAll, my_w, (k0 + j) & 31);
        if (k0 + j >= K) r[j] = -1;
        dot[j] = 0.0f;
      }
      if (live)
        for (int v = (warp % kWarps) * 32 + lane; v < nvec; v += kWarps * 32) {
          float g[8];
          unpack8<Half>(dy4[v], g);
          uint4 d[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (r[j] >= 0) d[j] = reinterpret_cast<const uint4*>(rows + r[j] * ld_rows)[v];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (r[j] < 0) continue;
            float f[8], o[8];
            unpack8<Half>(d[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              dot[j] = fmaf(g[i], f[i], dot[j]);
              o[i] = g[i] * w[j];
            }
            reinterpret_cast<uint4*>(drows + r[j] * ld_drows)[v] = pack8<Half>(o);
          }
        }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(kAll, dot[j], o);
        if (lane == j) s_part[warp][j] = dot[j];
      }
      if (kWarps > 1) __syncthreads(); else __syncwarp();
      if (live && warp % kWarps == 0 && lane < 8 && k0 + lane < K) {
        float sum = s_part[warp][lane];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) sum += s_part[warp + i][lane];
        dtopk_w[t * K + k0 + lane] = sum;
      }
      if (kWarps > 1) __syncthreads(); else __syncwarp();
    }
  }
}

// Warps for a token in the gradient. 16 warps are resident on an SM (126 registers
// a thread), so a rule on T by whole rounds of them: 8 a token while every token is
// in the first round, or nearly, with long rows; then 2, while those make one round
// or, with long rows, rounds enough that a short last one counts more than the
// sums' two barriers; 1 between and with short rows. us at 1 / 2 / 8, K = 8:
//    256 x 7168  35 /  21 /  13      1536 x 1024  12 /  13 /  19
//    512 x 7168  40 /  27 /  24      1536 x 7168  62 /  65 /  64
//    768 x 7168  43 /  33 /  35      3000 x 7168 122 / 113 / 116
//    768 x 1024 6.8 / 5.8 / 8.1      8192 x 1024  49 /  50 /  88
int backward_warps(int64_t T, int nvec) {
  const int64_t sms = device_sm_count();
  if (nvec <= 32) return 1;
  if (T <= 2 * sms || (T <= 4 * sms && nvec >= 512)) return 8;
  if (T <= 8 * sms) return 2;
  return T <= 16 * sms || nvec <= 128 ? 1 : 2;
}
constexpr int kCombineBlocks = 64;

}  // namespace
}  // namespace moe

extern "C" int moe_combine_rows(const void* rows, int64_t ld_rows, int dtype, const float* topk_w,
                                const int32_t* src2dst, const int32_t* d_n_valid, int64_t T, int H,
                                int K, int64_t M_cap, const void* residual, int64_t ld_res, void* out,
                                int64_t ld_out, int32_t* d_status, moe_stream_t stream) {
  MOE_REQUIRE(T >= 0 && K > 0 && K <= moe::kMaxK && M_cap >= 0 && M_cap <= INT32_MAX,
              "moe_combine_rows: bad sizes (K <= 32)");
  MOE_REQUIRE(T == 0 || ((rows || M_cap == 0) && src2dst && out), "moe_combine_rows: null pointer");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "moe_combine_rows: dtype must be MOE_BF16 or MOE_F16");
  MOE_REQUIRE(H > 0 && H % 8 == 0, "moe_combine_rows: H must be a positive multiple of 8");
  MOE_REQUIRE(ld_rows >= H && ld_out >= H && ld_rows % 8 == 0 && ld_out % 8 == 0 &&
                  (residual == nullptr || (ld_res >= H && ld_res % 8 == 0)),
              "moe_combine_rows: row strides must be multiples of 8, >= H");
  MOE_REQUIRE(moe::aligned(rows, 16) && moe::aligned(out, 16) && moe::aligned(residual, 16),
              "moe_combine_rows: rows, residual and out must be 16-byte aligned");
  MOE_REQUIRE(residual != out || residual == nullptr || ld_res == ld_out,
              "moe_combine_rows: in place needs the same row stride for residual and out");
  MOE_REQUIRE(rows != out || T == 0 || M_cap == 0, "moe_combine_rows: out must not be rows");
  MOE_REQUIRE_DEVICE();
  if (T == 0) return MOE_OK;
  // warps for a token: one where there are tokens for every warp that fits, up to
  // one for every 32 vectors where there are few
  const int chunks = (H / 8 + 31) / 32;
  const int64_t fit = static_cast<int64_t>(moe::device_sm_count()) * 48;
  const int parts = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(chunks, fit / T)));
  const int64_t need = (T * parts + moe::kCombineThreads / 32 - 1) / (moe::kCombineThreads / 32);
  const int64_t most = static_cast<int64_t>(moe::device_sm_count()) * moe::kCombineBlocks;
  const int64_t grid = need < most ? need : most;
  auto* kernel = dtype == MOE_F16 ? moe::combine_rows_kernel<true> : moe::combine_rows_kernel<false>;
  kernel<<<static_cast<unsigned>(grid), moe::kCombineThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(rows), ld_rows, topk_w, src2dst, d_n_valid, T, H / 8, K, M_cap,
      static_cast<const uint16_t*>(residual), ld_res, static_cast<uint16_t*>(out), ld_out, parts, d_status);
  return moe::check_launch("combine_rows_kernel");
}

extern "C" int moe_combine_rows_backward(const void* dy, int64_t ld_dy, const void* rows,
                                         int64_t ld_rows, int dtype, const float* topk_w,
                                         const int32_t* src2dst, const int32_t* psum,
                                         const int32_t* d_n_valid, int64_t T, int H, int K, int E,
                                         int align, int64_t M_cap, void* drows, int64_t ld_drows,
                                         float* dtopk_w, int32_t* d_status, moe_stream_t stream) {
  MOE_REQUIRE(T >= 0 && K > 0 && K <= moe::kMaxK && E > 0 && align > 0 && M_cap >= 0 && M_cap <= INT32_MAX,
              "moe_combine_rows_backward: bad sizes (K <= 32)");
  MOE_REQUIRE(psum && (M_cap == 0 || (rows && drows)), "moe_combine_rows_backward: null psum, rows or drows");
  MOE_REQUIRE(T == 0 || (dy && src2dst && dtopk_w), "moe_combine_rows_backward: null pointer");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16,
              "moe_combine_rows_backward: dtype must be MOE_BF16 or MOE_F16");
  MOE_REQUIRE(H > 0 && H % 8 == 0, "moe_combine_rows_backward: H must be a positive multiple of 8");
  MOE_REQUIRE(ld_dy >= H && ld_rows >= H && ld_drows >= H && ld_dy % 8 == 0 && ld_rows % 8 == 0 &&
                  ld_drows % 8 == 0,
              "moe_combine_rows_backward: row strides must be multiples of 8, >= H");
  MOE_REQUIRE(moe::aligned(dy, 16) && moe::aligned(rows, 16) && moe::aligned(drows, 16),
              "moe_combine_rows_backward: dy, rows and drows must be 16-byte aligned");
  MOE_REQUIRE(rows != drows || ld_rows == ld_drows,
              "moe_combine_rows_backward: in place needs the same row stride for rows and drows");
  const int64_t pad_per_expert = (align - 1 + moe::kPadRowsPerBlock - 1) / moe::kPadRowsPerBlock;
  const int64_t pad = M_cap == 0 ? 0 : pad_per_expert * E;
  MOE_REQUIRE(pad < (1ll << 30), "moe_combine_rows_backward: grid too large");
  MOE_REQUIRE(dy != drows || T == 0 || M_cap == 0, "moe_combine_rows_backward: drows must not be dy");
  MOE_REQUIRE_DEVICE();
  const int nvec = H / 8;
  const int64_t most = static_cast<int64_t>(moe::device_sm_count()) * (2048 / moe::kThreads) * 8;
  const int warps = moe::backward_warps(T, nvec);
  const int tokens = moe::kThreads / 32 / warps;   // of a block at a time
  const int64_t need = (T + tokens - 1) / tokens;
  const int64_t blocks = need < most ? need : most;
  if (pad + blocks == 0) return MOE_OK;
  auto pick = [warps](auto half) {
    constexpr bool kHalf = decltype(half)::value;
    return warps == 1   ? moe::combine_rows_backward_kernel<kHalf, 1>
           : warps == 2 ? moe::combine_rows_backward_kernel<kHalf, 2>
                        : moe::combine_rows_backward_kernel<kHalf, 8>;
  };
  auto* kernel = dtype == MOE_F16 ? pick(std::true_type{}) : pick(std::false_type{});
  kernel<<<static_cast<unsigned>(pad + blocks), moe::kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(dy), ld_dy, static_cast<const uint16_t*>(rows), ld_rows, topk_w, src2dst,
      psum, d_n_valid, T, nvec, K, align, M_cap, static_cast<uint16_t*>(drows), ld_drows, dtopk_w,
      static_cast<int>(pad_per_expert), static_cast<int>(pad), d_status);
  return moe::check_launch("combine_rows_backward_kernel");
}

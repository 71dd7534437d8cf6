// moe_swiglu / moe_swiglu_backward: the activation between the two 16-bit
// grouped products, with the pair's routing weight, and its gradient.
//   s = 1 / (1 + e^-g),  h = (g s) u w
//   dg = dh w u s (1 + g (1 - s)),  du = dh w g s,  dw = sum_i dh_i (g_i s_i) u_i
// per row of gu = [g | u]. All arithmetic is in fp32; h, dg and du are rounded
// once to the 16-bit type, dw stays fp32.
//
// Bytes a row: 6I + 4 forward, 10I + 8 backward, so both are bound by HBM. A
// group of kGroup lanes takes a row (the backward needs the row's sum): a
// warp, whose 16-byte vectors of g, u (and dh) are one contiguous 512-byte run
// per instruction, or, for rows of few vectors, the 8 or 16 lanes that leave
// the fewest idle.
// e^x is the hardware's base-2 exponential and the quotient its reciprocal: with
// correctly rounded ones the arithmetic, not HBM, would set the time of the
// backward. Their bounds are 2 + 1.173 |x| ulp (the argument is rounded before
// the exponential) and 2 ulp, so s is within 2^-19 of its value for |g| <= 8 and
// within 2^-16 at g = -60 (below -87, where it is under 2^-125, it is 0); h, dg
// and du are rounded to 2^-8 (bf16) or 2^-11 (fp16) anyway. For g > 0 the exponential
// is added to 1 and its error shrinks with it. dw is fp32 and takes the larger
// errors of its very negative g, in terms that are e^g of the others.
#include "dtype16.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

MOE_DEV float sigmoid_fast(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

template <bool Half, int kGroup>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(
    const uint16_t* __restrict__ gu, int64_t ld_gu, int nvec, const float* __restrict__ row_w,
    const int32_t* __restrict__ d_total, int64_t M_cap, uint16_t* __restrict__ h, int64_t ld_h) {
  const int lane = threadIdx.x % kGroup;
  int64_t total = *d_total;
  if (total > M_cap) total = M_cap;
  constexpr int kRows = kThreads / kGroup;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup; r < total;
       r += step) {
    const uint4* g4 = reinterpret_cast<const uint4*>(gu + r * ld_gu);
    const uint4* u4 = g4 + nvec;
    uint4* h4 = reinterpret_cast<uint4*>(h + r * ld_h);
    const float w = row_w != nullptr ? row_w[r] : 1.0f;
    for (int v = lane; v < nvec; v += kGroup) {
      float g[8], u[8];
      unpack8<Half>(__ldcs(g4 + v), g);
      unpack8<Half>(__ldcs(u4 + v), u);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = g[i] * sigmoid_fast(g[i]) * u[i] * w;
      h4[v] = pack8<Half>(g);
    }
  }
}

// dgu may be gu itself: a lane reads its vectors of g and u before it writes
// the same places, and no other lane touches them (so no __restrict__ or
// read-only loads on gu here).
template <bool Half, int kGroup>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(
    const uint16_t* __restrict__ dh, int64_t ld_dh, const uint16_t* gu, int64_t ld_gu, int nvec,
    const float* __restrict__ row_w, const int32_t* __restrict__ d_total, int64_t M_cap,
    uint16_t* dgu, int64_t ld_dgu, float* __restrict__ drow_w) {
  const int lane = threadIdx.x % kGroup;
  int64_t total = *d_total;
  if (total > M_cap) total = M_cap;
  constexpr int kRows = kThreads / kGroup;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kGroup; r < total;
       r += step) {
    const uint4* g4 = reinterpret_cast<const uint4*>(gu + r * ld_gu);
    const uint4* d4 = reinterpret_cast<const uint4*>(dh + r * ld_dh);
    uint4* o4 = reinterpret_cast<uint4*>(dgu + r * ld_dgu);
    const float w = row_w != nullptr ? row_w[r] : 1.0f;
    float sum = 0.0f;
    for (int v = lane; v < nvec; v += kGroup) {
      float g[8], u[8], d[8];
      unpack8<Half>(g4[v], g);
      unpack8<Half>(g4[nvec + v], u);
      unpack8<Half>(__ldcs(d4 + v), d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float s = sigmoid_fast(g[i]);
        const float a = g[i] * s;          // silu(g)
        const float dw = d[i] * w;
        sum += d[i] * (a * u[i]);
        g[i] = dw * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
        u[i] = dw * a;
      }
      o4[v] = pack8<Half>(g);
      o4[nvec + v] = pack8<Half>(u);
    }
    if (drow_w != nullptr) {
      // the row's own lanes: rows of one warp may end their loops apart
      const uint32_t lanes = kGroup == 32 ? 0xffffffffu
                                          : ((1u << (kGroup % 32)) - 1u) << (threadIdx.x % 32 / kGroup * kGroup);
#pragma unroll
      for (int o = kGroup / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(lanes, sum, o);
      if (lane == 0) drow_w[r] = sum;
    }
  }
}

// Lanes per row: a warp from two vectors a lane on (at I = 560 it takes 38 us
// for 65536 rows, eight lanes 43; at 1096 75 and 86), below that the group that
// idles least, the widest of equals (at 72 6.7 us with eight lanes, 12.0 with a
// warp; at 264 15.8 and 26.6).
int group_for(int nvec) {
  if (nvec >= 64) return 32;
  int best = 32, least = (nvec + 31) / 32 * 32;
  for (int g = 16; g >= 8; g /= 2) {
    const int n = (nvec + g - 1) / g * g;
    if (n < least) {
      best = g;
      least = n;
    }
  }
  return best;
}

// Up to eight times the blocks that fit at once: the hardware hands out rows
// as blocks finish, and rows of a large buffer past `total` cost little.
unsigned grid_for(int64_t rows, int group) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * (2048 / kThreads) * 8;
  const int64_t per = kThreads / group;
  const int64_t need = (rows + per - 1) / per;
  return static_cast<unsigned>(need < most ? need : most);
}

template <int kGroup>
void launch_forward(bool half, const uint16_t* gu, int64_t ld_gu, int nvec, const float* row_w,
                    const int32_t* d_total, int64_t M_cap, uint16_t* h, int64_t ld_h, cudaStream_t s) {
  auto* kernel = half ? swiglu_kernel<true, kGroup> : swiglu_kernel<false, kGroup>;
  kernel<<<grid_for(M_cap, kGroup), kThreads, 0, s>>>(gu, ld_gu, nvec, row_w, d_total, M_cap, h, ld_h);
}

template <int kGroup>
void launch_backward(bool half, const uint16_t* dh, int64_t ld_dh, const uint16_t* gu, int64_t ld_gu,
                     int nvec, const float* row_w, const int32_t* d_total, int64_t M_cap,
                     uint16_t* dgu, int64_t ld_dgu, float* drow_w, cudaStream_t s) {
  auto* kernel = half ? swiglu_backward_kernel<true, kGroup> : swiglu_backward_kernel<false, kGroup>;
  kernel<<<grid_for(M_cap, kGroup), kThreads, 0, s>>>(dh, ld_dh, gu, ld_gu, nvec, row_w, d_total, M_cap,
                                                      dgu, ld_dgu, drow_w);
}

}  // namespace
}  // namespace moe

extern "C" int moe_swiglu(const void* gu, int64_t ld_gu, int dtype, int I, const float* row_w,
                          const int32_t* d_total, int64_t M_cap, void* h, int64_t ld_h,
                          moe_stream_t stream) {
  MOE_REQUIRE(M_cap == 0 || (gu && d_total && h), "moe_swiglu: null pointer");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "moe_swiglu: dtype must be MOE_BF16 or MOE_F16");
  MOE_REQUIRE(I > 0 && I % 8 == 0 && M_cap >= 0 && M_cap <= INT32_MAX,
              "moe_swiglu: I must be a positive multiple of 8");
  MOE_REQUIRE(ld_gu >= 2ll * I && ld_h >= I && ld_gu % 8 == 0 && ld_h % 8 == 0,
              "moe_swiglu: row strides must be multiples of 8, at least the row");
  MOE_REQUIRE(moe::aligned(gu, 16) && moe::aligned(h, 16), "moe_swiglu: gu and h must be 16-byte aligned");
  MOE_REQUIRE_DEVICE();
  if (M_cap == 0) return MOE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int group = moe::group_for(I / 8);
  auto launch = group == 32 ? moe::launch_forward<32>
                            : (group == 16 ? moe::launch_forward<16> : moe::launch_forward<8>);
  launch(dtype == MOE_F16, static_cast<const uint16_t*>(gu), ld_gu, I / 8, row_w, d_total, M_cap,
         static_cast<uint16_t*>(h), ld_h, s);
  return moe::check_launch("swiglu_kernel");
}

extern "C" int moe_swiglu_backward(const void* dh, int64_t ld_dh, const void* gu, int64_t ld_gu,
                                   int dtype, int I, const float* row_w, const int32_t* d_total,
                                   int64_t M_cap, void* dgu, int64_t ld_dgu, float* drow_w,
                                   moe_stream_t stream) {
  MOE_REQUIRE(M_cap == 0 || (dh && gu && d_total && dgu), "moe_swiglu_backward: null pointer");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16,
              "moe_swiglu_backward: dtype must be MOE_BF16 or MOE_F16");
  MOE_REQUIRE(I > 0 && I % 8 == 0 && M_cap >= 0 && M_cap <= INT32_MAX,
              "moe_swiglu_backward: I must be a positive multiple of 8");
  MOE_REQUIRE(ld_gu >= 2ll * I && ld_dgu >= 2ll * I && ld_dh >= I && ld_gu % 8 == 0 &&
                  ld_dgu % 8 == 0 && ld_dh % 8 == 0,
              "moe_swiglu_backward: row strides must be multiples of 8, at least the row");
  MOE_REQUIRE(moe::aligned(dh, 16) && moe::aligned(gu, 16) && moe::aligned(dgu, 16),
              "moe_swiglu_backward: dh, gu and dgu must be 16-byte aligned");
  MOE_REQUIRE(gu != dgu || ld_gu == ld_dgu,
              "moe_swiglu_backward: in place needs the same row stride for gu and dgu");
  MOE_REQUIRE_DEVICE();
  if (M_cap == 0) return MOE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int group = moe::group_for(I / 8);
  auto launch = group == 32 ? moe::launch_backward<32>
                            : (group == 16 ? moe::launch_backward<16> : moe::launch_backward<8>);
  launch(dtype == MOE_F16, static_cast<const uint16_t*>(dh), ld_dh, static_cast<const uint16_t*>(gu),
         ld_gu, I / 8, row_w, d_total, M_cap, static_cast<uint16_t*>(dgu), ld_dgu, drow_w, s);
  return moe::check_launch("swiglu_backward_kernel");
}

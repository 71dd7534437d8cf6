// moe_route_topk / moe_route_topk_backward: the router's choice of K of E
// experts and their weights, and the gradient of its logits.
//   key_e = fl32(l_e + b_e);  ids = the K largest keys, ties to the lowest e
//   softmax: w_k = c p[i_k], p = softmax(l) over E, or over the chosen
//   sigmoid: w_k = c s[i_k], s = 1 / (1 + e^-l), or c s[i_k] / sum_j s[i_j]
// A warp takes a row; lane a holds the logits of experts [a n, a n + n), n =
// ceil(E / 32), so that of equal keys the lowest expert is the lowest lane's
// first. A round finds the largest key of the warp with one redux.sync on keys
// mapped to unsigned integers of the same order, and strikes it out.
#include "dtype16.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxK = 32;
constexpr int kMaxE = 1024;
constexpr uint32_t kAll = 0xffffffffu;

MOE_DEV float load_logit(const void* p, int64_t i, int dtype) {
  if (dtype == MOE_F32) return __ldg(static_cast<const float*>(p) + i);
  const uint32_t w = __ldg(static_cast<const uint16_t*>(p) + i);
  return dtype == MOE_F16 ? unpack2<true>(w).x : unpack2<false>(w).x;
}

MOE_DEV void store_logit(void* p, int64_t i, int dtype, float v) {
  if (dtype == MOE_F32)
    static_cast<float*>(p)[i] = v;
  else
    static_cast<uint16_t*>(p)[i] =
        static_cast<uint16_t>((dtype == MOE_F16 ? pack2<true>(v, 0.0f) : pack2<false>(v, 0.0f)) & 0xffffu);
}

// Unsigned integers in the order of the keys; 0: never chosen (-inf, NaN). -0
// and +0 are one key.
MOE_DEV uint32_t order_of(float key) {
  if (!(key > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(key + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

MOE_DEV float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
MOE_DEV float warp_max(float v) {   // of the values that are no NaN
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

MOE_DEV int64_t valid_rows(const int32_t* d_n_valid, int64_t T) {
  if (d_n_valid == nullptr) return T;
  const int64_t nv = *d_n_valid;
  return nv < 0 ? 0 : (nv > T ? T : nv);
}

// sigmoid(l) e^-shift, shift <= 0: with shift the smaller of 0 and the largest l
// of a row, the quotients of very negative logits keep their digits.
MOE_DEV float sigmoid_shifted(float l, float shift) {
  return l >= 0.0f ? 1.0f / (1.0f + expf(-l)) : expf(l - shift) / (1.0f + expf(l));
}

// The weights of the chosen, before the factor: lane k has pair k's logit
// (ok: it has one). m, sum: the row's largest logit and sum of e^(l - m).
MOE_DEV float weight_of(float l, bool ok, bool sigmoid, bool renormalize, float m, float sum) {
  if (!renormalize) {
    if (!ok) return 0.0f;
    return sigmoid ? sigmoid_shifted(l, 0.0f) : expf(l - m) / sum;
  }
  const float top = warp_max(ok ? l : -INFINITY);
  float s = 0.0f;
  if (ok) s = sigmoid ? sigmoid_shifted(l, fminf(top, 0.0f)) : expf(l - top);
  const float all = warp_sum(s);
  return ok ? s / all : 0.0f;
}

template <int kN>
__global__ void __launch_bounds__(kThreads) route_topk_kernel(
    const void* __restrict__ logits, int64_t ld, int dtype, const float* __restrict__ bias,
    const int32_t* __restrict__ d_n_valid, int64_t T, int E, int K, bool sigmoid, bool renormalize,
    float factor, int32_t* __restrict__ ids, float* __restrict__ weights) {
  const int lane = threadIdx.x & 31;
  const int64_t nv = valid_rows(d_n_valid, T);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  const int e0 = lane * kN;
  float b[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) b[j] = bias != nullptr && e0 + j < E ? bias[e0 + j] : 0.0f;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < nv;
       t += step) {
    float l[kN];
    uint32_t u[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      l[j] = e0 + j < E ? load_logit(logits, t * ld + e0 + j, dtype) : -INFINITY;
      u[j] = order_of(l[j] + b[j]);
    }
    float m = 0.0f, sum = 1.0f;
    if (!sigmoid && !renormalize) {
      m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) m = fmaxf(m, l[j]);
      m = warp_max(m);
      sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (e0 + j < E) sum += expf(l[j] - m);
      sum = warp_sum(sum);
    }
    int my = -1;
    for (int k = 0; k < K; ++k) {
      uint32_t best = 0;
#pragma unroll
      for (int j = 0; j < kN; ++j) best = max(best, u[j]);
      const uint32_t top = __reduce_max_sync(kAll, best);
      if (top == 0) break;
      const int owner = __ffs(__ballot_sync(kAll, best == top)) - 1;
      int e = 0;
      bool open = lane == owner;
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (open && u[j] == top) {
          u[j] = 0;
          e = e0 + j;
          open = false;
        }
      e = __shfl_sync(kAll, e, owner);
      if (lane == k) my = e;
    }
    const bool ok = my >= 0;
    const float w = weight_of(ok ? load_logit(logits, t * ld + my, dtype) : 0.0f, ok, sigmoid,
                              renormalize, m, sum);
    if (lane < K) {
      ids[t * K + lane] = my;
      weights[t * K + lane] = ok ? factor * w : 0.0f;
    }
  }
}

// dl over the whole row is written first where every expert has one (softmax
// over E) or zero; then lane k writes pair k's expert, the warp's stores being
// ordered by __syncwarp.
template <int kN>
__global__ void __launch_bounds__(kThreads) route_topk_backward_kernel(
    const float* __restrict__ dweights, const void* __restrict__ logits, int64_t ld, int dtype,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ d_n_valid, int64_t T, int E, int K,
    bool sigmoid, bool renormalize, float factor, void* dlogits, int64_t ld_d) {
  const int lane = threadIdx.x & 31;
  const int64_t nv = valid_rows(d_n_valid, T);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5); t < nv;
       t += step) {
    const int my = lane < K ? ids[t * K + lane] : -1;
    const bool ok = my >= 0 && my < E;
    const float g = ok ? factor * dweights[t * K + lane] : 0.0f;
    const float lk = ok ? load_logit(logits, t * ld + my, dtype) : 0.0f;
    float d;   // of pair k's logit
    if (!sigmoid && !renormalize) {
      float l[kN], m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int e = j * 32 + lane;
        l[j] = e < E ? load_logit(logits, t * ld + e, dtype) : -INFINITY;
        m = fmaxf(m, l[j]);
      }
      m = warp_max(m);
      const bool any = m > -INFINITY;   // else a row without experts: its gradient is 0
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        l[j] = any || l[j] != l[j] ? expf(l[j] - m) : 0.0f;
        if (j * 32 + lane < E) sum += l[j];
      }
      sum = warp_sum(sum);
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
      const float pk = ok ? expf(lk - m) * inv : 0.0f;
      const float mean = warp_sum(g * pk);
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int e = j * 32 + lane;
        if (e < E) store_logit(dlogits, t * ld_d + e, dtype, -(l[j] * inv) * mean);
      }
      // the same expert more than once: each of its pairs adds
      float ge = g;
      if (__any_sync(kAll, __popc(__match_any_sync(kAll, ok ? my : -1 - lane)) > 1)) {
        ge = 0.0f;
        for (int k = 0; k < K; ++k) {
          const int id = __shfl_sync(kAll, my, k);
          const float gk = __shfl_sync(kAll, g, k);
          if (id == my) ge += gk;
        }
      }
      d = pk * (ge - mean);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const int e = j * 32 + lane;
        if (e < E) store_logit(dlogits, t * ld_d + e, dtype, 0.0f);
      }
      if (renormalize) {
        const float r = weight_of(lk, ok, sigmoid, true, 0.0f, 1.0f);
        const float mean = warp_sum(ok ? g * r : 0.0f);
        d = r * (g - mean);
        if (sigmoid) d *= sigmoid_shifted(-lk, 0.0f);   // 1 - s
      } else {
        d = g * sigmoid_shifted(lk, 0.0f) * sigmoid_shifted(-lk, 0.0f);
      }
      if (__any_sync(kAll, __popc(__match_any_sync(kAll, ok ? my : -1 - lane)) > 1)) {
        float all = 0.0f;
        for (int k = 0; k < K; ++k) {
          const int id = __shfl_sync(kAll, my, k);
          const float dk = __shfl_sync(kAll, d, k);
          if (id == my) all += dk;
        }
        d = all;
      }
    }
    __syncwarp();
    if (ok) store_logit(dlogits, t * ld_d + my, dtype, d);
    __syncwarp();
  }
}

unsigned grid_for(int64_t rows) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * (2048 / kThreads) * 8;
  const int64_t need = (rows + kThreads / 32 - 1) / (kThreads / 32);
  return static_cast<unsigned>(need < most ? need : most);
}

}  // namespace
}  // namespace moe

#define MOE_BY_WIDTH(E, LAUNCH) \
  do {                          \
    const int n_ = (E + 31) / 32; \
    if (n_ <= 1) LAUNCH(1);       \
    else if (n_ <= 2) LAUNCH(2);  \
    else if (n_ <= 4) LAUNCH(4);  \
    else if (n_ <= 8) LAUNCH(8);  \
    else if (n_ <= 16) LAUNCH(16); \
    else LAUNCH(32);              \
  } while (0)

extern "C" int moe_route_topk(const void* logits, int64_t ld, int dtype, const float* bias,
                              const int32_t* d_n_valid, int64_t T, int E, int K, int score,
                              int renormalize, float factor, int32_t* topk_ids, float* topk_w,
                              moe_stream_t stream) {
  MOE_REQUIRE(T >= 0 && E > 0 && E <= moe::kMaxE && K > 0 && K <= moe::kMaxK && K <= E,
              "moe_route_topk: bad sizes (E <= 1024, K <= 32, K <= E)");
  MOE_REQUIRE(T == 0 || (logits && topk_ids && topk_w), "moe_route_topk: null pointer");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16 || dtype == MOE_F32, "moe_route_topk: unknown dtype");
  MOE_REQUIRE(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, "moe_route_topk: unknown score");
  MOE_REQUIRE(ld >= E, "moe_route_topk: the row stride must be at least E");
  MOE_REQUIRE(moe::aligned(logits, dtype == MOE_F32 ? 4 : 2) && moe::aligned(bias, 4) &&
                  moe::aligned(topk_ids, 4) && moe::aligned(topk_w, 4),
              "moe_route_topk: misaligned pointer");
  MOE_REQUIRE_DEVICE();
  if (T == 0) return MOE_OK;
#define LAUNCH(n)                                                                              \
  moe::route_topk_kernel<n><<<moe::grid_for(T), moe::kThreads, 0,                              \
                              reinterpret_cast<cudaStream_t>(stream)>>>(                       \
      logits, ld, dtype, bias, d_n_valid, T, E, K, score == MOE_SCORE_SIGMOID, renormalize != 0, \
      factor, topk_ids, topk_w)
  MOE_BY_WIDTH(E, LAUNCH);
#undef LAUNCH
  return moe::check_launch("route_topk_kernel");
}

extern "C" int moe_route_topk_backward(const float* dtopk_w, const void* logits, int64_t ld, int dtype,
                                       const int32_t* topk_ids, const int32_t* d_n_valid, int64_t T,
                                       int E, int K, int score, int renormalize, float factor,
                                       void* dlogits, int64_t ld_d, moe_stream_t stream) {
  MOE_REQUIRE(T >= 0 && E > 0 && E <= moe::kMaxE && K > 0 && K <= moe::kMaxK && K <= E,
              "moe_route_topk_backward: bad sizes (E <= 1024, K <= 32, K <= E)");
  MOE_REQUIRE(T == 0 || (dtopk_w && logits && topk_ids && dlogits), "moe_route_topk_backward: null pointer");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16 || dtype == MOE_F32,
              "moe_route_topk_backward: unknown dtype");
  MOE_REQUIRE(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID,
              "moe_route_topk_backward: unknown score");
  MOE_REQUIRE(ld >= E && ld_d >= E, "moe_route_topk_backward: row strides must be at least E");
  const uintptr_t size = dtype == MOE_F32 ? 4 : 2;
  MOE_REQUIRE(moe::aligned(logits, size) && moe::aligned(dlogits, size) && moe::aligned(dtopk_w, 4) &&
                  moe::aligned(topk_ids, 4),
              "moe_route_topk_backward: misaligned pointer");
  MOE_REQUIRE(logits != dlogits || T == 0, "moe_route_topk_backward: dlogits must not be logits");
  MOE_REQUIRE_DEVICE();
  if (T == 0) return MOE_OK;
#define LAUNCH(n)                                                                                 \
  moe::route_topk_backward_kernel<n><<<moe::grid_for(T), moe::kThreads, 0,                        \
                                       reinterpret_cast<cudaStream_t>(stream)>>>(                 \
      dtopk_w, logits, ld, dtype, topk_ids, d_n_valid, T, E, K, score == MOE_SCORE_SIGMOID,       \
      renormalize != 0, factor, dlogits, ld_d)
  MOE_BY_WIDTH(E, LAUNCH);
#undef LAUNCH
  return moe::check_launch("route_topk_backward_kernel");
}

// moe_route_topk / moe_route_topk_backward: the router's choice of K of E
// experts and their weights, and the gradient of its logits.
//   key_e = fl32(l_e + b_e);  ids = the K largest keys, ties to the lowest e
//   softmax: w_k = c p[i_k], p = softmax(l) over E, or over the chosen
//   sigmoid: w_k = c s[i_k], s = 1 / (1 + e^-l), or c s[i_k] / sum_j s[i_j]
// A group of lanes takes a row: a warp, or 8 lanes where there are many rows of few
// experts. Lane i of a group of n holds the logits and keys of experts i, i + n, ...
// Keys are mapped to unsigned integers of the same order; a round finds the
// largest of the group and the lowest expert that has it. A lane keeps its keys in
// sorted runs of up to six (a stable insertion sort): a round looks at the runs'
// heads, and the chosen one's run moves up.
//
// Bytes: a row's logits and 8K (12K and twice the logits back). The instructions
// of a row set the time, not the bytes: 32768 x 160 fp32, K = 8, sigmoid, take 15.0 us
// (1.5 TB/s; issue slots 65 % busy, the pipe of comparisons and selects 62 %), their
// softmax gradient 10.5 us (4.2 TB/s). Every key searched again each round took 36 us,
// one sorted run of 5 by a warp 19, runs by 8 lanes in blocks of 256 threads 17; 1024
// experts, 5120 rows, took 30 us unsorted and 18 in runs of 4.
#include "dtype16.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
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

// A lane's part of a row that begins at element `row`: every kLanes-th logit from the
// lane's own on; places from E on are -inf.
template <int kLanes, int kN>
MOE_DEV void load_part(const void* p, int64_t row, int lane, int E, int dtype, float (&l)[kN]) {
  if (dtype == MOE_F32) {
    const float* f = static_cast<const float*>(p) + row + lane;
#pragma unroll
    for (int j = 0; j < kN; ++j) l[j] = j * kLanes + lane < E ? __ldg(f + j * kLanes) : -INFINITY;
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p) + row + lane;
    uint32_t w[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j) w[j] = j * kLanes + lane < E ? __ldg(h + j * kLanes) : 0u;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      l[j] = dtype == MOE_F16 ? unpack2<true>(w[j]).x : unpack2<false>(w[j]).x;
      if (j * kLanes + lane >= E) l[j] = -INFINITY;
    }
  }
}
template <int kLanes, int kN>
MOE_DEV void store_part(void* p, int64_t row, int lane, int E, int dtype, const float (&v)[kN]) {
  if (dtype == MOE_F32) {
    float* f = static_cast<float*>(p) + row + lane;
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (j * kLanes + lane < E) f[j * kLanes] = v[j];
  } else {
    uint16_t* h = static_cast<uint16_t*>(p) + row + lane;
#pragma unroll
    for (int j = 0; j < kN; ++j)
      if (j * kLanes + lane < E)
        h[j * kLanes] = static_cast<uint16_t>(
            (dtype == MOE_F16 ? pack2<true>(v[j], 0.0f) : pack2<false>(v[j], 0.0f)) & 0xffffu);
  }
}

// Unsigned integers in the order of the keys; 0: never chosen (-inf, NaN). -0
// and +0 are one key.
MOE_DEV uint32_t order_of(float key) {
  if (!(key > -INFINITY)) return 0u;
  const uint32_t b = __float_as_uint(key + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Over the lanes of a group; every lane of the warp calls these.
template <int kLanes>
MOE_DEV float group_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
template <int kLanes>
MOE_DEV uint32_t group_max(uint32_t v) {
  if constexpr (kLanes == 32) return __reduce_max_sync(kAll, v);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int kLanes>
MOE_DEV uint32_t group_min(uint32_t v) {
  if constexpr (kLanes == 32) return __reduce_min_sync(kAll, v);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
template <int kLanes>
MOE_DEV float group_max(float v) {   // of the values that are no NaN; -inf if there are none
  if constexpr (kLanes == 32) {
    const uint32_t b = __float_as_uint(v);
    const uint32_t top = group_max<32>(v != v ? 0u : (b & 0x80000000u ? ~b : b | 0x80000000u));
    return top == 0u ? -INFINITY : __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
  }
  v = fmaxf(v, -INFINITY);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
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

// The weights of the chosen, before the factor: lane k of a group has pair k's
// logit (ok: it has one). m, sum: the row's largest logit and sum of e^(l - m).
template <int kLanes>
MOE_DEV float weight_of(float l, bool ok, bool sigmoid, bool renormalize, float m, float sum) {
  if (!renormalize) {
    if (!ok) return 0.0f;
    return sigmoid ? sigmoid_shifted(l, 0.0f) : expf(l - m) / sum;
  }
  const float top = group_max<kLanes>(ok ? l : -INFINITY);
  float s = 0.0f;
  if (ok) s = sigmoid ? sigmoid_shifted(l, fminf(top, 0.0f)) : expf(l - top);
  const float all = group_sum<kLanes>(s);
  return ok ? s / all : 0.0f;
}

// Keys of a sorted run, of the n of a lane.
constexpr int run_of(int n) { return n % 4 == 0 ? 4 : n; }

template <int kLanes, int kN>
__global__ void __launch_bounds__(kThreads) route_topk_kernel(
    const void* __restrict__ logits, int64_t ld, int dtype, const float* __restrict__ bias,
    const int32_t* __restrict__ d_n_valid, int64_t T, int E, int K, bool sigmoid, bool renormalize,
    float factor, int32_t* __restrict__ ids, float* __restrict__ weights) {
  constexpr int kRows = kThreads / kLanes;   // of a block
  constexpr int kRun = run_of(kN);
  const int lane = threadIdx.x % kLanes;
  const int64_t nv = valid_rows(d_n_valid, T);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  float b[kN];
#pragma unroll
  for (int j = 0; j < kN; ++j) b[j] = bias != nullptr && j * kLanes + lane < E ? bias[j * kLanes + lane] : 0.0f;
  // the warp goes round together; a group past the last row does it once more
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / 32 * (32 / kLanes); t0 < nv;
       t0 += step) {
    const int64_t row = t0 + threadIdx.x % 32 / kLanes;
    const bool live = row < nv;
    const int64_t t = live ? row : nv - 1;
    float l[kN];
    uint32_t u[kN];
    int at[kN];   // the keys' experts
    load_part<kLanes, kN>(logits, t * ld, lane, E, dtype, l);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      at[j] = j * kLanes + lane;
      u[j] = order_of(l[j] + b[j]);
    }
    float m = 0.0f, sum = 1.0f;
    if (!sigmoid && !renormalize) {
      m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) m = fmaxf(m, l[j]);
      m = group_max<kLanes>(m);
      sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kN; ++j)
        if (at[j] < E) sum += expf(l[j] - m);
      sum = group_sum<kLanes>(sum);
    }
#pragma unroll
    for (int h = 0; h < kN; h += kRun)
#pragma unroll
      for (int i = h + 1; i < h + kRun; ++i)
#pragma unroll
        for (int j = i; j > h; --j) {
          const bool up = u[j] > u[j - 1];
          const uint32_t hi = max(u[j], u[j - 1]), lo = min(u[j], u[j - 1]);
          u[j - 1] = hi;
          u[j] = lo;
          const int a = up ? at[j] : at[j - 1], c = up ? at[j - 1] : at[j];
          at[j - 1] = a;
          at[j] = c;
        }
    int my = -1;
    for (int k = 0; k < K; ++k) {
      uint32_t best = u[0];
      int e = at[0];
#pragma unroll
      for (int h = kRun; h < kN; h += kRun) {
        e = u[h] > best ? at[h] : e;
        best = max(best, u[h]);
      }
      const uint32_t top = group_max<kLanes>(best);
      if (kLanes == 32 && top == 0) break;
      const int first = static_cast<int>(group_min<kLanes>(best == top ? static_cast<uint32_t>(e) : ~0u));
      if (lane == k && top != 0) my = first;
#pragma unroll
      for (int h = 0; h < kN; h += kRun)
        if (at[h] == first) {   // an expert is one lane's
#pragma unroll
          for (int j = h; j + 1 < h + kRun; ++j) {
            u[j] = u[j + 1];
            at[j] = at[j + 1];
          }
          u[h + kRun - 1] = 0;
        }
    }
    const bool ok = my >= 0;
    const float w = weight_of<kLanes>(ok ? load_logit(logits, t * ld + my, dtype) : 0.0f, ok, sigmoid,
                                      renormalize, m, sum);
    if (lane < K && live) {
      ids[t * K + lane] = my;
      weights[t * K + lane] = ok ? factor * w : 0.0f;
    }
  }
}

// dl over the whole row is written first: what every expert has (softmax over E),
// or zero; then lane k writes pair k's expert, the warp's stores being ordered by
// __syncwarp.
template <int kLanes, int kN>
__global__ void __launch_bounds__(kThreads) route_topk_backward_kernel(
    const float* __restrict__ dweights, const void* __restrict__ logits, int64_t ld, int dtype,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ d_n_valid, int64_t T, int E, int K,
    bool sigmoid, bool renormalize, float factor, void* dlogits, int64_t ld_d) {
  constexpr int kRows = kThreads / kLanes;
  const int lane = threadIdx.x % kLanes;
  const int64_t nv = valid_rows(d_n_valid, T);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / 32 * (32 / kLanes); t0 < nv;
       t0 += step) {
    const int64_t row = t0 + threadIdx.x % 32 / kLanes;
    const bool live = row < nv;
    const int64_t t = live ? row : nv - 1;
    const int my = lane < K ? ids[t * K + lane] : -1;
    const bool ok = my >= 0 && my < E;
    const float g = ok ? factor * dweights[t * K + lane] : 0.0f;
    const float lk = ok ? load_logit(logits, t * ld + my, dtype) : 0.0f;
    bool again = false;   // an expert comes more than once: each of its pairs adds
    for (int i = 1; i < K; ++i) {
      const int other = __shfl_down_sync(kAll, my, i, kLanes);
      again = again || (ok && lane + i < K && other == my);
    }
    again = __any_sync(kAll, again);
    float l[kN], d;   // d: of pair k's logit
    if (!sigmoid && !renormalize) {
      load_part<kLanes, kN>(logits, t * ld, lane, E, dtype, l);
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kN; ++j) m = fmaxf(m, l[j]);
      m = group_max<kLanes>(m);
      const bool any = m > -INFINITY;   // else a row without experts: its gradient is 0
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        l[j] = any || l[j] != l[j] ? expf(l[j] - m) : 0.0f;
        if (j * kLanes + lane < E) sum += l[j];
      }
      sum = group_sum<kLanes>(sum);
      const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
      const float pk = ok ? expf(lk - m) * inv : 0.0f;
      const float mean = group_sum<kLanes>(g * pk), scale = -(inv * mean);
      const bool tiny = fabsf(scale) < 0x1p-100f;   // inv mean may be a subnormal where p mean is none
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = tiny ? -(l[j] * inv) * mean : l[j] * scale;
      float ge = g;
      if (again) {
        ge = 0.0f;
        for (int k = 0; k < K; ++k) {
          const int id = __shfl_sync(kAll, my, k, kLanes);
          const float gk = __shfl_sync(kAll, g, k, kLanes);
          if (id == my) ge += gk;
        }
      }
      d = pk * (ge - mean);
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) l[j] = 0.0f;
      if (renormalize) {
        const float r = weight_of<kLanes>(lk, ok, sigmoid, true, 0.0f, 1.0f);
        const float mean = group_sum<kLanes>(ok ? g * r : 0.0f);
        d = r * (g - mean);
        if (sigmoid) d *= sigmoid_shifted(-lk, 0.0f);   // 1 - s
      } else {
        d = g * sigmoid_shifted(lk, 0.0f) * sigmoid_shifted(-lk, 0.0f);
      }
      if (again) {
        float all = 0.0f;
        for (int k = 0; k < K; ++k) {
          const int id = __shfl_sync(kAll, my, k, kLanes);
          const float dk = __shfl_sync(kAll, d, k, kLanes);
          if (id == my) all += dk;
        }
        d = all;
      }
    }
    if (live) store_part<kLanes, kN>(dlogits, t * ld_d, lane, E, dtype, l);
    __syncwarp();
    if (ok && live) store_logit(dlogits, t * ld_d + my, dtype, d);
    __syncwarp();
  }
}

unsigned grid_for(int64_t rows, int lanes) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * (2048 / kThreads) * 2;
  const int64_t need = (rows * lanes + kThreads - 1) / kThreads;
  return static_cast<unsigned>(need < most ? need : most);
}

}  // namespace
}  // namespace moe

// 32 lanes a row
#define MOE_WIDE(E, LAUNCH)            \
  do {                                 \
    const int n_ = (E + 31) / 32;      \
    if (n_ <= 2) LAUNCH(32, 2);        \
    else if (n_ <= 3) LAUNCH(32, 3);   \
    else if (n_ <= 4) LAUNCH(32, 4);   \
    else if (n_ <= 5) LAUNCH(32, 5);   \
    else if (n_ <= 6) LAUNCH(32, 6);   \
    else if (n_ <= 8) LAUNCH(32, 8);   \
    else if (n_ <= 12) LAUNCH(32, 12); \
    else if (n_ <= 16) LAUNCH(32, 16); \
    else if (n_ <= 24) LAUNCH(32, 24); \
    else LAUNCH(32, 32);               \
  } while (0)
// 8 lanes a row, for E <= 64
#define MOE_NARROW(E, LAUNCH)       \
  do {                              \
    const int n_ = (E + 7) / 8;     \
    if (n_ <= 1) LAUNCH(8, 1);      \
    else if (n_ <= 2) LAUNCH(8, 2); \
    else if (n_ <= 4) LAUNCH(8, 4); \
    else if (n_ <= 6) LAUNCH(8, 6); \
    else LAUNCH(8, 8);              \
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
#define LAUNCH(lanes, n)                                                                       \
  moe::route_topk_kernel<lanes, n><<<moe::grid_for(T, lanes), moe::kThreads, 0,                \
                                     reinterpret_cast<cudaStream_t>(stream)>>>(                \
      logits, ld, dtype, bias, d_n_valid, T, E, K, score == MOE_SCORE_SIGMOID, renormalize != 0, \
      factor, topk_ids, topk_w)
  // 8 lanes a row save instructions, a warp time where all rows run at once (8
  // and 32 lanes, K = 8: 1024 x 64 3.5 and 2.7 us, 4096 x 32 3.3 and 3.5, 4096 x 64
  // 3.9 and 3.6, 16384 x 64 5.6 and 8.3, 4096 x 96 4.4 and 3.7, 8192 x 96 5.0 and 5.7,
  // 16384 x 160 10.1 and 10.9, 32768 x 128 14.8 and 16.4, x 192 20.7 and 21.4).
  const int64_t enough = (E <= 64 ? 24 : 48) * static_cast<int64_t>(moe::device_sm_count());
  if (K > 8 || E > 192 || T < enough)
    MOE_WIDE(E, LAUNCH);
  else if (E <= 64)
    MOE_NARROW(E, LAUNCH);
  else if (E <= 96)
    LAUNCH(8, 12);
  else if (E <= 128)
    LAUNCH(8, 16);
  else if (E <= 160)
    LAUNCH(8, 20);
  else
    LAUNCH(8, 24);
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
#define LAUNCH(lanes, n)                                                                          \
  moe::route_topk_backward_kernel<lanes, n><<<moe::grid_for(T, lanes), moe::kThreads, 0,          \
                                              reinterpret_cast<cudaStream_t>(stream)>>>(          \
      dtopk_w, logits, ld, dtype, topk_ids, d_n_valid, T, E, K, score == MOE_SCORE_SIGMOID,       \
      renormalize != 0, factor, dlogits, ld_d)
  // as above (8 and 32 lanes, K = 8: 1024 x 64 3.1 and 3.0 us, 4096 x 64 3.3 and 3.5,
  // 2048 x 128 3.7 and 3.1, 4096 x 128 4.0 and 3.7, 8192 x 128 4.6 and 5.4, 32768 x 160
  // 10.5 and 15.0, but 8192 x 256 6.4 and 6.4)
  const int64_t enough = (E <= 64 ? 16 : 32) * static_cast<int64_t>(moe::device_sm_count());
  if (K > 8 || E > 192 || T < enough)
    MOE_WIDE(E, LAUNCH);
  else if (E <= 64)
    MOE_NARROW(E, LAUNCH);
  else if (E <= 96)
    LAUNCH(8, 12);
  else if (E <= 128)
    LAUNCH(8, 16);
  else if (E <= 160)
    LAUNCH(8, 20);
  else
    LAUNCH(8, 24);
#undef LAUNCH
  return moe::check_launch("route_topk_backward_kernel");
}

// moe_adamw_step: one AdamW step over many tensors in one launch (a launch
// per 400 of them), with the two moments held in fp32 or in 8 bits.
//   g' = scale g
//   m = b1 m + (1 - b1) g',   v = b2 v + (1 - b2) g'^2,   r = sqrt(v)
//   p = p (1 - lr wd) - (m lr / (1 - b1^t)) / (r / sqrt(1 - b2^t) + eps)
// Every operation is rounded on its own (no contraction into fused
// multiply-adds), so a step gives the same bits as the formula written with
// elementwise fp32 tensor operations, whatever the tensors' split over
// launches, blocks or lanes (8-bit codes: to nearest or at random, see below).
//
// 8-bit states: m and r = sqrt(v), not v, are stored as e4m3 codes with an
// fp32 scale per 128 values (amax / 448). r has half of v's range in powers
// of two, so within a block it keeps what is down to 2^-18 of the largest (v:
// 2^-36); an r > 0 that would round to zero is stored as the smallest code
// instead, because a second moment lost to zero would divide its first moment
// by eps alone. A block whose largest value is below 1e-30 is stored as
// zeros (its scale's inverse would overflow). The step itself uses the new m
// and v before they are rounded.
//
// How codes are rounded. A step moves r by about 0.7 w of itself, w = (1 - b2) /
// (1 - b2^t) being the newest gradient's share of the average, and where the
// gradients get small by w / 2; a code's half step is 3 to 6 %. Where w is small,
// rounding to nearest puts nearly every code back where it was, and r stays at
// its old size for ever: with b2 = 0.98 to 0.999 and gradients that fall to 1 %
// in half of every block, r was 6 to 130 times too large after 4000 steps. So
// below w = 1/24 the codes of m and r are rounded up or down at random, with the
// chances that make the mean exact. A step's rounding then has a variance of at
// most w times a code's step of 9 %, forgotten over 1 / w steps: r follows its
// average with a deviation of 14 to 17 % (b2 = 0.98 to 0.999), a step's norm within
// 3 %. The bits come from the step's number and the value's place (tensor in the
// list, index), so a step gives the same codes every time. From w = 1/24 on (every
// step with b2 <= 0.958, the first 24 with any b2) the average moves by code steps;
// rounding to nearest has the smaller error there (8 % at b2 = 0.95, at random 12 %
// at 0.96) and takes 439 instead of 480 us (134 M values). One thing it would still
// hold: m's codes below 2^-6 are whole multiples of the least, and 0.9 of one rounds
// back to itself up to four, so a value whose gradients have ended would be moved
// on by 0.15 lr at every step, for ever. At a step whose gradient is zero those
// codes become zero (4 % of the time: 420 us without).
//
// Bytes a value: 8 (p) + 2|4 (g) + 16 (fp32 m, v) or 4 + 16/128 (8 bits) + 2
// (copy): bound by HBM with 32-bit states (577 us for 134 M values, fp32
// gradients, bf16 copies: 6.97 TB/s). With 8-bit states the time hardly depends
// on the gradients' bytes (439 us in fp32, 428 in bf16: 5.5 and 5.1 TB/s): there
// the instructions of the exactly rounded root, quotient and codes set it (82 %
// of the issue slots), and many small blocks keep them flowing (128 threads, 1024
// values, 14 blocks an SM; when they took 420 us, 256 threads, 4096 values and
// five blocks took 549). A warp takes 128 consecutive values, 4 per lane (16 bytes of
// each fp32 array), which is also one scale block, so its largest magnitudes are
// two warp reductions. The tensors' table is a kernel parameter: nothing is
// copied to the device before the launch. Types are asked at every access:
// kernels compiled for one set of types took 418 us then.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>

#include "common.cuh"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kThreads = 128;
constexpr int kBlocksPerSm = 14;            // 32 registers a thread
constexpr int kBlock = 128;                 // values that share a scale = values of a warp
constexpr int kChunk = 1024;                // values of a block: two scale blocks per warp
constexpr float kTinyAmax = 1e-30f;

struct Tensor {
  void* p;
  const void* g;
  void* copy;
  void* m;
  void* v;
  float* ms;
  float* vs;
  int64_t n;
  int32_t chunk_end;   // chunks of this and the earlier tensors of the launch
  uint8_t p_type, g_type, copy_type, vec;
};

template <int Max>
struct Table {
  Tensor t[Max];
  int count;
};

struct Hyper {
  float b1, c1, b2, c2;   // c = 1 - b
  float decay;            // 1 - lr wd
  float step_size;        // lr / (1 - b1^t)
  float root;             // 1 / sqrt(1 - b2^t)
  float eps;
  const float* scale;
  uint32_t step;          // random rounding: what its bits come from, besides a value's place
  uint32_t first;         // non-empty tensors of earlier launches
};

MOE_DEV float load16(uint16_t b, int type) {
  return type == MOE_F16 ? __half2float(__ushort_as_half(b)) : __bfloat162float(__ushort_as_bfloat16(b));
}
MOE_DEV uint16_t store16(float f, int type) {
  return type == MOE_F16 ? __half_as_ushort(__float2half_rn(f)) : __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

// Four values from index i (of n) of an array of the given type; `vec`: all
// four exist and the address is aligned to them.
MOE_DEV void load4(const void* a, int type, int64_t i, int64_t n, bool vec, float (&f)[4]) {
  if (type == MOE_F32) {
    const float* s = static_cast<const float*>(a) + i;
    if (vec) {
      const float4 t = *reinterpret_cast<const float4*>(s);
      f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = i + j < n ? s[j] : 0.0f;
    }
  } else {
    const uint16_t* s = static_cast<const uint16_t*>(a) + i;
    if (vec) {
      const ushort4 t = *reinterpret_cast<const ushort4*>(s);
      f[0] = load16(t.x, type); f[1] = load16(t.y, type);
      f[2] = load16(t.z, type); f[3] = load16(t.w, type);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = i + j < n ? load16(s[j], type) : 0.0f;
    }
  }
}

MOE_DEV void store4(void* a, int type, int64_t i, int64_t n, bool vec, const float (&f)[4]) {
  if (type == MOE_F32) {
    float* s = static_cast<float*>(a) + i;
    if (vec) {
      *reinterpret_cast<float4*>(s) = make_float4(f[0], f[1], f[2], f[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) s[j] = f[j];
    }
  } else {
    uint16_t* s = static_cast<uint16_t*>(a) + i;
    if (vec) {
      *reinterpret_cast<ushort4*>(s) = make_ushort4(store16(f[0], type), store16(f[1], type),
                                                    store16(f[2], type), store16(f[3], type));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < n) s[j] = store16(f[j], type);
    }
  }
}

// Four e4m3 codes (low byte first) as fp32, exactly: through fp16, which holds
// every e4m3 value.
MOE_DEV void decode4(uint32_t codes, float (&f)[4]) {
  uint32_t lo, hi;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(static_cast<uint16_t>(codes)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(static_cast<uint16_t>(codes >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}
MOE_DEV uint32_t encode4(const float (&f)[4]) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(f[1]), "f"(f[0]));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(f[3]), "f"(f[2]));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Four codes from index i (of n); those past n are zero.
MOE_DEV uint32_t load_codes(const void* a, int64_t i, int64_t n, bool vec) {
  const uint8_t* s = static_cast<const uint8_t*>(a) + i;
  if (vec) return *reinterpret_cast<const uint32_t*>(s);
  uint32_t c = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (i + j < n) c |= static_cast<uint32_t>(s[j]) << (8 * j);
  return c;
}

// 64 bits from a counter (x, y) and a key, seven rounds of the 2x32 multiply
// and exclusive-or generator of Salmon, Moraes, Dror and Shaw (2011).
MOE_DEV uint2 random_bits(uint32_t x, uint32_t y, uint32_t key) {
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    const uint64_t w = static_cast<uint64_t>(x) * 0xD256D193u;
    x = static_cast<uint32_t>(w >> 32) ^ key ^ y;
    y = static_cast<uint32_t>(w);
    key += 0x9E3779B9u;
  }
  return make_uint2(x, y);
}

// q rounded to one of its two neighbours among the codes' values, up where the
// 20 random bits exceed what is missing: added to the 20 bits of fp32's mantissa
// that a code does not have, they carry with that chance. Codes below 2^-6 are 2^-9
// apart, as those of [2^-6, 2^-5) are, so these are rounded there. From 448 on (and
// NaN) the conversion saturates.
MOE_DEV float round_random(float q, uint32_t bits) {
  const float a = fabsf(q);
  const float off = a < 0x1p-6f ? 0x1p-6f : 0.0f;
  const uint32_t up = (__float_as_uint(__fadd_rn(a, off)) + bits) & 0xFFF00000u;
  return a < 448.0f ? copysignf(__fsub_rn(__uint_as_float(up), off), q) : q;
}

// The block's values as codes (Floor: a positive value never becomes zero;
// Random: rounded at random with `bits`, else to nearest), given the block's
// largest magnitude; returns the block's scale.
template <bool Floor, bool Random>
MOE_DEV float store_codes(void* a, int64_t i, int64_t n, bool vec, const float (&f)[4], float amax,
                          uint2 bits) {
  const bool live = amax >= kTinyAmax;
  const float inv = live ? __fmul_rn(__frcp_rn(amax), 448.0f) : 0.0f;
  const float least = live ? 0x1p-9f : 0.0f;   // the smallest positive code
  float q[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q[j] = __fmul_rn(f[j], inv);
    if (Random) {
      const uint32_t w = j < 2 ? bits.x : bits.y;   // a value's high bits are nobody else's
      q[j] = round_random(q[j], j % 2 ? w >> 12 : w & 0xFFFFFu);
    }
    if (Floor && f[j] > 0.0f && q[j] < least) q[j] = least;
  }
  const uint32_t c = encode4(q);
  uint8_t* s = static_cast<uint8_t*>(a) + i;
  if (vec) {
    *reinterpret_cast<uint32_t*>(s) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j < n) s[j] = static_cast<uint8_t>(c >> (8 * j));
  }
  return live ? __fmul_rn(amax, 1.0f / 448.0f) : 0.0f;
}

MOE_DEV float largest4(const float (&f)[4]) {
  return fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
}

template <int Bits, bool Random, int Max>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) adamw_kernel(const __grid_constant__ Table<Max> tab,
                                                         const Hyper h) {
  const int chunk = blockIdx.x;
  int lo = 0, hi = tab.count - 1;   // first tensor whose chunk_end is past this chunk
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (tab.t[mid].chunk_end > chunk) hi = mid; else lo = mid + 1;
  }
  const Tensor& t = tab.t[lo];
  const int first = lo > 0 ? tab.t[lo - 1].chunk_end : 0;
  const int64_t n = t.n;
  const int64_t base = static_cast<int64_t>(chunk - first) * kChunk;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float scale = h.scale != nullptr ? *h.scale : 1.0f;
  const int p_type = t.p_type, g_type = t.g_type, copy_type = t.copy_type;
  const bool has_copy = t.copy != nullptr;
  constexpr int kIter = kChunk / kBlock / (kThreads / 32);
  struct In {
    float p[4], g[4];
    float m[4], v[4];       // 32-bit states
    uint32_t mc, vc;        // 8-bit states
    float ms, vs;
  };
  auto block_at = [&](int it) { return base + (it * (kThreads / 32) + warp) * kBlock; };
  auto load = [&](int64_t b, In& x) {
    const int64_t i = b + lane * 4;
    const bool vec = t.vec && i + 4 <= n;
    load4(t.g, g_type, i, n, vec, x.g);
    load4(t.p, p_type, i, n, vec, x.p);
    if (Bits == 32) {
      load4(t.m, MOE_F32, i, n, vec, x.m);
      load4(t.v, MOE_F32, i, n, vec, x.v);
    } else {
      x.mc = load_codes(t.m, i, n, vec);
      x.vc = load_codes(t.v, i, n, vec);
      x.ms = t.ms[b / kBlock];
      x.vs = t.vs[b / kBlock];
    }
  };
  auto step = [&](int64_t b, In& x) {
    const int64_t i = b + lane * 4;
    const bool vec = t.vec && i + 4 <= n;
    float (&p)[4] = x.p, (&g)[4] = x.g, (&m)[4] = x.m, (&v)[4] = x.v;
    float r[4];
    if (Bits == 8) {
      decode4(x.mc, m);
      decode4(x.vc, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = __fmul_rn(m[j], x.ms);
        v[j] = __fmul_rn(v[j], x.vs);
        v[j] = __fmul_rn(v[j], v[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (h.scale != nullptr) g[j] = __fmul_rn(g[j], scale);
      const bool ended = Bits == 8 && !Random && g[j] == 0.0f && fabsf(m[j]) < 0x1p-6f * x.ms;
      m[j] = __fadd_rn(__fmul_rn(m[j], h.b1), __fmul_rn(g[j], h.c1));
      v[j] = __fadd_rn(__fmul_rn(v[j], h.b2), __fmul_rn(__fmul_rn(g[j], g[j]), h.c2));
      r[j] = __fsqrt_rn(v[j]);
      const float d = __fadd_rn(__fmul_rn(r[j], h.root), h.eps);
      p[j] = __fsub_rn(__fmul_rn(p[j], h.decay), __fdiv_rn(__fmul_rn(m[j], h.step_size), d));
      if (ended) m[j] = 0.0f;
    }
    store4(t.p, p_type, i, n, vec, p);
    if (has_copy) store4(t.copy, copy_type, i, n, vec, p);
    if (Bits == 32) {
      store4(t.m, MOE_F32, i, n, vec, m);
      store4(t.v, MOE_F32, i, n, vec, v);
    } else {
      // values past n are zero and change no maximum
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j >= n) m[j] = r[j] = 0.0f;
      // The block's largest |m| and r: fp32 magnitudes compare as integers do.
      const uint32_t am = __reduce_max_sync(0xffffffffu, __float_as_uint(largest4(m)));
      const uint32_t ar = __reduce_max_sync(0xffffffffu, __float_as_uint(largest4(r)));
      // m and r share their bits: rounded the same way, their quotient moves least
      uint2 bits = make_uint2(0, 0);
      if (Random) {
        const uint64_t at = static_cast<uint64_t>(i) >> 2;
        bits = random_bits(static_cast<uint32_t>(at),
                           (h.first + lo) ^ (static_cast<uint32_t>(at >> 32) << 24), h.step);
      }
      const float ms = store_codes<false, Random>(t.m, i, n, vec, m, __uint_as_float(am), bits);
      const float vs = store_codes<true, Random>(t.v, i, n, vec, r, __uint_as_float(ar), bits);
      if (lane == 0) {
        t.ms[b / kBlock] = ms;
        t.vs[b / kBlock] = vs;
      }
    }
  };
#pragma unroll 1
  for (int it = 0; it < kIter; ++it) {
    const int64_t b = block_at(it);
    if (b >= n) break;   // the whole warp
    In x;
    load(b, x);
    step(b, x);
  }
}

// A launch's parameters may take 32,764 bytes: 400 tensors of 72 bytes. A
// table of 16 keeps the launch of a few tensors small (a call for one tensor
// takes 8.4 us with it, 9.8 to 12 with the large one).
constexpr int kMaxTensors = 400;
constexpr int kFewTensors = 16;

template <int Bits, bool Random, int Max>
int launch(const Table<kMaxTensors>& all, int chunks, const Hyper& h, cudaStream_t s) {
  if constexpr (Max == kMaxTensors) {
    adamw_kernel<Bits, Random, Max><<<chunks, kThreads, 0, s>>>(all, h);
  } else {
    Table<Max> few;
    for (int i = 0; i < all.count; ++i) few.t[i] = all.t[i];
    few.count = all.count;
    adamw_kernel<Bits, Random, Max><<<chunks, kThreads, 0, s>>>(few, h);
  }
  return check_launch("adamw_kernel");
}

template <int Bits, bool Random>
int launch_of(const Table<kMaxTensors>& tab, int chunks, const Hyper& h, cudaStream_t s) {
  return tab.count <= kFewTensors ? launch<Bits, Random, kFewTensors>(tab, chunks, h, s)
                                  : launch<Bits, Random, kMaxTensors>(tab, chunks, h, s);
}

int launch_all(const Table<kMaxTensors>& tab, int bits, bool random, int chunks, const Hyper& h,
               cudaStream_t s) {
  if (bits == 32) return launch_of<32, false>(tab, chunks, h, s);
  return random ? launch_of<8, true>(tab, chunks, h, s) : launch_of<8, false>(tab, chunks, h, s);
}

}  // namespace
}  // namespace moe

extern "C" int moe_adamw_step(const moe_adamw_tensor* tensors, int count, int state_bits, double lr,
                              double beta1, double beta2, double eps, double weight_decay,
                              int64_t step, const float* d_grad_scale, moe_stream_t stream) {
  MOE_REQUIRE(count >= 0 && (count == 0 || tensors), "moe_adamw_step: null tensor list");
  MOE_REQUIRE(state_bits == 32 || state_bits == 8, "moe_adamw_step: state_bits must be 32 or 8");
  MOE_REQUIRE(step >= 1, "moe_adamw_step: step counts from 1");
  MOE_REQUIRE(std::isfinite(lr) && beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 &&
                  eps >= 0.0 && std::isfinite(eps) && std::isfinite(weight_decay),
              "moe_adamw_step: betas must be in [0, 1), eps >= 0, lr and weight_decay finite");
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& a = tensors[i];
    MOE_REQUIRE(a.n >= 0, "moe_adamw_step: tensor %d: negative size", i);
    MOE_REQUIRE((a.n + moe::kChunk - 1) / moe::kChunk <= INT32_MAX,
                "moe_adamw_step: tensor %d is too large", i);
    if (a.n == 0) continue;
    MOE_REQUIRE(a.p && a.g && a.m && a.v && (state_bits == 32 || (a.m_scale && a.v_scale)),
                "moe_adamw_step: tensor %d: null pointer", i);
    MOE_REQUIRE(a.p_type >= MOE_BF16 && a.p_type <= MOE_F32 && a.g_type >= MOE_BF16 &&
                    a.g_type <= MOE_F32 && (!a.copy || (a.copy_type >= MOE_BF16 && a.copy_type <= MOE_F32)),
                "moe_adamw_step: tensor %d: bad type", i);
    MOE_REQUIRE(moe::aligned(a.p, a.p_type == MOE_F32 ? 4 : 2) &&
                    moe::aligned(a.g, a.g_type == MOE_F32 ? 4 : 2) &&
                    moe::aligned(a.copy, a.copy_type == MOE_F32 ? 4 : 2) &&
                    (state_bits == 8 || (moe::aligned(a.m, 4) && moe::aligned(a.v, 4))) &&
                    moe::aligned(a.m_scale, 4) && moe::aligned(a.v_scale, 4),
                "moe_adamw_step: tensor %d: pointer not aligned to its type", i);
  }
  MOE_REQUIRE_DEVICE();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // lr and the step's bias corrections are values of the launch, so a graph
  // would apply this one step's again at every replay
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) {
    const int rc = moe::check_launch("cudaStreamIsCapturing");
    return rc != MOE_OK ? rc : MOE_ERR_CUDA;
  }
  MOE_REQUIRE(capture == cudaStreamCaptureStatusNone,
              "moe_adamw_step: the stream is capturing a graph, whose replays would repeat this step's "
              "bias correction and lr");
  const double t = static_cast<double>(step);
  moe::Hyper h;
  h.b1 = static_cast<float>(beta1);
  h.c1 = static_cast<float>(1.0 - beta1);
  h.b2 = static_cast<float>(beta2);
  h.c2 = static_cast<float>(1.0 - beta2);
  h.decay = static_cast<float>(1.0 - lr * weight_decay);
  h.step_size = static_cast<float>(lr / (1.0 - std::pow(beta1, t)));
  h.root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(beta2, t)));
  h.eps = static_cast<float>(eps);
  h.scale = d_grad_scale;
  h.step = static_cast<uint32_t>(step);
  h.first = 0;
  const double newest = (1.0 - beta2) / (1.0 - std::pow(beta2, t));   // its share of the average
  const bool random = newest < 1.0 / 24.0;
  moe::Table<moe::kMaxTensors> tab;
  int64_t chunks = 0;
  tab.count = 0;
  const bool eight = state_bits == 8;
  for (int i = 0; i < count; ++i) {
    const moe_adamw_tensor& a = tensors[i];
    if (a.n == 0) continue;
    const int64_t mine = (a.n + moe::kChunk - 1) / moe::kChunk;
    if (tab.count == moe::kMaxTensors || chunks + mine > INT32_MAX) {
      const int rc = moe::launch_all(tab, state_bits, random, static_cast<int>(chunks), h, s);
      if (rc != MOE_OK) return rc;
      h.first += static_cast<uint32_t>(tab.count);
      tab.count = 0;
      chunks = 0;
    }
    chunks += mine;
    moe::Tensor& d = tab.t[tab.count++];
    d.p = a.p;
    d.g = a.g;
    d.copy = a.copy;
    d.m = a.m;
    d.v = a.v;
    d.ms = a.m_scale;
    d.vs = a.v_scale;
    d.n = a.n;
    d.chunk_end = static_cast<int32_t>(chunks);
    d.p_type = static_cast<uint8_t>(a.p_type);
    d.g_type = static_cast<uint8_t>(a.g_type);
    d.copy_type = static_cast<uint8_t>(a.copy_type);
    d.vec = moe::aligned(a.p, a.p_type == MOE_F32 ? 16 : 8) &&
            moe::aligned(a.g, a.g_type == MOE_F32 ? 16 : 8) &&
            moe::aligned(a.copy, a.copy_type == MOE_F32 ? 16 : 8) &&
            moe::aligned(a.m, eight ? 4 : 16) && moe::aligned(a.v, eight ? 4 : 16);
  }
  return tab.count > 0 ? moe::launch_all(tab, state_bits, random, static_cast<int>(chunks), h, s) : MOE_OK;
}

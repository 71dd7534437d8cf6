// moe_grouped_mm_w4: the experts' product over 4-bit weights with group scales,
//   out[r, n] = sum_k x[r, k] s[e, n, k / g] (q[e, n, k] - z[e, n, k / g]),
// for batches of single tokens, where the time is that of reading the weights.
//
// D = W X^T on mma.sync (m16n8k16): the weights are the first operand, so that
// they go from memory to registers and, as integers, into the tensor core with
// no stop in shared memory; 8 rows of x are the second operand's columns. Which
// of 128 contracted values stands at which place of the eight instructions is
// free as long as both operands agree, and is chosen so that a lane reads 16
// contiguous bytes of codes per weight row and the 8 values of x that go with
// each word of them. q - z is exact in 16 bits (q is put into the mantissa of
// 128 or 1024, and 128 + z or 1024 + z taken off); a group's sum is exact
// products in fp32, and the scale multiplies that sum in fp32, so nothing is
// rounded but the sums and, once, the result.
//
// A block does 64 weight rows by up to 32 rows of one expert; its warps share
// the weight rows (two) and the contraction (four), whose sums meet in shared
// memory in a fixed order.
#include <algorithm>

#include "dtype16.cuh"
#include "gemm_host.h"
#include "host_util.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxE = 1024;
constexpr int kRows = 32;      // rows of x of a block
constexpr int kTile = 64;      // weight rows of a block
constexpr int kSplit = 4;      // warps along the contraction
constexpr int kMT = 2;         // 16-row tiles of a warp
constexpr int kBlock = 128;    // contracted per step of a warp

struct W4Params {
  const int32_t* start;
  const int32_t* psum;
  const uint16_t* x;
  int64_t ld_x;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  int E, N, Kd, groups;   // groups along Kd
  int64_t M_cap;
  uint16_t* out;
  int64_t ld_out;
  int32_t* status;
};

template <bool Half>
MOE_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (Half)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Nibbles i and i + 4 of a word, less the zero point (already with the offset,
// twice): two 16-bit values.
template <bool Half, int i>
MOE_DEV uint32_t code_pair(uint32_t word, uint32_t off) {
  const uint32_t v = ((word >> (4 * i)) & 0x000f000fu) | (Half ? 0x64006400u : 0x43004300u);
  if constexpr (Half) {
    const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&v), *reinterpret_cast<const __half2*>(&off));
    return *reinterpret_cast<const uint32_t*>(&d);
  } else {
    const __nv_bfloat162 d =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), *reinterpret_cast<const __nv_bfloat162*>(&off));
    return *reinterpret_cast<const uint32_t*>(&d);
  }
}

template <bool Half>
MOE_DEV float to_f32(uint16_t v) {
  return unpack2<Half>(v).x;
}

// The contraction of one warp: its share of the steps, kMT x kNT tiles of sums.
// kGroup values share a scale. Word c of a lane (t = lane % 4) stands for the 8
// contracted values from offset(c) of a step on.
template <bool Half, int kGroup, int kNT>
MOE_DEV void contract(const W4Params& p, int e, int n0, int64_t row0, int rows, int split,
                      float (&acc)[kMT][kNT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  constexpr int kWide = kGroup / 32;   // words a lane reads at once: 4, 2 or 1
  const int64_t row_bytes = p.Kd / 2;
  const uint8_t* w[kMT][2];
  int64_t sc[kMT][2];
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int n = min(n0 + m * 16 + h * 8 + g, p.N - 1);   // past the last: not stored
      const int64_t row = static_cast<int64_t>(e) * p.N + n;
      w[m][h] = p.codes + row * row_bytes;
      sc[m][h] = row * p.groups;
    }
  const uint16_t* x[kNT];
#pragma unroll
  for (int j = 0; j < kNT; ++j) x[j] = p.x + (row0 + min(j * 8 + g, rows - 1)) * p.ld_x;
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][j][i] = 0.0f;

  const int steps = (p.Kd + kBlock - 1) / kBlock;
  for (int b = split; b < steps; b += kSplit) {
    const int k0 = b * kBlock;
    uint32_t word[kMT][2][4];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 4; c += kWide) {
          const int k = k0 + (c / kWide) * kGroup + t * (8 * kWide);
          uint32_t* to = &word[m][h][c];
          const uint8_t* from = w[m][h] + k / 2;
          if constexpr (kWide == 4) {
            const uint4 v = k < p.Kd ? __ldcs(reinterpret_cast<const uint4*>(from)) : make_uint4(0, 0, 0, 0);
            to[0] = v.x, to[1] = v.y, to[2] = v.z, to[3] = v.w;
          } else if constexpr (kWide == 2) {
            const uint2 v = k < p.Kd ? __ldg(reinterpret_cast<const uint2*>(from)) : make_uint2(0, 0);
            to[0] = v.x, to[1] = v.y;
          } else {
            to[0] = k < p.Kd ? __ldg(reinterpret_cast<const uint32_t*>(from)) : 0u;
          }
        }
#pragma unroll
    for (int q = 0; q < kBlock / kGroup; ++q) {
      const int gi = k0 / kGroup + q;
      const bool in = gi < p.groups;
      float s[kMT][2];
      uint32_t off[kMT][2];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s[m][h] = in ? to_f32<Half>(__ldg(p.scales + sc[m][h] + gi)) : 0.0f;
          const uint32_t z = p.zeros == nullptr ? 8u : (in ? __ldg(p.zeros + sc[m][h] + gi) & 15u : 0u);
          off[m][h] = (Half ? 0x64006400u : 0x43004300u) | (z * 0x00010001u);
        }
      float part[kMT][kNT][4];
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) part[m][j][i] = 0.0f;
#pragma unroll
      for (int cc = 0; cc < kWide; ++cc) {
        const int c = q * kWide + cc;
        const int k = k0 + q * kGroup + t * (8 * kWide) + cc * 8;
        uint4 xv[kNT];
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          xv[j] = k < p.Kd && j * 8 + g < rows ? __ldg(reinterpret_cast<const uint4*>(x[j] + k))
                                               : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a[kMT][4];
#pragma unroll
          for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              a[m][h] = half == 0 ? code_pair<Half, 0>(word[m][h][c], off[m][h])
                                  : code_pair<Half, 2>(word[m][h][c], off[m][h]);
              a[m][2 + h] = half == 0 ? code_pair<Half, 1>(word[m][h][c], off[m][h])
                                      : code_pair<Half, 3>(word[m][h][c], off[m][h]);
            }
#pragma unroll
          for (int j = 0; j < kNT; ++j) {
            // (x[i], x[i + 4]) for i = 2 half, 2 half + 1
            const uint32_t lo = half == 0 ? xv[j].x : xv[j].y, hi = half == 0 ? xv[j].z : xv[j].w;
            const uint32_t b0 = __byte_perm(lo, hi, 0x5410), b1 = __byte_perm(lo, hi, 0x7632);
#pragma unroll
            for (int m = 0; m < kMT; ++m) mma16816<Half>(part[m][j], a[m], b0, b1);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < kMT; ++m)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[m][j][i] = fmaf(s[m][i >> 1], part[m][j][i], acc[m][j][i]);
    }
  }
}

template <bool Half, int kGroup, int kNT>
MOE_DEV void tile(const W4Params& p, int e, int i0, int64_t row0, int rows, float* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int split = warp % kSplit, part = warp / kSplit;
  float acc[kMT][kNT][4];
  contract<Half, kGroup, kNT>(p, e, i0 + part * kMT * 16, row0, rows, split, acc);
  // sums[split][row][weight row]
#pragma unroll
  for (int m = 0; m < kMT; ++m)
#pragma unroll
    for (int j = 0; j < kNT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sums[(split * kRows + j * 8 + t * 2 + (i & 1)) * kTile + part * kMT * 16 + m * 16 + (i >> 1) * 8 + g] =
            acc[m][j][i];
  __syncthreads();
  for (int v = threadIdx.x; v < rows * (kTile / 8); v += kThreads) {
    const int r = v / (kTile / 8), n = v % (kTile / 8) * 8;
    if (i0 + n >= p.N) continue;
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f[i] = sums[r * kTile + n + i];
#pragma unroll
      for (int s = 1; s < kSplit; ++s) f[i] += sums[(s * kRows + r) * kTile + n + i];
    }
    *reinterpret_cast<uint4*>(p.out + (row0 + r) * p.ld_out + i0 + n) = pack8<Half>(f);
  }
}

template <bool Half, int kGroup>
__global__ void __launch_bounds__(kThreads, 2) grouped_w4_kernel(const W4Params p) {
  __shared__ float s_sums[kSplit * kRows * kTile];
  __shared__ int s_warp_sum[kThreads / 32];
  __shared__ int s_e, s_row, s_rows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ni = (p.N + kTile - 1) / kTile;
  const int chunk = static_cast<int>(blockIdx.x) / ni;
  const int i0 = (static_cast<int>(blockIdx.x) - chunk * ni) * kTile;
  // Which expert has chunk number `chunk`? Thread i counts the chunks of experts
  // per i .. per i + per - 1; segments are clamped into the buffer.
  constexpr int kPer = kMaxE / kThreads;
  const int per = (p.E + kThreads - 1) / kThreads;
  if (threadIdx.x == 0) s_e = -1;
  int a[kPer], n[kPer], mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = threadIdx.x * per + j;
    a[j] = n[j] = 0;
    if (j < per && e < p.E) {
      const int cap = static_cast<int>(p.M_cap);
      a[j] = min(max(p.start[e], 0), cap);
      n[j] = min(max(p.psum[e], a[j]), cap) - a[j];
      mine += (n[j] + kRows - 1) / kRows;
    }
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_warp_sum[warp] = incl;
  __syncthreads();
  int base = incl - mine;
  for (int w = 0; w < warp; ++w) base += s_warp_sum[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = (n[j] + kRows - 1) / kRows;
    if (chunk >= base && chunk < base + c) {
      s_e = threadIdx.x * per + j;
      s_row = a[j] + (chunk - base) * kRows;
      s_rows = min(kRows, n[j] - (chunk - base) * kRows);
    }
    base += c;
  }
  // more chunks than the grid has: the caller's bound on the rows was wrong
  if (blockIdx.x == 0 && threadIdx.x == kThreads - 1 &&
      static_cast<int64_t>(base) * ni > static_cast<int64_t>(gridDim.x))
    set_status(p.status, MOE_ERR_DEVICE_CHECK);
  __syncthreads();
  const int e = s_e, rows = s_rows;
  if (e < 0) return;
  if (rows <= 8)
    tile<Half, kGroup, 1>(p, e, i0, s_row, rows, s_sums);
  else if (rows <= 16)
    tile<Half, kGroup, 2>(p, e, i0, s_row, rows, s_sums);
  else
    tile<Half, kGroup, 4>(p, e, i0, s_row, rows, s_sums);
}

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_mm_w4(const void* x, int64_t ld_x, const uint8_t* codes, const void* scales,
                                 const uint8_t* zeros, int group, const int32_t* start,
                                 const int32_t* psum, int dtype, int E, int N, int Kd, int64_t M_cap,
                                 int64_t max_rows, void* out, int64_t ld_out, int32_t* d_status,
                                 moe_stream_t stream) {
  MOE_REQUIRE(start && psum, "moe_grouped_mm_w4: null segments");
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "moe_grouped_mm_w4: dtype must be MOE_BF16 or MOE_F16");
  MOE_REQUIRE(E > 0 && E <= moe::kMaxE, "moe_grouped_mm_w4: E must be in [1, 1024]");
  MOE_REQUIRE(group == 32 || group == 64 || group == 128, "moe_grouped_mm_w4: group must be 32, 64 or 128");
  MOE_REQUIRE(N > 0 && N % 8 == 0 && Kd > 0 && Kd % group == 0,
              "moe_grouped_mm_w4: N must be a positive multiple of 8, Kd of the group");
  MOE_REQUIRE(M_cap >= 0 && M_cap <= INT32_MAX && max_rows >= 0 && max_rows <= M_cap,
              "moe_grouped_mm_w4: M_cap and max_rows must fit each other and 32 bits");
  MOE_REQUIRE(codes && scales && (M_cap == 0 || (x && out)), "moe_grouped_mm_w4: operands must be non-null");
  MOE_REQUIRE(ld_x >= Kd && ld_out >= N && ld_x % 8 == 0 && ld_out % 8 == 0,
              "moe_grouped_mm_w4: a row stride must be a multiple of 8, at least the row");
  MOE_REQUIRE(moe::aligned(x, 16) && moe::aligned(codes, 16) && moe::aligned(out, 16) &&
                  moe::aligned(scales, 16),
              "moe_grouped_mm_w4: x, codes, scales and out must be 16-byte aligned");
  const int64_t live = std::min<int64_t>(E, max_rows);
  const int64_t tiles = (max_rows / moe::kRows + live) * ((N + moe::kTile - 1) / moe::kTile);
  MOE_REQUIRE(tiles <= INT32_MAX, "moe_grouped_mm_w4: sizes exceed 32-bit tile numbers");
  MOE_REQUIRE_DEVICE();
  if (max_rows == 0) return MOE_OK;
  moe::W4Params p;
  p.start = start;
  p.psum = psum;
  p.x = static_cast<const uint16_t*>(x);
  p.ld_x = ld_x;
  p.codes = codes;
  p.scales = static_cast<const uint16_t*>(scales);
  p.zeros = zeros;
  p.E = E;
  p.N = N;
  p.Kd = Kd;
  p.groups = Kd / group;
  p.M_cap = M_cap;
  p.out = static_cast<uint16_t*>(out);
  p.ld_out = ld_out;
  p.status = d_status;
  const bool half = dtype == MOE_F16;
  auto* kernel = group == 128  ? (half ? moe::grouped_w4_kernel<true, 128> : moe::grouped_w4_kernel<false, 128>)
                 : group == 64 ? (half ? moe::grouped_w4_kernel<true, 64> : moe::grouped_w4_kernel<false, 64>)
                               : (half ? moe::grouped_w4_kernel<true, 32> : moe::grouped_w4_kernel<false, 32>);
  kernel<<<static_cast<unsigned>(tiles), moe::kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return moe::check_launch("grouped_w4_kernel");
}

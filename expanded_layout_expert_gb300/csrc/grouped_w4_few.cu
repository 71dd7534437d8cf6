// The 4-bit product of grouped_w4.cu for chunks of at most 8 rows: an expert's
// few single tokens, or one.
//
// D = W X^T on mma.sync (m16n8k16), the weights as the first operand: from
// memory to a lane's registers through a ring of asynchronous copies, made
// 16-bit values there, and into the tensor core. Which of 128 contracted values
// stands at which place of the eight instructions is free as long as both
// operands agree: a lane (t = lane % 4) takes 8 neighbouring values per word of
// codes, and the 16 bytes of x that go with them. A group's sums are exact
// products in fp32; the scale multiplies that sum in fp32.
//
// mma.sync has a quarter of tcgen05's rate, enough for 8 rows at HBM's. What
// bounds the kernel is no one thing: one token of 8 out of 64 experts of 4096 x 7168 takes
// 27.4 us (4.4 TB/s of codes and scales, whose bytes alone take 17.9), 26.5 with the codes taken
// as they are, 25.8 without reading x, 22.4 without the copies, 14.0 without all three and 7.1
// with one step of the loop: the start (segments found, the first copies
// asked for and come) and the end of a single wave. A block of four warps does 32
// weight rows by one expert's chunk; the warps take every fourth 128 contracted
// values and meet once, at the end, in shared memory in a fixed order. Blocks
// are small so that those of a single token all fit the GPU at once (with six
// to an SM instead of seven 30 us).
#include <algorithm>
#include <atomic>

#include "gemm_host.h"
#include "host_util.h"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 32;        // weight rows
constexpr int kRows = 8;         // of x: the columns of an instruction's second operand
constexpr int kBlock = 128;      // contracted per step of a warp
constexpr int kStages = 3;
constexpr int kSlot = kTile * kBlock / 2;             // bytes of a warp's step
constexpr int kRing = kWarps * kStages * kSlot;

struct FewParams {
  const int32_t* start;
  const int32_t* psum;
  const uint16_t* x;
  int64_t ld_x;
  const uint8_t* codes;
  const uint16_t* scales;
  const uint8_t* zeros;
  int E, N, Kd, groups;   // groups along Kd
  int pitch;              // of a row's scales in shared memory
  int64_t M_cap;
  uint16_t* out;
  int64_t ld_out;
  int32_t* status;
};

// 16 bytes from global to shared memory; none of them read (zeros written) if !in.
MOE_DEV void copy16(uint32_t to, const void* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0)
               : "memory");
}
MOE_DEV void copy8(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
MOE_DEV void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
MOE_DEV void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// D = A B + (kFirst ? 0 : D)
template <bool Half, bool kFirst>
MOE_DEV void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  const float c[4] = {kFirst ? 0.0f : d[0], kFirst ? 0.0f : d[1], kFirst ? 0.0f : d[2], kFirst ? 0.0f : d[3]};
  if constexpr (Half)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
          "f"(c[3]));
}

template <bool Half, int kGroup, bool kZeros>
__global__ void __launch_bounds__(kThreads, 7) grouped_w4_few_kernel(const FewParams p) {
  extern __shared__ __align__(128) uint8_t smem[];   // ring, then the tile's scales and zero points
  __shared__ int s_warp_sum[kWarps], s_found[3];
  constexpr int kWide = kGroup / 32;   // words of a lane that share a group: 4, 2 or 1
  constexpr int kGroups = kBlock / kGroup;
  constexpr bool kRagged = kGroup < kBlock;   // the last step may be short
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ni = (p.N + kTile - 1) / kTile;
  const int chunk = static_cast<int>(blockIdx.x) / ni;
  const int i0 = (static_cast<int>(blockIdx.x) - chunk * ni) * kTile;
  const int all = w4_find_chunk<kThreads, kRows>(p.start, p.psum, p.E, p.M_cap, chunk, s_warp_sum, s_found);
  // more chunks than the grid has: the caller's bound on the rows was wrong
  if (blockIdx.x == 0 && threadIdx.x == kThreads - 1 &&
      static_cast<int64_t>(all) * ni > static_cast<int64_t>(gridDim.x))
    set_status(p.status, MOE_ERR_DEVICE_CHECK);
  const int e = s_found[0], rows = s_found[2];
  const int64_t row0 = s_found[1];
  if (e < 0) return;

  const int steps = (p.Kd + kBlock - 1) / kBlock;
  const int64_t w_row = static_cast<int64_t>(e) * p.N + i0;
  const int n_rows = min(kTile, p.N - i0);
  const uint32_t base = smem_u32(smem);
  uint8_t* s_scales = smem + kRing;
  uint8_t* s_zeros = s_scales + kTile * p.pitch * 2;
  // a lane copies 16 bytes of rows g, g + 8, g + 16 and g + 24 a step; rows past
  // the last are the last once more, and not stored
  const uint32_t place = g * 64 + ((t ^ ((g >> 1) & 3)) << 4);
  const uint32_t ring = base + warp * kStages * kSlot + place;
  const uint8_t* from[4];   // of the next step to be copied
#pragma unroll
  for (int h = 0; h < 4; ++h)
    from[h] = p.codes + (w_row + min(h * 8 + g, n_rows - 1)) * (p.Kd / 2) + warp * (kBlock / 2) + t * 16;
  auto copy_step = [&](int b, int slot) {
    if (b < steps) {
      // what is past the contraction is not read, and zero
      const bool in = !kRagged || b * (kBlock / 2) + t * 16 < p.Kd / 2;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        copy16(ring + slot * kSlot + h * 512, in ? from[h] : p.codes, in);
        from[h] += kWarps * (kBlock / 2);
      }
    }
    copies_commit();
  };
  // The scales and zero points of the tile's rows lie together; where their rows
  // are whole vectors, the copies are kept apart by one, so that the eight rows
  // that are read at a time lie in different banks.
  {
    const uint8_t* scales = reinterpret_cast<const uint8_t*>(p.scales + w_row * p.groups);
    const uint8_t* zeros = p.zeros + w_row * p.groups;
    if (p.pitch != p.groups) {
      const int r = threadIdx.x / 4;   // four lanes a row
      static_assert(kThreads == 4 * kTile, "a row of scales for every four threads");
      if (r < n_rows) {
        for (int i = t * 16; i < p.groups * 2; i += 64)
          copy16(smem_u32(s_scales) + r * p.pitch * 2 + i, scales + r * p.groups * 2 + i, true);
        if (kZeros)
          for (int i = t * 8; i < p.groups; i += 32)
            copy8(smem_u32(s_zeros) + r * p.pitch + i, zeros + r * p.groups + i);
      }
    } else {
      for (int i = threadIdx.x * 16; i < n_rows * p.groups * 2; i += kThreads * 16)
        copy16(smem_u32(s_scales) + i, scales + i, true);
      if (kZeros)
        for (int i = threadIdx.x * 8; i < n_rows * p.groups; i += kThreads * 8)
          copy8(smem_u32(s_zeros) + i, zeros + i);
    }
    copies_commit();
  }
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) copy_step(warp + s * kWarps, s);

  // Columns past the chunk's rows repeat its last row, and are not stored; the
  // steps past the last repeat it, and are not used.
  const uint16_t* x = p.x + (row0 + min(g, rows - 1)) * p.ld_x + t * (8 * kWide);
  auto load_x = [&](int b, int c) {
    const int k = b * kBlock + (c / kWide) * kGroup + (c % kWide) * 8;
    return !kRagged || k + t * (8 * kWide) < p.Kd ? __ldg(reinterpret_cast<const uint4*>(x + k))
                                                  : make_uint4(0, 0, 0, 0);
  };
  uint4 xv[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) xv[c] = load_x(min(warp, steps - 1), c);
  float2 acc[2][2];   // of weight rows g and g + 8, of 16 m + that
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) acc[m][h] = make_float2(0.0f, 0.0f);
  // rows g, g + 8, g + 16 and g + 24 in the scales and zero points
  int at[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) at[h] = min(h * 8 + g, n_rows - 1) * p.pitch;
  copies_wait<kStages - 1>();
  __syncthreads();   // the scales are there

  int slot = 0;
  for (int b = warp; b < steps; b += kWarps) {
    copies_wait<kStages - 2>();
    __syncwarp();   // every lane's copies of this step, and every lane has read the slot that is filled next
    copy_step(b + (kStages - 1) * kWarps, slot == 0 ? kStages - 1 : slot - 1);
    const uint8_t* codes = smem + (warp * kStages + slot) * kSlot + g * 64;
    const int b_next = min(b + kWarps, steps - 1);
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      const bool in = !kRagged || b * kGroups + q < p.groups;   // else products with zeros
      const int gi = in ? b * kGroups + q : 0;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float s[2];
        uint32_t off[2], word[2][kWide];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = at[m * 2 + h] + gi;
          s[h] = in ? unpack2<Half>(reinterpret_cast<const uint16_t*>(s_scales)[r]).x : 0.0f;
          off[h] = w4_offset<Half>(kZeros ? s_zeros[r] & 15u : kW4Zero);
          const uint8_t* c = codes + (m * 2 + h) * 512;
          const int swizzle = (g >> 1) & 3;
          if constexpr (kWide == 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(c + ((t ^ swizzle) << 4));
            word[h][0] = v.x, word[h][1] = v.y, word[h][2] = v.z, word[h][3] = v.w;
          } else if constexpr (kWide == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(c + (((2 * q + (t >> 1)) ^ swizzle) << 4) + (t & 1) * 8);
            word[h][0] = v.x, word[h][1] = v.y;
          } else {
            word[h][0] = *reinterpret_cast<const uint32_t*>(c + ((q ^ swizzle) << 4) + t * 4);
          }
        }
        float part[4];
#pragma unroll
        for (int c = 0; c < kWide; ++c) {
          const uint32_t l0 = word[0][c] & 0x0f0f0f0fu, h0 = word[0][c] & 0xf0f0f0f0u;   // row g
          const uint32_t l1 = word[1][c] & 0x0f0f0f0fu, h1 = word[1][c] & 0xf0f0f0f0u;   // row g + 8
          const uint4 v = xv[q * kWide + c];
          const uint32_t a[4] = {w4_pair<Half, 0>(l0, h0, off[0]), w4_pair<Half, 0>(l1, h1, off[1]),
                                 w4_pair<Half, 1>(l0, h0, off[0]), w4_pair<Half, 1>(l1, h1, off[1])};
          if (c == 0)
            mma16816<Half, true>(part, a, v.x, v.y);
          else
            mma16816<Half, false>(part, a, v.x, v.y);
          const uint32_t a2[4] = {w4_pair<Half, 2>(l0, h0, off[0]), w4_pair<Half, 2>(l1, h1, off[1]),
                                  w4_pair<Half, 3>(l0, h0, off[0]), w4_pair<Half, 3>(l1, h1, off[1])};
          mma16816<Half, false>(part, a2, v.z, v.w);
          if (m == 1) xv[q * kWide + c] = load_x(b_next, q * kWide + c);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) fma2(acc[m][h], s[h], part[2 * h], part[2 * h + 1]);
      }
    }
    if (++slot == kStages) slot = 0;
  }
  copies_wait<0>();
  __syncthreads();   // the ring is free
  // sums[warp][row of x][weight row]
  float* sums = reinterpret_cast<float*>(smem);
  constexpr int kLd = kTile + 4;   // rows apart in the banks
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sums[(warp * kRows + t * 2 + (i & 1)) * kLd + m * 16 + (i >> 1) * 8 + g] =
          i & 1 ? acc[m][i >> 1].y : acc[m][i >> 1].x;
  __syncthreads();
  for (int v = threadIdx.x; v < rows * (kTile / 2); v += kThreads) {
    const int r = v / (kTile / 2), n = v % (kTile / 2) * 2;
    if (n >= n_rows) continue;
    float2 f = *reinterpret_cast<const float2*>(sums + r * kLd + n);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float2 o = *reinterpret_cast<const float2*>(sums + (w * kRows + r) * kLd + n);
      f.x += o.x;
      f.y += o.y;
    }
    *reinterpret_cast<uint32_t*>(p.out + (row0 + r) * p.ld_out + i0 + n) =
        pack2<Half>(f.x * kW4Unit<Half>, f.y * kW4Unit<Half>);
  }
}

template <bool Half, int kGroup, bool kZeros>
int launch(const FewParams& p, int64_t tiles, size_t bytes, cudaStream_t s) {
  auto* kernel = grouped_w4_few_kernel<Half, kGroup, kZeros>;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRing + kW4FewScaleBytes) !=
        cudaSuccess)
      return check_launch("cudaFuncSetAttribute(grouped_w4_few_kernel)");
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  kernel<<<static_cast<unsigned>(tiles), kThreads, bytes, s>>>(p);
  return check_launch("grouped_w4_few_kernel");
}

template <bool Half, int kGroup>
int launch_zeros(const FewParams& p, int64_t tiles, size_t bytes, cudaStream_t s) {
  return p.zeros != nullptr ? launch<Half, kGroup, true>(p, tiles, bytes, s)
                            : launch<Half, kGroup, false>(p, tiles, bytes, s);
}

}  // namespace

int launch_grouped_w4_few(const W4Args& a, cudaStream_t s) {
  FewParams p;
  p.start = a.start;
  p.psum = a.psum;
  p.x = static_cast<const uint16_t*>(a.x);
  p.ld_x = a.ld_x;
  p.codes = a.codes;
  p.scales = static_cast<const uint16_t*>(a.scales);
  p.zeros = a.zeros;
  p.E = a.E;
  p.N = a.N;
  p.Kd = a.Kd;
  p.groups = a.Kd / a.group;
  p.pitch = w4_few_pitch(p.groups);
  p.M_cap = a.M_cap;
  p.out = a.out;
  p.ld_out = a.ld_out;
  p.status = a.status;
  const int64_t tiles =
      (a.max_rows / kRows + std::min<int64_t>(a.E, a.max_rows)) * ((a.N + kTile - 1) / kTile);
  MOE_REQUIRE(tiles <= INT32_MAX, "moe_grouped_mm_w4: sizes exceed 32-bit tile numbers");
  const size_t bytes = kRing + static_cast<size_t>(kTile) * p.pitch * (a.zeros != nullptr ? 3 : 2);
  auto* launch = a.group == 128  ? (a.half ? launch_zeros<true, 128> : launch_zeros<false, 128>)
                 : a.group == 64 ? (a.half ? launch_zeros<true, 64> : launch_zeros<false, 64>)
                                 : (a.half ? launch_zeros<true, 32> : launch_zeros<false, 32>);
  return launch(p, tiles, bytes, s);
}

}  // namespace moe

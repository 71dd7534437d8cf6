// The forward product and dgrad of grouped_mm16.cu for experts with few rows
// each: a batch of single tokens, where the time is that of reading the
// weights. Here the weights are the tensor core's first operand,
//   D[i, r] = sum_c W[i, c] X[r, c],   i = n (forward) or k (dgrad),
// so a tile is 128 weight rows by only as many activation rows (kRows: 16 to
// 128) as an expert is likely to have, and a stage holds 16 KB of weights and
// 2 to 16 KB of activations. The contraction of a tile is split over the CTAs
// of a cluster (1 to 8) when there are too few tiles to keep the GPU's memory
// system busy: each CTA leaves its partial sums in shared memory, the cluster
// meets, and each CTA adds the partials of its share of the rows, always in
// the same order, reading the others' through distributed shared memory.
//
// Bytes: the weights of every expert with rows, once (a second chunk of rows
// of one expert finds them in L2). Two CTAs fit an SM with about 100 KB of
// loads in flight each; a CTA does one tile, so that the hardware evens out
// the work and one CTA's start and end hide under the other's loads.
// Measured (in a graph): a decode batch of 32 rows for each of 64 experts of
// 4096 x 7168, 551 us, 6.8 TB/s of weights; one token of 8 of those experts, 73
// us (6.4 TB/s), where tiles of 256 weight rows by CTA pairs took 104; 18 experts
// of 96 x 4032 with a row each, 7.6 us (22 by pairs).
#include <algorithm>
#include <atomic>

#include "dtype16.cuh"
#include "gemm_host.h"
#include "host_util.h"
#include "mm16.cuh"

namespace moe {
namespace {

constexpr int kI = 128;                  // weight rows of a tile
constexpr int BC = 64;                   // contracted per stage
constexpr int kUmmaK = 16;
constexpr int kWBytes = kI * BC * 2;
constexpr int kThreads = 192;            // warps 0-3 epilogue, 4 TMA producer, 5 MMA issuer
constexpr int kMaxE = 1024;
constexpr int kMaxStages = 6;

struct FewParams {
  const int32_t* start;
  const int32_t* psum;
  int E;
  int width;            // D's weight rows: N (forward) or Kd (dgrad)
  int blocks;           // of BC along the contraction
  int rows;             // kRows of a tile: 16, 32, 64 or 128
  int stages;
  int splits;           // CTAs of a cluster
  int64_t M_cap;
  uint16_t* out;
  int64_t ld_out;
  int32_t* status;
};

template <bool kDgrad, bool Half>
__global__ void __launch_bounds__(kThreads, 2)
    grouped_mm16_few_kernel(const __grid_constant__ CUtensorMap tmW,
                            const __grid_constant__ CUtensorMap tmX, const FewParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done[1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ int s_warp_sum[kThreads / 32];
  __shared__ int s_e, s_row, s_rows;
  volatile int* abort_flag = &s_abort;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int splits = p.splits;
  const int rank = static_cast<int>(blockIdx.x) % splits;
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int ni = (p.width + kI - 1) / kI;
  const int chunk = tile / ni;
  const int i0 = (tile - chunk * ni) * kI;
  const int stage_bytes = kWBytes + p.rows * BC * 2;
  const uint32_t tmem_cols = static_cast<uint32_t>(max(p.rows, 32));

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(&done[0], 1);
    s_abort = 0;
    s_e = -1;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 5) {
    tmem_alloc(&s_tmem, tmem_cols);
    tmem_relinquish();
  }
  // Which expert has chunk number `chunk`? Thread t counts the chunks of
  // experts kPer t .. kPer t + kPer - 1; segments are clamped into the buffer.
  {
    constexpr int kPer = (kMaxE + kThreads - 1) / kThreads;
    const int per = (p.E + kThreads - 1) / kThreads;   // <= kPer
    int a[kPer], n[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = threadIdx.x * per + j;
      a[j] = n[j] = 0;
      if (j < per && e < p.E) {
        const int cap = static_cast<int>(p.M_cap);
        a[j] = min(max(p.start[e], 0), cap);
        n[j] = min(max(p.psum[e], a[j]), cap) - a[j];
        mine += (n[j] + p.rows - 1) / p.rows;
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
      const int c = (n[j] + p.rows - 1) / p.rows;
      if (chunk >= base && chunk < base + c) {
        s_e = threadIdx.x * per + j;
        s_row = a[j] + (chunk - base) * p.rows;
        s_rows = min(p.rows, n[j] - (chunk - base) * p.rows);
      }
      base += c;
    }
    // more chunks than the grid has: the caller's bound on the rows was wrong
    if (blockIdx.x == 0 && threadIdx.x == kThreads - 1 &&
        static_cast<int64_t>(base) * ni * splits > static_cast<int64_t>(gridDim.x))
      set_status(p.status, MOE_ERR_DEVICE_CHECK);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int e = s_e, row0 = s_row, rows = s_rows;
  const uint32_t tmem = s_tmem;

  if (e >= 0) {   // the same for the whole cluster
    const int b0 = p.blocks * rank / splits, b1 = p.blocks * (rank + 1) / splits;
    if (warp == 4 && lane == 0) {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      for (int b = b0; b < b1; ++b) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status)) break;
        uint8_t* sw = smem + stage * stage_bytes;
        const uint32_t bar = smem_u32(&full[stage]);
        mbar_arrive_expect_tx(&full[stage], stage_bytes);
        if (kDgrad) {
#pragma unroll
          for (int q = 0; q < kI / 64; ++q)
            load_3d<1>(sw + q * kMm16Panel, &tmW, i0 + q * 64, b * BC, e, bar);
        } else {
          load_3d<1>(sw, &tmW, b * BC, i0, e, bar);
        }
        load_2d<1>(sw + kWBytes, &tmX, b * BC, row0, bar);
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
      // every load has landed before the CTA can exit: each stage is released
      // once more
      for (int i = 0; i < p.stages; ++i) {
        if (!drain_wait(&empty[stage], phase ^ 1u)) break;
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
    } else if (warp == 5 && lane == 0) {
      // ---------------------------------------------------------- MMA issuer
      const uint32_t idesc = idesc_f16(Half, kDgrad, false, kI, p.rows);
      int stage = 0;
      uint32_t phase = 0;
      for (int b = b0; b < b1; ++b) {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t sw = smem_u32(smem + stage * stage_bytes);
        const uint32_t sx = sw + kWBytes;
#pragma unroll
        for (int k = 0; k < BC / kUmmaK; ++k)
          tc_mma_f16<1>(tmem,
                        kDgrad ? sw128_mnmajor_desc(sw + k * kUmmaK * 128)
                               : sw128_kmajor_desc(sw + k * kUmmaK * 2),
                        sw128_kmajor_desc(sx + k * kUmmaK * 2), idesc, (b > b0 || k > 0) ? 1u : 0u);
        tc_commit(&empty[stage]);
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      }
      tc_commit(&done[0]);
      drain_wait(&done[0], 0);   // also before TMEM is released
    } else if (warp < 4) {
      // ---------------------------------------------------------- epilogue
      // Thread t holds weight row i0 + t, a column of `out`; its TMEM columns
      // are the chunk's rows.
      const int i = i0 + threadIdx.x;
      const bool i_ok = i < p.width;
      const bool got = mbar_wait_warp(&done[0], 0, abort_flag, p.status);
      tc_fence_after();
      uint16_t* out = p.out + static_cast<int64_t>(row0) * p.ld_out + i;
      float* part = reinterpret_cast<float*>(smem);   // the ring is free: every MMA is done
      for (int r0 = 0; r0 < rows && got; r0 += 32) {
        uint32_t v[32];
        __syncwarp();   // lanes past the last weight row stored nothing
        tc_ld32_wait(tmem + (static_cast<uint32_t>(warp * 32) << 16) + r0, v);
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          if (r0 + r >= rows) break;
          if (splits > 1)
            part[(r0 + r) * kI + threadIdx.x] = __uint_as_float(v[r]);
          else if (i_ok)
            out[(r0 + r) * p.ld_out] =
                static_cast<uint16_t>(pack2<Half>(__uint_as_float(v[r]), 0.0f) & 0xffffu);
        }
      }
    }
    if (splits > 1) {
      cluster_sync();
      if (warp < 4) {
        // this CTA's share of the rows: the partials of all CTAs, in order
        const int i = i0 + threadIdx.x;
        const int ra = rows * rank / splits, rb = rows * (rank + 1) / splits;
        uint16_t* out = p.out + static_cast<int64_t>(row0) * p.ld_out + i;
        uint32_t from[8];
#pragma unroll
        for (int s = 0; s < 8; ++s)
          from[s] = s < splits ? cta_smem(smem, s) + static_cast<uint32_t>(threadIdx.x) * 4 : 0;
        for (int r = ra; r < rb; ++r) {
          float f[8], sum = 0.0f;
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (s < splits)
              asm volatile("ld.shared::cluster.f32 %0, [%1];"
                           : "=f"(f[s])
                           : "r"(from[s] + static_cast<uint32_t>(r * kI * 4)));
#pragma unroll
          for (int s = 0; s < 8; ++s)
            if (s < splits) sum += f[s];
          if (i < p.width && !*abort_flag)
            out[r * p.ld_out] = static_cast<uint16_t>(pack2<Half>(sum, 0.0f) & 0xffffu);
        }
      }
      cluster_sync();   // no CTA leaves while its partials are read
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    __syncwarp();   // lane 0 comes from the issuer's role
    tmem_dealloc(tmem, tmem_cols);
  }
}

// Ring of a CTA: two CTAs share an SM's 228 KB.
int stages_for(int rows) { return rows <= 16 ? 6 : (rows <= 32 ? 5 : (rows <= 64 ? 4 : 3)); }
int ring_bytes(int rows) { return stages_for(rows) * (kWBytes + rows * BC * 2) + 1024; }
constexpr int kMostSmem = 6 * (kWBytes + 16 * BC * 2) + 1024;

template <bool kDgrad, bool Half>
int launch(const CUtensorMap& tw, const CUtensorMap& tx, const FewParams& p, int64_t tiles,
           cudaStream_t s) {
  auto* kernel = grouped_mm16_few_kernel<kDgrad, Half>;
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem) != cudaSuccess)
      return check_launch("cudaFuncSetAttribute(grouped_mm16_few_kernel)");
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(ring_bytes(p.rows));
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(p.splits);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, tw, tx, p);
  return check_launch("grouped_mm16_few_kernel");
}

}  // namespace

int launch_grouped_mm16_few(bool dgrad, bool half, const void* a, int64_t ld_a, const void* w,
                            const int32_t* start, const int32_t* psum, int E, int N, int Kd,
                            int64_t M_cap, int64_t max_rows, uint16_t* out, int64_t ld_out,
                            int32_t* status, cudaStream_t s) {
  FewParams p;
  p.start = start;
  p.psum = psum;
  p.E = E;
  p.width = dgrad ? Kd : N;
  const int in = dgrad ? N : Kd;
  p.blocks = (in + BC - 1) / BC;
  p.M_cap = M_cap;
  p.out = out;
  p.ld_out = ld_out;
  p.status = status;
  // Experts that can have rows, and rows for about twice their mean: one token
  // of 8 out of 64 experts of 4096 x 7168 takes 73 us with 16 rows a tile, 112
  // with 128; 16 rows each of 32 experts of 4096 x 4096 164 us with 32, 172 with
  // 128.
  const int64_t live = std::min<int64_t>(E, max_rows);
  const int64_t mean = (max_rows + live - 1) / live;
  p.rows = mean <= 8 ? 16 : (mean <= 20 ? 32 : (mean <= 48 ? 64 : 128));
  p.stages = stages_for(p.rows);
  const int64_t ni = (p.width + kI - 1) / kI;
  // Splits: until every SM has a CTA, none with less than six blocks. More cost
  // more in their starts than they even out: one token of 8 out of 64 experts of
  // 4096 x 7168 takes 73 us whole (256 tiles), 76, 82 and 95 in two, four and
  // eight parts; six experts of 3416 x 6344 48 whole, 59 in two. Two experts' 96 x
  // 4032 take 7.6 us in eight parts, 9.4 in four; 512 x 512 takes 6.6 whole, 7.5 in
  // two.
  const int64_t want = device_sm_count();
  p.splits = 1;
  while (p.splits < 8 && live * ni * p.splits < want && p.blocks / (2 * p.splits) >= 6) p.splits *= 2;
  const int64_t tiles = (max_rows / p.rows + live) * ni;
  MOE_REQUIRE(tiles * p.splits <= INT32_MAX, "grouped product: sizes exceed 32-bit tile numbers");
  CUtensorMap tw, tx;
  int rc = make_tmap_weights16(&tw, w, Kd, N, E, dgrad ? 64 : kI);
  if (rc != MOE_OK) return rc;
  rc = make_tmap_rows16(&tx, a, in, M_cap, ld_a, p.rows);
  if (rc != MOE_OK) return rc;
  if (dgrad)
    return half ? launch<true, true>(tw, tx, p, tiles, s) : launch<true, false>(tw, tx, p, tiles, s);
  return half ? launch<false, true>(tw, tx, p, tiles, s) : launch<false, false>(tw, tx, p, tiles, s);
}

}  // namespace moe

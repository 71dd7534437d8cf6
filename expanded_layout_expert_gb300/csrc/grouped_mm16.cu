// moe_grouped_mm / _dgrad / _wgrad: the products of an MoE layer's experts in
// bf16 or fp16, over the rows that the expanded layout gives each expert
// (rows [start[e], psum[e]) of the activations, any number of them):
//
//   forward  y[r, n]    = sum_k x[r, k] w[e, n, k]
//   dgrad    dx[r, k]   = sum_n dy[r, n] w[e, n, k]
//   wgrad    dw[e, n, k] (+)= sum_r dy[r, n] x[r, k]     r in the segment of e
//
// One kernel computes D[i, j] = sum_c A[i, c] B[j, c] on the 5th-generation
// tensor cores for all three; they differ in what a tile's operands are:
//
//              i (rows of D)   j (columns)    c (contracted)   A, B in memory
//   forward    rows of x       n              k                c-contiguous both
//   dgrad      rows of dy      k              n                A c-contiguous, B j-contiguous
//   wgrad      n               k              rows             both i/j-contiguous
//
// The tensor core reads either order from shared memory (the "major" bits of
// the instruction descriptor), so no operand is ever transposed in memory.
// Weights go through a 3-D tensor map [E, N, Kd], so a tile that reaches past
// an expert's matrix reads zeros, never the next expert's values (which may be
// infinite or NaN). Rows past a segment's end do belong to other experts or to
// a gap: in forward and dgrad they only make rows of D that are not stored;
// in wgrad they are contracted over, so both operands' rows there are set to
// zero in shared memory before the tensor core reads them. That ragged block
// comes first in the tile, so that this is done while the tensor core still
// works on the tile before.
//
// Accumulation is in fp32 in tensor memory over the whole contraction; each
// result is rounded once.
//
// One persistent CTA per SM, warp-specialised as in grouped_gemm.cu: warp 0
// TMA producer, warp 1 tcgen05.mma issuer, warp 2 zeroes ragged rows (wgrad),
// warps 4-7 epilogue. Two 256-column accumulators let the epilogue of a tile
// run under the next tile's products.
#include "common.cuh"
#include "dtype16.cuh"
#include "gemm_host.h"
#include "host_util.h"

namespace moe {
namespace {

enum Mode { kForward = 0, kDgrad = 1, kWgrad = 2 };

constexpr int BM = 128;          // rows of D per tile
constexpr int BN = 256;          // columns of D per tile
constexpr int BC = 64;           // contracted per stage: one 128-byte swizzle row of 16-bit values
constexpr int kUmmaK = 16;       // contracted per tcgen05.mma
constexpr int kStages = 4;
constexpr int kABytes = BM * BC * 2;
constexpr int kBBytes = BN * BC * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kPanel = 64 * 128;   // 64 rows of 128 bytes: one TMA box of an i/j-contiguous operand
constexpr int kAcc = 2;
constexpr int kTmemCols = kAcc * BN;
constexpr int kEpiWarps = 4;
constexpr int kThreads = 256;
constexpr int kMaxE = 1024;
constexpr int kRaster = 8;       // tiles in a column of the raster (see tile_at)

constexpr int kStoreOffset = kStages * kStageBytes;             // per epilogue warp: 32 rows x 128 bytes
constexpr int kBarOffset = kStoreOffset + kEpiWarps * 32 * 128;
constexpr int kNumBars = 3 * kStages + 2 * kAcc + 1;
constexpr int kMiscOffset = kBarOffset + kNumBars * 8;          // tmem slot, abort flag
constexpr int kTableOffset = (kMiscOffset + 8 + 15) / 16 * 16;  // tile prefix [E+1], start [E], end [E]
constexpr int smem_bytes(int E) { return 1024 + kTableOffset + (3 * E + 1) * 4; }
static_assert(smem_bytes(kMaxE) <= 227 * 1024, "shared memory");

struct Params {
  const int32_t* start;
  const int32_t* psum;
  int E, N, Kd;          // weights [E, N, Kd]
  int64_t M_cap;
  void* out;             // forward [M_cap, ld_out = N..], dgrad [M_cap, Kd..], wgrad [E, N, Kd]
  int64_t ld_out;
  int32_t* status;
};

// Tensor-core operand whose contiguous axis is i/j, not c: panels of 64 c rows
// x 128 bytes (64 values), 128-byte swizzle. Groups of 8 c rows are 1024 bytes
// apart (stride byte offset), panels kPanel apart (leading byte offset).
MOE_DEV uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kPanel >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Instruction descriptor: dense, D = f32, A and B both fp16 or both bf16;
// a_mn / b_mn: the operand's contiguous axis is i / j.
constexpr uint32_t idesc_f16(bool half, bool a_mn, bool b_mn, int M, int N) {
  return (1u << 4) | ((half ? 0u : 1u) << 7) | ((half ? 0u : 1u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit operands, K = 16.
MOE_DEV void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

MOE_DEV void tma_load_3d(void* dst, const CUtensorMap* tm, int32_t x, int32_t y, int32_t z,
                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

MOE_DEV void tc_wait32(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tc_regs_landed(v);
}

MOE_DEV void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) {
    if (clock64() - t0 > kWaitLimitCycles) return;
  }
}

struct Tile {
  int e, i0, j0;   // expert; first row (forward, dgrad: within the segment) and column of D
  int row0, rows;  // the expert's segment
};

// Out16: D is stored in the operands' type, else (wgrad) in fp32. Add: D is
// added to what `out` holds.
template <int kMode, bool Half, bool Out16, bool Add>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_mm16_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOffset);
  uint64_t* empty = full + kStages;
  uint64_t* clean = empty + kStages;    // wgrad: the stage's ragged rows are zero
  uint64_t* tfull = clean + kStages;
  uint64_t* tempty = tfull + kAcc;
  uint64_t* mma_done = tempty + kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOffset);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOffset + 4);
  int* s_tp = reinterpret_cast<int*>(smem + kTableOffset);
  int* s_start = s_tp + p.E + 1;
  int* s_end = s_start + p.E;
  __shared__ int s_warp_sum[kThreads / 32];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kMode == kWgrad ? 2 : 1);   // MMA (and the zeroing warp)
      mbar_init(&clean[s], 1);
    }
    for (int b = 0; b < kAcc; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  // Segments, clamped into the buffer, and (forward, dgrad) the prefix of
  // their row tiles: thread t owns experts 4t .. 4t+3.
  {
    int mine = 0, cnt[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = threadIdx.x * 4 + j;
      if (e < p.E) {
        const int cap = static_cast<int>(p.M_cap);
        const int a = min(max(p.start[e], 0), cap);
        const int b = min(max(p.psum[e], a), cap);
        s_start[e] = a;
        s_end[e] = b;
        cnt[j] = (b - a + BM - 1) / BM;
        mine += cnt[j];
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
    for (int j = 0; j < 4; ++j) {
      const int e = threadIdx.x * 4 + j;
      if (e < p.E) {
        s_tp[e] = base;
        base += cnt[j];
        if (e == p.E - 1) s_tp[p.E] = base;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // D's columns, its column tiles and (wgrad) row tiles
  const int cols = kMode == kForward ? p.N : p.Kd;
  const int nj = (cols + BN - 1) / BN;
  const int ni_w = (p.N + BM - 1) / BM;
  const int num_tiles = kMode == kWgrad ? p.E * ni_w * nj : s_tp[p.E] * nj;

  // Tile id -> tile. Within an expert the tiles go in columns of kRaster row
  // tiles, row tile fastest, so the CTAs that run at one time share both
  // operands' panels in L2.
  auto tile_at = [&](int tile) {
    Tile t;
    int l, ni;
    if (kMode == kWgrad) {
      t.e = tile / (ni_w * nj);
      l = tile - t.e * ni_w * nj;
      ni = ni_w;
    } else {
      const int m = tile / nj;
      int lo = 0, hi = p.E - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tp[mid] <= m) lo = mid; else hi = mid - 1;
      }
      t.e = lo;
      l = tile - s_tp[lo] * nj;
      ni = s_tp[lo + 1] - s_tp[lo];
    }
    const int g = l / (kRaster * nj);
    const int in = l - g * kRaster * nj;
    const int gi = min(kRaster, ni - g * kRaster);
    t.i0 = (g * kRaster + in % gi) * BM;
    t.j0 = (in / gi) * BN;
    t.row0 = s_start[t.e];
    t.rows = s_end[t.e] - t.row0;
    return t;
  };
  // blocks of BC along the contracted axis
  const int blocks_fd = ((kMode == kForward ? p.Kd : p.N) + BC - 1) / BC;
  auto num_blocks = [&](const Tile& t) { return kMode == kWgrad ? (t.rows + BC - 1) / BC : blocks_fd; };
  // wgrad: rows of the ragged block (the tile's first), 0 if all are whole
  auto ragged = [&](const Tile& t) { return kMode == kWgrad ? t.rows % BC : 0; };

  if (warp == 0 && lane == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
      const Tile t = tile_at(tile);
      const int nb = num_blocks(t);
      const int rag = ragged(t);
      for (int b = 0; b < nb; ++b) {
        if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
        uint8_t* sa = smem + stage * kStageBytes;
        uint8_t* sb = sa + kABytes;
        mbar_arrive_expect_tx(&full[stage], kStageBytes);
        if (kMode == kForward) {
          tma_load_2d(sa, &tmA, b * BC, t.row0 + t.i0, &full[stage]);
          tma_load_3d(sb, &tmB, b * BC, t.j0, t.e, &full[stage]);
        } else if (kMode == kDgrad) {
          tma_load_2d(sa, &tmA, b * BC, t.row0 + t.i0, &full[stage]);
#pragma unroll
          for (int q = 0; q < BN / 64; ++q)
            tma_load_3d(sb + q * kPanel, &tmB, t.j0 + q * 64, b * BC, t.e, &full[stage]);
        } else {
          // the ragged block first: it is the segment's last
          const int c = rag ? (b == 0 ? t.rows - rag : (b - 1) * BC) : b * BC;
#pragma unroll
          for (int q = 0; q < BM / 64; ++q)
            tma_load_2d(sa + q * kPanel, &tmA, t.i0 + q * 64, t.row0 + c, &full[stage]);
#pragma unroll
          for (int q = 0; q < BN / 64; ++q)
            tma_load_2d(sb + q * kPanel, &tmB, t.j0 + q * 64, t.row0 + c, &full[stage]);
        }
        ++issued;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
    // Let the last loads land before the CTA can exit.
    const int outstanding = issued < kStages ? issued : kStages;
    for (int i = 1; i <= outstanding; ++i) {
      int s = stage - i;
      uint32_t ph = phase;
      if (s < 0) { s += kStages; ph ^= 1u; }
      drain_wait(&full[s], ph);
    }
  } else if (warp == 1 && lane == 0) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t idesc = idesc_f16(Half, kMode == kWgrad, kMode != kForward, BM, BN);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    uint32_t clean_phase[kStages] = {};
    bool ok = true;
    for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
      const Tile t = tile_at(tile);
      const int nb = num_blocks(t);
      if (nb == 0) continue;   // wgrad of an expert without rows: the epilogue stores zeros
      const int rag = ragged(t);
      if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, p.status)) break;
      const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
      for (int b = 0; b < nb; ++b) {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
        int steps = BC / kUmmaK;
        if (kMode == kWgrad && rag && b == 0) {
#pragma unroll
          for (int s = 0; s < kStages; ++s)
            if (s == stage) {
              ok = mbar_wait(&clean[s], clean_phase[s], abort_flag, p.status);
              clean_phase[s] ^= 1u;
            }
          if (!ok) break;
          steps = (rag + kUmmaK - 1) / kUmmaK;
        }
        tc_fence_after();
        const uint32_t sa = smem_u32(smem + stage * kStageBytes);
        const uint32_t sb = sa + kABytes;
        for (int k = 0; k < steps; ++k) {
          // 16 contracted values on: 32 bytes along a c-contiguous row, 16
          // rows of 128 bytes otherwise
          const uint64_t da = kMode == kWgrad ? sw128_mnmajor_desc(sa + k * kUmmaK * 128)
                                              : sw128_kmajor_desc(sa + k * kUmmaK * 2);
          const uint64_t db = kMode != kForward ? sw128_mnmajor_desc(sb + k * kUmmaK * 128)
                                                : sw128_kmajor_desc(sb + k * kUmmaK * 2);
          tc_mma_f16(d, da, db, idesc, (b > 0 || k > 0) ? 1u : 0u);
        }
        tc_commit(&empty[stage]);
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
      if (!ok) break;
      tc_commit(&tfull[acc]);
      if (++acc == kAcc) { acc = 0; acc_phase ^= 1u; }
    }
    // Every MMA issued so far must complete before TMEM is released.
    tc_commit(mma_done);
    drain_wait(mma_done, 0);
  } else if (warp == 2 && kMode == kWgrad) {
    // ------------------------------------------------- ragged rows to zero
    // Only the rows up to the next multiple of 16 are read by the tensor core.
    // The warp follows every block and has its own arrival on `empty`: a
    // parity wait is sound only for a waiter that is never two phases away.
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < num_tiles && ok; tile += gridDim.x) {
      const Tile t = tile_at(tile);
      const int nb = num_blocks(t);
      const int rag = ragged(t);
      for (int b = 0; b < nb; ++b) {
        if (!mbar_wait_warp(&full[stage], phase, abort_flag, p.status)) { ok = false; break; }
        if (rag && b == 0) {
          const int r1 = (rag + kUmmaK - 1) / kUmmaK * kUmmaK;
          uint8_t* s = smem + stage * kStageBytes;
          const int per_panel = (r1 - rag) * 8;   // 16-byte vectors
          for (int q = 0; q < (BM + BN) / 64; ++q)
            for (int v = lane; v < per_panel; v += 32)
              *reinterpret_cast<uint4*>(s + q * kPanel + rag * 128 + v * 16) = make_uint4(0, 0, 0, 0);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&clean[stage]);
        }
        if (lane == 0) mbar_arrive(&empty[stage]);
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    // A warp owns 32 rows of D (its TMEM lanes): it reads 32 or 64 columns,
    // converts, passes them through shared memory (swizzled, so that neither
    // side has bank conflicts) and stores whole row pieces. Where 16-bit
    // results are added to, the pieces stay in fp32 until after the addition,
    // so that the sum is rounded once.
    const int quarter = warp & 3;
    const uint32_t stg = smem_u32(smem + kStoreOffset + quarter * 32 * 128);
    constexpr int kElem = Out16 ? 2 : 4;
    constexpr bool kStage16 = Out16 && !Add;
    constexpr int kCols = kStage16 ? 64 : 32;   // columns of D per staged 128-byte row piece
    constexpr int kVec = kCols / 8;             // columns per staged 16-byte vector
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x) {
      const Tile t = tile_at(tile);
      const bool empty_tile = num_blocks(t) == 0;
      if (empty_tile && Add) continue;
      if (!empty_tile) {
        if (!mbar_wait_warp(&tfull[acc], acc_phase, abort_flag, p.status)) break;
        tc_fence_after();
      }
      const uint32_t tq = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                          static_cast<uint32_t>(acc * BN);
      const int ilim = kMode == kWgrad ? p.N : t.rows;   // rows of D that exist
      const int iw = t.i0 + quarter * 32;                // this warp's first row
      const int64_t orow = kMode == kWgrad ? static_cast<int64_t>(t.e) * p.N : t.row0;
      uint8_t* out = static_cast<uint8_t*>(p.out);
      for (int c0 = 0; c0 < BN; c0 += kCols) {
        uint32_t w[32];   // the thread's row, 128 bytes
        if (empty_tile) {
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = 0u;
        } else if (kStage16) {
          uint32_t va[32], vb[32];
          tc_ld32(tq + c0, va);
          tc_ld32(tq + c0 + 32, vb);
          tc_wait64(va, vb);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            w[i] = pack2<Half>(__uint_as_float(va[2 * i]), __uint_as_float(va[2 * i + 1]));
            w[16 + i] = pack2<Half>(__uint_as_float(vb[2 * i]), __uint_as_float(vb[2 * i + 1]));
          }
        } else {
          tc_ld32(tq + c0, w);
          tc_wait32(w);
        }
        if (!empty_tile && c0 + kCols == BN) {   // the last read has landed
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[acc]);
        }
        if (t.j0 + c0 >= cols || iw >= ilim) continue;   // the same for the whole warp
#pragma unroll
        for (int c = 0; c < 8; ++c)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                           stg + lane * 128 + ((c ^ (lane & 7)) << 4)),
                       "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                       : "memory");
        __syncwarp();
        const int c = lane & 7;
        const bool col_ok = t.j0 + c0 + c * kVec < cols;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3);
          uint4 v;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                       : "r"(stg + r * 128 + ((c ^ (r & 7)) << 4))
                       : "memory");
          if (iw + r < ilim && col_ok) {
            uint8_t* dst = out + ((orow + iw + r) * p.ld_out + t.j0 + c0 + c * kVec) * kElem;
            if (Add) {
              float f[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z),
                            __uint_as_float(v.w)};
              if (Out16) {
                const uint2 o = *reinterpret_cast<const uint2*>(dst);
                const float2 lo = unpack2<Half>(o.x), hi = unpack2<Half>(o.y);
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<Half>(lo.x + f[0], lo.y + f[1]),
                                                            pack2<Half>(hi.x + f[2], hi.y + f[3]));
              } else {
                const float4 o = *reinterpret_cast<const float4*>(dst);
                *reinterpret_cast<float4*>(dst) =
                    make_float4(o.x + f[0], o.y + f[1], o.z + f[2], o.w + f[3]);
              }
            } else {
              *reinterpret_cast<uint4*>(dst) = v;
            }
          }
        }
        __syncwarp();
      }
      if (!empty_tile && ++acc == kAcc) { acc = 0; acc_phase ^= 1u; }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <int kMode, bool Half, bool Out16, bool Add>
int launch(const CUtensorMap& ta, const CUtensorMap& tb, const Params& p, int64_t max_tiles,
           cudaStream_t s) {
  auto* kernel = grouped_mm16_kernel<kMode, Half, Out16, Add>;
  static bool attr_set[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 0 && dev < 64 && !attr_set[dev]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem_bytes(kMaxE)) != cudaSuccess)
      return check_launch("cudaFuncSetAttribute(grouped_mm16_kernel)");
    attr_set[dev] = true;
  }
  int64_t grid = device_sm_count();
  if (grid > max_tiles) grid = max_tiles;
  kernel<<<static_cast<unsigned>(grid), kThreads, smem_bytes(p.E), s>>>(ta, tb, p);
  return check_launch("grouped_mm16_kernel");
}

int check_sizes(const char* what, int dtype, int E, int N, int Kd, int64_t M_cap) {
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "%s: dtype must be MOE_BF16 or MOE_F16", what);
  MOE_REQUIRE(E > 0 && E <= kMaxE, "%s: E must be in [1, 1024]", what);
  MOE_REQUIRE(N > 0 && N % 8 == 0 && Kd > 0 && Kd % 8 == 0,
              "%s: N and Kd must be positive multiples of 8", what);
  MOE_REQUIRE(M_cap >= 0 && M_cap <= INT32_MAX - BM, "%s: bad M_cap", what);
  // linear tile ids are 32-bit
  const int64_t nj = (N > Kd ? N : Kd) / BN + 1;
  MOE_REQUIRE((M_cap / BM + E) * nj <= INT32_MAX && static_cast<int64_t>(E) * (N / BM + 1) * nj <= INT32_MAX,
              "%s: sizes exceed 32-bit tile numbers", what);
  return MOE_OK;
}

int check_rows(const char* what, const char* name, const void* a, int64_t ld, int width) {
  MOE_REQUIRE(a && aligned(a, 16), "%s: %s must be non-null and 16-byte aligned", what, name);
  MOE_REQUIRE(ld >= width && ld % 8 == 0, "%s: the row stride of %s must be a multiple of 8, at least %d",
              what, name, width);
  return MOE_OK;
}

#define MOE_TRY(expr)                  \
  do {                                 \
    const int rc_ = (expr);            \
    if (rc_ != MOE_OK) return rc_;     \
  } while (0)

// Forward and dgrad: rows [M_cap, in] times weights -> rows [M_cap, out].
int rows_times_weights(const char* what, bool dgrad, const void* a, int64_t ld_a, const void* w,
                       const int32_t* start, const int32_t* psum, int dtype, int E, int N, int Kd,
                       int64_t M_cap, void* out, int64_t ld_out, int32_t* d_status, cudaStream_t s) {
  MOE_TRY(check_sizes(what, dtype, E, N, Kd, M_cap));
  const int in = dgrad ? N : Kd, width = dgrad ? Kd : N;
  if (M_cap > 0) {
    MOE_REQUIRE(start && psum, "%s: null segments", what);
    MOE_TRY(check_rows(what, dgrad ? "dy" : "x", a, ld_a, in));
    MOE_TRY(check_rows(what, "w", w, Kd, Kd));
    MOE_TRY(check_rows(what, dgrad ? "dx" : "out", out, ld_out, width));
  }
  MOE_REQUIRE_DEVICE();
  if (M_cap == 0) return MOE_OK;
  CUtensorMap ta, tb;
  MOE_TRY(make_tmap_rows16(&ta, a, in, M_cap, ld_a, BM));
  MOE_TRY(make_tmap_weights16(&tb, w, Kd, N, E, dgrad ? 64 : BN));
  Params p;
  p.start = start;
  p.psum = psum;
  p.E = E;
  p.N = N;
  p.Kd = Kd;
  p.M_cap = M_cap;
  p.out = out;
  p.ld_out = ld_out;
  p.status = d_status;
  const int64_t m_tiles = M_cap / BM + (E < M_cap ? E : M_cap);
  const int64_t tiles = m_tiles * ((width + BN - 1) / BN);
  const bool half = dtype == MOE_F16;
  if (dgrad)
    return half ? launch<kDgrad, true, true, false>(ta, tb, p, tiles, s)
                : launch<kDgrad, false, true, false>(ta, tb, p, tiles, s);
  return half ? launch<kForward, true, true, false>(ta, tb, p, tiles, s)
              : launch<kForward, false, true, false>(ta, tb, p, tiles, s);
}

template <bool Half>
int launch_wgrad(const CUtensorMap& ta, const CUtensorMap& tb, const Params& p, int64_t tiles,
                 bool out16, bool add, cudaStream_t s) {
  if (out16)
    return add ? launch<kWgrad, Half, true, true>(ta, tb, p, tiles, s)
               : launch<kWgrad, Half, true, false>(ta, tb, p, tiles, s);
  return add ? launch<kWgrad, Half, false, true>(ta, tb, p, tiles, s)
             : launch<kWgrad, Half, false, false>(ta, tb, p, tiles, s);
}

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_mm(const void* x, int64_t ld_x, const void* w, const int32_t* start,
                              const int32_t* psum, int dtype, int E, int N, int Kd, int64_t M_cap,
                              void* out, int64_t ld_out, int32_t* d_status, moe_stream_t stream) {
  return moe::rows_times_weights("moe_grouped_mm", false, x, ld_x, w, start, psum, dtype, E, N, Kd,
                                 M_cap, out, ld_out, d_status, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_grouped_mm_dgrad(const void* dy, int64_t ld_dy, const void* w,
                                    const int32_t* start, const int32_t* psum, int dtype, int E,
                                    int N, int Kd, int64_t M_cap, void* dx, int64_t ld_dx,
                                    int32_t* d_status, moe_stream_t stream) {
  return moe::rows_times_weights("moe_grouped_mm_dgrad", true, dy, ld_dy, w, start, psum, dtype, E, N,
                                 Kd, M_cap, dx, ld_dx, d_status, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_grouped_mm_wgrad(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                    const int32_t* start, const int32_t* psum, int dtype, int E,
                                    int N, int Kd, int64_t M_cap, void* dw, int out_dtype,
                                    int accumulate, int32_t* d_status, moe_stream_t stream) {
  using namespace moe;
  const char* what = "moe_grouped_mm_wgrad";
  MOE_TRY(check_sizes(what, dtype, E, N, Kd, M_cap));
  MOE_REQUIRE(out_dtype == dtype || out_dtype == MOE_F32, "%s: dw must have the operands' type or be fp32",
              what);
  MOE_TRY(check_rows(what, "dw", dw, Kd, Kd));
  if (M_cap > 0) {
    MOE_REQUIRE(start && psum, "%s: null segments", what);
    MOE_TRY(check_rows(what, "dy", dy, ld_dy, N));
    MOE_TRY(check_rows(what, "x", x, ld_x, Kd));
  }
  MOE_REQUIRE_DEVICE();
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M_cap == 0) {   // no rows at all: the gradient is zero
    if (accumulate) return MOE_OK;
    const size_t bytes = static_cast<size_t>(E) * N * Kd * (out_dtype == MOE_F32 ? 4 : 2);
    if (cudaMemsetAsync(dw, 0, bytes, s) != cudaSuccess) return check_launch("cudaMemsetAsync(dw)");
    return MOE_OK;
  }
  CUtensorMap ta, tb;
  MOE_TRY(make_tmap_rows16(&ta, dy, N, M_cap, ld_dy, BC));
  MOE_TRY(make_tmap_rows16(&tb, x, Kd, M_cap, ld_x, BC));
  Params p;
  p.start = start;
  p.psum = psum;
  p.E = E;
  p.N = N;
  p.Kd = Kd;
  p.M_cap = M_cap;
  p.out = dw;
  p.ld_out = Kd;
  p.status = d_status;
  const int64_t tiles = static_cast<int64_t>(E) * ((N + BM - 1) / BM) * ((Kd + BN - 1) / BN);
  const bool out16 = out_dtype != MOE_F32, add = accumulate != 0;
  return dtype == MOE_F16 ? launch_wgrad<true>(ta, tb, p, tiles, out16, add, s)
                          : launch_wgrad<false>(ta, tb, p, tiles, out16, add, s);
}

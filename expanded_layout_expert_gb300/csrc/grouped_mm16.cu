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
// Accumulation is in fp32 and each result is rounded once. The tensor core
// truncates where it adds, so its sums drift towards zero by about 1e-6 of
// their size per 1024 contracted values (measured: 1.0e-6 at 1024 rows, 1.9e-5
// at 16384, 8.7e-5 at 65536 against 1e-7 to 5e-7 of fp32 products). In
// forward and dgrad that is far below the rounding to 16 bits. wgrad contracts
// over as many rows as an expert has, so its sums leave tensor memory after at
// most 512 rows (fp32 results; 4096 for 16-bit ones) and are added up, rounding to
// nearest, in the epilogue's registers.
//
// Persistent CTAs, one per SM, warp-specialised as in grouped_gemm.cu: warp 0
// TMA producer, warp 1 tcgen05.mma issuer, warp 2 zeroes ragged rows (wgrad),
// warps 4-11 epilogue. Two 256-column accumulators let the epilogue of a tile
// run under the next tile's products. Two CTAs work on one 256 x 256 tile
// (cta_group::2): each loads half of both operands, so a 64-deep block costs an
// SM 32 KB instead of 48. With one CTA per 128 x 256 tile a block took 705
// cycles (1024 rows an expert, 4096 x 4096, forward), with pairs 558; the
// tensor core's own time is 512. A segment's last tile, if it has at most 128
// rows, is done with 64 rows per CTA (300 rows an expert: 331 instead of 367
// us). wgrad has single-CTA tiles where N <= 128, and where tiles are so few that
// their rows are shared by a cluster; forward and dgrad of experts with few rows
// are grouped_mm16_few.cu's.
//
// What bounds it: power. Forward and dgrad of long segments run at 1.5 to 1.6
// PFLOP/s with the SM clock held near 1.4 GHz by the power limit, 92-97 % of what
// the library's product of the same rows and weights reaches there; segments of
// 160 to 600 rows are bound by whole tiles (300 rows an expert: 384 in tiles). wgrad (both operands i/j-contiguous)
// is bound by the rate at which the tensor core reads such an A: 668 cycles a
// block on long segments, against 531 for the others.
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "dtype16.cuh"
#include "gemm_host.h"
#include "host_util.h"
#include "mm16.cuh"

namespace moe {
namespace {

enum Mode { kForward = 0, kDgrad = 1, kWgrad = 2 };

constexpr int BMC = 128;         // rows of D per CTA
constexpr int BN = 256;          // columns of D per tile
constexpr int BC = 64;           // contracted per stage: one 128-byte swizzle row of 16-bit values
constexpr int kUmmaK = 16;       // contracted per tcgen05.mma
constexpr int kPanel = kMm16Panel;
constexpr int kAcc = 2;
constexpr int kTmemCols = kAcc * BN;
constexpr int kEpiWarps = 8;     // two per TMEM lane quarter
constexpr int kThreads = 32 * (4 + kEpiWarps);
constexpr int kMaxE = 1024;
// wgrad: blocks of BC summed in tensor memory at a time, at most. fp32 results:
// 512 rows, whose error is 5e-7 (plain fp32 products: 2e-7 to 1.7e-6); 896 rows were
// 9e-7 off and took 906-911 us instead of 910-919 (1024 rows an expert, 4096 x
// 4096). 16-bit results round to 2^-8 or 2^-11 anyway, and short chunks make the tensor
// core wait for an epilogue that is still storing the tile before: with 8 blocks
// they take 844-849 us there, with up to 64 813; those of the Zipf batch (124 k rows,
// 7168 x 2048) 2.62-2.65 and 2.52-2.55 ms.
constexpr int max_chunk(bool out16) { return out16 ? 64 : 8; }
// wgrad: warps 0-3 hand registers to the epilogue, whose threads hold 128 sums
// (56 * 128 + 224 * 256 = 168 * 384, the registers the block is launched with).
constexpr int kRegsLow = 56;
constexpr int kRegsHigh = 224;
static_assert(kRegsLow * 128 + kRegsHigh * 256 == 168 * kThreads, "register split");
// Row tiles in a column of the raster (see tile_at). Seconds long, at the power
// limit, it decides little: forward takes 4.76 ms with 4, 8 and 16 (Zipf batch, 124 k
// rows, 4096 x 7168); wgrad of that batch 2.51, 2.53 and 2.53 ms with 2, 4 and 8, and
// added to fp32 (1024 rows an expert, 4096 x 4096) 1.03, 1.06 and 1.04 ms.
constexpr int raster(int mode) { return mode == kWgrad ? 4 : 8; }

// kCtas CTAs work on one tile of kCtas * 128 x 256.
template <int kCtas>
struct Cfg {
  static constexpr int BM = kCtas * BMC;
  static constexpr int kBRows = BN / kCtas;             // columns of D whose operand this CTA loads
  static constexpr int kABytes = BMC * BC * 2;
  static constexpr int kBBytes = kBRows * BC * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // Of a row of D, staged at a time: 64 bytes leave room for six stages (with
  // 1024 ragged rows an expert and 4096 x 4096 weights wgrad took 767 cycles a
  // block so, 785 with 128 bytes and five stages, forward 558 and 577, wgrad
  // added to fp32 1.00 and 1.07 ms).
  static constexpr int kPieceBytes = 64;
  static constexpr int kStages = kCtas == 2 ? 6 : 3;
  static constexpr int kStoreOffset = kStages * kStageBytes;   // per epilogue warp: 32 rows of a piece
  static constexpr int kBarOffset = kStoreOffset + kEpiWarps * 32 * kPieceBytes;
  static constexpr int kNumBars = 4 * kStages + 2 * kAcc + 1;
  static constexpr int kMiscOffset = kBarOffset + kNumBars * 8;          // tmem slot, abort flag
  static constexpr int kTableOffset = (kMiscOffset + 8 + 15) / 16 * 16;  // prefix [E+1], start, end [E]
  static constexpr int smem_bytes(int E) { return 1024 + kTableOffset + (3 * E + 1) * 4; }
  static_assert(1024 + kTableOffset + (3 * kMaxE + 1) * 4 <= 227 * 1024, "shared memory");
};

struct Params {
  const int32_t* start;
  const int32_t* psum;
  int E, N, Kd;          // weights [E, N, Kd]
  int64_t M_cap;
  void* out;             // forward [M_cap, ld_out = N..], dgrad [M_cap, Kd..], wgrad [E, N, Kd]
  int64_t ld_out;
  int wide;              // rows of out begin on 32-byte boundaries
  int splits;            // CTAs of a cluster that share a tile's contraction (single-CTA wgrad)
  int32_t* status;
};

// Arrive once on `bar` (kCtas = 2: on the barrier at this place in both CTAs)
// when the MMAs issued so far have completed.
template <int kCtas>
MOE_DEV void tc_commit_all(uint64_t* bar) {
  if constexpr (kCtas == 1)
    tc_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
template <int kCtas>
MOE_DEV void tc_commit_own(uint64_t* bar) {
  if constexpr (kCtas == 1)
    tc_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

template <int kCtas>
MOE_DEV void tmem_alloc_n(uint32_t* slot, uint32_t ncols) {
  if constexpr (kCtas == 1) {
    tmem_alloc(slot, ncols);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(slot)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int kCtas>
MOE_DEV void tmem_dealloc_n(uint32_t taddr, uint32_t ncols) {
  __syncwarp();   // lane 0 comes from a role of its own
  if constexpr (kCtas == 1)
    tmem_dealloc(taddr, ncols);
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

MOE_DEV uint32_t leader_smem(const void* p) { return cta_smem(p, 0); }
// Arrive on a barrier of the pair's first CTA. The relaxed form is for a
// thread whose only business with the waiter is TMEM it has read (the loads
// are complete after tcgen05.wait::ld): a release would first wait for the
// thread's global stores to be visible, which has nothing to do with it.
MOE_DEV void mbar_arrive_leader(uint64_t* bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_smem(bar))
               : "memory");
}
MOE_DEV void mbar_arrive_leader_relaxed(uint64_t* bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(leader_smem(bar))
               : "memory");
}
// mbar_wait for a barrier that threads of the other CTA arrive on after
// writing shared memory of their own that this thread's MMAs read.
MOE_DEV bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort, int32_t* status) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kWaitSleepNs)
        : "memory");
    if (ok) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort = 1;
      set_status(status, MOE_ERR_TIMEOUT);
      return false;
    }
  }
}

// TMA store (kAdd: addition in fp32, done by L2) of a staged piece of 32
// rows; places past the tensor are not written.
template <bool kAdd>
MOE_DEV void tma_store_3d(const CUtensorMap* tm, uint32_t src, int32_t x, int32_t y, int32_t z) {
  if constexpr (kAdd)
    asm volatile(
        "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::
            "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
            reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(src)
        : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// The staged pieces have been read (may be overwritten) / the stores are done.
MOE_DEV void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
MOE_DEV void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// A 32-byte sector of a row of D that has `left` more values (a multiple of 8
// 16-bit values or of 8 fp32 ones; <= 0: none), `per` values a sector. wide:
// rows begin on 32-byte boundaries, so a thread moves a whole sector at once.
MOE_DEV void store_sector(uint8_t* a, const uint32_t* v, int left, int per, int wide) {
  if (left >= per && wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    if (left > 0) *reinterpret_cast<uint4*>(a) = make_uint4(v[0], v[1], v[2], v[3]);
    if (left >= per) *reinterpret_cast<uint4*>(a + 16) = make_uint4(v[4], v[5], v[6], v[7]);
  }
}
MOE_DEV void load_sector(const uint8_t* a, uint32_t* v, int left, int per, int wide) {
  if (left >= per && wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                   "=r"(v[6]), "=r"(v[7])
                 : "l"(a)
                 : "memory");
  } else {
    if (left > 0) {
      const uint4 x = *reinterpret_cast<const uint4*>(a);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    }
    if (left >= per) {
      const uint4 x = *reinterpret_cast<const uint4*>(a + 16);
      v[4] = x.x; v[5] = x.y; v[6] = x.z; v[7] = x.w;
    }
  }
}

struct Tile {
  int e, i0, j0;   // expert; first row (forward, dgrad: within the segment) and column of D
  int row0, rows;  // the expert's segment
  bool light;      // a pair's tile with at most 128 rows, 64 of them per CTA
};

// Out16: D is stored in the operands' type, else (wgrad) in fp32. Add: D is
// added to what `out` holds.
template <int kMode, bool Half, bool Out16, bool Add, int kCtas>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_mm16_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmD, const Params p) {
  using C = Cfg<kCtas>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  // the same offset in both CTAs of a pair: their windows begin alike
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOffset);
  uint64_t* empty = full + kStages;
  // wgrad, a tile's ragged block: it has landed in this CTA; its ragged rows
  // are zero in every CTA of the tile
  uint64_t* rlanded = empty + kStages;
  uint64_t* rzeroed = rlanded + kStages;
  uint64_t* tfull = rzeroed + kStages;
  uint64_t* tempty = tfull + kAcc;
  uint64_t* mma_done = tempty + kAcc;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMiscOffset);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMiscOffset + 4);
  int* s_tp = reinterpret_cast<int*>(smem + C::kTableOffset);
  int* s_start = s_tp + p.E + 1;
  int* s_end = s_start + p.E;
  __shared__ int s_warp_sum[kThreads / 32];

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = kCtas == 1 ? 0 : static_cast<int>(blockIdx.x % kCtas);   // in the pair

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&rlanded[s], 1);
      mbar_init(&rzeroed[s], kCtas);
    }
    for (int b = 0; b < kAcc; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kCtas * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&tmA);
    prefetch_tmap(&tmB);
    prefetch_tmap(&tmD);
  }
  if (warp == 1) tmem_alloc_n<kCtas>(tmem_slot, kTmemCols);
  // Segments, clamped into the buffer, and (forward, dgrad) the prefix of
  // their row tiles: thread t owns experts kPer t .. kPer t + kPer - 1.
  {
    constexpr int kPer = (kMaxE + kThreads - 1) / kThreads;
    int mine = 0, cnt[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = threadIdx.x * kPer + j;
      cnt[j] = 0;
      if (e < p.E) {
        const int cap = static_cast<int>(p.M_cap);
        const int a = min(max(p.start[e], 0), cap);
        const int b = min(max(p.psum[e], a), cap);
        s_start[e] = a;
        s_end[e] = b;
        cnt[j] = (b - a + C::BM - 1) / C::BM;
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
    for (int j = 0; j < kPer; ++j) {
      const int e = threadIdx.x * kPer + j;
      if (e < p.E) {
        s_tp[e] = base;
        base += cnt[j];
        if (e == p.E - 1) s_tp[p.E] = base;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (kCtas > 1) cluster_sync();   // the other CTA's barriers exist, its TMEM too
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // D's columns, its column tiles and (wgrad) row tiles
  const int cols = kMode == kForward ? p.N : p.Kd;
  const int nj = (cols + BN - 1) / BN;
  const int ni_w = (p.N + C::BM - 1) / C::BM;
  const int num_tiles = kMode == kWgrad ? p.E * ni_w * nj : s_tp[p.E] * nj;
  constexpr bool kCanSplit = kMode == kWgrad && kCtas == 1;
  const int splits = kCanSplit ? p.splits : 1;
  const int split = kCanSplit ? static_cast<int>(blockIdx.x) % splits : 0;
  const int first_tile = blockIdx.x / (kCtas * splits), tile_step = gridDim.x / (kCtas * splits);

  constexpr int kRaster = raster(kMode);
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
    t.i0 = (g * kRaster + in % gi) * C::BM;
    t.j0 = (in / gi) * BN;
    t.row0 = s_start[t.e];
    t.rows = s_end[t.e] - t.row0;
    t.light = kCtas == 2 && kMode != kWgrad && t.rows - t.i0 <= BMC;
    return t;
  };
  // blocks of BC along the contracted axis
  const int blocks_fd = ((kMode == kForward ? p.Kd : p.N) + BC - 1) / BC;
  auto num_blocks = [&](const Tile& t) { return kMode == kWgrad ? (t.rows + BC - 1) / BC : blocks_fd; };
  // this CTA's share of them: [first_block, end_block)
  auto first_block = [&](const Tile& t) { return kCanSplit ? num_blocks(t) * split / splits : 0; };
  auto end_block = [&](const Tile& t) {
    return kCanSplit ? num_blocks(t) * (split + 1) / splits : num_blocks(t);
  };
  // wgrad: blocks of a chunk, chunks being as equal as they can be
  constexpr int kMaxChunk = max_chunk(Out16);
  auto chunk_blocks = [&](int nb) {
    const int chunks = (nb + kMaxChunk - 1) / kMaxChunk;
    return (nb + chunks - 1) / chunks;
  };
  // wgrad: rows of the ragged block (the tile's first), 0 if all are whole
  auto ragged = [&](const Tile& t) { return kMode == kWgrad ? t.rows % BC : 0; };

  if (warp < 4) {
    if constexpr (kMode == kWgrad) regs_release<kRegsLow>();
    if (warp == 0 && lane == 0) {
      // ------------------------------------------------------------ producer
      // Both CTAs' bytes are counted on the first CTA's barrier, those of a
      // ragged block on each CTA's own, for the warp that zeroes rows there.
      constexpr int kGroup = kCtas;
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        const Tile t = tile_at(tile);
        const int nb = end_block(t);
        const int rag = ragged(t);
        const int i0 = t.i0 + rank * (t.light ? BMC / 2 : BMC), j0 = t.j0 + rank * C::kBRows;
        for (int b = first_block(t); b < nb; ++b) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          uint8_t* sa = smem + stage * C::kStageBytes;
          uint8_t* sb = sa + C::kABytes;
          uint32_t bar;
          if (kMode == kWgrad && rag && b == 0) {
            mbar_arrive_expect_tx(&rlanded[stage], C::kStageBytes);
            bar = kCtas == 1 ? smem_u32(&rlanded[stage]) : cta_smem(&rlanded[stage], rank);
          } else {
            if (rank == 0) mbar_arrive_expect_tx(&full[stage], kCtas * C::kStageBytes);
            bar = kCtas == 1 ? smem_u32(&full[stage]) : cta_smem(&full[stage], 0);
          }
          if (kMode == kForward) {
            load_2d<kGroup>(sa, &tmA, b * BC, t.row0 + i0, bar);
            load_3d<kGroup>(sb, &tmB, b * BC, j0, t.e, bar);
          } else if (kMode == kDgrad) {
            load_2d<kGroup>(sa, &tmA, b * BC, t.row0 + i0, bar);
#pragma unroll
            for (int q = 0; q < C::kBRows / 64; ++q)
              load_3d<kGroup>(sb + q * kPanel, &tmB, j0 + q * 64, b * BC, t.e, bar);
          } else {
            // the ragged block first: it is the segment's last
            const int c = rag ? (b == 0 ? t.rows - rag : (b - 1) * BC) : b * BC;
#pragma unroll
            for (int q = 0; q < BMC / 64; ++q)
              load_2d<kGroup>(sa + q * kPanel, &tmA, i0 + q * 64, t.row0 + c, bar);
#pragma unroll
            for (int q = 0; q < C::kBRows / 64; ++q)
              load_2d<kGroup>(sb + q * kPanel, &tmB, j0 + q * 64, t.row0 + c, bar);
          }
          if (++stage == kStages) { stage = 0; phase ^= 1u; }
        }
      }
      // Every load has landed before the CTA can exit: the tensor core has
      // consumed (released) each stage once more. After a wait that gave up,
      // this one is bounded too.
      for (int i = 0; i < kStages; ++i) {
        if (!drain_wait(&empty[stage], phase ^ 1u)) break;
        if (++stage == kStages) { stage = 0; phase ^= 1u; }
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ------------------------------------------------------------ MMA issuer
      constexpr uint32_t idesc_whole = idesc_f16(Half, kMode == kWgrad, kMode != kForward, C::BM, BN);
      constexpr uint32_t idesc_light = idesc_f16(Half, kMode == kWgrad, kMode != kForward, BMC, BN);
      int stage = 0, acc = 0;
      uint32_t acc_phase = 0;
      uint32_t full_phase = 0, rag_phase = 0;   // a bit per stage: uses so far
      bool ok = true;
      const uint32_t ring = smem_u32(smem);
      const uint64_t desc_a = kMode == kWgrad ? sw128_mnmajor_desc(ring) : sw128_kmajor_desc(ring);
      const uint64_t desc_b = kMode != kForward ? sw128_mnmajor_desc(ring + C::kABytes)
                                                : sw128_kmajor_desc(ring + C::kABytes);
      for (int tile = first_tile; tile < num_tiles && ok; tile += tile_step) {
        const Tile t = tile_at(tile);
        const int bf = first_block(t), nb = end_block(t);
        if (nb == bf) continue;   // wgrad of an expert without rows: the epilogue stores zeros
        const int rag = ragged(t);
        const uint32_t idesc = t.light ? idesc_light : idesc_whole;
        const int chunk = kMode == kWgrad ? chunk_blocks(nb - bf) : nb;
        for (int b0 = bf; b0 < nb && ok; b0 += chunk) {
          if (!mbar_wait(&tempty[acc], acc_phase ^ 1u, abort_flag, p.status)) { ok = false; break; }
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * BN);
          const int b1 = min(b0 + chunk, nb);
          for (int b = b0; b < b1; ++b) {
            const bool ragged_block = kMode == kWgrad && rag && b == 0;
            if (ragged_block) {
              ok = kCtas > 1 ? mbar_wait_cluster(&rzeroed[stage], (rag_phase >> stage) & 1u, abort_flag, p.status)
                             : mbar_wait(&rzeroed[stage], (rag_phase >> stage) & 1u, abort_flag, p.status);
              rag_phase ^= 1u << stage;
            } else {
              ok = mbar_wait(&full[stage], (full_phase >> stage) & 1u, abort_flag, p.status);
              full_phase ^= 1u << stage;
            }
            if (!ok) break;
            tc_fence_after();
            // the descriptors' addresses are in 16-byte units; 16 contracted
            // values on are 32 bytes along a c-contiguous row, 16 rows of 128
            // bytes otherwise
            const uint32_t at = static_cast<uint32_t>(stage * (C::kStageBytes >> 4));
            const uint64_t da0 = desc_a + at, db0 = desc_b + at;
            auto step = [&](int k) {
              constexpr int kAlong = kUmmaK * 2 / 16, kAcross = kUmmaK * 128 / 16;
              tc_mma_f16<kCtas>(d, da0 + k * (kMode == kWgrad ? kAcross : kAlong),
                                db0 + k * (kMode != kForward ? kAcross : kAlong), idesc,
                                (b > b0 || k > 0) ? 1u : 0u);
            };
            if (ragged_block) {
              for (int k = 0; k < (rag + kUmmaK - 1) / kUmmaK; ++k) step(k);
            } else {
#pragma unroll
              for (int k = 0; k < BC / kUmmaK; ++k) step(k);
            }
            tc_commit_all<kCtas>(&empty[stage]);
            if (++stage == kStages) stage = 0;
          }
          if (!ok) break;
          tc_commit_all<kCtas>(&tfull[acc]);
          if (++acc == kAcc) { acc = 0; acc_phase ^= 1u; }
        }
      }
      // Every MMA issued so far must complete before TMEM is released.
      tc_commit_own<kCtas>(mma_done);
      drain_wait(mma_done, 0);
    } else if (warp == 2 && kMode == kWgrad) {
      // ------------------------------------------------- ragged rows to zero
      // Only the rows up to the next multiple of 16 are read by the tensor core.
      int stage = 0;
      uint32_t uses = 0;   // a bit per stage
      for (int tile = first_tile; tile < num_tiles; tile += tile_step) {
        const Tile t = tile_at(tile);
        const int rag = first_block(t) == 0 && end_block(t) > 0 ? ragged(t) : 0;
        if (rag) {
          if (!mbar_wait_warp(&rlanded[stage], (uses >> stage) & 1u, abort_flag, p.status)) break;
          uses ^= 1u << stage;
          const int r1 = (rag + kUmmaK - 1) / kUmmaK * kUmmaK;
          uint8_t* s = smem + stage * C::kStageBytes;
          const int per_panel = (r1 - rag) * 8;   // 16-byte vectors
          for (int q = 0; q < C::kStageBytes / kPanel; ++q)
            for (int v = lane; v < per_panel; v += 32)
              *reinterpret_cast<uint4*>(s + q * kPanel + rag * 128 + v * 16) = make_uint4(0, 0, 0, 0);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (kCtas == 1) mbar_arrive(&rzeroed[stage]); else mbar_arrive_leader(&rzeroed[stage]);
          }
        }
        stage = (stage + end_block(t) - first_block(t)) % kStages;
      }
    }
    if (kCanSplit && splits > 1) {   // the epilogue's two meetings
      cluster_sync();
      cluster_sync();
    }
  } else {
    if constexpr (kMode == kWgrad) regs_claim<kRegsHigh>();
    // ------------------------------------------------------------ epilogue
    // A thread owns one row of D (its TMEM lane) and 128 columns, in pieces of
    // 64 bytes. A warp whose 32 rows are all D's (always in wgrad; in forward and
    // dgrad all but a segment's last) stages a piece in shared memory
    // (swizzled: no bank conflicts) and one TMA store takes it out; fp32
    // results that are added to `out` are added by that store, in L2. The
    // other rows go straight from registers, a 32-byte sector per thread, as
    // do 16-bit results that are added to, whose sum is rounded once: their
    // old values are asked for kAhead pieces early. Stores from registers alone
    // slowed the products: with 1024 rows an expert and 4096 x 4096 weights wgrad
    // took 930 cycles a block of 64 rows with them, 738 with TMA stores, 750 with
    // no stores at all.
    const int quarter = warp & 3;
    const int half_cols = ((warp - 4) >> 2) * (BN / 2);
    constexpr int kElem = Out16 ? 2 : 4;
    constexpr bool kAddHere = Add && Out16;     // added in registers
    constexpr bool kTma = !kAddHere;
    constexpr int kPiece = C::kPieceBytes;
    constexpr int kWords = kPiece / 4;
    constexpr int kCols = kPiece / kElem;       // columns of D per piece: 32 or 16
    constexpr int kPieces = BN / 2 / kCols;
    const uint32_t stg = smem_u32(smem + C::kStoreOffset + (warp - 4) * 32 * kPiece);
    constexpr int kAhead = kAddHere ? 2 : 1;
    constexpr int kSector = 32 / kElem;         // columns of a 32-byte sector
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int tile = first_tile; tile < num_tiles; tile += tile_step) {
      const Tile t = tile_at(tile);
      if (Add && num_blocks(t) == 0) continue;   // an expert without rows adds nothing
      const int ilim = kMode == kWgrad ? p.N : t.rows;                // rows of D that exist
      // this warp's first row and column of D, and of the accumulator; a light
      // tile's 64 rows lie in lanes 0-63 with D's columns 0-127 and in lanes
      // 64-127 with its columns 128-255, in accumulator columns 0-127
      const int iw = t.i0 + (t.light ? rank * (BMC / 2) + (quarter & 1) * 32 : rank * BMC + quarter * 32);
      const int acol = t.light ? half_cols / 2 : half_cols;
      const int j = t.j0 + (t.light ? (quarter >> 1) * (BN / 2) : 0) + acol;
      const int pieces = t.light ? kPieces / 2 : kPieces;
      const bool by_tma = kTma && (kMode == kWgrad || iw + 32 <= ilim);
      const int64_t orow = (kMode == kWgrad ? static_cast<int64_t>(t.e) * p.N : t.row0) + iw + lane;
      uint8_t* out = static_cast<uint8_t*>(p.out) + (orow * p.ld_out + j) * kElem;
      const int ncols = iw + lane < ilim ? cols - j : 0;              // columns to store from j on
      uint32_t old[kAhead][kWords];
      auto fetch = [&](int piece, uint32_t (&o)[kWords]) {
#pragma unroll
        for (int q = 0; q < kWords / 8; ++q)
          load_sector(out + piece * kPiece + q * 32, &o[q * 8], ncols - piece * kCols - q * kSector,
                      kSector, p.wide);
      };
      auto accumulator = [&]() {
        return tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
               static_cast<uint32_t>(acc * BN + acol);
      };
      auto release = [&]() {   // its last read has landed
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kCtas == 1) mbar_arrive(&tempty[acc]); else mbar_arrive_leader_relaxed(&tempty[acc]);
        }
        if (++acc == kAcc) { acc = 0; acc_phase ^= 1u; }
      };
      // wgrad: the thread's 128 results, the tile's chunks added up
      float sum[kMode == kWgrad ? BN / 2 : 1];
      uint32_t tq = 0;
      bool ok = true;
      if constexpr (kMode == kWgrad) {
        const int nb = end_block(t) - first_block(t);
        const int chunk = nb > 0 ? chunk_blocks(nb) : 1;
        if (nb == 0) {
#pragma unroll
          for (int k = 0; k < BN / 2; ++k) sum[k] = 0.0f;
        } else {
          ok = mbar_wait_warp(&tfull[acc], acc_phase, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = accumulator();
#pragma unroll
          for (int q = 0; q < BN / 32; ++q) {
            uint32_t a[16];
            tc_ld16_wait(ta + q * 16, a);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[q * 16 + k] = __uint_as_float(a[k]);
          }
          release();
        }
#pragma unroll 1
        for (int c = chunk; c < nb; c += chunk) {
          ok = mbar_wait_warp(&tfull[acc], acc_phase, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t ta = accumulator();
#pragma unroll
          for (int q = 0; q < BN / 32; ++q) {
            uint32_t a[16];
            tc_ld16_wait(ta + q * 16, a);
#pragma unroll
            for (int k = 0; k < 16; ++k) sum[q * 16 + k] += __uint_as_float(a[k]);
          }
          release();
        }
      } else {
        ok = mbar_wait_warp(&tfull[acc], acc_phase, abort_flag, p.status);
        tc_fence_after();
        tq = accumulator();
      }
      if (!ok) break;
      if constexpr (kCanSplit) {
        if (splits > 1) {
          // The ring is free: every MMA of this CTA, its only tile's, is done.
          float* part = reinterpret_cast<float*>(smem) + half_cols * BMC + quarter * 32 + lane;
#pragma unroll
          for (int k = 0; k < BN / 2; ++k) part[k * BMC] = sum[k];   // [column][row]
          break;
        }
      }
      if constexpr (kAddHere) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) fetch(a, old[a]);
      }
#pragma unroll
      for (int piece = 0; piece < kPieces; ++piece) {
        if (kCtas == 2 && kMode != kWgrad && piece >= pieces) break;
        uint32_t w[kWords];   // the thread's row of the piece
        float f[kCols];
        if constexpr (kMode == kWgrad) {
#pragma unroll
          for (int k = 0; k < kCols; ++k) f[k] = sum[piece * kCols + k];
        } else {
          uint32_t a[32];
          __syncwarp();   // the stores of the piece before differ from lane to lane
          tc_ld32_wait(tq + piece * kCols, a);
#pragma unroll
          for (int k = 0; k < kCols; ++k) f[k] = __uint_as_float(a[k]);
          if (piece == pieces - 1) release();
        }
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          if constexpr (Out16) {
            float x = f[2 * k], y = f[2 * k + 1];
            if constexpr (kAddHere) {
              const float2 was = unpack2<Half>(old[piece % kAhead][k]);
              x += was.x;
              y += was.y;
            }
            w[k] = pack2<Half>(x, y);
          } else {
            w[k] = __float_as_uint(f[k]);
          }
        }
        if (by_tma) {
          if (j + piece * kCols >= cols || iw >= ilim) continue;   // the same for the whole warp
          if (lane == 0) tma_store_read();   // the warp's last piece has left the buffer
          __syncwarp();
#pragma unroll
          for (int c = 0; c < kPiece / 16; ++c)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             stg + lane * kPiece +
                             ((c ^ ((lane >> 1) & 3)) << 4)),
                         "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                         : "memory");
          fence_async_smem();
          __syncwarp();
          if (lane == 0)
            tma_store_3d<Add>(&tmD, stg, j + piece * kCols, kMode == kWgrad ? iw : t.row0 + iw,
                              kMode == kWgrad ? t.e : 0);
        } else {
#pragma unroll
          for (int q = 0; q < kWords / 8; ++q)
            store_sector(out + piece * kPiece + q * 32, &w[q * 8], ncols - piece * kCols - q * kSector,
                         kSector, p.wide);
          if constexpr (kAddHere)
            if (piece + kAhead < kPieces) fetch(piece + kAhead, old[piece % kAhead]);
        }
      }
    }
    if (kTma && lane == 0) tma_store_done();
    if constexpr (kCanSplit) {
      if (splits > 1) {
        // The partial sums of the cluster's CTAs, each CTA for its share of the
        // columns, always in the same order. A lane takes four rows, so that a
        // warp reads the 512 bytes of a column at once (distributed shared
        // memory is slow where a warp's accesses are scattered: lanes that read
        // 16 bytes of a row each made this step three times as long).
        cluster_sync();
        const Tile t = tile_at(first_tile);
        const int i = t.i0 + lane * 4;
        const int cw = BN / kEpiWarps / splits;   // columns of a warp: 16, 8 or 4
        const int c0 = (split * kEpiWarps + (warp - 4)) * cw;
        const bool skip = (Add && num_blocks(t) == 0) || *abort_flag;
        for (int c = c0; c < c0 + cw && !skip; c += 4) {
          float f[4][4] = {};   // [row][column]
          for (int s = 0; s < splits; ++s) {
            const uint32_t from = cta_smem(smem, s) + static_cast<uint32_t>((c * BMC + lane * 4) * 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float4 x;
              asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                           : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                           : "r"(from + k * BMC * 4));
              f[0][k] += x.x;
              f[1][k] += x.y;
              f[2][k] += x.z;
              f[3][k] += x.w;
            }
          }
          if (t.j0 + c >= cols) continue;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            if (i + r >= p.N) break;
            uint8_t* out = static_cast<uint8_t*>(p.out) +
                           ((static_cast<int64_t>(t.e) * p.N + i + r) * p.ld_out + t.j0 + c) * kElem;
            if constexpr (Out16) {
              if (Add) {
                const uint2 o = *reinterpret_cast<const uint2*>(out);
                const float2 lo = unpack2<Half>(o.x), hi = unpack2<Half>(o.y);
                f[r][0] += lo.x; f[r][1] += lo.y; f[r][2] += hi.x; f[r][3] += hi.y;
              }
              *reinterpret_cast<uint2*>(out) =
                  make_uint2(pack2<Half>(f[r][0], f[r][1]), pack2<Half>(f[r][2], f[r][3]));
            } else {
              if (Add) {
                const float4 o = *reinterpret_cast<const float4*>(out);
                f[r][0] += o.x; f[r][1] += o.y; f[r][2] += o.z; f[r][3] += o.w;
              }
              *reinterpret_cast<float4*>(out) = make_float4(f[r][0], f[r][1], f[r][2], f[r][3]);
            }
          }
        }
        cluster_sync();   // no CTA leaves while its partial sums are read
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (kCtas > 1) cluster_sync();   // neither CTA leaves, or frees TMEM, under the other's work
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_n<kCtas>(tmem_base, kTmemCols);
  }
}

// Clusters of `size` CTAs of the kernel that the current device runs at one time
// (a GPC's SMs need not be a multiple of it), found once per device, and the
// kernel's shared memory allowed. 0 on an error (message set).
template <int kMode, bool Half, bool Out16, bool Add, int kCtas>
int resident_clusters(int size) {
  using C = Cfg<kCtas>;
  auto* kernel = grouped_mm16_kernel<kMode, Half, Out16, Add, kCtas>;
  static std::atomic<int> found[64][4];   // size 1, 2, 4, 8
  const int slot = size == 1 ? 0 : (size == 2 ? 1 : (size == 4 ? 2 : 3));
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  int n = found[dev][slot].load();
  if (n != 0) return n;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::smem_bytes(kMaxE)) != cudaSuccess) {
    check_launch("cudaFuncSetAttribute(grouped_mm16_kernel)");
    return 0;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(device_sm_count() / size * size));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::smem_bytes(kMaxE);
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(size);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    check_launch("cudaOccupancyMaxActiveClusters(grouped_mm16_kernel)");
    return 0;
  }
  if (n < 1) n = 1;
  found[dev][slot].store(n);
  return n;
}

template <int kMode, bool Half, bool Out16, bool Add, int kCtas>
int launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td, const Params& p,
           int64_t max_tiles, cudaStream_t s) {
  using C = Cfg<kCtas>;
  auto* kernel = grouped_mm16_kernel<kMode, Half, Out16, Add, kCtas>;
  const int cluster = kCtas * p.splits;
  const int n = resident_clusters<kMode, Half, Out16, Add, kCtas>(cluster);
  if (n == 0) return MOE_ERR_CUDA;
  // a split tile's cluster does that tile only
  const int64_t grid = p.splits > 1 || max_tiles < n ? max_tiles : n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::smem_bytes(p.E);
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(cluster);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, ta, tb, td, p);
  return check_launch("grouped_mm16_kernel");
}

int check_sizes(const char* what, int dtype, int E, int N, int Kd, int64_t M_cap) {
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "%s: dtype must be MOE_BF16 or MOE_F16", what);
  MOE_REQUIRE(E > 0 && E <= kMaxE, "%s: E must be in [1, 1024]", what);
  MOE_REQUIRE(N > 0 && N % 8 == 0 && Kd > 0 && Kd % 8 == 0,
              "%s: N and Kd must be positive multiples of 8", what);
  MOE_REQUIRE(M_cap >= 0 && M_cap <= INT32_MAX - 256, "%s: bad M_cap", what);
  // linear tile ids are 32-bit
  const int64_t nj = (N > Kd ? N : Kd) / BN + 1;
  MOE_REQUIRE((M_cap / BMC + E) * nj <= INT32_MAX && static_cast<int64_t>(E) * (N / BMC + 1) * nj <= INT32_MAX,
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

// Rows per expert, on average, up to which the few-rows form is taken. With 24
// rows it takes 171 us and the pairs 176 (32 experts of 4096 x 4096, forward;
// dgrad 166 and 166), with 48 rows 183 and 178 (180 and 169); with 32 rows of
// 64 experts of 4096 x 7168 it takes 551 and the pairs 587. The rows may all be
// one expert's: 160 experts of 2048 x 4096, 6080 rows, 1400 of them with one, take
// 427 us (dgrad 430), the weights alone 400 at HBM's rate.
constexpr int kFewRows = 40;

// Forward and dgrad: rows [M_cap, in] times weights -> rows [M_cap, out].
int rows_times_weights(const char* what, bool dgrad, const void* a, int64_t ld_a, const void* w,
                       const int32_t* start, const int32_t* psum, int dtype, int E, int N, int Kd,
                       int64_t M_cap, int64_t max_rows, void* out, int64_t ld_out, int32_t* d_status,
                       cudaStream_t s) {
  MOE_TRY(check_sizes(what, dtype, E, N, Kd, M_cap));
  const int in = dgrad ? N : Kd, width = dgrad ? Kd : N;
  MOE_REQUIRE(max_rows >= 0 && max_rows <= M_cap, "%s: max_rows must be in [0, M_cap]", what);
  if (M_cap > 0) {
    MOE_REQUIRE(start && psum, "%s: null segments", what);
    MOE_TRY(check_rows(what, dgrad ? "dy" : "x", a, ld_a, in));
    MOE_TRY(check_rows(what, "w", w, Kd, Kd));
    MOE_TRY(check_rows(what, dgrad ? "dx" : "out", out, ld_out, width));
  }
  MOE_REQUIRE_DEVICE();
  if (max_rows == 0) return MOE_OK;
  const bool half = dtype == MOE_F16;
  if (max_rows <= static_cast<int64_t>(E) * kFewRows)
    return launch_grouped_mm16_few(dgrad, half, a, ld_a, w, start, psum, E, N, Kd, M_cap, max_rows,
                                   static_cast<uint16_t*>(out), ld_out, d_status, s);
  CUtensorMap ta, tb, td;
  MOE_TRY(make_tmap_rows16(&ta, a, in, M_cap, ld_a, BMC));
  MOE_TRY(make_tmap_weights16(&tb, w, Kd, N, E, dgrad ? 64 : BN / 2));
  MOE_TRY(make_tmap_result(&td, out, false, width, M_cap, 1, ld_out));
  Params p;
  p.start = start;
  p.psum = psum;
  p.E = E;
  p.N = N;
  p.Kd = Kd;
  p.M_cap = M_cap;
  p.out = out;
  p.ld_out = ld_out;
  p.wide = aligned(out, 32) && ld_out % 16 == 0;
  p.splits = 1;
  p.status = d_status;
  const int64_t m_tiles = max_rows / (2 * BMC) + std::min<int64_t>(E, max_rows);
  const int64_t tiles = m_tiles * ((width + BN - 1) / BN);
  if (dgrad)
    return half ? launch<kDgrad, true, true, false, 2>(ta, tb, td, p, tiles, s)
                : launch<kDgrad, false, true, false, 2>(ta, tb, td, p, tiles, s);
  return half ? launch<kForward, true, true, false, 2>(ta, tb, td, p, tiles, s)
              : launch<kForward, false, true, false, 2>(ta, tb, td, p, tiles, s);
}

template <bool Half, int kCtas>
int launch_wgrad(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& td, const Params& p,
                 bool out16, bool add, cudaStream_t s) {
  const int64_t tiles = static_cast<int64_t>(p.E) * ((p.N + kCtas * BMC - 1) / (kCtas * BMC)) *
                        ((p.Kd + BN - 1) / BN);
  if (out16)
    return add ? launch<kWgrad, Half, true, true, kCtas>(ta, tb, td, p, tiles, s)
               : launch<kWgrad, Half, true, false, kCtas>(ta, tb, td, p, tiles, s);
  return add ? launch<kWgrad, Half, false, true, kCtas>(ta, tb, td, p, tiles, s)
             : launch<kWgrad, Half, false, false, kCtas>(ta, tb, td, p, tiles, s);
}

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_mm(const void* x, int64_t ld_x, const void* w, const int32_t* start,
                              const int32_t* psum, int dtype, int E, int N, int Kd, int64_t M_cap,
                              int64_t max_rows, void* out, int64_t ld_out, int32_t* d_status,
                              moe_stream_t stream) {
  return moe::rows_times_weights("moe_grouped_mm", false, x, ld_x, w, start, psum, dtype, E, N, Kd,
                                 M_cap, max_rows, out, ld_out, d_status, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" int moe_grouped_mm_dgrad(const void* dy, int64_t ld_dy, const void* w,
                                    const int32_t* start, const int32_t* psum, int dtype, int E,
                                    int N, int Kd, int64_t M_cap, int64_t max_rows, void* dx,
                                    int64_t ld_dx, int32_t* d_status, moe_stream_t stream) {
  return moe::rows_times_weights("moe_grouped_mm_dgrad", true, dy, ld_dy, w, start, psum, dtype, E, N,
                                 Kd, M_cap, max_rows, dx, ld_dx, d_status, reinterpret_cast<cudaStream_t>(stream));
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
  CUtensorMap ta, tb, td;
  MOE_TRY(make_tmap_result(&td, dw, out_dtype == MOE_F32, Kd, N, E, Kd));
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
  p.wide = aligned(dw, 32) && (Kd % 16 == 0 || out_dtype == MOE_F32);
  p.status = d_status;
  const bool out16 = out_dtype != MOE_F32, add = accumulate != 0;
  // One CTA a tile where a pair's second one would have no rows of D (128 rows
  // for each of 32 experts, N = 64, Kd = 4096 take 11.2 us, by pairs 16.9), and
  // where there are so few such tiles that the rows can be shared by the CTAs of
  // a cluster: all clusters run at once, each CTA has 12 blocks on average. One
  // expert of 512 x 512 and 32768 rows takes 41 us in eight parts, 176 whole;
  // eight of 4096 rows 28.7 in two, 29.7 whole; with 8 blocks a CTA (eight of 1024
  // rows) parts cost 16.4 instead of 14.3; 16 tiles in eight parts, of which 15
  // clusters run at once, 36 instead of 25 in four.
  const int64_t tiles = static_cast<int64_t>(E) * ((N + BMC - 1) / BMC) * ((Kd + BN - 1) / BN);
  const int64_t blocks = (M_cap / E + BC - 1) / BC;
  p.splits = 1;
  for (int k = 8; k > 1 && p.splits == 1; k /= 2)
    if (blocks / k >= 12 && tiles <= resident_clusters<kWgrad, false, true, false, 1>(k)) p.splits = k;
  if (N > BMC && p.splits == 1)
    return dtype == MOE_F16 ? launch_wgrad<true, 2>(ta, tb, td, p, out16, add, s)
                            : launch_wgrad<false, 2>(ta, tb, td, p, out16, add, s);
  return dtype == MOE_F16 ? launch_wgrad<true, 1>(ta, tb, td, p, out16, add, s)
                          : launch_wgrad<false, 1>(ta, tb, td, p, out16, add, s);
}

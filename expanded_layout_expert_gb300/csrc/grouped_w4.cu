// moe_grouped_mm_w4: the experts' product over 4-bit weights with group scales,
//   out[r, n] = sum_k x[r, k] s[e, n, k / g] (q[e, n, k] - z[e, n, k / g]),
// for batches of single tokens, where the time is that of reading the weights.
// This is the form for more than a few rows an expert; grouped_w4_few.cu has
// the other, and the end of this file the choice.
//
// The weights are the tensor core's first operand, read from tensor memory:
//   D[i, r] = sum_c W[i, c] X[r, c],
// a tile being 256 weight rows, 128 to each of two warpgroups, by kR activation
// rows (16 to 64) of one expert. TMA brings 128 contracted values at a time, 64
// bytes of codes a weight row and the rows of x; a thread takes one weight row,
// makes its codes 16-bit values (w4.cuh: exact) and stores them into its lane of
// tensor memory. Each scale group has sums of its own there, which the thread
// multiplies by its scale and adds up in fp32 registers. So nothing is rounded
// but the sums and, once, the result.
//
// Bound: no single unit (issue slots are half used, HBM at 0.7 to 0.77 of a copy's rate).
// 64 experts of 4096 x 7168 take, with 32 and with 8 rows each, 218 us (4.7 TB/s; the
// bytes alone 152) and 194 us (5.1 TB/s; 147). With parts taken out for timing: the
// products 216 and 191, the sums 213 and 187, the making of the values 203 and 167, all
// three 203 and 169, the copies of x 213 and 191, those and the three 178 and 166, the
// stores to tensor memory as well 169 and 156. One stage of a tile's 56 alone, so the
// starts and ends of 1024 tiles in 3.4 rounds of 304, takes 30 and 26.
// So with few rows it is the making of the values, half of the 350 instructions that
// each of four warps has for 128 x 128 codes, in a chain from the sums to the values,
// the barrier and the products (the SM's four warpgroups cover for each other); with
// more rows x stands behind it, brought anew for every 256 weight rows; and the starts
// behind both.
// What got there, in us for 32 rows: one CTA of four dequantising warps, a TMA
// and an MMA warp, sums waited for at once 490; the next values made meanwhile
// 386; no warps of their own for the loads and products, which poll for their
// turn with half of all instructions, 374; the operands of those known to be
// uniform 300; 256 rows a CTA, so that four stages fit, 279; the warpgroups'
// barriers apart 249; the loop's arithmetic off the uniform pipe 245; sums first and
// then the values, in few registers, 243; the scales moved up between them 234;
// tiles of 48 rows for them instead of 64 224; no branch in front of a barrier's test 218.
// Eight warps for 128 rows, three CTAs, were slower (362), and so were sums fetched
// while the next values are made (267) and the contraction split in two for fuller
// waves (279).
//
// With few tiles the contraction is split over the CTAs of a cluster, whose
// partial sums meet in a fixed order through distributed shared memory.
#include <algorithm>
#include <atomic>

#include "dtype16.cuh"
#include "gemm_host.h"
#include "host_util.h"
#include "mm16.cuh"
#include "w4.cuh"

namespace moe {
namespace {

constexpr int kHalf = 128;               // weight rows of a warpgroup
constexpr int kI = 2 * kHalf;            // of a tile
constexpr int BC = 128;                  // contracted per stage
constexpr int kUmmaK = 16;
constexpr int kHalfBytes = kHalf * BC / 2;
constexpr int kCodeBytes = 2 * kHalfBytes;
constexpr int kThreads = 256;
constexpr int kHalfCols = 128;           // tensor memory: at most 64 of a step's weights, 64 of its sums
constexpr int kTmemCols = 2 * kHalfCols;

// Contracted values of a step, a batch of products: their sums, of every scale
// group apart, have 64 columns.
constexpr int step_k(int group, int R) { return 64 / R * group < 128 ? 64 / R * group : 128; }

constexpr int stage_bytes(int R) { return kCodeBytes + R * BC * 2; }
// What the ring takes is lost to L1, where the scales' sectors wait for their next
// use, so the more scales a row has, the fewer stages (64 experts of 4096 x 7168 with 20
// rows each take, with 4 and 3 stages, 203 and 208 us in groups of 128, 253 and 231
// in groups of 64, 401 and 278 in groups of 32; with 8 rows 194 and 200, 224 and 218, 246
// and 238). Tiles of 16 rows in groups of 64 keep four all the same, for short
// contractions: 64 experts of 2048 x 4096 73 and 74 us, without zero points 71 and 73, 16
// of 4096 x 4096 with 12 rows 46.9 and 47.6, 160 of 1536 x 5120 164 and 166. Two
// stages are too few, and for more than 32 rows two CTAs have no room for four.
constexpr int stages_for(int group, int R) { return R > 32 || group <= 2 * R ? 3 : 4; }
constexpr int ring_bytes(int group, int R) { return stages_for(group, R) * stage_bytes(R) + 1024; }
// Two CTAs an SM is the most, because tensor memory has room for no third: nothing
// counts its columns when a CTA is placed, and an allocation waits for them without
// a limit, for CTAs perhaps that wait for their cluster's others behind it. Shared memory is
// counted, so every CTA takes enough of the SM's 228 KB (1 KB of them its own
// overhead) that no third fits, nor one of the 16-bit product for few rows (97 KB and up
// to 128 columns) beside two. The other kernels with tensor memory take all registers. It
// costs tiles of 16 rows in groups of 32 some L1 (64 experts of 4096 x 7168, 8 rows
// each: 230 -> 236 us), the others nothing.
constexpr int kMinSmem = 77 * 1024;
constexpr int smem_bytes(int group, int R) {
  return ring_bytes(group, R) > kMinSmem ? ring_bytes(group, R) : kMinSmem;
}
static_assert(512 / kTmemCols == 2 && 3 * (kMinSmem + 1024) > 228 * 1024, "two CTAs an SM at most");

// A copy that is left out: that of stage `block` of CTA `cta`; and how long waits wait.
struct W4Drop {
  long long limit;
  int cta, block;
};

struct W4Params {
  const int32_t* start;
  const int32_t* psum;
  const uint2* scales;    // 4 to a vector
  const uint32_t* zeros;  // 4 to a word, or NULL
  int E, N;
  int blocks;             // stages along the contraction
  int groups;             // scales of a row
  int splits;             // CTAs of a cluster
  int code_rows;          // rows of codes that a copy brings: 256 or 128
  int64_t M_cap;
  uint16_t* out;
  int64_t ld_out;
  int32_t* status;
  W4Drop drop = {};       // read by the kernel that moe_selftest_w4_wait runs, alone
};

// D[tmem] (+)= A[tmem] * B[smem]^T, 16-bit operands, K = 16. B's descriptor comes
// in halves, of which only the low one moves: a 64-bit sum takes two steps.
template <bool kAdd>
MOE_DEV void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t b_high, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_low), "r"(b_high), "r"(idesc), "n"(kAdd ? 1 : 0)
      : "memory");
}

MOE_DEV void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
MOE_DEV void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A row's scales and zero points, four groups at a time, in registers: those
// four, and the aligned vectors that the next four lie in, asked for in advance.
// N being a multiple of 8, the tensors are whole vectors.
struct GroupStream {
  const uint2* scales;
  const uint32_t* zeros;
  int next, last;   // vectors of four, from the row's first one
  int skew;         // of the first group in its vector
  uint2 s0, s1;
  uint32_t z0, z1;
  uint32_t s[2], z;   // the four
  MOE_DEV void load(uint2& s, uint32_t& z) {
    s = __ldg(scales + min(next, last));
    if (zeros != nullptr) z = __ldg(zeros + min(next, last));
  }
  MOE_DEV void begin(const uint2* sc, const uint32_t* ze, int64_t first, int64_t values) {
    scales = sc + (first >> 2);
    zeros = ze != nullptr ? ze + (first >> 2) : nullptr;
    last = static_cast<int>(min(static_cast<int64_t>(INT32_MAX), values / 4 - 1 - (first >> 2)));
    skew = static_cast<int>(first) & 3;
    z = 0x01010101u * kW4Zero;
    next = 0;
    load(s0, z0);   // neither is waited for here
    next = 1;
    load(s1, z1);
  }
  MOE_DEV void refill() {
    const bool up = skew & 2;
    const uint32_t a = up ? s0.y : s0.x, b = up ? s1.x : s0.y, c = up ? s1.y : s1.x;
    s[0] = __funnelshift_r(a, b, 16 * (skew & 1));
    s[1] = __funnelshift_r(b, c, 16 * (skew & 1));
    if (zeros != nullptr) z = __funnelshift_r(z0, z1, 8 * skew);
    s0 = s1;
    z0 = z1;
    ++next;
    load(s1, z1);
  }
  template <int n>   // n of the four are used up: 1, 2 or 4
  MOE_DEV void pass() {
    s[0] = n == 1 ? __funnelshift_r(s[0], s[1], 16) : s[1];
    s[1] = n == 1 ? s[1] >> 16 : 0u;
    if (zeros != nullptr && n < 4) z >>= 8 * (n & 3);
  }
};

// A value that all lanes hold, so that the compiler knows it: tensor core and TMA
// instructions take their operands from uniform registers, and where it does not
// know that they are uniform it loops over the lanes.
MOE_DEV int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// mbar_wait_warp on a barrier given by its shared-memory address: forming the
// address anew at every wait costs as much as the wait.
MOE_DEV bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return __all_sync(0xffffffffu, ok != 0);
}

// The 128 threads of a warpgroup meet.
MOE_DEV void meet(int group) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(group + 1) : "memory");
}

// Arrive once on `bar` when every tcgen05 operation this thread issued before has
// completed.
MOE_DEV void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// True in one lane of a converged warp.
MOE_DEV bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// kDrop: one copy is left out (p.drop), so that the wait for it runs out.
template <bool Half, int kGroup, int kR, bool kDrop = false>
__global__ void __launch_bounds__(kThreads, 2)
    grouped_w4_kernel(const __grid_constant__ CUtensorMap tmW,
                      const __grid_constant__ CUtensorMap tmX, const W4Params p) {
  constexpr int kStages = stages_for(kGroup, kR);
  constexpr int kStageBytes = stage_bytes(kR);
  constexpr int kGroups = BC / kGroup;   // of a stage
  constexpr int kStep = step_k(kGroup, kR);
  constexpr int kSteps = BC / kStep;     // of a stage: 1 or 2
  constexpr int kEnds = kStep / kGroup;  // groups of a step
  constexpr int kACols = kStep / 2;
  constexpr int kChunks = kStep / 32;    // of 32 values, a 16-byte vector of codes
  static_assert(kEnds >= 1 && kACols + kEnds * kR <= kHalfCols, "tensor memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  // full[s]: the barrier of a place in the ring; full[kStages + s]: the stages up to the
  // last one asked for there, of this CTA's
  __shared__ uint64_t full[2 * kStages], d_ready[2], done[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_used[kStages];
  __shared__ int s_warp_sum[kThreads / 32], s_found[3];
  volatile int* abort_flag = &s_abort;
  const int warp = uniform(threadIdx.x >> 5);
  const int splits = p.splits;
  const int rank = static_cast<int>(blockIdx.x) % splits;
  const int tile = static_cast<int>(blockIdx.x) / splits;
  const int ni = (p.N + kI - 1) / kI;
  const int chunk = tile / ni;
  const int i0 = (tile - chunk * ni) * kI;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      s_used[s] = 0;
      full[kStages + s] = 0;
    }
    for (int h = 0; h < 2; ++h) {
      mbar_init(&d_ready[h], 1);
      mbar_init(&done[h], 1);
    }
    s_abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmW);
    prefetch_tmap(&tmX);
  }
  if (warp == 0) {
    __syncwarp();
    tmem_alloc(&s_tmem, kTmemCols);
    tmem_relinquish();
  }
  const int all = w4_find_chunk<kThreads, kR>(p.start, p.psum, p.E, p.M_cap, chunk, s_warp_sum, s_found);
  // more chunks than the grid has: the caller's bound on the rows was wrong
  if (blockIdx.x == 0 && threadIdx.x == kThreads - 1 &&
      static_cast<int64_t>(all) * ni * splits > static_cast<int64_t>(gridDim.x))
    set_status(p.status, MOE_ERR_DEVICE_CHECK);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int e = uniform(s_found[0]), row0 = uniform(s_found[1]), rows = uniform(s_found[2]);
  const uint32_t tmem = uniform(s_tmem);

  if (e >= 0) {   // the same for the whole cluster
    const int b0 = p.blocks * rank / splits, b1 = p.blocks * (rank + 1) / splits;
    const uint32_t idesc = idesc_f16(Half, false, false, kHalf, (rows + 15) / 16 * 16);
    const uint64_t x0 = sw128_kmajor_desc(smem_u32(smem) + kCodeBytes);
    const bool both = i0 + kHalf < p.N;   // else the second warpgroup has no rows
    const int half = warp >> 2, row = threadIdx.x & (kHalf - 1);
    const uint32_t bars = smem_u32(full), d_bar = smem_u32(&d_ready[half]);
    // A wait that gave up, here or in another warp, ends the waits and the loads;
    // the rest of the loop goes on with whatever there is, and nothing of the tile is
    // stored.
    // The first test is made all the same: the lanes meet in it, as what follows wants
    // them to (the loads and stores of tensor memory are .aligned), after one of them
    // has issued products or copies.
    bool got = true;
    auto expect = [&](uint32_t bar, uint64_t* at, uint32_t parity) {
      const bool there = try_wait(bar, parity);
      if (!there && got)
        got = mbar_wait_warp(at, parity, abort_flag, p.status, kDrop ? p.drop.limit : kWaitLimitCycles);
    };
    // By one lane. The copies are few, because the warp that asks for them keeps
    // the other three waiting: 256 rows of codes at once where all are the
    // expert's, and all of the tile's rows of x, needed or not.
    auto load = [&](int b, int stage) {
      if (kDrop && static_cast<int>(blockIdx.x) == p.drop.cta && b - b0 == p.drop.block) return;
      full[kStages + stage] = static_cast<uint32_t>(b - b0 + 1);
      uint8_t* sw = smem + stage * kStageBytes;
      uint8_t* sx = sw + kCodeBytes;
      const uint32_t bar = smem_u32(&full[stage]);
      mbar_arrive_expect_tx(&full[stage], (both ? kCodeBytes : kHalfBytes) + kR * BC * 2);
      load_2d<1>(sw, &tmW, b * (BC / 2), e * p.N + i0, bar);
      if (both && p.code_rows == kHalf) load_2d<1>(sw + kHalfBytes, &tmW, b * (BC / 2), e * p.N + i0 + kHalf, bar);
      load_2d<1>(sx, &tmX, b * BC, row0, bar);
      load_2d<1>(sx + kR * 128, &tmX, b * BC + 64, row0, bar);
    };
    const int loaded = min(kStages, b1 - b0);   // stages asked for in advance
    if (warp == 1 && elect_one())
      for (int s = 0; s < loaded; ++s) load(b0 + s, s);
    // Thread t holds weight row i0 + t, a column of `out`. A warpgroup's TMEM
    // columns: a step's weights, then the chunk's rows, group by group.
    const int i = i0 + threadIdx.x;
    const bool i_ok = i < p.N;
    const uint32_t half_tmem = tmem + half * kHalfCols;
    const uint32_t my_tmem = half_tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    GroupStream groups;
    groups.begin(p.scales, p.zeros, (static_cast<int64_t>(e) * p.N + min(i, p.N - 1)) * p.groups + b0 * kGroups,
                 static_cast<int64_t>(p.E) * p.N * p.groups);
    float2 acc[kR / 2];
#pragma unroll
    for (int r = 0; r < kR / 2; ++r) acc[r] = make_float2(0.0f, 0.0f);
    // the last step's sums, times their scales
    float f[kEnds];
    auto add = [&] {
#pragma unroll
      for (int q = 0; q < kEnds; ++q)
#pragma unroll
        for (int r0 = 0; r0 < kR; r0 += 16) {
          if (r0 >= rows) break;
          uint32_t v[16];
          tc_ld16_wait(my_tmem + kACols + q * kR + r0, v);
#pragma unroll
          for (int r = 0; r < 16; r += 2)
            fma2(acc[(r0 + r) / 2], f[q], __uint_as_float(v[r]), __uint_as_float(v[r + 1]));
        }
    };
    // The loop's own arithmetic is kept short: what the compiler knows to be uniform
    // goes through a slower pipe, step after step in all warps.
    const uint32_t swizzle = ((row >> 1) & 3) << 4;
    uint32_t codes = smem_u32(smem) + threadIdx.x * 64, bar = bars;   // of the stage
    uint32_t xs = static_cast<uint32_t>(x0);
    const uint32_t x_high = static_cast<uint32_t>(x0 >> 32);
    uint32_t phase = 0, turn = 0;
    int slot = 0, old = 0;                     // the stage's place in the ring, and the one before's
    int left = half == 1 && !both ? 0 : b1 - b0, to_load = left - loaded;
    int groups_left = p.groups - b0 * kGroups;   // of the rows
    const bool some = left > 0;
    bool first = true;
    for (int n = 0; left > 0; --left, ++n) {
#pragma unroll
      for (int h = 0; h < kSteps; ++h) {
        auto values = [&](int c, uint32_t (&v)[16]) {   // of chunk c of the step
          const int piece = h * kChunks + c;            // of the stage's four
          uint4 w;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                       : "r"(codes + ((piece << 4) ^ swizzle))
                       : "memory");
          const uint32_t o = w4_offset<Half>((groups.z >> (piece * 32 / kGroup * 8)) & 15u);
          w4_values<Half>(w.x, o, v);
          w4_values<Half>(w.y, o, v + 4);
          w4_values<Half>(w.z, o, v + 8);
          w4_values<Half>(w.w, o, v + 12);
        };
        if (h > 0 || !first) {
          expect(d_bar, &d_ready[half], turn ^ 1u);
          tc_fence_after();
          add();
        }
        if (h == 0) {
          if (n % (4 / kGroups) == 0) groups.refill();
          expect(bar, &full[slot], phase);
        }
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          uint32_t v[16];
          values(c, v);
          tc_st16(my_tmem + c * 16, v);
        }
#pragma unroll
        for (int q = 0; q < kEnds; ++q) {   // a group past the contraction has products with zeros
          const int g = h * kEnds + q;
          const uint32_t s = g & 1 ? groups.s[g / 2] >> 16 : groups.s[g / 2] & 0xffffu;
          f[q] = kGroup == BC || g < groups_left ? unpack2<Half>(s).x : 0.0f;
        }
        tc_wait_st();
        tc_fence_before();
        meet(half);
        if ((warp & 3) == 0 && elect_one()) {
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kStep; k += kUmmaK) {
            const int c = h * kStep + k;   // of the stage
            const uint32_t d = half_tmem + kACols + k / kGroup * kR, x_low = xs + ((c / 64 * (kR * 128) + c % 64 * 2) >> 4);
            if (k % kGroup != 0)
              tc_mma_f16_ta<true>(d, half_tmem + k / 2, x_low, x_high, idesc);
            else
              tc_mma_f16_ta<false>(d, half_tmem + k / 2, x_low, x_high, idesc);
          }
          commit(d_bar);
        }
        if (h == 0 && !first && to_load > 0) {
          // this warpgroup has used up the stage before; the later one fills it
          if ((warp & 3) == 1 && got && elect_one()) {
            __threadfence_block();
            if (!both || atomicAdd(&s_used[old], 1) & 1) load(b1 - to_load, old);
          }
          --to_load;
        }
        turn ^= 1u;
      }
      first = false;
      groups.pass<kGroups>();
      groups_left -= kGroups;
      old = slot;
      codes += kStageBytes;
      bar += 8;
      xs += kStageBytes >> 4;
      if (++slot == kStages) {
        slot = 0;
        codes -= kStages * kStageBytes;
        bar = bars;
        xs = static_cast<uint32_t>(x0);
        phase ^= 1u;
      }
    }
    if (some) {
      expect(d_bar, &d_ready[half], turn ^ 1u);
      tc_fence_after();
      add();
      tc_fence_before();
    }
    const bool stop = __syncthreads_or(!got);   // the ring is free: every product is done
    if (stop) {
      // Nothing of this CTA is under way when it exits or gives back its tensor memory:
      // neither products, a warpgroup's all being one lane's (elect.sync's choice is the
      // same every time), nor copies. Of those a place has one under way at most, and
      // none behind one that was left out, for the next is asked for by a warp that has
      // waited for the one before.
      if ((warp & 3) == 0 && elect_one()) {
        tc_commit(&done[half]);
        drain_wait(&done[half], 0);
      }
      if (warp == 1 && elect_one())
        for (int s = 0; s < kStages; ++s) {
          const int upto = static_cast<int>(full[kStages + s]);
          if (upto > 0 && !drain_wait(&full[s], static_cast<uint32_t>((upto - 1) / kStages) & 1u)) break;
        }
    }
    uint16_t* out = p.out + static_cast<int64_t>(row0) * p.ld_out + i;
    float* part = reinterpret_cast<float*>(smem);
    if (!stop) {
#pragma unroll
      for (int r = 0; r < kR; ++r) {
        if (r >= rows) break;
        const float v = (r & 1 ? acc[r / 2].y : acc[r / 2].x) * kW4Unit<Half>;
        if (splits > 1)
          part[r * kI + threadIdx.x] = v;
        else if (i_ok)
          out[r * p.ld_out] = static_cast<uint16_t>(pack2<Half>(v, 0.0f) & 0xffffu);
      }
    }
    if (splits > 1) {
      cluster_sync();
      // A CTA that gave up has no partials, and its flag is up: then no one stores.
      const int lane = threadIdx.x & 31;
      int lost = 0;
      if (lane < splits)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(lost) : "r"(cta_smem(&s_abort, lane)) : "memory");
      const bool whole = !__any_sync(0xffffffffu, lost != 0);
      // this CTA's share of the rows: the partials of all CTAs, in order
      const int ra = rows * rank / splits, rb = rows * (rank + 1) / splits;
      uint32_t from[8];
#pragma unroll
      for (int c = 0; c < 8; ++c)
        from[c] = c < splits ? cta_smem(smem, c) + static_cast<uint32_t>(threadIdx.x) * 4 : 0;
      for (int r = ra; r < rb; ++r) {
        float v[8], sum = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < splits)
            asm volatile("ld.shared::cluster.f32 %0, [%1];"
                         : "=f"(v[c])
                         : "r"(from[c] + static_cast<uint32_t>(r * kI * 4)));
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < splits) sum += v[c];
        if (i_ok && whole) out[r * p.ld_out] = static_cast<uint16_t>(pack2<Half>(sum, 0.0f) & 0xffffu);
      }
      cluster_sync();   // no CTA leaves while its partials are read
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    __syncwarp();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <bool Half, int kGroup, int kR, bool kDrop = false>
int launch(const CUtensorMap& tw, const CUtensorMap& tx, const W4Params& p, int64_t tiles, cudaStream_t s) {
  auto* kernel = grouped_w4_kernel<Half, kGroup, kR, kDrop>;
  constexpr int kSmem = smem_bytes(kGroup, kR);
  static std::atomic<bool> attr_set[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !attr_set[dev].load()) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
      return check_launch("cudaFuncSetAttribute(grouped_w4_kernel)");
    if (dev >= 0 && dev < 64) attr_set[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = static_cast<unsigned>(p.splits);
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, kernel, tw, tx, p);
  return check_launch("grouped_w4_kernel");
}

template <bool Half, int kGroup>
int launch_rows(int R, const CUtensorMap& tw, const CUtensorMap& tx, const W4Params& p, int64_t tiles,
                cudaStream_t s) {
  if (R <= 16) return launch<Half, kGroup, 16>(tw, tx, p, tiles, s);
  if constexpr (kGroup > 32) {
    if (R > 48) return launch<Half, kGroup, 64>(tw, tx, p, tiles, s);
    if (R > 32) return launch<Half, kGroup, 48>(tw, tx, p, tiles, s);
  }
  return launch<Half, kGroup, 32>(tw, tx, p, tiles, s);
}

// R: rows of a tile, 16, 32, 48 or 64; at most 32 with scales of 32 values, whose sums
// have no room for more. With `drop`: bf16, groups of 128 and R = 32.
int launch_grouped_w4_many(const W4Args& a, int R, cudaStream_t s, const W4Drop* drop = nullptr) {
  if (a.group == 32) R = std::min(R, 32);
  W4Params p;
  p.start = a.start;
  p.psum = a.psum;
  p.scales = static_cast<const uint2*>(a.scales);
  p.zeros = reinterpret_cast<const uint32_t*>(a.zeros);
  p.E = a.E;
  p.N = a.N;
  p.blocks = (a.Kd + BC - 1) / BC;
  p.groups = a.Kd / a.group;
  p.M_cap = a.M_cap;
  p.out = a.out;
  p.ld_out = a.ld_out;
  p.status = a.status;
  const int64_t live = std::min<int64_t>(a.E, a.max_rows), ni = (a.N + kI - 1) / kI;
  const int64_t want = 2 * device_sm_count();
  p.splits = 1;
  while (p.splits < 8 && live * ni * p.splits < want && p.blocks / (2 * p.splits) >= 4) p.splits *= 2;
  const int64_t tiles = (a.max_rows / R + live) * ni;
  MOE_REQUIRE(tiles * p.splits <= INT32_MAX, "moe_grouped_mm_w4: sizes exceed 32-bit tile numbers");
  CUtensorMap tw, tx;
  p.code_rows = a.N % kI == 0 ? kI : kHalf;
  int rc = make_tmap_codes4(&tw, a.codes, a.Kd / 2, static_cast<uint64_t>(a.E) * a.N, p.code_rows);
  if (rc != MOE_OK) return rc;
  rc = make_tmap_rows16(&tx, a.x, a.Kd, a.M_cap, a.ld_x, R);
  if (rc != MOE_OK) return rc;
  if (drop != nullptr) {
    p.drop = *drop;
    return launch<false, 128, 32, true>(tw, tx, p, tiles, s);
  }
  auto* pick = a.group == 128  ? (a.half ? launch_rows<true, 128> : launch_rows<false, 128>)
               : a.group == 64 ? (a.half ? launch_rows<true, 64> : launch_rows<false, 64>)
                               : (a.half ? launch_rows<true, 32> : launch_rows<false, 32>);
  return pick(R, tw, tx, p, tiles, s);
}

int check(const W4Args& a) {
  MOE_REQUIRE(a.start && a.psum, "moe_grouped_mm_w4: null segments");
  MOE_REQUIRE(a.E > 0 && a.E <= kW4MaxE, "moe_grouped_mm_w4: E must be in [1, 1024]");
  MOE_REQUIRE(a.group == 32 || a.group == 64 || a.group == 128, "moe_grouped_mm_w4: group must be 32, 64 or 128");
  MOE_REQUIRE(a.N > 0 && a.N % 8 == 0 && a.Kd > 0 && a.Kd % a.group == 0,
              "moe_grouped_mm_w4: N must be a positive multiple of 8, Kd of the group");
  MOE_REQUIRE(a.M_cap >= 0 && a.M_cap <= INT32_MAX && a.max_rows >= 0 && a.max_rows <= a.M_cap,
              "moe_grouped_mm_w4: M_cap and max_rows must fit each other and 32 bits");
  MOE_REQUIRE(a.codes && a.scales && (a.M_cap == 0 || (a.x && a.out)),
              "moe_grouped_mm_w4: operands must be non-null");
  MOE_REQUIRE(a.ld_x >= a.Kd && a.ld_out >= a.N && a.ld_x % 8 == 0 && a.ld_out % 8 == 0,
              "moe_grouped_mm_w4: a row stride must be a multiple of 8, at least the row");
  MOE_REQUIRE(aligned(a.x, 16) && aligned(a.codes, 16) && aligned(a.out, 16) && aligned(a.scales, 16) &&
                  aligned(a.zeros, 8),
              "moe_grouped_mm_w4: x, codes, scales and out must be 16-byte aligned, zeros 8-byte");
  MOE_REQUIRE(static_cast<int64_t>(a.E) * a.N <= INT32_MAX, "moe_grouped_mm_w4: sizes exceed 32-bit row numbers");
  const int64_t live = std::min<int64_t>(a.E, a.max_rows);
  MOE_REQUIRE((a.max_rows / 8 + live) * ((a.N + 31) / 32) <= INT32_MAX,
              "moe_grouped_mm_w4: sizes exceed 32-bit tile numbers");
  MOE_REQUIRE(a.x != a.out || a.max_rows == 0, "moe_grouped_mm_w4: out must not be x");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

extern "C" int moe_grouped_mm_w4(const void* x, int64_t ld_x, const uint8_t* codes, const void* scales,
                                 const uint8_t* zeros, int group, const int32_t* start,
                                 const int32_t* psum, int dtype, int E, int N, int Kd, int64_t M_cap,
                                 int64_t max_rows, void* out, int64_t ld_out, int32_t* d_status,
                                 moe_stream_t stream) {
  MOE_REQUIRE(dtype == MOE_BF16 || dtype == MOE_F16, "moe_grouped_mm_w4: dtype must be MOE_BF16 or MOE_F16");
  const moe::W4Args a = {x,  ld_x, codes, scales,   zeros, group,
                         start, psum, dtype == MOE_F16, E, N, Kd, M_cap, max_rows,
                         static_cast<uint16_t*>(out), ld_out, d_status};
  const int rc = moe::check(a);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE_DEVICE();
  if (max_rows == 0) return MOE_OK;
  const int64_t live = std::min<int64_t>(E, max_rows);
  const int64_t mean = (max_rows + live - 1) / live;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Which form, by the mean rows of an expert with rows and the weights read.
  // Up to four rows mma.sync is the faster (64 experts of 2048 x 4096 with 1, 2 and
  // 4 rows: 42, 54 and 61 us, here 54, 59 and 66), from six on this form (70 there,
  // 66 here; with 8 rows 84 and 66); with fewer weights its few large tiles leave SMs
  // idle longer: 8 experts of 4096 x 4096 take 20 us there and 27 here with 8 rows, 34
  // and 29 with 16, 32 of 2048 x 4096 with 8 in groups of 64 52 and 46; 8 of 1024 x
  // 1024 5.2 and 7.9 with 8, 8.5 and 10.9 with 32.
  const int64_t weights = live * N * Kd;
  const int64_t scale_bytes = 32ll * moe::w4_few_pitch(Kd / group) * 3;
  if ((mean <= 4 || (mean <= 8 && weights <= (1ll << 27)) || (mean <= 32 && weights <= (1ll << 23))) &&
      scale_bytes <= moe::kW4FewScaleBytes)
    return moe::launch_grouped_w4_few(a, s);
  // Rows of a tile, by the mean of the rows there may be (max_rows: what there are,
  // only the device knows): 64 experts of 2048 x 4096 with 8 rows each take 66, 68
  // and 75 us with 16, 32 and 64, with 16 rows 83, 69 and 76; with 32 rows 87, 77 and 80
  // with 32, 48 and 64 (in groups of 64 98, 90 and 98), with 26 rows 71, 76 and 79, with
  // 44 rows 115, 90 and 82; scales of 32 values (more rows of their sums do not fit) 84
  // and 88 us with 8 rows in tiles of 16 and 32, 167 and 130 with 32.
  return moe::launch_grouped_w4_many(a, mean <= 12 ? 16 : (mean <= 26 ? 32 : (mean <= 40 ? 48 : 64)), s);
}

extern "C" int moe_selftest_w4_wait(const void* x, int64_t ld_x, const uint8_t* codes, const void* scales,
                                    const uint8_t* zeros, const int32_t* start, const int32_t* psum, int E,
                                    int N, int Kd, int64_t M_cap, int64_t max_rows, void* out, int64_t ld_out,
                                    int64_t limit_cycles, int cta, int block, int32_t* d_status,
                                    moe_stream_t stream) {
  const moe::W4Args a = {x,  ld_x, codes, scales,   zeros, 128,
                         start, psum, false, E, N, Kd, M_cap, max_rows,
                         static_cast<uint16_t*>(out), ld_out, d_status};
  const int rc = moe::check(a);
  if (rc != MOE_OK) return rc;
  MOE_REQUIRE(d_status, "moe_selftest_w4_wait: null status");
  MOE_REQUIRE(limit_cycles > 0 && limit_cycles <= moe::kWaitLimitCycles,
              "moe_selftest_w4_wait: limit must be in (0, 4e9] cycles");
  MOE_REQUIRE_DEVICE();
  if (max_rows == 0) return MOE_OK;
  const moe::W4Drop drop = {limit_cycles, cta, block};
  return moe::launch_grouped_w4_many(a, 32, reinterpret_cast<cudaStream_t>(stream), &drop);
}

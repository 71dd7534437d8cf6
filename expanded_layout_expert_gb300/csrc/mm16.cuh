// Shared-memory operand and instruction descriptors, MMA and TMA wrappers of
// the 16-bit grouped products.
#pragma once

#include "common.cuh"

namespace moe {

constexpr int kMm16Panel = 64 * 128;   // 64 rows of 128 bytes: a TMA box of an i/j-contiguous operand

// Tensor-core operand whose contiguous axis is i/j, not the contracted one c:
// panels of 64 c rows x 128 bytes (64 values), 128-byte swizzle. Groups of 8 c
// rows are 1024 bytes apart (stride byte offset), panels kMm16Panel apart
// (leading byte offset).
MOE_DEV uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kMm16Panel >> 4) << 16;
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

// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit operands, K = 16. kCtas = 2: issued
// by the pair's first CTA; each CTA's shared memory holds its half of A's rows
// and of B's, each CTA's TMEM its half of D's rows.
template <int kCtas>
MOE_DEV void tc_mma_f16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                        uint32_t accumulate) {
  if constexpr (kCtas == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Address of the same shared-memory place in the cluster's CTA of that rank.
MOE_DEV uint32_t cta_smem(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}

// The .aligned forms want the whole warp at the instruction, so the lanes meet
// first, wherever the branches before it have left them.
MOE_DEV void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// TMA loads whose bytes are counted on `bar` (a shared::cluster address): a
// barrier of this CTA, or (kCtas = 2) of the other one of its pair.
template <int kCtas>
MOE_DEV void load_2d(void* dst, const CUtensorMap* tm, int32_t x, int32_t y, uint32_t bar) {
  if constexpr (kCtas == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
template <int kCtas>
MOE_DEV void load_3d(void* dst, const CUtensorMap* tm, int32_t x, int32_t y, int32_t z, uint32_t bar) {
  if constexpr (kCtas == 1)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// 32 TMEM lanes x 32 columns, waited for.
MOE_DEV void tc_ld32_wait(uint32_t taddr, uint32_t (&v)[32]) {
  tc_ld32(taddr, v);
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  tc_regs_landed(v);
}

// 32 TMEM lanes x 16 columns, waited for.
MOE_DEV void tc_ld16_wait(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}

// Bounded wait used while draining: no abort check, only the time limit.
MOE_DEV bool drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait_sleep(bar, parity, kWaitSleepNs)) {
    if (clock64() - t0 > kWaitLimitCycles) return false;
  }
  return true;
}

}  // namespace moe

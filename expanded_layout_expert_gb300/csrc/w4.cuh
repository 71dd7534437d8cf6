// What the two forms of the 4-bit product share: codes to 16-bit values, and the
// expert of a tile.
//
// A word holds 8 codes, value 2j in the low and 2j + 1 in the high four bits of
// byte j. The bits of a 16-bit float below twice its smallest normal number, read
// as an integer n, stand for n times its smallest subnormal: so a code in bits
// 0-3 of a half word is q and one in bits 4-7 is 16 q such units, and one packed
// fma, times a power of two less z, makes (q - z) 2^-6 (bf16) or (q - z) 2^-9
// (fp16), exactly. Two masks and a byte permutation per pair, no shifts.
#pragma once

#include "dtype16.cuh"

namespace moe {

constexpr int kW4MaxE = 1024;

// What the 16-bit weights are short of.
template <bool Half>
constexpr float kW4Unit = Half ? 0x1p9f : 0x1p6f;

// -z / kW4Unit, twice, made in the same way.
template <bool Half>
MOE_DEV uint32_t w4_offset(uint32_t z) {
  uint32_t r;
  if constexpr (Half)
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(z * 0x00010001u), "r"(0xf800f800u));
  else
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(z * 0x00010001u), "r"(0xff00ff00u));
  return r;
}
constexpr uint32_t kW4Zero = 8;   // where there are no zero points

// acc += s (a, b), two fp32 values an instruction.
MOE_DEV void fma2(float2& acc, float s, float a, float b) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %2};\n\t"
      "mov.b64 y, {%3, %4};\n\t"
      "mov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "f"(s), "f"(a), "f"(b));
}

// Codes 2j and 2j + 1 of a word, given as low = its low four bits a byte and
// high = its high ones in place. A byte of `low` is below 16, so its sign, which
// prmt's selectors from 8 on copy, makes the zero bytes.
template <bool Half, int j>
MOE_DEV uint32_t w4_pair(uint32_t low, uint32_t high, uint32_t off) {
  uint32_t v, r;
  asm("prmt.b32 %0, %1, %2, %3;"
      : "=r"(v)
      : "r"(low), "r"(high), "n"(((8 + j) << 12) | ((4 + j) << 8) | ((8 + j) << 4) | j));
  if constexpr (Half)   // 2^15 and 2^11 times 2^-24
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x68007800u), "r"(off));
  else                  // 2^127 and 2^123 times 2^-133
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(v), "r"(0x7d007f00u), "r"(off));
  return r;
}

// A word's eight values, in order.
template <bool Half>
MOE_DEV void w4_values(uint32_t w, uint32_t off, uint32_t* to) {
  const uint32_t low = w & 0x0f0f0f0fu, high = w & 0xf0f0f0f0u;
  to[0] = w4_pair<Half, 0>(low, high, off);
  to[1] = w4_pair<Half, 1>(low, high, off);
  to[2] = w4_pair<Half, 2>(low, high, off);
  to[3] = w4_pair<Half, 3>(low, high, off);
}

// Which expert has chunk number `chunk`, of at most R of its rows? Thread t of
// kThreads counts the chunks of experts per t .. per t + per - 1; segments are
// clamped into the buffer. The block meets twice; `found` (shared: expert or
// -1, first row, rows) is valid after that. Returns all experts' chunks to the
// last thread.
template <int kThreads, int R>
MOE_DEV int w4_find_chunk(const int32_t* __restrict__ start, const int32_t* __restrict__ psum, int E,
                          int64_t M_cap, int chunk, int (&warp_sum)[kThreads / 32], int (&found)[3]) {
  constexpr int kPer = (kW4MaxE + kThreads - 1) / kThreads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (E + kThreads - 1) / kThreads;   // <= kPer
  const int cap = static_cast<int>(M_cap);
  if (threadIdx.x == 0) found[0] = -1;
  int a[kPer], n[kPer], mine = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = threadIdx.x * per + j;
    a[j] = n[j] = 0;
    if (j < per && e < E) {
      a[j] = min(max(start[e], 0), cap);
      n[j] = min(max(psum[e], a[j]), cap) - a[j];
      mine += (n[j] + R - 1) / R;
    }
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int base = incl - mine;
  for (int w = 0; w < warp; ++w) base += warp_sum[w];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int c = (n[j] + R - 1) / R;
    if (chunk >= base && chunk < base + c) {
      found[0] = threadIdx.x * per + j;
      found[1] = a[j] + (chunk - base) * R;
      found[2] = min(R, n[j] - (chunk - base) * R);
    }
    base += c;
  }
  __syncthreads();
  return base;
}

}  // namespace moe

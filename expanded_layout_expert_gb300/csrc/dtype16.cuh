// The two 16-bit formats of the training kernels, as one interface: eight
// values of a 16-byte vector to and from fp32, rounded to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace moe {

template <bool Half>
MOE_DEV float2 unpack2(uint32_t w) {
  if (Half) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <bool Half>
MOE_DEV uint32_t pack2(float a, float b) {
  if (Half) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <bool Half>
MOE_DEV void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack2<Half>(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

template <bool Half>
MOE_DEV uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack2<Half>(f[0], f[1]), pack2<Half>(f[2], f[3]), pack2<Half>(f[4], f[5]),
                    pack2<Half>(f[6], f[7]));
}

}  // namespace moe

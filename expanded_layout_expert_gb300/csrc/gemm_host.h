// Host-side pieces shared by the two grouped-GEMM implementations.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace moe {

// TMA descriptor for a 2-D uint8 tensor [outer, inner] with a row stride of
// `stride` bytes, copied in boxes of box_outer rows x 128 bytes with 128-byte
// swizzling; rows past `outer` read as zero. Returns MOE_OK or MOE_ERR_CUDA
// (message set).
int make_tmap_k128(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t stride, uint32_t box_outer);

// TMA descriptors for 16-bit operands, copied in boxes of 64 values (128
// bytes, 128-byte swizzling); places past the tensor read as zero.
// Rows: [rows, width] with a row stride of `ld` values, boxes of box_rows rows.
// Weights: [E, N, Kd] contiguous, boxes of box_n rows of one expert.
int make_tmap_rows16(CUtensorMap* tm, const void* base, uint64_t width, uint64_t rows, uint64_t ld,
                     uint32_t box_rows);
int make_tmap_weights16(CUtensorMap* tm, const void* base, uint64_t Kd, uint64_t N, uint64_t E,
                        uint32_t box_n);
// Results [E, rows, width] with a row stride of `ld` values, 16-bit or fp32,
// stored in boxes of 32 rows x 64 bytes (64-byte swizzling).
int make_tmap_result(CUtensorMap* tm, void* base, bool f32, uint64_t width, uint64_t rows, uint64_t E,
                     uint64_t ld);

// Arguments of the block-scaled (ue8m0) grouped GEMM, already validated.
struct MxGemmArgs {
  const uint8_t* A;
  const uint32_t* A_scale;  // packed ue8m0, column-major words [ceil(Kd/512), ld_as]
  int64_t ld_as;
  const int32_t* start;
  const int32_t* tile_prefix;
  const int32_t* d_total;
  const uint8_t* W;
  const uint8_t* W_scale;   // ue8m0 bytes [E, N/128, Kd/128]
  const float* row_w;       // non-null: output row r is multiplied by row_w[r]
  int E, N, Kd;
  int64_t M_cap;
  uint16_t* out;
  int32_t* status;
  unsigned long long* trace;  // optional per-CTA cycle counters
  // Non-null: W is W13 [E, N = 2I, Kd] and the kernel applies silu(gate)*up
  // and the ue8m0 fp8 quantiser in its epilogue, writing down_proj's input
  // di [M_cap, I] and its packed scales (int32 words [ceil(I/512), ld_ds],
  // addressed as bytes) instead of `out`.
  uint8_t* di = nullptr;
  uint8_t* di_scale = nullptr;
  int64_t ld_ds = 0;
};

// Forward (dgrad) product for experts with few rows each, arguments already
// validated: out = a times the weights. max_rows: rows of all segments
// together, at most.
int launch_grouped_mm16_few(bool dgrad, bool half, const void* a, int64_t ld_a, const void* w,
                            const int32_t* start, const int32_t* psum, int E, int N, int Kd,
                            int64_t M_cap, int64_t max_rows, uint16_t* out, int64_t ld_out,
                            int32_t* status, cudaStream_t s);

// Launches the tcgen05 block-scaled kernel (N % 256 == 0).
int launch_grouped_gemm_mx(const MxGemmArgs& a, cudaStream_t s);

}  // namespace moe

// fp8.h -- launcher interfaces of the E4M3 operators with a scale per 128 values.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nvfp4 {

struct Fp8QuantArgs {
  const void* x;        // [rows, k], or [rows, 2 k] for SwiGLU (gate | up)
  int dtype, act;
  int64_t rows;
  int k, block_rows;    // 1 or 128 rows share a scale
  uint8_t* codes;       // [rows, k]
  float* scale;         // [ceil(rows / block_rows), ceil(k / 128)]
};
hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, hipStream_t s);

struct Fp8GemmArgs {
  const uint8_t* a;     // [B, K]
  const float* as;      // [B, ceil(K / 128)]
  const uint8_t* w;     // [N, K]
  const float* ws;      // [ceil(N / 128), ceil(K / 128)]
  void* y;              // [B, N]
  int out_dtype;
  int B, N, K;
};
hipError_t launch_fp8_gemm(const Fp8GemmArgs& g, hipStream_t s);

}  // namespace nvfp4

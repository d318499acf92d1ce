// Block-FP8 linear layer (fp8_linear.cu, api_fp8_linear.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda.h>  // CUtensorMap (types only; the encoder is fetched at run time)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lingmoe {

constexpr int kF8Block = 128;     // inputs (and outputs of the weights) per scale
constexpr int kF8GemvMaxT = 8;    // tokens up to which the weights are streamed through mma.sync
constexpr int kF8TileM = 128;     // tokens per tensor-core tile
constexpr int kF8TileNs = 4;      // output tile widths 32, 64, 128, 256
__host__ __device__ constexpr int f8_tile_n(int i) { return 32 << i; }

// shared memory of the streaming kernel with T tokens' codes and scales, and its limit (two CTAs per SM)
constexpr int kF8GemvSmem = 104 * 1024;
__host__ __device__ constexpr size_t f8_gemv_smem(int T, int kb) { return (size_t)T * ((size_t)kb * kF8Block + 64 + 4 * kb); }

struct F8Maps {
  CUtensorMap x;                  // token codes, boxes of 128 rows
  CUtensorMap w[kF8TileNs];       // weight codes, boxes of f8_tile_n(i) rows
};

struct F8Params {
  const uint8_t* w;   // codes [rows padded to 128][kb * 128]
  const float* sw;    // [ceil(N / 128)][kb]
  const __nv_bfloat16* x;  // tokens (the streaming kernel quantises them itself)
  long long x_stride;
  int K, x_vec;
  const uint8_t* xq;  // codes [rows padded to 128][kb * 128]
  const float* sx;    // [kb][tpad]
  void* out;
  long long out_stride;  // elements
  int T, N, kb, tpad, out_bf16, vec;  // vec: rows of `out` take 16-byte stores
  int tiles_m, tiles_n;
  unsigned int* err;
  unsigned long long wait_ns;
  int skip_cta;       // test hook: this CTA's producer issues no copies (-1: none)
};

cudaError_t setup_fp8_linear();
cudaError_t f8_encode_maps(F8Maps* m, const uint8_t* w, int w_rows, const uint8_t* xq, int x_rows, int kbytes);
// x (bf16, row stride in elements) -> codes and scales
cudaError_t launch_f8_quantize(const __nv_bfloat16* x, long long x_stride, int T, int K, int kb, int tpad,
                               uint8_t* xq, float* sx, cudaStream_t s);
// fused: quantises p.x itself (f8_gemv_smem within kF8GemvSmem); otherwise p.xq and p.sx are filled
cudaError_t launch_f8_gemv(const F8Params& p, int sms, bool fused, cudaStream_t s);
cudaError_t launch_f8_gemm(const F8Maps& m, const F8Params& p, int tile, int ctas, cudaStream_t s);

}  // namespace lingmoe

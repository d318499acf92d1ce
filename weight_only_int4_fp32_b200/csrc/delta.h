// Gated delta rule (delta.cu, api_delta.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lingmoe {

constexpr int kDeltaChunk = 64;    // tokens per chunk of the prefill
constexpr int kDeltaMaxStep = 8;   // tokens per sequence of a step

// one chunk of one head: what the scan needs of q, k, v, g and beta (delta.cu)
__host__ __device__ constexpr int delta_tile_bytes(int dk) { return kDeltaChunk * dk * 2; }
__host__ __device__ constexpr int delta_ops_bytes(int dk) {
  return 5 * delta_tile_bytes(dk) + kDeltaChunk * kDeltaChunk * 2 + (dk + 2 * kDeltaChunk) * 4;
}
__host__ __device__ constexpr int delta_rec_bytes(int dk, int dv) { return delta_ops_bytes(dk) + kDeltaChunk * dv * 4; }

struct DeltaParams {
  const __nv_bfloat16 *q, *k, *v;
  const float *g, *beta;
  __nv_bfloat16* out;                  // contiguous [tokens, Hv, dv]
  long long q_b, q_t, q_h, k_b, k_t, k_h, v_b, v_t, v_h;  // strides in elements: sequence (step), token, head
  long long g_b, g_t, g_h, be_b, be_t, be_h;
  int g_c;                             // 1: a decay per channel, 0: per head
  int vec_qk, vec_v, vec_g;            // rows take 8-byte (q, k), 4-byte (v), 16-byte (g) loads
  int Hk, Hv, dv;
  int T;                               // prefill: tokens in all; step: tokens per sequence
  int nseq, num_slots;
  float* state;                        // [num_slots][Hv][dk][dv]
  const int32_t* slots;                // [nseq] or NULL
  const int32_t* cu;                   // prefill: [nseq + 1]
  const uint8_t* fresh;                // prefill: [nseq] or NULL
  const int32_t* accepted;             // step: [nseq] or NULL
  float scale;
  unsigned char* ws;                   // prefill: records of seg_chunks x Hv
  int seg0, seg_chunks;
  unsigned int* err;
  unsigned long long wait_ns;
  int skip;                            // test hook: the scan issues no copies
};

cudaError_t setup_delta();
cudaError_t launch_delta_step(const DeltaParams& p, int dk, int sms, cudaStream_t s);
cudaError_t launch_delta_prep(const DeltaParams& p, int dk, bool first, cudaStream_t s);
cudaError_t launch_delta_scan(const DeltaParams& p, int dk, cudaStream_t s);

}  // namespace lingmoe

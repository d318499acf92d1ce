// Beam search: selection over beams and vocabulary, and the in-place move of
// the beams' states (beam.cu, api_beam.cpp).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace lingmoe {

constexpr int kBeamMax = 16;        // beams per group
constexpr int kBeamMaxSegs = 32;    // pieces of a row, one lane each in the merge
constexpr int beam_tile(bool bf16) { return bf16 ? 8192 : 4096; }  // logits a CTA takes at a time: 256 threads x 64 bytes
constexpr int kBeamCtas = 4;        // CTAs of the selection that an SM holds at once
constexpr int kReorderTensors = 32; // tensors per reorder launch

// One piece of a row: max, at most 1 below its largest logit, the sum of
// exp(logit - max), and its best keys in order (0: none).  Key: order key of the logit above ~token.
struct BeamPart {
  double sum;
  float max;
  float pad;
  unsigned long long keys[kBeamMax];
};

struct BeamSelectParams {
  const void* logits;
  long long group_stride, beam_stride;  // elements
  const float* scores;
  const uint8_t* finished;  // may be NULL
  int groups, beams, vocab, eos, segs, seg_len;
  BeamPart* parts;          // [groups * beams][segs]
  unsigned int* arrived;    // [groups], zero between calls
  int32_t* tokens;
  int32_t* parents;
  float* scores_out;
  uint8_t* finished_out;
};
cudaError_t launch_beam_select(const BeamSelectParams& p, bool bf16, cudaStream_t s);

struct BeamReorderParams {
  unsigned char* state[kReorderTensors];
  unsigned long long row_bytes[kReorderTensors];
  const int32_t* parents;  // [groups][beams]
  const int32_t* slots;    // [groups][beams] or NULL: row g * beams + w
  int num_rows, beams;
};
// unit: bytes moved per thread (16, 4 or 1); every pointer and row size a multiple of it
cudaError_t launch_beam_reorder(const BeamReorderParams& p, int tensors, int groups, int unit, size_t longest_row,
                                cudaStream_t s);

}  // namespace lingmoe

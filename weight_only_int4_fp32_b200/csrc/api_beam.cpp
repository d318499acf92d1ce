// C entry points of beam search (beam.cu): argument checks, workspace, dispatch.
#include <atomic>
#include <cmath>
#include <new>

#include "api_common.h"
#include "beam.h"

using namespace lingmoe;

struct ling_moe_beam {
  int device = 0, sms = 0;
  int max_groups = 0, beams = 0, vocab = 0;
  BeamPart* parts = nullptr;
  unsigned int* arrived = nullptr;
  std::atomic<int64_t> launches{0};
  ~ling_moe_beam() {
    if (parts) cudaFree(parts);
    if (arrived) cudaFree(arrived);
  }
};

extern "C" {

int ling_moe_beam_create(int max_groups, int beams, int vocab, ling_moe_beam_t** out) {
  if (!out) return fail_arg(LING_MOE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (max_groups < 1 || beams < 1 || vocab < 1)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "max_groups, beams and vocab must be positive");
  if (beams > kBeamMax || max_groups > 65535 || vocab > (1 << 30))
    return fail_arg(LING_MOE_ERR_UNSUPPORTED, "at most %d beams, 65535 groups and 2^30 tokens", kBeamMax);
  int dev = 0, sms = 0;
  if (int rc = check_device(&dev, &sms)) return rc;
  ling_moe_beam* h = new (std::nothrow) ling_moe_beam();
  if (!h) return fail_arg(LING_MOE_ERR_OOM, "host allocation failed");
  h->device = dev;
  h->sms = sms;
  h->max_groups = max_groups;
  h->beams = beams;
  h->vocab = vocab;
  const size_t parts = (size_t)max_groups * beams * kBeamMaxSegs * sizeof(BeamPart);
  cudaError_t e = cudaMalloc(&h->parts, parts);
  if (e == cudaSuccess) e = cudaMalloc(&h->arrived, (size_t)max_groups * sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaMemset(h->arrived, 0, (size_t)max_groups * sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const int rc = fail_cuda(e, "beam workspace");
    delete h;
    return rc;
  }
  *out = h;
  return LING_MOE_OK;
}

int ling_moe_beam_select(ling_moe_beam_t* h, const void* logits, int logits_type, int64_t group_stride,
                         int64_t beam_stride, int groups, const float* scores, const uint8_t* finished, int eos,
                         int32_t* tokens, int32_t* parents, float* scores_out, uint8_t* finished_out, void* stream) {
  if (!h) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle is NULL");
  if (groups < 0 || groups > h->max_groups)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "groups=%d outside [0, %d]", groups, h->max_groups);
  if (logits_type != LING_MOE_TYPE_F32 && logits_type != LING_MOE_TYPE_BF16)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "unknown logits type %d", logits_type);
  if (eos < -1 || eos >= h->vocab) return fail_arg(LING_MOE_ERR_INVALID_ARG, "eos=%d outside [-1, %d)", eos, h->vocab);
  if (finished && eos < 0) return fail_arg(LING_MOE_ERR_INVALID_ARG, "finished beams need an eos token");
  if (groups == 0) return LING_MOE_OK;
  if (!logits || !scores || !tokens || !parents || !scores_out || !finished_out)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "a pointer is NULL");
  if (group_stride < 0 || beam_stride < 0) return fail_arg(LING_MOE_ERR_INVALID_ARG, "strides must not be negative");
  const size_t es = logits_type == LING_MOE_TYPE_F32 ? 4 : 2;
  if (!is_aligned(logits, es) || !is_aligned(scores, 4) || !is_aligned(tokens, 4) || !is_aligned(parents, 4) ||
      !is_aligned(scores_out, 4))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "a pointer is not aligned to its element size");
  const size_t rows = (size_t)groups * h->beams;
  const size_t lbytes = ((size_t)(groups - 1) * group_stride + (size_t)(h->beams - 1) * beam_stride + h->vocab) * es;
  const void* outs[4] = {tokens, parents, scores_out, finished_out};
  const size_t nb[4] = {rows * 4, rows * 4, rows * 4, rows};
  for (int i = 0; i < 4; ++i) {
    if (ranges_overlap(outs[i], nb[i], logits, lbytes))
      return fail_arg(LING_MOE_ERR_INVALID_ARG, "an output overlaps logits");
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(outs[i], nb[i], outs[j], nb[j]))
        return fail_arg(LING_MOE_ERR_INVALID_ARG, "two outputs overlap");
    // scores_out may be scores and finished_out may be finished, wholly
    if (outs[i] != (const void*)scores && ranges_overlap(outs[i], nb[i], scores, rows * 4))
      return fail_arg(LING_MOE_ERR_INVALID_ARG, "an output overlaps scores");
    if (i != 2 && outs[i] == (const void*)scores)
      return fail_arg(LING_MOE_ERR_INVALID_ARG, "an output overlaps scores");
    if (finished && !(i == 3 && outs[i] == (const void*)finished) && ranges_overlap(outs[i], nb[i], finished, rows))
      return fail_arg(LING_MOE_ERR_INVALID_ARG, "an output overlaps finished");
  }
  if (int rc = check_same_device(h->device)) return rc;

  // Segments: as many as keep the whole call within one wave of CTAs (kBeamCtas
  // per SM), each at least one tile.
  const int tile = beam_tile(logits_type == LING_MOE_TYPE_BF16), tiles = (h->vocab + tile - 1) / tile;
  int segs = (int)((long long)kBeamCtas * h->sms / (long long)rows);
  if (segs < 1) segs = 1;
  if (segs > kBeamMaxSegs) segs = kBeamMaxSegs;
  if (segs > tiles) segs = tiles;
  const int per = (tiles + segs - 1) / segs;
  segs = (tiles + per - 1) / per;
  BeamSelectParams p{};
  p.logits = logits;
  p.group_stride = group_stride;
  p.beam_stride = beam_stride;
  p.scores = scores;
  p.finished = finished;
  p.groups = groups;
  p.beams = h->beams;
  p.vocab = h->vocab;
  p.eos = eos;
  p.segs = segs;
  p.seg_len = per * tile;
  p.parts = h->parts;
  p.arrived = h->arrived;
  p.tokens = tokens;
  p.parents = parents;
  p.scores_out = scores_out;
  p.finished_out = finished_out;
  cudaError_t e = launch_beam_select(p, logits_type == LING_MOE_TYPE_BF16, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e, "beam selection launch");
  h->launches.fetch_add(1);
  return LING_MOE_OK;
}

int ling_moe_beam_reorder(void* const* states, const size_t* row_bytes, int n_states, int num_rows,
                          const int32_t* slots, const int32_t* parents, int groups, int beams, void* stream) {
  if (n_states < 0 || groups < 0 || num_rows < 0)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "n_states, groups and num_rows must not be negative");
  if (beams < 1 || beams > kBeamMax || groups > 65535)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "beams=%d outside [1, %d] or groups=%d above 65535", beams, kBeamMax, groups);
  if (n_states == 0 || groups == 0 || num_rows == 0) return LING_MOE_OK;
  if (!states || !row_bytes || !parents) return fail_arg(LING_MOE_ERR_INVALID_ARG, "a pointer is NULL");
  if (!slots && (int64_t)groups * beams > num_rows)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "%d groups of %d beams need that many rows (got %d)", groups, beams, num_rows);
  if (!is_aligned(parents, 4) || !is_aligned(slots, 4))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "parents and slots must be 4-byte aligned");
  const size_t ib = (size_t)groups * beams * 4;
  for (int i = 0; i < n_states; ++i) {
    if (!states[i] && row_bytes[i]) return fail_arg(LING_MOE_ERR_INVALID_ARG, "states[%d] is NULL", i);
    const size_t nb = row_bytes[i] * (size_t)num_rows;
    if (ranges_overlap(states[i], nb, parents, ib) || (slots && ranges_overlap(states[i], nb, slots, ib)))
      return fail_arg(LING_MOE_ERR_INVALID_ARG, "states[%d] overlaps parents or slots", i);
    for (int j = 0; j < i; ++j)
      if (ranges_overlap(states[i], nb, states[j], row_bytes[j] * (size_t)num_rows))
        return fail_arg(LING_MOE_ERR_INVALID_ARG, "states[%d] overlaps states[%d]", i, j);
  }
  // one launch per 32 tensors of the same unit (the widest that divides addresses and row sizes)
  for (int unit : {16, 4, 1}) {
    BeamReorderParams p{};
    p.parents = parents;
    p.slots = slots;
    p.num_rows = num_rows;
    p.beams = beams;
    int n = 0;
    size_t longest = 0;
    for (int i = 0; i <= n_states; ++i) {
      if (n == kReorderTensors || (i == n_states && n)) {
        cudaError_t e = launch_beam_reorder(p, n, groups, unit, longest, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return fail_cuda(e, "beam reorder launch");
        n = 0;
        longest = 0;
      }
      if (i == n_states || !row_bytes[i]) continue;
      const auto fits = [&](int u) { return is_aligned(states[i], u) && row_bytes[i] % u == 0; };
      if ((fits(16) ? 16 : fits(4) ? 4 : 1) != unit) continue;
      p.state[n] = static_cast<unsigned char*>(states[i]);
      p.row_bytes[n] = row_bytes[i];
      if (row_bytes[i] > longest) longest = row_bytes[i];
      ++n;
    }
  }
  return LING_MOE_OK;
}

int64_t ling_moe_beam_launch_count(const ling_moe_beam_t* h) { return h ? h->launches.load() : 0; }

void ling_moe_beam_destroy(ling_moe_beam_t* h) { delete h; }

}  // extern "C"

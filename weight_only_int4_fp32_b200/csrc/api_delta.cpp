// C entry points of the gated delta rule (delta.cu): argument checks,
// workspace, dispatch.
#include <atomic>
#include <cmath>
#include <new>

#include "api_common.h"
#include "delta.h"

using namespace lingmoe;

namespace {

constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s
// Records (chunk x head) of one half of the prefill's workspace: the operands of
// one segment of chunks, four waves of the preparation's CTAs (two per SM):
// 8 per SM and not 4: 172 us in place of 175 for 2048 tokens x 32 heads, 704 in place of 744 for 8192 packed tokens.
constexpr int kRecordsPerSm = 8;

struct Span { const char* lo; const char* hi; };
Span span(const void* p, size_t es, const int64_t n[4], const int64_t st[4]) {
  int64_t last = 0;
  for (int i = 0; i < 4; ++i) last += (n[i] - 1) * st[i];
  return {static_cast<const char*>(p), static_cast<const char*>(p) + (last + 1) * (int64_t)es};
}

}  // namespace

struct ling_moe_delta {
  int device = 0, sms = 0;
  ling_moe_delta_config_t cfg{};
  int seg_chunks = 0;
  size_t half_bytes = 0;  // of the workspace
  unsigned char* ws = nullptr;
  unsigned int* err = nullptr;
  std::atomic<int64_t> launches{0};
  int skip = 0;
  unsigned long long wait_ns = kWaitNs;
  ~ling_moe_delta() {
    if (ws) cudaFree(ws);
    if (err) cudaFree(err);
  }
};

static int64_t chunks_bound(int64_t tokens, int64_t seqs) { return tokens / kDeltaChunk + (seqs < tokens ? seqs : tokens); }

// What both calls check; `n` tokens per sequence for a step (batch = sequences), all tokens for a prefill (batch = 1).
static int fill(const ling_moe_delta_t* h, const ling_moe_delta_io_t* io, int batch, int n, DeltaParams* p) {
  const ling_moe_delta_config_t& c = h->cfg;
  if (!io->q || !io->k || !io->v || !io->g || !io->beta || !io->out || !io->state)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "a pointer is NULL");
  if (!is_aligned(io->q, 2) || !is_aligned(io->k, 2) || !is_aligned(io->v, 2) || !is_aligned(io->g, 4) ||
      !is_aligned(io->beta, 4) || !is_aligned(io->slots, 4))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "an input is not aligned to its element size");
  if (!is_aligned(io->out, 16) || !is_aligned(io->state, 16))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "out and state must be 16-byte aligned");
  if (io->num_slots < 1) return fail_arg(LING_MOE_ERR_INVALID_ARG, "num_slots must be positive");
  for (const int64_t* s : {io->q_stride, io->k_stride, io->v_stride, io->g_stride, io->beta_stride})
    for (int i = 0; i < 3; ++i)
      if (s[i] < 0) return fail_arg(LING_MOE_ERR_INVALID_ARG, "strides must not be negative");
  if (io->g_channel_stride != 0 && io->g_channel_stride != 1)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "g_channel_stride must be 1 (a decay per channel) or 0 (per head)");
  const size_t out_bytes = (size_t)batch * n * c.v_heads * c.head_v * 2;
  const size_t state_bytes = (size_t)io->num_slots * c.v_heads * c.head_k * c.head_v * 4;
  if (ranges_overlap(io->out, out_bytes, io->state, state_bytes))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "out overlaps state");
  const struct { const void* ptr; size_t es; const int64_t* st; int heads, dim; int64_t ch; } in[5] = {
      {io->q, 2, io->q_stride, c.k_heads, c.head_k, 1},  {io->k, 2, io->k_stride, c.k_heads, c.head_k, 1},
      {io->v, 2, io->v_stride, c.v_heads, c.head_v, 1},  {io->g, 4, io->g_stride, c.v_heads, c.head_k, io->g_channel_stride},
      {io->beta, 4, io->beta_stride, c.v_heads, 1, 1}};
  for (const auto& x : in) {
    const int64_t dims[4] = {batch, n, x.heads, x.dim}, st[4] = {x.st[0], x.st[1], x.st[2], x.ch};
    const Span s = span(x.ptr, x.es, dims, st);
    if (ranges_overlap(s.lo, (size_t)(s.hi - s.lo), io->out, out_bytes) ||
        ranges_overlap(s.lo, (size_t)(s.hi - s.lo), io->state, state_bytes))
      return fail_arg(LING_MOE_ERR_INVALID_ARG, "out or state overlaps an input");
  }
  if (int rc = check_same_device(h->device)) return rc;
  p->q = static_cast<const __nv_bfloat16*>(io->q);
  p->k = static_cast<const __nv_bfloat16*>(io->k);
  p->v = static_cast<const __nv_bfloat16*>(io->v);
  p->g = io->g;
  p->beta = io->beta;
  p->out = static_cast<__nv_bfloat16*>(io->out);
  p->q_b = io->q_stride[0], p->q_t = io->q_stride[1], p->q_h = io->q_stride[2];
  p->k_b = io->k_stride[0], p->k_t = io->k_stride[1], p->k_h = io->k_stride[2];
  p->v_b = io->v_stride[0], p->v_t = io->v_stride[1], p->v_h = io->v_stride[2];
  p->g_b = io->g_stride[0], p->g_t = io->g_stride[1], p->g_h = io->g_stride[2];
  p->be_b = io->beta_stride[0], p->be_t = io->beta_stride[1], p->be_h = io->beta_stride[2];
  p->g_c = (int)io->g_channel_stride;
  const auto mult = [](const int64_t* s, int m) { return s[0] % m == 0 && s[1] % m == 0 && s[2] % m == 0; };
  p->vec_qk = is_aligned(io->q, 8) && is_aligned(io->k, 8) && mult(io->q_stride, 4) && mult(io->k_stride, 4);
  p->vec_v = is_aligned(io->v, 4) && mult(io->v_stride, 2);
  p->vec_g = is_aligned(io->g, 16) && mult(io->g_stride, 4);
  p->Hk = c.k_heads;
  p->Hv = c.v_heads;
  p->dv = c.head_v;
  p->T = n;
  p->num_slots = io->num_slots;
  p->state = io->state;
  p->slots = io->slots;
  p->scale = c.scale;
  p->err = h->err;
  p->wait_ns = h->wait_ns;
  p->skip = h->skip;
  return LING_MOE_OK;
}

extern "C" {

int ling_moe_delta_create(const ling_moe_delta_config_t* cfg, ling_moe_delta_t** out) {
  if (!out) return fail_arg(LING_MOE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!cfg) return fail_arg(LING_MOE_ERR_INVALID_ARG, "cfg is NULL");
  if (cfg->k_heads < 1 || cfg->v_heads < 1 || cfg->head_k < 1 || cfg->head_v < 1 || cfg->max_tokens < 1 || cfg->max_seqs < 1)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "heads, head sizes, max_tokens and max_seqs must be positive");
  if (cfg->v_heads % cfg->k_heads) return fail_arg(LING_MOE_ERR_INVALID_ARG, "v_heads must be a multiple of k_heads");
  if (!std::isfinite(cfg->scale)) return fail_arg(LING_MOE_ERR_INVALID_ARG, "scale must be finite");
  if ((cfg->head_k != 64 && cfg->head_k != 128) || (cfg->head_v != 64 && cfg->head_v != 128))
    return fail_arg(LING_MOE_ERR_UNSUPPORTED, "head_k and head_v must be 64 or 128 (got %d, %d)", cfg->head_k, cfg->head_v);
  if (cfg->v_heads > 1024 || cfg->max_tokens > (1 << 24) || cfg->max_seqs > (1 << 18))
    return fail_arg(LING_MOE_ERR_UNSUPPORTED, "at most 1024 heads, 2^24 tokens and 2^18 sequences");
  int dev = 0, sms = 0;
  if (int rc = check_device(&dev, &sms)) return rc;
  cudaError_t e = setup_delta();
  if (e != cudaSuccess) return fail_cuda(e, "delta rule kernel attributes");
  ling_moe_delta* h = new (std::nothrow) ling_moe_delta();
  if (!h) return fail_arg(LING_MOE_ERR_OOM, "host allocation failed");
  h->device = dev;
  h->sms = sms;
  h->cfg = *cfg;
  if (h->cfg.scale == 0.f) h->cfg.scale = 1.f / std::sqrt((float)cfg->head_k);
  const int64_t need = chunks_bound(cfg->max_tokens, cfg->max_seqs);
  const int64_t fit = kRecordsPerSm * sms / cfg->v_heads > 0 ? kRecordsPerSm * sms / cfg->v_heads : 1;
  h->seg_chunks = (int)(need < fit ? need : fit);
  h->half_bytes = (size_t)h->seg_chunks * cfg->v_heads * delta_rec_bytes(cfg->head_k, cfg->head_v);
  e = cudaMalloc(&h->ws, h->half_bytes * (need > h->seg_chunks ? 2 : 1));
  if (e == cudaSuccess) e = cudaMalloc(&h->err, sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaMemset(h->err, 0, sizeof(unsigned int));
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const int rc = fail_cuda(e, "delta rule workspace");
    delete h;
    return rc;
  }
  *out = h;
  return LING_MOE_OK;
}

int ling_moe_delta_step(ling_moe_delta_t* h, const ling_moe_delta_io_t* io, int seqs, int tokens,
                        const int32_t* accepted, void* stream) {
  if (!h || !io) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle or io is NULL");
  if (seqs < 0 || seqs > h->cfg.max_seqs)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "seqs=%d outside [0, %d]", seqs, h->cfg.max_seqs);
  if (tokens < 0 || tokens > kDeltaMaxStep)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "tokens=%d outside [0, %d]", tokens, kDeltaMaxStep);
  if (seqs == 0 || tokens == 0) return LING_MOE_OK;
  if (!io->slots && seqs > io->num_slots)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "%d sequences need that many slots (got %d)", seqs, io->num_slots);
  if (!is_aligned(accepted, 4)) return fail_arg(LING_MOE_ERR_INVALID_ARG, "accepted must be 4-byte aligned");
  DeltaParams p{};
  if (int rc = fill(h, io, seqs, tokens, &p)) return rc;
  p.nseq = seqs;
  p.accepted = accepted;
  cudaError_t e = launch_delta_step(p, h->cfg.head_k, h->sms, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail_cuda(e, "delta rule step launch");
  h->launches.fetch_add(1);
  return LING_MOE_OK;
}

int ling_moe_delta_prefill(ling_moe_delta_t* h, const ling_moe_delta_io_t* io, int tokens, const int32_t* cu_seqlens,
                           int seqs, const uint8_t* fresh, void* stream_v) {
  if (!h || !io) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle or io is NULL");
  if (tokens < 0 || tokens > h->cfg.max_tokens)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "tokens=%d outside [0, %d]", tokens, h->cfg.max_tokens);
  if (seqs < 0 || seqs > h->cfg.max_seqs)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "seqs=%d outside [0, %d]", seqs, h->cfg.max_seqs);
  if (tokens == 0 || seqs == 0) return LING_MOE_OK;
  if (!cu_seqlens || !is_aligned(cu_seqlens, 4))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "cu_seqlens is NULL or not 4-byte aligned");
  if (!io->slots && seqs > io->num_slots)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "%d sequences need that many slots (got %d)", seqs, io->num_slots);
  DeltaParams p{};
  if (int rc = fill(h, io, 1, tokens, &p)) return rc;
  p.nseq = seqs;
  p.cu = cu_seqlens;
  p.fresh = fresh;
  cudaStream_t s = static_cast<cudaStream_t>(stream_v);
  const int64_t all = chunks_bound(tokens, seqs);
  for (int64_t c = 0; c < all; c += h->seg_chunks) {
    p.seg0 = (int)c;
    p.ws = h->ws + (c / h->seg_chunks % 2) * h->half_bytes;
    p.seg_chunks = (int)(all - c < h->seg_chunks ? all - c : h->seg_chunks);
    cudaError_t e = launch_delta_prep(p, h->cfg.head_k, c == 0, s);
    if (e == cudaSuccess) e = launch_delta_scan(p, h->cfg.head_k, s);
    if (e != cudaSuccess) return fail_cuda(e, "delta rule prefill launch");
    h->launches.fetch_add(2);
  }
  return LING_MOE_OK;
}

int ling_moe_delta_status(ling_moe_delta_t* h, void* stream_v) {
  if (!h) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle is NULL");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream_v));
  if (e != cudaSuccess) return fail_cuda(e, "stream synchronize");
  unsigned int err = 0;
  e = cudaMemcpy(&err, h->err, sizeof(err), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail_cuda(e, "read device error word");
  if (err) {
    cudaMemset(h->err, 0, sizeof(unsigned int));
    cudaDeviceSynchronize();
    return fail_arg(LING_MOE_ERR_DEVICE_TIMEOUT, "a bounded device-side wait of the delta rule gave up (error word %u)", err);
  }
  return LING_MOE_OK;
}

int64_t ling_moe_delta_launch_count(const ling_moe_delta_t* h) { return h ? h->launches.load() : 0; }

int ling_moe_delta_test_set_wait(ling_moe_delta_t* h, int skip, uint64_t wait_limit_ns) {
  if (!h) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle is NULL");
  h->skip = skip != 0;
  h->wait_ns = wait_limit_ns ? wait_limit_ns : kWaitNs;
  return LING_MOE_OK;
}

void ling_moe_delta_destroy(ling_moe_delta_t* h) { delete h; }

}  // extern "C"

// C entry points of the block-FP8 linear layer (fp8_linear.cu): argument
// checks, ownership, dispatch.
#include <atomic>
#include <new>

#include "api_common.h"
#include "fp8_linear.h"

using namespace lingmoe;

namespace {
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s
}

struct ling_moe_fp8_linear {
  int device = 0, sms = 0;
  int N = 0, K = 0, kb = 0, max_tokens = 0, tpad = 0;
  uint8_t* w = nullptr;
  float* sw = nullptr;
  uint8_t* xq = nullptr;
  float* sx = nullptr;
  unsigned int* err = nullptr;
  F8Maps maps{};
  std::atomic<int64_t> launches{0};
  int skip_cta = -1;
  unsigned long long wait_ns = kWaitNs;
  ~ling_moe_fp8_linear() {
    for (void* p : {(void*)w, (void*)sw, (void*)xq, (void*)sx, (void*)err})
      if (p) cudaFree(p);
  }
};

extern "C" {

int ling_moe_fp8_linear_create(const uint8_t* codes, const float* scales, int out_features, int in_features,
                               int max_tokens, ling_moe_fp8_linear_t** out) {
  if (!out) return fail_arg(LING_MOE_ERR_INVALID_ARG, "out is NULL");
  *out = nullptr;
  if (!codes || !scales) return fail_arg(LING_MOE_ERR_INVALID_ARG, "codes or scales is NULL");
  if (!is_aligned(scales, 4)) return fail_arg(LING_MOE_ERR_INVALID_ARG, "scales must be 4-byte aligned");
  if (out_features < 1 || in_features < 1 || max_tokens < 1)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "out_features, in_features and max_tokens must be positive");
  if (out_features > (1 << 24) || in_features > (1 << 22) || max_tokens > (1 << 24))
    return fail_arg(LING_MOE_ERR_UNSUPPORTED, "at most 2^24 outputs and tokens and 2^22 inputs");
  int dev = 0, sms = 0;
  if (int rc = check_device(&dev, &sms)) return rc;
  cudaError_t e = setup_fp8_linear();
  if (e != cudaSuccess) return fail_cuda(e, "linear kernel attributes");
  ling_moe_fp8_linear* h = new (std::nothrow) ling_moe_fp8_linear();
  if (!h) return fail_arg(LING_MOE_ERR_OOM, "host allocation failed");
  h->device = dev;
  h->sms = sms;
  h->N = out_features;
  h->K = in_features;
  h->kb = (in_features + kF8Block - 1) / kF8Block;
  h->max_tokens = max_tokens;
  h->tpad = (max_tokens + kF8TileM - 1) / kF8TileM * kF8TileM;
  const size_t pitch = (size_t)h->kb * kF8Block;
  const int wrows = (out_features + kF8Block - 1) / kF8Block * kF8Block;
  const size_t nsw = (size_t)(wrows / kF8Block) * h->kb * sizeof(float);
  const size_t nsx = (size_t)h->kb * h->tpad * sizeof(float);
  e = cudaDeviceSynchronize();  // the weights may still be on their way on any of the caller's streams
  struct { void** p; size_t n; } plan[] = {{(void**)&h->w, (size_t)wrows * pitch},
                                           {(void**)&h->sw, nsw},
                                           {(void**)&h->xq, (size_t)h->tpad * pitch},
                                           {(void**)&h->sx, nsx},
                                           {(void**)&h->err, sizeof(unsigned int)}};
  for (auto& a : plan)
    if (e == cudaSuccess) {
      e = cudaMalloc(a.p, a.n);
      if (e != cudaSuccess) *a.p = nullptr;
      // padding rows and inputs stay zero: they multiply to nothing
      else e = cudaMemset(*a.p, 0, a.n);
    }
  if (e == cudaSuccess)
    e = cudaMemcpy2D(h->w, pitch, codes, (size_t)in_features, (size_t)in_features, (size_t)out_features,
                     cudaMemcpyDeviceToDevice);
  if (e == cudaSuccess) e = cudaMemcpy(h->sw, scales, nsw, cudaMemcpyDeviceToDevice);
  if (e == cudaSuccess) e = f8_encode_maps(&h->maps, h->w, wrows, h->xq, h->tpad, (int)pitch);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  if (e != cudaSuccess) {
    const int rc = fail_cuda(e, "block-FP8 linear layer");
    delete h;
    return rc;
  }
  *out = h;
  return LING_MOE_OK;
}

int ling_moe_fp8_linear_forward(ling_moe_fp8_linear_t* h, const void* x, int64_t x_stride, int T, void* out,
                                int out_type, int64_t out_stride, void* stream_v) {
  if (!h) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle is NULL");
  if (T < 0 || T > h->max_tokens) return fail_arg(LING_MOE_ERR_INVALID_ARG, "T=%d outside [0, %d]", T, h->max_tokens);
  if (out_type != LING_MOE_TYPE_F32 && out_type != LING_MOE_TYPE_BF16)
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "unknown output type %d", out_type);
  if (T == 0) return LING_MOE_OK;
  if (!x || !out) return fail_arg(LING_MOE_ERR_INVALID_ARG, "x or out is NULL");
  const size_t es = out_type == LING_MOE_TYPE_F32 ? 4 : 2;
  if (!is_aligned(x, 2) || !is_aligned(out, es))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "x or out is not aligned to its element size");
  if (T > 1 && (x_stride < h->K || out_stride < h->N))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "a row stride is shorter than its row");
  if (ranges_overlap(x, ((size_t)(T - 1) * (T > 1 ? x_stride : 0) + h->K) * 2, out,
                     ((size_t)(T - 1) * (T > 1 ? out_stride : 0) + h->N) * es))
    return fail_arg(LING_MOE_ERR_INVALID_ARG, "out overlaps x");
  if (int rc = check_same_device(h->device)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream_v);
  const bool fused = T <= kF8GemvMaxT && f8_gemv_smem(T, h->kb) <= kF8GemvSmem;
  cudaError_t e = cudaSuccess;
  if (!fused)
    e = launch_f8_quantize(static_cast<const __nv_bfloat16*>(x), x_stride, T, h->K, h->kb, h->tpad, h->xq, h->sx, s);
  if (e != cudaSuccess) return fail_cuda(e, "token quantisation launch");
  F8Params p{};
  p.w = h->w;
  p.sw = h->sw;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.x_stride = x_stride;
  p.K = h->K;
  p.x_vec = is_aligned(x, 16) && (T == 1 || x_stride % 8 == 0);
  p.xq = h->xq;
  p.sx = h->sx;
  p.out = out;
  p.out_stride = out_stride;
  p.T = T;
  p.N = h->N;
  p.kb = h->kb;
  p.tpad = h->tpad;
  p.out_bf16 = out_type == LING_MOE_TYPE_BF16;
  p.vec = is_aligned(out, 16) && (T == 1 || (out_stride * es) % 16 == 0);
  p.err = h->err;
  p.wait_ns = h->wait_ns;
  p.skip_cta = h->skip_cta;
  if (T <= kF8GemvMaxT) {
    e = launch_f8_gemv(p, h->sms, fused, s);
  } else {
    // The tile width whose waves of tiles cost least.  A wave's time at K = 2560 is
    // 9.0, 10.2, 12.5 and 17.5 us for widths 32, 64, 128 and 256: a fixed part worth
    // some 200 columns, and the width.  Over 16 to 8192 tokens at 2560 x 1024, 2560 x 2560,
    // 8192 x 2560, 8192 x 4096 and 2560 x 8192 (outputs x inputs) it takes the quickest of
    // the four widths, or one within 6 % of it.
    p.tiles_m = (T + kF8TileM - 1) / kF8TileM;
    int tile = 0;
    long long best = 0;
    for (int i = 0; i < kF8TileNs; ++i) {
      const long long tiles = (long long)p.tiles_m * ((h->N + f8_tile_n(i) - 1) / f8_tile_n(i));
      const long long cost = (tiles + h->sms - 1) / h->sms * (f8_tile_n(i) + 200);
      if (i == 0 || cost <= best) {
        best = cost;
        tile = i;
      }
    }
    p.tiles_n = (h->N + f8_tile_n(tile) - 1) / f8_tile_n(tile);
    const long long tiles = (long long)p.tiles_m * p.tiles_n;
    e = launch_f8_gemm(h->maps, p, tile, (int)(tiles < h->sms ? tiles : h->sms), s);
  }
  if (e != cudaSuccess) return fail_cuda(e, "linear launch");
  h->launches.fetch_add(fused ? 1 : 2);
  return LING_MOE_OK;
}

int ling_moe_fp8_linear_status(ling_moe_fp8_linear_t* h, void* stream_v) {
  if (!h) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle is NULL");
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream_v));
  if (e != cudaSuccess) return fail_cuda(e, "stream synchronize");
  unsigned int err = 0;
  e = cudaMemcpy(&err, h->err, sizeof(err), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return fail_cuda(e, "read device error word");
  if (err) {
    cudaMemset(h->err, 0, sizeof(unsigned int));
    cudaDeviceSynchronize();
    return fail_arg(LING_MOE_ERR_DEVICE_TIMEOUT, "a bounded device-side wait of the linear layer gave up (error word %u)",
                    err);
  }
  return LING_MOE_OK;
}

int64_t ling_moe_fp8_linear_launch_count(const ling_moe_fp8_linear_t* h) { return h ? h->launches.load() : 0; }

int ling_moe_fp8_linear_test_set_wait(ling_moe_fp8_linear_t* h, int skip_cta, uint64_t wait_limit_ns) {
  if (!h) return fail_arg(LING_MOE_ERR_INVALID_ARG, "handle is NULL");
  if (skip_cta >= h->sms) return fail_arg(LING_MOE_ERR_INVALID_ARG, "skip_cta out of range");
  h->skip_cta = skip_cta < 0 ? -1 : skip_cta;
  h->wait_ns = wait_limit_ns ? wait_limit_ns : kWaitNs;
  return LING_MOE_OK;
}

void ling_moe_fp8_linear_destroy(ling_moe_fp8_linear_t* h) { delete h; }

}  // extern "C"

// Linear layer with block-scaled FP8 weights: y = x W^T.
//
//   W: e4m3 codes [N, K], one fp32 scale sw per block of 128 outputs x 128 inputs
//   x: bf16 tokens, quantised per call: for each token and each 128 inputs
//      sx = max|x| * (1 / 448) (1 for zeros), codes e4m3(x / sx); 1 / 448, the
//      product and the division each rounded once to fp32, the conversion to
//      nearest even, saturating
//   y[t, n] = sum over blocks b of  sx[t, b] sw[n / 128, b] (sum_k xq[t, k] wq[n, k])
//
// The inner sums are sums of exact products in fp32; each is scaled and added
// to an fp32 accumulator outside the tensor cores, since both scales change
// with every 128 inputs.  One rounding to the output type at the end.
//
// Two kernels follow the quantisation, launched as its programmatic
// dependent (their set-up and first weight loads overlap it):
//  * up to 8 tokens: weights streamed from HBM straight into mma.sync
//    fragments (e4m3 -> fp16 exactly), 16 outputs per CTA, the blocks of K
//    dealt to its 8 warps.  Bound: HBM, N x K bytes.
//  * more: tcgen05 (kind::f8f6f4) tiles of 128 tokens x 32..256 outputs.  Each
//    128-wide K block is one pipeline stage and one chain of four MMAs into
//    one of two TMEM buffers; 8 warps read a finished buffer, scale it and
//    add it to accumulators in registers while the next block multiplies.
//    Bound: tensor cores for many tokens, HBM for few.
// Source of the format: vLLM recipe page "inclusionAI/Ling-3.0-flash", section
// Overview (the block-FP8 checkpoint); the page does not define it, the
// definition above is this library's.
#include "common.cuh"
#include "fp8_linear.h"
#include "tcgen05.cuh"

namespace lingmoe {

namespace {

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// two floats -> two e4m3 codes; v0 in the low byte (the lower K index)
__device__ __forceinline__ uint32_t f8x2(float v0, float v1) {
  unsigned short r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v1), "f"(v0));
  return r;
}
// two e4m3 codes (a 16-bit pair) -> the same two values as fp16 (exact)
__device__ __forceinline__ uint32_t f8x2_to_f16x2(uint32_t pair) {
  uint32_t r;
  const unsigned short p = (unsigned short)pair;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(p));
  return r;
}

// ---------------------------------------------------------------- quantisation
// 16 lanes take one token's 128 inputs of block blockIdx.y, 8 each; a CTA
// takes 64 tokens.  HBM bound for many tokens (2 bytes read, 1 written).
constexpr int kQTokens = 64;

__global__ void __launch_bounds__(256) f8_quantize_kernel(const __nv_bfloat16* __restrict__ x, long long stride, int T,
                                                          int K, int kb, int tpad, int vec, uint8_t* __restrict__ xq,
                                                          float* __restrict__ sx) {
  pdl_launch_dependents();
  const int b = blockIdx.y, l = threadIdx.x & 15;
  const int k = b * kF8Block + 8 * l;
  for (int i = threadIdx.x >> 4; i < kQTokens; i += 16) {
    const long long t = (long long)blockIdx.x * kQTokens + i;
    if (t >= T) break;  // both halves of a warp: only whole 16-lane groups shuffle below
    const __nv_bfloat16* src = x + t * stride + k;
    uint32_t r[4] = {0u, 0u, 0u, 0u};
    if (vec && k + 8 <= K) {
      const uint4 v = *reinterpret_cast<const uint4*>(src);
      r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < K) r[e >> 1] |= (uint32_t) * reinterpret_cast<const unsigned short*>(src + e) << (16 * (e & 1));
    }
    float a = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) a = fmaxf(a, fmaxf(fabsf(bf16lo(r[e])), fabsf(bf16hi(r[e]))));
    const unsigned int half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, o));
    const float s = a > 0.f ? __fmul_rn(a, 1.0f / 448.0f) : 1.0f;
    uint32_t c[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = f8x2(__fdiv_rn(bf16lo(r[e]), s), __fdiv_rn(bf16hi(r[e]), s));
    *reinterpret_cast<uint2*>(xq + t * ((long long)kb * kF8Block) + k) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
    if (l == 0) sx[(long long)b * tpad + t] = s;
  }
}

// ---------------------------------------------------------------- 1..8 tokens
// A warp's share of K: blocks w, w + 8, ...; kU of them are in flight at once
// (4 x 16 bytes per lane each).  Lane (g, c) = (lane / 4, lane % 4) loads codes
// 16 c .. + 15 of each half block of rows g and g + 8; the K order inside the
// MMAs is a permutation of the 64 codes, the same for weights and tokens.
constexpr int kGemvRows = 16, kGemvWarps = 8, kU = 4;

__global__ void __launch_bounds__(kGemvWarps * 32) f8_gemv_kernel(const F8Params p) {
  __shared__ float red[kGemvWarps][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int row0 = blockIdx.x * kGemvRows;
  const size_t pitch = (size_t)p.kb * kF8Block;
  const uint8_t* wa = p.w + (size_t)(row0 + g) * pitch + 16 * c;  // the padded rows exist
  const uint8_t* wb = wa + 8 * pitch;
  const uint8_t* xr = p.xq + (size_t)g * pitch + 16 * c;          // rows >= T: any codes, results dropped
  const float* sw = p.sw + (size_t)(row0 / kF8Block) * p.kb;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  bool waited = false;
  for (int b0 = warp; b0 < p.kb; b0 += kGemvWarps * kU) {
    uint4 a[kU][2], b[kU][2];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int kb = b0 + kGemvWarps * u;
      if (kb < p.kb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          a[u][h] = ldg_stream(wa + (size_t)kb * kF8Block + 64 * h);
          b[u][h] = ldg_stream(wb + (size_t)kb * kF8Block + 64 * h);
        }
      }
    }
    if (!waited) {
      pdl_wait();  // the tokens' codes
      waited = true;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int kb = b0 + kGemvWarps * u;
      if (kb < p.kb) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 xv = __ldcg(reinterpret_cast<const uint4*>(xr + (size_t)kb * kF8Block + 64 * h));
          const uint32_t xp[4] = {xv.x, xv.y, xv.z, xv.w};
          const uint32_t pa[4] = {a[u][h].x, a[u][h].y, a[u][h].z, a[u][h].w};
          const uint32_t pb[4] = {b[u][h].x, b[u][h].y, b[u][h].z, b[u][h].w};
#pragma unroll
          for (int m = 0; m < 4; ++m)
            mma_16816(d[0], d[1], d[2], d[3], f8x2_to_f16x2(pa[m]), f8x2_to_f16x2(pb[m]), f8x2_to_f16x2(pa[m] >> 16),
                      f8x2_to_f16x2(pb[m] >> 16), f8x2_to_f16x2(xp[m]), f8x2_to_f16x2(xp[m] >> 16), d[0], d[1], d[2],
                      d[3]);
        }
        const float2 sx = __ldcg(reinterpret_cast<const float2*>(p.sx + (size_t)kb * p.tpad + 2 * c));
        const float s = __ldg(sw + kb);
        acc[0] = fmaf(d[0], s * sx.x, acc[0]);
        acc[1] = fmaf(d[1], s * sx.y, acc[1]);
        acc[2] = fmaf(d[2], s * sx.x, acc[2]);
        acc[3] = fmaf(d[3], s * sx.y, acc[3]);
      }
    }
  }
  *reinterpret_cast<float4*>(red[warp][lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  // thread (token, row): consecutive threads write consecutive outputs
  const int i = threadIdx.x;
  if (i < 8 * kGemvRows) {
    const int tok = i / kGemvRows, r = i % kGemvRows;
    const int n = row0 + r;
    if (tok < p.T && n < p.N) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kGemvWarps; ++w) s += red[w][4 * (r & 7) + (tok >> 1)][(r >> 3) * 2 + (tok & 1)];
      const size_t at = (size_t)tok * p.out_stride + n;
      if (p.out_bf16)
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(s);
      else
        static_cast<float*>(p.out)[at] = s;
    }
  }
}

// ---------------------------------------------------------------- tensor-core tiles
template <int BN>
struct F8Cfg {
  static constexpr int kStageA = kF8TileM * kF8Block;  // 16 KB
  static constexpr int kStageB = BN * kF8Block;
  static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 6 : 8;
  static constexpr int kBarOff = kStages * (kStageA + kStageB);
  static constexpr int kSmem = 1024 + kBarOff + 256;
  static constexpr int kTmemCols = 2 * BN;
};
constexpr int kF8EpiWarps = 8;
constexpr int kF8Threads = (kF8EpiWarps + 2) * 32;

__device__ __forceinline__ void tc_mma_f8(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}"
      :: "r"(tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(0), "r"(0), "r"(0), "r"(0));
}
__device__ __forceinline__ void tmem_ld16_async(uint32_t taddr, float v[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr));
}
// waits for every load issued so far; v is what the caller uses next
__device__ __forceinline__ void tmem_wait16(float v[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :: "memory");
}

}  // namespace

// Warps 0-7 promote and store (TMEM lanes 32 (w % 4).., column half w / 4), warp
// 8 issues the TMA loads, warp 9 the MMAs.  Every role walks the tiles
// blockIdx.x, + gridDim.x, ... (token tile fastest).
template <int BN>
__global__ void __launch_bounds__(kF8Threads, 1)
f8_gemm_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const F8Params p) {
  using C = F8Cfg<BN>;
  constexpr int S = C::kStages;
  extern __shared__ __align__(1024) unsigned char smem_raw_f8[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw_f8) + 1023) & ~uintptr_t(1023));
  unsigned char* sA = smem;
  unsigned char* sB = smem + S * C::kStageA;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + S;
  uint64_t* accf = empty + S;
  uint64_t* acce = accf + 2;
  uint64_t* drain = acce + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ntiles = p.tiles_m * p.tiles_n;

  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], kF8EpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kF8EpiWarps + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_u32(tmem_slot)), "r"(C::kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the tokens' codes and scales

  if (warp < kF8EpiWarps) {
    constexpr int HALF = BN / 2, NC = HALF / 16;
    const int q = warp & 3, half = warp >> 2;
    const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(half * HALF);
    int it = 0;  // K blocks so far: buffer it % 2
    bool ok = true;
    for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
      const int m0 = (tile % p.tiles_m) * kF8TileM, n0 = (tile / p.tiles_m) * BN + half * HALF;
      const int row = m0 + 32 * q + lane;
      const float* sx = p.sx + row;  // rows up to tpad exist
      const float* sw = p.sw + (size_t)min(n0 / kF8Block, (p.N - 1) / kF8Block) * p.kb;
      float acc[HALF];
#pragma unroll
      for (int j = 0; j < HALF; ++j) acc[j] = 0.f;
      float s_next = __ldcg(sx) * __ldg(sw);
#pragma unroll 1
      for (int kb = 0; kb < p.kb; ++kb, ++it) {
        const int b = it & 1;
        const float s = s_next;
        if (kb + 1 < p.kb) s_next = __ldcg(sx + (size_t)(kb + 1) * p.tpad) * __ldg(sw + kb + 1);
        if (lane == 0) ok = tc_wait(&accf[b], (it >> 1) & 1, p.err, abort_flag, p.wait_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
        float v[2][16];
        tmem_ld16_async(tb + b * BN, v[0]);
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          tmem_wait16(v[c & 1]);
          if (c + 1 < NC) {
            tmem_ld16_async(tb + b * BN + 16 * (c + 1), v[(c + 1) & 1]);
          } else {  // everything is read: the buffer may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acce[b]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[16 * c + j] = fmaf(v[c & 1][j], s, acc[16 * c + j]);
        }
      }
      if (!ok) break;
      if (row < p.T) {
        const size_t at = (size_t)row * p.out_stride + n0;
        if (p.out_bf16) {
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < HALF; j += 8) {
            if (p.vec && n0 + j + 8 <= p.N) {
              __nv_bfloat162 r[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) r[i] = __floats2bfloat162_rn(acc[j + 2 * i], acc[j + 2 * i + 1]);
              *reinterpret_cast<uint4*>(o + j) = *reinterpret_cast<const uint4*>(r);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (n0 + j + i < p.N) o[j + i] = __float2bfloat16_rn(acc[j + i]);
            }
          }
        } else {
          float* o = static_cast<float*>(p.out) + at;
#pragma unroll
          for (int j = 0; j < HALF; j += 4) {
            if (p.vec && n0 + j + 4 <= p.N) {
              *reinterpret_cast<float4*>(o + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (n0 + j + i < p.N) o[j + i] = acc[j + i];
            }
          }
        }
      }
    }
  } else if (warp == kF8EpiWarps) {
    if (lane == 0) {
      int g = 0;
      bool ok = (int)blockIdx.x != p.skip_cta;
      for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
        const int m0 = (tile % p.tiles_m) * kF8TileM, n0 = (tile / p.tiles_m) * BN;
#pragma unroll 1
        for (int kb = 0; kb < p.kb; ++kb, ++g) {
          const int s = g % S;
          if (!tc_wait(&empty[s], ((g / S) & 1) ^ 1, p.err, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], C::kStageA + C::kStageB);
          tma_load_2d(smem_u32(sA + s * C::kStageA), &tmX, kb * kF8Block, m0, &full[s]);
          tma_load_2d(smem_u32(sB + s * C::kStageB), &tmW, kb * kF8Block, n0, &full[s]);
        }
      }
      // after an abort, loads may still be landing: wait for every armed stage
      for (int i = g > S ? g - S : 0; i < g; ++i) mbar_wait(&full[i % S], (i / S) & 1, kTcWaitNs, p.err);
    }
    __syncwarp();
  } else {
    if (lane == 0) {
      const uint32_t idesc = make_idesc(BN);  // f32 accumulator; e4m3 is format 0, as f16 is in kind::f16
      int g = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
#pragma unroll 1
        for (int kb = 0; kb < p.kb; ++kb, ++g) {
          const int s = g % S, b = g & 1;
          if (!tc_wait(&full[s], (g / S) & 1, p.err, abort_flag, p.wait_ns) ||
              !tc_wait(&acce[b], ((g >> 1) & 1) ^ 1, p.err, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(sA + s * C::kStageA), b0 = smem_u32(sB + s * C::kStageB);
#pragma unroll
          for (int k4 = 0; k4 < kF8Block / 32; ++k4)
            tc_mma_f8(tmem + b * BN, sw128_desc(a0 + 32 * k4), sw128_desc(b0 + 32 * k4), idesc, k4 ? 1u : 0u);
          tc_commit(&empty[s]);
          tc_commit(&accf[b]);
        }
      }
      // no MMA may still be writing TMEM when it is freed
      tc_commit(drain);
      mbar_wait(drain, 0, kTcWaitNs, p.err);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kF8EpiWarps + 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(C::kTmemCols) : "memory");
  }
}

// ---------------------------------------------------------------- host
template <int BN>
static cudaError_t setup_tile() {
  return cudaFuncSetAttribute(f8_gemm_kernel<BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, F8Cfg<BN>::kSmem);
}
cudaError_t setup_fp8_linear() {
  cudaError_t e = setup_tile<32>();
  if (e == cudaSuccess) e = setup_tile<64>();
  if (e == cudaSuccess) e = setup_tile<128>();
  if (e == cudaSuccess) e = setup_tile<256>();
  return e;
}

cudaError_t f8_encode_maps(F8Maps* m, const uint8_t* w, int w_rows, const uint8_t* xq, int x_rows, int kbytes) {
  cudaError_t e = tma_encode_2d(&m->x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, xq, x_rows, kbytes, kF8Block, kF8TileM);
  for (int i = 0; i < kF8TileNs && e == cudaSuccess; ++i)
    e = tma_encode_2d(&m->w[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, w_rows, kbytes, kF8Block, f8_tile_n(i));
  return e;
}

cudaError_t launch_f8_quantize(const __nv_bfloat16* x, long long x_stride, int T, int K, int kb, int tpad,
                               uint8_t* xq, float* sx, cudaStream_t s) {
  const int vec = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && x_stride % 8 == 0;
  f8_quantize_kernel<<<dim3((T + kQTokens - 1) / kQTokens, kb), 256, 0, s>>>(x, x_stride, T, K, kb, tpad, vec, xq, sx);
  return cudaGetLastError();
}

// launched while the kernel before it in the stream may still run (it waits for it itself)
template <typename... A>
static cudaError_t launch_dependent(void (*kernel)(A...), int grid, int threads, int smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

cudaError_t launch_f8_gemv(const F8Params& p, cudaStream_t s) {
  return launch_dependent(f8_gemv_kernel, (p.N + kGemvRows - 1) / kGemvRows, kGemvWarps * 32, 0, s, p);
}

cudaError_t launch_f8_gemm(const F8Maps& m, const F8Params& p, int tile, int ctas, cudaStream_t s) {
  switch (tile) {
    case 0: return launch_dependent(f8_gemm_kernel<32>, ctas, kF8Threads, F8Cfg<32>::kSmem, s, m.x, m.w[0], p);
    case 1: return launch_dependent(f8_gemm_kernel<64>, ctas, kF8Threads, F8Cfg<64>::kSmem, s, m.x, m.w[1], p);
    case 2: return launch_dependent(f8_gemm_kernel<128>, ctas, kF8Threads, F8Cfg<128>::kSmem, s, m.x, m.w[2], p);
    default: return launch_dependent(f8_gemm_kernel<256>, ctas, kF8Threads, F8Cfg<256>::kSmem, s, m.x, m.w[3], p);
  }
}

}  // namespace lingmoe

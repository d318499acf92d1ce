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
// Two kernels:
//  * up to 8 tokens: weights streamed from HBM straight into mma.sync
//    fragments (e4m3 -> fp16 exactly), 16 outputs at a time per CTA, the blocks
//    of K dealt to its 8 warps, tokens quantised in the same launch.  Bound:
//    HBM, N x K bytes; at sizes of one projection, latency (2560 x 2560, one
//    token: 5.4 us on the device; 8192 x 2560, eight: 11.4 us, some 8 of them without
//    the quantisation).
//  * more: tcgen05 (kind::f8f6f4) tiles of 128 tokens x 32..256 outputs.  Each
//    128-wide K block is one pipeline stage and one chain of four MMAs into
//    one of two TMEM buffers; 16 warps read a finished buffer, scale it and
//    add it to accumulators in registers while the next block multiplies.
//    A quantisation kernel runs first, the tiles as its programmatic dependent.
//    Bound: the way of a buffer between MMAs and promotion, and filling 48 KB
//    per block, for many tokens (8192 x 8192 x 4096: 387 us, 1.42 PFLOP/s, in a row of
//    ten; 357 in the best burst, 411 call after call, by the card's power); HBM or one
//    tile's K loop for few (2560 x 2560: 13 us for 16 tokens, 15 for 256).
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
// 16 lanes take one token's 128 inputs of one block, 8 each.

// codes of x / s for 8 values.  The quotient's rounding matters only where a
// border between two codes lies within it: x times the rounded 1 / s is within
// 3 2^-24 of the rounded quotient, so where both ends of 2^-21 around it give
// the same code that is the answer; otherwise, and where 1 / s may overflow,
// the division decides.
__device__ __forceinline__ uint2 f8_codes(const uint32_t r[4], float s) {
  const float inv = __frcp_rn(s);
  bool sure = s > 1e-30f;
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x = __fmul_rn(bf16lo(r[e]), inv), y = __fmul_rn(bf16hi(r[e]), inv);
    c[e] = f8x2(fmaf(x, 0x1p-21f, x), fmaf(y, 0x1p-21f, y));
    sure &= c[e] == f8x2(fmaf(x, -0x1p-21f, x), fmaf(y, -0x1p-21f, y));
  }
  if (!sure) {
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = f8x2(__fdiv_rn(bf16lo(r[e]), s), __fdiv_rn(bf16hi(r[e]), s));
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// 8 inputs k .. of a row, zeros at and past K
__device__ __forceinline__ void load8(const __nv_bfloat16* src, int k, int K, int vec, uint32_t r[4]) {
  r[0] = r[1] = r[2] = r[3] = 0u;
  if (vec && k + 8 <= K) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (k + e < K) r[e >> 1] |= (uint32_t) * reinterpret_cast<const unsigned short*>(src + e) << (16 * (e & 1));
  }
}
// the block's scale, from the 16 lanes that hold it (all 16 take part)
__device__ __forceinline__ float block_scale16(const uint32_t r[4]) {
  float a = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) a = fmaxf(a, fmaxf(fabsf(bf16lo(r[e])), fabsf(bf16hi(r[e]))));
  const unsigned int half = 0xFFFFu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(half, a, o));
  return a > 0.f ? __fmul_rn(a, 1.0f / 448.0f) : 1.0f;
}

// A kernel of its own in front of the tensor-core tiles: 16 groups of 16 lanes,
// kQIter tokens each, whose loads are in flight together.  HBM bound for many
// tokens (2 bytes read, 1 written per input).
constexpr int kQIter = 2, kQTokens = 16 * kQIter;

__global__ void __launch_bounds__(256) f8_quantize_kernel(const __nv_bfloat16* __restrict__ x, long long stride, int T,
                                                          int K, int kb, int tpad, int vec, uint8_t* __restrict__ xq,
                                                          float* __restrict__ sx) {
  pdl_launch_dependents();
  const int b = blockIdx.y, l = threadIdx.x & 15;
  const int k = b * kF8Block + 8 * l;
  const int t0 = blockIdx.x * kQTokens + (threadIdx.x >> 4);
  uint32_t r[kQIter][4];
#pragma unroll
  for (int i = 0; i < kQIter; ++i)
    if (t0 + 16 * i < T) load8(x + (t0 + 16 * i) * stride + k, k, K, vec, r[i]);
#pragma unroll
  for (int i = 0; i < kQIter; ++i) {
    const long long t = t0 + 16 * i;
    if (t >= T) break;  // whole 16-lane groups: only they shuffle together
    const float s = block_scale16(r[i]);
    *reinterpret_cast<uint2*>(xq + t * ((long long)kb * kF8Block) + k) = f8_codes(r[i], s);
    if (l == 0) sx[(long long)b * tpad + t] = s;
  }
}

// ---------------------------------------------------------------- 1..8 tokens
// A CTA takes groups of 16 outputs, grid strided, and deals the blocks of K to
// its 8 warps: w, w + 8, ...; a warp keeps kU of them in flight (4 x 16 bytes
// per lane each), each replaced as soon as it is used, across groups too.  Lane
// (g, c) = (lane / 4, lane % 4) loads codes 16 c .. + 15 of each half block of
// rows g and g + 8; the K order inside the MMAs is a permutation of the 64
// codes, the same for weights and tokens.
//
// The CTAs of a cluster (one, or two where there is much to do) quantise the
// tokens into the shared memory of each while their first weights are on their
// way: one launch.  Where the tokens' codes do not fit there (FUSED false), the
// kernel above has left them in global memory.
constexpr int kGemvRows = 16, kGemvWarps = 8, kU = 4;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// the shared memory of CTA `rank` of the cluster, at this CTA's address
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

template <bool FUSED>
__global__ void __launch_bounds__(kGemvWarps * 32, 2) f8_gemv_kernel(const F8Params p) {
  __shared__ float red[kGemvWarps][32][4];
  extern __shared__ __align__(16) unsigned char gsm[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  if constexpr (FUSED) cluster_arrive();
  const int groups = (p.N + kGemvRows - 1) / kGemvRows;
  const size_t pitch = (size_t)p.kb * kF8Block;
  const uint8_t* wr = p.w + (size_t)g * pitch + 16 * c;  // the padded rows exist
  uint4 a[kU][2], b[kU][2];
  auto load = [&](int u, int grp, int kb) {
    if (grp >= groups || kb >= p.kb) return;
    const uint8_t* wa = wr + (size_t)grp * kGemvRows * pitch + (size_t)kb * kF8Block;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      a[u][h] = ldg_stream(wa + 64 * h);
      b[u][h] = ldg_stream(wa + 8 * pitch + 64 * h);
    }
  };
  // the tokens: row pitch in bytes (half a bank row off a multiple of 128), scales [kb][T]
  const int row = (int)pitch + 64;
  float* ssx = reinterpret_cast<float*>(gsm + (size_t)p.T * row);
  const int tg = min(g, p.T - 1), t0 = min(2 * c, p.T - 1), t1 = min(2 * c + 1, p.T - 1);  // past T: results dropped
  // quantisation: kQ pairs of token and block at a time per 16 lanes
  constexpr int kQ = 3;
  const int l = threadIdx.x & 15, pairs = FUSED ? p.T * p.kb : 0;
  const int ctas = FUSED ? (int)cluster_ctas() : 1, step = 16 * ctas;
  int qi = (threadIdx.x >> 4) + (FUSED ? 16 * (int)cluster_rank() : 0), qt = qi / p.kb, qb = qi - qt * p.kb;
  const int dt = step / p.kb, db = step - dt * p.kb;
  uint32_t qr[kQ][4];
  int at[kQ], as[kQ];
  auto fetch = [&] {
#pragma unroll
    for (int q = 0; q < kQ; ++q) {
      at[q] = -1;
      qr[q][0] = qr[q][1] = qr[q][2] = qr[q][3] = 0u;
      if (qi < pairs) {
        const int k = qb * kF8Block + 8 * l;
        load8(p.x + qt * p.x_stride + k, k, p.K, p.x_vec, qr[q]);
        at[q] = qt * row + k;
        as[q] = p.T * row + 4 * (qb * p.T + qt);
      }
      qi += step, qt += dt, qb += db;
      if (qb >= p.kb) qb -= p.kb, ++qt;
    }
  };
  if constexpr (FUSED) fetch();  // before the weights: they would wait behind them
#pragma unroll
  for (int u = 0; u < kU; ++u) load(u, blockIdx.x, warp + kGemvWarps * u);

  if constexpr (FUSED) {
    cluster_wait();  // every CTA of the cluster runs
    while (true) {
      float qs[kQ];
      uint2 codes[kQ];
#pragma unroll
      for (int q = 0; q < kQ; ++q) qs[q] = block_scale16(qr[q]);  // side by side: nothing leaves the loop early
#pragma unroll
      for (int q = 0; q < kQ; ++q) codes[q] = f8_codes(qr[q], qs[q]);
#pragma unroll
      for (int q = 0; q < kQ; ++q) {
        if (at[q] < 0) continue;
        for (int k = 0; k < ctas; ++k) {
          const uint32_t base = cluster_map(smem_u32(gsm), (uint32_t)k);
          asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" :: "r"(base + at[q]), "r"(codes[q].x), "r"(codes[q].y)
                       : "memory");
          if (l == 0) asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(base + as[q]), "f"(qs[q]) : "memory");
        }
      }
      if (qi >= pairs) break;
      fetch();
    }
    __syncwarp();  // the halves of a warp may leave after different rounds
    cluster_arrive();
    cluster_wait();
  } else {
    pdl_wait();  // the tokens' codes and scales
  }
  const uint8_t* xg = p.xq + (size_t)tg * pitch + 16 * c;
  const unsigned char* xs = gsm + (size_t)tg * row + 16 * c;

  for (int grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const float* sw = p.sw + (size_t)(grp * kGemvRows / kF8Block) * p.kb;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int b0 = warp; b0 < p.kb; b0 += kGemvWarps * kU) {
      // what follows this batch: the row's next blocks, or the next group's first
      const bool more = b0 + kGemvWarps * kU < p.kb;
      const int ngrp = more ? grp : grp + (int)gridDim.x, nb0 = more ? b0 + kGemvWarps * kU : warp;
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int kb = b0 + kGemvWarps * u;
        if (kb < p.kb) {
          float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};  // two chains of products
          uint32_t xp[2][4], pa[2][4], pb[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 xv;
            if constexpr (FUSED)
              xv = *reinterpret_cast<const uint4*>(xs + kb * kF8Block + 64 * h);
            else
              xv = __ldcg(reinterpret_cast<const uint4*>(xg + (size_t)kb * kF8Block + 64 * h));
            xp[h][0] = xv.x, xp[h][1] = xv.y, xp[h][2] = xv.z, xp[h][3] = xv.w;
            pa[h][0] = a[u][h].x, pa[h][1] = a[u][h].y, pa[h][2] = a[u][h].z, pa[h][3] = a[u][h].w;
            pb[h][0] = b[u][h].x, pb[h][1] = b[u][h].y, pb[h][2] = b[u][h].z, pb[h][3] = b[u][h].w;
          }
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mma_16816(d[h][0], d[h][1], d[h][2], d[h][3], f8x2_to_f16x2(pa[h][m]), f8x2_to_f16x2(pb[h][m]),
                        f8x2_to_f16x2(pa[h][m] >> 16), f8x2_to_f16x2(pb[h][m] >> 16), f8x2_to_f16x2(xp[h][m]),
                        f8x2_to_f16x2(xp[h][m] >> 16), d[h][0], d[h][1], d[h][2], d[h][3]);
          float sx0, sx1;
          if constexpr (FUSED) {
            sx0 = ssx[kb * p.T + t0], sx1 = ssx[kb * p.T + t1];
          } else {
            sx0 = __ldcg(p.sx + (size_t)kb * p.tpad + t0), sx1 = __ldcg(p.sx + (size_t)kb * p.tpad + t1);
          }
          const float s = __ldg(sw + kb);
          acc[0] = fmaf(d[0][0] + d[1][0], s * sx0, acc[0]);
          acc[1] = fmaf(d[0][1] + d[1][1], s * sx1, acc[1]);
          acc[2] = fmaf(d[0][2] + d[1][2], s * sx0, acc[2]);
          acc[3] = fmaf(d[0][3] + d[1][3], s * sx1, acc[3]);
        }
        load(u, ngrp, nb0 + kGemvWarps * u);
      }
    }
    *reinterpret_cast<float4*>(red[warp][lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    // thread (token, row): consecutive threads write consecutive outputs
    const int i = threadIdx.x;
    if (i < 8 * kGemvRows) {
      const int tok = i / kGemvRows, r = i % kGemvRows;
      const int n = grp * kGemvRows + r;
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
    __syncthreads();
  }
}

// ---------------------------------------------------------------- tensor-core tiles
constexpr int kF8Scales = 16;
template <int BN>
struct F8Cfg {
  static constexpr int kStageA = kF8TileM * kF8Block;  // 16 KB
  static constexpr int kStageB = BN * kF8Block;
  static constexpr int kStages = BN >= 256 ? 4 : BN >= 128 ? 6 : 8;
  static constexpr int kScaleOff = kStages * (kStageA + kStageB);  // the tokens' scales of kF8Scales blocks
  static constexpr int kBarOff = kScaleOff + kF8Scales * kF8TileM * 4;
  static constexpr int kSmem = 1024 + kBarOff + 256;
  static_assert(kStages + 3 <= kF8Scales, "a block's scales are read after its stage may be filled again");
  static constexpr int kTmemCols = 2 * BN;
};
constexpr int kF8EpiWarps = 16;
constexpr int kF8Threads = (kF8EpiWarps + 2) * 32;

__device__ __forceinline__ void tc_mma_f8(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, {%5, %5, %5, %5}, p;\n\t}"
      :: "r"(tmem), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(0));
}
// true in one lane of a whole warp, always the same
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
template <typename E>
__device__ __forceinline__ E to_out(float x) {
  if constexpr (sizeof(E) == 2)
    return __float2bfloat16_rn(x);
  else
    return x;
}
// P lanes with P pieces of 16 bytes each: lane i gets every lane's piece i
template <int P>
__device__ __forceinline__ void exchange(uint4 v[P]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = P / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (i & o) continue;
      const uint4 x = up ? v[i] : v[i | o];
      const uint4 y = make_uint4(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o),
                                 __shfl_xor_sync(0xffffffffu, x.z, o), __shfl_xor_sync(0xffffffffu, x.w, o));
      if (up)
        v[i] = y;
      else
        v[i | o] = y;
    }
  }
}
// A warp's 32 rows x COLS accumulators (a row per lane) to rows row0 .., columns n0 ..
// of the output.  Lanes exchange pieces first, so that a store writes whole lines
// of a few rows: a row per lane, a 256 x 256 tile's stores took 3.6 us.
template <typename E, int COLS>
__device__ __forceinline__ void store_tile(const F8Params& p, const float* acc, int row0, int n0) {
  constexpr int PE = 16 / sizeof(E), ALL = COLS / PE, P = ALL < 8 ? ALL : 8;  // elements of a piece, pieces of a row
  const int lane = threadIdx.x & 31;
  E* out = static_cast<E*>(p.out);
  if (!p.vec) {
    if (row0 + lane < p.T) {
#pragma unroll
      for (int j = 0; j < COLS; ++j)
        if (n0 + j < p.N) out[(size_t)(row0 + lane) * p.out_stride + n0 + j] = to_out<E>(acc[j]);
    }
    return;
  }
#pragma unroll
  for (int g = 0; g < ALL; g += P) {
    uint4 v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float* x = acc + (g + i) * PE;
      if constexpr (sizeof(E) == 2) {
        __nv_bfloat162 r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
        v[i] = *reinterpret_cast<const uint4*>(r);
      } else {
        v[i] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
      }
    }
    exchange<P>(v);
    const int n = n0 + (g + (lane & (P - 1))) * PE;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int row = row0 + (lane & ~(P - 1)) + j;
      if (row >= p.T) continue;
      E* dst = out + (size_t)row * p.out_stride + n;
      if (n + PE <= p.N) {
        *reinterpret_cast<uint4*>(dst) = v[j];
      } else {
        const E* e = reinterpret_cast<const E*>(&v[j]);
#pragma unroll
        for (int i = 0; i < PE; ++i)
          if (n + i < p.N) dst[i] = e[i];
      }
    }
  }
}

// N consecutive columns of this warp's 32 TMEM lanes, here when it returns
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  if constexpr (N == 32) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]),
          "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(taddr));
  } else if constexpr (N == 16) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
          "=f"(v[14]), "=f"(v[15])
                 : "r"(taddr));
  } else {
    static_assert(N == 8, "8, 16 or 32 columns");
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
          "=f"(v[7])
                 : "r"(taddr));
  }
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // not used before the wait
}

}  // namespace

// The order of the tiles: bands of kF8Band token tiles, inside a band the token
// tile fastest, so that the CTAs at work at one time share both their tokens
// and their weights.  Bands of 4, 8 and 16 take the same time within the run's noise at 16 to
// 8192 tokens x 2560 to 8192 outputs x 1024 to 8192 inputs (8192 x 8192 x 4096: 356, 357
// and 355 us); all token tiles in one band took an eighth longer.
constexpr int kF8Band = 8;
__device__ __forceinline__ void tile_place(const F8Params& p, int tile, int& m, int& n) {
  const int per = kF8Band * p.tiles_n, band = tile / per, in = tile - band * per;
  const int rows = min(kF8Band, p.tiles_m - band * kF8Band);
  m = band * kF8Band + in % rows;
  n = in / rows;
}

// Warps 0-15 promote and store (TMEM lanes 32 (w % 4).., column quarter w / 4),
// warp 16 issues the TMA loads, warp 17 the MMAs.  Every role walks the tiles
// blockIdx.x, + gridDim.x, ...
// (256 x 256 tiles over the two CTAs of a cluster, which read a third less, were
// slower by a twentieth, in one run, at 8192 x 8192 x 4096.  A buffer's way from the
// MMAs to the promotion and back takes longer between two CTAs, and it is what
// bounds the loop.)
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
  float* sX = reinterpret_cast<float*>(smem + C::kScaleOff);
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
    // a warp's columns, and those it reads at once (a thread of 18 warps has 96 registers)
    constexpr int COLS = BN / 4, CH = COLS == 64 ? 16 : COLS;
    const int q = warp & 3, part = warp >> 2;
    const uint32_t tb = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(part * COLS);
    int it = 0;  // K blocks so far: buffer it % 2
    bool ok = true;
    for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
      int tm, tn;
      tile_place(p, tile, tm, tn);
      const int m0 = tm * kF8TileM, n0 = tn * BN + part * COLS;
      // the weights' scales of 32 blocks, one per lane, loaded 32 blocks ahead
      const float* sw = p.sw + (size_t)min(n0 / kF8Block, (p.N - 1) / kF8Block) * p.kb;
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
      float sw_now = 0.f, sw_next = lane < p.kb ? __ldg(sw + lane) : 0.f;
#pragma unroll 1
      for (int kb = 0; kb < p.kb; ++kb, ++it) {
        const int b = it & 1;
        if ((kb & 31) == 0) {
          sw_now = sw_next;
          if (kb + 32 + lane < p.kb) sw_next = __ldg(sw + kb + 32 + lane);
        }
        if (lane == 0) ok = tc_wait(&accf[b], (it >> 1) & 1, p.err, abort_flag, p.wait_ns);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
        const float s = sX[(it % kF8Scales) * kF8TileM + 32 * q + lane] * __shfl_sync(0xffffffffu, sw_now, kb & 31);
#pragma unroll
        for (int c = 0; c < COLS; c += CH) {
          float v[CH];
          tmem_ld<CH>(tb + b * BN + c, v);
          if (c + CH == COLS) {  // everything is read: the buffer may be overwritten
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acce[b]);
          }
#pragma unroll
          for (int j = 0; j < CH; ++j) acc[c + j] = fmaf(v[j], s, acc[c + j]);
        }
      }
      if (!ok) break;
      if (p.out_bf16)
        store_tile<__nv_bfloat16, COLS>(p, acc, m0 + 32 * q, n0);
      else
        store_tile<float, COLS>(p, acc, m0 + 32 * q, n0);
    }
  } else if (warp == kF8EpiWarps) {
    // (here and below the whole warp walks the loop and one lane issues, so that
    // addresses and descriptors stay in uniform registers)
    int g = 0;
    bool ok = (int)blockIdx.x != p.skip_cta;
    for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
      int tm, tn;
      tile_place(p, tile, tm, tn);
      const int m0 = tm * kF8TileM, n0 = tn * BN;
      const float* sx = p.sx + m0;  // rows up to tpad exist
#pragma unroll 1
      for (int kb = 0; kb < p.kb; ++kb, ++g) {
        const int s = g % S;
        ok = __all_sync(0xffffffffu, tc_wait(&empty[s], ((g / S) & 1) ^ 1, p.err, abort_flag, p.wait_ns));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&full[s], C::kStageA + C::kStageB + kF8TileM * 4);
          bulk_g2s(sX + (g % kF8Scales) * kF8TileM, sx + (size_t)kb * p.tpad, kF8TileM * 4, &full[s]);
          tma_load_2d(smem_u32(sA + s * C::kStageA), &tmX, kb * kF8Block, m0, &full[s]);
          tma_load_2d(smem_u32(sB + s * C::kStageB), &tmW, kb * kF8Block, n0, &full[s]);
        }
        __syncwarp();
      }
    }
    // after an abort, loads may still be landing: wait for every armed stage
    for (int i = g > S ? g - S : 0; i < g; ++i) mbar_wait(&full[i % S], (i / S) & 1, kTcWaitNs, p.err);
    __syncwarp();
  } else {
    // f32 accumulator; e4m3 is format 0, as f16 is in kind::f16
    const uint32_t idesc = make_idesc(BN);
    const uint64_t da = sw128_desc(smem_u32(sA)), db = sw128_desc(smem_u32(sB));
    int g = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < ntiles && ok; tile += gridDim.x) {
#pragma unroll 1
      for (int kb = 0; kb < p.kb; ++kb, ++g) {
        const int s = g % S, b = g & 1;
        ok = __all_sync(0xffffffffu, tc_wait(&full[s], (g / S) & 1, p.err, abort_flag, p.wait_ns) &&
                                         tc_wait(&acce[b], ((g >> 1) & 1) ^ 1, p.err, abort_flag, p.wait_ns));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          // descriptors count 16 bytes
          const uint64_t a0 = da + (uint64_t)(s * (C::kStageA >> 4)), b0 = db + (uint64_t)(s * (C::kStageB >> 4));
#pragma unroll
          for (int k4 = 0; k4 < kF8Block / 32; ++k4)
            tc_mma_f8(tmem + b * BN, a0 + 2 * k4, b0 + 2 * k4, idesc, k4 ? 1u : 0u);
          tc_commit(&empty[s]);
          tc_commit(&accf[b]);
        }
        __syncwarp();
      }
    }
    // no MMA may still be writing TMEM when it is freed (the lane that issued them commits)
    if (elect_one()) tc_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, kTcWaitNs, p.err);
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
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f8_gemv_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kF8GemvSmem);
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

cudaError_t launch_f8_gemv(const F8Params& p, int sms, bool fused, cudaStream_t s) {
  const int groups = (p.N + kGemvRows - 1) / kGemvRows;
  int grid = groups < 2 * sms ? groups : 2 * sms;
  if (!fused) return launch_dependent(f8_gemv_kernel<false>, grid, kGemvWarps * 32, 0, s, p);
  // Two CTAs share the quantisation where one alone would take more than a round
  // or two of loads: 8 tokens x 2560 inputs, 8192 outputs, 11.4 us (alone 14.5, four
  // 12.2, eight 12.6).  Over 1 to 8 tokens x 1024 to 8192 inputs that is the quicker choice or
  // within 0.5 us of it, but for exactly 64 pairs: one token x 8192 inputs takes 10.5 us
  // alone and 8.8 shared, two x 4096 11.4 and 9.2.
  const int cluster = p.T * p.kb > 64 && grid >= 2 ? 2 : 1;
  grid = (grid + cluster - 1) / cluster * cluster;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3(kGemvWarps * 32);
  c.dynamicSmemBytes = f8_gemv_smem(p.T, p.kb);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, f8_gemv_kernel<true>, p);
}

template <int BN>
static cudaError_t gemm_launch(const F8Maps& m, const F8Params& p, int tile, int ctas, cudaStream_t s) {
  return launch_dependent(f8_gemm_kernel<BN>, ctas, kF8Threads, F8Cfg<BN>::kSmem, s, m.x, m.w[tile], p);
}
cudaError_t launch_f8_gemm(const F8Maps& m, const F8Params& p, int tile, int ctas, cudaStream_t s) {
  switch (tile) {
    case 0: return gemm_launch<32>(m, p, tile, ctas, s);
    case 1: return gemm_launch<64>(m, p, tile, ctas, s);
    case 2: return gemm_launch<128>(m, p, tile, ctas, s);
    default: return gemm_launch<256>(m, p, tile, ctas, s);
  }
}

}  // namespace lingmoe

// Gated delta rule: the recurrence of the model's linear-attention layers.
//
// Per value head, with unit keys and queries (x / sqrt(sum x^2 + 1e-6)), a
// log-decay g <= 0 per channel (or per head), a write strength b and a state S
// [dk, dv] in fp32:
//   S <- diag(exp g_t) S;  u = b_t (v_t - S^T k_t);  S <- S + k_t u^T;
//   o_t = scale * S^T q_t.
//
// Step (1..8 tokens per sequence): delta_step_kernel, the recurrence as it
// stands with the state in registers.  HBM bound: the state read and written once.
//
// Prefill: chunks of 64 tokens.  With G the running sum of g inside a chunk,
//   A[i,j] = b_i sum_c k_i k_j exp(G_i - G_j)  (j < i),   T = (I + A)^-1,
//   B[i,j] = sum_c q_i k_j exp(G_i - G_j)      (j <= i),
//   X = v - (k exp G) S0,   U = (T diag(b)) X,
//   O = (q exp G) S0 + B U,   S1 = diag(exp G_last) S0 + (k exp(G_last - G))^T U.
// delta_prep_kernel forms, for every chunk and head at once, the operands
// that do not depend on the state; delta_scan_kernel walks a sequence's
// chunks with the state in registers.  Every decay is a product of factors
// exp(g) <= 1 between two tokens, never a quotient, so that no decay, however
// strong, overflows.
//
// Precision: products run on mma.sync with fp16 operands and fp32 sums.  What
// feeds the state (fp32) is split into two fp16 terms (22 bits) after a power-
// of-two scale taken from each 16-row block's largest value, three products
// per pair of split operands; what feeds only the bf16 output takes one fp16
// term (half a step 2^-11, the output's own being 2^-8).
#include "common.cuh"
#include "delta.h"

namespace lingmoe {

namespace {

constexpr float kOpScale = 1024.f;  // k, q, T and B operands are stored times 2^10
constexpr float kNormEps = 1e-6f;
constexpr unsigned long long kLandNs = 2000000000ull;

__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_a(uint32_t addr, uint32_t r[4]) { ldsm_x4(addr, r[0], r[1], r[2], r[3]); }
__device__ __forceinline__ void mma(float d[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
  mma_16816(d[0], d[1], d[2], d[3], a[0], a[1], a[2], a[3], b0, b1, d[0], d[1], d[2], d[3]);
}
__device__ __forceinline__ uint32_t pack_half2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// (x, y) -> fp16 pair hi and the fp16 pair of what it leaves
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_half2(x - f.x, y - f.y);
}
// The power of two that brings values up to m into [2^13, 2^14), and its inverse.
__device__ __forceinline__ void block_scale(float m, float& s, float& inv) {
  const int e = max(-100, (int)(__float_as_uint(m) >> 23) - 127);
  s = pow2_int(13 - e);
  inv = pow2_int(e - 13);
}
__device__ __forceinline__ float warp_max_abs(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// One warp: the sequence and place of chunk `chunk` (counted over all
// sequences in order), or false.  Boundaries outside [0, T] or out of order
// are clamped.
__device__ bool find_chunk(const DeltaParams& p, int chunk, int& seq, int& start, int& len) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    const int i = i0 + lane;
    int s = 0, e = 0;
    if (i < p.nseq) {
      s = clamp_int(p.cu[i], 0, p.T);
      e = clamp_int(p.cu[i + 1], s, p.T);
    }
    const int n = (e - s + kDeltaChunk - 1) / kDeltaChunk;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const int at = chunk - base - (x - n);
    const unsigned int who = __ballot_sync(0xffffffffu, at >= 0 && at < n);
    if (who) {
      const int l = __ffs(who) - 1;
      seq = i0 + l;
      start = __shfl_sync(0xffffffffu, s + at * kDeltaChunk, l);
      len = min(kDeltaChunk, __shfl_sync(0xffffffffu, e, l) - start);
      return true;
    }
    base += __shfl_sync(0xffffffffu, x, 31);
  }
  return false;
}
// One warp: sequence seq's first chunk, its tokens [start, end).
__device__ void find_sequence(const DeltaParams& p, int seq, int& first, int& start, int& end) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (int i = lane; i < seq; i += 32) {
    const int s = clamp_int(p.cu[i], 0, p.T), e = clamp_int(p.cu[i + 1], s, p.T);
    n += (e - s + kDeltaChunk - 1) / kDeltaChunk;
  }
  first = __reduce_add_sync(0xffffffffu, n);
  start = clamp_int(p.cu[seq], 0, p.T);
  end = clamp_int(p.cu[seq + 1], start, p.T);
}
// the sequence's row of the state pool, -1 for none
__device__ __forceinline__ int slot_of(const DeltaParams& p, int seq) {
  const int s = p.slots ? p.slots[seq] : seq;
  return s >= 0 && s < p.num_slots ? s : -1;
}

// N consecutive channels of a bf16 row as floats
template <int N>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* src, bool vec, float* x) {
  if (vec) {
    if constexpr (N == 4) {
      const uint2 r = *reinterpret_cast<const uint2*>(src);
      x[0] = bf16lo(r.x), x[1] = bf16hi(r.x), x[2] = bf16lo(r.y), x[3] = bf16hi(r.y);
    } else {
      const uint32_t r = *reinterpret_cast<const uint32_t*>(src);
      x[0] = bf16lo(r), x[1] = bf16hi(r);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = __bfloat162float(src[i]);
  }
}
// N consecutive channels' log-decays (one for all where there is one per head)
template <int N>
__device__ __forceinline__ void load_decay(const float* src, int per_channel, bool vec, float* x) {
  if (!per_channel) {
    const float g = *src;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = g;
  } else if (vec) {
    if constexpr (N == 4) {
      const float4 r = *reinterpret_cast<const float4*>(src);
      x[0] = r.x, x[1] = r.y, x[2] = r.z, x[3] = r.w;
    } else {
      const float2 r = *reinterpret_cast<const float2*>(src);
      x[0] = r.x, x[1] = r.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = src[i];
  }
}
// two floats in one register pair, and the same operation on both
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// exp(g), 1 for g > 0; a NaN stays one
__device__ __forceinline__ float decay_of(float g) { return expf(g > 0.f ? 0.f : g); }

// lane l gets the warp's sum of v[l]
__device__ __forceinline__ float transpose_sum32(float v[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float keep = up ? v[i + o] : v[i], send = up ? v[i] : v[i + o];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  return v[0];
}

}  // namespace

// ---------------------------------------------------------------- step
// A warp takes 16 columns of one head's state and all of its rows: lane (rg, cl)
// = (lane / 4, lane % 4) holds columns 4 cl.. of rows rg R .. + R - 1 in
// registers, so that no token needs more than its own warp.  Both products with
// the decayed state, S^T k and S^T q, are formed together, and S_new^T q =
// S^T q + (k . q) u.  The warps of a CTA share the tokens' unit keys and
// queries and their decays, which a warp per token prepares while the state is
// on its way from HBM.
constexpr int kStepCols = 16;  // state columns of a warp
// the place of channel c among a token's channels: R of them per row group, padded so
// that the eight row groups' 16-byte reads fall into different banks
template <int DK>
__host__ __device__ constexpr int step_at(int c) { return c + 4 * (c / (DK / 8)); }

template <int DK>
struct StepTokens {  // a head's tokens, prepared
  float k[kDeltaMaxStep][DK + 32], q[kDeltaMaxStep][DK + 32], a[kDeltaMaxStep][DK + 32];
  float v[kDeltaMaxStep][128];
  float beta[kDeltaMaxStep], kq[kDeltaMaxStep];
};
// what a lane loads of a token: CPL channels each of q, k and g, two or four of v
template <int DK>
struct StepRaw {
  float q[DK / 32], k[DK / 32], g[DK / 32], v[4], beta;
  __device__ __forceinline__ void load(const DeltaParams& p, int b, int h, int t, int lane) {
    constexpr int CPL = DK / 32;
    const int hk = h / (p.Hv / p.Hk);
    load_bf16<CPL>(p.q + b * p.q_b + t * p.q_t + hk * p.q_h + CPL * lane, p.vec_qk, q);
    load_bf16<CPL>(p.k + b * p.k_b + t * p.k_t + hk * p.k_h + CPL * lane, p.vec_qk, k);
    load_decay<CPL>(p.g + b * p.g_b + t * p.g_t + h * p.g_h + p.g_c * CPL * lane, p.g_c, p.vec_g, g);
    const __nv_bfloat16* vp = p.v + b * p.v_b + t * p.v_t + h * p.v_h + 2 * lane;
    load_bf16<2>(vp, p.vec_v, v);
    if (p.dv > 64) load_bf16<2>(vp + 64, p.vec_v, v + 2);
    beta = p.beta[b * p.be_b + t * p.be_t + h * p.be_h];
  }
  __device__ __forceinline__ void finish(StepTokens<DK>& s, int t, int lane) {
    *reinterpret_cast<float2*>(&s.v[t][2 * lane]) = make_float2(v[0], v[1]);
    *reinterpret_cast<float2*>(&s.v[t][2 * lane + 64]) = make_float2(v[2], v[3]);
    constexpr int CPL = DK / 32;
    float qq = 0.f, kk = 0.f, kq = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) qq += q[c] * q[c], kk += k[c] * k[c];
    const float rq = 1.f / sqrtf(warp_sum(qq) + kNormEps), rk = 1.f / sqrtf(warp_sum(kk) + kNormEps);
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int at = step_at<DK>(CPL * lane + c);
      q[c] *= rq;
      k[c] *= rk;
      kq += q[c] * k[c];
      s.q[t][at] = q[c];
      s.k[t][at] = k[c];
      s.a[t][at] = decay_of(g[c]);
    }
    kq = warp_sum(kq);
    if (lane == 0) {
      s.kq[t] = kq;
      s.beta[t] = beta;
    }
  }
};
template <int DK>
__host__ __device__ constexpr int step_smem(int dv, bool ahead) {
  return (ahead ? 2 * (int)sizeof(StepTokens<DK>) + DK * dv * 4 : (int)sizeof(StepTokens<DK>)) + 16;
}

// AHEAD: a CTA takes whole heads, blockIdx.x, + gridDim.x, ...; while it
// computes one, a bulk copy brings the next one's state to shared memory and
// its tokens come to registers.  Otherwise one item (a head or a part of its
// columns) per CTA.
template <int DK, bool AHEAD>
__global__ void __launch_bounds__(256, 2) delta_step_kernel(const DeltaParams p) {
  constexpr int R = DK / 8;
  extern __shared__ __align__(128) unsigned char dsm[];
  float* sstate = reinterpret_cast<float*>(dsm);
  StepTokens<DK>* tok = reinterpret_cast<StepTokens<DK>*>(dsm + (AHEAD ? DK * p.dv * 4 : 0));
  uint64_t* bar = reinterpret_cast<uint64_t*>(tok + (AHEAD ? 2 : 1));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int splits = AHEAD ? 1 : p.dv / (kStepCols * warps);
  const int items = AHEAD ? p.nseq * p.Hv : (int)gridDim.x;
  const int cl = lane & 3, rg = lane >> 2;
  const int n = p.T;
  int item = blockIdx.x;
  // the next item at or after `i` that has a slot
  auto find = [&](int i) {
    if constexpr (AHEAD)
      while (i < items && slot_of(p, i / p.Hv) < 0) i += gridDim.x;
    return i;
  };
  item = find(item);
  if (item >= items) return;
  int split = item % splits, h = item / splits % p.Hv, b = item / splits / p.Hv, slot = slot_of(p, b);
  if (slot < 0) return;
  const int col = (split * warps + warp) * kStepCols + 4 * cl;
  const size_t off = (size_t)rg * R * p.dv + col;  // this lane's first element of a head's state
  if (AHEAD && threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  f2 S[R / 2][4];  // rows 2 r, 2 r + 1 of each column
  auto take = [&](const float* sp) {
#pragma unroll
    for (int r = 0; r < R; r += 2) {
      const float4 x = *reinterpret_cast<const float4*>(sp + (size_t)r * p.dv);
      const float4 y = *reinterpret_cast<const float4*>(sp + (size_t)(r + 1) * p.dv);
      S[r / 2][0] = pack2(x.x, y.x), S[r / 2][1] = pack2(x.y, y.y), S[r / 2][2] = pack2(x.z, y.z), S[r / 2][3] = pack2(x.w, y.w);
    }
  };
  take(p.state + ((size_t)slot * p.Hv + h) * DK * p.dv + off);
  for (int t = warp; t < n; t += warps) {
    StepRaw<DK> raw;
    raw.load(p, b, h, t, lane);
    raw.finish(tok[0], t, lane);
  }
  bool dead = false;  // a wait ran out: the results are void
  uint32_t phase = 0;
  for (int turn = 0;; turn ^= 1) {
    __syncthreads();  // the item's tokens are prepared, its state is out of shared memory
    const StepTokens<DK>& s = tok[AHEAD ? turn : 0];
    int next = items, nh = 0, nb = 0, nslot = 0;
    StepRaw<DK> raw;
    if constexpr (AHEAD) {
      next = find(item + gridDim.x);
      if (next < items) {
        nh = next % p.Hv, nb = next / p.Hv, nslot = slot_of(p, nb);
        if (threadIdx.x == 0) {
          mbar_arrive_expect_tx(bar, DK * p.dv * 4);
          if (!p.skip) bulk_g2s(sstate, p.state + ((size_t)nslot * p.Hv + nh) * DK * p.dv, DK * p.dv * 4, bar);
        }
        if (warp < n) raw.load(p, nb, nh, warp, lane);
      }
    }
    const int commit = p.accepted ? clamp_int(p.accepted[b], 0, n) : n;
    __nv_bfloat16* op = p.out + ((size_t)b * n * p.Hv + h) * p.dv + col;
    float* sp = p.state + ((size_t)slot * p.Hv + h) * DK * p.dv + off;
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
      f2 w[8];  // S^T k of the four columns, then S^T q; even and odd rows apart
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0ull;
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const int at = step_at<DK>(R) * rg + r;
        const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(&s.a[t][at]);
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&s.k[t][at]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&s.q[t][at]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            f2& x = S[r / 2 + i][c];
            x = mul2(x, i ? a.y : a.x);
            w[c] = fma2(x, i ? k.y : k.x, w[c]);
            w[4 + c] = fma2(x, i ? q.y : q.x, w[4 + c]);
          }
      }
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 x = unpack2(w[i]);
        z[i] = x.x + x.y;
      }
      // the sums over the row groups: lane (rg, cl) is left with the sum of z[rg]
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) {
        const bool up = rg & o;
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const float keep = up ? z[i + o] : z[i], send = up ? z[i] : z[i + o];
          z[i] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * o);
        }
      }
      const float beta = s.beta[t];
      const float4 v4 = *reinterpret_cast<const float4*>(&s.v[t][col]);
      const float v[4] = {v4.x, v4.y, v4.z, v4.w};
      float u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = beta * (v[i] - __shfl_sync(0xffffffffu, z[0], 4 * i + cl));
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const ulonglong2 k = *reinterpret_cast<const ulonglong2*>(&s.k[t][step_at<DK>(R) * rg + r]);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) S[r / 2 + i][c] = fma2(i ? k.y : k.x, pack2(u[c], u[c]), S[r / 2 + i][c]);
      }
      if (rg >= 4) {  // S^T q of column rg - 4
        const float ui = rg == 4 ? u[0] : rg == 5 ? u[1] : rg == 6 ? u[2] : u[3];
        op[(size_t)t * p.Hv * p.dv + rg - 4] = __float2bfloat16_rn(p.scale * fmaf(s.kq[t], ui, z[0]));
      }
      if (t + 1 == commit) {
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          float2 x[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) x[c] = unpack2(S[r / 2][c]);
          *reinterpret_cast<float4*>(sp + (size_t)r * p.dv) = make_float4(x[0].x, x[1].x, x[2].x, x[3].x);
          *reinterpret_cast<float4*>(sp + (size_t)(r + 1) * p.dv) = make_float4(x[0].y, x[1].y, x[2].y, x[3].y);
        }
      }
    }
    if (!AHEAD || next >= items) break;
    if (warp < n) raw.finish(tok[turn ^ 1], warp, lane);
    for (int t = warp + warps; t < n; t += warps) {
      raw.load(p, nb, nh, t, lane);
      raw.finish(tok[turn ^ 1], t, lane);
    }
    if (!dead) dead = !mbar_wait(bar, phase, p.wait_ns, p.err);
    dead = __syncthreads_or(dead);
    if (dead) {  // a copy that is late must have landed before the CTA ends
      if (threadIdx.x == 0 && !p.skip) mbar_wait(bar, phase, kLandNs, p.err);
      return;
    }
    phase ^= 1;
    item = next, h = nh, b = nb, slot = nslot;
    take(sstate + off);
  }
}

// ---------------------------------------------------------------- prefill: operands of every chunk
// One CTA per chunk and head, one warp per 8 rows.  Decays inside an 8-row block
// are prefix products p and suffix products s of exp(g); t is the block's whole
// product.  A 16-row tile a of A and B meets the 8-column tiles before it
// through its own start: rows (k_i or q_i) p_i [x t of its first half], columns
// k_j s_j x (the t of the blocks between).  Its second half meets its first half
// through the border between them.  Only the 8 x 8 blocks on the diagonal are
// left; their pairs are summed directly from running products.
//
// The record of a chunk and head (layout: rows of 2 dk or 128 bytes, 16-byte
// pieces exchanged by piece ^= row % 8 for conflict-free ldmatrix):
//   k exp(G) hi, lo | q exp(G) | T diag(b) hi, lo | B | exp(G_last) fp32 |
//   k exp(G_last - G) hi, lo
template <int DK>
struct PrepCfg {
  static constexpr int kRow = DK * 2 + 16;      // bytes of a k or q row in shared memory
  static constexpr int kPRow = DK + 8;          // floats of a p or s row
  static constexpr int kMRow = 68;              // floats of a row of a 64 x 64 matrix
  static constexpr int kK = 0, kQ = kDeltaChunk * kRow;
  static constexpr int kP = 2 * kDeltaChunk * kRow;
  static constexpr int kS = kP + kDeltaChunk * kPRow * 4;
  static constexpr int kEnd = kS + kDeltaChunk * kPRow * 4;
  // the matrices take the place of the operands once the products are done
  static constexpr int kMat = kDeltaChunk * kMRow * 4;
  static constexpr int kT = kEnd > 3 * kMat ? kEnd : 3 * kMat;  // t [8][DK]
  static constexpr int kRk = kT + 8 * DK * 4, kRq = kRk + 256, kB = kRq + 256, kInfo = kB + 256;
  static constexpr int kSmem = kInfo + 32;
};

template <int DK>
__global__ void __launch_bounds__(256, 2) delta_prep_kernel(const DeltaParams p) {
  using C = PrepCfg<DK>;
  constexpr int CPL = DK / 32;
  extern __shared__ __align__(128) unsigned char dsm[];
  float* sp = reinterpret_cast<float*>(dsm + C::kP);
  float* ss = reinterpret_cast<float*>(dsm + C::kS);
  float* st = reinterpret_cast<float*>(dsm + C::kT);
  float* srk = reinterpret_cast<float*>(dsm + C::kRk);
  float* srq = reinterpret_cast<float*>(dsm + C::kRq);
  float* sbeta = reinterpret_cast<float*>(dsm + C::kB);
  int* info = reinterpret_cast<int*>(dsm + C::kInfo);
  float* mA = reinterpret_cast<float*>(dsm);
  float* mB = reinterpret_cast<float*>(dsm + C::kMat);
  float* mT = reinterpret_cast<float*>(dsm + 2 * C::kMat);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.y, hk = h / (p.Hv / p.Hk);
  if (warp == 0) {
    int seq = 0, start = 0, len = 0;
    const bool ok = find_chunk(p, p.seg0 + blockIdx.x, seq, start, len) && slot_of(p, seq) >= 0;
    if (lane == 0) {
      info[0] = ok ? len : 0;
      info[1] = start;
    }
  }
  __syncthreads();
  const int len = info[0], start = info[1];
  if (len == 0) return;
  unsigned char* rec = p.ws + ((size_t)blockIdx.x * p.Hv + h) * delta_rec_bytes(DK);

  // ---- this warp's 8 rows, CPL channels per lane
  const int row0 = 8 * warp, c0 = CPL * lane;
  float q[8][CPL], k[8][CPL], a[8][CPL];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = row0 + i;
    if (r < len) {
      const long long t = start + r;
      load_bf16<CPL>(p.q + t * p.q_t + hk * p.q_h + c0, p.vec_qk, q[i]);
      load_bf16<CPL>(p.k + t * p.k_t + hk * p.k_h + c0, p.vec_qk, k[i]);
      load_decay<CPL>(p.g + t * p.g_t + h * p.g_h + p.g_c * c0, p.g_c, p.vec_g, a[i]);
    } else {  // past the sequence: no key, no query, no decay
#pragma unroll
      for (int c = 0; c < CPL; ++c) q[i][c] = k[i][c] = a[i][c] = 0.f;
    }
  }
  if (lane < 8) {
    const int r = row0 + lane;
    sbeta[r] = r < len ? p.beta[(long long)(start + r) * p.be_t + h * p.be_h] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float qq = 0.f, kk = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) qq += q[i][c] * q[i][c], kk += k[i][c] * k[i][c];
    const float rq = 1.f / sqrtf(warp_sum(qq) + kNormEps), rk = 1.f / sqrtf(warp_sum(kk) + kNormEps);
    uint32_t kw[CPL / 2], qw[CPL / 2];
#pragma unroll
    for (int c = 0; c < CPL / 2; ++c) {  // back to the bf16 they came from: exact
      const __nv_bfloat162 kb = __floats2bfloat162_rn(k[i][2 * c], k[i][2 * c + 1]);
      const __nv_bfloat162 qb = __floats2bfloat162_rn(q[i][2 * c], q[i][2 * c + 1]);
      kw[c] = *reinterpret_cast<const uint32_t*>(&kb);
      qw[c] = *reinterpret_cast<const uint32_t*>(&qb);
    }
#pragma unroll
    for (int c = 0; c < CPL / 2; ++c) {
      *reinterpret_cast<uint32_t*>(dsm + C::kK + (row0 + i) * C::kRow + 2 * c0 + 4 * c) = kw[c];
      *reinterpret_cast<uint32_t*>(dsm + C::kQ + (row0 + i) * C::kRow + 2 * c0 + 4 * c) = qw[c];
    }
    if (lane == 0) {
      srk[row0 + i] = rk;
      srq[row0 + i] = rq;
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      k[i][c] *= rk;
      q[i][c] *= rq;
      a[i][c] = decay_of(a[i][c]);
    }
  }
  // prefix and suffix products of the block
  {
    float x[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) x[c] = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        x[c] *= a[i][c];
        sp[(row0 + i) * C::kPRow + c0 + c] = x[c];
      }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      st[warp * DK + c0 + c] = x[c];
      x[c] = 1.f;
    }
#pragma unroll
    for (int i = 7; i >= 0; --i)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        ss[(row0 + i) * C::kPRow + c0 + c] = x[c];
        x[c] *= a[i][c];
      }
  }
  // the pairs inside the block: entry i (i - 1) / 2 + j of each list for j < i,
  // then the q.k of equal rows (0-3 in the first list, 4-7 in the second)
  float dkk, dqk;
  {
    float vk[32], vq[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x[CPL], y = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        x[c] = k[j][c];
        y += q[j][c] * x[c];
      }
      if (j < 4)
        vk[28 + j] = y;
      else
        vq[24 + j] = y;
#pragma unroll
      for (int i = j + 1; i < 8; ++i) {
        float u = 0.f, w = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          x[c] *= a[i][c];
          u = fmaf(k[i][c], x[c], u);
          w = fmaf(q[i][c], x[c], w);
        }
        vk[i * (i - 1) / 2 + j] = u;
        vq[i * (i - 1) / 2 + j] = w;
      }
    }
    dkk = transpose_sum32(vk);
    dqk = transpose_sum32(vq);
  }
  __syncthreads();

  // ---- the operands that meet the state
  {
    float before[CPL], after[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) before[c] = after[c] = kOpScale;
    for (int w = 0; w < 8; ++w)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const float t = st[w * DK + c0 + c];
        if (w < warp) before[c] *= t;
        if (w > warp) after[c] *= t;
      }
    constexpr int KT = delta_tile_bytes(DK);
    unsigned char* khat = rec + 3 * KT + delta_ta_bytes(DK);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = row0 + i;
      const size_t at = (size_t)r * DK * 2 + (((2 * c0) >> 4) ^ (r & 7)) * 16 + ((2 * c0) & 15);
      float kt[CPL], qt[CPL], kh[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const float e = before[c] * sp[r * C::kPRow + c0 + c];
        kt[c] = k[i][c] * e;
        qt[c] = q[i][c] * e;
        kh[c] = k[i][c] * (after[c] * ss[r * C::kPRow + c0 + c]);
      }
#pragma unroll
      for (int c = 0; c < CPL; c += 2) {
        uint32_t hi, lo;
        split2(kt[c], kt[c + 1], hi, lo);
        *reinterpret_cast<uint32_t*>(rec + at + 2 * c) = hi;
        *reinterpret_cast<uint32_t*>(rec + KT + at + 2 * c) = lo;
        *reinterpret_cast<uint32_t*>(rec + 2 * KT + at + 2 * c) = pack_half2(qt[c], qt[c + 1]);
        split2(kh[c], kh[c + 1], hi, lo);
        *reinterpret_cast<uint32_t*>(khat + at + 2 * c) = hi;
        *reinterpret_cast<uint32_t*>(khat + KT + at + 2 * c) = lo;
      }
    }
    if (warp == 7) {  // nothing after the last block: exp(G_last) = before x its own product
      float* dec = reinterpret_cast<float*>(rec + 3 * KT + 3 * kDeltaChunk * kDeltaChunk * 2);
#pragma unroll
      for (int c = 0; c < CPL; ++c) dec[c0 + c] = before[c] * (1.f / kOpScale) * st[7 * DK + c0 + c];
    }
  }

  // ---- tile row a of A and B, half the channels per warp
  const int ta = warp & 3, hh = warp >> 2, gq = lane >> 2, tq = lane & 3;
  float accA[7][4], accB[7][4];
#pragma unroll
  for (int u = 0; u < 7; ++u)
#pragma unroll
    for (int e = 0; e < 4; ++e) accA[u][e] = accB[u][e] = 0.f;
  {
    const int r0 = 16 * ta + gq, r1 = r0 + 8;
    const float rk0 = srk[r0] * kOpScale, rk1 = srk[r1] * kOpScale, rq0 = srq[r0] * kOpScale, rq1 = srq[r1] * kOpScale;
#pragma unroll 1
    for (int ks = hh * (DK / 32); ks < (hh + 1) * (DK / 32); ++ks) {
      uint32_t Ah[4], Al[4], Aq[4], Rh[4], Rl[4], Rq[4];
      float D[2][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // channels 2 tq, + 1 and + 8, + 9
        const int c = 16 * ks + 8 * half + 2 * tq;
        const uint32_t k0 = *reinterpret_cast<const uint32_t*>(dsm + C::kK + r0 * C::kRow + 2 * c);
        const uint32_t k1 = *reinterpret_cast<const uint32_t*>(dsm + C::kK + r1 * C::kRow + 2 * c);
        const uint32_t q0 = *reinterpret_cast<const uint32_t*>(dsm + C::kQ + r0 * C::kRow + 2 * c);
        const uint32_t q1 = *reinterpret_cast<const uint32_t*>(dsm + C::kQ + r1 * C::kRow + 2 * c);
        const float2 p0 = *reinterpret_cast<const float2*>(sp + r0 * C::kPRow + c);
        const float2 p1 = *reinterpret_cast<const float2*>(sp + r1 * C::kPRow + c);
        const float2 t0 = *reinterpret_cast<const float2*>(st + 2 * ta * DK + c);
        D[half][0] = D[half][1] = 1.f;
        split2(bf16lo(k0) * rk0 * p0.x, bf16hi(k0) * rk0 * p0.y, Ah[2 * half], Al[2 * half]);
        Aq[2 * half] = pack_half2(bf16lo(q0) * rq0 * p0.x, bf16hi(q0) * rq0 * p0.y);
        const float kx = bf16lo(k1) * rk1 * p1.x, ky = bf16hi(k1) * rk1 * p1.y;
        const float qx = bf16lo(q1) * rq1 * p1.x, qy = bf16hi(q1) * rq1 * p1.y;
        split2(kx * t0.x, ky * t0.y, Ah[2 * half + 1], Al[2 * half + 1]);
        Aq[2 * half + 1] = pack_half2(qx * t0.x, qy * t0.y);
        split2(kx, ky, Rh[2 * half + 1], Rl[2 * half + 1]);
        Rq[2 * half + 1] = pack_half2(qx, qy);
        Rh[2 * half] = Rl[2 * half] = Rq[2 * half] = 0u;
      }
      // column tile s of 8 rows: u = 6 the tile row's own first half, else s = 2 ta - 1 - u
#pragma unroll
      for (int u = 6; u >= -1; --u) {
        if (u == -1) break;
        const int uu = u == 6 ? 6 : 5 - u;  // 6, then 0, 1, .. 5
        const int s = u == 6 ? 2 * ta : 2 * ta - 1 - uu;
        if (s >= 0) {
          const int j = 8 * s + gq;
          const float rk = srk[j] * kOpScale;
          uint32_t Bh[2], Bl[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int c = 16 * ks + 8 * half + 2 * tq;
            const uint32_t kj = *reinterpret_cast<const uint32_t*>(dsm + C::kK + j * C::kRow + 2 * c);
            const float2 sj = *reinterpret_cast<const float2*>(ss + j * C::kPRow + c);
            float x = bf16lo(kj) * rk * sj.x, y = bf16hi(kj) * rk * sj.y;
            if (u != 6) {
              const float2 t = *reinterpret_cast<const float2*>(st + s * DK + c);
              x *= D[half][0];
              y *= D[half][1];
              D[half][0] *= t.x;
              D[half][1] *= t.y;
            }
            split2(x, y, Bh[half], Bl[half]);
          }
          const uint32_t* ah = u == 6 ? Rh : Ah;
          const uint32_t* al = u == 6 ? Rl : Al;
          const uint32_t* aq = u == 6 ? Rq : Aq;
          mma(accA[uu], ah, Bh[0], Bh[1]);
          mma(accB[uu], aq, Bh[0], Bh[1]);
          mma(accA[uu], al, Bh[0], Bh[1]);
          mma(accA[uu], ah, Bl[0], Bl[1]);
        }
      }
    }
  }
  __syncthreads();  // the operands are read: the matrices take their place
  for (int i = tid; i < 3 * C::kMat / 16; i += 256) reinterpret_cast<float4*>(dsm)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  __syncthreads();
  constexpr float kUn = 1.f / (kOpScale * kOpScale);
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    if (hh == turn) {
#pragma unroll
      for (int uu = 0; uu < 7; ++uu) {
        const int s = uu == 6 ? 2 * ta : 2 * ta - 1 - uu;
        if (s < 0) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * ta + gq + (e >= 2 ? 8 : 0), c = 8 * s + 2 * tq + (e & 1);
          if (uu == 6 && e < 2) continue;
          mA[r * C::kMRow + c] += accA[uu][e] * (kUn * sbeta[r]);
          mB[r * C::kMRow + c] += accB[uu][e] * kUn;
        }
      }
    }
    if (turn == 0) {
      int i = 1, j;
      if (lane < 28) {
        while (i * (i + 1) / 2 <= lane) ++i;
        j = lane - i * (i - 1) / 2;
        mA[(row0 + i) * C::kMRow + row0 + j] = dkk * sbeta[row0 + i];
        mB[(row0 + i) * C::kMRow + row0 + j] = dqk;
      } else {
        i = row0 + lane - 28;
        mB[i * C::kMRow + i] = dkk;
        mB[(i + 4) * C::kMRow + i + 4] = dqk;
      }
    }
    __syncthreads();
  }

  // ---- T = (I + A)^-1: 16 x 16 blocks on the diagonal by substitution, one
  // column per lane, then the blocks below, diagonal by diagonal
  if (warp < 4 && lane < 16) {
    const int b = 16 * warp;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) y = fmaf(-mA[(b + i) * C::kMRow + b + m], x[m], y);
      x[i] = y;
      mT[(b + i) * C::kMRow + b + lane] = y;
    }
  }
  __syncthreads();
#pragma unroll 1
  for (int d = 1; d < 4; ++d) {
    // block (bi, bi - d): 64 threads, 4 columns each
    const int bi = d + (tid >> 6), bj = bi - d;
    const int i = (tid & 63) >> 2, j = 4 * (tid & 3);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    if (bi < 4) {
      for (int m = 16 * bj; m < 16 * bi; ++m) {
        const float x = mA[(16 * bi + i) * C::kMRow + m];
        const float4 t = *reinterpret_cast<const float4*>(mT + m * C::kMRow + 16 * bj + j);
        y.x = fmaf(x, t.x, y.x), y.y = fmaf(x, t.y, y.y), y.z = fmaf(x, t.z, y.z), y.w = fmaf(x, t.w, y.w);
      }
    }
    // A T of the block goes above the diagonal, to block (bj, bi), which nothing reads
    if (bi < 4) *reinterpret_cast<float4*>(mA + (16 * bj + i) * C::kMRow + 16 * bi + j) = y;
    __syncthreads();
    if (bi < 4) {
      y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const float x = -mT[(16 * bi + i) * C::kMRow + 16 * bi + m];
        const float4 t = *reinterpret_cast<const float4*>(mA + (16 * bj + m) * C::kMRow + 16 * bi + j);
        y.x = fmaf(x, t.x, y.x), y.y = fmaf(x, t.y, y.y), y.z = fmaf(x, t.z, y.z), y.w = fmaf(x, t.w, y.w);
      }
      *reinterpret_cast<float4*>(mT + (16 * bi + i) * C::kMRow + 16 * bj + j) = y;
    }
    __syncthreads();
  }
  // ---- T diag(b) and B to the record
  {
    const int r = tid >> 2;
    unsigned char* out = rec + 3 * delta_tile_bytes(DK);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int piece = 2 * (tid & 3) + half, c = 8 * piece;
      uint32_t hi[4], lo[4], bw[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 t = *reinterpret_cast<const float2*>(mT + r * C::kMRow + c + 2 * e);
        const float2 b = *reinterpret_cast<const float2*>(mB + r * C::kMRow + c + 2 * e);
        split2(t.x * sbeta[c + 2 * e] * kOpScale, t.y * sbeta[c + 2 * e + 1] * kOpScale, hi[e], lo[e]);
        bw[e] = pack_half2(b.x * kOpScale, b.y * kOpScale);
      }
      const size_t at = (size_t)r * 128 + ((piece ^ (r & 7)) * 16);
      *reinterpret_cast<uint4*>(out + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(out + 8192 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      *reinterpret_cast<uint4*>(out + 16384 + at) = make_uint4(bw[0], bw[1], bw[2], bw[3]);
    }
  }
}

// ---------------------------------------------------------------- prefill: the chain of chunks
// One CTA per sequence, head and 32 state columns, the state in the
// accumulators of its warps (warp w: rows 16 w ..).  Per chunk three products
// in a row, with a barrier after each operand has been written: X from the
// state, U from X, the new state from U; the output hangs beside them.  The
// records arrive by bulk copies ahead of use: the first piece (k exp G, q exp G)
// into one buffer that is free after X, the others into two buffers each.
template <int DK>
struct ScanCfg {
  static constexpr int kKq = 3 * delta_tile_bytes(DK);
  static constexpr int kTa = delta_ta_bytes(DK);
  static constexpr int kKh = 2 * delta_tile_bytes(DK);
  static constexpr int oKq = 0, oTa = kKq, oKh = oTa + 2 * kTa;
  static constexpr int kSt = DK * kDeltaCols * 2, kXt = kDeltaChunk * kDeltaCols * 2;
  static constexpr int oS = oKh + 2 * kKh, oX = oS + 2 * kSt, oU = oX + 2 * kXt;
  static constexpr int oSc = oU + 2 * kXt;           // scales: state [8], X [4][2], U [4][2]
  static constexpr int oBar = oSc + 24 * 4, oInfo = oBar + 5 * 8;
  static constexpr int kSmem = oInfo + 24;
};
// byte of (row, 16-byte piece) in a [rows][32] fp16 tile
__device__ __forceinline__ int tile32(int row, int piece) { return row * 64 + ((piece ^ ((row >> 1) & 3)) << 4); }

template <int DK>
__global__ void __launch_bounds__(256, 1) delta_scan_kernel(const DeltaParams p) {
  using C = ScanCfg<DK>;
  constexpr int NB = DK / 16;  // 16-row blocks of the state
  extern __shared__ __align__(128) unsigned char dsm[];
  float* sc_s = reinterpret_cast<float*>(dsm + C::oSc);
  float* sc_x = sc_s + 8;
  float* sc_u = sc_x + 8;
  uint64_t* bar = reinterpret_cast<uint64_t*>(dsm + C::oBar);  // kq, ta 0, ta 1, kh 0, kh 1
  int* info = reinterpret_cast<int*>(dsm + C::oInfo);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int splits = p.dv / kDeltaCols;
  const int split = blockIdx.x % splits, h = blockIdx.x / splits % p.Hv, seq = blockIdx.x / splits / p.Hv;
  if (warp == 0) {
    int first, start, end;
    find_sequence(p, seq, first, start, end);
    if (lane == 0) {
      info[0] = first, info[1] = start, info[2] = end, info[3] = slot_of(p, seq);
      for (int i = 0; i < 5; ++i) mbar_init(bar + i, 1);
      fence_mbar_init();
    }
  }
  __syncthreads();
  const int first = info[0], start = info[1], end = info[2], slot = info[3];
  const int chunks = (end - start + kDeltaChunk - 1) / kDeltaChunk;
  const int c0 = max(first, p.seg0), c1 = min(first + chunks, p.seg0 + p.seg_chunks);
  if (slot < 0 || c0 >= c1) return;
  const int n = c1 - c0;
  const unsigned char* rec0 = p.ws + ((size_t)(c0 - p.seg0) * p.Hv + h) * delta_rec_bytes(DK);
  const size_t rec_step = (size_t)p.Hv * delta_rec_bytes(DK);
  const bool copies = tid == 0 && !p.skip;
  auto issue_kq = [&](int c) {
    mbar_arrive_expect_tx(bar, C::kKq);
    bulk_g2s(dsm + C::oKq, rec0 + c * rec_step, C::kKq, bar);
  };
  auto issue_rest = [&](int c) {
    const int b = c & 1;
    mbar_arrive_expect_tx(bar + 1 + b, C::kTa);
    bulk_g2s(dsm + C::oTa + b * C::kTa, rec0 + c * rec_step + C::kKq, C::kTa, bar + 1 + b);
    mbar_arrive_expect_tx(bar + 3 + b, C::kKh);
    bulk_g2s(dsm + C::oKh + b * C::kKh, rec0 + c * rec_step + C::kKq + C::kTa, C::kKh, bar + 3 + b);
  };
  if (copies) {
    issue_kq(0);
    issue_rest(0);
    if (n > 1) issue_rest(1);
  }

  const int gq = lane >> 2, tq = lane & 3;
  const int col0 = split * kDeltaCols;
  float* sp = p.state + ((size_t)slot * p.Hv + h) * DK * p.dv + col0;
  float S[4][4];
  const bool zero = c0 == first && p.fresh && p.fresh[seq];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      float2 v = make_float2(0.f, 0.f);
      if (warp < NB && !zero)
        v = *reinterpret_cast<const float2*>(sp + (size_t)(16 * warp + gq + 8 * hi) * p.dv + 8 * nt + 2 * tq);
      S[nt][2 * hi] = v.x;
      S[nt][2 * hi + 1] = v.y;
    }
  const int ta = warp & 3, half = warp >> 2;  // row tile and column half of X, U and the output
  // v of rows 16 ta + gq (+ 8), columns 16 half + 8 nt + 2 tq; zeros past the sequence
  auto load_v = [&](int c, float v[2][4]) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi) {
        const int t = start + (c0 - first + c) * kDeltaChunk + 16 * ta + gq + 8 * hi;
        float x = 0.f, y = 0.f;
        if (t < end) {
          const __nv_bfloat16* src = p.v + (long long)t * p.v_t + h * p.v_h + col0 + 16 * half + 8 * nt + 2 * tq;
          if (p.vec_v) {
            const uint32_t r = *reinterpret_cast<const uint32_t*>(src);
            x = bf16lo(r);
            y = bf16hi(r);
          } else {
            x = __bfloat162float(src[0]);
            y = __bfloat162float(src[1]);
          }
        }
        v[nt][2 * hi] = x;
        v[nt][2 * hi + 1] = y;
      }
  };
  float v[2][4];
  load_v(0, v);
  bool dead = false;  // a wait ran out: no further waits, the results are void
  auto wait = [&](uint64_t* b, uint32_t parity) {
    if (!dead) dead = !mbar_wait(b, parity, p.wait_ns, p.err);
  };
  const uint32_t base = smem_u32(dsm);
  const int arow = 16 * ta + (lane & 15), apc = lane >> 4;  // ldmatrix rows and pieces of an A tile
  const int brow = lane & 15, bpc = 2 * half + (lane >> 4);  // of a B tile's 16 rows, this half's columns

#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    const int b = c & 1;
    // ---- the state as two fp16 terms
    if (warp < NB) {
      float m = 0.f;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(S[nt][e]));
      float s, inv;
      block_scale(warp_max_abs(m), s, inv);
      if (lane == 0) sc_s[warp] = inv * (1.f / kOpScale);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          uint32_t xh, xl;
          split2(S[nt][2 * hi] * s, S[nt][2 * hi + 1] * s, xh, xl);
          const int at = tile32(16 * warp + gq + 8 * hi, nt) + 4 * tq;
          *reinterpret_cast<uint32_t*>(dsm + C::oS + at) = xh;
          *reinterpret_cast<uint32_t*>(dsm + C::oS + C::kSt + at) = xl;
        }
    }
    __syncthreads();
    if (copies && c >= 1 && c + 1 < n) issue_rest(c + 1);
    wait(bar, c & 1);
    // ---- X = v - (k exp G) S, and (q exp G) S
    float X[2][4], O[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        X[nt][e] = v[nt][e];
        O[nt][e] = 0.f;
      }
#pragma unroll
    for (int ks = 0; ks < NB; ++ks) {
      uint32_t kh[4], kl[4], qh[4], sh[4], sl[4];
      const uint32_t aoff = base + C::oKq + arow * DK * 2 + (((2 * ks + apc) ^ (arow & 7)) << 4);
      ldsm_a(aoff, kh);
      ldsm_a(aoff + delta_tile_bytes(DK), kl);
      ldsm_a(aoff + 2 * delta_tile_bytes(DK), qh);
      const uint32_t boff = base + C::oS + tile32(16 * ks + brow, bpc);
      ldsm_x4_t(boff, sh);
      ldsm_x4_t(boff + C::kSt, sl);
      const float f = sc_s[ks];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float d[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
        mma(d, kh, sh[2 * nt], sh[2 * nt + 1]);
        mma(e, qh, sh[2 * nt], sh[2 * nt + 1]);
        mma(d, kl, sh[2 * nt], sh[2 * nt + 1]);
        mma(d, kh, sl[2 * nt], sl[2 * nt + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          X[nt][i] = fmaf(-f, d[i], X[nt][i]);
          O[nt][i] = fmaf(f, e[i], O[nt][i]);
        }
      }
    }
    // a 16 x 16 block (rows 16 ta.., this column half) to shared memory as two terms
    auto put = [&](const float x[2][4], int off, float* sc) {
      float m = 0.f;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(x[nt][e]));
      float s, inv;
      block_scale(warp_max_abs(m), s, inv);
      if (lane == 0) sc[2 * ta + half] = inv * (1.f / kOpScale);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int hi = 0; hi < 2; ++hi) {
          uint32_t xh, xl;
          split2(x[nt][2 * hi] * s, x[nt][2 * hi + 1] * s, xh, xl);
          const int at = tile32(16 * ta + gq + 8 * hi, 2 * half + nt) + 4 * tq;
          *reinterpret_cast<uint32_t*>(dsm + off + at) = xh;
          *reinterpret_cast<uint32_t*>(dsm + off + C::kXt + at) = xl;
        }
    };
    put(X, C::oX, sc_x);
    if (c + 1 < n) load_v(c + 1, v);
    __syncthreads();
    if (copies && c + 1 < n) issue_kq(c + 1);
    wait(bar + 1 + b, (c >> 1) & 1);
    // ---- U = T diag(b) X (T is lower triangular)
    float U[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) U[nt][e] = 0.f;
    const uint32_t toff = base + C::oTa + b * C::kTa + arow * 128;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks > ta) continue;
      uint32_t th[4], tl[4], xh[4], xl[4];
      ldsm_a(toff + (((2 * ks + apc) ^ (arow & 7)) << 4), th);
      ldsm_a(toff + 8192 + (((2 * ks + apc) ^ (arow & 7)) << 4), tl);
      const uint32_t boff = base + C::oX + tile32(16 * ks + brow, bpc);
      ldsm_x4_t(boff, xh);
      ldsm_x4_t(boff + C::kXt, xl);
      const float f = sc_x[2 * ks + half];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma(d, th, xh[2 * nt], xh[2 * nt + 1]);
        mma(d, tl, xh[2 * nt], xh[2 * nt + 1]);
        mma(d, th, xl[2 * nt], xl[2 * nt + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) U[nt][i] = fmaf(f, d[i], U[nt][i]);
      }
    }
    put(U, C::oU, sc_u);
    __syncthreads();
    wait(bar + 3 + b, (c >> 1) & 1);
    // ---- S = diag(exp G_last) S + (k exp(G_last - G))^T U
    if (warp < NB) {
      const float* dec = reinterpret_cast<const float*>(dsm + C::oTa + b * C::kTa + 3 * 8192);
      const float d0 = dec[16 * warp + gq], d1 = dec[16 * warp + gq + 8];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        S[nt][0] *= d0;
        S[nt][1] *= d0;
        S[nt][2] *= d1;
        S[nt][3] *= d1;
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t kh[4], kl[4];
        const int row = 16 * ks + (lane & 7) + ((lane & 16) >> 1);
        const uint32_t aoff =
            base + C::oKh + b * C::kKh + row * DK * 2 + (((2 * warp + ((lane >> 3) & 1)) ^ (row & 7)) << 4);
        ldsm_x4_t(aoff, kh);
        ldsm_x4_t(aoff + delta_tile_bytes(DK), kl);
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t uh[4], ul[4];
          const uint32_t boff = base + C::oU + tile32(16 * ks + brow, 2 * hf + (lane >> 4));
          ldsm_x4_t(boff, uh);
          ldsm_x4_t(boff + C::kXt, ul);
          const float f = sc_u[2 * ks + hf];
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            mma(d, kh, uh[2 * nt], uh[2 * nt + 1]);
            mma(d, kl, uh[2 * nt], uh[2 * nt + 1]);
            mma(d, kh, ul[2 * nt], ul[2 * nt + 1]);
#pragma unroll
            for (int i = 0; i < 4; ++i) S[2 * hf + nt][i] = fmaf(f, d[i], S[2 * hf + nt][i]);
          }
        }
      }
    }
    // ---- output: + B U (B is lower triangular with its diagonal)
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      if (ks > ta) continue;
      uint32_t bh[4], uh[4];
      ldsm_a(toff + 16384 + (((2 * ks + apc) ^ (arow & 7)) << 4), bh);
      ldsm_x4_t(base + C::oU + tile32(16 * ks + brow, bpc), uh);
      const float f = sc_u[2 * ks + half];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma(d, bh, uh[2 * nt], uh[2 * nt + 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) O[nt][i] = fmaf(f, d[i], O[nt][i]);
      }
    }
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int t = start + (c0 - first + c) * kDeltaChunk + 16 * ta + gq + 8 * hi;
      if (t < end) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          *reinterpret_cast<__nv_bfloat162*>(p.out + ((size_t)t * p.Hv + h) * p.dv + col0 + 16 * half + 8 * nt + 2 * tq) =
              __floats2bfloat162_rn(p.scale * O[nt][2 * hi], p.scale * O[nt][2 * hi + 1]);
      }
    }
  }
  // after a time-out copies may still be landing: wait for the last of each buffer
  if (copies && dead) {
    mbar_wait(bar, (n - 1) & 1, kLandNs, p.err);
    for (int c = max(0, n - 2); c < n; ++c) {
      mbar_wait(bar + 1 + (c & 1), (c >> 1) & 1, kLandNs, p.err);
      mbar_wait(bar + 3 + (c & 1), (c >> 1) & 1, kLandNs, p.err);
    }
  }
  if (warp < NB) {
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int hi = 0; hi < 2; ++hi)
        *reinterpret_cast<float2*>(sp + (size_t)(16 * warp + gq + 8 * hi) * p.dv + 8 * nt + 2 * tq) =
            make_float2(S[nt][2 * hi], S[nt][2 * hi + 1]);
  }
}

// ---------------------------------------------------------------- host
template <int DK>
static cudaError_t setup_dk() {
  cudaError_t e = cudaFuncSetAttribute(delta_prep_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       PrepCfg<DK>::kSmem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(delta_step_kernel<DK, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             step_smem<DK>(128, true));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(delta_scan_kernel<DK>, cudaFuncAttributeMaxDynamicSharedMemorySize, ScanCfg<DK>::kSmem);
  return e;
}
cudaError_t setup_delta() {
  const cudaError_t e = setup_dk<64>();
  return e != cudaSuccess ? e : setup_dk<128>();
}

template <int DK, bool AHEAD>
static void step_launch(const DeltaParams& p, unsigned grid, int warps, cudaStream_t s) {
  delta_step_kernel<DK, AHEAD><<<grid, 32 * warps, step_smem<DK>(p.dv, AHEAD), s>>>(p);
}
// More heads than CTAs fit at once: whole heads with the next one's state on its
// way.  Otherwise one item per CTA, a part of a head's columns where whole heads
// would leave SMs without work.
cudaError_t launch_delta_step(const DeltaParams& p, int dk, int sms, cudaStream_t s) {
  const long long heads = (long long)p.nseq * p.Hv;
  int warps = p.dv / kStepCols;
  const int fit = sms * 16 / warps;  // 16 warps per SM (registers)
  if (heads > fit) {
    if (dk == 64)
      step_launch<64, true>(p, (unsigned)fit, warps, s);
    else
      step_launch<128, true>(p, (unsigned)fit, warps, s);
    return cudaGetLastError();
  }
  while (warps > 2 && heads * (p.dv / kStepCols / warps) < 2ll * sms) warps /= 2;
  const unsigned grid = (unsigned)(heads * (p.dv / kStepCols / warps));
  if (dk == 64)
    step_launch<64, false>(p, grid, warps, s);
  else
    step_launch<128, false>(p, grid, warps, s);
  return cudaGetLastError();
}
cudaError_t launch_delta_prep(const DeltaParams& p, int dk, cudaStream_t s) {
  const dim3 grid((unsigned)p.seg_chunks, (unsigned)p.Hv);
  if (dk == 64)
    delta_prep_kernel<64><<<grid, 256, PrepCfg<64>::kSmem, s>>>(p);
  else
    delta_prep_kernel<128><<<grid, 256, PrepCfg<128>::kSmem, s>>>(p);
  return cudaGetLastError();
}
cudaError_t launch_delta_scan(const DeltaParams& p, int dk, cudaStream_t s) {
  const unsigned grid = (unsigned)p.nseq * p.Hv * (p.dv / kDeltaCols);
  if (dk == 64)
    delta_scan_kernel<64><<<grid, 256, ScanCfg<64>::kSmem, s>>>(p);
  else
    delta_scan_kernel<128><<<grid, 256, ScanCfg<128>::kSmem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace lingmoe

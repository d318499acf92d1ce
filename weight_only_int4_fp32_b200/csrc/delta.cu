// Gated delta rule: the recurrence of the model's linear-attention layers.
//
// Per value head, with unit keys and queries (x / sqrt(sum x^2 + 1e-6)), a
// log-decay g <= 0 per channel (or per head), a write strength b and a state S
// [dk, dv] in fp32:
//   S <- diag(exp g_t) S;  u = b_t (v_t - S^T k_t);  S <- S + k_t u^T;
//   o_t = scale * S^T q_t.
//
// Step (1..8 tokens per sequence): delta_step_kernel, the recurrence as it
// stands with the state in registers: the state read and written once.
//
// Prefill: chunks of 64 tokens.  With G the running sum of g inside a chunk,
//   A[i,j] = b_i sum_c k_i k_j exp(G_i - G_j)  (j < i),
//   B[i,j] = sum_c q_i k_j exp(G_i - G_j)      (j <= i),
//   (I + A) [W, U~] = diag(b) [k exp G, v],
//   U = U~ - W S0,
//   O = (q exp G) S0 + B U,   S1 = diag(exp G_last) S0 + (k exp(G_last - G))^T U.
// delta_prep_kernel forms, for every chunk and head at once, the operands
// that do not depend on the state; delta_scan_kernel walks a sequence's
// chunks with the state in registers.  Every decay is a product of factors
// exp(g) <= 1 between two tokens, never a quotient below 2^-16, so that no decay,
// however strong, overflows.
//
// A token's slowest decay, that of its largest log-decay over the channels, is
// shared by all of them: the operands hold what the channels decay beyond it, and
// the products of the slowest decays are fp32 factors of tokens, on the way into
// and out of the tensor cores (W and q: from the chunk's start; U: to its end; B:
// between its tokens; A, on U~'s side of the solution: through block borders).
// So what a chunk leaves of early writes or of its first state, however little
// that is where nothing is written after them, keeps its relative precision.
//
// Precision: products run on mma.sync with fp16 operands and fp32 sums.  What
// feeds the state (fp32) is split into two fp16 terms (22 bits) after a power-
// of-two scale taken from each row's largest value (fixed where the values are
// bounded: there the terms end at 2^-35), three products per pair of split operands; what
// feeds only the bf16 output takes one fp16 term (half a step 2^-11, the output's own
// being 2^-8; B's ends at 2^-35 too).
#include "common.cuh"
#include "delta.h"

namespace lingmoe {

namespace {

constexpr float kOpScale = 1024.f;  // operands that are 2 at most are stored times 2^10
// A 16-row block's slowest decays in all, below which U~ is solved for without dividing by them:
// of what is split after that division, the first rows keep 2^-38 / 2^-16 of the last ones.
constexpr float kSteep = 0x1p-16f;
constexpr uint32_t kLargeV = (127 + 100) << 7;  // bf16 2^100: such values are not divided by a decay either
constexpr float kTopScale = 8192.f;  // block_scale brings the largest value to 2^13 at least
constexpr float kNormEps = 1e-6f;
// A row whose sum of squares passes fp32 is taken times 2^-40, twice at most: 128 of the largest
// bf16 numbers, 2^88 and then 2^48, and the sum stays above 2^48, beside which the 1e-6 is nothing.
constexpr float kNormDown = 0x1p-40f;
constexpr int kNormPasses = 2;
constexpr unsigned long long kLandNs = 2000000000ull;

__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared.b64 _, [%0];" :: "r"(smem_u32(bar)) : "memory");
}
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

// the sequence's row of the state pool, -1 for none
__device__ __forceinline__ int slot_of(const DeltaParams& p, int seq) {
  const int s = p.slots ? p.slots[seq] : seq;
  return s >= 0 && s < p.num_slots ? s : -1;
}
// One warp, sequence i = a multiple of 32 + lane: its tokens [start, end).  A boundary
// counts as the largest of those up to it, each clamped to [0, T]: sequences never
// overlap, so that they have no more chunks than the host made room for.  `run` is the
// boundary before the 32 sequences, and then the one behind them.
__device__ __forceinline__ void scan_bounds(const DeltaParams& p, int i, int& run, int& start, int& end) {
  const int lane = threadIdx.x & 31;
  end = i < p.nseq ? clamp_int(p.cu[i + 1], 0, p.T) : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, end, o);
    if (lane >= o) end = max(end, y);
  }
  end = max(end, run);
  start = __shfl_up_sync(0xffffffffu, end, 1);
  if (lane == 0) start = run;
  run = __shfl_sync(0xffffffffu, end, 31);
}
__device__ __forceinline__ int chunks_of(int tokens) { return (tokens + kDeltaChunk - 1) / kDeltaChunk; }
// One warp: the place of chunk `chunk` (counted over all sequences in order) and
// its sequence's slot, or false.
__device__ bool find_chunk(const DeltaParams& p, int chunk, int& slot, int& start, int& len) {
  const int lane = threadIdx.x & 31;
  int base = 0, run = clamp_int(p.cu[0], 0, p.T);
  for (int i0 = 0; i0 < p.nseq; i0 += 32) {
    const int i = i0 + lane;
    int s, e;
    scan_bounds(p, i, run, s, e);
    const int sl = i < p.nseq ? slot_of(p, i) : -1;
    const int n = chunks_of(e - s);
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
      slot = __shfl_sync(0xffffffffu, sl, l);
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
  int n = 0, run = clamp_int(p.cu[0], 0, p.T);
  for (int i0 = 0;; i0 += 32) {
    int s, e;
    scan_bounds(p, i0 + lane, run, s, e);
    if (i0 + lane < seq) n += chunks_of(e - s);
    if (seq < i0 + 32) {
      start = __shfl_sync(0xffffffffu, s, seq - i0);
      end = __shfl_sync(0xffffffffu, e, seq - i0);
      break;
    }
  }
  first = __reduce_add_sync(0xffffffffu, n);
}
// N consecutive channels of a bf16 row, two to a word; converted apart from the
// load, so that a thread's loads are in flight together
template <int N>
__device__ __forceinline__ void load_bf16(const __nv_bfloat16* src, bool vec, uint32_t* r) {
  if (vec) {
    if constexpr (N == 4) {
      const uint2 x = *reinterpret_cast<const uint2*>(src);
      r[0] = x.x, r[1] = x.y;
    } else {
      r[0] = *reinterpret_cast<const uint32_t*>(src);
    }
  } else {
    const unsigned short* e = reinterpret_cast<const unsigned short*>(src);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) r[i] = e[2 * i] | (uint32_t)e[2 * i + 1] << 16;
  }
}
template <int N>
__device__ __forceinline__ void from_bf16(const uint32_t* r, float* x) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) x[2 * i] = bf16lo(r[i]), x[2 * i + 1] = bf16hi(r[i]);
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
// Many heads: 64 sequences x 4 tokens, 32 heads of 128 x 128, 65 us, 268 MB of states
// at 4.1 TB/s (32 columns per CTA with an exchange between its warps per token: 89 us;
// without packed arithmetic and the next head's state on its way: 86).  DRAM is at 42 %
// of its peak: a CTA's load, dependent tokens and stores follow one another,
// and two CTAs per SM do not fill the gaps.  One sequence, one token: 4.4 us on the device.
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
  uint32_t rq[DK / 64], rk[DK / 64], rv[2];
  float g[DK / 32], beta;
  __device__ __forceinline__ void load(const DeltaParams& p, int b, int h, int t, int lane) {
    constexpr int CPL = DK / 32;
    const int hk = h / (p.Hv / p.Hk);
    load_bf16<CPL>(p.q + b * p.q_b + t * p.q_t + hk * p.q_h + CPL * lane, p.vec_qk, rq);
    load_bf16<CPL>(p.k + b * p.k_b + t * p.k_t + hk * p.k_h + CPL * lane, p.vec_qk, rk);
    load_decay<CPL>(p.g + b * p.g_b + t * p.g_t + h * p.g_h + p.g_c * CPL * lane, p.g_c, p.vec_g, g);
    const __nv_bfloat16* vp = p.v + b * p.v_b + t * p.v_t + h * p.v_h + 2 * lane;
    load_bf16<2>(vp, p.vec_v, rv);
    rv[1] = 0u;
    if (p.dv > 64) load_bf16<2>(vp + 64, p.vec_v, rv + 1);
    beta = p.beta[b * p.be_b + t * p.be_t + h * p.be_h];
  }
  __device__ __forceinline__ void finish(StepTokens<DK>& s, int t, int lane) {
    *reinterpret_cast<float2*>(&s.v[t][2 * lane]) = make_float2(bf16lo(rv[0]), bf16hi(rv[0]));
    *reinterpret_cast<float2*>(&s.v[t][2 * lane + 64]) = make_float2(bf16lo(rv[1]), bf16hi(rv[1]));
    constexpr int CPL = DK / 32;
    float q[CPL], k[CPL];
    from_bf16<CPL>(rq, q);
    from_bf16<CPL>(rk, k);
    float qq, kk, kq = 0.f;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      qq = kk = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) qq += q[c] * q[c], kk += k[c] * k[c];
      qq = warp_sum(qq), kk = warp_sum(kk);
      if (pass == kNormPasses || !(qq == INFINITY || kk == INFINITY)) break;
      const float dq = qq == INFINITY ? kNormDown : 1.f, dk = kk == INFINITY ? kNormDown : 1.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) q[c] *= dq, k[c] *= dk;
    }
    const float rq = 1.f / sqrtf(qq + kNormEps), rk = 1.f / sqrtf(kk + kNormEps);
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
// (I + A) [W U~] = diag(b) [k exp(G), v] is then solved by 16-row blocks, the
// right sides transposed: a warp takes 16 of the 2 x 128 columns through all four
// blocks in registers (what a product leaves is the next one's operand), with the
// inverses of the diagonal blocks formed by substitution before.
//
// The record of a chunk and head: W^T hi, lo in the order of the B operands that
// it becomes | q exp(G) [64][dk] | k exp(G_last - G) hi, lo [64][dk] | B [64][64] |
// exp(G_last) fp32 [dk] | each token's slowest decays from the chunk's start [64] and
// to its end, times k's power of two [64] | U~^T fp32 in the order of the accumulators that take
// it.  W, q and k without the slowest decays.  fp16 rows have their 16-byte pieces
// exchanged, piece ^= row % 8, for conflict-free ldmatrix.
//
// 114 us for 1024 records of 128 x 128 heads (81 KB read, 124 KB written each): two
// CTAs per SM (shared memory; 128 registers, 200 bytes a thread spilled), whose own
// loads, dependent phases and instruction fetches (a long program, once per CTA) are
// what the time goes to, not a rate.  What keeps the precision of decayed writes is 16 us of it.
template <int DK>
struct PrepCfg {
  static constexpr int kFRow = DK + 8;            // floats of a row of k p or k s
  static constexpr int kHRow = DK * 2 + 16;       // bytes of a row of q p
  static constexpr int kVRow = 128 * 2 + 16;      // bytes of a row of v
  static constexpr int kMRow = 68;                // floats of a row of a 64 x 64 matrix
  static constexpr int kMat = kDeltaChunk * kMRow * 4;
  static constexpr int max2(int a, int b) { return a > b ? a : b; }
  static constexpr int oKp = 0;
  static constexpr int oKs = oKp + kDeltaChunk * kFRow * 4;
  static constexpr int oQ = oKs + max2(kDeltaChunk * kFRow * 4, 2 * kMat);
  static constexpr int oQ8 = oQ + max2(kDeltaChunk * kHRow, kDeltaChunk * kVRow);  // second halves of the tiles
  static constexpr int oT = oQ8 + kDeltaChunk / 2 * kHRow;                         // t [8][DK]
  static constexpr int oBefore = oT + 8 * DK * 4;                                  // [8][DK]
  static constexpr int oB = oBefore + 8 * DK * 4, oInfo = oB + 256;
  // the slowest channel's decays: each token's, their products from the start of its 8-row block
  // and behind it to the end, the blocks' whole; the same from the start of its 16-row
  // block, beta over that, and the powers of two of k's rows
  static constexpr int oE = oInfo + 32, oEp = oE + 256, oEs = oEp + 256, oP = oEs + 256, oBp = oP + 256;
  static constexpr int oEt = oBp + 256, oPk = oEt + 32;
  static constexpr int kSmem = oPk + 256;
  // once the products are done: A and B in place of k s, v in place of q p, then
  // A's blocks below the diagonal and the inverses on it as fp16 in place of B
  static constexpr int oA = oKs, oBm = oKs + kMat, oV = oQ, oA16 = oBm;
  static_assert(2 * kDeltaChunk * 128 <= kMat, "A as fp16 hi and lo");
};

// Four values of two rows (rows gq and gq + 8 of a 16 x 8 accumulator pair) as an
// A operand of two fp16 terms, each row times its scale
__device__ __forceinline__ void split_frag(const float x[4], const float y[4], float s0, float s1, uint32_t hi[4],
                                           uint32_t lo[4]) {
  split2(x[0] * s0, x[1] * s0, hi[0], lo[0]);
  split2(x[2] * s1, x[3] * s1, hi[1], lo[1]);
  split2(y[0] * s0, y[1] * s0, hi[2], lo[2]);
  split2(y[2] * s1, y[3] * s1, hi[3], lo[3]);
}
// an 8 x 8 tile of 16-bit values, rows and columns exchanged
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// the largest of a row, held by the four lanes of a quad
__device__ __forceinline__ float quad_max(float m) {
  m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
  return fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
}

// 16 columns of W or U~ (`tile`): one warp, from a CTA's shared memory to its record.  U~'s
// rows of a 16-row block are taken over the shared decay P from the block's start, and
// multiplied by that in the end.  Where P gets steep (STEEP, U~ only), the inverses on
// the diagonal, whose entries then fall with the decays as the rows of the result
// do where nothing is written, are applied in fp32 instead.
template <int DK, bool STEEP>
__device__ __forceinline__ void solve_tile(unsigned char* dsm, unsigned char* rec, int tile) {
  using C = PrepCfg<DK>;
  const int lane = threadIdx.x & 31, gq = lane >> 2, tq = lane & 3;
  const float* skp = reinterpret_cast<const float*>(dsm + C::oKp);
  const float* sbefore = reinterpret_cast<const float*>(dsm + C::oBefore);
  const float* sbeta = reinterpret_cast<const float*>(dsm + C::oB);
  const float* sEs = reinterpret_cast<const float*>(dsm + C::oEs);
  const float* sEt = reinterpret_cast<const float*>(dsm + C::oEt);
  const float* sP = reinterpret_cast<const float*>(dsm + C::oP);
  const float* sBp = reinterpret_cast<const float*>(dsm + C::oBp);
  const float* mA = reinterpret_cast<const float*>(dsm + C::oA);
  const uint32_t a16 = smem_u32(dsm + C::oA16);
  const int brow = (lane & 7) + ((lane >> 4) << 3), bpc = (lane >> 3) & 1;  // ldmatrix rows and pieces of a 16 x 16 block
  const bool is_w = !STEEP && tile < DK / 16;
  auto store_u = [&](int i, const float z[2][4]) {
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
      *reinterpret_cast<float4*>(rec + delta_ops_bytes(DK) + ((((tile - DK / 16) * 8 + 2 * i + nt) * 32 + lane) << 4)) =
          make_float4(z[nt][0], z[nt][1], z[nt][2], z[nt][3]);
  };
  const int c = 16 * (is_w ? tile : tile - DK / 16) + gq;  // column of rows 0, 1 of the accumulators; + 8 of 2, 3
  uint32_t fh[3][4], fl[3][4];
  float f[3][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float* scale = is_w || STEEP ? sbeta : sBp;
    float y[2][4];
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = 16 * i + 8 * nt + 2 * tq + (e & 1), cc = c + (e >= 2 ? 8 : 0);
        const float x = is_w ? skp[n * C::kFRow + cc] * sbefore[(2 * i + nt) * DK + cc]
                             : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(dsm + C::oV + n * C::kVRow + 2 * cc));
        y[nt][e] = x * scale[n];
      }
    uint32_t bh[4], bl[4];
#pragma unroll
    for (int j = 0; j < i; ++j) {
      const uint32_t at = a16 + (16 * i + brow) * 128 + (((2 * j + bpc) ^ (brow & 7)) << 4);
      ldsm_a(at, bh);
      ldsm_a(at + 8192, bl);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma(d, fh[j], bh[2 * nt], bh[2 * nt + 1]);
        mma(d, fl[j], bh[2 * nt], bh[2 * nt + 1]);
        mma(d, fh[j], bl[2 * nt], bl[2 * nt + 1]);
        if constexpr (STEEP) {
          const float2 r = *reinterpret_cast<const float2*>(sP + 16 * i + 8 * nt + 2 * tq);
          d[0] *= r.x, d[1] *= r.y, d[2] *= r.x, d[3] *= r.y;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) y[nt][e] = fmaf(-f[j][e >> 1], d[e], y[nt][e]);
      }
    }
    // the block's inverse times y, and the block as the next ones' operand
    float s0, s1, i0, i1, w[2][4];
    uint32_t oh[4], ol[4];
    if constexpr (STEEP) {
      float z[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) w[nt][e] = 0.f;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int o = 0; o < 4; ++o) {  // tokens 8 half + 2 o, + 1, which lane o of the quad holds
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = __shfl_sync(0xffffffffu, y[half][e], (lane & 28) | o);
#pragma unroll
          for (int nt = half; nt < 2; ++nt)
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float2 t = *reinterpret_cast<const float2*>(mA + (16 * i + 8 * nt + 2 * tq + b) * C::kMRow + 16 * i +
                                                                8 * half + 2 * o);
              w[nt][b] = fmaf(t.x, x[0], fmaf(t.y, x[1], w[nt][b]));
              w[nt][2 + b] = fmaf(t.x, x[2], fmaf(t.y, x[3], w[nt][2 + b]));
            }
        }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // decayed to the block's end
          const int n = 16 * i + 8 * nt + 2 * tq + (e & 1);
          z[nt][e] = w[nt][e];
          w[nt][e] *= sEs[n] * (nt ? 1.f : sEt[2 * i + 1]);
        }
      store_u(i, z);
    } else {
      uint32_t yh[4], yl[4];
      block_scale(quad_max(fmaxf(fmaxf(fabsf(y[0][0]), fabsf(y[0][1])), fmaxf(fabsf(y[1][0]), fabsf(y[1][1])))), s0, i0);
      block_scale(quad_max(fmaxf(fmaxf(fabsf(y[0][2]), fabsf(y[0][3])), fmaxf(fabsf(y[1][2]), fabsf(y[1][3])))), s1, i1);
      split_frag(y[0], y[1], s0, s1, yh, yl);
      const uint32_t at = a16 + (16 * i + brow) * 128 + (((2 * i + bpc) ^ (brow & 7)) << 4);
      ldsm_a(at, bh);
      ldsm_a(at + 8192, bl);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma(d, yh, bh[2 * nt], bh[2 * nt + 1]);
        mma(d, yl, bh[2 * nt], bh[2 * nt + 1]);
        mma(d, yh, bl[2 * nt], bl[2 * nt + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[nt][e] = d[e] * ((e >= 2 ? i1 : i0) * (1.f / kOpScale));
      }
      if (!is_w) {
        float z[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float2 r = *reinterpret_cast<const float2*>(sP + 16 * i + 8 * nt + 2 * tq);
          z[nt][0] = w[nt][0] * r.x, z[nt][1] = w[nt][1] * r.y, z[nt][2] = w[nt][2] * r.x, z[nt][3] = w[nt][3] * r.y;
        }
        store_u(i, z);
      }
    }
    if (is_w) {  // W's terms are the record's
      s0 = s1 = kOpScale;
      i0 = i1 = 1.f / kOpScale;
    } else {
      block_scale(quad_max(fmaxf(fmaxf(fabsf(w[0][0]), fabsf(w[0][1])), fmaxf(fabsf(w[1][0]), fabsf(w[1][1])))), s0, i0);
      block_scale(quad_max(fmaxf(fmaxf(fabsf(w[0][2]), fabsf(w[0][3])), fmaxf(fabsf(w[1][2]), fabsf(w[1][3])))), s1, i1);
    }
    split_frag(w[0], w[1], s0, s1, oh, ol);
    if (is_w) {  // 8 x 8 tiles turned: the B operand of 16 channels and tokens 16 i ..
      uint4* dst = reinterpret_cast<uint4*>(rec) + (tile * 4 + i) * 32 + lane;
      *dst = make_uint4(turn8(oh[0]), turn8(oh[1]), turn8(oh[2]), turn8(oh[3]));
      dst[delta_tile_bytes(DK) / 16] = make_uint4(turn8(ol[0]), turn8(ol[1]), turn8(ol[2]), turn8(ol[3]));
    }
    if (i < 3) {
#pragma unroll
      for (int m = 0; m < 4; ++m) fh[i][m] = oh[m], fl[i][m] = ol[m];
      // decayed to where the next block starts: this block's whole, unless that is in w
      const float t = is_w || STEEP ? 1.f : sP[16 * i + 15];
      f[i][0] = i0 * (1.f / kOpScale) * t;
      f[i][1] = i1 * (1.f / kOpScale) * t;
      if (!is_w) {
#pragma unroll
        for (int j = 0; j < i; ++j) f[j][0] *= sP[16 * i + 15], f[j][1] *= sP[16 * i + 15];
      }
    }
  }
}

template <int DK>
__global__ void __launch_bounds__(256, 2) delta_prep_kernel(const DeltaParams p) {
  using C = PrepCfg<DK>;
  constexpr int CPL = DK / 32;
  extern __shared__ __align__(128) unsigned char dsm[];
  float* skp = reinterpret_cast<float*>(dsm + C::oKp);
  float* sks = reinterpret_cast<float*>(dsm + C::oKs);
  float* st = reinterpret_cast<float*>(dsm + C::oT);
  float* sbefore = reinterpret_cast<float*>(dsm + C::oBefore);
  float* sbeta = reinterpret_cast<float*>(dsm + C::oB);
  int* info = reinterpret_cast<int*>(dsm + C::oInfo);
  float* sE = reinterpret_cast<float*>(dsm + C::oE);
  float* sEp = reinterpret_cast<float*>(dsm + C::oEp);
  float* sEs = reinterpret_cast<float*>(dsm + C::oEs);
  float* sEt = reinterpret_cast<float*>(dsm + C::oEt);
  float* sP = reinterpret_cast<float*>(dsm + C::oP);
  float* sBp = reinterpret_cast<float*>(dsm + C::oBp);
  float* spk = reinterpret_cast<float*>(dsm + C::oPk);
  float* mA = reinterpret_cast<float*>(dsm + C::oA);
  float* mB = reinterpret_cast<float*>(dsm + C::oBm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % p.Hv, hk = h / (p.Hv / p.Hk);
  pdl_launch_dependents();
  if (warp == 0) {
    int slot = -1, start = 0, len = 0;
    const bool ok = find_chunk(p, p.seg0 + (int)(blockIdx.x / p.Hv), slot, start, len) && slot >= 0;
    if (lane == 0) {
      info[0] = ok ? len : 0;
      info[1] = start;
    }
  }
  __syncthreads();
  const int len = info[0], start = info[1];
  // This kernel runs beside the scan before it, whose records are in the other
  // half of the workspace.  It ends after that scan: the next one starts from its
  // states, the next preparation writes to its half.
  const bool last = blockIdx.x == gridDim.x - 1;
  if (len == 0) {
    if (last) pdl_wait();
    return;
  }
  unsigned char* rec = p.ws + (size_t)blockIdx.x * delta_rec_bytes(DK, p.dv);
  if (tid < len) {  // v is used last: to L2 by then
    const char* row = reinterpret_cast<const char*>(p.v + (long long)(start + tid) * p.v_t + h * p.v_h);
    for (int i = 0; i < 2 * p.dv; i += 128) asm volatile("prefetch.global.L2 [%0];" :: "l"(row + i));
  }

  // ---- this warp's 8 rows, CPL channels per lane
  const int row0 = 8 * warp, c0 = CPL * lane;
  float q[8][CPL], k[8][CPL], a[8][CPL];
  {
    uint32_t rq[8][CPL / 2], rk[8][CPL / 2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = row0 + i;
      if (r < len) {
        const long long t = start + r;
        load_bf16<CPL>(p.q + t * p.q_t + hk * p.q_h + c0, p.vec_qk, rq[i]);
        load_bf16<CPL>(p.k + t * p.k_t + hk * p.k_h + c0, p.vec_qk, rk[i]);
        load_decay<CPL>(p.g + t * p.g_t + h * p.g_h + p.g_c * c0, p.g_c, p.vec_g, a[i]);
      } else {  // past the sequence: no key, no query, no decay
#pragma unroll
        for (int c = 0; c < CPL; ++c) rq[i][c / 2] = rk[i][c / 2] = 0u, a[i][c] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      from_bf16<CPL>(rq[i], q[i]);
      from_bf16<CPL>(rk[i], k[i]);
    }
  }
  if (lane < 8) {
    const int r = row0 + lane;
    sbeta[r] = r < len ? p.beta[(long long)(start + r) * p.be_t + h * p.be_h] : 0.f;
  }
  {
    // lanes 2 i and 2 i + 1: the sum of squares of query i, lanes 16 + 2 i and 17 + 2 i of key i
    float sum;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
      float n[16];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        n[i] = n[8 + i] = 0.f;
#pragma unroll
        for (int c = 0; c < CPL; ++c) n[i] = fmaf(q[i][c], q[i][c], n[i]), n[8 + i] = fmaf(k[i][c], k[i][c], n[8 + i]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        const bool up = lane & (2 * o);
#pragma unroll
        for (int i = 0; i < o; ++i) {
          const float keep = up ? n[i + o] : n[i], send = up ? n[i] : n[i + o];
          n[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * o);
        }
      }
      sum = n[0] + __shfl_xor_sync(0xffffffffu, n[0], 1);
      if (pass == kNormPasses || !__any_sync(0xffffffffu, sum == INFINITY)) break;
      const float down = sum == INFINITY ? kNormDown : 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float dq = __shfl_sync(0xffffffffu, down, 2 * i), dk = __shfl_sync(0xffffffffu, down, 16 + 2 * i);
#pragma unroll
        for (int c = 0; c < CPL; ++c) q[i][c] *= dq, k[i][c] *= dk;
      }
    }
    const float r = 1.f / sqrtf(sum + kNormEps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float rq = __shfl_sync(0xffffffffu, r, 2 * i), rk = __shfl_sync(0xffffffffu, r, 16 + 2 * i);
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        q[i][c] *= rq;
        k[i][c] *= rk;
      }
    }
    // each token's slowest decay (e^-200 is 0), and the channels' beyond it
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float m = INFINITY;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        a[i][c] = a[i][c] > 0.f ? 0.f : a[i][c];
        m = fminf(m, fabsf(a[i][c]));
      }
      const float slow = fminf(__uint_as_float(__reduce_min_sync(0xffffffffu, __float_as_uint(m))), 200.f);
      if (lane == i) mine = slow;
#pragma unroll
      for (int c = 0; c < CPL; ++c) a[i][c] = expf(a[i][c] + slow);
    }
    // lane i < 8: products of the slowest decays up to token i, and behind it
    const float e = expf(-mine);
    float ep = e, es = e;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float x = __shfl_up_sync(0xffffffffu, ep, o, 8), y = __shfl_down_sync(0xffffffffu, es, o, 8);
      if ((lane & 7) >= o) ep *= x;
      if ((lane & 7) + o < 8) es *= y;
    }
    es = __shfl_down_sync(0xffffffffu, es, 1, 8);
    if (lane < 8) {
      sE[row0 + lane] = e;
      sEp[row0 + lane] = ep;
      sEs[row0 + lane] = lane < 7 ? es : 1.f;
      if (lane == 7) sEt[warp] = ep;
    }
  }
  auto store_row = [&](float* dst, const float* x) {
    if constexpr (CPL == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[1]);
  };
  auto store_half = [&](unsigned char* dst, const float* x, float s) {
    if constexpr (CPL == 4)
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_half2(x[0] * s, x[1] * s), pack_half2(x[2] * s, x[3] * s));
    else
      *reinterpret_cast<uint32_t*>(dst) = pack_half2(x[0] * s, x[1] * s);
  };
  // k p and k s; the block's whole product; q p of a tile's second half (for its border)
  {
    float x[CPL], y[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) x[c] = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) x[c] *= a[i][c], y[c] = k[i][c] * x[c];
      store_row(skp + (row0 + i) * C::kFRow + c0, y);
      if (warp & 1) {
#pragma unroll
        for (int c = 0; c < CPL; ++c) y[c] = q[i][c] * x[c];
        store_half(dsm + C::oQ8 + (8 * (warp >> 1) + i) * C::kHRow + 2 * c0, y, kOpScale);
      }
    }
    store_row(st + warp * DK + c0, x);
#pragma unroll
    for (int c = 0; c < CPL; ++c) x[c] = 1.f;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
#pragma unroll
      for (int c = 0; c < CPL; ++c) y[c] = k[i][c] * x[c], x[c] *= a[i][c];
      store_row(sks + (row0 + i) * C::kFRow + c0, y);
    }
  }
  // the pairs inside the block: entry i (i - 1) / 2 + j of each list for j < i,
  // then the q.k of equal rows (0-3 in the first list, 4-7 in the second)
  float dkk, dqk;
  {
    float vk[32], vq[32];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f2 x[CPL / 2], y = 0ull;
#pragma unroll
      for (int c = 0; c < CPL / 2; ++c) {
        x[c] = pack2(k[j][2 * c], k[j][2 * c + 1]);
        y = fma2(pack2(q[j][2 * c], q[j][2 * c + 1]), x[c], y);
      }
      const float2 yy = unpack2(y);
      if (j < 4)
        vk[28 + j] = yy.x + yy.y;
      else
        vq[24 + j] = yy.x + yy.y;
#pragma unroll
      for (int i = j + 1; i < 8; ++i) {
        f2 u = 0ull, w = 0ull;
#pragma unroll
        for (int c = 0; c < CPL / 2; ++c) {
          x[c] = mul2(x[c], pack2(a[i][2 * c], a[i][2 * c + 1]));
          u = fma2(pack2(k[i][2 * c], k[i][2 * c + 1]), x[c], u);
          w = fma2(pack2(q[i][2 * c], q[i][2 * c + 1]), x[c], w);
        }
        const float2 uu = unpack2(u), ww = unpack2(w);
        vk[i * (i - 1) / 2 + j] = uu.x + uu.y;
        vq[i * (i - 1) / 2 + j] = ww.x + ww.y;
      }
    }
    dkk = transpose_sum32(vk);
    dqk = transpose_sum32(vq);
  }
  __syncthreads();

  // ---- the operands that meet the state, and q p of the tiles
  {
    float before[CPL], after[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) before[c] = after[c] = 1.f;
    for (int w = 0; w < 8; ++w)
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        const float t = st[w * DK + c0 + c];
        if (w < warp) before[c] *= t;
        if (w > warp) after[c] *= t;
      }
    store_row(sbefore + warp * DK + c0, before);
    float x[CPL], first[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      x[c] = 1.f;
      first[c] = warp & 1 ? st[(warp - 1) * DK + c0 + c] : 1.f;
    }
    constexpr int KT = delta_tile_bytes(DK);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = row0 + i;
      const size_t at = (size_t)r * DK * 2 + (((2 * c0) >> 4) ^ (r & 7)) * 16 + ((2 * c0) & 15);
      float qt[CPL], qp[CPL], kh[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        x[c] *= a[i][c];
        const float y = q[i][c] * x[c];
        qt[c] = y * before[c];
        qp[c] = y * first[c];
        kh[c] = after[c] * sks[r * C::kFRow + c0 + c];
      }
      store_half(dsm + C::oQ + r * C::kHRow + 2 * c0, qp, kOpScale);
      store_half(rec + 2 * KT + at, qt, kOpScale);
      // k's row is scaled by its largest value: what the channels decay beyond the slowest adds up
      float sk, ik, mk = 0.f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) mk = fmaxf(mk, fabsf(kh[c]));
      block_scale(warp_max_abs(mk), sk, ik);
      if (lane == 0) spk[r] = ik * kTopScale;
      uint32_t hi[CPL / 2], lo[CPL / 2];
#pragma unroll
      for (int c = 0; c < CPL / 2; ++c) split2(kh[2 * c] * sk, kh[2 * c + 1] * sk, hi[c], lo[c]);
      if constexpr (CPL == 4) {
        *reinterpret_cast<uint2*>(rec + 3 * KT + at) = make_uint2(hi[0], hi[1]);
        *reinterpret_cast<uint2*>(rec + 4 * KT + at) = make_uint2(lo[0], lo[1]);
      } else {
        *reinterpret_cast<uint32_t*>(rec + 3 * KT + at) = hi[0];
        *reinterpret_cast<uint32_t*>(rec + 4 * KT + at) = lo[0];
      }
    }
  }
  __syncthreads();
  // the record's factors, those of the solution
  if (tid < DK) {
    float* f = reinterpret_cast<float*>(rec + 5 * delta_tile_bytes(DK) + kDeltaChunk * kDeltaChunk * 2);
    float all = 1.f;
    if (tid < kDeltaChunk) {
      const int w = tid >> 3;
      float up = 1.f, down = 1.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float t = sEt[i];
        all *= t;
        if (i < w - (w & 1)) up *= t;
        if (i > w) down *= t;
      }
      const float x = sEp[tid] * (w & 1 ? sEt[w - 1] : 1.f);
      sP[tid] = x;
      sBp[tid] = sbeta[tid] / x;
      f[DK + tid] = x * up;
      f[DK + 64 + tid] = sEs[tid] * down * spk[tid];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) all *= sEt[i];
    }
    f[tid] = sbefore[7 * DK + tid] * st[7 * DK + tid] * all;
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
#pragma unroll 1
    for (int ks = hh * (DK / 32); ks < (hh + 1) * (DK / 32); ++ks) {
      uint32_t Ah[4], Al[4], Aq[4], Rh[4], Rl[4], Rq[4];
      float D[2][2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // channels 2 tq, + 1 and + 8, + 9
        const int c = 16 * ks + 8 * half + 2 * tq;
        const float2 k0 = *reinterpret_cast<const float2*>(skp + r0 * C::kFRow + c);
        const float2 k1 = *reinterpret_cast<const float2*>(skp + r1 * C::kFRow + c);
        const float2 t0 = *reinterpret_cast<const float2*>(st + 2 * ta * DK + c);
        D[half][0] = D[half][1] = kOpScale;
        const float kx = k1.x * kOpScale, ky = k1.y * kOpScale;
        split2(k0.x * kOpScale, k0.y * kOpScale, Ah[2 * half], Al[2 * half]);
        split2(kx * t0.x, ky * t0.y, Ah[2 * half + 1], Al[2 * half + 1]);
        split2(kx, ky, Rh[2 * half + 1], Rl[2 * half + 1]);
        Aq[2 * half] = *reinterpret_cast<const uint32_t*>(dsm + C::oQ + r0 * C::kHRow + 2 * c);
        Aq[2 * half + 1] = *reinterpret_cast<const uint32_t*>(dsm + C::oQ + r1 * C::kHRow + 2 * c);
        Rq[2 * half + 1] = *reinterpret_cast<const uint32_t*>(dsm + C::oQ8 + (8 * ta + gq) * C::kHRow + 2 * c);
        Rh[2 * half] = Rl[2 * half] = Rq[2 * half] = 0u;
      }
      // column tile s of 8 rows: unit 6 the tile row's own first half, else s = 2 ta - 1 - unit
#pragma unroll
      for (int n = 0; n < 7; ++n) {
        const int u = n == 0 ? 6 : n - 1;
        const int s = u == 6 ? 2 * ta : 2 * ta - 1 - u;
        if (s >= 0) {
          uint32_t Bh[2], Bl[2];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int c = 16 * ks + 8 * half + 2 * tq;
            float2 kj = *reinterpret_cast<const float2*>(sks + (8 * s + gq) * C::kFRow + c);
            kj.x *= D[half][0];
            kj.y *= D[half][1];
            if (u != 6) {
              const float2 t = *reinterpret_cast<const float2*>(st + s * DK + c);
              D[half][0] *= t.x;
              D[half][1] *= t.y;
            }
            split2(kj.x, kj.y, Bh[half], Bl[half]);
          }
          const uint32_t* ah = u == 6 ? Rh : Ah;
          const uint32_t* al = u == 6 ? Rl : Al;
          const uint32_t* aq = u == 6 ? Rq : Aq;
          mma(accA[u], ah, Bh[0], Bh[1]);
          mma(accB[u], aq, Bh[0], Bh[1]);
          mma(accA[u], al, Bh[0], Bh[1]);
          mma(accA[u], ah, Bl[0], Bl[1]);
        }
      }
    }
  }
  __syncthreads();  // the operands are read: the matrices and v take their place
  for (int i = tid; i < 2 * C::kMat / 16; i += 256) reinterpret_cast<float4*>(dsm + C::oA)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  uint32_t vmax = 0u;  // the largest |v| among this thread's, even and odd channels apart
  {
    uint32_t x[8][2];
#pragma unroll
    for (int n = 0; n < 8; ++n) {  // 256 threads x 8 x 4 values: dv = 128
      const int i = n * 256 + tid, r = i / (p.dv / 4), c = 4 * (i % (p.dv / 4));
      x[n][0] = x[n][1] = 0u;
      if (r < len) {
        const __nv_bfloat16* src = p.v + (long long)(start + r) * p.v_t + h * p.v_h + c;
        load_bf16<2>(src, p.vec_v, x[n]);
        load_bf16<2>(src + 2, p.vec_v, x[n] + 1);
      }
    }
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int i = n * 256 + tid, r = i / (p.dv / 4), c = 4 * (i % (p.dv / 4));
      if (r < kDeltaChunk) *reinterpret_cast<uint2*>(dsm + C::oV + r * C::kVRow + 2 * c) = make_uint2(x[n][0], x[n][1]);
      vmax = __vmaxu2(vmax, __vmaxu2(x[n][0] & 0x7FFF7FFFu, x[n][1] & 0x7FFF7FFFu));
    }
  }
  const bool large = __syncthreads_or((vmax & 0xFFFFu) >= kLargeV || (vmax >> 16) >= kLargeV);
  constexpr float kUn = 1.f / (kOpScale * kOpScale);
  {  // B's slowest decays: from the column to its block's end, from there to the row
    float d0 = sP[16 * ta + gq] * kUn, d1 = sP[16 * ta + gq + 8] * kUn;
#pragma unroll
    for (int u = 0; u < 7; ++u) {
      const int s = u == 6 ? 2 * ta : 2 * ta - 1 - u;
      if (s < 0) continue;
      const float2 x = *reinterpret_cast<const float2*>(sEs + 8 * s + 2 * tq);
      if (u == 6) d1 = sEp[16 * ta + gq + 8] * kUn;
      accB[u][0] *= d0 * x.x, accB[u][1] *= d0 * x.y, accB[u][2] *= d1 * x.x, accB[u][3] *= d1 * x.y;
      d0 *= sEt[s], d1 *= sEt[s];
    }
  }
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    if (hh == turn) {
#pragma unroll
      for (int u = 0; u < 7; ++u) {
        const int s = u == 6 ? 2 * ta : 2 * ta - 1 - u;
        if (s < 0) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * ta + gq + (e >= 2 ? 8 : 0), c = 8 * s + 2 * tq + (e & 1);
          if (u == 6 && e < 2) continue;
          mA[r * C::kMRow + c] += accA[u][e] * (kUn * sbeta[r]);
          mB[r * C::kMRow + c] += accB[u][e];
        }
      }
    }
    if (turn == 0) {
      int i = 1, j;
      if (lane < 28) {
        while (i * (i + 1) / 2 <= lane) ++i;
        j = lane - i * (i - 1) / 2;
        mA[(row0 + i) * C::kMRow + row0 + j] = dkk * sbeta[row0 + i];
        float d = dqk;
#pragma unroll
        for (int m = 1; m < 8; ++m) d *= j + m <= i ? sE[row0 + j + m] : 1.f;
        mB[(row0 + i) * C::kMRow + row0 + j] = d;
      } else {
        i = row0 + lane - 28;
        mB[i * C::kMRow + i] = dkk;
        mB[(i + 4) * C::kMRow + i + 4] = dqk;
      }
    }
    __syncthreads();
  }

  // ---- warps 0-3: the inverses of I + A's 16 x 16 diagonal blocks by substitution, a
  // column per lane, in the blocks' place; warps 4-7: B to the record
  if (warp < 4) {
    const int b = 16 * warp;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float y = i == lane ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) y = fmaf(-mA[(b + i) * C::kMRow + b + m], x[m], y);
      x[i] = y;
    }
    __syncwarp();
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) mA[(b + i) * C::kMRow + b + lane] = x[i];
    }
  } else {
    unsigned char* out = rec + 5 * delta_tile_bytes(DK);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int i = n * 128 + tid - 128, r = i >> 3, piece = i & 7;
      const float4 x = *reinterpret_cast<const float4*>(mB + r * C::kMRow + 8 * piece);
      const float4 y = *reinterpret_cast<const float4*>(mB + r * C::kMRow + 8 * piece + 4);
      *reinterpret_cast<uint4*>(out + r * 128 + ((piece ^ (r & 7)) << 4)) =
          make_uint4(pack_half2(x.x * kOpScale, x.y * kOpScale), pack_half2(x.z * kOpScale, x.w * kOpScale),
                     pack_half2(y.x * kOpScale, y.y * kOpScale), pack_half2(y.z * kOpScale, y.w * kOpScale));
    }
  }
  __syncthreads();
  // ---- A below the diagonal and the inverses on it as two fp16 terms
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int i = n * 256 + tid, r = i >> 3, piece = i & 7;
    const float4 x = *reinterpret_cast<const float4*>(mA + r * C::kMRow + 8 * piece);
    const float4 y = *reinterpret_cast<const float4*>(mA + r * C::kMRow + 8 * piece + 4);
    uint32_t hi[4], lo[4];
    split2(x.x * kOpScale, x.y * kOpScale, hi[0], lo[0]);
    split2(x.z * kOpScale, x.w * kOpScale, hi[1], lo[1]);
    split2(y.x * kOpScale, y.y * kOpScale, hi[2], lo[2]);
    split2(y.z * kOpScale, y.w * kOpScale, hi[3], lo[3]);
    unsigned char* dst = dsm + C::oA16 + r * 128 + ((piece ^ (r & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(dst + 8192) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();

  // ---- where a block's decay is steep, or values are too large to divide by it: the inverses times the decays between their tokens,
  // a row of a block and four of its columns per thread
  const bool steep = large || fminf(fminf(sP[15], sP[31]), fminf(sP[47], sP[63])) < kSteep;
  if (steep) {
    const int r = tid >> 2, c0 = (r & 48) + 4 * (tid & 3);
    float d = 0.f;
    for (int c = r; c >= c0; --c) {
      d = c == r ? 1.f : d * sE[c + 1];
      if (c < c0 + 4) mA[r * C::kMRow + c] *= d;
    }
    __syncthreads();
  }
  // ---- the solution, 16 columns at a time
#pragma unroll 1
  for (int tile = warp; tile < (DK + p.dv) / 16; tile += 8) {
    if (steep && tile >= DK / 16)
      solve_tile<DK, true>(dsm, rec, tile);
    else
      solve_tile<DK, false>(dsm, rec, tile);
  }
  if (last) pdl_wait();
}

// ---------------------------------------------------------------- prefill: the chain of chunks
// One CTA per sequence, head and 32 state columns; two warps per 16 columns.
// (64 columns per CTA read the records half as often, but a chunk then takes 4.5
// us in place of 2.5: worth it only where many sequences share a segment, and
// then by a tenth.)
// Everything is transposed, so that what one product leaves in its accumulators
// is the next one's A operand in the same registers:
//   U^T = U~^T - S^T W^T,  O^T = S^T (q exp G)^T + U^T B^T,
//   S^T = S^T diag(exp G_last) + U^T (k exp(G_last - G)).
// Of the pair, warp hf holds the channels' half hf of S^T and forms the tokens'
// half hf of U^T and O^T; the halves of S^T and U^T go to the other warp as
// operands through shared memory, with a barrier of the two each.  Operands are
// two fp16 terms, a power of two per state column and half.  One more warp
// brings the records, two ahead, by bulk copies.
// A chunk takes 2.4 us (32 chunks x 32 heads: 76 us alone), mma.sync at 56 % of its rate
// on each of the four schedulers; with a barrier of the whole CTA after each of three
// products, and the inverse applied here, it took 4.5.
constexpr int kScanTiles = 2;  // 16-column tiles per CTA

template <int DK>
struct ScanCfg {
  static constexpr int MT = kScanTiles;
  static constexpr int kWarps = 2 * MT;
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int kOps = delta_ops_bytes(DK);
  static constexpr int kKs = DK / 32;                      // 16-channel steps of a half
  static constexpr int kXS = 2 * kKs * 2 * 512;            // a column tile's S^T operand: halves, steps, terms
  static constexpr int kXU = 2 * 2 * 3 * 512;              // its U^T operands: to the chunk's end, two terms; as it is, one
  static constexpr int oX = 2 * kOps, oU = oX + MT * kXS;
  static constexpr int oFs = oU + MT * kXU, oFu = oFs + MT * 2 * 16 * 4;  // inverse scales [MT][half][16]
  static constexpr int oFb = oFu + MT * 2 * 16 * 4;
  static constexpr int oBar = oFb + MT * 2 * 16 * 4, oInfo = oBar + 4 * 8;
  static constexpr int kSmem = oInfo + 32;
  static_assert(kSmem <= 232448, "two records and the operands exceed 227 KB of shared memory");
};

template <int DK>
__global__ void __launch_bounds__(ScanCfg<DK>::kThreads, 1) delta_scan_kernel(const DeltaParams p) {
  using C = ScanCfg<DK>;
  constexpr int MT = C::MT, KS = C::kKs, NT = 2 * KS, KT = delta_tile_bytes(DK);
  extern __shared__ __align__(128) unsigned char dsm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(dsm + C::oBar);
  uint64_t* empty = full + 2;
  int* info = reinterpret_cast<int*>(dsm + C::oInfo);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int splits = p.dv / (16 * MT);
  const int split = blockIdx.x % splits, h = blockIdx.x / splits % p.Hv, seq = blockIdx.x / splits / p.Hv;
  if (warp == 0) {
    int first, start, end;
    find_sequence(p, seq, first, start, end);
    if (lane == 0) {
      info[0] = first, info[1] = start, info[2] = end, info[3] = slot_of(p, seq);
      for (int i = 0; i < 2; ++i) {
        mbar_init(full + i, 1);
        mbar_init(empty + i, C::kWarps);
      }
      fence_mbar_init();
    }
  }
  __syncthreads();
  // The records, and the states of the scan before.  Every CTA waits, those
  // without work too: the next preparation may start once all have passed.
  pdl_wait();
  pdl_launch_dependents();
  const int first = info[0], start = info[1], end = info[2], slot = info[3];
  const int chunks = chunks_of(end - start);
  const int c0 = max(first, p.seg0), c1 = min(first + chunks, p.seg0 + p.seg_chunks);
  if (slot < 0 || c0 >= c1) return;
  const int n = c1 - c0;
  const unsigned char* rec0 = p.ws + ((size_t)(c0 - p.seg0) * p.Hv + h) * delta_rec_bytes(DK, p.dv);
  const size_t rec_step = (size_t)p.Hv * delta_rec_bytes(DK, p.dv);

  if (warp == C::kWarps) {  // the records
    if (lane == 0 && !p.skip) {
      int c = 0;
      for (; c < n; ++c) {
        const int b = c & 1;
        if (c >= 2 && !mbar_wait(empty + b, ((c >> 1) & 1) ^ 1, p.wait_ns, p.err)) break;
        mbar_arrive_expect_tx(full + b, C::kOps);
        bulk_g2s(dsm + b * C::kOps, rec0 + c * rec_step, C::kOps, full + b);
      }
      // the CTA's shared memory stays until every copy has landed
      for (int i = max(0, c - 2); i < c; ++i) mbar_wait(full + (i & 1), (i >> 1) & 1, kLandNs, p.err);
    }
    return;
  }

  const int mt = warp >> 1, hf = warp & 1;
  const int gq = lane >> 2, tq = lane & 3;
  const int col = (split * MT + mt) * 16;  // state columns col .. + 15; this lane's col + gq and + 8
  float* sp = p.state + (((size_t)slot * p.Hv + h) * DK + hf * (DK / 2) + 2 * tq) * p.dv + col + gq;
  float S[NT][4];  // S^T: rows the columns, channels 8 nt + 2 tq, + 1 of the half
  const bool zero = c0 == first && p.fresh && p.fresh[seq];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[nt][e] = zero ? 0.f : sp[(size_t)(8 * nt + (e & 1)) * p.dv + (e >= 2 ? 8 : 0)];
  uint4* xs = reinterpret_cast<uint4*>(dsm + C::oX + mt * C::kXS);  // [half][step][term][lane]
  uint4* xu = reinterpret_cast<uint4*>(dsm + C::oU + mt * C::kXU);
  float* fs = reinterpret_cast<float*>(dsm + C::oFs) + mt * 32;
  float* fu = reinterpret_cast<float*>(dsm + C::oFu) + mt * 32;
  float* fb = reinterpret_cast<float*>(dsm + C::oFb) + mt * 32;
  auto pair_sync = [&] {
    __syncwarp();
    asm volatile("bar.sync %0, 64;" :: "r"(mt + 1) : "memory");
  };
  bool dead = false;  // a wait ran out: no further waits, the results are void
  // U~ of this warp's tokens: 4 tiles of 8
  const unsigned char* ut = rec0 + C::kOps + (((size_t)(split * MT + mt) * 8 + 4 * hf) * 32 + lane) * 16;
  float4 un[4];
#pragma unroll
  for (int nt = 0; nt < 4; ++nt) un[nt] = __ldcg(reinterpret_cast<const float4*>(ut + nt * 512));
  const uint32_t base = smem_u32(dsm);
  const int trow = (lane & 7) + (lane & 8), tpc = lane >> 4;                // ldmatrix.trans of a 16 (k) x 16 (n) block
  const int brow = (lane & 7) + ((lane >> 4) << 3), bpc = (lane >> 3) & 1;  // ldmatrix of a 16 (n) x 16 (k) block

#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    const int b = c & 1;
    const uint32_t ops = base + b * C::kOps;
    // exp(G_last) of the channels; of this half's tokens the factors of W and q, and of U
    const float* dec = reinterpret_cast<const float*>(dsm + b * C::kOps + 5 * KT + kDeltaChunk * kDeltaChunk * 2);
    const float* tokf = dec + DK + 32 * hf + 2 * tq;
    // ---- this half of S^T as operand
    {
      float m0 = 0.f, m1 = 0.f, s0, s1, i0, i1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        m0 = fmaxf(m0, fmaxf(fabsf(S[nt][0]), fabsf(S[nt][1])));
        m1 = fmaxf(m1, fmaxf(fabsf(S[nt][2]), fabsf(S[nt][3])));
      }
      block_scale(quad_max(m0), s0, i0);
      block_scale(quad_max(m1), s1, i1);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t hi[4], lo[4];
        split_frag(S[2 * ks], S[2 * ks + 1], s0, s1, hi, lo);
        xs[((hf * KS + ks) * 2 + 0) * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        xs[((hf * KS + ks) * 2 + 1) * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      if (tq == 0) {
        fs[hf * 16 + gq] = i0 * (1.f / kOpScale);
        fs[hf * 16 + gq + 8] = i1 * (1.f / kOpScale);
      }
    }
    pair_sync();
    // one answer for the warp: warp-wide instructions follow
    if (!dead) dead = !mbar_wait_warp(full + b, (c >> 1) & 1, p.wait_ns, p.err);
    // ---- U^T and the state's part of O^T for this half of the tokens: W S0 and q S0 first
    float U[4][4], O[4][4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      U[nt][0] = U[nt][1] = U[nt][2] = U[nt][3] = 0.f;
      O[nt][0] = O[nt][1] = O[nt][2] = O[nt][3] = 0.f;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float d[4][4], o[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[nt][e] = o[nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint4 h4 = xs[((half * KS + ks) * 2 + 0) * 32 + lane], l4 = xs[((half * KS + ks) * 2 + 1) * 32 + lane];
        const uint32_t ah[4] = {h4.x, h4.y, h4.z, h4.w}, al[4] = {l4.x, l4.y, l4.z, l4.w};
        uint32_t wh[2][4], wl[2][4], qh[2][4];
        const int kr = 16 * (half * KS + ks);
#pragma unroll
        for (int g = 0; g < 2; ++g) {  // 16 tokens
          const uint4* wat = reinterpret_cast<const uint4*>(dsm + b * C::kOps) + ((half * KS + ks) * 4 + 2 * hf + g) * 32 + lane;
          const uint4 x = wat[0], y = wat[KT / 16];
          wh[g][0] = x.x, wh[g][1] = x.y, wh[g][2] = x.z, wh[g][3] = x.w;
          wl[g][0] = y.x, wl[g][1] = y.y, wl[g][2] = y.z, wl[g][3] = y.w;
          const int qr = 32 * hf + 16 * g + brow;
          ldsm_a(ops + 2 * KT + qr * DK * 2 + (((kr / 8 + bpc) ^ (qr & 7)) << 4), qh[g]);
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma(d[nt], ah, wh[nt >> 1][2 * (nt & 1)], wh[nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma(o[nt], ah, qh[nt >> 1][2 * (nt & 1)], qh[nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma(d[nt], al, wh[nt >> 1][2 * (nt & 1)], wh[nt >> 1][2 * (nt & 1) + 1]);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma(d[nt], ah, wl[nt >> 1][2 * (nt & 1)], wl[nt >> 1][2 * (nt & 1) + 1]);
      }
      const float f0 = fs[half * 16 + gq], f1 = fs[half * 16 + gq + 8];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          U[nt][e] = fmaf(e >= 2 ? f1 : f0, d[nt][e], U[nt][e]);
          O[nt][e] = fmaf(e >= 2 ? f1 : f0, o[nt][e], O[nt][e]);
        }
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const float2 x = *reinterpret_cast<const float2*>(tokf + 8 * nt);
      U[nt][0] = fmaf(-x.x, U[nt][0], un[nt].x), U[nt][1] = fmaf(-x.y, U[nt][1], un[nt].y);
      U[nt][2] = fmaf(-x.x, U[nt][2], un[nt].z), U[nt][3] = fmaf(-x.y, U[nt][3], un[nt].w);
      O[nt][0] *= x.x, O[nt][1] *= x.y, O[nt][2] *= x.x, O[nt][3] *= x.y;
    }
    if (c + 1 < n) {
      ut += rec_step;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) un[nt] = __ldcg(reinterpret_cast<const float4*>(ut + nt * 512));
    }
    // ---- this half of U^T as operands: of the output as it is, of the state decayed to the end
    {
      float V[4][4], m[4] = {0.f, 0.f, 0.f, 0.f}, sc[4], inv[4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const float2 x = *reinterpret_cast<const float2*>(tokf + 64 + 8 * nt);
        V[nt][0] = U[nt][0] * x.x, V[nt][1] = U[nt][1] * x.y, V[nt][2] = U[nt][2] * x.x, V[nt][3] = U[nt][3] * x.y;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[e] = fmaxf(m[e], fmaxf(fabsf(V[nt][2 * e]), fabsf(V[nt][2 * e + 1])));
          m[2 + e] = fmaxf(m[2 + e], fmaxf(fabsf(U[nt][2 * e]), fabsf(U[nt][2 * e + 1])));
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) block_scale(quad_max(m[e]), sc[e], inv[e]);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        uint32_t hi[4], lo[4];
        split_frag(V[2 * ks], V[2 * ks + 1], sc[0], sc[1], hi, lo);
        xu[((hf * 2 + ks) * 3 + 0) * 32 + lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        xu[((hf * 2 + ks) * 3 + 1) * 32 + lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        const float* x = U[2 * ks];
        const float* y = U[2 * ks + 1];
        xu[((hf * 2 + ks) * 3 + 2) * 32 + lane] =
            make_uint4(pack_half2(x[0] * sc[2], x[1] * sc[2]), pack_half2(x[2] * sc[3], x[3] * sc[3]),
                       pack_half2(y[0] * sc[2], y[1] * sc[2]), pack_half2(y[2] * sc[3], y[3] * sc[3]));
      }
      if (tq == 0) {
        fu[hf * 16 + gq] = inv[0] * (1.f / kTopScale);
        fu[hf * 16 + gq + 8] = inv[1] * (1.f / kTopScale);
        fb[hf * 16 + gq] = inv[2] * (1.f / kOpScale);
        fb[hf * 16 + gq + 8] = inv[3] * (1.f / kOpScale);
      }
    }
    pair_sync();
    // ---- S^T of this half of the channels, O^T of this half of the tokens
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = *reinterpret_cast<const float2*>(dec + hf * (DK / 2) + 2 * tq + 8 * nt);
      S[nt][0] *= x.x, S[nt][1] *= x.y, S[nt][2] *= x.x, S[nt][3] *= x.y;
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float d[NT][4], o[4][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[nt][e] = 0.f;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const uint4 h4 = xu[((half * 2 + ks) * 3 + 0) * 32 + lane], l4 = xu[((half * 2 + ks) * 3 + 1) * 32 + lane];
        const uint32_t ah[4] = {h4.x, h4.y, h4.z, h4.w}, al[4] = {l4.x, l4.y, l4.z, l4.w};
        const int kr = 16 * (2 * half + ks);
        uint32_t kh[KS][4];
        const auto load_k = [&](uint32_t off) {
#pragma unroll
          for (int g = 0; g < KS; ++g)  // 16 channels
            ldsm_x4_t(ops + off + (kr + trow) * DK * 2 + (((hf * (DK / 16) + 2 * g + tpc) ^ (trow & 7)) << 4), kh[g]);
        };
        load_k(3 * KT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(d[nt], ah, kh[nt >> 1][2 * (nt & 1)], kh[nt >> 1][2 * (nt & 1) + 1]);
        if (half <= hf) {  // B is lower triangular
          const uint4 o4 = xu[((half * 2 + ks) * 3 + 2) * 32 + lane];
          const uint32_t ao[4] = {o4.x, o4.y, o4.z, o4.w};
          uint32_t bh[2][4];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int r = 32 * hf + 16 * g + brow;
            ldsm_a(ops + 5 * KT + r * 128 + (((kr / 8 + bpc) ^ (r & 7)) << 4), bh[g]);
          }
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) mma(o[nt], ao, bh[nt >> 1][2 * (nt & 1)], bh[nt >> 1][2 * (nt & 1) + 1]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(d[nt], al, kh[nt >> 1][2 * (nt & 1)], kh[nt >> 1][2 * (nt & 1) + 1]);
        load_k(4 * KT);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma(d[nt], ah, kh[nt >> 1][2 * (nt & 1)], kh[nt >> 1][2 * (nt & 1) + 1]);
      }
      const float f0 = fu[half * 16 + gq], f1 = fu[half * 16 + gq + 8];
      const float b0 = fb[half * 16 + gq], b1 = fb[half * 16 + gq + 8];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[nt][e] = fmaf(e >= 2 ? f1 : f0, d[nt][e], S[nt][e]);
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) O[nt][e] = fmaf(e >= 2 ? b1 : b0, o[nt][e], O[nt][e]);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(empty + b);  // the record is read
    __syncwarp();
    // ---- out: 8 x 8 tiles turned, so that a lane has two columns of one token
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      const int t = start + (c0 - first + c) * kDeltaChunk + 32 * hf + 8 * nt + gq;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(p.scale * O[nt][2 * r], p.scale * O[nt][2 * r + 1]);
        const uint32_t y = turn8(*reinterpret_cast<const uint32_t*>(&x));
        if (t < end)
          *reinterpret_cast<uint32_t*>(p.out + ((size_t)t * p.Hv + h) * p.dv + col + 8 * r + 2 * tq) = y;
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) sp[(size_t)(8 * nt + (e & 1)) * p.dv + (e >= 2 ? 8 : 0)] = S[nt][e];
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
  // what an SM holds: 16 warps (registers), 227 KB of shared memory
  const int smem = (dk == 64 ? step_smem<64>(p.dv, true) : step_smem<128>(p.dv, true)) + 1024;
  const int fit = sms * (16 / warps < 227 * 1024 / smem ? 16 / warps : 227 * 1024 / smem);
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
// launched while the kernel before it in the stream may still run (it waits for it itself)
static cudaError_t launch_dependent(void (*kernel)(DeltaParams), unsigned grid, int threads, int smem, bool dependent,
                                    cudaStream_t s, const DeltaParams& p) {
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, p);
}
// The first preparation of a call follows what is before it in the stream; the
// others run beside the scan before them.
cudaError_t launch_delta_prep(const DeltaParams& p, int dk, bool first, cudaStream_t s) {
  const unsigned grid = (unsigned)p.seg_chunks * p.Hv;
  if (dk == 64) return launch_dependent(delta_prep_kernel<64>, grid, 256, PrepCfg<64>::kSmem, !first, s, p);
  return launch_dependent(delta_prep_kernel<128>, grid, 256, PrepCfg<128>::kSmem, !first, s, p);
}
cudaError_t launch_delta_scan(const DeltaParams& p, int dk, cudaStream_t s) {
  const unsigned grid = (unsigned)p.nseq * p.Hv * (p.dv / (16 * kScanTiles));
  if (dk == 64) return launch_dependent(delta_scan_kernel<64>, grid, ScanCfg<64>::kThreads, ScanCfg<64>::kSmem, true, s, p);
  return launch_dependent(delta_scan_kernel<128>, grid, ScanCfg<128>::kThreads, ScanCfg<128>::kSmem, true, s, p);
}

}  // namespace lingmoe

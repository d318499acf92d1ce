// Beam search over the logits of the LM head: selection and reordering.
//
// Selection.  For group g, beam w with accumulated score c_w and logits z:
//   candidate (w, t):  c_w + z_t - log sum_j exp(z_j)     (a live beam)
//   candidate (w, eos): c_w                               (a finished beam)
// and the W best candidates of the group in order.  Terms exp(z - m) are fp32
// (each off by (|z - m| + 4) 2^-23 of itself at most); a thread adds the 16 or 32
// of a tile in fp32 and the tiles with compensation, threads and pieces join in 64
// bits: log sum exp is off by 6e-7 and the terms' mean error, some 2e-6 in all,
// however long the row.  Scores are formed from it in 64 bits and rounded to fp32
// once, at the end.  Inside a row the order of the candidates is that of the
// logits themselves, ties to the lower token, whatever the scores round to.
//
// One pass over the logits, one launch.  A row is cut into segments of whole
// tiles of 4096 (bf16: 8192) logits; a CTA walks one segment, each thread
// keeping the (max, sum) of its own logits, with nothing shared on the way.
// The W-th largest of the 256 threads' maxima is a bound that W candidates
// reach, and only the few threads whose maximum reaches it own such candidates:
// their logits are read once more (from L2; 8 of 256) and the best W kept.  A
// key is (order key of the logit, ~token): all distinct, larger is better.
// Where equal logits let too many through, the segment is walked a second time
// with a bound on whole keys, tau, that rises as keys are found: where many
// threads exceed it, it becomes the W-th largest of 32 group maxima first,
// which bounds what can pass to W groups x 8 threads' keys; the buffer is cut to
// its best W, and tau raised to the W-th, when the next tile might not fit.
// The last CTA of a group to finish merges: a warp per row joins the segments'
// sums and merges their sorted lists (a lane per segment), then one warp merges
// the rows (a lane per row).
//
// Bound: latency.  Large batches (224 live rows x 157184 bf16: 30 us, 70 MB at 2.3
// TB/s; 55 us with candidates collected tile by tile) wait for their loads most (5.2
// cycles per instruction; 68 % of the busiest scheduler's slots are used): an SM holds
// three or four CTAs with one tile on its way each, and at 64 registers a thread of the
// bf16 kernel spills 192 bytes.  One request (9 us) is one or two tiles and two
// merges.  The segments depend on the call's sizes alone, not on
// alignment, so equal rows give equal sums to the last bit.
#include "beam.h"
#include "common.cuh"

namespace lingmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kManyHits = 64;                          // threads that may push without raising tau
constexpr int kBufKeys = kBeamMax + kBeamMax * 8 * 32;  // what is kept, and what a tile may push: W groups of 8 threads
constexpr int kChosen = 32;                            // threads whose logits are read once more
constexpr unsigned long long kNoKey = 0x007FFFFFFFFFFFFFull;  // every key of a logit above -inf is larger
constexpr float kLowest = -3.402823466e38f;

// a thread's logits of a tile: 4 vectors of 16 bytes
template <bool BF16> struct Tile;
template <> struct Tile<false> {
  static constexpr int kVecs = 4, kVec = 4, kPer = 16, kLogits = beam_tile(false);
  __device__ static float max(const uint4* r) {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < kPer; ++e) m = fmaxf(m, get(r, e));
    return m;
  }
  __device__ static float get(const uint4* r, int e) {
    const uint4& v = r[e >> 2];
    const uint32_t b = (e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w;
    return __uint_as_float(b);
  }
};
template <> struct Tile<true> {
  static constexpr int kVecs = 4, kVec = 8, kPer = 32, kLogits = beam_tile(true);
  // the largest of a tile (NaN aside), two at a time
  __device__ static float max(const uint4* r) {
    __nv_bfloat162 m[2];
    m[0] = m[1] = __halves2bfloat162(__ushort_as_bfloat16(0xFF80u), __ushort_as_bfloat16(0xFF80u));
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const uint32_t w[4] = {r[v].x, r[v].y, r[v].z, r[v].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) m[i & 1] = __hmax2(m[i & 1], *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    }
    m[0] = __hmax2(m[0], m[1]);
    return fmaxf(__low2float(m[0]), __high2float(m[0]));
  }
  __device__ static float get(const uint4* r, int e) {
    const uint4& v = r[e >> 3];
    const int k = (e & 7) >> 1;
    const uint32_t b = k == 0 ? v.x : k == 1 ? v.y : k == 2 ? v.z : v.w;
    return (e & 1) ? bf16hi(b) : bf16lo(b);
  }
};
// element e of thread tid in a tile
template <bool BF16> __device__ __forceinline__ int tile_at(int tid, int e) {
  constexpr int VE = Tile<BF16>::kVec;
  return (e / VE) * (kThreads * VE) + tid * VE + e % VE;
}

// the vector of logits i .. of a row, those at and past `end` as -inf
template <bool BF16>
__device__ __forceinline__ void load_vec(uint4& r, const unsigned char* row, int i, int end, bool al) {
  constexpr int VE = Tile<BF16>::kVec, ES = BF16 ? 2 : 4;
  if (al && i + VE <= end) {
    r = ldg_stream(row + (size_t)i * ES);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (BF16) {
        const unsigned short* p = reinterpret_cast<const unsigned short*>(row);
        const uint32_t lo = i + 2 * k < end ? p[i + 2 * k] : 0xFF80u;
        const uint32_t hi = i + 2 * k + 1 < end ? p[i + 2 * k + 1] : 0xFF80u;
        w[k] = lo | (hi << 16);
      } else {
        w[k] = i + k < end ? reinterpret_cast<const uint32_t*>(row)[i + k] : 0xFF800000u;
      }
    }
    r = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The tile that starts at `base`.  The element a thread gets does not depend on
// the row's alignment.
template <bool BF16>
__device__ __forceinline__ void load_tile(uint4* r, const unsigned char* row, int base, int end, int tid, bool al) {
  constexpr int VE = Tile<BF16>::kVec;
#pragma unroll
  for (int v = 0; v < Tile<BF16>::kVecs; ++v) load_vec<BF16>(r[v], row, base + v * (kThreads * VE) + tid * VE, end, al);
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
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;
// exp(x), x <= 0, to 2 ulp of the result (and 2^-24 |x| for the product); arguments below 2^-126 count as 0
__device__ __forceinline__ float exp_neg(float x) { return ex2(x * kLog2e); }
// NaN counts as -inf; -0 as +0 (equal logits tie)
__device__ __forceinline__ float clean(float z) { return fmaxf(z, -INFINITY) + 0.0f; }
__device__ __forceinline__ unsigned long long make_key(float z, int token) {
  return ((unsigned long long)f32_order_key(z) << 32) | (unsigned long long)(0xFFFFFFFFu - (uint32_t)token);
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((unsigned long long)hi << 32) | lo;
}
// order-preserving key of a double (no NaN)
__device__ __forceinline__ unsigned long long f64_order_key(double d) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(d);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

struct SelectSmem {
  union {
    unsigned long long buf[kBufKeys];                            // candidates of a segment
    unsigned long long list[kThreads / 32][kBeamMaxSegs * kBeamMax];  // merge: a row's lists, one per warp
  };
  unsigned long long best[kBeamMax];
  unsigned long long grp[32];
  __align__(16) uint32_t tops[kThreads];
  int who[kChosen];
  int chosen;
  uint32_t bound;
  unsigned long long tau;
  unsigned long long row_key[kBeamMax][kBeamMax];
  double row_score[kBeamMax][kBeamMax];
  double red_s[kThreads / 32];
  float red_m[kThreads / 32];
  int count;
  int last;
};

// The `count` keys in sm.buf -> the best K of them, sorted, in sm.best and
// sm.buf[0 .. K).  Every thread of the CTA calls it; ends with a barrier.
__device__ __forceinline__ void keep_best(SelectSmem& sm, int K, int tid) {
  const int n = sm.count;
  if (tid < kBeamMax) sm.best[tid] = 0ull;
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) {
    const unsigned long long k = sm.buf[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += sm.buf[j] > k;
    if (r < K) sm.best[r] = k;
  }
  __syncthreads();
  if (tid < K) sm.buf[tid] = sm.best[tid];
  if (tid == 0) {
    sm.count = n < K ? n : K;
    if (n >= K && sm.best[K - 1] > sm.tau) sm.tau = sm.best[K - 1];
  }
  __syncthreads();
}

}  // namespace

template <bool BF16>
__global__ void __launch_bounds__(kThreads, kBeamCtas) beam_select_kernel(const BeamSelectParams p) {
  __shared__ SelectSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.segs, seg = blockIdx.x % p.segs;
  const int g = row / p.beams, w = row % p.beams;
  const int K = p.beams;
  const float score = p.scores[row];
  const bool live = score > -INFINITY && !(p.finished && p.finished[row]);  // false for NaN
  constexpr int NV = Tile<BF16>::kVecs, VE = Tile<BF16>::kVec;
  constexpr int kPerThread = Tile<BF16>::kPer, kBeamTile = Tile<BF16>::kLogits;
  constexpr int kTilePush = kBeamMax * 8 * kPerThread;
  static_assert(kManyHits * kPerThread <= kTilePush && kBeamMax + kTilePush <= kBufKeys, "push bound");
  BeamPart* part = p.parts + (size_t)row * p.segs + seg;

  if (live) {
    const unsigned char* z = static_cast<const unsigned char*>(p.logits) +
                             ((long long)g * p.group_stride + (long long)w * p.beam_stride) * (BF16 ? 2 : 4);
    const bool al = (reinterpret_cast<uintptr_t>(z) & 15u) == 0;
    const int begin = seg * p.seg_len;
    const int end = min(p.vocab, begin + p.seg_len);
    if (tid == 0) {
      sm.count = 0;
      sm.chosen = 0;
      sm.tau = kNoKey;
    }
    // ---- one pass: the thread's largest logit and its sum of exp(logit - m).  m follows the
    // largest only when that is more than 1 above it, so that what a rescaling rounds has
    // shrunk by e: however many there are, they add 2^-22 (1 + 1 / e + ...) at most.  s - low
    // is the sum, each tile's added with compensation.
    float m = kLowest, s = 0.f, low = 0.f, top = -INFINITY;
    {
      uint4 cur[NV], nxt[NV];
      load_tile<BF16>(cur, z, begin, end, tid, al);
      for (int base = begin; base < end; base += kBeamTile) {
        if (base + kBeamTile < end) load_tile<BF16>(nxt, z, base + kBeamTile, end, tid, al);
        const float mx = Tile<BF16>::max(cur);
        top = fmaxf(top, mx);
        if (mx > m + 1.f) {
          const float f = exp_neg(m - mx);
          s *= f;
          low *= f;
          m = mx;
        }
        f2 t[2] = {0ull, 0ull};
        const f2 off = pack2(-m, -m), scale = pack2(kLog2e, kLog2e);
#pragma unroll
        for (int e = 0; e < kPerThread; e += 2) {
          const float2 x = unpack2(mul2(add2(pack2(Tile<BF16>::get(cur, e), Tile<BF16>::get(cur, e + 1)), off), scale));
          t[(e >> 1) & 1] = add2(t[(e >> 1) & 1], pack2(ex2(x.x), ex2(x.y)));
        }
        const float2 ts = unpack2(add2(t[0], t[1]));
        float sum = ts.x + ts.y;
        if (!(sum == sum)) {  // a NaN among them: it counts as -inf
          sum = 0.f;
#pragma unroll 1
          for (int v = 0; v < NV; ++v) {
            const uint4 one[1] = {v == 0 ? cur[0] : v == 1 ? cur[1] : v == 2 ? cur[2] : cur[3]};
#pragma unroll
            for (int e = 0; e < VE; ++e) sum += exp_neg(fmaxf(Tile<BF16>::get(one, e), -INFINITY) - m);
          }
        }
        sum -= low;
        const float t2 = s + sum;
        low = (t2 - s) - sum;
        s = t2;
#pragma unroll
        for (int v = 0; v < NV; ++v) cur[v] = nxt[v];
      }
    }
    // ---- the K-th largest of the threads' maxima: K candidates reach it, and
    // whatever does belongs to a thread that does
    // (the order keys' low 8 bits give way to the thread, so that all differ; the
    // bound is that much lower at most)
    const uint32_t mine = (f32_order_key(clean(top)) & ~255u) | (uint32_t)tid;
    sm.tops[tid] = mine;
    __syncthreads();
    if (warp == 0) {
      uint32_t k[kThreads / 32], best = 0u;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) k[i] = sm.tops[32 * i + lane];
      for (int i = 0; i < K; ++i) {
        uint32_t own = 0u;
#pragma unroll
        for (int j = 0; j < kThreads / 32; ++j) own = k[j] > own ? k[j] : own;
        best = __reduce_max_sync(0xffffffffu, own);
#pragma unroll
        for (int j = 0; j < kThreads / 32; ++j) k[j] = k[j] == best ? 0u : k[j];
      }
      if (lane == 0) sm.bound = best & ~255u;
    }
    __syncthreads();
    const uint32_t bound = sm.bound;
    if (mine >= bound && top > -INFINITY) {
      const int at = atomicAdd(&sm.chosen, 1);
      if (at < kChosen) sm.who[at] = tid;
    }
    __syncthreads();
    const int chosen = sm.chosen;
    // ---- those threads' logits once more, a vector at a time
    if (chosen <= kChosen) {
      const int tiles = (end - begin + kBeamTile - 1) / kBeamTile;
      const float boundf = bound > f32_order_key(-INFINITY) ? f32_from_order_key(bound) : -INFINITY;
      for (int i = tid; i < chosen * tiles * NV; i += kThreads) {
        const int v = i % NV, t = i / NV % tiles, owner = sm.who[i / NV / tiles];
        const int at = begin + t * kBeamTile + v * (kThreads * VE) + owner * VE;
        uint4 one[1];
        load_vec<BF16>(one[0], z, at, end, al);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float x = clean(Tile<BF16>::get(one, e));
          if (x >= boundf && x > -INFINITY) {
            const int slot = atomicAdd(&sm.count, 1);
            if (slot < kBufKeys) sm.buf[slot] = make_key(x, at + e);
          }
        }
      }
      __syncthreads();
    }
    // ---- many equal logits: too many threads or candidates reach the bound; tile by tile with a rising tau
    if (chosen > kChosen || sm.count > kBufKeys) {
      __syncthreads();
      if (tid == 0) sm.count = 0;
      __syncthreads();
      unsigned long long tau = kNoKey;
      int held = 0;  // the buffer has at most this many keys (the same in every thread)
#pragma unroll 1
      for (int base = begin; base < end; base += kBeamTile) {
        uint4 cur[NV];
        load_tile<BF16>(cur, z, base, end, tid, al);
        // the thread's best key of the tile
        unsigned long long best = 0ull;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
          const unsigned long long k = make_key(clean(Tile<BF16>::get(cur, e)), base + tile_at<BF16>(tid, e));
          if (k > best) best = k;
        }
        const bool hit = best > tau;
        const int hits = __syncthreads_count(hit);
        if (!hits) continue;
        if (hits > kManyHits) {
          // raise tau to just below the K-th largest of 32 group maxima
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            const unsigned long long x = __shfl_xor_sync(0xffffffffu, best, o);
            best = x > best ? x : best;
          }
          if ((lane & 7) == 0) sm.grp[tid >> 3] = best;
          __syncthreads();
          if (warp == 0) {
            const unsigned long long k = sm.grp[lane];
            int r = 0;
            for (int j = 0; j < 32; ++j) r += sm.grp[j] > k;
            if (r == K - 1 && k - 1 > sm.tau) sm.tau = k - 1;  // keys of logits above -inf are distinct: one lane
          }
          __syncthreads();
          tau = sm.tau;
        }
        const int push = hits > kManyHits ? kTilePush : hits * kPerThread;
        if (held + push > kBufKeys) {  // what earlier tiles pushed stands: a barrier since
          keep_best(sm, K, tid);
          tau = sm.tau;
          held = K;
        }
        held += push;
        if (hit) {
#pragma unroll
          for (int e = 0; e < kPerThread; ++e) {
            const float x = clean(Tile<BF16>::get(cur, e));
            const unsigned long long k = make_key(x, base + tile_at<BF16>(tid, e));
            if (k > tau && x > -INFINITY) {
              const int at = atomicAdd(&sm.count, 1);
              if (at < kBufKeys) sm.buf[at] = k;
            }
          }
        }
      }
      __syncthreads();
    }
    keep_best(sm, K, tid);
    // the segment's max and sum, joined in 64 bits
    float bm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
    if (lane == 0) sm.red_m[warp] = bm;
    __syncthreads();
    bm = sm.red_m[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) bm = fmaxf(bm, sm.red_m[i]);
    double ds = ((double)s - (double)low) * (double)expf(m - bm);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ds += __shfl_xor_sync(0xffffffffu, ds, o);
    if (lane == 0) sm.red_s[warp] = ds;
    __syncthreads();
    if (tid == 0) {
      double t = 0.0;
      for (int i = 0; i < kThreads / 32; ++i) t += sm.red_s[i];
      part->sum = t;
      part->max = bm;
    }
    if (tid < K) part->keys[tid] = sm.best[tid];
  }

  // the last CTA of the group merges
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    const unsigned int all = (unsigned int)(p.beams * p.segs) - 1u;
    sm.last = atomicInc(p.arrived + g, all) == all;  // wraps to 0 for the next call
    __threadfence();
  }
  __syncthreads();
  if (!sm.last) return;

  for (int r = warp; r < K; r += kThreads / 32) {
    const int grow = g * K + r;
    const float c = p.scores[grow];
    const bool done = p.finished && p.finished[grow];
    if (!(c > -INFINITY) || done) {
      if (lane < K) {
        const bool keep = lane == 0 && done && c > -INFINITY;
        sm.row_key[r][lane] = keep ? make_key(0.f, p.eos) : 0ull;
        sm.row_score[r][lane] = keep ? (double)c : -INFINITY;
      }
      continue;
    }
    const BeamPart* q = p.parts + (size_t)grow * p.segs;
    float pm = kLowest;
    double ps = 0.0;
    if (lane < p.segs) {
      pm = __ldcg(&q[lane].max);
      ps = __ldcg(&q[lane].sum);
    }
    for (int i = lane; i < p.segs * K; i += 32) sm.list[warp][i] = __ldcg(&q[i / K].keys[i % K]);
    float M = pm;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    ps *= exp((double)pm - (double)M);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
    // +inf among the logits: the softmax is not defined and the row has no candidates
    const bool ok = ps > 0.0 && M < INFINITY;
    const double lse = ok ? (double)M + log(ps) : 0.0;
    __syncwarp();
    int at = 0;
    unsigned long long head = ok && lane < p.segs ? sm.list[warp][lane * K] : 0ull;
    for (int i = 0; i < K; ++i) {
      const unsigned long long k = warp_max_u64(head);
      if (lane == 0) {
        sm.row_key[r][i] = k;
        sm.row_score[r][i] = k ? (double)f32_from_order_key((uint32_t)(k >> 32)) - lse + (double)c : -INFINITY;
      }
      if (k != 0ull && head == k) {
        ++at;
        head = at < K ? sm.list[warp][lane * K + at] : 0ull;
      }
    }
    __syncwarp();
  }
  __syncthreads();
  if (warp != 0) return;
  // a lane per row: its best candidate left; ties between rows go to the lower one
  int at = 0;
  for (int i = 0; i < K; ++i) {
    const double v = lane < K && at < K ? sm.row_score[lane][at] : -INFINITY;
    const unsigned long long k = v > -INFINITY ? f64_order_key(v + 0.0) : 0ull;
    const unsigned long long top = warp_max_u64(k);
    const unsigned int who = __ballot_sync(0xffffffffu, k == top && top != 0ull);
    const int out = g * K + i;
    if (who == 0u) {
      if (lane == 0) {
        p.tokens[out] = -1;
        p.parents[out] = i;
        p.scores_out[out] = -INFINITY;
        p.finished_out[out] = 1;
      }
      continue;
    }
    const int src = __ffs(who) - 1;
    if (lane == src) {
      const int token = (int)(0xFFFFFFFFu - (uint32_t)sm.row_key[lane][at]);
      p.tokens[out] = token;
      p.parents[out] = lane;
      p.scores_out[out] = (float)v;
      // a finished beam's only candidate is its own end
      p.finished_out[out] = token == p.eos;
      ++at;
    }
    __syncwarp();
  }
}

cudaError_t launch_beam_select(const BeamSelectParams& p, bool bf16, cudaStream_t s) {
  const unsigned grid = (unsigned)(p.groups * p.beams * p.segs);
  if (bf16)
    beam_select_kernel<true><<<grid, kThreads, 0, s>>>(p);
  else
    beam_select_kernel<false><<<grid, kThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- reorder
// row[place w] <- row[place parent(w)] for every place of a group at once, in
// place.  A thread owns one unit (16 bytes) of the columns of all the group's
// rows: it loads that unit of every row that moves, then stores them, so a
// row that is both read and overwritten (a chain or a cycle of parents) needs
// no copy elsewhere.  Places whose parent is themselves are neither read nor
// written.  Bound: HBM, moved rows read (shared parents once, the repeats hit
// the caches) and written once: 48 rows of 2 MB moved in 32 us, 6.3 TB/s.
template <typename U, int MAXW>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const BeamReorderParams p) {
  const int g = blockIdx.y, t = blockIdx.z;
  const size_t units = p.row_bytes[t] / sizeof(U);
  if ((size_t)blockIdx.x * kThreads >= units) return;
  __shared__ int s_from[kBeamMax], s_to[kBeamMax], s_moves;
  if (threadIdx.x < 32) {
    const int w = threadIdx.x;
    int from = -1, to = -1;
    if (w < p.beams) {
      const int par = p.parents[g * p.beams + w];
      if (par >= 0 && par < p.beams && par != w) {
        from = p.slots ? p.slots[g * p.beams + par] : g * p.beams + par;
        to = p.slots ? p.slots[g * p.beams + w] : g * p.beams + w;
      }
    }
    const bool mv = from >= 0 && from < p.num_rows && to >= 0 && to < p.num_rows && from != to;
    const unsigned int mask = __ballot_sync(0xffffffffu, mv);
    if (mv) {
      const int at = __popc(mask & ((1u << w) - 1u));
      s_from[at] = from;
      s_to[at] = to;
    }
    if (w == 0) s_moves = __popc(mask);
  }
  __syncthreads();
  const int moves = s_moves;
  U* base = reinterpret_cast<U*>(p.state[t]);
  for (size_t c = (size_t)blockIdx.x * kThreads + threadIdx.x; c < units; c += (size_t)gridDim.x * kThreads) {
    U v[MAXW];
#pragma unroll
    for (int i = 0; i < MAXW; ++i)
      if (i < moves) v[i] = base[(size_t)s_from[i] * units + c];
#pragma unroll
    for (int i = 0; i < MAXW; ++i)
      if (i < moves) base[(size_t)s_to[i] * units + c] = v[i];
  }
}

template <typename U>
static void reorder_unit(const BeamReorderParams& p, dim3 grid, cudaStream_t s) {
  if (p.beams <= 4)
    beam_reorder_kernel<U, 4><<<grid, kThreads, 0, s>>>(p);
  else if (p.beams <= 8)
    beam_reorder_kernel<U, 8><<<grid, kThreads, 0, s>>>(p);
  else
    beam_reorder_kernel<U, kBeamMax><<<grid, kThreads, 0, s>>>(p);
}

cudaError_t launch_beam_reorder(const BeamReorderParams& p, int tensors, int groups, int unit, size_t longest_row,
                                cudaStream_t s) {
  const size_t blocks = (longest_row / unit + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(blocks < 4096 ? blocks : 4096), (unsigned)groups, (unsigned)tensors);
  if (unit == 16)
    reorder_unit<uint4>(p, grid, s);
  else if (unit == 4)
    reorder_unit<uint32_t>(p, grid, s);
  else
    reorder_unit<unsigned char>(p, grid, s);
  return cudaGetLastError();
}

}  // namespace lingmoe

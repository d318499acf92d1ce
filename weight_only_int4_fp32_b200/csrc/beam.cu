// Beam search over the logits of the LM head: selection and reordering.
//
// Selection.  For group g, beam w with accumulated score c_w and logits z:
//   candidate (w, t):  c_w + z_t - log sum_j exp(z_j)     (a live beam)
//   candidate (w, eos): c_w                               (a finished beam)
// and the W best candidates of the group in order.  Scores are formed in 64
// bits (fp32 terms exp(z - max), summed in fp32 per thread over at most a few
// hundred terms and in 64 bits above that), so that two beams' candidates
// compare by more than the 2^-24 of an fp32 score; they are rounded to fp32
// once, at the end.  Inside a row the order of the candidates is that of the
// logits themselves, ties to the lower token, whatever the scores round to.
//
// One pass over the logits, one launch.  A row is cut into segments of whole
// tiles of 4096 logits; a CTA walks one segment with the tile in registers,
// keeping per thread the running (max, sum) and per CTA the best W keys.  A
// key is (order key of the logit, ~token): all distinct, larger is better.
// Only keys above the W-th best so far (tau) are looked at: from the second
// tile on that is a handful per tile.  Where many threads exceed tau (the
// first tile, ascending rows) it is raised first to the W-th largest of 32
// group maxima, which bounds what can pass to W groups x 128 keys.  The last
// CTA of a group to finish merges: a warp per row joins the segments' sums
// and merges their sorted lists (a lane per segment), then one warp merges
// the rows (a lane per row).
//
// Bound: HBM for large batches, latency (one tile, two merges) for one
// request.  The segments depend on the call's sizes alone, not on
// alignment, so equal rows give equal sums to the last bit.
#include "beam.h"
#include "common.cuh"

namespace lingmoe {

namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = kBeamTile / kThreads;             // 16
constexpr int kBufKeys = kBeamMax + kBeamMax * 8 * kPerThread;  // kept + W groups of 8 threads
constexpr int kManyHits = 64;                                // threads that may push without raising tau
static_assert(kManyHits * kPerThread <= kBeamMax * 8 * kPerThread, "push bound");
constexpr unsigned long long kNoKey = 0x007FFFFFFFFFFFFFull;  // every key of a logit above -inf is larger
constexpr float kLowest = -3.402823466e38f;

// 16 logits per thread, NV vectors of 16 bytes
template <bool BF16> struct Tile;
template <> struct Tile<false> {
  static constexpr int kVecs = 4, kVec = 4;
  __device__ static float get(const uint4* r, int e) {
    const uint4& v = r[e >> 2];
    const uint32_t b = (e & 3) == 0 ? v.x : (e & 3) == 1 ? v.y : (e & 3) == 2 ? v.z : v.w;
    return __uint_as_float(b);
  }
};
template <> struct Tile<true> {
  static constexpr int kVecs = 2, kVec = 8;
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

// The tile that starts at `base`, logits at and past `end` as -inf.  The
// element a thread gets does not depend on the row's alignment.
template <bool BF16>
__device__ __forceinline__ void load_tile(uint4* r, const unsigned char* row, int base, int end, int tid, bool al) {
  constexpr int VE = Tile<BF16>::kVec, ES = BF16 ? 2 : 4;
#pragma unroll
  for (int v = 0; v < Tile<BF16>::kVecs; ++v) {
    const int i = base + v * (kThreads * VE) + tid * VE;
    if (al && i + VE <= end) {
      r[v] = ldg_stream(row + (size_t)i * ES);
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
      r[v] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

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
    if (n >= K) sm.tau = sm.best[K - 1];
  }
  __syncthreads();
}

}  // namespace

template <bool BF16>
__global__ void __launch_bounds__(kThreads) beam_select_kernel(const BeamSelectParams p) {
  __shared__ SelectSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / p.segs, seg = blockIdx.x % p.segs;
  const int g = row / p.beams, w = row % p.beams;
  const int K = p.beams;
  const float score = p.scores[row];
  const bool live = score > -INFINITY && !(p.finished && p.finished[row]);  // false for NaN
  BeamPart* part = p.parts + (size_t)row * p.segs + seg;

  if (live) {
    const unsigned char* z = static_cast<const unsigned char*>(p.logits) +
                             ((long long)g * p.group_stride + (long long)w * p.beam_stride) * (BF16 ? 2 : 4);
    const bool al = (reinterpret_cast<uintptr_t>(z) & 15u) == 0;
    const int begin = seg * p.seg_len;
    const int end = min(p.vocab, begin + p.seg_len);
    if (tid == 0) {
      sm.count = 0;
      sm.tau = kNoKey;
    }
    float m = kLowest, s = 0.f;
    uint4 cur[Tile<BF16>::kVecs], nxt[Tile<BF16>::kVecs];
    load_tile<BF16>(cur, z, begin, end, tid, al);
    __syncthreads();
    unsigned long long tau = sm.tau;
    for (int base = begin; base < end; base += kBeamTile) {
      if (base + kBeamTile < end) load_tile<BF16>(nxt, z, base + kBeamTile, end, tid, al);
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) mx = fmaxf(mx, Tile<BF16>::get(cur, e));
      const float mn = fmaxf(m, mx);
      s *= __expf(m - mn);
      m = mn;
#pragma unroll
      for (int e = 0; e < kPerThread; ++e) s += __expf(clean(Tile<BF16>::get(cur, e)) - m);
      bool hit = f32_order_key(clean(mx)) >= (uint32_t)(tau >> 32) && mx > -INFINITY;
      const int hits = __syncthreads_count(hit);
      if (hits) {
        if (hits > kManyHits) {
          // raise tau to just below the K-th largest of 32 group maxima
          unsigned long long best = 0ull;
#pragma unroll
          for (int e = 0; e < kPerThread; ++e) {
            const float v = clean(Tile<BF16>::get(cur, e));
            const unsigned long long k = make_key(v, base + tile_at<BF16>(tid, e));
            if (k > best) best = k;
          }
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
#pragma unroll 8
            for (int j = 0; j < 32; ++j) r += __shfl_sync(0xffffffffu, k, j) > k;
            if (r == K - 1 && k - 1 > sm.tau) sm.tau = k - 1;  // keys are distinct: one lane
          }
          __syncthreads();
          tau = sm.tau;
        }
        if (hit) {
#pragma unroll
          for (int e = 0; e < kPerThread; ++e) {
            const float v = clean(Tile<BF16>::get(cur, e));
            const unsigned long long k = make_key(v, base + tile_at<BF16>(tid, e));
            if (k > tau && v > -INFINITY) {
              const int at = atomicAdd(&sm.count, 1);
              if (at < kBufKeys) sm.buf[at] = k;
            }
          }
        }
        __syncthreads();
        if (sm.count > K) keep_best(sm, K, tid);
        tau = sm.tau;
      }
#pragma unroll
      for (int v = 0; v < Tile<BF16>::kVecs; ++v) cur[v] = nxt[v];
    }
    keep_best(sm, K, tid);  // at most K keys: sorts them
    // the segment's max and sum, joined in 64 bits
    float bm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, o));
    if (lane == 0) sm.red_m[warp] = bm;
    __syncthreads();
    bm = sm.red_m[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) bm = fmaxf(bm, sm.red_m[i]);
    double ds = (double)s * (double)expf(m - bm);
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
// the caches) and written once.
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

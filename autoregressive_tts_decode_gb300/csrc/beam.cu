// beam.cu -- beam selection over beams and vocabulary, and the reordering of
// per-beam state that follows it.
//
// Row (g, b) holds the logits of beam b of group g.  With x the logits after
// the repetition penalty and the mask of special codes (the sampler's rule),
//   score(b, v) = scores[b] + (x_v - max x) - log sum_v e^(x_v - max x),
// and a group keeps the k candidates with the largest scores among its beams'
// vocabularies.  Scores are sums of two floats, so that candidates of one beam order
// exactly as their logits do; between beams they are as exact as the rows' sums,
// fp32 sums of fp32 exponentials (up to about 2^-20 relative, a few 2^-24 as a rule).
// Equal scores go to the lower beam, then the larger logit, then the lower code.  A
// finished beam offers one candidate, its end code at its own score.
//
// Within a row scores order as logits do, so a row's own k best logits are all
// it can contribute.  One pass over a row keeps the running maximum and sum of
// its softmax and a buffer of candidates above a bound of its k best logits
// (first the k-th largest maximum of 32 groups of threads, then, whenever the
// buffer fills, the k-th best itself), so most tiles of a long row need one
// barrier and no selection at all.  A CTA scans a row, or a piece of a long one
// where there are few.  Up to eight whole rows of a group are a cluster, whose
// first CTA joins their maxima, sums and lists through distributed shared memory;
// otherwise they are left in a workspace and a second kernel joins a group's.
// (Clusters of 16 for 8 groups of 16 beams over 131072 codes took 47 us, against
// 29 in two kernels: no more than 7 such clusters run at once, or their CTAs share
// SMs.)
// Measured with the reordering of a state of 2048 floats a beam: 4 beams of 4096
// codes 9.2 us, 32 groups of 4 beams of 2048 11.3, both latency; 8 groups of 16 beams of 131072
// codes (67 MB) 30 us, of which the scan takes 18 (a plain read 14.5): it waits at
// a barrier per tile.
// The GPU's fp64 rate is low: a row's log sum is computed in fp64, a candidate's
// score as a sum of two floats, and compared as an ordered integer.
#include <cooperative_groups.h>

#include <atomic>

#include "ops.cuh"

namespace cg = cooperative_groups;

namespace q3 {

namespace {

constexpr int BM_THREADS = 512, BM_WARPS = BM_THREADS / 32;
constexpr int BM_PER = 16;                       // logits of a thread per tile
constexpr int BM_TILE = BM_THREADS * BM_PER;     // logits of a tile
constexpr int BM_MAXK = 32;                      // candidates kept
constexpr int BM_MAXB = 32;                      // beams of a group
constexpr int BM_LISTS = 128;                    // lists (rows or pieces of rows) of a group at most
constexpr int BM_GROUP = 8;                      // beams of a group that a cluster takes (the portable size)
constexpr int BM_FULL = 256;                     // buffered candidates that call for a selection
constexpr int BM_CAND = BM_FULL + BM_TILE;       // a tile adds all of its logits at most
static_assert(BM_LISTS >= BM_MAXB, "a list for every beam");

typedef unsigned long long u64;

// Ordered integers: larger value, larger integer.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
// Larger key: larger logit (-0 is +0), then lower code.  Keys of a row are
// distinct; 0 is below every key.
__device__ __forceinline__ u64 make_key(float x, int v) { return ((u64)ordered(x + 0.f) << 32) | (uint32_t)~v; }
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int key_code(u64 k) { return (int)~(uint32_t)k; }

// What a scan leaves of its piece (in the workspace): the maximum, the sum of
// e^(x - maximum), and the best keys in order (0: none).
struct Piece {
  float mx, sum;
  u64 list[BM_MAXK];
};

struct BeamSmem {
  float red[2][32];
  float group[64], bound;
  u64 best[BM_MAXK], top[BM_MAXK];
  int n_cand;
  u64 cand[BM_CAND];
};

struct JoinSmem {
  float hi[BM_MAXB], lo[BM_MAXB];  // the beam's score less the log of its row's sum (relative to its maximum), in two floats
  float mx[BM_MAXB];
  uint32_t group[128], bound;
  int n_cand;
  u64 score[BM_LISTS * BM_MAXK], key[BM_LISTS * BM_MAXK];  // the candidates that may be kept
  int row[BM_LISTS * BM_MAXK];
};

// The k-th largest of the G group values g[0 .. G) into *out (k <= G).  Each warp
// ranks its share of them, 32 comparisons a ballot.  All threads; ends in a
// block barrier, and expects one since g was written.
template <int G, class T>
__device__ __forceinline__ void kth_group(const T* g, int k, T* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int PER = G / BM_WARPS;
  T v[G / 32];
#pragma unroll
  for (int c = 0; c < G / 32; ++c) v[c] = g[c * 32 + lane];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int me = warp * PER + i;
    const T x = g[me];
    int r = 0;  // how many come before it: larger, or equal and earlier
#pragma unroll
    for (int c = 0; c < G / 32; ++c)
      r += __popc(__ballot_sync(0xffffffffu, v[c] > x || (v[c] == x && c * 32 + lane < me)));
    if (r == k - 1 && lane == 0) *out = x;
  }
  __syncthreads();
}

// The k best of sm.cand[0 .. n) into sm.best, in order, the rest 0.  All
// threads.  More candidates than threads (equal or ascending logits): the k-th
// largest key by bisection first (keys are distinct, so exactly k are at or
// above it), then those are ranked.
__device__ void keep_best(BeamSmem& sm, int n, int k) {
  const int tid = threadIdx.x;
  const u64* from = sm.cand;
  if (n > BM_THREADS) {
    u64 lo = 0, hi = ~0ull;  // count(key >= lo) >= k > count(key > hi)
    while (lo < hi) {
      const u64 mid = lo + (hi - lo) / 2 + 1;
      float c = 0.f;  // at most BM_CAND: exact
      for (int i = tid; i < n; i += BM_THREADS) c += sm.cand[i] >= mid ? 1.f : 0.f;
      c = block_sum(c, sm.red[0]);
      if (c >= (float)k) lo = mid; else hi = mid - 1;
    }
    if (tid == 0) sm.n_cand = 0;
    __syncthreads();
    for (int i = tid; i < n; i += BM_THREADS)
      if (sm.cand[i] >= lo) sm.top[atomicAdd(&sm.n_cand, 1)] = sm.cand[i];
    from = sm.top;
    n = k;
  }
  if (tid < BM_MAXK) sm.best[tid] = 0;
  __syncthreads();
  // a warp ranks every sixteenth, 32 comparisons a ballot
  const int lane = tid & 31;
  for (int i = tid >> 5; i < n; i += BM_WARPS) {
    const u64 key = from[i];
    int r = 0;
    for (int j = 0; j < n; j += 32) r += __popc(__ballot_sync(0xffffffffu, j + lane < n && from[j + lane] > key));
    if (lane == 0 && r < k) sm.best[r] = key;
  }
  __syncthreads();
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Pairs of floats, one instruction each.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
constexpr float kLog2e = 1.4426950408889634f;
// e^(x - m), with e^0 = 1 where both are infinite (and 0 where nothing can be picked)
__device__ __forceinline__ float exp_off(float x, float m) {
  return x == m ? (x == -INFINITY ? 0.f : 1.f) : exp2_fast((x - m) * kLog2e);
}

// A tile's logits (and history bytes) of one thread, four codes in a row at a
// time; codes from v1 on are -inf.
template <bool HIST>
__device__ __forceinline__ void load_tile(const float* x, const uint8_t* hist, bool vec, int t0, int v1,
                                          float (&f)[BM_PER], uint32_t (&hb)[BM_PER / 4]) {
  const int tid = threadIdx.x;
  if (vec && t0 + BM_TILE <= v1) {  // a whole tile: every load under way before the first is waited for
    const float4* p = reinterpret_cast<const float4*>(x + t0) + tid;
    float4 w[BM_PER / 4];
#pragma unroll
    for (int j = 0; j < BM_PER / 4; ++j) w[j] = __ldcs(p + j * BM_THREADS);
#pragma unroll
    for (int j = 0; j < BM_PER / 4; ++j)
      if (HIST) hb[j] = __ldcs(reinterpret_cast<const unsigned int*>(hist + t0) + j * BM_THREADS + tid);
#pragma unroll
    for (int j = 0; j < BM_PER / 4; ++j) {
      f[4 * j] = w[j].x;
      f[4 * j + 1] = w[j].y;
      f[4 * j + 2] = w[j].z;
      f[4 * j + 3] = w[j].w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < BM_PER / 4; ++j) {
    const int c = t0 + (j * BM_THREADS + tid) * 4;
    float4 w = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    uint32_t h = 0;
    if (vec && c + 4 <= v1) {
      w = __ldcs(reinterpret_cast<const float4*>(x + c));
      if (HIST) h = __ldcs(reinterpret_cast<const unsigned int*>(hist + c));
    } else if (c < v1) {
      w.x = x[c];
      if (c + 1 < v1) w.y = x[c + 1];
      if (c + 2 < v1) w.z = x[c + 2];
      if (c + 3 < v1) w.w = x[c + 3];
      if (HIST)
        for (int e = 0; e < 4; ++e)
          if (c + e < v1) h |= (uint32_t)hist[c + e] << (8 * e);
    }
    f[4 * j] = w.x;
    f[4 * j + 1] = w.y;
    f[4 * j + 2] = w.z;
    f[4 * j + 3] = w.w;
    if (HIST) hb[j] = h;
  }
}

// sum of e^(f[i] - m), m the largest of them or more, finite
__device__ __forceinline__ float tile_sum(const float (&f)[BM_PER], float m) {
  const float2 mm = make_float2(-m, -m), ll = make_float2(kLog2e, kLog2e);
  float2 acc = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < BM_PER; i += 2) {
    const float2 d = mul2(add2(make_float2(f[i], f[i + 1]), mm), ll);
    acc = add2(acc, make_float2(exp2_fast(d.x), exp2_fast(d.y)));
  }
  return acc.x + acc.y;
}

// One row's codes [v0, v1): running maximum and sum, and the k best keys.
template <bool HIST>
__device__ __forceinline__ void scan_piece(BeamSmem& sm, Piece& out, const BeamArgs& a, const float* x,
                                           const uint8_t* hist, int v0, int v1) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
  const bool vec = ((uintptr_t)(x + v0) & 15) == 0 && (!HIST || ((uintptr_t)(hist + v0) & 3) == 0);
  float m = -INFINITY, s = 0.f;
  float thr = -INFINITY;  // only logits above it can still be among the k best
  if (tid == 0) sm.n_cand = 0;
  float nf[BM_PER];  // the next tile, on its way while this one is worked on
  uint32_t nh[BM_PER / 4];
  load_tile<HIST>(x, hist, vec, v0, v1, nf, nh);
  for (int t0 = v0; t0 < v1; t0 += BM_TILE) {
    float f[BM_PER];
    uint32_t hb[BM_PER / 4];
#pragma unroll
    for (int i = 0; i < BM_PER; ++i) f[i] = nf[i];
#pragma unroll
    for (int i = 0; i < BM_PER / 4; ++i)
      if (HIST) hb[i] = nh[i];
    if (t0 + BM_TILE < v1) load_tile<HIST>(x, hist, vec, t0 + BM_TILE, v1, nf, nh);
    // the sampler's rule: penalty on the codes of the history, special codes masked
    if (HIST) {
#pragma unroll
      for (int i = 0; i < BM_PER; ++i)
        if ((hb[i >> 2] >> (8 * (i & 3))) & 0xffu) f[i] = f[i] > 0.f ? f[i] / a.penalty : f[i] * a.penalty;
    }
    if (a.special_from > 0 && t0 + BM_TILE > a.special_from) {
#pragma unroll
      for (int i = 0; i < BM_PER; ++i) {
        const int v = t0 + ((i >> 2) * BM_THREADS + tid) * 4 + (i & 3);
        if (v >= a.special_from && v != a.eos) f[i] = -INFINITY;
      }
    }
    float tm = -INFINITY;  // of the numbers among them: a NaN is passed over
#pragma unroll
    for (int i = 0; i < BM_PER; ++i) tm = fmaxf(tm, f[i]);
    if (tm > m) {
      s *= exp_off(m, tm);
      m = tm;
    }
    if (m > -INFINITY && m < INFINITY) {
      float ts = tile_sum(f, m);
      if (ts != ts) {  // a NaN logit counts as -inf
#pragma unroll
        for (int i = 0; i < BM_PER; ++i) f[i] = fmaxf(f[i], -INFINITY);
        ts = tile_sum(f, m);
      }
      s += ts;
    } else if (m == INFINITY) {
#pragma unroll
      for (int i = 0; i < BM_PER; ++i) s += exp_off(fmaxf(f[i], -INFINITY), m);
    }
    const int some = __syncthreads_count(tm > thr);
    if (some == 0) continue;
    float bound = -INFINITY;
    if (some > BM_FULL / 4) {
      // many: the k-th largest of the maxima of 64 groups of 8 threads has at
      // least k of this tile's logits at or above it
      float gm = tm;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
      if ((lane & 7) == 0) sm.group[warp * 4 + (lane >> 3)] = gm;
      __syncthreads();
      kth_group<64>(sm.group, k, &sm.bound);
      bound = sm.bound;
    }
    int at = -1;
    if (tm > thr && tm >= bound) {
#pragma unroll
      for (int i = 0; i < BM_PER; ++i)
        if (f[i] > thr && f[i] >= bound) {
          at = atomicAdd(&sm.n_cand, 1);
          sm.cand[at] = make_key(f[i], t0 + ((i >> 2) * BM_THREADS + tid) * 4 + (i & 3));
        }
    }
    // k logits with lower codes are at or above the bound: a later one must pass it
    thr = fmaxf(thr, bound);
    // the buffer is full, or this was the first of several tiles: from now on a
    // logit must pass the k-th best so far
    if (__syncthreads_or(at >= BM_FULL || (at >= k && t0 == v0 && t0 + BM_TILE < v1))) {
      keep_best(sm, sm.n_cand, k);
      if (tid < k) sm.cand[tid] = sm.best[tid];
      if (tid == 0) sm.n_cand = k;
      thr = key_value(sm.best[k - 1]);
      __syncthreads();
    }
  }
  __syncthreads();
  keep_best(sm, sm.n_cand, k);
  // the threads' maxima and sums
  const float wm = warp_max(m);
  const float ws = warp_sum(s * exp_off(m, wm));
  if (lane == 0) {
    sm.red[0][warp] = wm;
    sm.red[1][warp] = ws;
  }
  __syncthreads();
  if (warp == 0) {
    const float m1 = lane < BM_WARPS ? sm.red[0][lane] : -INFINITY;
    const float s1 = lane < BM_WARPS ? sm.red[1][lane] : 0.f;
    const float mm = warp_max(m1);
    const float ss = warp_sum(s1 * exp_off(m1, mm));
    if (lane == 0) {
      out.mx = mm;
      out.sum = ss;
    }
    if (lane < k) out.list[lane] = sm.best[lane];
  }
}

// Codes from v0 on of row gb (a finished beam: its one candidate, where they start).
template <bool HIST>
__device__ __forceinline__ void scan_row(BeamSmem& sm, Piece& out, const BeamArgs& a, int gb, int v0, int len) {
  const int row = a.row_ids ? a.row_ids[gb] : gb, tid = threadIdx.x;
  if (a.finished && a.finished[row]) {
    if (tid < a.k) out.list[tid] = v0 == 0 && tid == 0 ? make_key(0.f, a.eos) : 0;
    if (tid == 0) {
      out.mx = 0.f;
      out.sum = v0 == 0 ? 1.f : 0.f;
    }
    return;
  }
  scan_piece<HIST>(sm, out, a, a.logits + (size_t)row * a.ld, HIST ? a.history + (size_t)row * a.vocab : nullptr, v0,
                   min(a.vocab, v0 + len));
}

template <bool HIST>
__global__ void __launch_bounds__(BM_THREADS, 2) beam_scan_kernel(BeamArgs a, int pieces, int piece_len, Piece* ws) {
  extern __shared__ __align__(16) uint8_t bm_raw[];
  pdl_wait();
  pdl_trigger();
  scan_row<HIST>(*reinterpret_cast<BeamSmem*>(bm_raw), ws[blockIdx.x], a, blockIdx.x / pieces,
                 (int)(blockIdx.x % pieces) * piece_len, piece_len);
}

// Natural logarithm of a positive normal number to about 1e-10: x = 2^e m with m
// in [sqrt(1/2), sqrt(2)), log m = 2 atanh(t) = 2 (t + t^3/3 + t^5/5 + ..), t =
// (m - 1) / (m + 1), |t| <= 0.172 (the first term left out is below 2e-11).  A
// short chain: the fp64 units are slow, and the sums it is taken of are fp32's.
__device__ __forceinline__ double log_of(double x) {
  const long long b = __double_as_longlong(x);
  int e = (int)(b >> 52) - 1023;
  double m = __longlong_as_double((b & 0xfffffffffffffll) | 0x3ff0000000000000ll);
  if (m > 1.4142135623730951) {
    m *= 0.5;
    e += 1;
  }
  const double d = m + 1.0;
  double r = (double)(1.0f / (float)d);
  r = fma(r, fma(-d, r, 1.0), r);  // one Newton step
  const double t = (m - 1.0) * r, t2 = t * t;
  const double p = fma(t2, fma(t2, fma(t2, fma(t2, 1.0 / 11.0, 1.0 / 9.0), 1.0 / 7.0), 1.0 / 5.0), 1.0 / 3.0);
  return fma((double)e, 0.6931471805599453, 2.0 * fma(t * t2, p, t));
}

// score = (hi + lo) + (x - mx) as an ordered integer, 0 for none (-inf or NaN): a
// sum of two floats (about 48 bits), the larger one's bits above the smaller
// one's.  (The fp64 units are too slow for a thousand of these.)
__device__ __forceinline__ u64 score_key(float hi, float lo, float x, float mx) {
  if (!(hi > -INFINITY)) return 0;
  float h, l;
  if (fabsf(hi) < 1e36f && (x == mx || (fabsf(x) < 1e36f && fabsf(mx) < 1e36f))) {
    // x - mx = d + e exactly (infinite logits share the weight: 0)
    const float d = x == mx ? 0.f : x - mx;
    const float t = d - x, e = x == mx ? 0.f : (x - (d - t)) + (-mx - t);
    // hi + d = s + f exactly
    const float s = hi + d, u = s - hi, f = (hi - (s - u)) + (d - u);
    const float r = f + (lo + e);
    h = s + r;
    l = h - h == 0.f ? (s - h) + r : 0.f;
  } else {  // sums that may leave fp32's range
    const double v = ((double)hi + (double)lo) + (x == mx ? 0.0 : (double)x - (double)mx);
    if (!(v > -INFINITY)) return 0;
    h = (float)fmin(fmax(v, -3.4028234663852886e38), 3.4028234663852886e38);
    l = (float)(v - (double)h);
    if (v == INFINITY) h = INFINITY, l = 0.f;
  }
  return ((u64)ordered(h) << 32) | ordered(l + 0.f);
}
// The score of a key, rounded once.
__device__ __forceinline__ float score_of(u64 k) { return key_value(k) + key_value(k << 32); }

// Joins group g's lists, at most LISTS (list(u): the u-th, piece by piece of beam by
// beam): every entry's score, a bound that the k best are at or above (as in the
// scan), and the order of what passes it.  Lane i of a warp holds entry i of its
// lists.
template <int LISTS, class List>
__device__ __forceinline__ void join_lists(JoinSmem& jn, const BeamArgs& a, int g, int pieces, List list) {
  constexpr int PER = LISTS / BM_WARPS;  // lists of a warp
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
  const int lists = a.beams * pieces;
  u64 key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int u = warp + i * BM_WARPS;
    key[i] = u < lists && lane < k ? list(u)->list[lane] : 0;
  }
  if (tid < a.beams) {
    float mm = -INFINITY;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) mm = fmaxf(mm, list(tid * pieces + p)->mx);
    double ss = 0.0;
#pragma unroll 4
    for (int p = 0; p < pieces; ++p) {
      const Piece* q = list(tid * pieces + p);
      ss += (double)(q->sum * exp_off(q->mx, mm));
    }
    // what a candidate's logit is scored against
    const double base = (double)a.scores[g * a.beams + tid] - (ss > 0.0 ? log_of(ss) : 0.0);
    jn.hi[tid] = (float)base;
    jn.lo[tid] = fabs(base) < INFINITY ? (float)(base - (double)(float)base) : 0.f;
    jn.mx[tid] = mm;
  }
  if (tid == 0) jn.n_cand = 0;
  __syncthreads();
  u64 sc[PER], best = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    sc[i] = 0;
    if (key[i] != 0) {
      const int b = (warp + i * BM_WARPS) / pieces;
      sc[i] = score_key(jn.hi[b], jn.lo[b], key_value(key[i]), jn.mx[b]);
    }
    best = sc[i] > best ? sc[i] : best;
  }
  // groups of lanes l, l + 8, l + 16 and l + 24 (of sorted lists: the larger
  // entries apart), by the scores' high words
  uint32_t top = (uint32_t)(best >> 32);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
  if (lane < 8) jn.group[warp * 8 + lane] = top;
  __syncthreads();
  kth_group<128>(jn.group, k, &jn.bound);
  const uint32_t bound = jn.bound;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (sc[i] != 0 && (uint32_t)(sc[i] >> 32) >= bound) {
      const int at = atomicAdd(&jn.n_cand, 1);
      jn.score[at] = sc[i];
      jn.key[at] = key[i];
      jn.row[at] = (warp + i * BM_WARPS) / pieces;
    }
  __syncthreads();
  const int n = jn.n_cand;
  for (int i = warp; i < n; i += BM_WARPS) {
    const u64 s0 = jn.score[i], k0 = jn.key[i];
    const int b0 = jn.row[i];
    int r = 0;
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      bool before = false;
      if (j < n) {
        const u64 s1 = jn.score[j];
        before = s1 > s0 || (s1 == s0 && (jn.row[j] < b0 || (jn.row[j] == b0 && jn.key[j] > k0)));
      }
      r += __popc(__ballot_sync(0xffffffffu, before));
    }
    if (lane == 0 && r < k) {
      a.tokens[g * k + r] = key_code(k0);
      a.parents[g * k + r] = b0;
      a.scores_out[g * k + r] = score_of(s0);
    }
  }
  if (tid >= n && tid < k) {  // no candidate left for the slot
    a.tokens[g * k + tid] = -1;
    a.parents[g * k + tid] = 0;
    a.scores_out[g * k + tid] = -INFINITY;
  }
}

__global__ void __launch_bounds__(BM_THREADS) beam_join_kernel(BeamArgs a, int pieces, const Piece* ws) {
  extern __shared__ __align__(16) uint8_t bm_raw[];
  pdl_wait();
  pdl_trigger();
  const Piece* pc = ws + (size_t)blockIdx.x * a.beams * pieces;
  join_lists<BM_LISTS>(*reinterpret_cast<JoinSmem*>(bm_raw), a, blockIdx.x, pieces, [&](int u) { return pc + u; });
}

// A group of up to BM_GROUP beams whose rows are scanned whole: a cluster with a
// CTA for each row, the first of which joins the lists.
template <bool HIST>
__global__ void __launch_bounds__(BM_THREADS, 2) beam_group_kernel(BeamArgs a) {
  extern __shared__ __align__(16) uint8_t bm_raw[];
  __shared__ Piece mine;
  cg::cluster_group cl = cg::this_cluster();
  pdl_wait();
  pdl_trigger();
  scan_row<HIST>(*reinterpret_cast<BeamSmem*>(bm_raw), mine, a, blockIdx.x, 0, a.vocab);
  cl.sync();
  if (cl.block_rank() == 0)
    join_lists<BM_WARPS>(*reinterpret_cast<JoinSmem*>(bm_raw), a, blockIdx.x / a.beams, 1,
                         [&](int u) -> const Piece* { return cl.map_shared_rank(&mine, u); });
  cl.sync();  // the first CTA has read the others' lists
}

// --------------------------------------------------------------- reordering
//
// Bytes moved once: a block column per row (or, in place, per group) and set, all
// sets of a kind in one launch; a word of every row of a group is read before one
// is written in place.  32 groups of 4 beams' 12 KB: 2.4 us; 64 of 32 beams' 266 KB
// (1.1 GB moved, some of it read twice): 135 us, in place 174.

constexpr int RO_SETS = 8;
constexpr int RO_THREADS = 256;
constexpr int RO_UNROLL = 4;  // loads in flight per thread

struct RowSets {
  q3tts_rows set[RO_SETS];
};

template <class W>
__device__ __forceinline__ void gather_row(const q3tts_rows& r, int src_row, int dst_row, size_t w0, size_t words) {
  const W* s = reinterpret_cast<const W*>(static_cast<const uint8_t*>(r.src) + (size_t)src_row * r.src_stride);
  W* d = reinterpret_cast<W*>(static_cast<uint8_t*>(r.dst) + (size_t)dst_row * r.dst_stride);
  const size_t step = (size_t)gridDim.x * RO_THREADS;
  if (step >= words) {
    if (w0 < words) d[w0] = s[w0];
    return;
  }
  for (size_t w = w0; w < words; w += RO_UNROLL * step) {
    W v[RO_UNROLL];
#pragma unroll
    for (int u = 0; u < RO_UNROLL; ++u)
      if (w + u * step < words) v[u] = s[w + u * step];
#pragma unroll
    for (int u = 0; u < RO_UNROLL; ++u)
      if (w + u * step < words) d[w + u * step] = v[u];
  }
}

// dst row (g, j) = src row (g, parents[g][j]); src and dst do not overlap.
__global__ void __launch_bounds__(RO_THREADS) gather_rows_kernel(const __grid_constant__ RowSets sets,
                                                                 const int* row_ids, const int* parents, int beams_in,
                                                                 int beams_out, int* status) {
  pdl_wait();
  pdl_trigger();
  const q3tts_rows& r = sets.set[blockIdx.z];
  const int g = blockIdx.y / beams_out;
  const int p = parents[blockIdx.y];
  if (p < 0 || p >= beams_in) {
    if (threadIdx.x == 0 && blockIdx.x == 0) op_status(status, Q3TTS_ERR_ARG);
    return;
  }
  const int si = g * beams_in + p, di = blockIdx.y;
  const int sr = row_ids ? row_ids[si] : si, dr = row_ids ? row_ids[di] : di;
  const size_t w0 = (size_t)blockIdx.x * RO_THREADS + threadIdx.x;
  const uintptr_t al = (uintptr_t)r.src | (uintptr_t)r.dst | r.src_stride | r.dst_stride | r.row_bytes;
  if ((al & 15) == 0)
    gather_row<uint4>(r, sr, dr, w0, r.row_bytes / 16);
  else if ((al & 3) == 0)
    gather_row<uint32_t>(r, sr, dr, w0, r.row_bytes / 4);
  else
    gather_row<uint8_t>(r, sr, dr, w0, r.row_bytes);
}

// In place: a thread reads its word of every row of the group before it writes
// any of them.
template <class W, int MAXB>
__device__ __forceinline__ void permute_word(const q3tts_rows& r, const int* row, const int* par, int beams, size_t w) {
  W v[MAXB];
#pragma unroll
  for (int j = 0; j < MAXB; ++j)
    if (j < beams && par[j] != j)
      v[j] = reinterpret_cast<const W*>(static_cast<const uint8_t*>(r.src) + (size_t)row[par[j]] * r.src_stride)[w];
#pragma unroll
  for (int j = 0; j < MAXB; ++j)
    if (j < beams && par[j] != j)
      reinterpret_cast<W*>(static_cast<uint8_t*>(r.dst) + (size_t)row[j] * r.dst_stride)[w] = v[j];
}

template <int MAXB>
__global__ void __launch_bounds__(RO_THREADS) permute_rows_kernel(const __grid_constant__ RowSets sets,
                                                                  const int* row_ids, const int* parents, int beams,
                                                                  int* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ int row[MAXB], par[MAXB];
  const q3tts_rows& r = sets.set[blockIdx.z];
  const int g = blockIdx.y;
  if (threadIdx.x < beams) {
    const int i = g * beams + threadIdx.x;
    int p = parents[i];
    if (p < 0 || p >= beams) {  // reported; the row stays as it is
      op_status(status, Q3TTS_ERR_ARG);
      p = threadIdx.x;
    }
    par[threadIdx.x] = p;
    row[threadIdx.x] = row_ids ? row_ids[i] : i;
  }
  __syncthreads();
  const uintptr_t al = (uintptr_t)r.src | r.src_stride | r.row_bytes;
  const size_t w0 = (size_t)blockIdx.x * RO_THREADS + threadIdx.x, step = (size_t)gridDim.x * RO_THREADS;
  if ((al & 15) == 0)
    for (size_t w = w0; w < r.row_bytes / 16; w += step) permute_word<uint4, MAXB>(r, row, par, beams, w);
  else if ((al & 3) == 0)
    for (size_t w = w0; w < r.row_bytes / 4; w += step) permute_word<uint32_t, MAXB>(r, row, par, beams, w);
  else
    for (size_t w = w0; w < r.row_bytes; w += step) permute_word<uint8_t, MAXB>(r, row, par, beams, w);
}

}  // namespace

// Pieces of a row: enough CTAs for two on every SM, each of whole tiles, and no
// more lists in a group than the join holds.
static int beam_pieces(int groups, int beams, int vocab, int n_sm, int* len) {
  const int tiles = (vocab + BM_TILE - 1) / BM_TILE;
  const long rows = (long)groups * beams;
  long p = 2l * n_sm / rows;
  p = p < BM_LISTS / beams ? p : BM_LISTS / beams;
  p = p < 1 ? 1 : (p < tiles ? p : tiles);
  const int per = (tiles + (int)p - 1) / (int)p;
  *len = per * BM_TILE;
  return (tiles + per - 1) / per;
}

size_t beam_workspace(int groups, int beams, int vocab, int n_sm) {
  int len = 0;
  const int pieces = beam_pieces(groups, beams, vocab, n_sm, &len);
  return pieces == 1 && beams <= BM_GROUP ? 0 : sizeof(Piece) * (size_t)groups * beams * pieces;
}

int launch_beam_select(const BeamArgs& a, void* workspace, cudaStream_t s) {
  if (a.groups <= 0) return Q3TTS_OK;
  int dev = 0, n_sm = 0;
  if (!current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  static std::atomic<bool> ready[kMaxDevices];  // the attributes are the device's
  constexpr size_t kGroupSmem = sizeof(BeamSmem) > sizeof(JoinSmem) ? sizeof(BeamSmem) : sizeof(JoinSmem);
  if (!ready[dev].load(std::memory_order_acquire)) {
    auto allow = [](auto kernel, size_t smem) {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
    };
    if (!allow(beam_scan_kernel<false>, sizeof(BeamSmem)) || !allow(beam_scan_kernel<true>, sizeof(BeamSmem)) ||
        !allow(beam_join_kernel, sizeof(JoinSmem)) || !allow(beam_group_kernel<false>, kGroupSmem) ||
        !allow(beam_group_kernel<true>, kGroupSmem))
      return Q3TTS_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  int len = 0;
  const int pieces = beam_pieces(a.groups, a.beams, a.vocab, n_sm, &len);
  if (pieces == 1 && a.beams <= BM_GROUP) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.groups * a.beams));
    cfg.blockDim = dim3(BM_THREADS);
    cfg.dynamicSmemBytes = kGroupSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.beams;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = pdl_enabled() ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, a.history ? beam_group_kernel<true> : beam_group_kernel<false>, a) == cudaSuccess
               ? Q3TTS_OK
               : Q3TTS_ERR_CUDA;
  }
  Piece* ws = static_cast<Piece*>(workspace);
  const dim3 grid((unsigned)((long)a.groups * a.beams * pieces));
  const cudaError_t e = launch_pdl(a.history ? beam_scan_kernel<true> : beam_scan_kernel<false>, grid, dim3(BM_THREADS),
                                   sizeof(BeamSmem), s, a, pieces, len, ws);
  if (e != cudaSuccess ||
      launch_pdl(beam_join_kernel, dim3(a.groups), dim3(BM_THREADS), sizeof(JoinSmem), s, a, pieces, (const Piece*)ws) !=
          cudaSuccess)
    return Q3TTS_ERR_CUDA;
  return Q3TTS_OK;
}

int launch_reorder_rows(const q3tts_rows* sets, int n_sets, const int* row_ids, const int* parents, int groups,
                        int beams_in, int beams_out, int* status, cudaStream_t s) {
  if (groups <= 0) return Q3TTS_OK;
  int dev = 0, n_sm = 0;
  if (!current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  for (int inplace = 0; inplace < 2; ++inplace) {
    for (int i0 = 0; i0 < n_sets;) {
      RowSets p = {};
      int m = 0;
      size_t most = 0;
      for (; i0 < n_sets && m < RO_SETS; ++i0)
        if ((sets[i0].src == sets[i0].dst) == (inplace != 0) && sets[i0].row_bytes) {
          p.set[m++] = sets[i0];
          const size_t words = sets[i0].row_bytes / 16 + 1;
          most = words > most ? words : most;
        }
      if (!m) continue;
      const size_t blocks = (most + RO_THREADS - 1) / RO_THREADS;
      // a row of a gather goes to more CTAs only while there are few rows (64 x 32 rows
      // of 262 KB: 346 us with a CTA for each 4 KB of a row)
      const size_t few = (size_t)(8 * n_sm / (groups * beams_out * m) + 1), most_x = inplace ? 1024 : few;
      const unsigned bx = (unsigned)(blocks < most_x ? blocks : most_x);
      cudaError_t e;
      if (!inplace)
        e = launch_pdl(gather_rows_kernel, dim3(bx, groups * beams_out, m), dim3(RO_THREADS), 0, s, p, row_ids, parents,
                       beams_in, beams_out, status);
      else if (beams_out <= 8)
        e = launch_pdl(permute_rows_kernel<8>, dim3(bx, groups, m), dim3(RO_THREADS), 0, s, p, row_ids, parents,
                       beams_out, status);
      else
        e = launch_pdl(permute_rows_kernel<BM_MAXB>, dim3(bx, groups, m), dim3(RO_THREADS), 0, s, p, row_ids, parents,
                       beams_out, status);
      if (e != cudaSuccess) return Q3TTS_ERR_CUDA;
    }
  }
  return Q3TTS_OK;
}

}  // namespace q3

// beam.cu -- beam selection over beams and vocabulary, and the reordering of
// per-beam state that follows it.
//
// Row (g, b) holds the logits of beam b of group g.  With x the logits after
// the repetition penalty and the mask of special codes (the sampler's rule),
//   score(b, v) = scores[b] + (x_v - max x) - log sum_v e^(x_v - max x),
// and a group keeps the k candidates with the largest scores among its beams'
// vocabularies.  Scores are compared in 64 bits, so that candidates of
// different beams order as their exact values do; equal scores go to the lower
// beam, then the larger logit, then the lower code.  A finished beam offers one
// candidate, its end code at its own score.
//
// Within a row scores order as logits do, so a row's own k best logits are all
// it can contribute.  One pass over a row keeps the running maximum and sum of
// its softmax and its k best logits; the CTAs of one cluster share a group's
// rows (and pieces of long rows) and the first of them joins the lists through
// distributed shared memory: one launch, no workspace.
#include <cooperative_groups.h>

#include "ops.cuh"

namespace cg = cooperative_groups;

namespace q3 {

namespace {

constexpr int BM_THREADS = 512, BM_WARPS = BM_THREADS / 32;
constexpr int BM_PER = 16;                       // logits of a thread per tile
constexpr int BM_TILE = BM_THREADS * BM_PER;     // logits of a tile
constexpr int BM_MAXK = 32;                      // candidates kept
constexpr int BM_MAXB = 32;                      // beams of a group
constexpr int BM_MAXC = 8;                       // CTAs of a cluster
constexpr int BM_UNITS = BM_MAXB;                // units a CTA can hold (a cluster of one)
constexpr int BM_CAND = BM_TILE + BM_MAXK;       // candidates of one tile at most

typedef unsigned long long u64;

// Larger key: larger logit, then lower code.  Keys of a row are distinct; 0 is
// below every key.
__device__ __forceinline__ u64 make_key(float x, int v) {
  const uint32_t b = __float_as_uint(x);
  const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((u64)o << 32) | (uint32_t)~v;
}
__device__ __forceinline__ float key_value(u64 k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}
__device__ __forceinline__ int key_code(u64 k) { return (int)~(uint32_t)k; }

struct BeamSmem {
  u64 list[BM_UNITS][BM_MAXK];  // a unit's best keys in order (0: none)
  float mx[BM_UNITS], sum[BM_UNITS];
  int done[BM_UNITS];
  float red[2][32];
  float group[32];
  u64 best[BM_MAXK], top[BM_MAXK];
  int n_cand;
  u64 cand[BM_CAND];
};

// What the first CTA joins: candidates of all rows, at most max(beams, CTAs) k.
struct JoinSmem {
  double lse[BM_MAXB];  // log of the row's sum, relative to its maximum
  float mx[BM_MAXB];
  double score[BM_MAXB * BM_MAXK];
  u64 key[BM_MAXB * BM_MAXK];
  int row[BM_MAXB * BM_MAXK];
};
static_assert(sizeof(JoinSmem) <= sizeof(u64) * BM_CAND, "the join reuses the candidate buffer");

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
  if (tid < n) {
    const u64 key = from[tid];
    int r = 0;
    for (int j = 0; j < n; ++j) r += from[j] > key;
    if (r < k) sm.best[r] = key;
  }
  __syncthreads();
}

// A finite or +inf logit after penalty and mask; -inf where it cannot be
// picked (NaN counts as -inf).
__device__ __forceinline__ float rule(float x, int v, bool seen, const BeamArgs& a) {
  if (seen) x = x > 0.f ? x / a.penalty : x * a.penalty;
  if (a.special_from > 0 && v >= a.special_from && v != a.eos) x = -INFINITY;
  return x > -INFINITY ? x : -INFINITY;
}

// e^(x - m), with e^0 = 1 where both are infinite
__device__ __forceinline__ float exp_off(float x, float m) { return x == m ? (x == -INFINITY ? 0.f : 1.f) : expf(x - m); }

// One row's codes [v0, v1): running maximum and sum, and the k best keys.
__device__ void scan_piece(BeamSmem& sm, const BeamArgs& a, const float* x, const uint8_t* hist, int v0, int v1,
                           int unit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
  const bool vec = ((uintptr_t)(x + v0) & 15) == 0 && (!hist || ((uintptr_t)(hist + v0) & 3) == 0);
  float m = -INFINITY, s = 0.f;
  int have = 0;  // candidates kept so far
  float thr = -INFINITY;
  if (tid < BM_MAXK) sm.best[tid] = 0;
  for (int t0 = v0; t0 < v1; t0 += BM_TILE) {
    float f[BM_PER];
    int code0[BM_PER / 4];
#pragma unroll
    for (int j = 0; j < BM_PER / 4; ++j) {
      const int c = t0 + (j * BM_THREADS + tid) * 4;
      code0[j] = c;
      float4 w = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      uint32_t hb = 0;
      if (vec && c + 4 <= v1) {
        w = __ldcs(reinterpret_cast<const float4*>(x + c));
        if (hist) hb = __ldcs(reinterpret_cast<const unsigned int*>(hist + c));
      } else {
        if (c < v1) w.x = x[c];
        if (c + 1 < v1) w.y = x[c + 1];
        if (c + 2 < v1) w.z = x[c + 2];
        if (c + 3 < v1) w.w = x[c + 3];
        if (hist)
          for (int e = 0; e < 4; ++e)
            if (c + e < v1) hb |= (uint32_t)hist[c + e] << (8 * e);
      }
      f[4 * j] = rule(w.x, c, hb & 0xffu, a);
      f[4 * j + 1] = rule(w.y, c + 1, hb & 0xff00u, a);
      f[4 * j + 2] = rule(w.z, c + 2, hb & 0xff0000u, a);
      f[4 * j + 3] = rule(w.w, c + 3, hb & 0xff000000u, a);
    }
    float tm = f[0];
#pragma unroll
    for (int i = 1; i < BM_PER; ++i) tm = fmaxf(tm, f[i]);
    const float mn = fmaxf(m, tm);
    s *= exp_off(m, mn);
#pragma unroll
    for (int i = 0; i < BM_PER; ++i) s += exp_off(f[i], mn);
    m = mn;
    // candidates: logits above the k-th kept one (a later equal logit has a
    // higher code and loses)
    if (!__syncthreads_or(tm > thr)) continue;
    // a bound from this tile: the k-th largest of the maxima of 32 groups of
    // 16 threads has at least k logits at or above it
    float gm = tm;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, o));
    if ((lane & 15) == 0) sm.group[warp * 2 + (lane >> 4)] = gm;
    if (tid < have) sm.cand[tid] = sm.best[tid];
    if (tid == 0) sm.n_cand = have;
    __syncthreads();
    const float gv = sm.group[lane];
    int r = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(0xffffffffu, gv, j);
      r += o > gv || (o == gv && j < lane);
    }
    const unsigned at = __ballot_sync(0xffffffffu, r == k - 1);
    const float bound = __shfl_sync(0xffffffffu, gv, __ffs(at) - 1);
    if (tm > thr && tm >= bound) {
#pragma unroll
      for (int i = 0; i < BM_PER; ++i)
        if (f[i] > thr && f[i] >= bound) {
          const int c = code0[i >> 2] + (i & 3);
          sm.cand[atomicAdd(&sm.n_cand, 1)] = make_key(f[i], c);
        }
    }
    __syncthreads();
    const int n = sm.n_cand;
    keep_best(sm, n, k);
    have = min(n, k);
    if (have == k) thr = key_value(sm.best[k - 1]);
  }
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
      sm.mx[unit] = mm;
      sm.sum[unit] = ss;
    }
  }
  if (tid < BM_MAXK) sm.list[unit][tid] = tid < have ? sm.best[tid] : 0;
  __syncthreads();
}

__global__ void __launch_bounds__(BM_THREADS) beam_select_kernel(BeamArgs a, int pieces, int piece_len) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) uint8_t bm_raw[];
  BeamSmem& sm = *reinterpret_cast<BeamSmem*>(bm_raw);
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int g = blockIdx.x / C, tid = threadIdx.x, k = a.k;
  const int units = a.beams * pieces;
  for (int u = rank, slot = 0; u < units; u += C, ++slot) {
    const int b = u / pieces, piece = u % pieces;
    const int row = a.row_ids ? a.row_ids[g * a.beams + b] : g * a.beams + b;
    const bool done = a.finished && a.finished[row];
    if (tid == 0) sm.done[slot] = done;
    if (done) {  // one candidate, from the first piece
      if (tid < BM_MAXK) sm.list[slot][tid] = piece == 0 && tid == 0 ? make_key(0.f, a.eos) : 0;
      if (tid == 0) {
        sm.mx[slot] = 0.f;
        sm.sum[slot] = piece == 0 ? 1.f : 0.f;
      }
      __syncthreads();
    } else {
      const int v0 = piece * piece_len, v1 = min(a.vocab, v0 + piece_len);
      scan_piece(sm, a, a.logits + (size_t)row * a.ld, a.history ? a.history + (size_t)row * a.vocab : nullptr, v0, v1,
                 slot);
    }
  }
  cl.sync();
  if (rank == 0) {
    JoinSmem& jn = *reinterpret_cast<JoinSmem*>(sm.cand);
    // log of each row's sum, relative to its maximum, in 64 bits
    if (tid < a.beams) {
      float mm = -INFINITY;
      for (int p = 0; p < pieces; ++p) {
        const int u = tid * pieces + p;
        mm = fmaxf(mm, *cl.map_shared_rank(&sm.mx[u / C], u % C));
      }
      double ss = 0.0;
      for (int p = 0; p < pieces; ++p) {
        const int u = tid * pieces + p;
        const float pm = *cl.map_shared_rank(&sm.mx[u / C], u % C);
        ss += (double)*cl.map_shared_rank(&sm.sum[u / C], u % C) * (double)exp_off(pm, mm);
      }
      jn.lse[tid] = log(ss);
      jn.mx[tid] = mm;
    }
    if (tid == 0) sm.n_cand = 0;
    __syncthreads();
    for (int e = tid; e < units * k; e += BM_THREADS) {
      const int u = e / k, b = u / pieces;
      const u64 key = *cl.map_shared_rank(&sm.list[u / C][e % k], u % C);
      if (key == 0) continue;
      const float x = key_value(key), mm = jn.mx[b];
      // (x - max) - log sum; infinite logits share the weight
      const double d = x == mm ? 0.0 : (double)x - (double)mm;
      const double sc = (double)a.scores[g * a.beams + b] + (d - jn.lse[b]);
      if (!(sc > -INFINITY)) continue;
      const int i = atomicAdd(&sm.n_cand, 1);
      jn.score[i] = sc;
      jn.key[i] = key;
      jn.row[i] = b;
    }
    __syncthreads();
    const int n = sm.n_cand;
    for (int i = tid; i < n; i += BM_THREADS) {
      const double sc = jn.score[i];
      const u64 key = jn.key[i];
      const int b = jn.row[i];
      int r = 0;
      for (int j = 0; j < n && r < k; ++j) {
        const double so = jn.score[j];
        r += so > sc || (so == sc && (jn.row[j] < b || (jn.row[j] == b && jn.key[j] > key)));
      }
      if (r < k) {
        a.tokens[g * k + r] = key_code(key);
        a.parents[g * k + r] = b;
        a.scores_out[g * k + r] = (float)sc;
      }
    }
    if (tid >= n && tid < k) {  // no candidate left for the slot
      a.tokens[g * k + tid] = -1;
      a.parents[g * k + tid] = 0;
      a.scores_out[g * k + tid] = -INFINITY;
    }
  }
  cl.sync();  // rank 0 still reads the others' lists until here
}

// --------------------------------------------------------------- reordering

constexpr int RO_SETS = 8;
constexpr int RO_THREADS = 256;

struct RowSets {
  q3tts_rows set[RO_SETS];
};

template <class W>
__device__ __forceinline__ void gather_row(const q3tts_rows& r, int src_row, int dst_row, size_t w0, size_t words) {
  const W* s = reinterpret_cast<const W*>(static_cast<const uint8_t*>(r.src) + (size_t)src_row * r.src_stride);
  W* d = reinterpret_cast<W*>(static_cast<uint8_t*>(r.dst) + (size_t)dst_row * r.dst_stride);
  for (size_t w = w0; w < words; w += (size_t)gridDim.x * RO_THREADS) d[w] = s[w];
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

int launch_beam_select(const BeamArgs& a, cudaStream_t s) {
  if (a.groups <= 0) return Q3TTS_OK;
  int dev = 0, n_sm = 0;
  if (!current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  static bool ready[kMaxDevices] = {};
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(beam_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(BeamSmem)) !=
        cudaSuccess)
      return Q3TTS_ERR_CUDA;
    ready[dev] = true;
  }
  // CTAs of a group: one per tile of its rows, at most the portable cluster
  // size; rows are cut into pieces where a group has fewer rows than CTAs
  const int tiles = (a.vocab + BM_TILE - 1) / BM_TILE;
  int c = 1;
  while (c < BM_MAXC && c < a.beams * tiles) c *= 2;
  const int want = a.beams < c ? c / a.beams : 1;
  const int per = (tiles + want - 1) / want;  // tiles of a piece
  const int pieces = (tiles + per - 1) / per;
  if ((long)a.groups * c > 0x7fffffffL) return Q3TTS_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.groups * c));
  cfg.blockDim = dim3(BM_THREADS);
  cfg.dynamicSmemBytes = sizeof(BeamSmem);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, beam_select_kernel, a, pieces, per * BM_TILE) == cudaSuccess ? Q3TTS_OK
                                                                                              : Q3TTS_ERR_CUDA;
}

int launch_reorder_rows(const q3tts_rows* sets, int n_sets, const int* row_ids, const int* parents, int groups,
                        int beams_in, int beams_out, int* status, cudaStream_t s) {
  if (groups <= 0) return Q3TTS_OK;
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
      const unsigned bx = (unsigned)(blocks < 1024 ? blocks : 1024);
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

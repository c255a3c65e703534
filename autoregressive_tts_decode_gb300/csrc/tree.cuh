// tree.cuh -- what the two kernels of tree attention share (tree_attention.cu,
// tree_wide.cu): the work items, the tensor-core and copy instructions, the
// bounded wait.
#pragma once

#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "ops.cuh"

namespace q3 {

// Trees of more than 64 rows (nodes x q heads of a group) over a bf16 cache whose
// pages TMA boxes fit (tree_wide.cu).
int launch_tree_wide(const TreeArgs& a, int layers, int dev, int n_sm, cudaStream_t s);

namespace {

// What a CTA works on; false when it has no rows.  Lengths and row offsets
// come from device memory, so they are checked here: a sequence whose entries
// do not fit the cache or the buffers is left out and reported.
struct TreeSeq {
  int L, T, row0, P;  // committed positions, nodes, first row of q/out, L + T
};
__device__ __forceinline__ bool tree_seq(const TreeArgs& a, int seq, TreeSeq& t) {
  t.L = a.lengths[seq];
  t.row0 = a.node_start[seq];
  const int end = a.node_start[seq + 1];
  const long long cap = (long long)a.kv.pages_per_stream * a.kv.page_size;
  if (t.row0 < 0 || end < t.row0 || end > a.n_rows || end - t.row0 > a.max_nodes || t.L < 0 ||
      (long long)t.L + (end - t.row0) > cap) {
    op_status(a.status, Q3TTS_ERR_ARG);
    return false;
  }
  t.T = end - t.row0;
  t.P = t.L + t.T;
  return t.T > 0;
}

constexpr int TM_PT = 128;       // positions of a tile
constexpr int TM_SORT = 256;     // sequences that are dealt by length, at most (no more than threads)
constexpr long long TM_LAND_CYCLES = 500000000ll;  // ~0.25 s: copies and products in flight on giving up
constexpr float TM_FLOOR = -1e30f;  // base of a row that has seen nothing: below every score (which are limited to 2^27:
                                    // c s - base is rounded where base is, by up to 2^-24 of it, a power of two to the weights)
constexpr float TM_SLACK = 8.f;     // how far (log2) a score may pass its row's base

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(uint32_t b, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(b), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 128-byte swizzled operand tiles: rows of 128 bytes, 8-row atoms 1024 bytes
// apart (stride byte offset), descriptor version 1, swizzle mode 2.  K-major:
// the leading offset is not used.  M-major (V^T: 64 head-dim elements are a
// row's 128 bytes, positions the rows): the leading offset is the distance of
// the second 64 elements' block.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lead = 16) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lead & 0x3FFFFu) >> 4) << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16: D fp32, A and B bf16, B K-major; A K-major or M-major (bit 15).
__host__ __device__ constexpr uint32_t f16_idesc(int M, int N, bool a_m_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_m_major ? 1u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_bf16(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(
          tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// One lane of the warp, in a form that lets the compiler keep the MMAs' operands in
// uniform registers; under a plain comparison of the lane each MMA took up to 95
// cycles to issue (45 with this).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n selp.u32 %0, 1, 0, e;\n}" : "=r"(p));
  return p != 0;
}
// 16 fp32 columns of the warp's 32 lanes, one lane per thread (complete after wait::ld).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Pairs of floats (one 64-bit register pair, one instruction each).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Two floats to bf16 (x in the low half).
__device__ __forceinline__ uint32_t pack_bf16(float2 v) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(v.y), "f"(v.x));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Infinities and NaN in 16 bytes of bf16: an exponent of ones carries into the sign
// bit's place (bits 15 and 31 of the result, gathered by or).
__device__ __forceinline__ uint32_t not_finite(uint4 u, uint32_t found) {
  found |= (u.x & 0x7f807f80u) + 0x00800080u;
  found |= (u.y & 0x7f807f80u) + 0x00800080u;
  found |= (u.z & 0x7f807f80u) + 0x00800080u;
  return found | ((u.w & 0x7f807f80u) + 0x00800080u);
}
// Bounded wait on an mbarrier phase; false on expiry or when another role of
// the CTA has given up (abort_w[0]; abort_w[1]: the limit in units of 1024 cycles).
__device__ __noinline__ bool tm_wait_long(uint32_t bar, uint32_t parity, volatile int* abort_w, int* status) {
  const long long t0 = clock64();
  unsigned it = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++it & 63u) == 0) {
      if (*abort_w) return false;
      if ((clock64() - t0) >> 10 >= abort_w[1]) {
        *abort_w = 1;
        op_status(status, Q3TTS_ERR_TIMEOUT);
        return false;
      }
    }
  }
  return true;
}
__device__ __forceinline__ bool tm_wait(uint32_t bar, uint32_t parity, volatile int* abort_w, int* status) {
  return mbar_try_wait(bar, parity) || tm_wait_long(bar, parity, abort_w, status);
}

// What a CTA that has given up waits for (bounded) before it leaves, once all its
// roles have ended: any of them may have been the one, with copies of a loading
// warp that was itself done still on their way into shared memory, or products
// into the tensor memory that is about to be given back.

// Copies of loading warp w (copies: the last eight ring tiles of S places that each
// of the two has filled, -1: none).  A place that was filled again had landed.
template <int S>
__device__ __forceinline__ void land_copies(const int (&copies)[2][8], int w, unsigned long long* full) {
  const int lane = threadIdx.x & 31, it = lane < 8 ? copies[w][lane] : -1;
  bool last = it >= 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int o = copies[j >> 3][j & 7];
    last = last && !(o > it && (o - it) % S == 0);
  }
  const long long c0 = clock64();
  while (last && !mbar_try_wait(su32(&full[it % S]), (uint32_t)(it / S) & 1u) && clock64() - c0 < TM_LAND_CYCLES) {
  }
}
// Products issued by the calling thread (`done`: a barrier of one arrival, not used before).
__device__ __forceinline__ void land_products(uint32_t done) {
  mma_commit(done);
  const long long c0 = clock64();
  while (!mbar_try_wait(done, 0u) && clock64() - c0 < TM_LAND_CYCLES) {
  }
}

// Ring position of tile t's K and V among n tiles: K0 K1 V0 K2 V1 .. V(n-1).
__device__ __forceinline__ int k_item(int t) { return t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int v_item(int t, int n) { return t == n - 1 ? 2 * n - 1 : 2 * t + 2; }

// One item of work.
struct TmItem {
  TreeSeq t;
  int seq, g, n0, rows;  // kv head, first row of the tile, rows
  int t0, nt;            // first position tile, tiles
};

// How the items are dealt.
struct TmDeal {
  int items, row_tiles, rows;  // rows of a tile
  int stride, first;           // clusters, this one
  int rank, cl;                // CTA of the cluster, CTAs
  const uint16_t* order;       // sequences, longest first, or NULL
};

// The k-th item of a CTA: 1 if there is one, 0 if it has no rows (or does not
// fit, which is reported), -1 past the last.
__device__ __forceinline__ int tm_item(const TreeArgs& a, const TmDeal& d, int k, TmItem& m) {
  if ((long long)k * d.stride >= d.items) return -1;
  const int idx = k * d.stride + ((k & 1) ? d.stride - 1 - d.first : d.first);
  if (idx >= d.items) return 0;
  const int rep = a.Hq / a.kv.Hkv;
  m.g = idx / d.row_tiles % a.kv.Hkv;
  m.seq = idx / d.row_tiles / a.kv.Hkv;
  if (d.order) m.seq = d.order[m.seq];
  m.n0 = idx % d.row_tiles * d.rows;
  if (!tree_seq(a, m.seq, m.t) || m.n0 >= m.t.T * rep) return 0;
  m.rows = min(d.rows, m.t.T * rep - m.n0);
  const int all = (m.t.P + TM_PT - 1) / TM_PT, per = (all + d.cl - 1) / d.cl;
  m.t0 = min(all, d.rank * per);
  m.nt = min(all, m.t0 + per) - m.t0;
  return 1;
}

// row / rep for rows of an item (rep_inv = ceil(2^32 / rep); exact for rows and rep up to 2^16)
__device__ __forceinline__ int div_rep(int row, int rep, unsigned rep_inv) {
  return rep == 1 ? row : (int)__umulhi((unsigned)row, rep_inv);
}

// Row of the pool ([layer][page][k|v][kv head][position]) of a position on `page`;
// a page that is not the pool's is reported and read as page 0.
__device__ __forceinline__ int pool_row(const TreeArgs& a, int g, bool values, int page, int pos) {
  const int ps = a.kv.page_size;
  if (page < 0 || page >= a.kv.n_pages) {
    op_status(a.status, Q3TTS_ERR_ARG);
    page = 0;
  }
  const long long plane = (long long)a.kv.Hkv * ps;  // rows of a page's keys (or values)
  return (int)((((long long)a.layer * a.kv.n_pages + page) * 2 + (values ? 1 : 0)) * plane + (long long)g * ps + pos % ps);
}

// A warp's TMA loads of the keys (or the values) of all items of the CTA into
// their places of a ring of S tiles.  Lane (b, blk) copies block blk of page b's
// rows of a tile.  A warp's lanes issue one by one, 55 cycles each: from one warp
// for keys and values the 32 copies of 2 KB of a tile of 16-position pages took
// longer than the tile's bytes.  copies: the last eight ring tiles filled, for
// land_copies.  S is at least three: a warp skips two ring tiles at most, which its
// parity waits bear.
template <int HD, int S>
__device__ __forceinline__ bool tma_loads(const CUtensorMap* map, const TreeArgs& a, const TmDeal& deal, int box, bool values,
                                          uint32_t ring, unsigned long long* full, unsigned long long* empty,
                                          int (&copies)[8], volatile int* abort_w) {
  static_assert(S >= 3 && S <= 8, "ring");
  constexpr int BLK = HD / 64;
  constexpr uint32_t SLOT = TM_PT * HD * 2;
  const int lane = threadIdx.x & 31, b = lane / BLK, blk = lane % BLK;
  const int boxes = TM_PT / box, ps = a.kv.page_size;
  TmItem m;
  int have, ic = 0, issued = 0;  // position tiles so far, TMA copies of this warp
  bool ok = true;
  for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
    if (have == 0 || m.nt == 0) continue;
    const int* table = a.kv.page_table + (size_t)m.seq * a.kv.pages_per_stream;
    // the page of this lane's box in tile i; looked up two tiles ahead and not
    // touched until then, so the lookup's latency is never waited for
    auto page_of = [&](int i) -> int {
      const int pos = (m.t0 + i) * TM_PT + b * box;
      return b < boxes && i < m.nt && pos < m.t.P ? __ldg(table + pos / ps) : 0;
    };
    int page_even = page_of(0), page_odd = page_of(1);
    for (int tile = 0; tile < m.nt; ++tile) {
      const int it = 2 * ic + (values ? v_item(tile, m.nt) : k_item(tile)), slot = it % S;
      const int pos = (m.t0 + tile) * TM_PT + b * box;
      const int page = (tile & 1) ? page_odd : page_even;
      const uint32_t fb = su32(&full[slot]);
      ok = __all_sync(0xffffffffu, tm_wait(su32(&empty[slot]), ((uint32_t)(it / S) & 1u) ^ 1u, abort_w, a.status));
      if (!ok) break;
      const int held = min(TM_PT, m.t.P - (m.t0 + tile) * TM_PT);
      if (lane == 0) mbar_expect_tx(fb, (uint32_t)((held + box - 1) / box * box * HD * 2));
      __syncwarp();
      if (b < boxes && pos < m.t.P)
        tma_load(ring + slot * SLOT + blk * (TM_PT * 128) + b * box * 128, map, blk * 64, pool_row(a, m.g, values, page, pos), fb);
      // the page two tiles on takes this one's place
      if (tile & 1) page_odd = page_of(tile + 2); else page_even = page_of(tile + 2);
      if (lane == 0) copies[issued % 8] = it;
      ++issued;
    }
    ic += m.nt;
  }
  return ok;
}

// The first item's lengths, row offsets and page ids on their way to the L2 before
// anything is known that leads to them.
__device__ __forceinline__ void prefetch_first(const TreeArgs& a, const TmDeal& d) {
  const int i = threadIdx.x, seq = d.first / d.row_tiles / a.kv.Hkv;
  if (seq >= a.n_seqs) return;
  const int* p = i == 0 ? a.lengths + seq : i == 1 ? a.node_start + seq : a.kv.page_table + (size_t)seq * a.kv.pages_per_stream + (i - 2) * 32;
  if (i < 2 || (i < 32 && (i - 2) * 32 < a.kv.pages_per_stream)) asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// The queries of an item as three bf16 terms (x = their sum), K-major swizzled
// tiles of N rows, by QT threads: four elements of a row each, up to sixteen loads
// on their way at a time, the first before `ready` says that Q's place is free.
template <int HD, int N, int QT, class Ready>
__device__ __forceinline__ bool load_queries(const TreeArgs& a, const TmItem& m, int rep, unsigned rep_inv, bool wide, int lane,
                                             uint8_t* dst0, Ready ready) {
  constexpr int CH = HD / 4, ALL = N * CH / QT, UNITS = ALL < 16 ? ALL : 16;
  static_assert(ALL % UNITS == 0, "whole batches");
  constexpr uint32_t TERM = N * 128;
#pragma unroll 1
  for (int u0 = 0; u0 < ALL; u0 += UNITS) {
    float4 x[UNITS];
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int e = (u0 + u) * QT + lane, n = e / CH, row = m.n0 + n, node = div_rep(row, rep, rep_inv);
      const float* q = a.q + (size_t)(m.t.row0 + node) * a.ldq + (size_t)(m.g * rep + row - node * rep) * HD + e % CH * 4;
      x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n < m.rows) x[u] = wide ? *reinterpret_cast<const float4*>(q) : make_float4(q[0], q[1], q[2], q[3]);
    }
    if (u0 == 0 && !ready()) return false;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int e = (u0 + u) * QT + lane, n = e / CH, c = e % CH;
      uint8_t* dst = dst0 + (c >> 4) * 3 * TERM + n * 128 + ((((c >> 1) & 7) ^ (n & 7)) << 4) + (c & 1) * 8;
      float2 v = make_float2(x[u].x, x[u].y), w = make_float2(x[u].z, x[u].w);
#pragma unroll
      for (int term = 0; term < 3; ++term) {
        const uint32_t p = pack_bf16(v), r = pack_bf16(w);
        *reinterpret_cast<uint2*>(dst + term * TERM) = make_uint2(p, r);
        v = add2(v, make_float2(-__uint_as_float(p << 16), -__uint_as_float(p & 0xffff0000u)));
        w = add2(w, make_float2(-__uint_as_float(r << 16), -__uint_as_float(r & 0xffff0000u)));
      }
    }
  }
  return true;
}

// The end of an item whose positions a cluster has shared: what each share's
// output of a row counts for (fac [CL][N] in shared memory), then every CL-th row.
// base, sum [N] and os [N][LD] are each share's own.
template <int HD, int N, int THREADS, int LD>
__device__ __forceinline__ void join_shares(const TreeArgs& a, const TmItem& m, int rep, unsigned rep_inv, bool wide, float* base,
                                            float* sum, float* fac, float* os, volatile int* abort_w) {
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank(), tid = threadIdx.x;
  cl.sync();
  if (tid < N) {
    float bs[8], sm[8], mx = TM_FLOOR, all = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      bs[r] = r < CL ? *cl.map_shared_rank(&base[tid], r) : TM_FLOOR;
      sm[r] = r < CL ? *cl.map_shared_rank(&sum[tid], r) : 0.f;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) mx = fmaxf(mx, bs[r]);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      bs[r] = sm[r] == 0.f ? 0.f : exp2_fast(bs[r] - mx);  // 0: the share saw nothing
      all = fmaf(sm[r], bs[r], all);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
      if (r < CL) fac[r * N + tid] = all == 0.f ? 0.f : bs[r] / all;
  }
  __syncthreads();
  constexpr int LPR = HD / 4;  // lanes of a row
  if (!*abort_w) {
    for (int n = rank + CL * (tid / LPR); n < m.rows; n += CL * (THREADS / LPR)) {
      const int d = tid % LPR * 4;
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)  // a share without tiles wrote no output: its factor is 0
        v[r] = r < CL && fac[r * N + n] != 0.f
                   ? *reinterpret_cast<const float4*>(cl.map_shared_rank(os, r) + n * LD + d)
                   : make_float4(0.f, 0.f, 0.f, 0.f);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < CL) {
          const float f = fac[r * N + n];
          o.x = fmaf(v[r].x, f, o.x);
          o.y = fmaf(v[r].y, f, o.y);
          o.z = fmaf(v[r].z, f, o.z);
          o.w = fmaf(v[r].w, f, o.w);
        }
      const int row = m.n0 + n, node = div_rep(row, rep, rep_inv);
      float* dst = a.out + (size_t)(m.t.row0 + node) * a.ldo + (size_t)(m.g * rep + row - node * rep) * HD + d;
      if (wide) {
        *reinterpret_cast<float4*>(dst) = o;
      } else {
        dst[0] = o.x;
        dst[1] = o.y;
        dst[2] = o.z;
        dst[3] = o.w;
      }
    }
  }
  cl.sync();  // the others may still read this CTA's shared memory
}

// The sequences longest first (all threads of the CTA; at most TM_SORT of them).
__device__ __forceinline__ void sort_lengths(const TreeArgs& a, int* len, uint16_t* order) {
  const int tid = threadIdx.x, mine = tid < a.n_seqs ? a.lengths[tid] : 0;
  if (tid < TM_SORT) len[tid] = mine;
  __syncthreads();
  int r = 0;
#pragma unroll 8
  for (int j = 0; j < a.n_seqs; ++j) {
    const int o = len[j];
    r += o > mine || (o == mine && j < tid);
  }
  if (tid < a.n_seqs) order[r] = (uint16_t)tid;
}

// ------------------------------------------------------------- host side

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  });
  return fn;
}

// What the host keeps of a kernel, for each device.
struct TmKernel {
  std::atomic<bool> ready{false};
  std::mutex filling;
  int clusters[9] = {};  // clusters of that many CTAs that run at once
};

// CTAs of a cluster (which splits the positions of one item), of those that run
// all at once.  A tile more to a CTA costs about a microsecond (8 nodes over 12
// tiles: 17.5 us whole, 9.5 in shares), the shares' join two (3 tiles: 8.5 whole,
// 8.6 in shares), and more CTAs start later (6 tiles of 24 items: 10.9 us with 144,
// 9.7 with 72): the cheapest by that, in 64ths of a tile.
inline int cluster_size(long items, int tiles, const TmKernel& k) {
  int best = 1;
  long least = 64l * tiles + items;
  for (int c = 2; c <= 8; ++c) {
    const long cost = 64l * ((tiles + c - 1) / c) + 128 + items * c;
    if (items <= k.clusters[c] && cost < least) {
      best = c;
      least = cost;
    }
  }
  return best;
}

// The pool as a matrix of head-dim rows, read one page's rows (at most a tile's)
// by 64 elements at a time.
inline bool pool_map(const TreeArgs& a, int layers, int box, CUtensorMap* map) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)a.kv.hd, (cuuint64_t)((long long)layers * a.kv.n_pages * 2 * a.kv.Hkv * a.kv.page_size)};
  const cuuint64_t strides[1] = {(cuuint64_t)a.kv.hd * 2};
  const cuuint32_t boxd[2] = {64, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.kv.pool, dims, strides, boxd, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch: a cluster for each item whose positions it splits, or a CTA on
// every SM that works through whole items.
template <class Kernel>
int launch_items(Kernel kernel, TmKernel& known, int threads, size_t smem, bool tma, int tile_rows, const TreeArgs& a, int layers,
                 int n_sm, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  if (!known.ready.load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> one(known.filling);
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return Q3TTS_ERR_CUDA;
    cfg.numAttrs = 1;
    for (int c = 2; c <= 8 && !known.ready.load(std::memory_order_relaxed); ++c) {
      cfg.gridDim = dim3(c);
      at[0].val.clusterDim.x = c;
      if (cudaOccupancyMaxActiveClusters(&known.clusters[c], kernel, &cfg) != cudaSuccess) return Q3TTS_ERR_CUDA;
    }
    known.ready.store(true, std::memory_order_release);
  }
  const int box = a.kv.page_size < TM_PT ? a.kv.page_size : TM_PT;
  CUtensorMap map = {};
  if (tma && !pool_map(a, layers, box, &map)) return Q3TTS_ERR_CUDA;
  const int row_tiles = (a.max_nodes * (a.Hq / a.kv.Hkv) + tile_rows - 1) / tile_rows;
  const long items = (long)a.n_seqs * a.kv.Hkv * row_tiles;
  const int tiles = (int)(((long)a.kv.pages_per_stream * a.kv.page_size + TM_PT - 1) / TM_PT);
  if (items > 0x7fffffffL / 2) return Q3TTS_ERR_UNSUPPORTED;
  const int c = cluster_size(items, tiles, known);
  const long grid = c > 1 ? items * c : (items < n_sm ? items : n_sm);
  const int vec = (((uintptr_t)a.q & 15) == 0 && a.ldq % 4 == 0 ? 1 : 0) |  // float4 loads of q, stores of out
                  (((uintptr_t)a.out & 15) == 0 && a.ldo % 4 == 0 ? 2 : 0);
  const unsigned rep = (unsigned)(a.Hq / a.kv.Hkv), rep_inv = (unsigned)(((1ull << 32) + rep - 1) / rep);
  cfg.gridDim = dim3((unsigned)grid);
  at[0].val.clusterDim.x = c;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, map, a, row_tiles, box, (int)items, vec, rep_inv) == cudaSuccess ? Q3TTS_OK
                                                                                                         : Q3TTS_ERR_CUDA;
}

}  // namespace
}  // namespace q3

// kv8_tiles.cuh -- what the tensor-core kernels of the 8-bit cache's attention share
// (kv8_attention.cu, kv8_wide.cu): items of work, the loading of code tiles, operand
// descriptors, the launch.
#pragma once

#include <limits.h>

#include "kv8.cuh"
#include "tree.cuh"

namespace q3 {

// Tiles of 128 rows (kv8_wide.cu); tma: whether pages come in boxes (load_tiles).
int launch_kv8_wide(const Kv8AttnArgs& a, int layers, int dtype, bool tma, int dev, cudaStream_t s);

namespace {

constexpr int KF_SORT = 256;  // sequences that are dealt by length, at most
// Exponents of the values' powers that count: -KV8_EXP .. KV8_EXP.  A weight with its value's power is 2^-80 of
// another's at the least for equal scores then, and fp32's exponents leave 2^-40 for what the scores differ by: weights
// below that have no part in the softmax's sum (with 60 it was 2^-7 between blocks 2^120 apart).
constexpr int KV8_EXP = 40;

struct KfDeal {
  int row_tiles, box;
  int vec;  // four elements of a row in one access: 1 of q, 2 of out
  unsigned rep_inv;
  int sorted;  // the sequences are taken longest first
  int wait_1024, lost_tile;
  // powers: blocks of a page, from a key block's to its value block's; 128 positions are step_pages
  // pages, step_blocks blocks and step_rem positions
  int per_page, to_values, step_pages, step_blocks, step_rem;
};

// tm_wait without a call, which a kernel that moves registers between its warps cannot
// make, and with a longer sleep between looks, whose instructions the working warps would wait for.
__device__ __forceinline__ bool kv8_wait(uint32_t bar, uint32_t parity, volatile int* abort_w, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(20000)  // ns, at most
        : "memory");
    if (ok) return true;
    if (*abort_w) return false;
    if ((clock64() - t0) >> 10 >= abort_w[1]) {
      *abort_w = 1;
      op_status(status, Q3TTS_ERR_TIMEOUT);
      return false;
    }
  }
}

struct KfItem {
  Kv8Seq t;
  int seq, g, n0, rows;  // kv head, first row of the tile, rows
  int end;               // positions that its rows may see
  int t0, nt;            // first position tile, tiles
};

// The CTA's row tile and kv head; returns its sequence, or that one's place by length. The
// last rows of a sequence, which see the most, come first.
__device__ __forceinline__ int first_item(const Kv8AttnArgs& a, const KfDeal& d, int cl, int rows, KfItem& m) {
  const int idx = (int)blockIdx.x / cl;
  m.g = idx % a.c.Hkv;
  m.n0 = (d.row_tiles - 1 - idx / a.c.Hkv % d.row_tiles) * rows;
  return idx / a.c.Hkv / d.row_tiles;
}
// The sequence that is the wanted-th longest (all threads; len: room for KF_SORT; ordered by
// the caller's next barrier).
template <int THREADS>
__device__ __forceinline__ void find_sequence(const Kv8Rows& rows, int wanted, int* len, int* seq) {
  for (int i = threadIdx.x; i < (rows.n_seqs + 3 & ~3); i += THREADS) len[i] = i < rows.n_seqs ? rows.lengths[i] : INT_MIN;
  __syncthreads();
  for (int i = threadIdx.x; i < rows.n_seqs; i += THREADS) {
    const int mine = len[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < rows.n_seqs; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(len + j);
      r += (o.x > mine || (o.x == mine && j < i)) + (o.y > mine || (o.y == mine && j + 1 < i)) +
           (o.z > mine || (o.z == mine && j + 2 < i)) + (o.w > mine || (o.w == mine && j + 3 < i));
    }
    if (r == wanted) *seq = i;
  }
}
// The item's rows and positions, of which the CTA has its share; false when it has no rows
// (or the sequence does not fit, which is reported).
__device__ __forceinline__ bool take_item(const Kv8AttnArgs& a, const KfDeal& d, int cl, int rank, int rows, KfItem& m) {
  const int rep = a.Hq / a.c.Hkv;
  m.rows = m.nt = m.t0 = m.end = 0;
  if (!kv8_seq(a.r, a.c.page, m.seq, true, m.t) || m.n0 >= m.t.n * rep) return false;
  m.rows = min(rows, m.t.n * rep - m.n0);
  m.end = m.t.L + (a.masks ? m.t.n : kv8_div(m.n0 + m.rows - 1, rep, d.rep_inv) + 1);
  const int all = (m.end + TM_PT - 1) / TM_PT, per = (all + cl - 1) / cl;
  m.t0 = min(all, rank * per);
  m.nt = min(all, m.t0 + per) - m.t0;
  return true;
}

// The powers of a lane's N positions, 32 apart, of each of an item's tiles, on their way a
// tile ahead, and their pages, which lead to them, two: neither is waited for.  Blocks and pages
// are stepped over without a division (KfDeal), which took longer than the rest of it; all N are looked
// up before the first is used.
template <int N>
struct Powers {
  int k[N], v[N];  // bytes of a position's key block and value block (127 past what is seen)
  // of the next tile's positions when a tile's are used: page; of the one after that: their entry of
  // the table's row, block of the page, place in the block
  int page[N], entry[N], block[N], rem[N];
  const uint8_t* layer;  // the kv head's key powers on page 0

  __device__ __forceinline__ Powers(const Kv8AttnArgs& a, const KfDeal& d, const KfItem& m, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int pos = m.t0 * TM_PT + lane + 32 * j;
      entry[j] = kv8_div(pos, a.c.page, a.c.page_inv);
      const int slot = pos - entry[j] * a.c.page;
      block[j] = kv8_div(slot, a.c.block, a.c.block_inv);
      rem[j] = slot - block[j] * a.c.block;
    }
    layer = a.c.powers + ((long long)a.c.layer * a.c.n_pages * 2 * a.c.Hkv + m.g) * d.per_page;
    look(a, m, 0, lane);
    next(a, d, m, -1, lane);
  }
  // after tile i's have been used
  __device__ __forceinline__ void next(const Kv8AttnArgs& a, const KfDeal& d, const KfItem& m, int i, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int pg = (unsigned)page[j] < (unsigned)a.c.n_pages ? page[j] : 0;  // (reported by the loading warps)
      const uint8_t* p = layer + (long long)pg * (2 * d.to_values) + block[j];
      const bool is = there(m, i + 1, lane + 32 * j);
      k[j] = is ? *p : 127;
      v[j] = is ? p[d.to_values] : 127;
      // 128 positions on
      rem[j] += d.step_rem;
      block[j] += d.step_blocks;
      if (rem[j] >= a.c.block) {
        rem[j] -= a.c.block;
        ++block[j];
      }
      entry[j] += d.step_pages;
      if (block[j] >= d.per_page) {
        block[j] -= d.per_page;
        ++entry[j];
      }
    }
    look(a, m, i + 2, lane);
  }

 private:
  __device__ __forceinline__ bool there(const KfItem& m, int i, int at) const { return i < m.nt && (m.t0 + i) * TM_PT + at < m.end; }
  __device__ __forceinline__ void look(const Kv8AttnArgs& a, const KfItem& m, int i, int lane) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      page[j] = there(m, i, lane + 32 * j) ? a.r.page_table[(size_t)m.seq * a.r.pps + entry[j]] : 0;
  }
};
// Swizzled operand tiles with rows of W bytes (128 or 64) in atoms of eight rows.
template <int W>
__device__ __forceinline__ uint64_t sw_desc(uint32_t saddr, uint32_t lead = 16) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)((lead & 0x3FFFFu) >> 4) << 16) | ((uint64_t)(8 * W >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)(W == 128 ? 2 : 4) << 61);
}
// Byte offset of 16-byte chunk c of row r in such a tile.
template <int W>
__device__ __forceinline__ uint32_t sw_at(int r, int c) {
  const uint32_t o = (uint32_t)(r * W + c * 16);
  return W == 128 ? o ^ ((o >> 3) & 0x70u) : o ^ ((o >> 3) & 0x30u);
}

// Four consecutive elements of a row of q.
__device__ __forceinline__ float4 q4(const float* p, bool wide) {
  return wide ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ float4 q4(const bf16* p, bool wide) {
  if (!wide) return make_float4(to_f(p[0]), to_f(p[1]), to_f(p[2]), to_f(p[3]));
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}

// Four consecutive elements of a row of out.
__device__ __forceinline__ void store4(float* p, float4 v, bool wide) {
  if (wide) {
    *reinterpret_cast<float4*>(p) = v;
  } else {
    p[0] = v.x;
    p[1] = v.y;
    p[2] = v.z;
    p[3] = v.w;
  }
}
__device__ __forceinline__ void store4(bf16* p, float4 v, bool wide) {
  if (wide) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(make_float2(v.x, v.y)), pack_bf16(make_float2(v.z, v.w)));
  } else {
    p[0] = from_f<bf16>(v.x);
    p[1] = from_f<bf16>(v.y);
    p[2] = from_f<bf16>(v.z);
    p[3] = from_f<bf16>(v.w);
  }
}

// A warp's loads of the key and value tiles of an item, as codes, into a ring of S tiles
// (K0 V0 K1 V1 ..).  TMA: pages of 8 positions or more that fill a tile a whole number of
// times (or whole tiles of larger pages) come in boxes, swizzled on the way; other pages row by row in
// 16-byte asynchronous copies, by all lanes.  SPLIT: two warps, the keys (kv 0) and the
// values (1).  issued: tiles under way or there, up to the warp's last.
template <int HD, int S, bool TMA, bool SPLIT>
__device__ __forceinline__ bool load_tiles(const CUtensorMap* map, const Kv8AttnArgs& a, const KfItem& m, int box, uint32_t ring,
                                           unsigned long long* full, unsigned long long* empty, int kv, int& issued,
                                           volatile int* abort_w) {
  // tiles of the copying warp that stay on their way: fewer than its places of the ring
  constexpr int AHEAD = SPLIT ? 1 : 2;
  static_assert(SPLIT ? S >= 4 && S % 2 == 0 : S >= 3, "places");
  const int first = SPLIT ? kv : 0, last = SPLIT ? kv : 1;
  const int lane = threadIdx.x & 31, ps = a.c.page;
  const int* table = a.r.page_table + (size_t)m.seq * a.r.pps;
  int* status = a.r.status;
  bool ok = true;
  // a page that is not the pool's is reported and read as page 0
  auto checked = [&](int page) -> int {
    if (page >= 0 && page < a.c.n_pages) return page;
    op_status(status, Q3TTS_ERR_ARG);
    return 0;
  };
  if constexpr (TMA) {
    // lane (keys or values, b): box b of a tile
    const int my = SPLIT ? kv : lane >> 4, b = lane & 15, boxes = TM_PT / box;
    auto page_of = [&](int i) -> int {
      const int pos = (m.t0 + i) * TM_PT + b * box;
      return b < boxes && i < m.nt && pos < m.end ? table[kv8_div(pos, ps, a.c.page_inv)] : 0;
    };
    int page0 = page_of(0), page1 = page_of(1);  // looked up two tiles ahead
    for (int i = 0; i < m.nt; ++i) {
      const int pos = (m.t0 + i) * TM_PT + b * box;
      const int held = min(TM_PT, m.end - (m.t0 + i) * TM_PT);
      const bool mine = b < boxes && pos < m.end && !(SPLIT && lane > 15);
      const int row = mine ? (int)kv8_row(a.c, checked(page0), my, m.g, pos - kv8_div(pos, ps, a.c.page_inv) * ps) : 0;
      for (int h = first; h <= last; ++h) {
        const int it = 2 * i + h, slot = it % S;
        ok = ok && kv8_wait(su32(&empty[slot]), ((uint32_t)(it / S) & 1u) ^ 1u, abort_w, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t fb = su32(&full[slot]);
        if (lane == 0) mbar_expect_tx(fb, (uint32_t)((held + box - 1) / box * box * HD));
        __syncwarp();
        if (mine && my == h) tma_load(ring + slot * (TM_PT * HD) + b * box * HD, map, 0, row, fb);
        issued = it + 1;
      }
      if (!ok) break;
      page0 = page1;
      page1 = page_of(i + 2);
    }
  } else {
    // 16-byte copies, row by row: lane l has chunk l % CH of rows l / CH, ..
    constexpr int CH = HD / 16, RPI = 32 / CH;
    const int c = lane % CH;
    const long long plane = (long long)a.c.Hkv * ps;
    int row[TM_PT / 32], page[TM_PT / 32];  // pool rows of positions lane + 32 j of the tile; the next tile's pages
    auto look_up = [&](int i) {
#pragma unroll
      for (int j = 0; j < TM_PT / 32; ++j) {
        const int pos = (m.t0 + i) * TM_PT + lane + 32 * j;
        page[j] = i < m.nt && pos < m.end ? table[kv8_div(pos, ps, a.c.page_inv)] : 0;
      }
    };
    look_up(0);
    int sent = 0, arrived = 0;  // of the warp's tiles
    auto arrive = [&](int n) { mbar_arrive(su32(&full[(SPLIT ? 2 * n + kv : n) % S])); };
    for (int i = 0; i < m.nt && ok; ++i) {
#pragma unroll
      for (int j = 0; j < TM_PT / 32; ++j) {
        const int pos = (m.t0 + i) * TM_PT + lane + 32 * j;
        row[j] = pos < m.end ? (int)kv8_row(a.c, checked(page[j]), 0, m.g, pos - kv8_div(pos, ps, a.c.page_inv) * ps) : -1;
      }
      look_up(i + 1);
      for (int h = first; h <= last; ++h) {
        const int it = 2 * i + h, slot = it % S;
        ok = kv8_wait(su32(&empty[slot]), ((uint32_t)(it / S) & 1u) ^ 1u, abort_w, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = ring + slot * (TM_PT * HD);
        const uint8_t* src = a.c.codes + (h ? plane * HD : 0) + c * 16;
#pragma unroll
        for (int j = 0; j < TM_PT / 32; ++j)
#pragma unroll 8
          for (int e = lane / CH; e < 32; e += RPI) {
            const int from = __shfl_sync(0xffffffffu, row[j], e);
            if (from >= 0)
              asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + sw_at<HD>(32 * j + e, c)),
                           "l"(src + (size_t)from * HD)
                           : "memory");
          }
        asm volatile("cp.async.commit_group;" ::: "memory");
        issued = it + 1;
        if (++sent - arrived > AHEAD) {
          asm volatile("cp.async.wait_group %0;" ::"n"(AHEAD) : "memory");
          proxy_fence();
          arrive(arrived++);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    proxy_fence();
    for (; arrived < sent; ++arrived) arrive(arrived);
  }
  return ok;
}

// The codes as a matrix of head-dim rows, read one page's rows (at most a tile's) at a time.
bool codes_map(const Kv8Cache& c, int layers, int box, CUtensorMap* map) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)c.hd, (cuuint64_t)((long long)layers * c.n_pages * 2 * c.Hkv * c.page)};
  const cuuint64_t strides[1] = {(cuuint64_t)c.hd};
  const cuuint32_t boxd[2] = {(cuuint32_t)c.hd, (cuuint32_t)box};
  const cuuint32_t estr[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, c.codes, dims, strides, boxd, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             c.hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One launch: a CTA, or a cluster that splits the positions, for each item.
template <class Kernel>
int launch_tiles(Kernel kernel, TmKernel& known, int threads, size_t smem, bool tma, int rows, size_t vec_bytes,
                 const Kv8AttnArgs& a, int layers, cudaStream_t s) {
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
    for (int c = 1; c <= 8 && !known.ready.load(std::memory_order_relaxed); ++c) {
      cfg.gridDim = dim3(c);
      at[0].val.clusterDim.x = c;
      if (cudaOccupancyMaxActiveClusters(&known.clusters[c], kernel, &cfg) != cudaSuccess) return Q3TTS_ERR_CUDA;
    }
    known.ready.store(true, std::memory_order_release);
  }
  KfDeal d;
  d.box = a.c.page < TM_PT ? a.c.page : TM_PT;
  CUtensorMap map = {};
  if (tma && !codes_map(a.c, layers, d.box, &map)) return Q3TTS_ERR_CUDA;
  const int rep = a.Hq / a.c.Hkv;
  d.row_tiles = (int)(((long)a.r.max_rows * rep + rows - 1) / rows);
  const long items = (long)a.r.n_seqs * a.c.Hkv * d.row_tiles;
  if (items > 0x7fffffffL / 8) return Q3TTS_ERR_UNSUPPORTED;
  const int tiles = (int)(((long)a.r.pps * a.c.page + TM_PT - 1) / TM_PT);
  const int c = cluster_size(items, tiles, known);
  d.vec = (((uintptr_t)a.q & (vec_bytes - 1)) == 0 && a.ldq % 4 == 0 ? 1 : 0) |
          (((uintptr_t)a.out & (vec_bytes - 1)) == 0 && a.ldo % 4 == 0 ? 2 : 0);
  d.rep_inv = kv8_inverse(rep);
  d.sorted = items * c > known.clusters[1] && a.r.n_seqs > 1 && a.r.n_seqs <= KF_SORT;
  d.per_page = a.c.page / a.c.block;
  d.to_values = a.c.Hkv * d.per_page;
  d.step_pages = TM_PT / a.c.block / d.per_page;
  d.step_blocks = TM_PT / a.c.block % d.per_page;
  d.step_rem = TM_PT % a.c.block;
  d.wait_1024 = a.wait_1024;
  d.lost_tile = a.lost_tile;
  cfg.gridDim = dim3((unsigned)(items * c));
  at[0].val.clusterDim.x = c;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, map, a, d) == cudaSuccess ? Q3TTS_OK : Q3TTS_ERR_CUDA;
}

}  // namespace
}  // namespace q3

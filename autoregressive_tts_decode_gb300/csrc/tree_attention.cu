// tree_attention.cu -- attention of drafted tree nodes over a paged cache, on the
// 5th-generation tensor cores.
//
// A sequence holds L committed positions and T drafted nodes, whose keys and
// values sit in its pages at positions L .. L + T - 1 in node order.  Node i
// sees every committed position and the nodes j of its mask (bit j of a 64-bit
// word: its ancestors and itself), so for head h of kv head g
//   s_p = q . k_p / sqrt(hd),  o = sum_p e^(s_p - m) v_p / sum_p e^(s_p - m)
// over the positions p it sees, m about their largest score; o = 0 when it sees
// none.  One node whose mask is its own bit is the ordinary decode of a single
// token, a chain of nodes the causal attention of a short chunk.
//
// The few query rows that share a kv head (nodes x q heads of the group) are
// the MMA's N side, 128 cached positions its M side, so that one row costs no
// more lanes than sixteen:
//   S^T = K Q^T   M 128 positions, K the head dimension; K arrives by TMA, page
//                 by page, as it lies in the cache;
//   P^T = 2^(c S^T - base)  c = log2(e) / sqrt(hd), in registers, a running
//                 base per row;
//   O^T = V^T P^T M the head dimension, K 128 positions; V is read as it lies in
//                 the cache (an M-major operand).
// The base of a row follows its largest score only when a score passes it by
// more than 2^8: until then weights up to 256 are exact multiples that the
// final division removes, and a tile needs one vote of the softmax threads
// instead of a maximum over them.
//
// Precision.  Keys and values are bf16 as cached; Q and P enter as three bf16
// terms each, which hold all 24 bits of an fp32 value (two terms of P alone
// leave 2e-6 of the output).  The terms are stacked along N, so that a tile of
// K or V is read from shared memory once for all of them; each has its own
// accumulator columns (of 64 rows, the two small ones share) and they are added
// in fp32 registers, like the outputs of successive tiles: the tensor cores
// truncate as they accumulate, and summed in tensor memory over 32768 positions
// the error was 3.7e-5 of the output.
//
// Roles of a CTA (one per SM): two to eight warps bring the keys and values into a
// ring of tiles, one thread issues the MMAs (scores of tile t + 1 before the
// outputs of tile t), one warp brings in the queries of the items after the
// first, and four warps are the softmax (eight, each four with half of the rows,
// for tiles of 32 and 64 rows: 118 -> 113 us for 128 sequences with 32).  A CTA
// works through several items (sequence, kv head, tile of rows) and the roles run
// ahead into the next one, so only the first pays the latency of its start.  Items
// are dealt longest first, in rounds of alternating direction: on 128 sequences of
// 256..2048 positions the SMs then end together.  Few items are split over the
// positions in clusters, whose CTAs join their shares through each other's shared
// memory.
//
// How the cache is read follows its type and page size.  bf16 pages that TMA boxes
// fit come in whole boxes; other page sizes row by row, in 16-byte asynchronous
// copies (128 sequences of 1000 positions, 8 nodes: 88 us in boxes, 96 in rows);
// fp32 rows are loaded, split into three bf16 terms on the way by eight warps and
// multiplied term by term (100 sequences of 1000 positions, 8 nodes: 207 us, 4.1
// TB/s; four warps with twice the loads each: 291).  Tiles have the smallest of 16, 32 and 64 rows that hold a sequence's
// (there, 16 rows in tiles of 16, 32 or 64: 88, 97, 126 us; 32 rows in tiles of 32
// or 64: 99, 130).
//
// The bound is the cache's bytes, read once for up to 64 rows: 128 sequences of
// 256..2048 positions, 16 nodes with two heads each: 113 us, 5.7 TB/s.  Short
// calls are bound by latency (the launch, the chain from lengths to page ids to
// first rows, a tile's way through the tensor cores): 131 positions, 8 nodes: 7.6 us.
// Every wait is bounded; on expiry the CTA records Q3TTS_ERR_TIMEOUT, waits
// (bounded) for its copies and MMAs in flight, frees its tensor memory and
// writes nothing more.
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace q3 {

namespace {

constexpr int TM_QTHREADS = 32;
constexpr int TM_MASKS = 4;      // items whose masks are held: the softmax's, and the scores may be three ahead

// How a tile of K or V gets from the cache into shared memory.
enum TmLoad {
  kTma,    // bf16, pages of 8, 16, 32, 64 or a multiple of 128 positions: a TMA box per page
  kCopy,   // bf16, any page size: 16-byte asynchronous copies, row by row
  kSplit,  // fp32, any page size: loaded, split into three bf16 terms, stored as three tiles
};

template <int HD, int N, int MODE>
struct TmCfg {
  // softmax groups of four warps, each with its share of the rows; then a warp
  // for the MMAs, one for the queries, and 2 LW for the keys and values (rows
  // copied by 8 instead of 4 warps: 96 us, 103; beside 64 rows' softmax, for want
  // of registers, 4: 161 us, 8: 214, 2: 181)
  static constexpr int SW = N <= 16 ? 1 : 2, NC = N / SW;
  static constexpr int LW = MODE == kSplit || (MODE == kCopy && N <= 32) ? 4 : MODE == kTma ? 1 : 2;
  static constexpr int MMA_WARP = 4 * SW, QUERY_WARP = MMA_WARP + 1, LOAD_WARP = MMA_WARP + 2;
  static constexpr int THREADS = 128 * SW + 64 + 64 * LW;
  static constexpr int TERMS = MODE == kSplit ? 3 : 1;   // ring tiles of a K or V tile
  static constexpr uint32_t FULL = MODE == kTma ? 1 : 64 * LW;  // arrivals that fill a ring tile
  static constexpr int BLK = HD / 64;               // 128-byte swizzle blocks of a row
  static constexpr uint32_t SLOT = TM_PT * HD * 2;  // a K or V tile
  static constexpr uint32_t TERM = N * 128;         // one term of one 64-element block (of Q or P)
  static constexpr uint32_t QBYTES = BLK * 3 * TERM, PBYTES = 2 * 3 * TERM;
  static constexpr int G = N <= 32 ? 3 : 2;         // accumulator groups: the terms, or the large one and the others
  static constexpr uint32_t Q = 0, P = QBYTES, RING = P + PBYTES;  // (a second P would cost a place of the ring: 125 against 122 us, 16 nodes)
  static constexpr uint32_t CTL_BYTES = 6144;
  static constexpr int FIT = (int)((227u * 1024 - 1024 - CTL_BYTES - RING) / SLOT);
  static constexpr int S = FIT < 8 ? FIT : 8;       // tiles in the ring
  static constexpr uint32_t CTL = RING + S * SLOT;
  static constexpr size_t SMEM = 1024 + CTL + CTL_BYTES;
  static constexpr uint32_t TM_S = G * N, TM_O = 2 * TM_S;  // columns: S twice, O twice
  static constexpr uint32_t TMEM_COLS = 4 * G * N <= 256 ? 256 : 512;
  // three places: a TMA warp skips two ring tiles at most, which its parity waits
  // bear; the softmax of tile t waits for V_t, which takes the place of K_t (or,
  // split, of K_(t + 1)'s terms) at the latest; a split tile is stored whole
  static_assert(S >= 3 && (MODE != kSplit || G == 3) && 4 * G * N <= 512 && N * HD * 4 <= (int)PBYTES, "ring, tensor memory, output rows");
};

// Control block (shared memory).
template <int N, int S>
struct TmCtl {
  unsigned long long full[S], empty[S], s_full[2], s_free[2], p_full, p_free, q_first, q_full[TM_MASKS], q_free, done, v_full[2];
  uint32_t tmem;
  int abort_w[2];  // given up, limit of the waits
  float base[N], corr[N], sum[N];  // a row's base, the factor of its last rise, its sum of weights
  float part[4][N];
  unsigned bad[4];
  unsigned long long mask[TM_MASKS][N];
  int len[TM_SORT];
  uint16_t order[TM_SORT];  // sequences, longest first
  int copies[2][8];  // TMA: the last ring tiles that each loading warp has filled
};

// N fp32 columns of 16 lanes, eight columns at a time in the fragment order of
// an 8 x 8 matrix store: registers 4 b and 4 b + 1 hold columns 8 b + 2 (lane % 4)
// and the next of lane / 4, registers 4 b + 2 and 4 b + 3 the same of
// lane / 4 + 8.
template <int N>
__device__ __forceinline__ void tmem_frag(uint32_t taddr, uint32_t (&r)[N / 2]);
template <>
__device__ __forceinline__ void tmem_frag<16>(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
template <>
__device__ __forceinline__ void tmem_frag<32>(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
// Four 8 x 8 matrices of 16-bit elements, transposed on the way: matrix m goes
// to the rows at lanes 8 m .. 8 m + 7's addresses.
__device__ __forceinline__ void store_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// Barrier and vote of the 128 threads of softmax group wg.
__device__ __forceinline__ void soft_sync(int wg) {
  asm volatile("barrier.cta.sync %0, 128;" ::"r"(1 + 2 * wg) : "memory");
}
__device__ __forceinline__ bool soft_any(bool p, int wg) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(2 + 2 * wg)
      : "memory");
  return r != 0;
}
// Barrier and vote of all softmax threads; giving up is decided here alone, so
// that both groups leave together.
template <int COUNT>
__device__ __forceinline__ bool all_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 5, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(COUNT)
      : "memory");
  return r != 0;
}

// Max or sum over the lanes that hold the same columns (lane % 4).
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int HD, int N, int MODE>
__global__ void __launch_bounds__(TmCfg<HD, N, MODE>::THREADS, 1)
    tree_mma_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeArgs a, int row_tiles, int box, int items, int vec,
                    unsigned rep_inv) {
  using C = TmCfg<HD, N, MODE>;
  using Ctl = TmCtl<N, C::S>;
  static_assert(sizeof(Ctl) <= C::CTL_BYTES, "control block");
  extern __shared__ uint8_t tm_raw[];
  const uint32_t raw = su32(tm_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* sp = tm_raw + (sbase - raw);
  Ctl& ctl = *reinterpret_cast<Ctl*>(sp + C::CTL);
  volatile int* abort_w = ctl.abort_w;

  cg::cluster_group cl = cg::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rep = a.Hq / a.kv.Hkv;

  TmDeal deal{items, row_tiles, N, (int)gridDim.x / CL, (int)blockIdx.x / CL, rank, CL, nullptr};
  prefetch_first(a, deal);
  if (tid == 0) {
    for (int i = 0; i < C::S; ++i) {
      mbar_init(su32(&ctl.full[i]), C::FULL);
      mbar_init(su32(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(su32(&ctl.s_full[i]), 1);
      mbar_init(su32(&ctl.s_free[i]), 128 * C::SW);
    }
    mbar_init(su32(&ctl.p_full), 128 * C::SW);
    mbar_init(su32(&ctl.p_free), 1);
    for (int i = 0; i < TM_MASKS; ++i) mbar_init(su32(&ctl.q_full[i]), TM_QTHREADS);
    mbar_init(su32(&ctl.q_first), 128 * C::SW);
    mbar_init(su32(&ctl.q_free), 1);
    mbar_init(su32(&ctl.done), 1);
    for (int i = 0; i < 2; ++i) mbar_init(su32(&ctl.v_full[i]), 64 * C::LW);
    ctl.abort_w[0] = 0;
    ctl.abort_w[1] = a.wait_1024;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid >= 32 && tid < 48) ctl.copies[(tid >> 3) & 1][tid & 7] = -1;
  pdl_wait();  // q and the appended keys and values come from the previous kernels
  // (tensor memory after the wait: a kernel before may still be about to take its own)
  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&ctl.tmem)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const bool sorted = items > (int)gridDim.x / CL && a.n_seqs <= TM_SORT;
  if (sorted) {
    deal.order = ctl.order;
    sort_lengths(a, ctl.len, ctl.order);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  const uint32_t ring = sbase + C::RING;

  // the queries and masks of the CTA's qi-th item
  auto q_wait = [&](int qi) -> bool {
    return qi == 0 ? tm_wait(su32(&ctl.q_first), 0u, abort_w, a.status)
                   : tm_wait(su32(&ctl.q_full[qi % TM_MASKS]), (uint32_t)((qi - 1) / TM_MASKS) & 1u, abort_w, a.status);
  };
  TmItem m;
  int have = 0;
  bool ok = true;

  if (warp >= C::LOAD_WARP) {
    // ---- loads
    if constexpr (MODE == kTma) {
      const int w = warp - C::LOAD_WARP;  // a warp for the keys and one for the values
      ok = tma_loads<HD, C::S>(&map, a, deal, box, w > 0, ring, ctl.full, ctl.empty, ctl.copies[w], abort_w);
    } else {
      const int ps = a.kv.page_size;
      const long long plane = (long long)a.kv.Hkv * ps;  // rows of a page's keys (or values)
      int ic = 0;                                        // position tiles so far
      for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
        if (have == 0 || m.nt == 0) continue;
        const int* table = a.kv.page_table + (size_t)m.seq * a.kv.pages_per_stream;
        // all loading warps share every tile, in the ring's order (so that a place
        // is waited for at every phase of its barrier); warp lw has rows lw RW ..
        // of it, lane l the pool rows of the l-th of them (and the 32nd after it)
        constexpr int LWN = 2 * C::LW, RW = TM_PT / LWN, H = RW < 32 ? 1 : RW / 32;
        const int lw = warp - C::LOAD_WARP;
        const uint8_t* pool = static_cast<const uint8_t*>(a.kv.pool);
        int pages[H], pages2[H], row_even[H], row_odd[H];  // pages of the next two tiles, key rows of the last two
        auto look_up = [&](int i, int (&pg)[H]) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const int pos = (m.t0 + i) * TM_PT + lw * RW + lane + 32 * h;
            pg[h] = i < m.nt && pos < m.t.P ? __ldg(table + pos / ps) : 0;
          }
        };
        auto find_rows = [&](int i, int (&rows)[H]) {
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const int pos = (m.t0 + i) * TM_PT + lw * RW + lane + 32 * h;
            rows[h] = i < m.nt && pos < m.t.P ? pool_row(a, m.g, false, pages[h], pos) : -1;
            pages[h] = pages2[h];
            // the next tile on its way to the L2: the loads that follow keep too few
            // bytes in flight for the memory's latency
            if (MODE == kSplit && lane < RW && i + 1 < m.nt && pos + TM_PT < m.t.P) {
              const uint8_t* p = pool + (size_t)pool_row(a, m.g, false, pages[h], pos + TM_PT) * (HD * 4);
#pragma unroll
              for (int line = 0; line < HD * 4; line += 128) {
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + line));
                asm volatile("prefetch.global.L2 [%0];" ::"l"(p + plane * (HD * 4) + line));
              }
            }
          }
          look_up(i + 2, pages2);
        };
        // what the i-th ring tile of the item holds
        auto is_value = [&](int i) -> bool { return i == 2 * m.nt - 1 || (i >= 2 && (i & 1) == 0); };
        auto tile_of = [&](int i) -> int {
          return is_value(i) ? (i == 2 * m.nt - 1 ? m.nt - 1 : i / 2 - 1) : (i + 1) / 2;
        };
        look_up(0, pages);
        look_up(1, pages2);
        if constexpr (MODE == kCopy) {
          constexpr int CH = HD / 8;  // 16-byte pieces of a row
          const int c = lane % CH;
          int pending = -1;           // the ring tile whose copies are on their way
          for (int i = 0; i < 2 * m.nt; ++i) {
            const int it = 2 * ic + i, tile = tile_of(i);
            const bool v = is_value(i);
            if (!v) {
              if (tile & 1) find_rows(tile, row_odd); else find_rows(tile, row_even);
            }
            ok = __all_sync(0xffffffffu, tm_wait(su32(&ctl.empty[it % C::S]), ((uint32_t)(it / C::S) & 1u) ^ 1u, abort_w, a.status));
            if (!ok) break;
            const uint8_t* src = pool + c * 16 + (v ? plane * (HD * 2) : 0);
            const uint32_t dst = ring + it % C::S * C::SLOT + (c >> 3) * (TM_PT * 128);
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const int mine = (tile & 1) ? row_odd[h] : row_even[h];
#pragma unroll 8
              for (int q = lane / CH; q < (RW < 32 ? RW : 32); q += 32 / CH) {
                const int r = lw * RW + 32 * h + q, row = __shfl_sync(0xffffffffu, mine, q);
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 dst + r * 128 + (((c & 7) ^ (r & 7)) << 4)),
                             "l"(src + (size_t)max(row, 0) * (HD * 2)), "r"(row >= 0 ? 16 : 0)
                             : "memory");
              }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
            if (pending >= 0) {  // the tile before has arrived
              asm volatile("cp.async.wait_group 1;" ::: "memory");
              proxy_fence();
              mbar_arrive(su32(&ctl.full[pending % C::S]));
            }
            pending = it;
          }
          asm volatile("cp.async.wait_group 0;" ::: "memory");
          if (pending >= 0) {
            proxy_fence();
            mbar_arrive(su32(&ctl.full[pending % C::S]));
          }
        } else {
          // four elements of a row per lane, eight loads on their way while the eight
          // before them are split and stored
          constexpr int CH = HD / 4, U = 8, RPI = 32 / CH == 0 ? 1 : 32 / CH, BATCHES = RW / (U * RPI);
          static_assert(BATCHES >= 1 && CH <= 32, "a warp's rows in whole batches");
          const int c = lane % CH;
          auto load = [&](int i, int batch, float4 (&x)[U]) {
            i = min(i, 2 * m.nt - 1);  // (past the item: its last tile again, not used)
            const int tile = tile_of(i);
            const bool v = is_value(i);
            if (!v && batch == 0) {
              if (tile & 1) find_rows(tile, row_odd); else find_rows(tile, row_even);
            }
            const int mine = (tile & 1) ? row_odd[0] : row_even[0];
            const uint8_t* src = pool + c * 16 + (v ? plane * (HD * 4) : 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              // a row past the sequence is read from the pool's first and zeroed when stored: a
              // load under a branch would be waited for at the branch's end
              const int row = __shfl_sync(0xffffffffu, mine, (batch * U + u) * RPI + lane / CH);
              x[u] = __ldg(reinterpret_cast<const float4*>(src + (size_t)max(row, 0) * (HD * 4)));
            }
          };
          float4 x[U], y[U];
          load(0, 0, x);
          for (int i = 0; i < 2 * m.nt; ++i) {
            const int it = (2 * ic + i) * 3;
            // the last of the three places is free last
            const uint32_t eb = su32(&ctl.empty[(it + 2) % C::S]), ep = ((uint32_t)((it + 2) / C::S) & 1u) ^ 1u;
            for (int term = 0; term < 2; ++term)
              ok = tm_wait(su32(&ctl.empty[(it + term) % C::S]), ((uint32_t)((it + term) / C::S) & 1u) ^ 1u, abort_w, a.status) && ok;
            ok = __all_sync(0xffffffffu, tm_wait(eb, ep, abort_w, a.status) && ok);
            if (!ok) break;
#pragma unroll
            for (int batch = 0; batch < BATCHES; ++batch) {
              if (batch + 1 < BATCHES) load(i, batch + 1, y); else load(i + 1, 0, y);
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const int r = lw * RW + (batch * U + u) * RPI + lane / CH;
                const uint32_t off = (c >> 4) * (TM_PT * 128) + r * 128 + ((((c >> 1) & 7) ^ (r & 7)) << 4) + (c & 1) * 8;
                float2 v = make_float2(x[u].x, x[u].y), z = make_float2(x[u].z, x[u].w);
                if ((m.t0 + tile_of(i)) * TM_PT + r >= m.t.P) v = z = make_float2(0.f, 0.f);
#pragma unroll
                for (int term = 0; term < 3; ++term) {
                  const uint32_t p = pack_bf16(v), q = pack_bf16(z);
                  *reinterpret_cast<uint2*>(sp + C::RING + (it + term) % C::S * C::SLOT + off) = make_uint2(p, q);
                  v = add2(v, make_float2(-__uint_as_float(p << 16), -__uint_as_float(p & 0xffff0000u)));
                  z = add2(z, make_float2(-__uint_as_float(q << 16), -__uint_as_float(q & 0xffff0000u)));
                }
              }
#pragma unroll
              for (int u = 0; u < U; ++u) x[u] = y[u];
            }
            proxy_fence();
#pragma unroll
            for (int term = 0; term < 3; ++term) mbar_arrive(su32(&ctl.full[(it + term) % C::S]));
            if (is_value(i)) mbar_arrive(su32(&ctl.v_full[(ic + tile_of(i)) & 1]));
          }
        }
        ic += m.nt;
      }
    }
  } else if (warp == C::MMA_WARP) {
    // ---- MMA issue
    if (elect_one()) {
      constexpr uint32_t idS = f16_idesc(TM_PT, (C::G == 3 ? 3 : 2) * N, false), idS1 = f16_idesc(TM_PT, N, false);
      constexpr uint32_t idO = f16_idesc(TM_PT, (C::G == 3 ? 3 : 2) * N, true), idO1 = f16_idesc(TM_PT, N, true);
      // a head dimension of 64 fills half of M: the other half's rows are read
      // from the next atom and their results are not used
      constexpr uint32_t v_lead = HD == 128 ? TM_PT * 128 : 1024;
      const int lost = blockIdx.x == 0 ? a.lost_tile : -1;
      int ic = 0, tc = 0, qi = 0;  // ring tiles, position tiles and items so far
      for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
        if (have == 0 || m.nt == 0) continue;
        ok = q_wait(qi);
        tc_fence_after();
        for (int i = 0; i <= m.nt && ok; ++i) {
          if (i < m.nt) {  // scores of tile i
            const int it = (ic + k_item(i)) * C::TERMS, t = tc + i;
            ok = t != lost && tm_wait(su32(&ctl.s_free[t & 1]), ((uint32_t)(t >> 1) & 1u) ^ 1u, abort_w, a.status);
            const uint32_t d = tmem + (t & 1) * C::TM_S;
#pragma unroll
            for (int term = 0; term < C::TERMS; ++term) {
              // term j of K meets the first 3 - j of Q, in the accumulators of the products' size
              const int slot = (it + term) % C::S;
              ok = ok && tm_wait(su32(&ctl.full[slot]), (uint32_t)((it + term) / C::S) & 1u, abort_w, a.status);
              if (!ok) break;
              tc_fence_after();
              const uint32_t kb = ring + slot * C::SLOT;
#pragma unroll
              for (int blk = 0; blk < C::BLK; ++blk) {
                const uint64_t dk = sw128_desc(kb + blk * (TM_PT * 128));
                const uint64_t dq = sw128_desc(sbase + C::Q + blk * 3 * C::TERM);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                  mma_bf16(d + term * N, dk + s * 2, dq + s * 2, idS - (uint32_t)((term * N) >> 3 << 17),
                           (term | blk | s) != 0 ? 1u : 0u);
                  if constexpr (C::G == 2) mma_bf16(d + N, dk + s * 2, dq + ((2 * C::TERM) >> 4) + s * 2, idS1, 1u);
                }
              }
              mma_commit(su32(&ctl.empty[slot]));
            }
            if (!ok) break;
            mma_commit(su32(&ctl.s_full[t & 1]));
            if (i == m.nt - 1) mma_commit(su32(&ctl.q_free));
          }
          if (i > 0) {  // outputs of tile i - 1
            const int it = (ic + v_item(i - 1, m.nt)) * C::TERMS, t = tc + i - 1;
            ok = tm_wait(su32(&ctl.p_full), (uint32_t)t & 1u, abort_w, a.status);
            const uint32_t pbuf = sbase + C::P, d = tmem + C::TM_O + (t & 1) * C::TM_S;
#pragma unroll
            for (int term = 0; term < C::TERMS; ++term) {
              const int slot = (it + term) % C::S;
              ok = ok && tm_wait(su32(&ctl.full[slot]), (uint32_t)((it + term) / C::S) & 1u, abort_w, a.status);
              if (!ok) break;
              tc_fence_after();
              const uint32_t vb = ring + slot * C::SLOT;
#pragma unroll
              for (int s = 0; s < 8; ++s) {
                const uint64_t dv = sw128_desc(vb + s * 2048, v_lead);
                const uint64_t dp = sw128_desc(pbuf + (s >> 2) * 3 * C::TERM) + (s & 3) * 2;
                mma_bf16(d + term * N, dv, dp, idO - (uint32_t)((term * N) >> 3 << 17), (term | s) != 0 ? 1u : 0u);
                if constexpr (C::G == 2) mma_bf16(d + N, dv, dp + ((2 * C::TERM) >> 4), idO1, 1u);
              }
              mma_commit(su32(&ctl.empty[slot]));
            }
            if (!ok) break;
            mma_commit(su32(&ctl.p_free));
          }
        }
        ic += 2 * m.nt;
        tc += m.nt;
        ++qi;
      }
    }
    __syncwarp();
  } else if (warp == C::QUERY_WARP) {
    // ---- queries and masks of the items after the first, as soon as the scores of the one before are done
    int qi = -1;
    for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
      if (have == 0 || m.nt == 0 || ++qi == 0) continue;
      constexpr int MK = (N + 31) / 32;
      unsigned long long mask[MK];
#pragma unroll
      for (int j = 0; j < MK; ++j) {
        const int n = lane + 32 * j;
        mask[j] = n < m.rows ? a.masks[m.t.row0 + div_rep(m.n0 + n, rep, rep_inv)] : 0ull;
      }
      ok = load_queries<HD, N, TM_QTHREADS>(a, m, rep, rep_inv, vec & 1, lane, sp + C::Q, [&] {
        if (!tm_wait(su32(&ctl.q_free), ((uint32_t)qi & 1u) ^ 1u, abort_w, a.status)) return false;
#pragma unroll
        for (int j = 0; j < MK; ++j)
          if (lane + 32 * j < N) ctl.mask[qi % TM_MASKS][lane + 32 * j] = mask[j];
        return true;
      });
      if (!ok) break;
      proxy_fence();
      mbar_arrive(su32(&ctl.q_full[qi % TM_MASKS]));
    }
  } else {
    // ---- softmax: group wg has rows c0 .. c0 + NC - 1 of the tile, one thread a position
    constexpr int NC = C::NC;
    const int wg = warp >> 2, wt = tid & 127, w4 = warp & 3, c0 = wg * NC;
    const float c = 1.4426950408889634f / sqrtf((float)HD);
    const float2 c2 = make_float2(c, c);
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    constexpr int NB = NC / 8;  // blocks of eight rows; this thread holds rows n2, n2 + 1 of each
    const int n2 = c0 + (lane & 3) * 2;
    // where this lane's row of the four matrices of a block starts in P: row
    // lane % 8, positions 32 w4 + 8 (lane / 8) ..
    const uint32_t p_lane = (uint32_t)(w4 >> 1) * (3 * C::TERM) + (c0 + (lane & 7)) * 128 +
                            (((((w4 & 1) * 4) + (lane >> 3)) ^ (lane & 7)) << 4);
    int ic = 0, tc = 0, qi = 0;
    for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
      if (have == 0) continue;
      if (m.nt > 0 && qi == 0) {  // the first item's queries: nothing else to do yet
        if (tid < N) ctl.mask[0][tid] = tid < m.rows ? a.masks[m.t.row0 + div_rep(m.n0 + tid, rep, rep_inv)] : 0ull;
        load_queries<HD, N, 128 * C::SW>(a, m, rep, rep_inv, vec & 1, tid, sp + C::Q, [] { return true; });
        proxy_fence();
        mbar_arrive(su32(&ctl.q_first));
      }
      float2 base[NB], l[NB];  // negated base, sum of the weights
      float o[NC];             // element wt of the running output's rows
      bool scaled = false;     // the bases rose with this tile: the outputs before it are still to be scaled
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        base[b] = make_float2(-TM_FLOOR, -TM_FLOOR);
        l[b] = make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) o[n] = 0.f;
      if (wt < NC) {
        ctl.base[c0 + wt] = TM_FLOOR;
        ctl.sum[c0 + wt] = 0.f;
      }
      if (m.nt > 0) {  // the item's masks are there
        ok = q_wait(qi);
        if (all_any<128 * C::SW>(!ok)) {
          ok = false;
          break;
        }
      }
      for (int i = 0; i <= m.nt; ++i) {
        const int t = tc + i;
        if (i < m.nt) {
        ok = tm_wait(su32(&ctl.s_full[t & 1]), (uint32_t)(t >> 1) & 1u, abort_w, a.status) && ok;
        if (all_any<128 * C::SW>(!ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // scores of positions 32 w4 + 16 h + 8 r + lane / 4, 32 rows at a time
        uint32_t f[2][NC / 2];
        constexpr int W = NC < 32 ? NC : 32;
#pragma unroll
        for (int n = 0; n < NC; n += W) {
          uint32_t v[C::G][2][W / 2];
#pragma unroll
          for (int gr = 0; gr < C::G; ++gr)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tmem_frag<W>(tmem + (t & 1) * C::TM_S + gr * N + c0 + n + lanes + ((uint32_t)(16 * h) << 16), v[gr][h]);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < W / 2; e += 2) {
              float2 r = make_float2(__uint_as_float(v[C::G - 1][h][e]), __uint_as_float(v[C::G - 1][h][e + 1]));
#pragma unroll
              for (int gr = C::G - 2; gr >= 0; --gr)
                r = add2(r, make_float2(__uint_as_float(v[gr][h][e]), __uint_as_float(v[gr][h][e + 1])));
              f[h][n / 2 + e] = __float_as_uint(r.x);
              f[h][n / 2 + e + 1] = __float_as_uint(r.y);
            }
        }
        tc_fence_before();
        mbar_arrive(su32(&ctl.s_free[t & 1]));
        const int p0 = (m.t0 + i) * TM_PT + w4 * 32;  // the warp's first position
        if ((m.t0 + i + 1) * TM_PT > m.t.L) {  // the tile reaches past the committed positions
          // the value row of a position no row may meet is zeroed: one past the
          // sequence (whatever lies there), or a node's with an infinity or NaN
          const int it = (ic + v_item(i, m.nt)) * C::TERMS, pos = p0 + lane;
          // split tiles have a barrier of their own here: the places' may be a phase behind
          ok = MODE == kSplit ? tm_wait(su32(&ctl.v_full[t & 1]), (uint32_t)(t >> 1) & 1u, abort_w, a.status)
                              : tm_wait(su32(&ctl.full[it % C::S]), (uint32_t)(it / C::S) & 1u, abort_w, a.status);
          if (wg == 0) {  // (the wait may have run out for some lanes of a warp: all of them come to its ballot)
            uint4* vr = reinterpret_cast<uint4*>(sp + C::RING + it % C::S * C::SLOT + wt * 128);
            uint32_t bits = 0;
            if (ok && pos >= m.t.L && pos < m.t.P) {
#pragma unroll
              for (int e = 0; e < C::BLK * 8; ++e)
                bits = not_finite(vr[(e >> 3) * (TM_PT * 8) + ((e ^ lane) & 7)], bits);
            }
            const bool mine = (bits & 0x80008000u) != 0;
            if (ok && (pos >= m.t.P || mine))
              for (int term = 0; term < C::TERMS; ++term) {
                uint4* z = reinterpret_cast<uint4*>(sp + C::RING + (it + term) % C::S * C::SLOT + wt * 128);
#pragma unroll 4
                for (int e = 0; e < C::BLK * 8; ++e) z[(e >> 3) * (TM_PT * 8) + ((e ^ lane) & 7)] = make_uint4(0, 0, 0, 0);
              }
            // positions of the warp whose values are infinite or NaN: a row that sees one is NaN
            const unsigned found = __ballot_sync(0xffffffffu, mine);
            if (lane == 0) ctl.bad[w4] = found;
          }
          if (all_any<128 * C::SW>(!ok)) {
            ok = false;
            break;
          }
          const unsigned bad = ctl.bad[w4];
          // this lane's positions, counted from the first node (negative: committed)
          const uint32_t* words = reinterpret_cast<const uint32_t*>(ctl.mask[qi % TM_MASKS]) + 2 * n2;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int off = 8 * q + (lane >> 2), j = p0 + off - m.t.L;
            if (j >= 0) {
              const uint32_t past = j >= m.t.T ? 0u : ~0u, seen = (bad >> off) & 1u ? 0x7fc00000u : 0u;
              const uint32_t* w = words + (min(j, 63) >> 5);
#pragma unroll
              for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  uint32_t& x = f[q >> 1][4 * b + 2 * (q & 1) + e];
                  const bool sees = ((w[16 * b + 2 * e] & past) >> (j & 31)) & 1u;
                  x = sees ? (seen ? seen : x) : 0xff800000u;  // -inf
                }
            }
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t* x = &f[q >> 1][4 * b + 2 * (q & 1)];
            const float2 v = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, base[b]);
            top = fmaxf(top, fmaxf(v.x, v.y));
          }
        if (soft_any(top > TM_SLACK, wg)) {
          // new bases: the rows' largest scores so far
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            float mx = -INFINITY, my = -INFINITY;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mx = fmaxf(mx, __uint_as_float(f[q >> 1][4 * b + 2 * (q & 1)]));
              my = fmaxf(my, __uint_as_float(f[q >> 1][4 * b + 2 * (q & 1) + 1]));
            }
            mx = lanes_max(mx);
            my = lanes_max(my);
            if (lane < 4) {
              ctl.part[w4][8 * b + n2] = mx * c;
              ctl.part[w4][8 * b + n2 + 1] = my * c;
            }
          }
          soft_sync(wg);
          if (wt < NC) {
            const int n = c0 + wt;
            const float old = ctl.base[n];
            const float nb =
                fmaxf(fmaxf(fmaxf(ctl.part[0][n], ctl.part[1][n]), fmaxf(ctl.part[2][n], ctl.part[3][n])), old);
            ctl.corr[n] = nb == old ? 1.f : exp2_fast(old - nb);
            ctl.base[n] = nb;
          }
          soft_sync(wg);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const int n = 8 * b + n2;
            base[b] = make_float2(-ctl.base[n], -ctl.base[n + 1]);
            l[b].x *= ctl.corr[n];
            l[b].y *= ctl.corr[n + 1];
          }
          scaled = true;
        }
        ok = tm_wait(su32(&ctl.p_free), ((uint32_t)t & 1u) ^ 1u, abort_w, a.status) && ok;
        __syncwarp();
        const uint32_t ph = sbase + C::P + p_lane;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float2 p[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t* x = &f[q >> 1][4 * b + 2 * (q & 1)];
            const float2 e = fma2(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, base[b]);
            p[q] = make_float2(exp2_fast(e.x), exp2_fast(e.y));
            l[b] = add2(l[b], p[q]);
          }
#pragma unroll
          for (int term = 0; term < 3; ++term) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              w[q] = pack_bf16(p[q]);
              p[q] = add2(p[q], make_float2(-__uint_as_float(w[q] << 16), -__uint_as_float(w[q] & 0xffff0000u)));
            }
            store_t(ph + term * C::TERM + b * 1024, w[0], w[1], w[2], w[3]);
          }
        }
        proxy_fence();
        tc_fence_before();
        mbar_arrive(su32(&ctl.p_full));
        }
        // the output of the tile before joins the running one: it was complete before
        // this tile's P was written (whose barrier may be a phase on)
        if (i > 0) {
          if (i == m.nt) ok = tm_wait(su32(&ctl.p_free), (uint32_t)(t - 1) & 1u, abort_w, a.status) && ok;
          __syncwarp();
          tc_fence_after();
          const uint32_t src = tmem + C::TM_O + ((t - 1) & 1) * C::TM_S + lanes;
#pragma unroll
          for (int n = 0; n < NC; n += 16) {
            uint32_t v[C::G][16];
#pragma unroll
            for (int gr = 0; gr < C::G; ++gr) tmem_ld16(src + gr * N + c0 + n, v[gr]);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 r = make_float2(__uint_as_float(v[C::G - 1][e]), __uint_as_float(v[C::G - 1][e + 1]));
#pragma unroll
              for (int gr = C::G - 2; gr >= 0; --gr)
                r = add2(r, make_float2(__uint_as_float(v[gr][e]), __uint_as_float(v[gr][e + 1])));
              r = add2(r, make_float2(o[n + e], o[n + e + 1]));
              o[n + e] = r.x;
              o[n + e + 1] = r.y;
            }
          }
          if (scaled) {
#pragma unroll
            for (int n = 0; n < NC; ++n) o[n] *= ctl.corr[c0 + n];
          }
        }
        scaled = false;
      }
      if (m.nt > 0) {
        if (all_any<128 * C::SW>(!ok)) {  // every softmax thread comes here, whichever of them gave up
          ok = false;
          break;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float sx = lanes_sum(l[b].x), sy = lanes_sum(l[b].y);
          if (lane < 4) {
            ctl.part[w4][8 * b + n2] = sx;
            ctl.part[w4][8 * b + n2 + 1] = sy;
          }
        }
        soft_sync(wg);
        if (wt < NC) {
          const int n = c0 + wt;
          const float sum = (ctl.part[0][n] + ctl.part[1][n]) + (ctl.part[2][n] + ctl.part[3][n]);
          ctl.sum[n] = CL > 1 ? sum : (sum == 0.f ? 0.f : 1.f / sum);  // a row that saw nothing: zeroes
        }
        // the rows, through P's place (its readers are done) to whole lines
        float* os = reinterpret_cast<float*>(sp + C::P);  // [N][HD]
        if (wt < HD) {
#pragma unroll
          for (int n = 0; n < NC; ++n) os[(c0 + n) * HD + wt] = o[n];
        }
        soft_sync(wg);
        if (CL == 1) {
          constexpr int LPR = HD / 4;  // lanes of a row
#pragma unroll 1
          for (int n = c0 + wt / LPR; n < min(m.rows, c0 + NC); n += 128 / LPR) {
            const int row = m.n0 + n, node = div_rep(row, rep, rep_inv), d = wt % LPR * 4;
            const float4 v = *reinterpret_cast<const float4*>(os + n * HD + d);
            const float f = ctl.sum[n];
            float* dst = a.out + (size_t)(m.t.row0 + node) * a.ldo + (size_t)(m.g * rep + row - node * rep) * HD + d;
            if (vec & 2) {
              *reinterpret_cast<float4*>(dst) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
            } else {
              dst[0] = v.x * f;
              dst[1] = v.y * f;
              dst[2] = v.z * f;
              dst[3] = v.w * f;
            }
          }
          all_any<128 * C::SW>(false);  // P and the sums may be written again
        }
        ic += 2 * m.nt;
        tc += m.nt;
        ++qi;
      }
      if (CL > 1) break;  // one item for a cluster
    }
    if (!ok) *abort_w = 1;
  }
  if (CL > 1 && (have = tm_item(a, deal, 0, m)) == 1) {
    static_assert(sizeof(ctl.mask) >= 8 * N * sizeof(float), "a factor per share and row, where the masks were");
    join_shares<HD, N, C::THREADS, HD>(a, m, rep, rep_inv, vec & 2, ctl.base, ctl.sum, reinterpret_cast<float*>(ctl.mask),
                                       reinterpret_cast<float*>(sp + C::P), abort_w);
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_w) {
    if (MODE == kTma && warp >= C::LOAD_WARP) land_copies<C::S>(ctl.copies, warp - C::LOAD_WARP, ctl.full);
    if (warp == C::MMA_WARP && elect_one()) land_products(su32(&ctl.done));
    __syncwarp();
  }
  if (warp == C::MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
}

// ------------------------------------------------------------- host side

template <int HD, int N, int MODE>
int launch_mma(const TreeArgs& a, int layers, int dev, int n_sm, cudaStream_t s) {
  using C = TmCfg<HD, N, MODE>;
  static TmKernel known[kMaxDevices];
  return launch_items(tree_mma_kernel<HD, N, MODE>, known[dev], C::THREADS, C::SMEM, MODE == kTma, N, a, layers, n_sm, s);
}

// Whether tiles of 128 rows (tree_wide.cu) are done sooner than tiles of 64 on
// twice the CTAs.  A round of items costs about 6 us and 1.3 us for a tile of
// positions here, 9 and 1.65 us there; 64 nodes with two heads each (tiles of
// positions: us here, us there): 8 kv heads 1: 9.2, 11.4, 64: 25.2, 27.2; 32 kv
// heads 8: 16.3, 17.3, 16: 23.3, 21.0; 152 kv heads 1: 18.8, 13.2, 64: 209, 138;
// 512 kv heads 64: 711, 532.
bool wide_pays(const TreeArgs& a, int n_sm) {
  const long rows = (long)a.max_nodes * (a.Hq / a.kv.Hkv), heads = (long)a.n_seqs * a.kv.Hkv;
  const long tiles = ((long)a.kv.pages_per_stream * a.kv.page_size + TM_PT - 1) / TM_PT;
  auto us = [&](long items, double item, double tile) {
    const long rounds = (items + n_sm - 1) / n_sm, most = n_sm / items < 8 ? n_sm / items : 8, share = rounds > 1 ? 1 : most;
    return rounds * (item + tile * ((tiles + share - 1) / share));
  };
  return us(heads * ((rows + 127) / 128), 9, 1.65) < us(heads * ((rows + 63) / 64), 6, 1.3);
}

template <int HD, int MODE>
int launch_rows(const TreeArgs& a, int layers, int dev, int n_sm, cudaStream_t s) {
  const int rows = a.max_nodes * (a.Hq / a.kv.Hkv);
  if (rows <= 16) return launch_mma<HD, 16, MODE>(a, layers, dev, n_sm, s);
  if (rows <= 32 || MODE == kSplit) return launch_mma<HD, 32, MODE>(a, layers, dev, n_sm, s);
  if (MODE == kTma && rows > 64 && wide_pays(a, n_sm)) return launch_tree_wide(a, layers, dev, n_sm, s);
  return launch_mma<HD, MODE == kSplit ? 32 : 64, MODE>(a, layers, dev, n_sm, s);
}

template <int HD>
int launch_mode(const TreeArgs& a, int layers, int kdt, int dev, int n_sm, cudaStream_t s) {
  if (kdt == Q3TTS_F32) return launch_rows<HD, kSplit>(a, layers, dev, n_sm, s);
  // TMA boxes are pages of whole swizzle atoms (8 rows) that fill a tile a whole
  // number of times, or whole tiles of larger pages
  const int ps = a.kv.page_size;
  if ((ps >= 8 && ps <= TM_PT && TM_PT % ps == 0) || ps % TM_PT == 0)
    return launch_rows<HD, kTma>(a, layers, dev, n_sm, s);
  return launch_rows<HD, kCopy>(a, layers, dev, n_sm, s);
}

}  // namespace

int launch_tree_attention(const TreeArgs& a, int layers, int kdt, cudaStream_t s) {
  if (a.n_seqs <= 0 || a.n_rows <= 0) return Q3TTS_OK;
  int dev = 0, n_sm = 0;
  if (!current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  return a.kv.hd == 128 ? launch_mode<128>(a, layers, kdt, dev, n_sm, s) : launch_mode<64>(a, layers, kdt, dev, n_sm, s);
}

}  // namespace q3

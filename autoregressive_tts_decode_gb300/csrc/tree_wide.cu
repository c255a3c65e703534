// tree_wide.cu -- attention of drafted trees with more than 64 rows to a kv head
// (nodes x q heads of its group): 128 rows to a tile.
//
// The mathematics are tree_attention.cu's, which lays a tile of up to 64 rows
// along the MMA's N side, so that few rows cost little.  From 65 rows on they
// fill its M side instead:
//   S = Q K^T  M 128 rows, N 128 positions: Q as three bf16 terms in shared
//              memory, K as it lies in the cache;
//   O = P V    P as three bf16 terms in tensor memory, where it takes its scores'
//              place, V as it lies in the cache (an N-major operand).
// K and V are then read once for twice the rows, a row's scores are two threads',
// and P does not pass through shared memory.  The small terms are multiplied
// first into one accumulator, which the large one's truncated sums follow; the
// outputs of successive tiles are added in fp32 registers.
//
// Roles of a CTA (one per SM): a warp loads the keys by TMA, one the values, one
// thread issues the MMAs (scores of tile t + 1 before the outputs of tile t), one
// warp splits the queries of the items after the first, and two groups of four
// warps are the softmax, each with half of a tile's positions and half of the
// output's elements (one thread a row and half).  The tensor cores work in order,
// which orders most of what shares tensor memory: the scores of tile t + 2 come
// after the outputs of tile t, which have read P where they go; the outputs of
// tile t + 1 wait for its P, which the softmax announces when it has also read
// the outputs of tile t.
//
// The bound is the tensor cores' time for six products of 128 x 128 x 128 a tile:
// four sequences of 30011 .. 32768 positions, 64 nodes with two heads each: 127 us
// (tiles of 64 rows: 197), of which the products alone take 99 on the 128 SMs that
// 32 items in clusters of four fill.
#include "tree.cuh"

namespace q3 {

namespace {

constexpr int TW_ROWS = 128;     // rows of a tile
constexpr int TW_SOFT = 256;     // softmax threads

template <int HD>
struct TwCfg {
  static constexpr int MMA_WARP = 8, KEY_WARP = 9, VALUE_WARP = 10, QUERY_WARP = 11, THREADS = 384;
  static constexpr int BLK = HD / 64;               // 128-byte swizzle blocks of a row
  static constexpr uint32_t SLOT = TM_PT * HD * 2;  // a K or V tile
  static constexpr uint32_t TERM = TW_ROWS * 128;   // one term of one 64-element block of Q
  static constexpr uint32_t QBYTES = BLK * 3 * TERM;
  static constexpr uint32_t CTL_BYTES = 2048;
  static constexpr int S = HD == 128 ? 4 : 8;       // tiles in the ring
  static constexpr uint32_t RING = QBYTES, CTL = RING + S * SLOT;
  static constexpr size_t SMEM = 1024 + CTL + CTL_BYTES;
  static constexpr int LD = HD + 4;                 // a row of the shares' outputs: float4 stores without conflicts
  // columns: scores and P of even and of odd tiles, outputs
  static constexpr uint32_t TM_B = 192, TM_LO = 128, TM_O = 2 * TM_B;
  static_assert(SMEM <= 227 * 1024 && TM_O + HD <= 512 && TW_ROWS * LD * 4 <= S * SLOT && 10 * TW_ROWS * 4 <= QBYTES,
                "shared and tensor memory");
};

template <int S>
struct TwCtl {
  unsigned long long full[S], empty[S], s_full[2], p_full, o_full, q_first, q_full, q_free, done;
  uint32_t tmem;
  int abort_w[2];  // given up, limit of the waits
  unsigned bad[2][4];
  int copies[2][8];
  uint16_t order[TM_SORT];  // sequences, longest first
  float part[2][TW_ROWS];   // each group's largest score of a row, and its sum at the end
};

// 32 fp32 columns of the warp's 32 lanes, one lane per thread (complete after wait::ld).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
        "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]),
        "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// A in tensor memory: a lane per row, two elements of K to a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t tmem_d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(
          tmem_d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}

// Lanes `away` apart exchange b of the lower for a of the upper.
__device__ __forceinline__ void exchange(float4& a, float4& b, bool upper, int away) {
  const float4 give = upper ? a : b;
  float4 take;
  take.x = __shfl_xor_sync(0xffffffffu, give.x, away);
  take.y = __shfl_xor_sync(0xffffffffu, give.y, away);
  take.z = __shfl_xor_sync(0xffffffffu, give.z, away);
  take.w = __shfl_xor_sync(0xffffffffu, give.w, away);
  if (upper)
    a = take;
  else
    b = take;
}
// Barrier and vote of the softmax threads.
__device__ __forceinline__ bool vote(bool p, int id) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id)
      : "memory");
  return r != 0;
}

template <int HD>
__global__ void __launch_bounds__(TwCfg<HD>::THREADS, 1)
    tree_wide_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ TreeArgs a, int row_tiles, int box, int items,
                     int vec, unsigned rep_inv) {
  using C = TwCfg<HD>;
  using Ctl = TwCtl<C::S>;
  static_assert(sizeof(Ctl) <= C::CTL_BYTES && sizeof(Ctl::part) >= TM_SORT * sizeof(int), "control block");
  extern __shared__ uint8_t tw_raw[];
  const uint32_t raw = su32(tw_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* sp = tw_raw + (sbase - raw);
  Ctl& ctl = *reinterpret_cast<Ctl*>(sp + C::CTL);
  volatile int* abort_w = ctl.abort_w;

  namespace cg = cooperative_groups;
  const int CL = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rep = a.Hq / a.kv.Hkv;

  TmDeal deal{items, row_tiles, TW_ROWS, (int)gridDim.x / CL, (int)blockIdx.x / CL, rank, CL, nullptr};
  prefetch_first(a, deal);
  if (tid == 0) {
    for (int i = 0; i < C::S; ++i) {
      mbar_init(su32(&ctl.full[i]), 1);
      mbar_init(su32(&ctl.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(su32(&ctl.s_full[i]), 1);
    mbar_init(su32(&ctl.p_full), TW_SOFT);
    mbar_init(su32(&ctl.o_full), 1);
    mbar_init(su32(&ctl.q_first), TW_SOFT);
    mbar_init(su32(&ctl.q_full), 32);
    mbar_init(su32(&ctl.q_free), 1);
    mbar_init(su32(&ctl.done), 1);
    ctl.abort_w[0] = 0;
    ctl.abort_w[1] = a.wait_1024;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid >= 32 && tid < 48) ctl.copies[(tid >> 3) & 1][tid & 7] = -1;
  pdl_wait();  // q and the appended keys and values come from the previous kernels
  // (tensor memory after the wait: a kernel before may still be about to take its own)
  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&ctl.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  const bool sorted = items > (int)gridDim.x / CL && a.n_seqs <= TM_SORT;
  if (sorted) {
    deal.order = ctl.order;
    sort_lengths(a, reinterpret_cast<int*>(ctl.part), ctl.order);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  const uint32_t ring = sbase + C::RING;
  float* shares = reinterpret_cast<float*>(sp);  // bases and sums for the other shares of the item, factors; in Q's place

  TmItem m;
  int have = 0;
  bool ok = true;

  if (warp == C::KEY_WARP || warp == C::VALUE_WARP) {
    const int w = warp - C::KEY_WARP;
    ok = tma_loads<HD, C::S>(&map, a, deal, box, w > 0, ring, ctl.full, ctl.empty, ctl.copies[w], abort_w);
  } else if (warp == C::MMA_WARP) {
    // ---- MMA issue
    if (elect_one()) {
      constexpr uint32_t idS = f16_idesc(TW_ROWS, TM_PT, false), idO = f16_idesc(TW_ROWS, HD, false) | 1u << 16;  // B N-major
      const int lost = blockIdx.x == 0 ? a.lost_tile : -1;
      int ic = 0, tc = 0, qi = 0;  // ring tiles, position tiles and items so far
      for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
        if (have == 0 || m.nt == 0) continue;
        ok = tm_wait(su32(qi == 0 ? &ctl.q_first : &ctl.q_full), (uint32_t)(qi == 0 ? 0 : qi - 1) & 1u, abort_w, a.status);
        tc_fence_after();
        for (int i = 0; i <= m.nt && ok; ++i) {
          if (i < m.nt) {  // scores of tile i
            const int it = ic + k_item(i), t = tc + i, slot = it % C::S;
            ok = t != lost && tm_wait(su32(&ctl.full[slot]), (uint32_t)(it / C::S) & 1u, abort_w, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t d = tmem + (t & 1) * C::TM_B;
            const uint64_t dk = sw128_desc(ring) + slot * (C::SLOT >> 4), dq = sw128_desc(sbase);
#pragma unroll
            for (int term = 2; term >= 0; --term)
#pragma unroll
              for (int s = 0; s < HD / 16; ++s)
                mma_bf16(d, dq + (((s >> 2) * 3 + term) * C::TERM >> 4) + (s & 3) * 2, dk + ((s >> 2) * TM_PT * 128 >> 4) + (s & 3) * 2,
                         idS, (term < 2 || s != 0) ? 1u : 0u);
            mma_commit(su32(&ctl.empty[slot]));
            mma_commit(su32(&ctl.s_full[t & 1]));
            if (i == m.nt - 1) mma_commit(su32(&ctl.q_free));
          }
          if (i > 0) {  // outputs of tile i - 1
            const int it = ic + v_item(i - 1, m.nt), t = tc + i - 1, slot = it % C::S;
            ok = tm_wait(su32(&ctl.full[slot]), (uint32_t)(it / C::S) & 1u, abort_w, a.status) &&
                 tm_wait(su32(&ctl.p_full), (uint32_t)t & 1u, abort_w, a.status);
            if (!ok) break;
            tc_fence_after();
            const uint32_t p = tmem + (t & 1) * C::TM_B;
            const uint64_t dv = sw128_desc(ring, HD == 128 ? TM_PT * 128 : 1024) + slot * (C::SLOT >> 4);
#pragma unroll
            for (int term = 2; term >= 0; --term)
#pragma unroll
              for (int s = 0; s < 8; ++s) {  // 16 positions: eight columns of a term
                const uint32_t at = term == 2 ? C::TM_LO + 8 * s : 32 * (s >> 1) + 16 * term + 8 * (s & 1);
                mma_bf16_ts(tmem + C::TM_O, p + at, dv + (s * 2048 >> 4), idO, (term < 2 || s != 0) ? 1u : 0u);
              }
            mma_commit(su32(&ctl.empty[slot]));
            mma_commit(su32(&ctl.o_full));
          }
        }
        ic += 2 * m.nt;
        tc += m.nt;
        ++qi;
      }
    }
    __syncwarp();
  } else if (warp >= C::QUERY_WARP) {
    // ---- queries of the items after the first, as soon as the scores of the one before are done
    int qi = 0;
    for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
      if (have == 0 || m.nt == 0 || qi++ == 0) continue;
      ok = load_queries<HD, TW_ROWS, 32>(a, m, rep, rep_inv, vec & 1, lane, sp, [&] {
        return tm_wait(su32(&ctl.q_free), (uint32_t)qi & 1u, abort_w, a.status);
      });
      if (!ok) break;
      proxy_fence();
      mbar_arrive(su32(&ctl.q_full));
    }
  } else {
    // ---- softmax: group wg has positions 64 wg .. of a tile, elements wg HD / 2 .. of the output
    const float c = 1.4426950408889634f / sqrtf((float)HD);
    const float2 c2 = make_float2(c, c);
    constexpr int HW = HD / 2;  // elements of the output that a thread holds
    const int wg = warp >> 2, w4 = warp & 3, r = tid & 127;  // the thread's row
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    int ic = 0, tc = 0, qi = 0;  // ring tiles, position tiles, items so far
    for (int k = 0; ok && (have = tm_item(a, deal, k, m)) >= 0; ++k) {
      if (have == 0) continue;
      const int row = m.n0 + r, node = div_rep(row, rep, rep_inv);
      unsigned long long mask = r < m.rows ? a.masks[m.t.row0 + node] : 0ull;
      if (m.t.T < 64) mask &= (1ull << m.t.T) - 1;
      if (m.nt > 0 && qi++ == 0) {
        load_queries<HD, TW_ROWS, TW_SOFT>(a, m, rep, rep_inv, vec & 1, tid, sp, [] { return true; });
        proxy_fence();
        mbar_arrive(su32(&ctl.q_first));
      }
      float base = TM_FLOOR, l = 0.f, corr = 1.f;  // the row's base, sum of weights, factor of the base's last rise
      float2 o[HW / 2];
#pragma unroll
      for (int n = 0; n < HW / 2; ++n) o[n] = make_float2(0.f, 0.f);
      for (int i = 0; i <= m.nt; ++i) {
        const int t = tc + i;
        const bool scores = i < m.nt;
        if (scores) {
          ok = tm_wait(su32(&ctl.s_full[t & 1]), (uint32_t)(t >> 1) & 1u, abort_w, a.status) && ok;
          const int p0 = (m.t0 + i) * TM_PT;
          const bool edge = p0 + TM_PT > m.t.L;  // the tile reaches past the committed positions
          if (edge) {
            // the value row of a position no row may meet is zeroed: one past the
            // sequence (whatever lies there), or a node's with an infinity or NaN
            const int it = ic + v_item(i, m.nt), pos = p0 + r;
            ok = tm_wait(su32(&ctl.full[it % C::S]), (uint32_t)(it / C::S) & 1u, abort_w, a.status) && ok;
            if (wg == 0) {
              uint4* vr = reinterpret_cast<uint4*>(sp + C::RING + it % C::S * C::SLOT + r * 128);
              uint32_t bits = 0;
              if (ok && pos >= m.t.L && pos < m.t.P) {
#pragma unroll
                for (int e = 0; e < C::BLK * 8; ++e) bits = not_finite(vr[(e >> 3) * (TM_PT * 8) + ((e ^ lane) & 7)], bits);
              }
              const bool mine = (bits & 0x80008000u) != 0;
              if (ok && (pos >= m.t.P || mine)) {
#pragma unroll 4
                for (int e = 0; e < C::BLK * 8; ++e) vr[(e >> 3) * (TM_PT * 8) + ((e ^ lane) & 7)] = make_uint4(0, 0, 0, 0);
                proxy_fence();
              }
              // positions whose values are infinite or NaN: a row that sees one is NaN
              const unsigned found = __ballot_sync(0xffffffffu, mine);
              if (lane == 0) ctl.bad[t & 1][w4] = found;
            }
          }
          // (giving up is decided by votes of all softmax threads, so that they leave together)
          if (vote(!ok, 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t src = tmem + (t & 1) * C::TM_B + lanes;
          // 32 scores of the tile; -inf where the row does not see the position
          auto take = [&](int ch, float (&x)[32]) {
            tmem_ld32(src + 32 * ch, x);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
            const int d = p0 + 32 * ch - m.t.L;  // its first position, counted from the first node
            if (d > -32) {
              const uint32_t sees = d >= 64 ? 0u : d >= 0 ? (uint32_t)(mask >> d) : (uint32_t)(mask << -d) | ((1u << -d) - 1);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = (sees >> e) & 1u ? x[e] : -INFINITY;
              const uint32_t bad = ctl.bad[t & 1][ch];
              if (bad & sees) x[0] = __uint_as_float(0x7fc00000u);
            }
          };
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x[32];
            take(2 * wg + h, x);
#pragma unroll
            for (int e = 0; e < 32; ++e) top[e & 3] = fmaxf(top[e & 3], x[e]);
          }
          float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
          corr = 1.f;
          const bool rises = mx - base > TM_SLACK;
          if (vote(rises, 2)) {  // both halves of a row have the same base
            ctl.part[wg][r] = mx;
            vote(false, 1);
            mx = fmaxf(mx, ctl.part[wg ^ 1][r]);
            if (mx - base > TM_SLACK) {
              corr = exp2_fast(base - mx);
              base = mx;
              l *= corr;
            }
          }
          const float2 nb = make_float2(-base, -base);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int ch = 2 * wg + h;
            float x[32];
            take(ch, x);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 v = fma2(make_float2(x[e], x[e + 1]), c2, nb);
              const float2 p = make_float2(exp2_fast(v.x), exp2_fast(v.y));
              sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], p);
              x[e] = p.x;
              x[e + 1] = p.y;
            }
#pragma unroll
            for (int term = 0; term < 3; ++term) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float2 v = make_float2(x[2 * e], x[2 * e + 1]);
                w[e] = pack_bf16(v);
                const float2 rest = add2(v, make_float2(-__uint_as_float(w[e] << 16), -__uint_as_float(w[e] & 0xffff0000u)));
                x[2 * e] = rest.x;
                x[2 * e + 1] = rest.y;
              }
              tmem_st16(src + (term < 2 ? 32 * ch + 16 * term : C::TM_LO + 16 * ch), w);
            }
          }
          // (the running sum takes a tile's at a time: its own roundings stay few)
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
        // the output of the tile before joins the running one: the tensor cores
        // have had this tile's softmax to finish it
        if (i > 0) {
          ok = tm_wait(su32(&ctl.o_full), (uint32_t)(t - 1) & 1u, abort_w, a.status) && ok;
          __syncwarp();
          tc_fence_after();
#pragma unroll
          for (int n = 0; n < HW; n += 32) {
            float x[32];
            tmem_ld32(tmem + C::TM_O + wg * HW + n + lanes, x);
            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
            for (int e = 0; e < 32; e += 2) o[(n + e) / 2] = add2(o[(n + e) / 2], make_float2(x[e], x[e + 1]));
          }
          if (__any_sync(0xffffffffu, scores && corr != 1.f)) {
#pragma unroll
            for (int n = 0; n < HW / 2; ++n) o[n] = make_float2(o[n].x * corr, o[n].y * corr);
          }
        }
        if (scores) {
          tc_fence_before();
          mbar_arrive(su32(&ctl.p_full));
        }
      }
      if (m.nt > 0) ctl.part[wg][r] = l;
      if (vote(!ok, 1)) {
        ok = false;
        break;
      }
      if (m.nt > 0) l = ctl.part[0][r] + ctl.part[1][r];
      ic += 2 * m.nt;
      tc += m.nt;
      if (CL > 1) {  // one item for a cluster; the ring's copies and MMAs are done
        if (wg == 0) {
          shares[r] = base;
          shares[TW_ROWS + r] = l;
        }
        float* os = reinterpret_cast<float*>(sp + C::RING) + r * C::LD + wg * HW;
#pragma unroll
        for (int n = 0; n < HW; n += 4)
          *reinterpret_cast<float4*>(os + n) = make_float4(o[n / 2].x, o[n / 2].y, o[n / 2 + 1].x, o[n / 2 + 1].y);
        break;
      }
      // four lanes exchange quarters of their rows, so that they write 64 bytes of one
      // row after the other
      const float f = l == 0.f ? 0.f : 1.f / l;  // a row that saw nothing: zeroes
#pragma unroll
      for (int n = 0; n < HW; n += 16) {
        float4 v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
          v[q] = make_float4(o[n / 2 + 2 * q].x * f, o[n / 2 + 2 * q].y * f, o[n / 2 + 2 * q + 1].x * f, o[n / 2 + 2 * q + 1].y * f);
        exchange(v[0], v[1], lane & 1, 1);
        exchange(v[2], v[3], lane & 1, 1);
        exchange(v[0], v[2], lane & 2, 2);
        exchange(v[1], v[3], lane & 2, 2);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r4 = (r & ~3) + q, row4 = m.n0 + r4, node4 = div_rep(row4, rep, rep_inv);
          float* dst = a.out + (size_t)(m.t.row0 + node4) * a.ldo + (size_t)(m.g * rep + row4 - node4 * rep) * HD + wg * HW + n +
                       (lane & 3) * 4;
          if (r4 < m.rows) {
            if (vec & 2) {
              *reinterpret_cast<float4*>(dst) = v[q];
            } else {
              dst[0] = v[q].x;
              dst[1] = v[q].y;
              dst[2] = v[q].z;
              dst[3] = v[q].w;
            }
          }
        }
      }
    }
    if (!ok) *abort_w = 1;
  }
  if (CL > 1 && (have = tm_item(a, deal, 0, m)) == 1)
    join_shares<HD, TW_ROWS, C::THREADS, C::LD>(a, m, rep, rep_inv, vec & 2, shares, shares + TW_ROWS, shares + 2 * TW_ROWS,
                                                reinterpret_cast<float*>(sp + C::RING), abort_w);
  tc_fence_before();
  __syncthreads();
  if (*abort_w) {
    if (warp == C::KEY_WARP || warp == C::VALUE_WARP) land_copies<C::S>(ctl.copies, warp - C::KEY_WARP, ctl.full);
    if (warp == C::MMA_WARP && elect_one()) land_products(su32(&ctl.done));
    __syncwarp();
  }
  if (warp == C::MMA_WARP) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <int HD>
int launch_wide(const TreeArgs& a, int layers, int dev, int n_sm, cudaStream_t s) {
  using C = TwCfg<HD>;
  static TmKernel known[kMaxDevices];
  return launch_items(tree_wide_kernel<HD>, known[dev], C::THREADS, C::SMEM, true, TW_ROWS, a, layers, n_sm, s);
}

}  // namespace

int launch_tree_wide(const TreeArgs& a, int layers, int dev, int n_sm, cudaStream_t s) {
  return a.kv.hd == 128 ? launch_wide<128>(a, layers, dev, n_sm, s) : launch_wide<64>(a, layers, dev, n_sm, s);
}

}  // namespace q3

// kv8_wide.cu -- attention of many new rows over the 8-bit cache (chunks of prompts, large
// drafted trees): 128 rows (new rows x q heads of a kv head's group) to a tile.
//
// The mathematics are kv8_attention.cu's.  From some rows on the tensor cores are the bound, and
// two fp16 products cost less than eight of E4M3: fp16 holds every E4M3 code, and two fp16
// terms hold 22 bits of a query or a weight.  Of bf16 rows a query is one term (fp16 has the more bits, and
// the row is scaled so that its largest element is 2^14 or more), and so is a weight: its 11 bits are
// rounded off by half a step, 2^-11 of it, against the output's own 2^-8.
//   S = Q K^T  M 128 rows, N 128 positions: Q in tensor memory, K converted;
//   O = P V    P in tensor memory, in its scores' place, V converted (an N-major operand).
// The small terms are multiplied first into one accumulator; the outputs of successive tiles
// are added in fp32 registers.  Keys' powers are factors of the scores, values' powers of the
// weights; a row's base is its largest score and power so far, a whole number, less 8 (weights of
// 2^8, and up to 2^15 before the base follows: fp16's smallest step is 2^-24).
//
// Roles of a CTA (one per SM): two warps load codes, two convert the keys and two the values (a row's
// 16 codes a lane), one looks up the powers, one thread issues the MMAs, two groups of four warps are
// the softmax, of the even and of the odd tiles (one thread a row, which needs no word of another), and
// two add up the outputs (a row's half a thread).  While one group works on its scores, the tensor cores make the
// other's, or outputs: scores of tile t + 2 follow the outputs of tile t, whose P they overwrite, and are the time in
// which those outputs are read.
//
// Four sequences of 30011 .. 32768 positions, 64 nodes with two heads each, fp32: 119 us, 1.7 a tile of 128 x 128 (the
// products take 1.05); 2048 bf16 rows after 14336: 318 us, 1.25 a tile (0.53).  Without the softmax's work these are 86
// and 221 us, without the conversion 107 and 269, without adding up 116 and 311, with a sixteenth of the products 92
// and 277: no unit is full (a scheduler issues in half of its cycles), the instructions of all roles share it.  An item
// begins and ends in about 11 us.
#include "kv8_tiles.cuh"

namespace q3 {

namespace {

constexpr int KW_ROWS = 128;  // rows of a tile
constexpr int KW_SOFT = 256;  // softmax threads, and as many that add up
constexpr int KW_CONV = 64;   // threads that convert keys, and as many that convert values
constexpr float KW_TINY = 1e-37f;  // the least factor of a score: a masked one stays -inf
constexpr float KW_BASE = 8.f, KW_MOST = 15.f;  // log2 of the weights at the base, and at most

template <class T, int HD>
struct KwCfg {
  static constexpr int SUM_WARP = 8, MMA_WARP = 16, LOAD_WARP = 17, CONV_WARP = 19, POWER_WARP = 23, THREADS = 768;
  static constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;
  static constexpr uint32_t TILE = TM_PT * HD * 2;   // a converted K or V tile
  static constexpr uint32_t SLOT = TM_PT * HD;       // a tile of codes
  static constexpr int S = 4 * (128 / HD);           // tiles of codes in their ring
  static constexpr uint32_t K = 0, V = 2 * TILE, RING = 4 * TILE, CTL = RING + S * SLOT;
  static constexpr int LD = HD + 4;                  // a row of the outputs in shared memory
  static constexpr size_t SMEM = 227 * 1024;         // (all of an SM's, as of its tensor memory)
  // columns: scores and P of even and of odd tiles, outputs, queries
  static constexpr uint32_t TM_O = 256, TM_Q = 384, TM_QT = HD / 2;
  static_assert(KW_ROWS * LD * 4 <= 4 * TILE, "the outputs, where the converted tiles were");
};

template <int S>
struct KwCtl {
  unsigned long long full[S], empty[S], k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full, o_free, q_full, done, pw_full[4], pw_empty[4], bad_full[4], base_full[4];
  uint32_t tmem;
  int abort_w[2];  // given up, limit of the waits
  int seq;
  alignas(16) unsigned none[4][4];  // positions of a tile whose values do not count
  unsigned bad[4][4];               // of them, new rows with a NaN
  float4 power[4][TM_PT];     // of a position (or those that share a block): key power x 2^-15, value power's exponent, its inverse
  float bases[4][KW_ROWS];    // of the rows in a tile
  float end[2][2][KW_ROWS];   // each softmax group's last base and sum
  float base[KW_ROWS], sum[KW_ROWS];
  float fac[8][KW_ROWS];
  alignas(16) int len[KF_SORT];
};

// kind::f16: D fp32, A and B fp16, A in tensor memory; B K-major or N-major (bit 16).
__host__ __device__ constexpr uint32_t h16_idesc(int M, int N, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(
          tmem_d),
      "r"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
// 32 or 8 columns of the warp's 32 lanes, one lane per thread (complete after wait::ld).
__device__ __forceinline__ void tmem_ld32f(uint32_t taddr, float (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]),
        "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]),
        "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(taddr));
}
// 16 columns into r[O ..] and the largest of them.
template <int O>
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, float (&r)[32], float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, %16, [%17];"
      : "=f"(r[O]), "=f"(r[O + 1]), "=f"(r[O + 2]), "=f"(r[O + 3]), "=f"(r[O + 4]), "=f"(r[O + 5]), "=f"(r[O + 6]), "=f"(r[O + 7]),
        "=f"(r[O + 8]), "=f"(r[O + 9]), "=f"(r[O + 10]), "=f"(r[O + 11]), "=f"(r[O + 12]), "=f"(r[O + 13]), "=f"(r[O + 14]),
        "=f"(r[O + 15]), "=f"(top)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8u(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8u(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Two floats to fp16 (x in the low half), and back.
__device__ __forceinline__ uint32_t pack_half(float x, float y) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(y), "f"(x));
  return r;
}
__device__ __forceinline__ float2 unpack_half(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2*>(&h)); }
// Four E4M3 codes as fp16.
__device__ __forceinline__ uint2 codes_half(uint32_t w) {
  uint2 r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.x) : "h"(static_cast<unsigned short>(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r.y) : "h"(static_cast<unsigned short>(w >> 16)));
  return r;
}
// Registers, of 80 a thread at the launch (768 x 80 in all): the softmax's two warpgroups take
// what loading, converting and the issue of the MMAs do not need (256 x (104 + 80 + 56)).
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 104;"); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 56;"); }
// Barrier and vote of COUNT threads.
template <int COUNT = KW_SOFT>
__device__ __forceinline__ bool kw_vote(bool p, int id) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, %3, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "n"(COUNT)
      : "memory");
  return r != 0;
}

template <class T, int HD, int GRAN, bool TMA>
__global__ void __launch_bounds__(KwCfg<T, HD>::THREADS, 1)
    kv8_wide_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Kv8AttnArgs a, const KfDeal d) {
  using C = KwCfg<T, HD>;
  using Ctl = KwCtl<C::S>;
  static_assert(1024 + C::CTL + sizeof(Ctl) <= C::SMEM, "shared memory");
  extern __shared__ uint8_t kw_raw[];
  const uint32_t raw = su32(kw_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* sp = kw_raw + (sbase - raw);
  Ctl& ctl = *reinterpret_cast<Ctl*>(sp + C::CTL);
  volatile int* abort_w = ctl.abort_w;
  int* status = a.r.status;

  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  const int CL = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int rep = a.Hq / a.c.Hkv;

  if (tid == 0) {
    for (int i = 0; i < C::S; ++i) {
      mbar_init(su32(&ctl.full[i]), TMA ? 1 : 32);
      mbar_init(su32(&ctl.empty[i]), KW_CONV);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(su32(&ctl.k_full[i]), KW_CONV);
      mbar_init(su32(&ctl.v_full[i]), KW_CONV);
      mbar_init(su32(&ctl.k_empty[i]), 1);
      mbar_init(su32(&ctl.v_empty[i]), 1);
      mbar_init(su32(&ctl.s_full[i]), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(su32(&ctl.p_full[i]), KW_ROWS);
    for (int i = 0; i < 4; ++i) {
      mbar_init(su32(&ctl.pw_full[i]), 32);
      mbar_init(su32(&ctl.pw_empty[i]), KW_ROWS + KW_CONV);
      mbar_init(su32(&ctl.bad_full[i]), KW_CONV);
      mbar_init(su32(&ctl.base_full[i]), KW_ROWS);
    }
    mbar_init(su32(&ctl.o_full), 1);
    mbar_init(su32(&ctl.o_free), KW_SOFT);
    mbar_init(su32(&ctl.q_full), KW_SOFT);
    mbar_init(su32(&ctl.done), 1);
    ctl.abort_w[0] = 0;
    ctl.abort_w[1] = d.wait_1024;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();  // q and the rows written to the cache come from the previous kernels
  pdl_trigger();
  // (tensor memory after the wait: a kernel before may still be about to take its own)
  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&ctl.tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  KfItem m;
  const int wanted = first_item(a, d, CL, KW_ROWS, m);
  if (d.sorted) find_sequence<C::THREADS>(a.r, wanted, ctl.len, &ctl.seq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  m.seq = d.sorted ? ctl.seq : wanted;
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  const bool have = take_item(a, d, CL, rank, KW_ROWS, m);
  bool ok = true;
  int issued = 0;  // tiles that the loading warp has filled or is filling
  float* os = reinterpret_cast<float*>(sp);  // [KW_ROWS][LD]: the outputs, where the converted tiles were

  if (m.nt > 0) {
    if (warp == C::LOAD_WARP || warp == C::LOAD_WARP + 1) {
      give_registers();
      // (one warp for both: issuing the boxes of 16-position pages took longer than a tile's products)
      ok = load_tiles<HD, C::S, TMA, true>(&map, a, m, d.box, sbase + C::RING, ctl.full, ctl.empty, warp - C::LOAD_WARP, issued, abort_w);
    } else if (warp == C::MMA_WARP) {
      // ---- MMA issue
      give_registers();
      if (elect_one()) {
        constexpr uint32_t idS = h16_idesc(KW_ROWS, TM_PT, false), idO = h16_idesc(KW_ROWS, HD, true);
        const int lost = blockIdx.x == 0 ? d.lost_tile : -1;
        auto wait = [&](unsigned long long* bar, int phase) { return kv8_wait(su32(bar), (uint32_t)phase & 1u, abort_w, status); };
        auto scores = [&](int t) -> bool {
          const int b = t & 1;
          if (t == lost || !wait(&ctl.k_full[b], t >> 1)) return false;
          tc_fence_after();
          const uint64_t dk = sw128_desc(sbase + C::K + b * C::TILE);
#pragma unroll
          for (int term = C::TERMS - 1; term >= 0; --term)
#pragma unroll
            for (int s = 0; s < HD / 16; ++s)
              mma_f16_ts(tmem + b * 128, tmem + C::TM_Q + term * C::TM_QT + s * 8, dk + ((s >> 2) * TM_PT * 128 >> 4) + (s & 3) * 2, idS,
                         term < C::TERMS - 1 || s != 0);
          mma_commit(su32(&ctl.k_empty[b]));
          mma_commit(su32(&ctl.s_full[b]));
          return true;
        };
        ok = wait(&ctl.q_full, 0) && scores(0) && (m.nt < 2 || scores(1));
        for (int t = 0; t < m.nt && ok; ++t) {
          const int b = t & 1;
          ok = wait(&ctl.v_full[b], t >> 1) && wait(&ctl.p_full[b], t >> 1) && (t == 0 || wait(&ctl.o_free, t - 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t dv = sw128_desc(sbase + C::V + b * C::TILE, HD == 128 ? TM_PT * 128 : 1024);
#pragma unroll
          for (int term = C::TERMS - 1; term >= 0; --term)
#pragma unroll
            for (int s = 0; s < 8; ++s)  // 16 positions: eight columns of a term
              mma_f16_ts(tmem + C::TM_O, tmem + b * 128 + 16 * s + 8 * term, dv + (s * 2048 >> 4), idO,
                         term < C::TERMS - 1 || s != 0);
          mma_commit(su32(&ctl.v_empty[b]));
          mma_commit(su32(&ctl.o_full));
          if (t + 2 < m.nt) ok = scores(t + 2);
        }
      }
      __syncwarp();
    } else if (warp == C::POWER_WARP) {
      // ---- powers, four positions a lane
      give_registers();
      Powers<4> pw(a, d, m, lane);
      for (int t = 0; t < m.nt; ++t) {
        ok = kv8_wait(su32(&ctl.pw_empty[t & 3]), ((uint32_t)(t >> 2) & 1u) ^ 1u, abort_w, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int n = lane + 32 * j, pos = (m.t0 + t) * TM_PT + n, e = min(max(pw.v[j] - 127, -KV8_EXP), KV8_EXP);
          // a new row's block of NaN: rows that see it are told by its bit alone
          const bool bad = pos >= m.t.L && (pw.k[j] == 255 || pw.v[j] == 255);
          const bool none = bad || pw.v[j] < 127 - KV8_EXP || pos >= m.end;  // no values, or none that count
          if (n % GRAN == 0)
            ctl.power[t & 3][n / GRAN] = make_float4(bad ? 1.f : kv8_power(pw.k[j]) * 0x1p-15f, pw.v[j] == 255 && !bad ? kv8_power(255) : (float)e,
                                                     __int_as_float((127 - e) << 23), 0.f);
          const unsigned b0 = __ballot_sync(0xffffffffu, bad), n0 = __ballot_sync(0xffffffffu, none);
          if (lane == 0) {
            ctl.bad[t & 3][j] = b0;
            ctl.none[t & 3][j] = n0;
          }
        }
        mbar_arrive(su32(&ctl.pw_full[t & 3]));
        pw.next(a, d, m, t, lane);
      }
    } else if (warp >= C::CONV_WARP) {
      // ---- codes to fp16: two warps the keys, two the values.  A thread has chunk c (16 codes) of every RPI-th
      // row.  Eight lanes have four chunks of rows r and r ^ 5, whose places in the swizzle are apart
      // both in the codes' tile and (at twice the chunk) in fp16's; rows RPI apart, a multiple of 8, have the same.
      give_registers();
      constexpr int RPI = KW_CONV / (HD / 16), ROWS = TM_PT / RPI, U = 4;
      static_assert(RPI % 8 == 0 && ROWS % U == 0, "rows of a thread");
      const int h = (warp - C::CONV_WARP) >> 1, ct = ((warp - C::CONV_WARP) & 1) * 32 + lane;
      const int oct = ct >> 3, pair = HD == 128 ? oct >> 1 : oct & 3, c = (lane & 3) + (HD == 128 ? (oct & 1) * 4 : 0);
      const int r0 = (lane & 4 ? pair ^ 5 : pair) + (HD == 128 ? 0 : (oct >> 2) * 8);
      // the lanes of this thread's rows
      const unsigned row_lanes = HD == 128 ? 0x0f0fu << ((lane & 16) + (lane & 4)) : 0xfu << (lane & 28);
      const uint8_t* src = sp + C::RING + sw_at<HD>(r0, c);
      uint8_t* dst = sp + (h ? C::V : C::K) + (c >> 2) * (TM_PT * 128) + r0 * 128;
      const uint32_t x0 = ((2 * (c & 3)) ^ (r0 & 7)) << 4, x1 = ((2 * (c & 3) + 1) ^ (r0 & 7)) << 4;
      unsigned long long* const to_full = h ? ctl.v_full : ctl.k_full;
      unsigned long long* const to_empty = h ? ctl.v_empty : ctl.k_empty;
      for (int i = 0; i < m.nt; ++i) {
        const int b = i & 1, p0 = (m.t0 + i) * TM_PT, it = 2 * i + h, slot = it % C::S;
        ok = kv8_wait(su32(&ctl.full[slot]), (uint32_t)(it / C::S) & 1u, abort_w, status) &&
             kv8_wait(su32(&to_empty[b]), ((uint32_t)(i >> 1) & 1u) ^ 1u, abort_w, status) &&
             (!h || kv8_wait(su32(&ctl.pw_full[i & 3]), (uint32_t)(i >> 2) & 1u, abort_w, status)) &&
             (i != 1 || kv8_wait(su32(&ctl.q_full), 0u, abort_w, status));  // (the queries passed through its place)
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        bool some = false;
        if (h) {
          const uint4 z = *reinterpret_cast<const uint4*>(ctl.none[i & 3]);
          some = p0 + TM_PT > m.t.L || (z.x | z.y | z.z | z.w);  // (an edge tile: it reaches past the committed positions)
        }
#pragma unroll 1
        for (int u0 = 0; u0 < ROWS; u0 += U) {
          uint4 x[U];
#pragma unroll
          for (int u = 0; u < U; ++u) x[u] = *reinterpret_cast<const uint4*>(src + slot * C::SLOT + (u0 + u) * (RPI * HD));
          if (some) {
            // the value row of a position no row may meet is zeroed: one behind the last that is
            // seen (whatever lies there), or a new row's with a NaN
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int r = r0 + (u0 + u) * RPI, pos = p0 + r;
              const uint32_t bits = ((x[u].x & 0x7f7f7f7fu) + 0x01010101u) | ((x[u].y & 0x7f7f7f7fu) + 0x01010101u) |
                                    ((x[u].z & 0x7f7f7f7fu) + 0x01010101u) | ((x[u].w & 0x7f7f7f7fu) + 0x01010101u);
              const bool nan = (__ballot_sync(0xffffffffu, (bits & 0x80808080u) != 0) & row_lanes) != 0 && pos >= m.t.L && pos < m.end;
              if (nan || ((ctl.none[i & 3][r >> 5] >> (r & 31)) & 1u)) x[u] = make_uint4(0, 0, 0, 0);
              if (nan && c == 0) atomicOr(&ctl.bad[i & 3][r >> 5], 1u << (r & 31));
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint2 h0 = codes_half(x[u].x), h1 = codes_half(x[u].y), h2 = codes_half(x[u].z), h3 = codes_half(x[u].w);
            uint8_t* row = dst + b * C::TILE + (u0 + u) * (RPI * 128);
            *reinterpret_cast<uint4*>(row + x0) = make_uint4(h0.x, h0.y, h1.x, h1.y);
            *reinterpret_cast<uint4*>(row + x1) = make_uint4(h2.x, h2.y, h3.x, h3.y);
          }
        }
        mbar_arrive(su32(&ctl.empty[slot]));
        proxy_fence();
        mbar_arrive(su32(&to_full[b]));
        if (h) {
          mbar_arrive(su32(&ctl.bad_full[i & 3]));
          mbar_arrive(su32(&ctl.pw_empty[i & 3]));
        }
      }
    } else if (warp >= C::SUM_WARP) {
      // ---- outputs: group wg adds up elements wg HD / 2 .. of the rows
      constexpr int HW = HD / 2;
      const int wg = (warp - C::SUM_WARP) >> 2, r = tid & 127;
      const uint32_t src = tmem + C::TM_O + wg * HW + ((uint32_t)((warp & 3) * 32) << 16);
      float base = TM_FLOOR;  // what the sums are relative to: no tile's base is more than 2^10 above
      float2 o[HW / 2];
#pragma unroll
      for (int n = 0; n < HW / 2; ++n) o[n] = make_float2(0.f, 0.f);
      for (int t = 0; t < m.nt; ++t) {
        ok = kv8_wait(su32(&ctl.o_full), (uint32_t)t & 1u, abort_w, status) &&
             kv8_wait(su32(&ctl.base_full[t & 3]), (uint32_t)(t >> 2) & 1u, abort_w, status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float nb = ctl.bases[t & 3][r];
        const bool rises = nb - base > 10.f;
        if (__any_sync(0xffffffffu, rises)) {
          const float corr = rises ? exp2_fast(base - nb) : 1.f;
          if (rises) base = nb;
#pragma unroll
          for (int n = 0; n < HW / 2; ++n) o[n] = make_float2(o[n].x * corr, o[n].y * corr);
        }
        const float f = exp2_fast(nb - base);  // (whole numbers: exact)
#pragma unroll
        for (int n = 0; n < HW; n += 8) {
          uint32_t x[8];
          tmem_ld8u(src + n, x);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int e = 0; e < 8; e += 2)
            o[(n + e) / 2] = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(f, f), o[(n + e) / 2]);
        }
        tc_fence_before();
        mbar_arrive(su32(&ctl.o_free));
      }
      if (!ok) *abort_w = 1;
      if (wg == 0) ctl.base[r] = base;
#pragma unroll
      for (int n = 0; n < HW; n += 4)
        *reinterpret_cast<float4*>(os + r * C::LD + wg * HW + n) = make_float4(o[n / 2].x, o[n / 2].y, o[n / 2 + 1].x, o[n / 2 + 1].y);
    } else {
      // ---- softmax: group wg has the tiles of its parity, a thread a row
      take_registers();
      constexpr int HW = HD / 2;  // elements of its query that a thread brings in
      const int wg = warp >> 2, r = tid & 127;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const int row = m.n0 + r, node = kv8_div(min(row, m.n0 + m.rows - 1), rep, d.rep_inv);
      float qs;
      {
        // the queries, scaled to 2^14 .. 2^15, go to tensor memory, a lane a row, by way of shared
        // memory: a warp reads whole rows (a lane its own row: 3.5 us more).  Their place is that of
        // the odd tiles, whose conversion waits for it.
        // All its rows are on their way at once; half of them at a time are converted (unrolled over all,
        // fetching the instructions took longer).
        constexpr int LPR = HD / 4, RPW = 32 / LPR, ALL = KW_ROWS / (KW_SOFT / 32) / RPW, U = ALL / 2;
        const int sub = lane / LPR, e = lane % LPR * 4, last = m.n0 + m.rows - 1;
        const T* q0 = static_cast<const T*>(a.q) + (size_t)m.t.row0 * a.ldq + (size_t)m.g * rep * HD + e;
        float4 x[U], next[U];
#pragma unroll
        for (int u = 0; u < ALL; ++u) {
          const int at = min(m.n0 + (warp * ALL + u) * RPW + sub, last), of = kv8_div(at, rep, d.rep_inv);
          (u < U ? x[u % U] : next[u % U]) = q4(q0 + (size_t)of * a.ldq + (at - of * rep) * HD, d.vec & 1);
        }
#pragma unroll 1
        for (int u0 = 0; u0 < ALL; u0 += U) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int at = (warp * ALL + u0 + u) * RPW + sub;
            uint32_t top = max(max(__float_as_uint(x[u].x) & 0x7fffffffu, __float_as_uint(x[u].y) & 0x7fffffffu),
                               max(__float_as_uint(x[u].z) & 0x7fffffffu, __float_as_uint(x[u].w) & 0x7fffffffu));
            top = __reduce_max_sync(LPR == 32 ? 0xffffffffu : 0xffffu << (16 * sub), top);
            // |q| < 2^E, of the largest and of subnormal ones: 2^(15 - E) and 2^E in two factors; of its inverse the
            // keys' powers have 2^-15 (large keys meet small queries, and the reverse)
            const int E = min(max((int)(top >> 23) - 126, -125), 128), half = (15 - E) >> 1;
            // (a row with an infinity or NaN becomes NaN: an infinity's scores might all be -inf, as if it saw nothing)
            const float by = top >= 0x7f800000u ? __int_as_float(0x7fc00000) : __int_as_float((127 + 15 - E - half) << 23);
            const float by1 = __int_as_float((127 + half) << 23);
            if (lane % LPR == 0) ctl.sum[at] = 2.f * 1.4426950408889634f / sqrtf((float)HD) * __int_as_float((126 + E) << 23);
            float v[4] = {x[u].x * by * by1, x[u].y * by * by1, x[u].z * by * by1, x[u].w * by * by1};
#pragma unroll
            for (int term = 0; term < C::TERMS; ++term) {
              const uint2 w = make_uint2(pack_half(v[0], v[1]), pack_half(v[2], v[3]));
              *reinterpret_cast<uint2*>(sp + (term ? C::V : C::K) + C::TILE + at * (HD * 2) + (((e >> 3) ^ (at & 7)) << 4) + (e & 4) * 2) = w;
              const float2 h0 = unpack_half(w.x), h1 = unpack_half(w.y);
              v[0] -= h0.x;
              v[1] -= h0.y;
              v[2] -= h1.x;
              v[3] -= h1.y;
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) x[u] = next[u];
        }
        kw_vote(false, 1);
        qs = ctl.sum[r];
#pragma unroll
        for (int term = 0; term < C::TERMS; ++term)
#pragma unroll
          for (int c0 = 0; c0 < HW / 8; c0 += 4) {
            uint32_t w[16];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              *reinterpret_cast<uint4*>(w + 4 * c) = *reinterpret_cast<const uint4*>(
                  sp + (term ? C::V : C::K) + C::TILE + r * (HD * 2) + (((wg * (HW / 8) + c0 + c) ^ (r & 7)) << 4));
            tmem_st16u(tmem + C::TM_Q + term * C::TM_QT + wg * (HW / 2) + c0 * 4 + lanes, w);
          }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        mbar_arrive(su32(&ctl.q_full));
      }
      // what the row sees of the new rows
      unsigned long long mask = a.masks && r < m.rows ? a.masks[m.t.row0 + node] : 0ull;
      if (m.t.n < 64) mask &= (1ull << m.t.n) - 1;
      float base = TM_FLOOR, l = 0.f;  // the row's base and sum of weights, without the values' powers
      for (int t = wg; t < m.nt; t += 2) {
        const int p0 = (m.t0 + t) * TM_PT;
        ok = kv8_wait(su32(&ctl.s_full[wg]), (uint32_t)(t >> 1) & 1u, abort_w, status) &&
             kv8_wait(su32(&ctl.pw_full[t & 3]), (uint32_t)(t >> 2) & 1u, abort_w, status) &&
             // (a tile that reaches past the committed positions: its values' bits)
             (p0 + TM_PT <= m.t.L || kv8_wait(su32(&ctl.bad_full[t & 3]), (uint32_t)(t >> 2) & 1u, abort_w, status));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t src = tmem + wg * 128 + lanes;
        const float4* pw = ctl.power[t & 3];
        // The tile in chunks of 32 positions.  Weights are 2^(score + power - base); without the
        // power they join the sum.
        constexpr int CK = 32;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
        for (int ch = 0; ch < TM_PT / CK; ++ch) {
          float x[CK], most[2];  // (blocks of 16 positions or more: the largest score of each 16, found by the load)
          if constexpr (GRAN == 16) {
            tmem_ld16_max<0>(src + CK * ch, x, most[0]);
            tmem_ld16_max<16>(src + CK * ch + 16, x, most[1]);
          } else {
            tmem_ld32f(src + CK * ch, x);
          }
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
          const int dd = p0 + CK * ch - m.t.L;  // its first position, counted from the first new row
          if (dd > -CK) {
            // -inf where the row does not see the position, NaN where a value that it sees is
            uint32_t sees;
            if (a.masks) {
              sees = dd >= 64 ? 0u : dd >= 0 ? (uint32_t)(mask >> dd) : (uint32_t)(mask << -dd) | ((1u << -dd) - 1);
            } else {
              const int n = node + 1 - dd;
              sees = n >= CK ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
            }
            const uint32_t nan = ctl.bad[t & 3][ch];
#pragma unroll
            for (int e = 0; e < CK; ++e)
              x[e] = !((sees >> e) & 1u) ? -INFINITY : (nan >> e) & 1u ? __uint_as_float(0x7fc00000u) : x[e];
            if constexpr (GRAN == 16) {
              most[0] = most[1] = -INFINITY;
#pragma unroll
              for (int e = 0; e < CK; ++e) most[e / 16] = fmaxf(most[e / 16], x[e]);
            }
          }
          const float4* pc = pw + CK / GRAN * ch;
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < CK; e += GRAN) {
            float mx = x[e];
            if constexpr (GRAN == 16) {
              mx = most[e / 16];
            } else {
#pragma unroll
              for (int f = 1; f < GRAN; ++f) mx = fmaxf(mx, x[e + f]);
            }
            top = fmaxf(top, fmaf(mx, fmaxf(pc[e / GRAN].x * qs, KW_TINY), pc[e / GRAN].y));
          }
          const bool rises = top - base > KW_MOST;
          if (__any_sync(0xffffffffu, rises)) {
            // a new base: the tile's weights so far are scaled to it (by powers of two)
            const float nb = rises ? ceilf(top) - KW_BASE : base, corr = exp2_fast(base - nb);
            base = nb;
            l *= corr;
            sum[0] = make_float2(sum[0].x * corr, sum[0].y * corr);
            sum[1] = make_float2(sum[1].x * corr, sum[1].y * corr);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
#pragma unroll 1
            for (int col = 0; col < CK * ch; col += 8) {
              // (of each 16 columns the first term has eight, the second, if there is one, the others)
              if (C::TERMS == 1 && (col & 8)) continue;
              uint32_t w[8];
              tmem_ld8u(src + col, w);
              asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 v = unpack_half(w[e]);
                w[e] = pack_half(v.x * corr, v.y * corr);
              }
              tmem_st8u(src + col, w);
            }
          }
#pragma unroll
          for (int e = 0; e < CK; e += GRAN) {
            const float4 p = pc[e / GRAN];
            const float kq = fmaxf(p.x * qs, KW_TINY), nb = p.y - base;
            if constexpr (GRAN == 1) {
              x[e] = exp2_fast(fmaf(x[e], kq, nb));
              sum[0].x = fmaf(x[e], p.z, sum[0].x);
            } else {
              float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
              for (int f = 0; f < GRAN; f += 2) {
                const float2 v = fma2(make_float2(x[e + f], x[e + f + 1]), make_float2(kq, kq), make_float2(nb, nb));
                x[e + f] = exp2_fast(v.x);
                x[e + f + 1] = exp2_fast(v.y);
                part[(f >> 1) & 1] = add2(part[(f >> 1) & 1], make_float2(x[e + f], x[e + f + 1]));
              }
              sum[0] = fma2(add2(part[0], part[1]), make_float2(p.z, p.z), sum[0]);
            }
          }
#pragma unroll
          for (int q = 0; q < CK; q += 16) {
            uint32_t w[8];
            if constexpr (C::TERMS == 2) {
              // the upper 11 bits, and what is left of the weight
              float2 lo[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float2 v = make_float2(x[q + 2 * e], x[q + 2 * e + 1]);
                const float2 hi = make_float2(__uint_as_float(__float_as_uint(v.x) & 0xffffe000u), __uint_as_float(__float_as_uint(v.y) & 0xffffe000u));
                w[e] = pack_half(hi.x, hi.y);
                lo[e] = fma2(hi, make_float2(-1.f, -1.f), v);
              }
              tmem_st8u(src + CK * ch + q, w);
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = pack_half(lo[e].x, lo[e].y);
              tmem_st8u(src + CK * ch + q + 8, w);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = pack_half(x[q + 2 * e], x[q + 2 * e + 1]);
              tmem_st8u(src + CK * ch + q, w);
            }
          }
        }
        sum[0] = add2(sum[0], sum[1]);
        ctl.bases[t & 3][r] = base;
        mbar_arrive(su32(&ctl.base_full[t & 3]));
        // (the running sum takes a tile's at a time: its own roundings stay few)
        l += sum[0].x + sum[0].y;
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
        mbar_arrive(su32(&ctl.p_full[wg]));
        mbar_arrive(su32(&ctl.pw_empty[t & 3]));
      }
      if (!ok) *abort_w = 1;
      ctl.end[wg][0][r] = base;
      ctl.end[wg][1][r] = l;
    }
  } else if (have && tid < KW_ROWS) {
    ctl.base[tid] = TM_FLOOR;
    ctl.sum[tid] = 0.f;
  }
  __syncthreads();
  if (m.nt > 0 && tid < KW_ROWS)
    ctl.sum[tid] = ctl.end[0][1][tid] * exp2_fast(ctl.end[0][0][tid] - ctl.base[tid]) + ctl.end[1][1][tid] * exp2_fast(ctl.end[1][0][tid] - ctl.base[tid]);
  // the shares of an item are joined: what each counts for, then every CL-th row
  if (CL > 1)
    cl.sync();
  else
    __syncthreads();
  if (have && CL == 1) {
    if (tid < KW_ROWS) ctl.fac[0][tid] = ctl.sum[tid] == 0.f ? 0.f : 1.f / ctl.sum[tid];
  } else if (have && tid < KW_ROWS) {
    float bs[8], sm[8], mx = TM_FLOOR, all = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      bs[s] = s < CL ? *cl.map_shared_rank(&ctl.base[tid], s) : TM_FLOOR;
      sm[s] = s < CL ? *cl.map_shared_rank(&ctl.sum[tid], s) : 0.f;
      mx = fmaxf(mx, bs[s]);
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      bs[s] = sm[s] == 0.f ? 0.f : exp2_fast(bs[s] - mx);  // 0: the share saw nothing
      all = fmaf(sm[s], bs[s], all);
    }
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < CL) ctl.fac[s][tid] = all == 0.f ? 0.f : bs[s] / all;
  }
  __syncthreads();
  if (have && !*abort_w) {
    constexpr int LPR = HD / 4, RPI = C::THREADS / LPR, U = 2;  // lanes of a row, rows at a time, loads on their way
    const int e = tid % LPR * 4;
    T* out = static_cast<T*>(a.out) + (size_t)m.t.row0 * a.ldo + (size_t)m.g * rep * HD + e;
    for (int n0 = rank + CL * (tid / LPR); n0 < m.rows; n0 += CL * RPI * U) {
      float4 sum[U];
#pragma unroll
      for (int u = 0; u < U; ++u) sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s = 0; s < CL; ++s) {
        const float* from = CL > 1 ? cl.map_shared_rank(os, s) : os;
        float4 v[U];
        float f[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int n = min(n0 + u * CL * RPI, m.rows - 1);
          f[u] = ctl.fac[s][n];
          v[u] = *reinterpret_cast<const float4*>(from + n * C::LD + e);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (f[u] != 0.f)  // 0: a share without tiles wrote no output
            sum[u] = make_float4(fmaf(v[u].x, f[u], sum[u].x), fmaf(v[u].y, f[u], sum[u].y), fmaf(v[u].z, f[u], sum[u].z), fmaf(v[u].w, f[u], sum[u].w));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int n = n0 + u * CL * RPI;
        if (n >= m.rows) break;
        const int row = m.n0 + n, node = kv8_div(row, rep, d.rep_inv);
        store4(out + (size_t)node * a.ldo + (size_t)(row - node * rep) * HD, sum[u], d.vec & 2);
      }
    }
  }
  if (CL > 1) cl.sync();  // the others may still read this CTA's shared memory
  tc_fence_before();
  __syncthreads();
  if (*abort_w) {  // what is on its way lands first
    if (TMA && (warp == C::LOAD_WARP || warp == C::LOAD_WARP + 1)) {
      const long long c0 = clock64();
      for (int it = max(warp - C::LOAD_WARP, issued - C::S + 1); it < issued; it += 2)
        while (!mbar_try_wait(su32(&ctl.full[it % C::S]), (uint32_t)(it / C::S) & 1u) && clock64() - c0 < TM_LAND_CYCLES) {
        }
    }
    if (warp == C::MMA_WARP && elect_one()) land_products(su32(&ctl.done));
    __syncwarp();
  }
  if (warp == C::MMA_WARP) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

template <class T, int HD, int GRAN, bool TMA>
int launch_wide(const Kv8AttnArgs& a, int layers, int dev, cudaStream_t s) {
  using C = KwCfg<T, HD>;
  static TmKernel known[kMaxDevices];
  return launch_tiles(kv8_wide_kernel<T, HD, GRAN, TMA>, known[dev], C::THREADS, C::SMEM, TMA, KW_ROWS, 4 * sizeof(T), a, layers, s);
}

template <class T, int HD>
int launch_wide_of(const Kv8AttnArgs& a, int layers, bool tma, int dev, cudaStream_t s) {
  if (a.c.block % 16 == 0) return tma ? launch_wide<T, HD, 16, true>(a, layers, dev, s) : launch_wide<T, HD, 16, false>(a, layers, dev, s);
  if (a.c.block % 4 == 0) return tma ? launch_wide<T, HD, 4, true>(a, layers, dev, s) : launch_wide<T, HD, 4, false>(a, layers, dev, s);
  return tma ? launch_wide<T, HD, 1, true>(a, layers, dev, s) : launch_wide<T, HD, 1, false>(a, layers, dev, s);
}

}  // namespace

int launch_kv8_wide(const Kv8AttnArgs& a, int layers, int dtype, bool tma, int dev, cudaStream_t s) {
  if (dtype == Q3TTS_F32) return a.c.hd == 128 ? launch_wide_of<float, 128>(a, layers, tma, dev, s) : launch_wide_of<float, 64>(a, layers, tma, dev, s);
  return a.c.hd == 128 ? launch_wide_of<bf16, 128>(a, layers, tma, dev, s) : launch_wide_of<bf16, 64>(a, layers, tma, dev, s);
}

}  // namespace q3

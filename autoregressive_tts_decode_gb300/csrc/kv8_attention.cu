// kv8_attention.cu -- attention of few new rows over the 8-bit cache (decode steps,
// small drafted trees), on the 5th-generation tensor cores.
//
// For row i of a sequence and head h of kv head g, with p over the positions it sees,
//   s_p = 2^(a_p) q . c_p / sqrt(hd),  o = sum_p 2^(s_p') 2^(b_p) d_p / sum_p 2^(s_p'),  s' = log2(e) s - m,
// c_p and d_p the E4M3 codes of key and value, 2^(a_p) and 2^(b_p) their blocks' powers; o = 0
// when it sees none.
//
// Codes go from the cache to the tensor cores as they lie (kind::f8f6f4): no element
// is converted, and shared memory holds 8 bits of each.  The other operand has to be
// E4M3 too, and is: the codes 0 .. 15 of E4M3 (its subnormals and first binade) are the
// whole numbers 0 .. 15 times 2^-9.  A query row, scaled to 32-bit whole numbers by its
// largest element, and a row's weights as 32-bit fixed-point numbers are each eight hexadecimal digits,
// eight rows of the MMA's N side; the eight products are added in fp32 registers:
//   S^T = K Q^T   M 128 positions, N 8 digits x R rows, K the head dimension;
//   O^T = V^T W^T M the head dimension, N the same, K 128 positions (V read as it lies, M-major).
// The products are exact and the tensor cores keep 25 bits below the largest of a sum.
//
// The weights carry the values' powers: W = 2^(c s_p - base + b_p), where a row's base is its
// largest c s_p + b_p so far.  It is followed only when a weight passes 2^3: weights up to 2^4
// have a step of 2^-28, and a tile needs one vote of the softmax threads instead of
// a maximum over them.  The sum of 2^(c s_p - base) is held beside it in fp32.
//
// A CTA has one item: a sequence, a kv head, up to R = 2, 4, 8 or 16 rows, and with few items in a call
// a share of the positions, joined in a cluster.  One warp loads, one thread issues the MMAs, four warps
// are the softmax (a thread a position of the tile, and an element of the output).  Scores, weights and
// outputs of a tile follow one another; what overlaps are the CTAs of an SM, four for two rows, whose
// rings of three tiles keep 192 KB on their way.  Sequences are taken longest first, so that the
// last ones to start are short.
//
// The bound is the cache's bytes: 128 sequences of 256 .. 2048 positions, one token of 16 heads over 8: 54 us,
// 5.7 TB/s (loading alone 50; three CTAs with rings of four 59.6).  Short calls are latency, the chain from
// lengths to pages to codes and a tile's way: 131 positions 6 us, 16 sequences of 32 .. 512 9 us.  More rows cost
// their digits: 128 x 1152 positions, 2, 4, 8 new rows of two heads: 68, 85, 132 us.
#include "kv8_tiles.cuh"

namespace q3 {

namespace {

constexpr int KF_DIGITS = 8;
constexpr float KF_SLACK = 8.f;         // how large a weight may be
constexpr float KF_STEP = 268435456.f;  // 2^28: its fixed-point step

template <int HD, int R>
struct KfCfg {
  static constexpr int LOAD_WARP = 4, MMA_WARP = 5, THREADS = 192;
  static constexpr int N = KF_DIGITS * R;
  static constexpr uint32_t SLOT = TM_PT * HD;  // a K or V tile
  static constexpr uint32_t Q = 0, P = N * HD, RING = P + N * TM_PT;
  static constexpr int S = (R <= 8 ? 3 : 4) * (128 / HD);  // tiles in the ring
  static constexpr uint32_t CTL = RING + S * SLOT, CTL_BYTES = 2048;
  static constexpr uint32_t TMEM_COLS = 2 * N < 32 ? 32 : 2 * N;  // scores, outputs
  // A CTA's share of an SM's 512 columns of tensor memory is never larger than its share of the
  // 228 KB of shared memory (each with 1 KB of the system's), so that what fits there has its columns too.
  static constexpr size_t NEEDS = 1024 + CTL + CTL_BYTES, SHARE = TMEM_COLS * 456 - 1024;
  static constexpr size_t SMEM = NEEDS < SHARE ? SHARE : NEEDS;
  static_assert(SMEM <= 227 * 1024 && R * HD * 4 <= S * SLOT, "shared memory");
};

template <int R, int S>
struct KfCtl {
  unsigned long long full[S], empty[S], s_full, p_full, o_full, q_full, done;
  uint32_t tmem;
  int abort_w[2];  // given up, limit of the waits
  int seq;
  float qscale[R];
  float base[R], corr[R], sum[R];
  float part[4][R];
  unsigned bad[4];
  unsigned long long mask[R];
  float fac[8][R];
};

// kind::f8f6f4: D fp32, A and B E4M3, B K-major; A K-major or M-major (bit 15).
__host__ __device__ constexpr uint32_t f8_idesc(int M, int N, bool a_m_major) {
  return (1u << 4) | (a_m_major ? 1u << 15 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t tmem_d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(
          tmem_d),
      "l"(a), "l"(b), "r"(idesc), "r"(accum)
      : "memory");
}
__device__ __forceinline__ bool kf_vote(bool p) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"((uint32_t)p)
      : "memory");
  return r != 0;
}

template <class T, int HD, int R, bool TMA>
__global__ void __launch_bounds__(KfCfg<HD, R>::THREADS)
    kv8_few_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Kv8AttnArgs a, const KfDeal d) {
  using C = KfCfg<HD, R>;
  using Ctl = KfCtl<R, C::S>;
  static_assert(sizeof(Ctl) + 512 <= C::CTL_BYTES, "control block (and what an MMA of 64 rows reads behind the ring)");
  extern __shared__ uint8_t kf_raw[];
  const uint32_t raw = su32(kf_raw), sbase = (raw + 1023u) & ~1023u;
  uint8_t* sp = kf_raw + (sbase - raw);
  Ctl& ctl = *reinterpret_cast<Ctl*>(sp + C::CTL + 512);
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
      mbar_init(su32(&ctl.empty[i]), 1);
    }
    mbar_init(su32(&ctl.s_full), 1);
    mbar_init(su32(&ctl.p_full), 128);
    mbar_init(su32(&ctl.o_full), 1);
    mbar_init(su32(&ctl.q_full), 128);
    mbar_init(su32(&ctl.done), 1);
    ctl.abort_w[0] = 0;
    ctl.abort_w[1] = d.wait_1024;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_wait();  // q and the rows written to the cache come from the previous kernels
  pdl_trigger();
  // (tensor memory after the wait: a kernel before may still be about to take its own)
  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(su32(&ctl.tmem)),
                 "r"(C::TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  KfItem m;
  const int wanted = first_item(a, d, CL, R, m);
  if (d.sorted) find_sequence<C::THREADS>(a.r, wanted, reinterpret_cast<int*>(sp), &ctl.seq);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  m.seq = d.sorted ? ctl.seq : wanted;
  const uint32_t tmem = __shfl_sync(0xffffffffu, ctl.tmem, 0);
  const uint32_t ring = sbase + C::RING;
  const bool have = take_item(a, d, CL, rank, R, m);
  bool ok = true;
  int issued = 0;  // tiles that the loading warp has filled or is filling

  if (m.nt > 0) {
    if (warp == C::LOAD_WARP) {
      ok = load_tiles<HD, C::S, TMA, false>(&map, a, m, d.box, ring, ctl.full, ctl.empty, 0, issued, abort_w);
    } else if (warp == C::MMA_WARP) {
      if (elect_one()) {
        constexpr uint32_t idS = f8_idesc(TM_PT, C::N, false), idO = f8_idesc(TM_PT, C::N, true);
        const int lost = blockIdx.x == 0 ? d.lost_tile : -1;
        auto wait = [&](unsigned long long* bar, int phase) { return kv8_wait(su32(bar), (uint32_t)phase & 1u, abort_w, status); };
        auto scores = [&](int i) -> bool {
          const int it = 2 * i, slot = it % C::S;
          if (i == lost || !wait(&ctl.full[slot], it / C::S)) return false;
          tc_fence_after();
          const uint64_t dk = sw_desc<HD>(ring + slot * C::SLOT), dqd = sw_desc<HD>(sbase + C::Q);
#pragma unroll
          for (int s = 0; s < HD / 32; ++s) mma_f8(tmem, dk + s * 2, dqd + s * 2, idS, s != 0);
          mma_commit(su32(&ctl.empty[slot]));
          mma_commit(su32(&ctl.s_full));
          return true;
        };
        ok = wait(&ctl.q_full, 0) && scores(0);
        for (int i = 0; i < m.nt && ok; ++i) {
          const int it = 2 * i + 1, slot = it % C::S;
          ok = wait(&ctl.full[slot], it / C::S) && wait(&ctl.p_full, i);
          if (!ok) break;
          tc_fence_after();
          // (a head dimension of 64 fills half of M: the other half's results are not used)
          const uint64_t dv = sw_desc<HD>(ring + slot * C::SLOT, 512), dp = sw_desc<128>(sbase + C::P);
#pragma unroll
          for (int s = 0; s < TM_PT / 32; ++s) mma_f8(tmem + C::N, dv + (s * 32 * HD >> 4), dp + s * 2, idO, s != 0);
          mma_commit(su32(&ctl.empty[slot]));
          mma_commit(su32(&ctl.o_full));
          if (i + 1 < m.nt) ok = scores(i + 1);
        }
      }
      __syncwarp();
    } else {
      // ---- softmax: a thread has a position of the tile and an element of the output
      const uint32_t lanes = (uint32_t)(warp * 32) << 16;
      Powers<1> pw(a, d, m, tid);
      // the queries' digits: a warp a row, magnitudes as 32-bit whole numbers with the sign in each digit
      for (int r = warp; r < R; r += 4) {
        constexpr int EPL = 4, LPR = HD / EPL;  // (a head dimension of 64: half of the lanes)
        const int row = m.n0 + min(r, m.rows - 1), node = kv8_div(row, rep, d.rep_inv);
        const T* q = static_cast<const T*>(a.q) + (size_t)(m.t.row0 + node) * a.ldq + (size_t)(m.g * rep + row - node * rep) * HD;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (lane < LPR) x = q4(q + lane * EPL, d.vec & 1);
        const float f[4] = {x.x, x.y, x.z, x.w};
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
        top = __reduce_max_sync(0xffffffffu, top);
        // |q| < 2^E, of the largest and of subnormal ones: 2^(32 - E) and, below, 2^E in two factors
        const int E = min(max((int)(top >> 23) - 126, -125), 128), half = (32 - E) >> 1;
        const float by0 = __int_as_float((127 + 32 - E - half) << 23), by1 = __int_as_float((127 + half) << 23);
        uint32_t ev[4], od[4], sg[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t u;
          asm("cvt.rni.u32.f32 %0, %1;" : "=r"(u) : "f"(fabsf(f[e]) * by1 * by0));
          ev[e] = u & 0x0f0f0f0fu;
          od[e] = (u >> 4) & 0x0f0f0f0fu;
          sg[e] = __float_as_uint(f[e]) >> 31 << 7;
        }
        const uint32_t sign = sg[0] | sg[1] << 8 | sg[2] << 16 | sg[3] << 24;
        if (lane < LPR) {
#pragma unroll
          for (int nib = 0; nib < 8; ++nib) {
            const uint32_t* v = nib & 1 ? od : ev;
            const int sh = nib / 2 * 8;
            const uint32_t w = ((v[0] >> sh) & 15u) | ((v[1] >> sh) & 15u) << 8 | ((v[2] >> sh) & 15u) << 16 | ((v[3] >> sh) & 15u) << 24;
            *reinterpret_cast<uint32_t*>(sp + C::Q + sw_at<HD>(r * 8 + nib, lane >> 2) + (lane & 3) * 4) = w | sign;
          }
        }
        if (lane == 0) {
          // q is its digits' sum (the top one whole, codes for 2^-9 of a digit) x 2^(E - 32 + 28 + 9), of which the
          // sum takes 2^5.  Infinities and NaN, which have no digits: NaN, and with it every score that the row sees
          ctl.qscale[r] = top >= 0x7f800000u ? __int_as_float(0x7fc00000)
                                             : 2.f * 1.4426950408889634f / sqrtf((float)HD) * __int_as_float((126 + E) << 23);
          ctl.mask[r] = r >= m.rows ? 0ull : a.masks ? a.masks[m.t.row0 + node] : 0ull;
          ctl.base[r] = TM_FLOOR;
        }
      }
      proxy_fence();
      mbar_arrive(su32(&ctl.q_full));
      kf_vote(false);  // scales, masks and bases are there
      float l[R], o[R];
#pragma unroll
      for (int r = 0; r < R; ++r) l[r] = o[r] = 0.f;
      uint32_t pat[8];  // this position's byte of the eight digits of row 0
#pragma unroll
      for (int nib = 0; nib < 8; ++nib) pat[nib] = sbase + C::P + sw_at<128>(nib, tid >> 4) + (tid & 15);
      for (int i = 0; i < m.nt; ++i) {
        const int pos = (m.t0 + i) * TM_PT + tid, j = pos - m.t.L;
        const float kf = kv8_power(pw.k[0]), vf = kv8_power(pw.v[0]), eb = (float)min(max(pw.v[0] - 127, -KV8_EXP), KV8_EXP);
        pw.next(a, d, m, i, tid);
        const float vl = fmaxf(vf, kv8_power(127 - KV8_EXP));  // as in eb: weights of values below it stay in range too
        bool isbad = false;
        const bool edge = (m.t0 + i + 1) * TM_PT > m.t.L;  // the tile reaches past the committed positions
        if (edge) {
          // the value row of a position no row may meet is zeroed: one behind the last that
          // is seen (whatever lies there), or a new row's with a NaN
          const int it = 2 * i + 1;
          ok = kv8_wait(su32(&ctl.full[it % C::S]), (uint32_t)(it / C::S) & 1u, abort_w, status) && ok;
          uint8_t* vr = sp + C::RING + it % C::S * C::SLOT;
          if (ok && j >= 0 && pos < m.end) {
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < HD / 16; ++e) {
              const uint4 u = *reinterpret_cast<const uint4*>(vr + sw_at<HD>(tid, e));
              bits |= ((u.x & 0x7f7f7f7fu) + 0x01010101u) | ((u.y & 0x7f7f7f7fu) + 0x01010101u) |
                      ((u.z & 0x7f7f7f7fu) + 0x01010101u) | ((u.w & 0x7f7f7f7fu) + 0x01010101u);
            }
            isbad = (bits & 0x80808080u) != 0 || vf != vf;
          }
          if (ok && (isbad || pos >= m.end)) {
#pragma unroll
            for (int e = 0; e < HD / 16; ++e) *reinterpret_cast<uint4*>(vr + sw_at<HD>(tid, e)) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        ok = kv8_wait(su32(&ctl.s_full), (uint32_t)i & 1u, abort_w, status) && ok;
        __syncwarp();
        tc_fence_after();
        // scores in units of log2; -inf where the row does not see the position
        float x[R];
        bool over = false;
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          uint32_t v[16];
          tmem_ld16(tmem + r * 8 + lanes, v);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s = __uint_as_float(v[8 * h]);
#pragma unroll
            for (int nib = 1; nib < 8; ++nib) s = fmaf(s, 0.0625f, __uint_as_float(v[8 * h + nib]));
            x[r + h] = s * 32.f * (kf * ctl.qscale[r + h]);  // (large keys meet small queries, and the reverse)
          }
        }
        if (edge && j >= 0) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const bool sees = pos < m.end && (a.masks ? (ctl.mask[r] >> min(j, 63)) & 1ull
                                                      : j <= kv8_div(m.n0 + r, rep, d.rep_inv));
            x[r] = !sees ? -INFINITY : isbad ? __int_as_float(0x7fc00000) : x[r];
          }
        }
        float w[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          w[r] = exp2_fast(x[r] - ctl.base[r]);
          over = over || w[r] * vl > KF_SLACK;
        }
        if (kf_vote(over || !ok)) {
          // new bases: the rows' largest score and power so far
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float top = warp_max(x[r] + eb);
            if (lane == 0) ctl.part[warp][r] = top;
          }
          if (kf_vote(!ok)) {
            ok = false;
            break;
          }
          if (tid < R) {
            const float old = ctl.base[tid];
            const float nb = fmaxf(fmaxf(fmaxf(ctl.part[0][tid], ctl.part[1][tid]), fmaxf(ctl.part[2][tid], ctl.part[3][tid])), old);
            ctl.corr[tid] = nb == old ? 1.f : exp2_fast(old - nb);
            ctl.base[tid] = nb;
          }
          kf_vote(false);
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const float corr = ctl.corr[r];
            l[r] *= corr;
            o[r] *= corr;
            w[r] = exp2_fast(x[r] - ctl.base[r]);
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          l[r] += w[r];
          uint32_t u;
          asm("cvt.rni.u32.f32 %0, %1;" : "=r"(u) : "f"(w[r] * vf * KF_STEP));
          const uint32_t ev = u & 0x0f0f0f0fu, od = (u >> 4) & 0x0f0f0f0fu;
#pragma unroll
          for (int nib = 0; nib < 8; ++nib)
            asm volatile("st.shared.u8 [%0], %1;" ::"r"(pat[nib] + r * 1024), "r"((nib & 1 ? od : ev) >> (nib / 2 * 8)) : "memory");
        }
        proxy_fence();
        tc_fence_before();
        mbar_arrive(su32(&ctl.p_full));
        // the tile's output joins the running one
        ok = kv8_wait(su32(&ctl.o_full), (uint32_t)i & 1u, abort_w, status);
        __syncwarp();
        tc_fence_after();
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          uint32_t v[16];
          tmem_ld16(tmem + C::N + r * 8 + lanes, v);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float s = __uint_as_float(v[8 * h]);
#pragma unroll
            for (int nib = 1; nib < 8; ++nib) s = fmaf(s, 0.0625f, __uint_as_float(v[8 * h + nib]));
            o[r + h] += s;
          }
        }
        tc_fence_before();
      }
      if (kf_vote(!ok)) {
        ok = false;
        *abort_w = 1;
      }
      // (the sums have the top digit whole, 16^7 steps of 2^-28, and codes for 2^-9 of a digit)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float sum = warp_sum(l[r]);
        if (lane == 0) ctl.part[warp][r] = sum;
        o[r] *= 512.f;
      }
      kf_vote(false);
      if (tid < R) ctl.sum[tid] = (ctl.part[0][tid] + ctl.part[1][tid]) + (ctl.part[2][tid] + ctl.part[3][tid]);
      kf_vote(false);
      if (CL > 1) {
        float* os = reinterpret_cast<float*>(sp + C::RING);  // (its tiles have been read)
        if (tid < HD) {
#pragma unroll
          for (int r = 0; r < R; ++r) os[r * HD + tid] = o[r];
        }
      } else if (ok && tid < HD) {
        T* out = static_cast<T*>(a.out);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          if (r >= m.rows) break;
          const int row = m.n0 + r, node = kv8_div(row, rep, d.rep_inv);
          const float sum = ctl.sum[r];
          out[(size_t)(m.t.row0 + node) * a.ldo + (size_t)(m.g * rep + row - node * rep) * HD + tid] =
              from_f<T>(sum == 0.f ? 0.f : o[r] / sum);
        }
      }
    }
  } else if (have && tid < R) {
    ctl.base[tid] = TM_FLOOR;
    ctl.sum[tid] = 0.f;
  }
  __syncwarp();
  // Tensor memory is given back before the CTA waits for the others of its cluster.  One of those may be waiting for
  // columns that a CTA of another stream's call holds (the tree attention's 32 rows at a head dimension of 64 take all columns
  // and leave room in shared memory for a CTA here), whose cluster may be waiting for the columns held here.
  tc_fence_before();
  __syncthreads();
  if (*abort_w) {  // what is on its way lands first
    if (TMA && warp == C::LOAD_WARP) {
      const long long c0 = clock64();
      for (int it = max(0, issued - C::S); it < issued; ++it)
        while (!mbar_try_wait(su32(&ctl.full[it % C::S]), (uint32_t)(it / C::S) & 1u) && clock64() - c0 < TM_LAND_CYCLES) {
        }
    }
    if (warp == C::MMA_WARP && elect_one()) land_products(su32(&ctl.done));
    __syncwarp();
  }
  if (warp == C::MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS) : "memory");
  if (CL > 1) {
    // the shares of an item are joined: what each counts for, then every CL-th row
    cl.sync();
    if (have && tid < R) {
      float bs[8], sm[8], mx = TM_FLOOR, all = 0.f;
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        bs[r] = r < CL ? *cl.map_shared_rank(&ctl.base[tid], r) : TM_FLOOR;
        sm[r] = r < CL ? *cl.map_shared_rank(&ctl.sum[tid], r) : 0.f;
        mx = fmaxf(mx, bs[r]);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        bs[r] = sm[r] == 0.f ? 0.f : exp2_fast(bs[r] - mx);  // 0: the share saw nothing
        all = fmaf(sm[r], bs[r], all);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) ctl.fac[r][tid] = all == 0.f ? 0.f : bs[r] / all;
    }
    __syncthreads();
    if (have && !*abort_w) {
      float* os = reinterpret_cast<float*>(sp + C::RING);
      T* out = static_cast<T*>(a.out);
      for (int e = tid; e < R * HD; e += C::THREADS) {
        const int r = e / HD, n = r * CL + rank;
        if (n >= m.rows) break;
        float v[8], sum = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s)  // a share without tiles wrote no output: its factor is 0
          v[s] = s < CL && ctl.fac[s][n] != 0.f ? *(cl.map_shared_rank(os, s) + n * HD + e % HD) : 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s < CL) sum = fmaf(v[s], ctl.fac[s][n], sum);
        const int row = m.n0 + n, node = kv8_div(row, rep, d.rep_inv);
        out[(size_t)(m.t.row0 + node) * a.ldo + (size_t)(m.g * rep + row - node * rep) * HD + e % HD] = from_f<T>(sum);
      }
    }
    cl.sync();  // the others may still read this CTA's shared memory
  }
}

template <class T, int HD, int R, bool TMA>
int launch_few(const Kv8AttnArgs& a, int layers, int dev, cudaStream_t s) {
  using C = KfCfg<HD, R>;
  static TmKernel known[kMaxDevices];
  return launch_tiles(kv8_few_kernel<T, HD, R, TMA>, known[dev], C::THREADS, C::SMEM, TMA, R, 4 * sizeof(T), a, layers, s);
}

template <class T, int HD, bool TMA>
int launch_few_rows(const Kv8AttnArgs& a, int layers, int dev, cudaStream_t s) {
  const long rows = (long)a.r.max_rows * (a.Hq / a.c.Hkv);
  if (rows <= 2) return launch_few<T, HD, 2, TMA>(a, layers, dev, s);
  if (rows <= 4) return launch_few<T, HD, 4, TMA>(a, layers, dev, s);
  if (rows <= 8) return launch_few<T, HD, 8, TMA>(a, layers, dev, s);
  return launch_few<T, HD, 16, TMA>(a, layers, dev, s);
}

// Whether tiles of 128 rows (kv8_wide.cu) are done sooner than tiles of 16, whose cache is read
// again for each of them.  A round of items costs about 7 us and 2.3 us for a tile of positions here,
// of two CTAs on an SM, 11 and 1.75 us there, one on an SM; positions are split in up to eight where
// that leaves one round.  8 kv heads of two q heads, fp32 (sequences x positions, new rows: us here,
// us there): 1 x 112, 32: 10.9, 14.5; 1 x 2000, 16: 13.2, 18.8; 4 x 8000, 9: 62, 40; 16 x 112, 32: 25.7, 15.5;
// 64 x 112, 9: 41, 48; 64 x 2000, 16: 179, 148; 64 x 8000, 32: 966, 447.
bool wide_pays(const Kv8AttnArgs& a, int n_sm) {
  const long rows = (long)a.r.max_rows * (a.Hq / a.c.Hkv), heads = (long)a.r.n_seqs * a.c.Hkv;
  if (rows <= 16) return false;  // one tile: the rest of a wide one would be empty
  const long tiles = ((long)a.r.pps * a.c.page + TM_PT - 1) / TM_PT;
  auto us = [&](long items, long slots, double item, double tile) {
    const long rounds = (items + slots - 1) / slots, most = slots / items < 8 ? slots / items : 8, share = rounds > 1 ? 1 : most;
    return rounds * (item + tile * ((tiles + share - 1) / share));
  };
  return us(heads * ((rows + 127) / 128), n_sm, 11, 1.75) < us(heads * ((rows + 15) / 16), 2l * n_sm, 7, 2.3);
}

template <class T>
int launch_few_of(const Kv8AttnArgs& a, int layers, bool tma, int dev, cudaStream_t s) {
  if (a.c.hd == 128) return tma ? launch_few_rows<T, 128, true>(a, layers, dev, s) : launch_few_rows<T, 128, false>(a, layers, dev, s);
  return tma ? launch_few_rows<T, 64, true>(a, layers, dev, s) : launch_few_rows<T, 64, false>(a, layers, dev, s);
}

}  // namespace

int launch_kv8_attention(const Kv8AttnArgs& a, int layers, int dtype, cudaStream_t s) {
  int dev = 0, n_sm = 0;
  if (!current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  // TMA boxes are pages of whole swizzle atoms (8 rows) that fill a tile a whole
  // number of times, or whole tiles of larger pages
  const int ps = a.c.page;
  const bool tma = (ps >= 8 && ps <= TM_PT && TM_PT % ps == 0) || ps % TM_PT == 0;
  if (wide_pays(a, n_sm)) return launch_kv8_wide(a, layers, dtype, tma, dev, s);
  return dtype == Q3TTS_F32 ? launch_few_of<float>(a, layers, tma, dev, s) : launch_few_of<bf16>(a, layers, tma, dev, s);
}

}  // namespace q3

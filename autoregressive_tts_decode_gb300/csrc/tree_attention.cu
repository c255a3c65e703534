// tree_attention.cu -- attention of drafted tree nodes over a paged cache.
//
// A sequence holds L committed positions and T drafted nodes, whose keys and
// values sit in its pages at positions L .. L + T - 1 in node order.  Node i
// sees every committed position and the nodes j of its mask (bit j of a 64-bit
// word: its ancestors and itself), so for head h of kv head g
//   s_p = q . k_p / sqrt(hd),  o = sum_p e^(s_p - m) v_p / sum_p e^(s_p - m)
// over the positions p it sees, m their largest score; o = 0 when it sees none.
// One node whose mask is its own bit is the ordinary decode of a single token,
// a chain of nodes the causal attention of a short chunk.
//
// The rows of a sequence that share a kv head are the T nodes times the q
// heads of the group (row n: node n / rep, head g rep + n % rep), so each cache
// row is read once for all of them.  A CTA takes one tile of those rows and a
// share of the positions; the CTAs of one thread-block cluster split the
// positions of the same rows and join their (max, sum, output) through
// distributed shared memory: no workspace, no counters, one launch, and the
// same result on every run.
#include <cooperative_groups.h>

#include "ops.cuh"
#include "tree.cuh"

namespace cg = cooperative_groups;

namespace q3 {

namespace {

// Element offset of (position, k|v, kv head) of a sequence; a page id outside
// the pool is reported and page 0 read in its place.
__device__ __forceinline__ size_t tree_offset(const TreeArgs& a, const int* table, int pos, int kvsel, int g) {
  const KVDesc& kv = a.kv;
  int page = table[pos / kv.page_size];
  if (page < 0 || page >= kv.n_pages) {
    op_status(a.status, Q3TTS_ERR_ARG);
    page = 0;
  }
  return ((((size_t)a.layer * kv.n_pages + page) * 2 + kvsel) * kv.Hkv + g) * kv.page_size * kv.hd +
         (size_t)(pos % kv.page_size) * kv.hd;
}

__device__ __forceinline__ bool node_sees(unsigned long long mask, int pos, int L) {
  return pos < L || ((mask >> (pos - L)) & 1ull) != 0;
}

// ------------------------------------------------------- fp32 arithmetic
//
// Any cache type, page size and head dimension 64 or 128.  Tiles of 32
// positions are copied into shared memory (cp.async, two stages), scores and
// outputs are fp32 FMAs in registers, the running maximum and sum stay in fp32.
constexpr int TF_THREADS = 128, TF_PT = 32;

template <class KT, int HD, int RT>
struct TfCfg {
  static constexpr int KLD = HD + 16 / (int)sizeof(KT);  // padded row: consecutive rows start in other banks
  static constexpr int TILE = TF_PT * KLD;               // elements of a K or V tile
  static constexpr size_t SMEM =
      sizeof(KT) * 4 * (size_t)TILE + sizeof(float) * ((size_t)RT * HD * 2 + (size_t)RT * TF_PT + 3 * RT) + 8 * RT;
};

__device__ __forceinline__ uint32_t su32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
__device__ __forceinline__ void load4(const bf16* p, float (&f)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
  f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
}

template <class KT, int HD, int RT>
__global__ void __launch_bounds__(TF_THREADS) tree_fma_kernel(TreeArgs a, int row_tiles) {
  using C = TfCfg<KT, HD, RT>;
  constexpr int CG = HD / 4, RG = TF_THREADS / CG;  // output: column groups of 4, row groups
  constexpr int OR = (RT + RG - 1) / RG;            // output rows of a thread
  constexpr int SR = (RT + 7) / 8;                  // score rows of a thread (8 row groups x 16 position pairs)
  pdl_wait();  // q and the appended keys and values come from the previous kernels
  extern __shared__ __align__(16) uint8_t tf_raw[];
  KT* kt = reinterpret_cast<KT*>(tf_raw);  // [2 stages][K | V][TILE]
  float* qs = reinterpret_cast<float*>(kt + 4 * C::TILE);  // [RT][HD]
  float* os = qs + RT * HD;                                // [RT][HD] this CTA's output
  float* ps = os + RT * HD;                                // [RT][TF_PT]
  float* mrow = ps + RT * TF_PT;                           // running max, sum, rescale factor
  float* lrow = mrow + RT;
  float* crow = lrow + RT;
  unsigned long long* mk = reinterpret_cast<unsigned long long*>(crow + RT);

  cg::cluster_group cl = cg::this_cluster();
  const int C_ = (int)cl.num_blocks(), rank = (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int item = blockIdx.x / C_;
  const int rt = item % row_tiles, g = item / row_tiles % a.kv.Hkv, seq = item / row_tiles / a.kv.Hkv;
  const int rep = a.Hq / a.kv.Hkv, n0 = rt * RT;
  TreeSeq t;
  // every CTA of the cluster sees the same entries, so all of them leave here
  if (!tree_seq(a, seq, t) || n0 >= t.T * rep) return;
  const int rows = min(RT, t.T * rep - n0);
  const float scale = 1.0f / sqrtf((float)HD);
  for (int e = tid; e < RT * HD; e += TF_THREADS) {
    const int r = e / HD, i = e % HD, n = n0 + r;
    qs[e] = r < rows ? a.q[(size_t)(t.row0 + n / rep) * a.ldq + (size_t)(g * rep + n % rep) * HD + i] * scale : 0.f;
  }
  for (int r = tid; r < RT; r += TF_THREADS) {
    mrow[r] = -INFINITY;
    lrow[r] = 0.f;
    mk[r] = r < rows ? a.masks[t.row0 + (n0 + r) / rep] : 0ull;
  }
  const int* table = a.kv.page_table + (size_t)seq * a.kv.pages_per_stream;
  const int ntiles = (t.P + TF_PT - 1) / TF_PT, per = (ntiles + C_ - 1) / C_;
  const int t0 = min(ntiles, rank * per), t1 = min(ntiles, t0 + per);

  constexpr int CH = HD * (int)sizeof(KT) / 16;  // 16-byte pieces of a row
  auto stage = [&](int tile) {
    if (tile < t1) {
      KT* dst = kt + (size_t)(tile & 1) * 2 * C::TILE;
      for (int e = tid; e < 2 * TF_PT * CH; e += TF_THREADS) {
        const int c = e % CH, r = e / CH % TF_PT, sel = e / CH / TF_PT;
        const int pos = tile * TF_PT + r;
        const bool in = pos < t.P;  // rows past the last node are zeroes (unwritten words may hold NaN)
        const KT* src = (const KT*)a.kv.pool + (in ? tree_offset(a, table, pos, sel, g) : 0) + c * (16 / sizeof(KT));
        cp_async16(su32(dst + (size_t)sel * C::TILE + r * C::KLD) + c * 16, src, in ? 16 : 0);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  float o[OR][4];
#pragma unroll
  for (int i = 0; i < OR; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  const int oc = (tid % CG) * 4, og = tid / CG;       // output columns, row group
  const int sp = (tid & 15) * 2, sg = tid >> 4;       // score positions, row group
  stage(t0);
  for (int tile = t0; tile < t1; ++tile) {
    stage(tile + 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const KT* kb = kt + (size_t)(tile & 1) * 2 * C::TILE;
    const KT* vb = kb + C::TILE;
    float sc[SR][2];
#pragma unroll
    for (int i = 0; i < SR; ++i) sc[i][0] = sc[i][1] = 0.f;
#pragma unroll 4
    for (int c = 0; c < HD; c += 4) {
      float k0[4], k1[4];
      load4(kb + sp * C::KLD + c, k0);
      load4(kb + (sp + 1) * C::KLD + c, k1);
#pragma unroll
      for (int i = 0; i < SR; ++i) {
        const float4 qv = *reinterpret_cast<const float4*>(qs + min(sg + 8 * i, RT - 1) * HD + c);
        sc[i][0] = fmaf(qv.x, k0[0], fmaf(qv.y, k0[1], fmaf(qv.z, k0[2], fmaf(qv.w, k0[3], sc[i][0]))));
        sc[i][1] = fmaf(qv.x, k1[0], fmaf(qv.y, k1[1], fmaf(qv.z, k1[2], fmaf(qv.w, k1[3], sc[i][1]))));
      }
    }
#pragma unroll
    for (int i = 0; i < SR; ++i) {
      const int r = sg + 8 * i;
      if (r < RT) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pos = tile * TF_PT + sp + e;
          ps[r * TF_PT + sp + e] = (r < rows && pos < t.P && node_sees(mk[r], pos, t.L)) ? sc[i][e] : -INFINITY;
        }
      }
    }
    __syncthreads();
    // softmax of the tile: one warp per row, one position per lane
    for (int r = warp; r < rows; r += TF_THREADS / 32) {
      const float s = ps[r * TF_PT + lane];
      const float mo = mrow[r], mn = fmaxf(mo, warp_max(s));
      const float p = s == -INFINITY ? 0.f : expf(s - mn);
      const float sum = warp_sum(p);
      ps[r * TF_PT + lane] = p;
      if (lane == 0) {
        const float corr = mo == -INFINITY ? 0.f : expf(mo - mn);
        crow[r] = corr;
        lrow[r] = lrow[r] * corr + sum;
        mrow[r] = mn;
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < OR; ++i) {
      const int r = og + RG * i;
      if (r < rows) {
        const float corr = crow[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= corr;
      }
    }
    // a row must not meet the values of nodes it does not see (they may be
    // infinite or NaN): tiles with nodes skip weights of zero
    const bool drafts = (tile + 1) * TF_PT > t.L;
#pragma unroll 4
    for (int p = 0; p < TF_PT; ++p) {
      float v[4];
      load4(vb + p * C::KLD + oc, v);
#pragma unroll
      for (int i = 0; i < OR; ++i) {
        const int r = og + RG * i;
        const float w = r < rows ? ps[r * TF_PT + p] : 0.f;
        if (drafts && w == 0.f) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] = fmaf(w, v[e], o[i][e]);
      }
    }
    __syncthreads();  // the stage and ps may be written again
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  pdl_trigger();
  if (C_ == 1) {
#pragma unroll
    for (int i = 0; i < OR; ++i) {
      const int r = og + RG * i, n = n0 + r;
      if (r < rows) {
        const float l = lrow[r];
        float* dst = a.out + (size_t)(t.row0 + n / rep) * a.ldo + (size_t)(g * rep + n % rep) * HD + oc;
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = l == 0.f ? 0.f : o[i][e] / l;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < OR; ++i) {
    const int r = og + RG * i;
    if (r < RT)
      *reinterpret_cast<float4*>(os + r * HD + oc) = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
  }
  cl.sync();
  // join: the cluster's CTAs take the rows in turn
  for (int r = rank + C_ * warp; r < rows; r += C_ * (TF_THREADS / 32)) {
    float m = -INFINITY;
    for (int c = 0; c < C_; ++c) m = fmaxf(m, *cl.map_shared_rank(mrow + r, c));
    float l = 0.f, acc[HD / 32];
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) acc[e] = 0.f;
    for (int c = 0; c < C_; ++c) {
      const float mc = *cl.map_shared_rank(mrow + r, c);
      if (mc == -INFINITY) continue;  // no position of this share is seen
      const float f = expf(mc - m);
      l = fmaf(*cl.map_shared_rank(lrow + r, c), f, l);
      const float* oc_ = cl.map_shared_rank(os + r * HD, c);
#pragma unroll
      for (int e = 0; e < HD / 32; ++e) acc[e] = fmaf(oc_[lane + 32 * e], f, acc[e]);
    }
    const int n = n0 + r;
    float* dst = a.out + (size_t)(t.row0 + n / rep) * a.ldo + (size_t)(g * rep + n % rep) * HD;
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) dst[lane + 32 * e] = l == 0.f ? 0.f : acc[e] / l;
  }
  cl.sync();  // the others may still read this CTA's shared memory
}

template <class KT, int HD, int RT>
int launch_fma(const TreeArgs& a, int dev, int n_sm, cudaStream_t s) {
  using C = TfCfg<KT, HD, RT>;
  static bool ready[kMaxDevices] = {};  // the attribute is the device's
  if (!ready[dev]) {
    if (cudaFuncSetAttribute(tree_fma_kernel<KT, HD, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)C::SMEM) != cudaSuccess)
      return Q3TTS_ERR_CUDA;
    ready[dev] = true;
  }
  const int rep = a.Hq / a.kv.Hkv, row_tiles = (a.max_nodes * rep + RT - 1) / RT;
  const long items = (long)a.n_seqs * a.kv.Hkv * row_tiles;
  const int tiles = (int)(((long)a.kv.pages_per_stream * a.kv.page_size + TF_PT - 1) / TF_PT);
  const int c = tree_cluster(items, tiles, 4 * n_sm);
  if (items * c > 0x7fffffffL) return Q3TTS_ERR_UNSUPPORTED;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * c));
  cfg.blockDim = dim3(TF_THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = c;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, tree_fma_kernel<KT, HD, RT>, a, row_tiles) == cudaSuccess ? Q3TTS_OK
                                                                                           : Q3TTS_ERR_CUDA;
}

template <class KT>
int launch_fma_any(const TreeArgs& a, int dev, int n_sm, cudaStream_t s) {
  const int rows = a.max_nodes * (a.Hq / a.kv.Hkv);
  if (a.kv.hd == 128) return rows <= 8 ? launch_fma<KT, 128, 8>(a, dev, n_sm, s) : launch_fma<KT, 128, 32>(a, dev, n_sm, s);
  return rows <= 8 ? launch_fma<KT, 64, 8>(a, dev, n_sm, s) : launch_fma<KT, 64, 32>(a, dev, n_sm, s);
}

}  // namespace

int tree_cluster(long items, int tiles, long slots) {
  int c = 1;
  while (c < 8 && items * c * 2 <= slots && c * 2 <= tiles) c *= 2;
  return c;
}

int launch_tree_attention(const TreeArgs& a, int layers, int kdt, cudaStream_t s) {
  if (a.n_seqs <= 0 || a.n_rows <= 0) return Q3TTS_OK;
  int dev = 0, n_sm = 0;
  if (!current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  if (tree_mma_ok(a, layers, kdt)) return launch_tree_mma(a, layers, dev, n_sm, s);
  return kdt == Q3TTS_BF16 ? launch_fma_any<bf16>(a, dev, n_sm, s) : launch_fma_any<float>(a, dev, n_sm, s);
}

}  // namespace q3

// kv8_cache.cu -- quantising keys and values as they are written to the 8-bit
// cache, and reading them back.
//
// A block of B positions of a kv head's keys (or values) has one power of two,
//   2^e = the least with max |x| <= 448 x 2^e over its finite elements,  code = RN_e4m3(x / 2^e),
// so scaling is exact and the code is the only rounding.  448 = 1.75 x 2^8: with
// bits the fp32 pattern of the largest magnitude, e + 127 is the exponent field of
// bits + 0x1fffff (a mantissa above .75 carries into it) less 8.  While a block
// fills its power only rises; codes that are there already are then rounded again,
// which loses nothing but what falls under the format's smallest step.
//
// Both are bound by the bytes they move, rows in one form and codes in the other: 125,000 rows of
// eight kv heads read back to bf16 (771 MB): 123 us, 6.3 TB/s, 92 % of a plain copy (141 us with 64-bit
// divisions in the addresses: three quarters of the issue slots were taken); eight fp32 prompts of 2 ..
// 1982 rows written (81 MB): 15.7 us, 5.2 TB/s, waves of warps that each wait for their rows (17.9 with every
// element looked at for infinities and NaN).  Calls for single tokens are a launch and three dependent
// loads, 2.5 to 3 us.
#include "kv8.cuh"

namespace q3 {

namespace {

constexpr int KV8_THREADS = 256;  // of the reads
constexpr int KV8_WRITE_THREADS = 128;

// Four consecutive elements of a row, as they lie and as fp32.
__device__ __forceinline__ float4 load4(const float* p, bool wide) {
  return wide ? *reinterpret_cast<const float4*>(p) : make_float4(p[0], p[1], p[2], p[3]);
}
__device__ __forceinline__ uint2 load4(const bf16* p, bool wide) {
  if (wide) return *reinterpret_cast<const uint2*>(p);
  const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
  return make_uint2(u[0] | (uint32_t)u[1] << 16, u[2] | (uint32_t)u[3] << 16);
}
__device__ __forceinline__ float4 as_f(float4 v) { return v; }
__device__ __forceinline__ float4 as_f(uint2 u) {
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
template <class T>
struct Four {
  using V = float4;
};
template <>
struct Four<bf16> {
  using V = uint2;
};
// Whether x is an infinity or NaN.
__device__ __forceinline__ bool special(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
// The largest of the magnitudes' bits; ALL: infinities and NaN among them.
template <bool ALL>
__device__ __forceinline__ uint32_t top_bits(uint32_t top, float4 f) {
  const float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (ALL || !special(x[i])) top = max(top, __float_as_uint(x[i]) & 0x7fffffffu);
  return top;
}

// A warp per block, kv head and k or v; a lane has four elements of a row, a load
// RPL rows.  Up to U loads of rows stay in registers between the maximum and the
// rounding (blocks of more rows are read twice, the second time from the caches).  Five CTAs of 128
// threads to an SM for fp32 rows, eight for bf16, which stay as they lie (two of 256 threads, all rows as
// fp32: 20.8 us for the prompts above).
template <class T, int HD, int U>
__global__ void __launch_bounds__(KV8_WRITE_THREADS, U == 1 || sizeof(T) == 2 ? 8 : 5)
    kv8_write_kernel(Kv8Cache c, Kv8Rows r, const T* k, int ldk, const T* v, int ldv, int blocks, unsigned units, int wide) {
  pdl_wait();
  pdl_trigger();
  constexpr int RPL = 128 / HD;
  const int lane = threadIdx.x & 31, sub = lane / (HD / 4), e0 = lane % (HD / 4) * 4;
  const unsigned unit = blockIdx.x * (KV8_WRITE_THREADS / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const unsigned planes = 2 * c.Hkv, of = unit / planes, seq = of / blocks;
  const int jh = unit - of * planes, j = jh >= c.Hkv, head = jh - j * c.Hkv, nth = of - seq * blocks;
  Kv8Seq t;
  if (!kv8_seq(r, c.page, seq, true, t)) return;
  const int p0 = (kv8_div(t.L, c.block, c.block_inv) + nth) * c.block;  // the block's first position
  const int from = max(p0, t.L), to = min(p0 + c.block, t.L + t.n);  // new ones in it
  if (from >= to) return;
  const int m = to - from, held = from - p0;  // held: rows that were there
  const int ld = j ? ldv : ldk;
  const T* src = (j ? v : k) + (long long)(t.row0 + from - t.L) * ld + head * HD + e0;
  using V = typename Four<T>::V;
  V x[U];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPL + sub;
      x[u] = V{};
      if (i < m) x[u] = load4(src + (long long)i * ld, wide);
    }
  };
  const int entry = kv8_div(p0, c.page, c.page_inv), slot = p0 - entry * c.page;
  const int page = r.page_table[(size_t)seq * r.pps + entry];
  // (infinities and NaN do not count: sorted out, here and when rounding, only where there are any)
  uint32_t top = 0;
  for (int i0 = 0; i0 < m; i0 += U * RPL) {
    load(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) top = top_bits<true>(top, as_f(x[u]));
  }
  top = __reduce_max_sync(0xffffffffu, top);
  const bool odd = top >= 0x7f800000u;
  if (odd) {
    top = 0;
    for (int i0 = 0; i0 < m; i0 += U * RPL) {
      if (m > U * RPL) load(i0);
#pragma unroll
      for (int u = 0; u < U; ++u) top = top_bits<false>(top, as_f(x[u]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
  }
  if (page < 0 || page >= c.n_pages) {
    if (lane == 0) op_status(r.status, Q3TTS_ERR_ARG);
    return;
  }
  const Kv8Plane at(c, j, head);
  const long long row = at.row + (long long)page * at.rows + slot;
  uint8_t* power = c.powers + at.power + (long long)page * at.powers + kv8_div(slot, c.block, c.block_inv);
  int byte = max((int)((top + 0x1fffffu) >> 23) - 8, 0);
  if (held > 0) {
    const int before = *power;
    __syncwarp();  // all lanes have read it before lane 0 writes it
    if (byte > before) {
      // what is there is rounded again
      const float by = kv8_power(before - byte + 127);
      for (int i = sub; i < held; i += RPL) {
        uint32_t* code = reinterpret_cast<uint32_t*>(c.codes + (row + i) * HD + e0);
        float f[4];
        fp8x4_to_f32(*code, f);
        *code = kv8_codes(f[0] * by, f[1] * by, f[2] * by, f[3] * by);
      }
    }
    byte = max(byte, before);
  }
  const float by = kv8_power(254 - byte);
  uint8_t* dst = c.codes + (row + held) * HD + e0;
  for (int i0 = 0; i0 < m; i0 += U * RPL) {
    if (m > U * RPL) load(i0);
    const float nan = __int_as_float(0x7fc00000);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * RPL + sub;
      float4 f = as_f(x[u]);
      if (odd) f = make_float4(special(f.x) ? nan : f.x, special(f.y) ? nan : f.y, special(f.z) ? nan : f.z, special(f.w) ? nan : f.w);
      if (i < m) *reinterpret_cast<uint32_t*>(dst + i * HD) = kv8_codes(f.x * by, f.y * by, f.z * by, f.w * by);
    }
  }
  if (lane == 0) *power = (uint8_t)byte;
}

__device__ __forceinline__ void store16(float* p, const float* f, bool wide) {
  if (wide) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + i), "f"(f[i]), "f"(f[i + 1]), "f"(f[i + 2]),
                   "f"(f[i + 3]), "f"(f[i + 4]), "f"(f[i + 5]), "f"(f[i + 6]), "f"(f[i + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = f[i];
  }
}
__device__ __forceinline__ void store16(bf16* p, const float* f, bool wide) {
  if (wide) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = __float2bfloat16_rn(f[i]);
  }
}

// 16 codes, which are not read again.
__device__ __forceinline__ uint4 kv8_load16(const uint8_t* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// A warp per 16 rows, kv head and k or v; a lane has 16 codes of a row.
constexpr int KV8_READ_ROWS = 16;

template <class T, int HD>
__global__ void __launch_bounds__(KV8_THREADS) kv8_read_kernel(Kv8Cache c, Kv8Rows r, const int* path, T* k, int ldk, T* v,
                                                               int ldv, int chunks, unsigned units, int wide) {
  pdl_wait();
  pdl_trigger();
  constexpr int LPR = HD / 16, RPL = 32 / LPR, U = KV8_READ_ROWS / RPL;
  const int lane = threadIdx.x & 31, sub = lane / LPR, e0 = lane % LPR * 16;
  const unsigned unit = blockIdx.x * (KV8_THREADS / 32) + (threadIdx.x >> 5);
  if (unit >= units) return;
  const unsigned planes = 2 * c.Hkv, of = unit / planes, seq = of / chunks;
  const int jh = unit - of * planes, j = jh >= c.Hkv, head = jh - j * c.Hkv, i0 = (of - seq * chunks) * KV8_READ_ROWS;
  Kv8Seq t;
  if (!kv8_seq(r, c.page, seq, path == nullptr, t) || i0 >= t.n) return;
  const long long cap = (long long)r.pps * c.page;
  const Kv8Plane at(c, j, head);
  const int* table = r.page_table + (size_t)seq * r.pps;
  const uint8_t *codes = c.codes + at.row * HD + e0, *powers = c.powers + at.power;
  uint4 x[U];
  int power[U];
  bool have[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + u * RPL + sub;
    have[u] = i < t.n;
    const int off = have[u] && path ? path[t.row0 + i] : i;
    bool ok = off >= 0 && (long long)t.L + off < cap;
    const int pos = ok ? t.L + off : 0, entry = kv8_div(pos, c.page, c.page_inv), slot = pos - entry * c.page;
    int page = 0;
    if (have[u] && ok) {
      page = table[entry];
      ok = (unsigned)page < (unsigned)c.n_pages;
    }
    if (have[u] && !ok) op_status(r.status, Q3TTS_ERR_ARG);
    have[u] = have[u] && ok;
    x[u] = make_uint4(0, 0, 0, 0);
    power[u] = 0;
    if (have[u]) {
      x[u] = kv8_load16(codes + ((long long)page * at.rows + slot) * HD);
      power[u] = powers[(long long)page * at.powers + kv8_div(slot, c.block, c.block_inv)];
    }
  }
  const int ld = j ? ldv : ldk;
  T* dst = (j ? v : k) + (long long)(t.row0 + i0 + sub) * ld + head * HD + e0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!have[u]) continue;
    float f[16];
    fp8x4_to_f32(x[u].x, f);
    fp8x4_to_f32(x[u].y, f + 4);
    fp8x4_to_f32(x[u].z, f + 8);
    fp8x4_to_f32(x[u].w, f + 12);
    const float by = kv8_power(power[u]);
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] *= by;
    store16(dst + (long long)(u * RPL) * ld, f, wide);
  }
}

int grid_of(long long units, int threads, unsigned* grid) {
  const int warps = threads / 32;
  if (units > 0x7fffffffll) return Q3TTS_ERR_UNSUPPORTED;  // (warps are numbered in 32 bits)
  *grid = (unsigned)((units + warps - 1) / warps);
  return Q3TTS_OK;
}

template <class T, int HD, int U>
int launch_write(const Kv8Cache& c, const Kv8Rows& r, const void* k, int ldk, const void* v, int ldv, cudaStream_t s) {
  const int blocks = (int)(((long long)r.max_rows + 2ll * c.block - 2) / c.block);  // touched at most, from any offset
  const long long units = (long long)r.n_seqs * blocks * 2 * c.Hkv;
  unsigned grid;
  const int rc = grid_of(units, KV8_WRITE_THREADS, &grid);
  if (rc != Q3TTS_OK) return rc;
  const int wide = (((uintptr_t)k | (uintptr_t)v) & (4 * sizeof(T) - 1)) == 0 && ldk % 4 == 0 && ldv % 4 == 0;
  return launch_pdl(kv8_write_kernel<T, HD, U>, dim3(grid), dim3(KV8_WRITE_THREADS), 0, s, c, r, static_cast<const T*>(k), ldk,
                    static_cast<const T*>(v), ldv, blocks, (unsigned)units, wide) == cudaSuccess
             ? Q3TTS_OK
             : Q3TTS_ERR_CUDA;
}

template <class T, int HD>
int launch_write_rows(const Kv8Cache& c, const Kv8Rows& r, const void* k, int ldk, const void* v, int ldv, cudaStream_t s) {
  if (r.max_rows == 1 || c.block == 1) return launch_write<T, HD, 1>(c, r, k, ldk, v, ldv, s);
  return launch_write<T, HD, HD / 8>(c, r, k, ldk, v, ldv, s);  // 16 rows
}

template <class T, int HD>
int launch_read(const Kv8Cache& c, const Kv8Rows& r, const int* path, void* k, int ldk, void* v, int ldv, cudaStream_t s) {
  const int chunks = (int)(((long long)r.max_rows + KV8_READ_ROWS - 1) / KV8_READ_ROWS);
  const long long units = (long long)r.n_seqs * chunks * 2 * c.Hkv;
  unsigned grid;
  const int rc = grid_of(units, KV8_THREADS, &grid);
  if (rc != Q3TTS_OK) return rc;
  const size_t al = 32 / sizeof(T);
  const int wide = (((uintptr_t)k | (uintptr_t)v) & 31) == 0 && ldk % al == 0 && ldv % al == 0;
  return launch_pdl(kv8_read_kernel<T, HD>, dim3(grid), dim3(KV8_THREADS), 0, s, c, r, path, static_cast<T*>(k), ldk,
                    static_cast<T*>(v), ldv, chunks, (unsigned)units, wide) == cudaSuccess
             ? Q3TTS_OK
             : Q3TTS_ERR_CUDA;
}

}  // namespace

int launch_kv8_write(const Kv8Cache& c, const Kv8Rows& r, int dtype, const void* k, int ldk, const void* v, int ldv,
                     cudaStream_t s) {
  if (dtype == Q3TTS_F32)
    return c.hd == 128 ? launch_write_rows<float, 128>(c, r, k, ldk, v, ldv, s) : launch_write_rows<float, 64>(c, r, k, ldk, v, ldv, s);
  return c.hd == 128 ? launch_write_rows<bf16, 128>(c, r, k, ldk, v, ldv, s) : launch_write_rows<bf16, 64>(c, r, k, ldk, v, ldv, s);
}

int launch_kv8_read(const Kv8Cache& c, const Kv8Rows& r, const int* path, int dtype, void* k, int ldk, void* v, int ldv,
                    cudaStream_t s) {
  if (dtype == Q3TTS_F32)
    return c.hd == 128 ? launch_read<float, 128>(c, r, path, k, ldk, v, ldv, s) : launch_read<float, 64>(c, r, path, k, ldk, v, ldv, s);
  return c.hd == 128 ? launch_read<bf16, 128>(c, r, path, k, ldk, v, ldv, s) : launch_read<bf16, 64>(c, r, path, k, ldk, v, ldv, s);
}

}  // namespace q3

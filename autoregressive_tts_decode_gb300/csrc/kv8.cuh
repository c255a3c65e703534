// kv8.cuh -- the paged cache in 8 bits: its descriptor, what its kernels share
// and their launchers.  Arguments are checked by the callers (kv8_api.cu); a
// launcher returns a status code.
//
// A kernel here may begin while the one before it on the stream, which writes the codes and powers that
// it reads, still runs (it waits before it reads anything).  So it reads no memory through the non-coherent
// path, which is for data that nothing writes in a kernel's whole lifetime.
#pragma once

#include "ops.cuh"
#include "q3tts_kv8.h"

namespace q3 {

// Rows of a call: sequence s has rows start[s] .. start[s + 1] - 1 at positions
// lengths[s] and on.
struct Kv8Rows {
  const int* page_table;  // [n_seqs][pps]
  const int* lengths;
  const int* start;  // [n_seqs + 1]
  int pps, n_seqs, n_rows, max_rows;
  int* status;
};

// Row r of codes ([layer][page][k|v][kv head][slot], head dim bytes each); powers are
// one byte for each `block` slots of it.
struct Kv8Cache {
  uint8_t* codes;
  uint8_t* powers;
  int n_pages, Hkv, page, hd, block, layer;
  unsigned page_inv, block_inv;  // for kv8_div
};
// n / d for whole numbers below 2^31, with inv = ceil(2^32 / d): the product is the quotient or,
// of large ones, one more.
__device__ __forceinline__ int kv8_div(int n, int d, unsigned inv) {
  if (d == 1) return n;
  const int q = (int)__umulhi((unsigned)n, inv);
  return q - (q * d > n);
}
inline unsigned kv8_inverse(int d) { return (unsigned)(((1ull << 32) + d - 1) / d); }
// Rows of codes and bytes of powers of one kv head's keys or values in a layer: of page 0, and
// from one page to the next.
struct Kv8Plane {
  long long row, power;
  int rows, powers, per_page;
  __device__ __forceinline__ Kv8Plane(const Kv8Cache& c, int kv, int head) {
    const long long first = ((long long)c.layer * c.n_pages * 2 + kv) * c.Hkv + head;
    per_page = kv8_div(c.page, c.block, c.block_inv);
    row = first * c.page;
    power = first * per_page;
    rows = 2 * c.Hkv * c.page;
    powers = 2 * c.Hkv * per_page;
  }
};
__device__ __forceinline__ long long kv8_row(const Kv8Cache& c, int page, int kv, int head, int slot) {
  return ((((long long)c.layer * c.n_pages + page) * 2 + kv) * c.Hkv + head) * c.page + slot;
}

struct Kv8Seq {
  int L, n, row0;
};
// Lengths and rows come from device memory, so they are checked here: a sequence
// whose entries do not fit is left out and reported.
__device__ __forceinline__ bool kv8_seq(const Kv8Rows& r, long long page, int seq, bool positions, Kv8Seq& t) {
  t.L = r.lengths[seq];
  t.row0 = r.start[seq];
  const int end = r.start[seq + 1];
  t.n = end - t.row0;
  const bool ok = t.row0 >= 0 && end >= t.row0 && end <= r.n_rows && t.n <= r.max_rows && t.L >= 0 &&
                  (!positions || (long long)t.L + t.n <= r.pps * page);
  if (!ok) op_status(r.status, Q3TTS_ERR_ARG);
  return ok && t.n > 0;
}

// 2^(byte - 127) as fp32 (2^-127 is a denormal; 255: NaN).
__device__ __forceinline__ float kv8_power(int byte) {
  return __int_as_float(byte <= 0 ? 1 << 22 : byte >= 255 ? 0x7fc00000 : byte << 23);
}

// Four fp32 values (448 at most in size) to E4M3, nearest even; NaN stays NaN.
__device__ __forceinline__ uint32_t kv8_codes(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

struct Kv8AttnArgs {
  Kv8Cache c;
  Kv8Rows r;
  const unsigned long long* masks;  // [n_rows], or NULL: causal
  const void* q;
  void* out;
  int ldq, ldo, Hq;
  // the limit of the waits inside the kernels in units of 1024 cycles and, for the test of
  // their running out, the position tile at which the first CTA's products are lost (-1: none)
  int wait_1024 = 4 << 20;  // ~2 s
  int lost_tile = -1;
};

// Quantising writes and reading back (kv8_cache.cu).
int launch_kv8_write(const Kv8Cache& c, const Kv8Rows& r, int dtype, const void* k, int ldk, const void* v, int ldv,
                     cudaStream_t s);
int launch_kv8_read(const Kv8Cache& c, const Kv8Rows& r, const int* path, int dtype, void* k, int ldk, void* v, int ldv,
                    cudaStream_t s);
// Attention (kv8_attention.cu).
int launch_kv8_attention(const Kv8AttnArgs& a, int layers, int dtype, cudaStream_t s);

}  // namespace q3

// kv_pages.cu -- copying pages of a paged cache and compacting accepted rows.
//
// Both move bytes and compute nothing: their floor is the moved bytes read once
// and written once at the memory's copy rate.  A page is one block per layer
// ([k|v][kv head][position][head dim], contiguous), a row the head-dim elements
// of one position, kv head and k or v.
#include "ops.cuh"

namespace q3 {

namespace {

// ------------------------------------------------------------ page copies
//
// The page ids are host data (the allocator's), so they travel as kernel
// parameters: no upload, and a captured launch keeps its own copy of them.  300
// pages of 28 layers (1.1 GB moved): 159 us, 6.9 TB/s, the rate of a plain copy; 3
// pages: 3.6 us, a launch's time.
constexpr int CP_PAIRS = 448;   // pairs of a launch (kernel parameters: 3.5 KB of the 4 KB every device takes)
constexpr int CP_THREADS = 256;
constexpr int CP_UNROLL = 8;    // 16-byte loads in flight per thread
constexpr int CP_CHUNK = CP_THREADS * CP_UNROLL;  // 16-byte words of a CTA's chunk: 32 KB

struct CopyPairs {
  int src[CP_PAIRS], dst[CP_PAIRS];
};

__global__ void __launch_bounds__(CP_THREADS) copy_pages_kernel(uint4* pool, long long n_pages, int words,
                                                                const __grid_constant__ CopyPairs pr) {
  pdl_wait();
  pdl_trigger();
  const int pair = blockIdx.y;
  const uint4* s = pool + ((size_t)blockIdx.z * n_pages + pr.src[pair]) * words;
  uint4* d = pool + ((size_t)blockIdx.z * n_pages + pr.dst[pair]) * words;
  const int w0 = blockIdx.x * CP_CHUNK + threadIdx.x;
  uint4 v[CP_UNROLL];
#pragma unroll
  for (int i = 0; i < CP_UNROLL; ++i)
    if (w0 + i * CP_THREADS < words) v[i] = ld_stream16(s + w0 + i * CP_THREADS);
#pragma unroll
  for (int i = 0; i < CP_UNROLL; ++i)
    if (w0 + i * CP_THREADS < words) __stcs(d + w0 + i * CP_THREADS, v[i]);
}

// ------------------------------------------------------------- compaction
//
// Row L + path[i] moves to row L + i, for every layer, kv head, k and v.  The
// path ascends, so path[i] >= i: rows are taken in order, a chunk of them is
// loaded whole before any of it is stored, and a row is never written before it
// has been read.  A CTA moves one sequence's rows in one layer: path and pages
// are looked up once for all heads (a CTA per head: 21.4 us).  64 sequences, up to
// 12 rows of 28 layers (81 MB moved): 18 us, 4.5 TB/s, bound by the latency of
// three dependent loads in each of three waves of CTAs; 4, 6 or 12 loads in flight
// per thread or five to eight CTAs per SM were no faster.
constexpr int CR_THREADS = 256;
constexpr int CR_UNROLL = 8;  // 16-byte loads in flight per thread
constexpr int CR_ROWS = CR_THREADS;  // rows looked up at a time

__global__ void __launch_bounds__(CR_THREADS) compact_rows_kernel(KVDesc kv, int row_shift, const int* lengths,
                                                                  const int* path, int max_path, const int* path_len,
                                                                  int* status) {
  pdl_wait();
  pdl_trigger();
  __shared__ long long from[CR_ROWS], to[CR_ROWS];  // 16-byte words from the layer's start: a row's first key head
  const int seq = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int n = path_len[seq], L = lengths[seq];
  const int* pa = path + (size_t)seq * max_path;
  const int* table = kv.page_table + (size_t)seq * kv.pages_per_stream;
  const long long cap = (long long)kv.pages_per_stream * kv.page_size;
  // the row's place, -1 if its page is outside the pool
  auto place = [&](int pos) -> long long {
    const int page = table[pos / kv.page_size];
    if (page < 0 || page >= kv.n_pages) return -1;
    return ((long long)page * 2 * kv.Hkv * kv.page_size + pos % kv.page_size) << row_shift;
  };
  bool ok = n >= 0 && n <= max_path && L >= 0;
  if (ok)
    for (int i = tid; i < n; i += CR_THREADS) {
      const int p = pa[i], before = i ? pa[i - 1] : -1;
      ok = ok && p > before && (long long)L + p < cap;
      const long long f = ok ? place(L + p) : -1, t = ok ? place(L + i) : -1;
      ok = ok && f >= 0 && t >= 0;
      if (i < CR_ROWS) {  // (longer paths: looked up again below)
        from[i] = f;
        to[i] = p == i ? -1 : t;  // -1: already there
      }
    }
  if (!__syncthreads_and(ok)) {
    if (tid == 0 && layer == 0) op_status(status, Q3TTS_ERR_ARG);
    return;
  }
  uint4* pool = reinterpret_cast<uint4*>(kv.pool) +
                (((long long)layer * kv.n_pages * 2 * kv.Hkv * kv.page_size) << row_shift);
  const int units = 2 * kv.Hkv;                                        // (k|v, head)
  const long long unit_words = (long long)kv.page_size << row_shift;  // from one to the next
  const int c = tid & ((1 << row_shift) - 1), step = CR_THREADS >> row_shift;
  for (int i0 = 0; i0 < n; i0 += CR_ROWS) {
    const int m = min(CR_ROWS, n - i0);
    if (i0) {
      __syncthreads();
      if (tid < m) {
        const int i = i0 + tid, p = pa[i];
        from[tid] = place(L + p);
        to[tid] = p == i ? -1 : place(L + i);
      }
      __syncthreads();
    }
    for (int e0 = tid >> row_shift; e0 - (tid >> row_shift) < m * units; e0 += step * CR_UNROLL) {
      uint4 v[CR_UNROLL];
      long long dst[CR_UNROLL];
#pragma unroll
      for (int u = 0; u < CR_UNROLL; ++u) {
        const int e = e0 + u * step, i = e / units;
        dst[u] = e < m * units ? to[i] : -1;
        const long long off = (long long)(e - i * units) * unit_words + c;
        v[u] = pool[dst[u] < 0 ? c : from[i] + off];  // (a row that stays: some word, not stored)
        dst[u] = dst[u] < 0 ? -1 : dst[u] + off;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < CR_UNROLL; ++u)
        if (dst[u] >= 0) pool[dst[u]] = v[u];
    }
  }
}

}  // namespace

int launch_copy_pages(const KVDesc& kv, int layers, int esz, const int32_t* src, const int32_t* dst, int n,
                      cudaStream_t s) {
  const long long words = 2ll * kv.Hkv * kv.page_size * kv.hd * esz / 16;  // of a page in one layer
  if (layers > 65535 || words > 0x7fffffff - CP_CHUNK) return Q3TTS_ERR_UNSUPPORTED;
  for (int i0 = 0; i0 < n; i0 += CP_PAIRS) {
    CopyPairs p;
    const int m = n - i0 < CP_PAIRS ? n - i0 : CP_PAIRS;
    for (int i = 0; i < m; ++i) {
      p.src[i] = src[i0 + i];
      p.dst[i] = dst[i0 + i];
    }
    const dim3 grid((unsigned)((words + CP_CHUNK - 1) / CP_CHUNK), m, layers);
    if (launch_pdl(copy_pages_kernel, grid, dim3(CP_THREADS), 0, s, reinterpret_cast<uint4*>(kv.pool),
                   (long long)kv.n_pages, (int)words, p) != cudaSuccess)
      return Q3TTS_ERR_CUDA;
  }
  return Q3TTS_OK;
}

int launch_compact_rows(const KVDesc& kv, int layers, int esz, int n_seqs, const int* lengths, const int* path,
                        int max_path, const int* path_len, int* status, cudaStream_t s) {
  if (n_seqs <= 0 || max_path <= 0) return Q3TTS_OK;
  if (layers > 65535) return Q3TTS_ERR_UNSUPPORTED;
  int row_shift = 0;  // 16-byte words of a row: 8, 16 or 32
  while ((16 << row_shift) < kv.hd * esz) ++row_shift;
  return launch_pdl(compact_rows_kernel, dim3(n_seqs, layers), dim3(CR_THREADS), 0, s, kv, row_shift, lengths, path,
                    max_path, path_len, status) == cudaSuccess
             ? Q3TTS_OK
             : Q3TTS_ERR_CUDA;
}

}  // namespace q3

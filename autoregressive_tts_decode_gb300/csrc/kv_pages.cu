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
// parameters: no upload, and a captured launch keeps its own copy of them.
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
// path ascends, so path[i] >= i: rows are taken in order, a chunk is loaded
// whole before any of it is stored, and a row is never written before it has
// been read.  One warp moves the rows of one (sequence, layer, k|v, head).
constexpr int CR_WARPS = 4;
constexpr int CR_UNROLL = 8;  // 16-byte loads in flight per lane

__global__ void __launch_bounds__(CR_WARPS * 32) compact_rows_kernel(KVDesc kv, int row_words, const int* lengths,
                                                                     const int* path, int max_path,
                                                                     const int* path_len, int units, int* status) {
  pdl_wait();
  pdl_trigger();
  const int seq = blockIdx.y, lane = threadIdx.x & 31;
  const int unit = blockIdx.x * CR_WARPS + (threadIdx.x >> 5);  // (layer, k|v, head)
  if (unit >= units) return;
  const int n = path_len[seq], L = lengths[seq];
  const int* pa = path + (size_t)seq * max_path;
  const long long cap = (long long)kv.pages_per_stream * kv.page_size;
  bool ok = n >= 0 && n <= max_path && L >= 0;
  if (ok)
    for (int i = lane; i < n; i += 32) {
      const int p = pa[i];
      ok = ok && p >= 0 && (long long)L + p < cap && (i == 0 || p > pa[i - 1]);
    }
  if (!__all_sync(0xffffffffu, ok)) {
    if (lane == 0) op_status(status, Q3TTS_ERR_ARG);
    return;
  }
  const int head = unit % kv.Hkv, sel = unit / kv.Hkv % 2, layer = unit / kv.Hkv / 2;
  const int* table = kv.page_table + (size_t)seq * kv.pages_per_stream;
  uint4* pool = reinterpret_cast<uint4*>(kv.pool);
  auto at = [&](int pos) -> uint4* {
    const int page = table[pos / kv.page_size];
    if (page < 0 || page >= kv.n_pages) {
      op_status(status, Q3TTS_ERR_ARG);
      return nullptr;
    }
    return pool + (((((size_t)layer * kv.n_pages + page) * 2 + sel) * kv.Hkv + head) * kv.page_size +
                   pos % kv.page_size) * row_words;
  };
  const int words = n * row_words;
  for (int w0 = 0; w0 < words; w0 += 32 * CR_UNROLL) {
    uint4 v[CR_UNROLL];
    uint4* dst[CR_UNROLL];
#pragma unroll
    for (int i = 0; i < CR_UNROLL; ++i) {
      const int w = w0 + i * 32 + lane, r = w / row_words, c = w % row_words;
      dst[i] = nullptr;
      if (w < words && pa[r] != r) {
        const uint4* s = at(L + pa[r]);
        uint4* d = at(L + r);
        if (s && d) {
          v[i] = s[c];
          dst[i] = d + c;
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < CR_UNROLL; ++i)
      if (dst[i]) *dst[i] = v[i];
    __syncwarp();
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
  const long long units = 2ll * layers * kv.Hkv;
  if (n_seqs > 65535 || units > 0x7fffffff - CR_WARPS) return Q3TTS_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)((units + CR_WARPS - 1) / CR_WARPS), n_seqs);
  return launch_pdl(compact_rows_kernel, grid, dim3(CR_WARPS * 32), 0, s, kv, kv.hd * esz / 16, lengths, path, max_path,
                    path_len, (int)units, status) == cudaSuccess
             ? Q3TTS_OK
             : Q3TTS_ERR_CUDA;
}

}  // namespace q3

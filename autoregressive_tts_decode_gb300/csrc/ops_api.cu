// ops_api.cu -- C entries of the branching-decode operators over caller-owned
// buffers (declared in include/q3tts_branch.h): argument checks, then one launch.
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <utility>
#include <vector>

#include "ops.cuh"

namespace q3 {

bool current_device(int* dev, int* n_sm) {
  static std::atomic<int> sms[kMaxDevices];
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) return false;
  int n = sms[*dev].load(std::memory_order_relaxed);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess || n < 1) return false;
    sms[*dev].store(n, std::memory_order_relaxed);
  }
  *n_sm = n;
  return true;
}

}  // namespace q3

namespace {

// q3tts_debug_lose_tile, for the thread's next attention.
struct Lose {
  bool armed;
  int tile, wait_us;
};
thread_local Lose lose = {};

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

int esz(int dtype) { return dtype == Q3TTS_F32 ? 4 : 2; }

int check_cache(const q3tts_kv_cache* kv) {
  if (!kv || !kv->pool || !aligned(kv->pool, 16)) return Q3TTS_ERR_ARG;
  if (kv->layers < 1 || kv->n_pages < 1 || kv->n_kv_heads < 1 || kv->page_size < 1) return Q3TTS_ERR_ARG;
  if (kv->kv_dtype != Q3TTS_F32 && kv->kv_dtype != Q3TTS_BF16) return Q3TTS_ERR_ARG;
  if (kv->head_dim != 64 && kv->head_dim != 128) return Q3TTS_ERR_UNSUPPORTED;
  return Q3TTS_OK;
}

q3::KVDesc desc(const q3tts_kv_cache& c, const int32_t* table, int pps) {
  q3::KVDesc d;
  d.pool = c.pool;
  d.page_table = table;
  d.pages_per_stream = pps;
  d.page_size = c.page_size;
  d.n_pages = c.n_pages;
  d.Hkv = c.n_kv_heads;
  d.hd = c.head_dim;
  return d;
}

// positions of a sequence are 32-bit with room to spare
bool table_ok(const q3tts_kv_cache& c, int pps) { return pps >= 1 && (long long)pps * c.page_size <= 1 << 30; }

bool beam_shape(int groups, int beams, int vocab, int k) {
  return groups >= 0 && beams >= 1 && beams <= Q3TTS_MAX_BEAMS && vocab >= 1 && vocab <= 1 << 24 && k >= 1 &&
         k <= Q3TTS_MAX_BEAMS && (long long)groups * Q3TTS_MAX_BEAMS <= 1 << 24;
}

// [p, p + n) and [q, q + m) share a byte
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + m && b < a + n;
}

// Rows of a call: n of `bytes` bytes, `stride` (at least bytes) apart.
struct Span {
  const void* p;
  size_t bytes, stride;
  long long n;
};
uintptr_t start_of(const Span& r) { return (uintptr_t)r.p; }
uintptr_t end_of(const Span& r) { return (uintptr_t)r.p + (size_t)(r.n - 1) * r.stride + r.bytes; }

// A row of a and a row of b share a byte (rows that lie between each other's, as
// the fields of records do, need not).
bool rows_overlap(const Span& a, const Span& b) {
  if (!a.bytes || !b.bytes || a.n < 1 || b.n < 1) return false;
  if (start_of(a) >= end_of(b) || start_of(b) >= end_of(a)) return false;
  if (a.stride == b.stride) {
    // row i + d of b starts diff + d stride after row i of a: the least d in range for
    // which it does not end before that row, and whether it then starts before its end
    const long long st = (long long)a.stride, diff = (long long)start_of(b) - (long long)start_of(a);
    long long d = (-diff - (long long)b.bytes) / st - 1;
    while (diff + d * st <= -(long long)b.bytes) ++d;  // (two steps at most)
    d = std::max(d, 1 - a.n);
    return d < b.n && diff + d * st < (long long)a.bytes;
  }
  uintptr_t x = start_of(a), y = start_of(b);
  for (long long i = 0, j = 0; i < a.n && j < b.n;) {
    if (x + a.bytes <= y) {  // (all of a's rows up to the one that y may meet)
      const long long skip = (long long)((y - x - a.bytes) / a.stride) + 1;
      i += skip;
      x += (size_t)skip * a.stride;
    } else if (y + b.bytes <= x) {
      const long long skip = (long long)((x - y - b.bytes) / b.stride) + 1;
      j += skip;
      y += (size_t)skip * b.stride;
    } else {
      return true;
    }
  }
  return false;
}
// Rows that are numbered by one list of ids: whether row r of one meets row r of
// the other, whatever r is (other strides: not known).
bool same_rows_overlap(const Span& a, const Span& b) {
  return a.bytes && b.bytes && a.n > 0 && b.n > 0 && a.stride == b.stride && overlap(a.p, a.bytes, b.p, b.bytes);
}

// Whether a set writes what another one reads or writes (rows by number, or by ids).
bool sets_meet(const q3tts_rows* sets, int n_sets, bool ids, long long n_in, long long n_out) {
  auto meet = [&](const Span& a, const Span& b) { return ids ? same_rows_overlap(a, b) : rows_overlap(a, b); };
  auto span = [&](const q3tts_rows& r, bool dst) {
    return dst ? Span{r.dst, r.row_bytes, r.dst_stride, n_out} : Span{r.src, r.row_bytes, r.src_stride, n_in};
  };
  if (n_sets > 8 && !ids && n_in > 0) {
    // many sets: the spans by their starts; where none begins inside one before it
    // (two that are only read aside), none meet
    std::vector<std::pair<Span, bool>> all;
    for (int i = 0; i < n_sets; ++i)
      for (int d = sets[i].src == sets[i].dst; d < 2; ++d)
        if (sets[i].row_bytes) all.emplace_back(span(sets[i], d != 0), d != 0);
    std::sort(all.begin(), all.end(), [](const auto& a, const auto& b) { return start_of(a.first) < start_of(b.first); });
    uintptr_t read = 0, written = 0;
    bool close = false;
    for (const auto& e : all) {
      close = close || start_of(e.first) < (e.second ? std::max(read, written) : written);
      uintptr_t& end = e.second ? written : read;
      end = std::max(end, end_of(e.first));
    }
    if (!close) return false;
  }
  for (int i = 0; i < n_sets; ++i)
    for (int j = 0; j < n_sets; ++j)
      if (i != j && (meet(span(sets[i], true), span(sets[j], false)) ||
                     (j < i && meet(span(sets[i], true), span(sets[j], true)))))
        return true;
  return false;
}

}  // namespace

extern "C" {

int q3tts_tree_attention(const q3tts_kv_cache* kv, int layer, const int32_t* page_table_dev, int pages_per_seq,
                         int n_seqs, const int32_t* lengths_dev, const int32_t* node_start_dev,
                         const uint64_t* masks_dev, int n_rows, int max_nodes, int n_q_heads, const float* q_dev,
                         int ldq, float* out_dev, int ldo, int32_t* status_dev, void* cuda_stream) {
  const int rc = check_cache(kv);
  if (rc != Q3TTS_OK) return rc;
  if (layer < 0 || layer >= kv->layers || n_seqs < 0 || n_rows < 0 || n_q_heads < 1 || n_q_heads % kv->n_kv_heads ||
      max_nodes < 1 || max_nodes > Q3TTS_MAX_TREE_NODES)
    return Q3TTS_ERR_ARG;
  if (n_seqs == 0 || n_rows == 0) return Q3TTS_OK;
  if (!page_table_dev || !lengths_dev || !node_start_dev || !masks_dev || !q_dev || !out_dev ||
      !aligned(page_table_dev, 4) || !aligned(lengths_dev, 4) || !aligned(node_start_dev, 4) ||
      !aligned(masks_dev, 8) || !aligned(q_dev, 4) || !aligned(out_dev, 4) || !aligned(status_dev, 4))
    return Q3TTS_ERR_ARG;
  if (!table_ok(*kv, pages_per_seq) || (long long)n_q_heads * kv->head_dim > ldq ||
      (long long)n_q_heads * kv->head_dim > ldo)
    return Q3TTS_ERR_ARG;
  if (!q3::tree_attention_ok(desc(*kv, page_table_dev, pages_per_seq), kv->layers, n_q_heads))
    return Q3TTS_ERR_UNSUPPORTED;
  // rows of one sequence are written while another's queries are still read
  const size_t row = sizeof(float) * (size_t)n_q_heads * kv->head_dim;
  if (rows_overlap(Span{q_dev, row, sizeof(float) * (size_t)ldq, n_rows}, Span{out_dev, row, sizeof(float) * (size_t)ldo, n_rows}))
    return Q3TTS_ERR_ARG;
  q3::TreeArgs a;
  a.kv = desc(*kv, page_table_dev, pages_per_seq);
  a.layer = layer;
  a.n_seqs = n_seqs;
  a.lengths = lengths_dev;
  a.node_start = node_start_dev;
  a.masks = reinterpret_cast<const unsigned long long*>(masks_dev);
  a.n_rows = n_rows;
  a.max_nodes = max_nodes;
  a.Hq = n_q_heads;
  a.q = q_dev;
  a.ldq = ldq;
  a.out = out_dev;
  a.ldo = ldo;
  a.status = status_dev;
  if (lose.armed) {
    a.lost_tile = lose.tile;
    a.wait_1024 = 2 * lose.wait_us;  // (at the highest SM clock, 2070 MHz; less than 2 << 22)
    lose.armed = false;
  }
  return q3::launch_tree_attention(a, kv->layers, kv->kv_dtype, (cudaStream_t)cuda_stream);
}

int q3tts_debug_lose_tile(int tile, int wait_us) {
  if (tile < 0 || wait_us < 1 || wait_us > 2000000) return Q3TTS_ERR_ARG;
  lose = {true, tile, wait_us};
  return Q3TTS_OK;
}

int q3tts_copy_pages(const q3tts_kv_cache* kv, const int32_t* src, const int32_t* dst, int n, void* cuda_stream) {
  const int rc = check_cache(kv);
  if (rc != Q3TTS_OK) return rc;
  if (n < 0 || (n && (!src || !dst))) return Q3TTS_ERR_ARG;
  for (int i = 0; i < n; ++i)
    if (src[i] < 0 || src[i] >= kv->n_pages || dst[i] < 0 || dst[i] >= kv->n_pages) return Q3TTS_ERR_ARG;
  try {
    // no page is written twice, and none is both read and written
    std::vector<int32_t> d(dst, dst + n);
    std::sort(d.begin(), d.end());
    if (std::adjacent_find(d.begin(), d.end()) != d.end()) return Q3TTS_ERR_ARG;
    for (int i = 0; i < n; ++i)
      if (std::binary_search(d.begin(), d.end(), src[i])) return Q3TTS_ERR_ARG;
  } catch (...) {
    return Q3TTS_ERR_CAPACITY;  // no host memory for the check
  }
  return q3::launch_copy_pages(desc(*kv, nullptr, 0), kv->layers, esz(kv->kv_dtype), src, dst, n,
                               (cudaStream_t)cuda_stream);
}

int q3tts_compact_rows(const q3tts_kv_cache* kv, const int32_t* page_table_dev, int pages_per_seq, int n_seqs,
                       const int32_t* lengths_dev, const int32_t* path_dev, int max_path, const int32_t* path_len_dev,
                       int32_t* status_dev, void* cuda_stream) {
  const int rc = check_cache(kv);
  if (rc != Q3TTS_OK) return rc;
  if (n_seqs < 0 || max_path < 0 || !table_ok(*kv, pages_per_seq)) return Q3TTS_ERR_ARG;
  if (n_seqs == 0 || max_path == 0) return Q3TTS_OK;
  if (!page_table_dev || !lengths_dev || !path_dev || !path_len_dev || !aligned(page_table_dev, 4) ||
      !aligned(lengths_dev, 4) || !aligned(path_dev, 4) || !aligned(path_len_dev, 4) || !aligned(status_dev, 4))
    return Q3TTS_ERR_ARG;
  if (max_path > pages_per_seq * kv->page_size) return Q3TTS_ERR_ARG;
  return q3::launch_compact_rows(desc(*kv, page_table_dev, pages_per_seq), kv->layers, esz(kv->kv_dtype), n_seqs,
                                 lengths_dev, path_dev, max_path, path_len_dev, status_dev,
                                 (cudaStream_t)cuda_stream);
}

size_t q3tts_beam_workspace_size(int groups, int beams, int vocab, int k) {
  int dev = 0, n_sm = 0;
  if (!beam_shape(groups, beams, vocab, k) || !q3::current_device(&dev, &n_sm)) return 0;
  return groups ? q3::beam_workspace(groups, beams, vocab, n_sm) : 0;
}

int q3tts_beam_select(const float* logits_dev, size_t ld, const int32_t* row_ids_dev, int groups, int beams, int vocab,
                      const float* scores_dev, const uint8_t* finished_dev, const uint8_t* history_dev, int eos_token,
                      int special_from, float repetition_penalty, int k, int32_t* tokens_dev, int32_t* parents_dev,
                      float* scores_out_dev, void* workspace_dev, size_t workspace_bytes, void* cuda_stream) {
  if (groups < 0 || beams < 1 || vocab < 1 || k < 1 || ld < (size_t)vocab) return Q3TTS_ERR_ARG;
  if (!beam_shape(groups, beams, vocab, k)) return Q3TTS_ERR_UNSUPPORTED;
  if (!(repetition_penalty > 0.f) || eos_token >= vocab || special_from > vocab) return Q3TTS_ERR_ARG;
  if (finished_dev && eos_token < 0) return Q3TTS_ERR_ARG;  // a finished beam's candidate is its end code
  if (groups == 0) return Q3TTS_OK;
  if (!logits_dev || !scores_dev || !tokens_dev || !parents_dev || !scores_out_dev || !aligned(logits_dev, 4) ||
      !aligned(row_ids_dev, 4) || !aligned(scores_dev, 4) || !aligned(tokens_dev, 4) || !aligned(parents_dev, 4) ||
      !aligned(scores_out_dev, 4) || !aligned(workspace_dev, 8))
    return Q3TTS_ERR_ARG;
  // a group's scores are read after another group's may have been written
  if (overlap(scores_dev, sizeof(float) * (size_t)groups * beams, scores_out_dev, sizeof(float) * (size_t)groups * k) &&
      !(scores_dev == scores_out_dev && k == beams))
    return Q3TTS_ERR_ARG;
  q3::BeamArgs a;
  a.logits = logits_dev;
  a.ld = ld;
  a.row_ids = row_ids_dev;
  a.groups = groups;
  a.beams = beams;
  a.vocab = vocab;
  a.scores = scores_dev;
  a.finished = finished_dev;
  a.history = repetition_penalty != 1.f ? history_dev : nullptr;
  a.eos = eos_token;
  a.special_from = special_from;
  a.penalty = repetition_penalty;
  a.k = k;
  a.tokens = tokens_dev;
  a.parents = parents_dev;
  a.scores_out = scores_out_dev;
  int dev = 0, n_sm = 0;
  if (!q3::current_device(&dev, &n_sm)) return Q3TTS_ERR_CUDA;
  const size_t need = q3::beam_workspace(groups, beams, vocab, n_sm);
  if (need && (!workspace_dev || workspace_bytes < need)) return Q3TTS_ERR_ARG;
  return q3::launch_beam_select(a, workspace_dev, (cudaStream_t)cuda_stream);
}

int q3tts_reorder_rows(const q3tts_rows* sets, int n_sets, const int32_t* row_ids_dev, const int32_t* parents_dev,
                       int groups, int beams_in, int beams_out, int32_t* status_dev, void* cuda_stream) {
  if (n_sets < 0 || (n_sets && !sets) || groups < 0 || beams_in < 1 || beams_out < 1) return Q3TTS_ERR_ARG;
  if (beams_in > Q3TTS_MAX_BEAMS || beams_out > Q3TTS_MAX_BEAMS || (long long)groups * Q3TTS_MAX_BEAMS > 65535)
    return Q3TTS_ERR_UNSUPPORTED;
  if (row_ids_dev && beams_in != beams_out) return Q3TTS_ERR_ARG;
  if (!aligned(row_ids_dev, 4) || !aligned(status_dev, 4)) return Q3TTS_ERR_ARG;
  const long long n_in = (long long)groups * beams_in, n_out = (long long)groups * beams_out;
  for (int i = 0; i < n_sets; ++i) {
    const q3tts_rows& r = sets[i];
    if (r.row_bytes == 0) continue;
    if (!r.src || !r.dst || r.src_stride < r.row_bytes || r.dst_stride < r.row_bytes) return Q3TTS_ERR_ARG;
    const Span src{r.src, r.row_bytes, r.src_stride, n_in}, dst{r.dst, r.row_bytes, r.dst_stride, n_out};
    if (r.src == r.dst) {  // in place
      if (r.src_stride != r.dst_stride || beams_in != beams_out) return Q3TTS_ERR_ARG;
    } else if (row_ids_dev ? same_rows_overlap(src, dst) : rows_overlap(src, dst)) {
      return Q3TTS_ERR_ARG;
    }
    if (!row_ids_dev && parents_dev && rows_overlap(dst, Span{parents_dev, sizeof(int32_t) * (size_t)n_out, r.dst_stride, 1}))
      return Q3TTS_ERR_ARG;
  }
  try {
    if (n_sets > 1 && sets_meet(sets, n_sets, row_ids_dev != nullptr, n_in, n_out)) return Q3TTS_ERR_ARG;
  } catch (...) {
    return Q3TTS_ERR_CAPACITY;  // no host memory for the check
  }
  if (groups == 0 || n_sets == 0) return Q3TTS_OK;
  if (!parents_dev || !aligned(parents_dev, 4)) return Q3TTS_ERR_ARG;
  return q3::launch_reorder_rows(sets, n_sets, row_ids_dev, parents_dev, groups, beams_in, beams_out, status_dev,
                                 (cudaStream_t)cuda_stream);
}

}  // extern "C"

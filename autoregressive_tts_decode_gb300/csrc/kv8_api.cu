// kv8_api.cu -- C entries of the 8-bit cache's operators (declared in
// include/q3tts_kv8.h): argument checks, then one launch.
#include "api_checks.h"
#include "kv8.cuh"

namespace {

int check_cache(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows) {
  if (!kv || !rows || !kv->codes || !kv->powers || !aligned(kv->codes, 16)) return Q3TTS_ERR_ARG;
  if (kv->layers < 1 || kv->n_pages < 1 || kv->n_kv_heads < 1 || kv->page_size < 1) return Q3TTS_ERR_ARG;
  if (kv->block < 1 || kv->page_size % kv->block || rows->layer < 0 || rows->layer >= kv->layers) return Q3TTS_ERR_ARG;
  if (kv->head_dim != 64 && kv->head_dim != 128) return Q3TTS_ERR_UNSUPPORTED;
  return Q3TTS_OK;
}

q3::Kv8Cache desc(const q3tts_kv8_cache& c, int layer) {
  q3::Kv8Cache d;
  d.codes = static_cast<uint8_t*>(c.codes);
  d.powers = static_cast<uint8_t*>(c.powers);
  d.n_pages = c.n_pages;
  d.Hkv = c.n_kv_heads;
  d.page = c.page_size;
  d.hd = c.head_dim;
  d.block = c.block;
  d.layer = layer;
  d.page_inv = q3::kv8_inverse(c.page_size);
  d.block_inv = q3::kv8_inverse(c.block);
  return d;
}

// Whether the kernels that number a page's rows (its keys and its values) in 32 bits take them.
bool pages_ok(const q3tts_kv8_cache& c) { return 2ll * c.n_kv_heads <= 0x7fffffffll / c.page_size; }

bool dtype_ok(int d) { return d == Q3TTS_F32 || d == Q3TTS_BF16; }
size_t esz(int d) { return d == Q3TTS_F32 ? 4 : 2; }

// What the calls have in common; *work: whether there is any.
int check_rows(const q3tts_kv8_cache& c, const q3tts_kv8_rows& q, q3::Kv8Rows* r, bool* work) {
  *work = false;
  if (q.n_seqs < 0 || q.n_rows < 0 || q.max_rows < 1 || !dtype_ok(q.row_dtype)) return Q3TTS_ERR_ARG;
  if (q.n_seqs == 0 || q.n_rows == 0) return Q3TTS_OK;
  if (!q.page_table || !q.lengths || !q.row_start || !aligned(q.page_table, 4) || !aligned(q.lengths, 4) ||
      !aligned(q.row_start, 4) || !aligned(q.status, 4))
    return Q3TTS_ERR_ARG;
  // positions of a sequence are 32-bit with room to spare
  if (q.pages_per_seq < 1 || (long long)q.pages_per_seq * c.page_size > 1 << 30) return Q3TTS_ERR_ARG;
  r->page_table = q.page_table;
  r->lengths = q.lengths;
  r->start = q.row_start;
  r->pps = q.pages_per_seq;
  r->n_seqs = q.n_seqs;
  r->n_rows = q.n_rows;
  r->max_rows = q.max_rows < q.n_rows ? q.max_rows : q.n_rows;
  r->status = q.status;
  *work = true;
  return Q3TTS_OK;
}

bool rows_ok(const void* p, int ld, int heads, int hd, int dtype) {
  return p && aligned(p, esz(dtype)) && (long long)heads * hd <= ld;
}

Span span(const void* p, int ld, int heads, int hd, int dtype, int n) {
  return Span{p, esz(dtype) * (size_t)heads * hd, esz(dtype) * (size_t)ld, n};
}

}  // namespace

extern "C" {

int q3tts_kv8_write(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows, const void* k_dev, int ldk,
                    const void* v_dev, int ldv, void* cuda_stream) {
  int rc = check_cache(kv, rows);
  if (rc != Q3TTS_OK) return rc;
  q3::Kv8Rows r;
  bool work;
  rc = check_rows(*kv, *rows, &r, &work);
  if (rc != Q3TTS_OK || !work) return rc;
  const int dtype = rows->row_dtype;
  if (!rows_ok(k_dev, ldk, kv->n_kv_heads, kv->head_dim, dtype) || !rows_ok(v_dev, ldv, kv->n_kv_heads, kv->head_dim, dtype))
    return Q3TTS_ERR_ARG;
  // (a block's codes are numbered in 32 bits too)
  if (!pages_ok(*kv) || (long long)kv->block * kv->head_dim > 0x7fffffffll) return Q3TTS_ERR_UNSUPPORTED;
  return q3::launch_kv8_write(desc(*kv, rows->layer), r, dtype, k_dev, ldk, v_dev, ldv, (cudaStream_t)cuda_stream);
}

int q3tts_kv8_read(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows, const int32_t* path_dev, void* k_out_dev,
                   int ldk, void* v_out_dev, int ldv, void* cuda_stream) {
  int rc = check_cache(kv, rows);
  if (rc != Q3TTS_OK) return rc;
  q3::Kv8Rows r;
  bool work;
  rc = check_rows(*kv, *rows, &r, &work);
  if (rc != Q3TTS_OK || !work) return rc;
  const int heads = kv->n_kv_heads, hd = kv->head_dim, dtype = rows->row_dtype;
  if (!rows_ok(k_out_dev, ldk, heads, hd, dtype) || !rows_ok(v_out_dev, ldv, heads, hd, dtype) || !aligned(path_dev, 4))
    return Q3TTS_ERR_ARG;
  if (rows_overlap(span(k_out_dev, ldk, heads, hd, dtype, r.n_rows), span(v_out_dev, ldv, heads, hd, dtype, r.n_rows)))
    return Q3TTS_ERR_ARG;
  if (!pages_ok(*kv)) return Q3TTS_ERR_UNSUPPORTED;
  return q3::launch_kv8_read(desc(*kv, rows->layer), r, path_dev, dtype, k_out_dev, ldk, v_out_dev, ldv,
                             (cudaStream_t)cuda_stream);
}

int q3tts_kv8_attention(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows, const uint64_t* masks_dev,
                        const void* q_dev, int ldq, void* out_dev, int ldo, int n_q_heads, void* cuda_stream) {
  int rc = check_cache(kv, rows);
  if (rc != Q3TTS_OK) return rc;
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads || (masks_dev && rows->max_rows > Q3TTS_MAX_TREE_NODES)) return Q3TTS_ERR_ARG;
  q3::Kv8AttnArgs a;
  bool work;
  rc = check_rows(*kv, *rows, &a.r, &work);
  if (rc != Q3TTS_OK || !work) return rc;
  const int hd = kv->head_dim, dtype = rows->row_dtype, n = a.r.n_rows;
  if (!rows_ok(q_dev, ldq, n_q_heads, hd, dtype) || !rows_ok(out_dev, ldo, n_q_heads, hd, dtype) || !aligned(masks_dev, 8))
    return Q3TTS_ERR_ARG;
  if (n_q_heads / kv->n_kv_heads > 1024 ||
      2ll * kv->layers * kv->n_pages > 0x7fffffffll / kv->n_kv_heads / kv->page_size)
    return Q3TTS_ERR_UNSUPPORTED;
  // rows of one sequence are written while another's queries are still read
  if (rows_overlap(span(q_dev, ldq, n_q_heads, hd, dtype, n), span(out_dev, ldo, n_q_heads, hd, dtype, n))) return Q3TTS_ERR_ARG;
  a.c = desc(*kv, rows->layer);
  a.masks = reinterpret_cast<const unsigned long long*>(masks_dev);
  a.q = q_dev;
  a.out = out_dev;
  a.ldq = ldq;
  a.ldo = ldo;
  a.Hq = n_q_heads;
  const q3::Lose l = q3::take_lose();
  if (l.armed) {
    a.lost_tile = l.tile;
    a.wait_1024 = l.wait_1024();
  }
  return q3::launch_kv8_attention(a, kv->layers, dtype, (cudaStream_t)cuda_stream);
}

}  // extern "C"

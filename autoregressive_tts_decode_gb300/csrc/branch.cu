// branch.cu -- the handle's branching calls (declared in include/q3tts_branch.h):
// forking streams, checking a tree of drafted frames, and beam frames.
//
// A stream's context is a list of pages.  Whole pages are shared between
// streams that hold the same positions (page_ref counts the holders) and are
// never written again; the last, partly filled page is what a branch copies.
#include <algorithm>
#include <vector>

#include "engine.cuh"
#include "ops.cuh"

namespace q3 {
namespace {

q3tts_kv_cache cache_of(const q3tts_handle* h) {
  q3tts_kv_cache c;
  c.pool = h->kv_pool;
  c.layers = h->c.talker_layers;
  c.n_pages = h->n_pages;
  c.n_kv_heads = h->Hkv;
  c.page_size = h->c.page_size;
  c.head_dim = h->hd;
  c.kv_dtype = h->c.kv_dtype;
  return c;
}

// New contexts for the streams ids[0..n): stream ids[b] takes over the first
// len positions of src[b] (a stream; its own id: unchanged).  Planned in full
// before anything changes.
struct Branches {
  std::vector<int> ids, src;
  std::vector<std::vector<int>> pages;   // the new lists, -1 for a page to be taken
  std::vector<int> copy_from, copy_to;   // partly filled pages to copy
  std::vector<int> len;
};

// Plans the page lists; extra[b] more pages are wanted by stream ids[b] right
// after.  False when the pool would run out (nothing has changed).
bool plan(const q3tts_handle* h, Branches& br, const std::vector<int>& extra) {
  const int n = (int)br.ids.size(), ps = h->c.page_size;
  std::vector<int> ref = h->page_ref;
  std::vector<char> moved(h->c.max_streams, 0), kept(h->c.max_streams, 0);
  for (int b = 0; b < n; ++b) {
    moved[br.ids[b]] = 1;
    for (int p : h->pages[br.ids[b]]) --ref[p];
  }
  // a parent that carries on itself keeps its last page; otherwise its first
  // child takes it, and the further ones copy it
  for (int b = 0; b < n; ++b)
    if (br.src[b] == br.ids[b]) kept[br.src[b]] = 1;
  br.pages.assign(n, std::vector<int>());
  br.len.assign(n, 0);
  long need = 0;
  for (int b = 0; b < n; ++b) {
    const int s = br.src[b], len = h->len[s], whole = len / ps;
    br.len[b] = len;
    br.pages[b].assign(h->pages[s].begin(), h->pages[s].begin() + whole);
    for (int p : br.pages[b]) ++ref[p];
    if (len % ps) {
      const int last = h->pages[s][whole];
      const bool own = s == br.ids[b] || (moved[s] && !kept[s]);
      if (own) {
        if (s != br.ids[b]) kept[s] = 1;
        br.pages[b].push_back(last);
        ++ref[last];
      } else {
        br.pages[b].push_back(-1);
        br.copy_from.push_back(last);
        ++need;
      }
    }
    need += extra[b];
  }
  long room = (long)h->free_pages.size();
  for (int b = 0; b < n; ++b)
    for (int p : h->pages[br.ids[b]])
      if (ref[p] == 0) {
        ++room;
        ref[p] = -1;  // counted
      }
  return need <= room;
}

// Carries the plan out: host lists, page copies, page-table rows.
int apply(q3tts_handle* h, Branches& br) {
  const int n = (int)br.ids.size();
  for (int b = 0; b < n; ++b)
    for (int p : br.pages[b])
      if (p >= 0) ++h->page_ref[p];
  for (int b = 0; b < n; ++b) {
    for (int p : h->pages[br.ids[b]]) drop_page(h, p);
    if (h->tree_sid == br.ids[b]) h->tree_sid = -1;
  }
  br.copy_to.clear();
  for (int b = 0; b < n; ++b) {
    std::vector<int>& list = br.pages[b];
    if (!list.empty() && list.back() < 0) {
      list.back() = h->free_pages.back();
      h->free_pages.pop_back();
      h->page_ref[list.back()] = 1;
      br.copy_to.push_back(list.back());
    }
    h->pages[br.ids[b]].assign(list.begin(), list.end());
    h->len[br.ids[b]] = br.len[b];
  }
  const int m = (int)br.copy_from.size();
  if (m) {
    const q3tts_kv_cache c = cache_of(h);
    const int rc = q3tts_copy_pages(&c, br.copy_from.data(), br.copy_to.data(), m, h->s);
    if (rc != Q3TTS_OK) return rc;
    h->launches += (m + 447) / 448;
  }
  // pageable sources: staged before each call returns
  for (int b = 0; b < n; ++b) {
    const std::vector<int>& list = br.pages[b];
    if (br.src[b] != br.ids[b] && !list.empty() &&
        cudaMemcpyAsync(h->page_table + (size_t)br.ids[b] * h->pps, list.data(), sizeof(int) * list.size(),
                        cudaMemcpyHostToDevice, h->s) != cudaSuccess)
      return Q3TTS_ERR_CUDA;
  }
  return Q3TTS_OK;
}

int upload(q3tts_handle* h, void* dst, const void* src, size_t bytes) {
  return cudaMemcpyAsync(dst, src, bytes, cudaMemcpyHostToDevice, h->s) == cudaSuccess ? Q3TTS_OK : Q3TTS_ERR_CUDA;
}

int fork(q3tts_handle* h, int src, const int32_t* dst, int n) {
  Branches br;
  br.ids.assign(dst, dst + n);
  br.src.assign(n, src);
  if (!plan(h, br, std::vector<int>(n, 0))) return Q3TTS_ERR_CAPACITY;
  int rc = apply(h, br);
  // pending state, history and stop flag: rows of `src` into the others', up
  // to a beam group at a time
  const q3tts_rows sets[4] = {
      {h->pending_h, h->pending_h, sizeof(float) * h->Dt, sizeof(float) * h->Dt, sizeof(float) * h->Dt},
      {h->pending_logits, h->pending_logits, sizeof(float) * h->Vt, sizeof(float) * h->Vt, sizeof(float) * h->Vt},
      {h->history, h->history, (size_t)h->Vt, (size_t)h->Vt, (size_t)h->Vt},
      {h->finished, h->finished, 1, 1, 1}};
  for (int i0 = 0; i0 < n && rc == Q3TTS_OK; i0 += Q3TTS_MAX_BEAMS - 1) {
    const int m = std::min(n - i0, Q3TTS_MAX_BEAMS - 1);
    int ids[Q3TTS_MAX_BEAMS] = {src}, parents[Q3TTS_MAX_BEAMS] = {};
    std::copy(dst + i0, dst + i0 + m, ids + 1);
    rc = upload(h, h->beam_ids, ids, sizeof(int) * (m + 1));
    if (rc == Q3TTS_OK) rc = upload(h, h->beam_parents, parents, sizeof(int) * (m + 1));
    if (rc == Q3TTS_OK)
      rc = launch_reorder_rows(sets, 4, h->beam_ids, h->beam_parents, 1, m + 1, m + 1, h->d_err, h->s);
    h->launches += 1;
  }
  if (rc != Q3TTS_OK)
    for (int b = 0; b < n; ++b) h->len[dst[b]] = -1;  // no prompt until a prefill or a fork succeeds
  return rc;
}

int tree_step(q3tts_handle* h, int sid, const int32_t* codes_dev, const int32_t* parents, int n, float* hidden_dev,
              float* logits_dev) {
  const int len = h->len[sid], need = pages_for(h, len + n);
  // the tree before this one makes room
  const int freed = h->tree_sid < 0 ? 0 : tree_pages(h, h->len[h->tree_sid]);
  const int have = (int)h->pages[sid].size() - (h->tree_sid == sid ? freed : 0);
  if (need - have > (int)h->free_pages.size() + freed) return Q3TTS_ERR_CAPACITY;
  if (h->tree_sid >= 0) drop_tree(h, h->len[h->tree_sid]);
  for (int i = have; i < need; ++i) {
    const int page = h->free_pages.back();
    h->free_pages.pop_back();
    take_page(h, sid, page);
  }
  TreeMeta t = {};
  unsigned long long masks[Q3TTS_MAX_TREE_NODES];
  int depth[Q3TTS_MAX_TREE_NODES];
  t.length = len;
  t.node_start[1] = n;
  for (int i = 0; i < n; ++i) {
    depth[i] = parents[i] < 0 ? 0 : depth[parents[i]] + 1;
    masks[i] = (1ull << i) | (parents[i] < 0 ? 0ull : masks[parents[i]]);
    t.rope_pos[i] = len + depth[i];
  }
  int rc = Q3TTS_OK;
  if (need > have)
    rc = upload(h, h->page_table + (size_t)sid * h->pps + have, h->pages[sid].data() + have,
                sizeof(int) * (need - have));
  if (rc == Q3TTS_OK) rc = upload(h, h->tree_meta, &t, sizeof(t));
  if (rc == Q3TTS_OK) rc = upload(h, h->tree_masks, masks, sizeof(masks[0]) * n);
  if (rc == Q3TTS_OK && cudaMemcpyAsync(h->tree_codes, codes_dev, sizeof(int32_t) * (size_t)n * Q3TTS_N_CODEBOOKS,
                                        cudaMemcpyDeviceToDevice, h->s) != cudaSuccess)
    rc = Q3TTS_ERR_CUDA;
  if (rc == Q3TTS_OK) rc = tree_layered(h, sid, n);
  if (rc == Q3TTS_OK &&
      ((hidden_dev && cudaMemcpyAsync(hidden_dev, h->tree_h, sizeof(float) * (size_t)n * h->Dt,
                                      cudaMemcpyDeviceToDevice, h->s) != cudaSuccess) ||
       (logits_dev && cudaMemcpyAsync(logits_dev, h->tree_logits, sizeof(float) * (size_t)n * h->Vt,
                                      cudaMemcpyDeviceToDevice, h->s) != cudaSuccess)))
    rc = Q3TTS_ERR_CUDA;
  if (rc != Q3TTS_OK) {
    trim_pages(h, sid, len);
    return rc;
  }
  h->tree_sid = sid;
  h->tree_n = n;
  std::copy(parents, parents + n, h->tree_parent);
  return Q3TTS_OK;
}

int tree_accept(q3tts_handle* h, int sid, const int32_t* path, int n) {
  int rc = Q3TTS_OK;
  h->tree_sid = -1;
  if (n > 0) {
    bool move = false;
    for (int i = 0; i < n; ++i) move = move || path[i] != i;
    rc = upload(h, h->tree_meta->path, path, sizeof(int) * n);
    if (rc == Q3TTS_OK) rc = upload(h, &h->tree_meta->path_len, &n, sizeof(int));
    if (rc == Q3TTS_OK) rc = tree_commit(h, sid, n, path[n - 1], move);
    // the rows may have moved in part: no prompt until a prefill succeeds
    h->len[sid] = rc == Q3TTS_OK ? h->len[sid] + n : -1;
  }
  trim_pages(h, sid, h->len[sid]);  // pages that only other nodes used go back to the pool
  return rc;
}

int beam_frame(q3tts_handle* h, const q3tts_sampling& sp, const int32_t* ids, int groups, int beams, float* scores_dev,
               const float* uniforms_dev, int32_t* codes_dev, int32_t* parents_out) {
  const int n = groups * beams;
  int rc = upload(h, h->beam_ids, ids, sizeof(int) * n);
  if (rc != Q3TTS_OK) return rc;
  BeamArgs a = {};
  a.logits = h->pending_logits;
  a.ld = h->Vt;
  a.row_ids = h->beam_ids;
  a.groups = groups;
  a.beams = beams;
  a.vocab = h->Vt;
  a.scores = scores_dev;
  a.finished = sp.eos_token >= 0 ? h->finished : nullptr;
  a.history = sp.repetition_penalty != 1.f ? h->history : nullptr;
  a.eos = sp.eos_token;
  a.special_from = sp.special_from;
  a.penalty = sp.repetition_penalty;
  a.k = beams;
  a.tokens = h->beam_tokens;
  a.parents = h->beam_parents;
  a.scores_out = h->beam_scores;
  rc = launch_beam_select(a, h->beam_ws, h->s);
  if (rc != Q3TTS_OK) return rc;
  h->launches += beam_workspace(groups, beams, h->Vt, 1) ? 2 : 1;  // a second kernel where the lists go through it
  // the page lists are host data: the parents are read back before the streams move
  std::vector<int> par(n);
  if (cudaMemcpyAsync(par.data(), h->beam_parents, sizeof(int) * n, cudaMemcpyDeviceToHost, h->s) != cudaSuccess ||
      cudaStreamSynchronize(h->s) != cudaSuccess)
    return Q3TTS_ERR_CUDA;
  Branches br;
  br.ids.assign(ids, ids + n);
  br.src.resize(n);
  std::vector<int> extra(n, 0);
  for (int i = 0; i < n; ++i) {
    br.src[i] = ids[i / beams * beams + par[i]];
    const int len = h->len[br.src[i]];
    if (len % h->c.page_size == 0) extra[i] = 1;  // the frame's own position opens a page
  }
  if (!plan(h, br, extra)) return Q3TTS_ERR_CAPACITY;
  rc = apply(h, br);
  // what the frame reads of a stream besides its pages; the pending logits are
  // replaced by the frame
  const q3tts_rows sets[3] = {
      {h->pending_h, h->pending_h, sizeof(float) * h->Dt, sizeof(float) * h->Dt, sizeof(float) * h->Dt},
      {h->history, h->history, (size_t)h->Vt, (size_t)h->Vt, (size_t)h->Vt},
      {h->finished, h->finished, 1, 1, 1}};
  if (rc == Q3TTS_OK)
    rc = launch_reorder_rows(sets, 3, h->beam_ids, h->beam_parents, groups, beams, beams, h->d_err, h->s);
  if (rc == Q3TTS_OK && cudaMemcpyAsync(scores_dev, h->beam_scores, sizeof(float) * n, cudaMemcpyDeviceToDevice, h->s) !=
                            cudaSuccess)
    rc = Q3TTS_ERR_CUDA;
  h->launches += 1;
  static thread_local StepDesc d;
  d.n = n;
  int taken = 0;
  for (int b = 0; b < n; ++b) {
    d.sid[b] = ids[b];
    d.pos[b] = h->len[ids[b]];
    d.sp[b] = device_sampling(sp, h->Vt);
    d.newpage[b] = extra[b] ? h->free_pages[h->free_pages.size() - 1 - taken++] : -1;
  }
  if (rc == Q3TTS_OK) rc = step_layered(h, d, uniforms_dev, codes_dev, nullptr, nullptr, true);
  if (rc != Q3TTS_OK) {
    for (int b = 0; b < n; ++b) h->len[ids[b]] = -1;  // no prompt until a prefill or a fork succeeds
    return rc;
  }
  h->free_pages.resize(h->free_pages.size() - taken);
  for (int b = 0; b < n; ++b) {
    if (d.newpage[b] >= 0) take_page(h, ids[b], d.newpage[b]);
    h->len[ids[b]] += 1;
  }
  if (parents_out) std::copy(par.begin(), par.end(), parents_out);
  return Q3TTS_OK;
}

// Runs f; running out of host memory is a status, not an exception.
template <class F>
int guarded(F f) {
  try {
    return f();
  } catch (...) {
    return Q3TTS_ERR_CAPACITY;
  }
}

}  // namespace
}  // namespace q3

extern "C" {

int q3tts_fork(q3tts_handle* h, int src, const int32_t* dst_ids, int n) {
  if (!h || src < 0 || src >= h->c.max_streams || n < 1 || n >= h->c.max_streams || !dst_ids) return Q3TTS_ERR_ARG;
  bool seen[Q3TTS_MAX_STREAMS] = {};
  seen[src] = true;
  for (int i = 0; i < n; ++i) {
    if (dst_ids[i] < 0 || dst_ids[i] >= h->c.max_streams || seen[dst_ids[i]]) return Q3TTS_ERR_ARG;
    seen[dst_ids[i]] = true;
  }
  if (h->len[src] < 1) return Q3TTS_ERR_STATE;
  return q3::guarded([&] { return q3::fork(h, src, dst_ids, n); });
}

int q3tts_tree_step(q3tts_handle* h, int stream_id, const int32_t* codes_dev, const int32_t* parents, int n_nodes,
                    float* hidden_dev, float* logits_dev) {
  if (!h || stream_id < 0 || stream_id >= h->c.max_streams || !codes_dev || !parents || n_nodes < 1 ||
      n_nodes > Q3TTS_MAX_TREE_NODES)
    return Q3TTS_ERR_ARG;
  for (int i = 0; i < n_nodes; ++i)
    if (parents[i] < -1 || parents[i] >= i) return Q3TTS_ERR_ARG;
  if (!q3::tree_attention_ok(q3::talker_kv(h), h->c.talker_layers, h->Hq)) return Q3TTS_ERR_UNSUPPORTED;
  if (h->len[stream_id] < 1) return Q3TTS_ERR_STATE;
  if (h->len[stream_id] + n_nodes > h->c.kv_cap_steps) return Q3TTS_ERR_CAPACITY;
  return q3::guarded(
      [&] { return q3::tree_step(h, stream_id, codes_dev, parents, n_nodes, hidden_dev, logits_dev); });
}

int q3tts_tree_accept(q3tts_handle* h, int stream_id, const int32_t* path, int n) {
  if (!h || stream_id < 0 || stream_id >= h->c.max_streams || n < 0 || (n && !path)) return Q3TTS_ERR_ARG;
  if (h->tree_sid != stream_id) return Q3TTS_ERR_STATE;
  if (n > h->tree_n) return Q3TTS_ERR_ARG;
  for (int i = 0; i < n; ++i) {
    if (path[i] < 0 || path[i] >= h->tree_n) return Q3TTS_ERR_ARG;
    if (h->tree_parent[path[i]] != (i ? path[i - 1] : -1)) return Q3TTS_ERR_ARG;
  }
  return q3::guarded([&] { return q3::tree_accept(h, stream_id, path, n); });
}

int q3tts_beam_frame(q3tts_handle* h, const q3tts_sampling* params, const int32_t* stream_ids, int groups, int beams,
                     float* scores_dev, const float* uniforms_dev, int32_t* codes_dev, int32_t* parents) {
  if (!h || !params || !stream_ids || !scores_dev || !uniforms_dev || !codes_dev) return Q3TTS_ERR_ARG;
  if (groups < 1 || beams < 1 || beams > Q3TTS_MAX_BEAMS || groups > h->c.max_streams ||
      groups * beams > h->c.max_streams || !q3::check_sampling(*params, h->Vt))
    return Q3TTS_ERR_ARG;
  bool seen[Q3TTS_MAX_STREAMS] = {};
  for (int i = 0; i < groups * beams; ++i) {
    const int s = stream_ids[i];
    if (s < 0 || s >= h->c.max_streams || seen[s]) return Q3TTS_ERR_ARG;
    seen[s] = true;
  }
  for (int i = 0; i < groups * beams; ++i) {
    if (h->len[stream_ids[i]] < 1) return Q3TTS_ERR_STATE;
    if (h->len[stream_ids[i]] >= h->c.kv_cap_steps) return Q3TTS_ERR_CAPACITY;
  }
  return q3::guarded([&] {
    return q3::beam_frame(h, *params, stream_ids, groups, beams, scores_dev, uniforms_dev, codes_dev, parents);
  });
}

}  // extern "C"

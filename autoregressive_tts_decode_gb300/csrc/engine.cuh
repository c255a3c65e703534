// engine.cuh -- the handle behind the C ABI and the workspace layout.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <vector>

#include "common.cuh"
#include "q3tts_branch.h"

namespace q3 {

// Per-call description of a frame step, passed by value to the set-up kernel.
struct StepDesc {
  int n;
  int sid[Q3TTS_MAX_STREAMS];       // stream id of active slot b
  int pos[Q3TTS_MAX_STREAMS];       // Talker position the frame writes
  int newpage[Q3TTS_MAX_STREAMS];   // page id to enter at pos / page_size, or -1
  q3tts_sampling sp[Q3TTS_MAX_STREAMS];
};

// Where a layered step's fed codes come from: the draws, the caller's forced
// codes, or a beam selection's semantic codes (h->beam_tokens) with the
// acoustic codes drawn.
enum class FeedMode { kDrawn, kForced, kBeam };

// Per-call arrays of a drafted tree, uploaded in one copy.
struct TreeMeta {
  int length;         // committed positions
  int node_start[2];  // 0, nodes
  int path_len;
  int path[Q3TTS_MAX_TREE_NODES];
  int rope_pos[Q3TTS_MAX_TREE_NODES];
};

struct FrameKernelState;  // persistent frame kernel (frame_kernel.cu)

}  // namespace q3

struct q3tts_handle {
  q3tts_config c;
  std::vector<q3tts_layer_weights> tl, cl;
  q3tts_weights w;
  cudaStream_t s;
  int dev, n_sm;

  // dimensions
  int Dt, Dc, Ft, Fc, Hq, Hkv, hd, Vt, Vc, qkv_rows, pps, n_pages, chunk, m_max, esz;

  // workspace carve-up
  float* rope_cos;  // [kv_cap][hd/2]
  float* rope_sin;
  void* kv_pool;    // Talker KV, paged
  int* page_table;  // [max_streams][pps]
  float* cp_kv;     // CodePredictor KV: one 16-slot page per stream, fp32
  int* cp_page_table;
  float* pending_h;       // [max_streams][D_t]
  float* pending_logits;  // [max_streams][V_t]
  uint8_t* history;       // [max_streams][V_t]
  uint8_t* finished;      // [max_streams]: the stream fed its end-of-stream code
  int* d_sid;             // [max_streams]
  int* d_pos;
  q3tts_sampling* d_sp;
  int* d_fed;             // [max_streams][16] codes fed forward
  int* d_tok_stream;      // [m_max]
  int* d_tok_pos;         // [m_max]
  float *x, *hb, *qkv, *att, *gu, *act, *uin, *cpx, *logits;
  // hi/lo bf16 terms of the activations the tensor-core projections read
  // ([m_max][K] each); tc: bf16 weights whose every inner dimension is a
  // multiple of 64 take that path (Q3TTS_TC=0 turns it off)
  q3::bf16 *xh, *xl;
  bool tc = false;
  bool tc_failed = false;  // a projection could not be launched
  // split-context attention: span results [m_max][Hq][spl_nsmax][hd + 2] and
  // per-(token, kv head) counters [m_max][Hkv] (zero between launches)
  float* spl_part;
  int* spl_cnt;
  int spl_nsmax;
  int* d_err;
  // layered step replayed as a CUDA graph: the step's descriptor and its
  // per-call inputs/outputs pass through these fixed device buffers
  q3::StepDesc* d_desc;
  float* g_uni;      // [max_streams][16]
  int32_t* g_forced;  // [max_streams][16]
  int32_t* g_codes;   // [max_streams][16]
  // drafted trees (q3tts_tree_step): the latest tree's node states and the
  // small arrays its kernels read
  int32_t* tree_codes;  // [Q3TTS_MAX_TREE_NODES][16]
  float* tree_h;        // [Q3TTS_MAX_TREE_NODES][D_t] final-normed hiddens
  float* tree_logits;   // [Q3TTS_MAX_TREE_NODES][V_t]
  unsigned long long* tree_masks;  // [Q3TTS_MAX_TREE_NODES]
  q3::TreeMeta* tree_meta;
  // beams (q3tts_beam_frame): [max_streams] each
  int* beam_ids;
  int32_t* beam_tokens;
  int32_t* beam_parents;
  float* beam_scores;
  char* beam_ws;  // the selection's workspace (rows of up to 4096 codes are scanned whole)

  // host-side stream bookkeeping.  A page holds positions of one stream, or of
  // several (forks, beams) that share a prefix; page_ref counts its holders.
  // Only whole pages are shared, and positions are only ever appended, so a
  // shared page is never written.
  std::vector<int> len;  // Talker positions held; -1 = no prompt yet
  std::vector<std::vector<int>> pages;  // reserved to their longest at create: they never grow later
  std::vector<int> free_pages;
  std::vector<int> page_ref;
  // the latest drafted tree (tree_sid -1: none): its stream, nodes and parents
  int tree_sid = -1, tree_n = 0;
  int tree_parent[Q3TTS_MAX_TREE_NODES];

  q3::FrameKernelState* fk;
  char* fk_base;           // workspace region of the persistent frame kernel
  bool frame_kernel_off;   // Q3TTS_FRAME_KERNEL=0: always use the layered step
  bool used_static = false;   // q3tts_step_frame_static has run on this handle
  // failure-path test (q3tts_debug_fail_barrier), armed for one persistent launch
  int dbg_fail_bar = -1;
  long long dbg_wait_cycles = 0;
  uint64_t launches = 0;
  // streaming chunks (q3tts_step_frames): one event per frame, recorded after
  // the frame's codes are copied out
  cudaEvent_t chunk_ev[Q3TTS_MAX_CHUNK] = {};
  int chunk_n = 0;
  // the captured layered step (valid for g_n active streams, with or without
  // forced codes); g_launches kernels per replay
  cudaGraphExec_t gexec = nullptr;
  int g_n = 0;
  q3::FeedMode g_feed = q3::FeedMode::kDrawn;
  uint64_t g_launches = 0;
  cudaStream_t cap_stream = nullptr;  // stream the step is captured on
  bool graph_off = false;             // Q3TTS_GRAPH=0: launch the layered step kernel by kernel
};

namespace q3 {

// Layered frame step (one kernel per operation), any number of streams.
int step_layered(q3tts_handle* h, const StepDesc& d, const float* uniforms, int32_t* codes,
                 const int32_t* forced, float* logits, bool beam = false);
// Talker pass over the n nodes of the tree described by h->tree_meta,
// tree_masks and tree_codes; leaves tree_h and tree_logits.
int tree_layered(q3tts_handle* h, int sid, int n);
// Rows h->tree_meta->path of stream sid moved behind its context, the codes'
// history marked and the last node's state made pending.
int tree_commit(q3tts_handle* h, int sid, int n, int last, bool move);
int prefill_layered(q3tts_handle* h, int sid, const float* embeds, int len);
void step_graph_destroy(q3tts_handle* h);

// Page bookkeeping (api.cu).
void take_page(q3tts_handle* h, int sid, int page);  // a page off the free list joins sid's
void drop_page(q3tts_handle* h, int page);           // one holder less; free at none
int pages_for(const q3tts_handle* h, int len);       // pages of a context of len positions
void trim_pages(q3tts_handle* h, int sid, int len);  // the pages past those go back
// The drafted tree's pages past the first len positions of its stream: how many,
// and their return (the tree is forgotten).  No other stream holds such pages.
int tree_pages(const q3tts_handle* h, int len);
void drop_tree(q3tts_handle* h, int len);
bool check_sampling(const q3tts_sampling& p, int Vt);
q3tts_sampling device_sampling(const q3tts_sampling& p, int Vt);

KVDesc talker_kv(const q3tts_handle* h);
KVDesc cp_kv(const q3tts_handle* h);

}  // namespace q3

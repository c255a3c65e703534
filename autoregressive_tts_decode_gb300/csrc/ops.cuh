// ops.cuh -- launchers of the branching-decode operators: attention of drafted
// trees over a paged cache, page copies, compaction of accepted rows, beam
// selection and reordering of states.  The C entries over caller-owned buffers
// (ops_api.cu) and the handle's branching calls (branch.cu) both use them.
// Arguments are checked by the callers; a launcher returns a status code.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"
#include "q3tts_branch.h"

namespace q3 {

constexpr int kMaxDevices = 64;  // devices the per-device launch settings cover

// SM count of the current device and its index; false on a CUDA error or an
// index past kMaxDevices.
bool current_device(int* dev, int* n_sm);

// q3tts_debug_lose_tile, for the calling thread's next attention (which takes it).
struct Lose {
  bool armed;
  int tile, wait_us;
  int wait_1024() const { return 2 * wait_us; }  // (at the highest SM clock, 2070 MHz; less than 2 << 22)
};
Lose take_lose();

// Records err in *status (device int, may be NULL) unless one is recorded.
__device__ __forceinline__ void op_status(int* status, int err) {
  if (status) atomicCAS(status, 0, err);
}

// Attention of drafted tree nodes (tree_attention.cu); kv.page_table is
// [n_seqs][pages_per_stream].
struct TreeArgs {
  KVDesc kv;
  int layer;
  int n_seqs;
  const int* lengths;     // [n_seqs] committed positions
  const int* node_start;  // [n_seqs + 1] rows of each sequence's nodes
  const unsigned long long* masks;  // [n_rows]
  int n_rows, max_nodes, Hq;
  const float* q;  // [n_rows][ldq]
  int ldq;
  float* out;  // [n_rows][ldo]
  int ldo;
  int* status;
  // the limit of the waits inside the kernels in units of 1024 cycles and, for the test of
  // their running out, the position tile at which the first CTA's products are lost (-1: none)
  int wait_1024 = 4 << 20;  // ~2 s
  int lost_tile = -1;
};
// Whether the cache and head counts are ones it takes (the pool's rows of head
// dim elements are numbered in 32 bits).
inline bool tree_attention_ok(const KVDesc& kv, int layers, int Hq) {
  return Hq / kv.Hkv <= 1024 && 2ll * layers * kv.n_pages <= 0x7fffffffll / kv.Hkv / kv.page_size;
}
int launch_tree_attention(const TreeArgs& a, int layers, int kdt, cudaStream_t s);

// Page copies and compaction (kv_pages.cu).
int launch_copy_pages(const KVDesc& kv, int layers, int esz, const int32_t* src, const int32_t* dst, int n,
                      cudaStream_t s);
int launch_compact_rows(const KVDesc& kv, int layers, int esz, int n_seqs, const int* lengths, const int* path,
                        int max_path, const int* path_len, int* status, cudaStream_t s);

// Beam selection and reordering (beam.cu).
struct BeamArgs {
  const float* logits;
  size_t ld;           // floats between logits rows
  const int* row_ids;  // row of logits, finished and history of beam (g, b); NULL: g * beams + b
  int groups, beams, vocab;
  const float* scores;
  const uint8_t* finished;  // per row, or NULL
  const uint8_t* history;   // [row][vocab], or NULL
  int eos, special_from;
  float penalty;
  int k;
  int32_t* tokens;
  int32_t* parents;
  float* scores_out;
};
// 8-byte aligned bytes of workspace a selection needs on a GPU of n_sm SMs.
size_t beam_workspace(int groups, int beams, int vocab, int n_sm);
int launch_beam_select(const BeamArgs& a, void* workspace, cudaStream_t s);
int launch_reorder_rows(const q3tts_rows* sets, int n_sets, const int* row_ids, const int* parents, int groups,
                        int beams_in, int beams_out, int* status, cudaStream_t s);

}  // namespace q3

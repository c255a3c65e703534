// tree.cuh -- what the two forms of tree attention share (tree_attention.cu,
// tree_mma.cu).
#pragma once

#include "ops.cuh"

namespace q3 {

// What a CTA works on; false when it has no rows.  Lengths and row offsets
// come from device memory, so they are checked here: a sequence whose entries
// do not fit the cache or the buffers is left out and reported.
struct TreeSeq {
  int L, T, row0, P;  // committed positions, nodes, first row of q/out, L + T
};
__device__ __forceinline__ bool tree_seq(const TreeArgs& a, int seq, TreeSeq& t) {
  t.L = a.lengths[seq];
  t.row0 = a.node_start[seq];
  const int end = a.node_start[seq + 1];
  const long long cap = (long long)a.kv.pages_per_stream * a.kv.page_size;
  if (t.row0 < 0 || end < t.row0 || end > a.n_rows || end - t.row0 > a.max_nodes || t.L < 0 ||
      (long long)t.L + (end - t.row0) > cap) {
    op_status(a.status, Q3TTS_ERR_ARG);
    return false;
  }
  t.T = end - t.row0;
  t.P = t.L + t.T;
  return t.T > 0;
}

// CTAs of a cluster (which splits the positions of one item): enough to fill
// the slots, no more than there are tiles at the sequences' capacity, at most 8
// (the portable cluster size).
int tree_cluster(long items, int tiles, long slots);

long long tree_pool_rows(const KVDesc& kv, int layers);
bool tree_mma_ok(const TreeArgs& a, int layers, int kdt);
int launch_tree_mma(const TreeArgs& a, int layers, int dev, int n_sm, cudaStream_t s);

}  // namespace q3

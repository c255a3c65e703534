/*
 * q3tts_branch.h -- C ABI of libq3tts, second part: branching decode.
 *
 * Streams of one handle that share a prompt, drafted frames checked in trees
 * and beam search, and the operators they are made of for programs that keep
 * their own paged caches.  Conventions, status codes and dtypes are q3tts.h's.
 */
#ifndef Q3TTS_BRANCH_H
#define Q3TTS_BRANCH_H

#include "q3tts.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q3TTS_MAX_TREE_NODES 64  /* nodes of a drafted tree */
#define Q3TTS_MAX_BEAMS 32       /* beams of a group */

/* ---- Branching decode on a handle -------------------------------------
 * Takes of one prompt, trees of drafted frames and beam search.  q3tts.h
 * knows persistent streams only; these calls add ways for a stream to split.
 * A stream's KV pages that are full are shared by the streams that hold the
 * same positions and return to the pool when the last of them lets go; only
 * the last, partly filled page is copied. */

/* Makes each of the n streams dst_ids (host array, distinct, not src; n <
 * max_streams) what `src` is now: its context, pending state, semantic history
 * and stop flag.  What they held is forgotten.  Asynchronous.
 * Q3TTS_ERR_STATE if src has no prompt; Q3TTS_ERR_CAPACITY if the pool lacks
 * the pages (one per copy when the context ends inside a page), with every
 * stream left as it was. */
int q3tts_fork(q3tts_handle* h, int src, const int32_t* dst_ids, int n);

/* Runs the Talker over a tree of n_nodes (1 .. Q3TTS_MAX_TREE_NODES) drafted
 * frames that continue the stream, all of them in one pass.  What it tells of a
 * frame is its semantic code: the CodePredictor does not run, so whether the model
 * would have drawn a frame's 15 acoustic codes is not known from it.
 *   codes_dev   device int32 [n_nodes][16]: each drafted frame's codes.  A code
 *               outside its vocabulary makes q3tts_sync_status return
 *               Q3TTS_ERR_ARG, and the results are unspecified.
 *   parents     host int32 [n_nodes]: the node each one follows (a smaller
 *               index), -1 for the stream's context.
 *   hidden_dev, logits_dev  NULL, or device fp32 [n_nodes][D_t] and
 *               [n_nodes][V_t]: after each node, what q3tts_read_pending gives
 *               after a frame with those codes.
 * The stream itself does not advance; q3tts_tree_accept makes a path of the
 * tree part of it.  The handle holds one tree, the latest; a call that changes
 * its stream drops it, and its pages return to the pool.  Asynchronous.
 * Q3TTS_ERR_STATE without a prompt, Q3TTS_ERR_CAPACITY if the stream's capacity
 * or the pool lacks room for n_nodes more positions (the tree before stays then). */
int q3tts_tree_step(q3tts_handle* h, int stream_id, const int32_t* codes_dev, const int32_t* parents, int n_nodes,
                    float* hidden_dev, float* logits_dev);

/* Appends the n nodes path[0..n) (host array: path[0] a child of the context,
 * each next a child of the one before) of the handle's tree, which must be of
 * this stream (else Q3TTS_ERR_STATE), to the stream: it then is where it would
 * be after n frames with those codes fed.  Stop conditions are not applied: end
 * the path at an end code.  n = 0 drops the tree.  Either way pages that only
 * other nodes used return to the pool.  Asynchronous. */
int q3tts_tree_accept(q3tts_handle* h, int stream_id, const int32_t* path, int n);

/* One acoustic frame of a beam search over the semantic codes.  The
 * groups x beams streams stream_ids (host array, distinct; beams <=
 * Q3TTS_MAX_BEAMS) hold each group's beams, and scores_dev (device fp32,
 * groups x beams, read and written) their log probabilities so far: for a
 * prompt prefilled into a group's first stream and forked into the others,
 * start with 0 and -INFINITY.  From the pending logits q3tts_beam_select keeps
 * each group's best `beams` continuations under the semantic controls
 * special_from, eos_token and repetition_penalty of *params (one set for all;
 * do_sample, top_k, top_p and temperature do not apply to the semantic code);
 * slot b of a group becomes parent's state plus the selected code, and the
 * frame runs as q3tts_step_frame's with that code fed and the acoustic codes
 * drawn under the sub_* controls.
 *   uniforms_dev  device fp32 [groups x beams][16] (column 0 is not read).
 *   codes_dev     device int32 [groups x beams][16].
 *   parents       NULL, or host int32 [groups x beams]: the beam of the group
 *                 each slot continues.
 * A beam that has fed the end code keeps its score and yields -1 codes; a slot
 * that no continuation is left for has score -INFINITY and feeds code 0.
 * Waits for the handle's stream once, for the parents.  Q3TTS_ERR_STATE if a
 * stream has no prompt; Q3TTS_ERR_CAPACITY if a stream is full or the pool
 * lacks the pages, with streams and scores left as they were.  After a CUDA
 * error the streams have no prompt. */
int q3tts_beam_frame(q3tts_handle* h, const q3tts_sampling* params, const int32_t* stream_ids, int groups, int beams,
                     float* scores_dev, const float* uniforms_dev, int32_t* codes_dev, int32_t* parents);

/* ---- Operators over caller-owned buffers -------------------------------
 * What the calls above are made of, for programs that keep their own caches
 * and beams.  Device buffers are caller-owned and must stay valid until the
 * work has run; everything is enqueued on cuda_stream (a stream of the current
 * device) and is asynchronous; nothing is allocated on the device, and the
 * calls can be captured into a CUDA graph (host arrays are read during the
 * call).  Sizes of zero are no work.
 * status_dev, where a call has it, is NULL or a device int32: what can only be
 * checked on the device (lengths, paths, page ids, parents) and is wrong is
 * left out, and Q3TTS_ERR_ARG put there unless it already holds a code; the
 * caller clears it.  Q3TTS_ERR_TIMEOUT there: the attention gave up a wait
 * inside a kernel; its output is unspecified. */

/* A paged cache: pool is device memory, 16-byte aligned, of
 * [layers][n_pages][k|v][n_kv_heads][page_size][head_dim] elements of kv_dtype
 * (Q3TTS_F32 or Q3TTS_BF16); head_dim 64 or 128.  A sequence's position p is
 * slot p % page_size of page page_table[p / page_size], in every layer. */
typedef struct q3tts_kv_cache {
  void* pool;
  int layers, n_pages, n_kv_heads, page_size, head_dim;
  int kv_dtype;
} q3tts_kv_cache;

/* Attention of drafted tree nodes over the cache, in one layer.  Sequence s
 * holds lengths_dev[s] committed positions (0 or more), and the keys and values
 * of its nodes i = 0, 1, .. sit at the positions after them, in node order.
 * Its nodes are rows node_start_dev[s] .. node_start_dev[s + 1] - 1 of q, out
 * and masks (max_nodes bounds every sequence's count, 1 ..
 * Q3TTS_MAX_TREE_NODES).  A node sees every committed position, and node j if
 * bit j of its mask is set (its ancestors and itself, as a rule); one that sees
 * nothing gets zeroes.  One node with its own bit is a decode step's token.
 * What a row does not see does not touch it, infinities and NaN among it; a
 * row that sees such a key or value is unspecified, like one with scores (q . k /
 * sqrt(head_dim)) above 2^27 or values above 2^90 in size.
 *   page_table_dev  int32 [n_seqs][pages_per_seq]; entries past a sequence's
 *                   last position are not read.
 *   masks_dev       uint64 [n_rows], 8-byte aligned.
 *   q_dev, out_dev  fp32 [n_rows] rows of n_q_heads x head_dim, ldq and ldo
 *                   elements apart; q head h reads kv head
 *                   h / (n_q_heads / n_kv_heads), at most 1024 of them one;
 *                   scale 1 / sqrt(head_dim).
 * Caches of up to 2^31 rows of head_dim elements in all (else
 * Q3TTS_ERR_UNSUPPORTED).
 * Rows outside every sequence's range are left as they were, like the rows of
 * a sequence whose length or offsets do not fit; page ids outside the pool leave
 * the sequence's rows unspecified (both reported in status_dev).  No row of out
 * may share a byte with one of q (Q3TTS_ERR_ARG).  Accumulation in fp32; a row's
 * result does not depend on the run, but may on n_seqs, max_nodes and pages_per_seq,
 * which decide how positions are split: the table's width stands for the lengths,
 * which the host does not know, so a short sequence in a wide table is split as a
 * long one. */
int q3tts_tree_attention(const q3tts_kv_cache* kv, int layer, const int32_t* page_table_dev, int pages_per_seq,
                         int n_seqs, const int32_t* lengths_dev, const int32_t* node_start_dev,
                         const uint64_t* masks_dev, int n_rows, int max_nodes, int n_q_heads, const float* q_dev,
                         int ldq, float* out_dev, int ldo, int32_t* status_dev, void* cuda_stream);

/* Test hook for the attention's failure path: arms the calling thread's next
 * q3tts_tree_attention that reaches the device so that the products of its first
 * CTA are lost from position tile `tile` (0-based, 128 positions each) on, and
 * every wait inside the kernel gives up after about wait_us microseconds.  No GPU
 * fault, trap or endless wait is involved: the waits for those products run out,
 * the CTA records Q3TTS_ERR_TIMEOUT, lets its copies and products in flight land
 * and returns.  A tile past the CTA's last one changes nothing but the limit.
 * Q3TTS_ERR_ARG for tile < 0 or wait_us outside 1..2,000,000. */
int q3tts_debug_lose_tile(int tile, int wait_us);

/* Copies page src[i] to page dst[i] in every layer, i < n (host arrays).
 * Q3TTS_ERR_ARG if an id is outside the pool, a page is written twice, or one
 * is both read and written. */
int q3tts_copy_pages(const q3tts_kv_cache* kv, const int32_t* src, const int32_t* dst, int n, void* cuda_stream);

/* Compacts accepted nodes: for each sequence s and i < path_len_dev[s], the
 * keys and values at position lengths_dev[s] + path[i] move to position
 * lengths_dev[s] + i, in every layer and in place; path is row s of path_dev
 * (int32 [n_seqs][max_path]), ascending and not negative.  A sequence whose
 * entries do not hold to this or to its table is left as it was (reported in
 * status_dev).  No page that is written may belong to two sequences. */
int q3tts_compact_rows(const q3tts_kv_cache* kv, const int32_t* page_table_dev, int pages_per_seq, int n_seqs,
                       const int32_t* lengths_dev, const int32_t* path_dev, int max_path, const int32_t* path_len_dev,
                       int32_t* status_dev, void* cuda_stream);

/* Beam search's selection.  Beam b of group g reads row r = row_ids_dev[g x
 * beams + b] (row_ids_dev NULL: g x beams + b) of logits_dev (fp32 rows of
 * vocab, ld elements apart), of finished_dev (NULL, or uint8 per row) and of
 * history_dev (NULL, or uint8 rows of vocab: the codes the penalty applies to).
 * The logits get the repetition penalty and the mask of special codes (codes
 * from special_from on except eos_token; special_from <= 0: none) as in
 * q3tts_sampling; a NaN logit counts as -INFINITY.  A candidate (b, v) scores
 * scores_dev[g x beams + b] + log softmax(logits of b)[v]; a finished beam
 * offers one, eos_token (which must be a code then) at its own score.  The k
 * best of each group are written in order: tokens_dev, parents_dev (b) and
 * scores_out_dev, [groups][k] each (scores_out_dev may be scores_dev when k ==
 * beams).  Candidates of one beam come in the exact order of their logits.  Scores
 * carry the error of their row's fp32 sum of exponentials, up to about 2^-20, and one
 * rounding: candidates of different beams that are closer than that may come in
 * either order.  Of equal ones the lower beam comes first, then the larger logit
 * (-0 equals +0), then the lower code.  A slot without a candidate above -INFINITY
 * gets token -1, parent 0 and score -INFINITY; a beam whose score is -INFINITY or
 * NaN has none.  beams and k up to Q3TTS_MAX_BEAMS, vocab up to 2^24.  Row ids
 * are not checked.  workspace_dev: device memory, 8-byte aligned, of at least
 * q3tts_beam_workspace_size bytes (on the current device; 0: none is needed, and
 * it may be NULL, or the shape is not taken), whose contents do not matter before and after; calls that may
 * run at the same time need one each. */
size_t q3tts_beam_workspace_size(int groups, int beams, int vocab, int k);
int q3tts_beam_select(const float* logits_dev, size_t ld, const int32_t* row_ids_dev, int groups, int beams, int vocab,
                      const float* scores_dev, const uint8_t* finished_dev, const uint8_t* history_dev, int eos_token,
                      int special_from, float repetition_penalty, int k, int32_t* tokens_dev, int32_t* parents_dev,
                      float* scores_out_dev, void* workspace_dev, size_t workspace_bytes, void* cuda_stream);

/* Per-beam state to be reordered: rows of row_bytes, src_stride and dst_stride
 * bytes apart, in device memory. */
typedef struct q3tts_rows {
  const void* src;
  void* dst;
  size_t row_bytes, src_stride, dst_stride;
} q3tts_rows;

/* Row (g, j) of each set's dst = row (g, parents_dev[g x beams_out + j]) of its
 * src (sets: host array).  Rows are numbered g x beams_in + b in src and g x
 * beams_out + j in dst, or both by row_ids_dev (int32 [groups x beams], then
 * beams_in == beams_out; distinct rows, not checked).  dst is src (in place;
 * strides and beams equal then), or no row of it shares a byte with one of src.
 * The sets of a call may run at once: no row of a dst may share a byte with a row
 * of another set's src or dst, or with parents_dev (Q3TTS_ERR_ARG, where it can be
 * told: under row_ids_dev only for equal strides).  groups x Q3TTS_MAX_BEAMS up
 * to 65535. */
int q3tts_reorder_rows(const q3tts_rows* sets, int n_sets, const int32_t* row_ids_dev, const int32_t* parents_dev,
                       int groups, int beams_in, int beams_out, int32_t* status_dev, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* Q3TTS_BRANCH_H */

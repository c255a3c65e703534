/*
 * q3tts_kv8.h -- C ABI of libq3tts, third part: a paged cache held in 8 bits.
 *
 * Operators for programs that keep their own paged caches (as those of
 * q3tts_branch.h): keys and values are quantised as they are written, read back,
 * and attended over as they lie.  Conventions, status codes and dtypes are
 * q3tts.h's.
 */
#ifndef Q3TTS_KV8_H
#define Q3TTS_KV8_H

#include "q3tts_branch.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The cache: codes is device memory, 16-byte aligned, of
 * [layers][n_pages][k|v][n_kv_heads][page_size][head_dim] FP8 E4M3 codes, powers of
 * [layers][n_pages][k|v][n_kv_heads][page_size / block] E8M0 bytes; head_dim 64
 * or 128, block a divisor of page_size.  The element with code c in a block with
 * byte b is c x 2^(b - 127); a byte of 255 stands for NaN in the whole block.  A
 * sequence's position p is slot p % page_size of page page_table[p / page_size],
 * in every layer.  No block that a call writes may belong to two sequences of it. */
typedef struct q3tts_kv8_cache {
  void* codes;
  void* powers;
  int layers, n_pages, n_kv_heads, page_size, head_dim;
  int block;
} q3tts_kv8_cache;

/* The sequences and rows of a call, in one layer: sequence s holds lengths[s]
 * positions (0 or more), and its rows, row_start[s] .. row_start[s + 1] - 1 of the
 * call's rows, stand at the positions after them in order; max_rows (1 or more)
 * bounds every sequence's count and sizes the launch, as if each had as many: the
 * closer, the faster (a write's and a read's n_seqs x 2 n_kv_heads x its blocks, or
 * sixteens of rows, are 2^31 at most, an attention's n_seqs x n_kv_heads x its tiles
 * of 16 or 128 rows 2^28; else Q3TTS_ERR_UNSUPPORTED).  A table has up to 2^30
 * positions for a sequence (else Q3TTS_ERR_ARG).  page_table (int32
 * [n_seqs][pages_per_seq]), lengths, row_start and status (may be NULL;
 * q3tts_branch.h's status_dev) are device memory; the table's entries past a
 * sequence's last position are not read.  Rows are n_rows of fp32 or bf16 elements
 * (row_dtype: Q3TTS_F32 or Q3TTS_BF16), their pitch (ldk, ldv, ldq, ldo) counted in
 * elements.  A sequence whose length or rows do not fit its table, the rows or
 * max_rows is left out, and page ids outside the pool are not followed (both
 * reported in status). */
typedef struct q3tts_kv8_rows {
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* row_start;
  int32_t* status;
  int layer, pages_per_seq, n_seqs;
  int row_dtype, n_rows, max_rows;
} q3tts_kv8_rows;

/* Quantises the keys and values of new rows (n_rows of n_kv_heads x head_dim
 * elements) and writes them to one layer.  A block's power is the smallest of 2^-127
 * and up that brings the largest finite magnitude of its rows to 448 or below;
 * codes are rounded to the nearest, ties to even; infinities and NaN become NaN
 * and do not count for the power.  In a block whose first rows are positions that
 * the sequence holds already the power does not fall: where it rises, those rows'
 * codes are rounded again to the new one.  Rows of a block behind the last one
 * written are left as they were.  A block on a page outside the pool is left out.
 * Pages of up to 2^31 rows of head_dim elements, blocks of up to 2^31 elements (else
 * Q3TTS_ERR_UNSUPPORTED). */
int q3tts_kv8_write(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows, const void* k_dev, int ldk,
                    const void* v_dev, int ldv, void* cuda_stream);

/* Reads keys and values back into rows, each element rounded once to row_dtype.  Row
 * i of sequence s is position lengths[s] + i, or lengths[s] + path_dev[row]
 * where path_dev (int32 [n_rows]; not negative, any order) is given; an entry
 * outside the sequence's table or on a page outside the pool leaves its row as it
 * was (reported in status), like rows outside every sequence.  With a path,
 * reading the accepted nodes of a drafted tree and writing them as new rows at
 * lengths moves them to the places after the last position held.  No row of
 * k_out may share a byte with one of v_out (Q3TTS_ERR_ARG).  Pages of up to
 * 2^31 rows (else Q3TTS_ERR_UNSUPPORTED). */
int q3tts_kv8_read(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows, const int32_t* path_dev, void* k_out_dev,
                   int ldk, void* v_out_dev, int ldv, void* cuda_stream);

/* Attention of new rows over the cache, in one layer; the rows' own keys and values
 * have been written to it.  q_dev and out_dev: n_rows rows of n_q_heads x head_dim
 * of row_dtype; q head h reads kv head h / (n_q_heads / n_kv_heads), at most 1024
 * of them one; scale 1 / sqrt(head_dim).  A row sees every position held and, of
 * the sequence's new rows, itself and those before it (masks_dev NULL: a prompt's
 * chunk, or one token), or row j if bit j of its mask is set (masks_dev: uint64
 * [n_rows], 8-byte aligned; a drafted tree, max_rows up to
 * Q3TTS_MAX_TREE_NODES).  One that sees nothing gets zeroes.  What a row does not
 * see does not touch it, NaN among it; a row that sees a NaN is unspecified, like
 * one with scores above 2^27, an element of its query times a key block's power above
 * 2^100, or a value block's power above 2^40.  A head's query with an infinity or NaN
 * makes its output NaN, if it sees anything.  Values in blocks whose power is below 2^-40
 * may count as zeroes.  Rows outside every sequence's range are left as they were;
 * page ids outside the pool leave the sequence's rows unspecified.  No row of out may
 * share a byte with one of q (Q3TTS_ERR_ARG).  Caches of up to 2^31 rows of head_dim
 * elements in all (else Q3TTS_ERR_UNSUPPORTED).
 *
 * Scores, softmax statistics and sums are held in 32 bits, a query's elements to
 * 2^-22 of the head's largest.  A weight is a power of two to 2^-22, whose exponent
 * (score and value power less the row's largest) is off by 2^-24 of its size.  It
 * meets the values off by up to 2^-28 of the row's largest weight x value power and
 * 2^-22 of itself (2^-11 where row_dtype is bf16 and the call is one for tiles of 128
 * rows), and is whole in the softmax's sum; the result is rounded once to row_dtype.
 * It does not depend on the run, but may, in its roundings, on n_seqs, max_rows and
 * pages_per_seq, which decide the tiles and how positions are split, and on the other
 * rows of its tile.
 * q3tts_debug_lose_tile arms this call too. */
int q3tts_kv8_attention(const q3tts_kv8_cache* kv, const q3tts_kv8_rows* rows, const uint64_t* masks_dev,
                        const void* q_dev, int ldq, void* out_dev, int ldo, int n_q_heads, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* Q3TTS_KV8_H */

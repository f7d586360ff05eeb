/*
 * tm_attention.h -- C ABI of the attention window's operators on MI355X
 * (gfx950): rotary positions, a paged key/value cache held in 8 bits, the
 * attention that reads it, and the housekeeping of its pages.
 *
 * Memory as a context runs attention over a window of persistent tokens, the
 * memory's recalled vectors and the segment (tm_mac_window in tm.h, which
 * leaves that attention to the caller).  These calls are such an attention,
 * for whole segments and for single tokens; they need no tm_ctx.  They live
 * in the same library and follow tm.h's conventions: caller-owned device
 * memory, asynchronous on `stream`, a tm_status from every call, argument
 * checks on the host before anything is launched.
 *
 * Tensors.  Token arrays are [batch][n_tokens][heads][head_dim] of bf16 or
 * fp32 (tm_dtype).  The last two axes are contiguous; the distances between
 * batch entries and between tokens are given in elements (so that queries,
 * keys and values may be views of one projection's output).  Token arrays
 * are 16-byte aligned and their distances are multiples of 8 elements
 * (tm_rotary takes any).  A call whose launch would have 2^32 threads or
 * more along an axis is refused (TM_ERR_INVALID).
 *
 * The cache.  A cache holds n_seqs sequences of up to seq_pages * 64 tokens
 * in n_pages pages of 64 tokens, in one caller-owned blob of
 * tm_cache_bytes bytes, 256-byte aligned, with these regions in this order,
 * each 256-byte aligned (tm_cache_layout gives their offsets):
 *   meta    int32: status [64], lengths [n_seqs], refs [n_pages] (how many
 *           table entries hold the page; 0: the page is free), table
 *           [n_seqs][seq_pages] (page i of a sequence holds its tokens
 *           64 i ..; entries behind its last page mean nothing)
 *   scales  uint8 [n_pages][kv_heads][2 (keys, values)][4]: e + 127 of the
 *           power of two 2^e that each block of 16 tokens is scaled by
 *   keys    e4m3 (4-bit exponent, 3-bit mantissa, largest value 448)
 *           [n_pages][kv_heads][64][head_dim]
 *   values  e4m3 [n_pages][kv_heads][head_dim][64] (tokens innermost)
 * A copy of meta is a snapshot of the sequences' bookkeeping.  status[0]
 * holds sticky flags (below); status[1] and status[2] are the calls' own: 0 in a
 * new cache, and status[2] is 0 between calls, in a blob or a snapshot that is
 * given back too (an append that finds it otherwise sets TM_CACHE_BAD_ENTRY,
 * and the bookkeeping and codes mean nothing until tm_cache_init).
 * Quantisation: a block's exponent is the least e in [-110, 119] with
 * max |x| <= 448 2^e over its tokens, a code is x 2^-e rounded to nearest
 * even.  A block that is appended to keeps the larger of its exponent and
 * the new tokens'; where it grows, the codes it held are rounded to the new
 * scale (exactly, but for those that become subnormal: scales are powers of
 * two).  An element beyond 448 * 2^119 (2.98e38) is held as that.  A
 * non-finite element of k or v is held as zero and sets TM_CACHE_NONFINITE.
 * Pages.  Sequences may share pages (tm_cache_fork); a call never writes to
 * a page that others hold too: tm_cache_append first gives the sequence a
 * copy of a shared last page.  Pages are handed out the lowest free one
 * first, in the order of the call's entries, so the bookkeeping does not
 * depend on how a call was scheduled.
 * Lists of sequences.  seqs, src, dst: device int32, values in [0, n_seqs);
 * seqs null means 0, 1, 2, ...  counts: device int32 [batch], tokens of each
 * entry (clamped to 0 .. n_tokens), null: n_tokens each.  The host cannot
 * see these values; an entry that cannot be served is left out, alone, and
 * sets a flag.  Everything a kernel reads from the blob or from a list is
 * checked there before it is used as an index.
 * Concurrency: calls that write a cache are ordered by the caller; reads of
 * it (attend, read) may run at the same time, with workspaces of their own.
 * The handle is immutable and may be shared between threads.
 */
#ifndef TM_ATTENTION_H
#define TM_ATTENTION_H

#include "tm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- rotary positions ---- */

typedef enum {
    TM_ROPE_HALF = 0,         /* pair i is (x[i], x[i + rot_dim / 2]) */
    TM_ROPE_INTERLEAVED = 1   /* pair i is (x[2 i], x[2 i + 1]) */
} tm_rope_layout;

typedef enum {
    TM_ROPE_NONE = 0,
    TM_ROPE_LINEAR = 1,   /* every frequency divided by factor */
    TM_ROPE_BASE = 2,     /* base raised to base * factor^(rot_dim / (rot_dim - 2)) (rot_dim > 2) */
    TM_ROPE_PARTS = 3     /* by wavelength: pairs that turn at least beta_fast times within original_len
                             positions keep their frequency, those that turn at most beta_slow times are
                             divided by factor, and between them the share goes linearly with the pair's
                             index, from the last whole index that turns beta_fast times to the first
                             that turns beta_slow times (wherever those lie: no pair need turn so much or
                             so little); *result_scale = 0.1 ln(factor) + 1 for factor > 1 */
} tm_rope_scaling;

/* Host only: freq [rot_dim / 2] = base^(-2 i / rot_dim), scaled as `scaling`
 * says (factor > 0; original_len, beta_fast > beta_slow > 0 for
 * TM_ROPE_PARTS), and the factor the rotated elements take (1 unless
 * TM_ROPE_PARTS).  rot_dim: even, 2 .. 1024; base > 1; a scaled base or a
 * frequency that would overflow is refused. */
tm_status tm_rotary_frequencies(int rot_dim, double base, tm_rope_scaling scaling, double factor,
                                double original_len, double beta_fast, double beta_slow, double* freq,
                                double* result_scale);

/* Rotates each pair i of the first rot_dim elements of every head vector by
 * the angle position * freq[i] and multiplies it by result_scale:
 *   (a, b) -> result_scale (a cos - b sin, a sin + b cos);
 * the elements behind rot_dim are copied.  inverse != 0 rotates by the
 * negative angle: the gradient with respect to x of a call with inverse = 0
 * (the transpose of result_scale times a rotation).  Angles are formed and
 * reduced in 64 bits, so positions up to the range of int32 keep their
 * accuracy; the rotation is fp32, rounded once to the dtype.
 * positions: device int32, [batch][n_tokens] (per_token != 0), or [batch]
 * (per_token == 0: token t of entry b stands at positions[b] + t).  freq:
 * device fp64 [rot_dim / 2].  y may be x (with the same distances); it must
 * not overlap it otherwise.  head_dim 1 .. 1024, rot_dim even, 2 ..
 * head_dim.  x, y: aligned to their element type.  batch * n_tokens == 0 is
 * a no-op. */
tm_status tm_rotary(const void* x, long x_batch, long x_token, void* y, long y_batch, long y_token,
                    const int* positions, int per_token, const double* freq, double result_scale, int batch,
                    int n_tokens, int heads, int head_dim, int rot_dim, tm_rope_layout layout, int inverse,
                    tm_dtype dtype, void* stream);

/* ---- the cache ---- */

#define TM_CACHE_PAGE 64    /* tokens of a page */
#define TM_CACHE_BLOCK 16   /* tokens of a block with one scale */

/* status[0] of a cache: sticky until tm_cache_init */
#define TM_CACHE_NONFINITE 1   /* a non-finite key or value was held as zero */
#define TM_CACHE_NO_PAGES 2    /* an append was left out: not enough free pages */
#define TM_CACHE_FULL 4        /* an append was left out: longer than seq_pages * 64 tokens */
#define TM_CACHE_BAD_ENTRY 8   /* an entry was left out: a sequence out of range or listed before in the
                                  call, a fork into a sequence that is not empty, a table entry out of range;
                                  or an append found status[2] other than 0 */

typedef struct tm_cache tm_cache;

/* kv_heads 1 .. 1024; head_dim a multiple of 32, 32 .. 256; n_pages 1 ..
 * 2^24; n_seqs 1 .. 8192; seq_pages 1 .. 2^20 (n_seqs * seq_pages at most
 * 2^30).  On success *out owns a handle to release with tm_cache_destroy. */
tm_status tm_cache_create(int kv_heads, int head_dim, int n_pages, int n_seqs, int seq_pages, tm_cache** out);
void tm_cache_destroy(tm_cache* cache);

/* Bytes of the blob, and the offsets of meta, scales, keys and values in it. */
size_t tm_cache_bytes(const tm_cache* cache);
tm_status tm_cache_layout(const tm_cache* cache, size_t offsets[4]);

/* All sequences empty, all pages free, flags cleared (the codes are not
 * touched). */
tm_status tm_cache_init(const tm_cache* cache, void* blob, void* stream);

/* Workspace bytes of tm_cache_append, tm_cache_compact, and of
 * tm_cache_attend for a call of `batch` entries of n_tokens query tokens of
 * `heads` heads (heads 0: append and compact only).  256-byte aligned, holds
 * no data between calls. */
size_t tm_cache_workspace_bytes(const tm_cache* cache, int batch, int n_tokens, int heads);

/* Writes counts[b] tokens of k and v [batch][n_tokens][kv_heads][head_dim]
 * behind the tokens that sequence seqs[b] holds.  Pages are taken as needed.
 * An entry whose pages do not suffice, counted with those of the entries
 * before it, is left out (TM_CACHE_NO_PAGES), as is one that would grow
 * beyond seq_pages * 64 tokens (TM_CACHE_FULL), and the second of two equal
 * ones (TM_CACHE_BAD_ENTRY).  batch at most n_seqs; n_tokens above
 * seq_pages * 64 needs counts (TM_ERR_INVALID).  batch * n_tokens == 0 is a
 * no-op. */
tm_status tm_cache_append(const tm_cache* cache, void* blob, const int* seqs, const int* counts, const void* k,
                          long k_batch, long k_token, const void* v, long v_batch, long v_token, int batch,
                          int n_tokens, tm_dtype dtype, void* workspace, void* stream);

/* out[b][i][h] = sum_j p_j v_j, p = softmax over the visible tokens j of
 * score_scale * (q[b][i][h] . k_j), keys and values of head h / (heads /
 * kv_heads) of sequence seqs[b].  The counts[b] query tokens are the last of
 * the sequence (which holds their keys already): query i stands at position
 * length - counts[b] + i and sees the tokens j at or before it, with
 * window > 0 only the `window` last of them and the first `sink` of the
 * sequence.  A query that sees nothing (a sequence shorter than counts[b],
 * one out of range) gives zeros; rows i >= counts[b] of out are left as they
 * were.  A page whose table entry is out of range counts as not visible.
 * heads: a multiple of kv_heads, at most 64 * kv_heads.  out: contiguous
 * [batch][n_tokens][heads][head_dim] of dtype; it may be q, if q is contiguous,
 * and must not overlap it otherwise.  Products of bf16 calls are
 * of bf16 operands with fp32 accumulation (the cache's values are exact in
 * bf16; the softmax weights keep 16 bits where n_tokens * heads / kv_heads is
 * at most 64, and are rounded to bf16 above), those of fp32 calls keep 24
 * bits of q and of the weights; statistics are fp32.
 * max_len: at least the longest listed sequence's length lets the call
 * choose its launch (0: seq_pages * 64); results are right whatever it is.
 * The result of a row does not depend on the other rows of the call, but may
 * depend on batch, n_tokens and max_len in its rounding (how the sequence is
 * divided). */
tm_status tm_cache_attend(const tm_cache* cache, const void* blob, const int* seqs, const int* counts,
                          const void* q, long q_batch, long q_token, void* out, int batch, int n_tokens, int heads,
                          float score_scale, int window, int sink, int max_len, tm_dtype dtype, void* workspace,
                          void* stream);

/* The tokens start .. start + n_tokens - 1 of each sequence as the values
 * their codes stand for (rounded to dtype; exact in both), k and v contiguous
 * [batch][n_tokens][kv_heads][head_dim]; rows behind a sequence's end are
 * left as they were. */
tm_status tm_cache_read(const tm_cache* cache, const void* blob, const int* seqs, int start, void* k, void* v,
                        int batch, int n_tokens, tm_dtype dtype, void* stream);

/* dst[i] becomes a copy of sequence src[i] that shares its pages.  dst[i]
 * must be empty and listed once; sources are read as they were before the
 * call.  An entry whose dst is not empty or listed before, or whose src is
 * listed as a dst, is left out (TM_CACHE_BAD_ENTRY).  n at most n_seqs. */
tm_status tm_cache_fork(const tm_cache* cache, void* blob, const int* src, const int* dst, int n, void* stream);

/* Drops the tokens from keep[i] (device int32; null: 0) on of sequence
 * seqs[i]; pages that no sequence holds any more become free.  Listing a
 * sequence twice is the first entry's call (TM_CACHE_BAD_ENTRY). */
tm_status tm_cache_free(const tm_cache* cache, void* blob, const int* seqs, const int* keep, int n, void* stream);

/* Moves the pages in use to the lowest numbers: with U pages in use, the
 * i-th used page at or above U moves to the i-th free page below U, and the
 * tables follow.  Afterwards the pages U .. are free. */
tm_status tm_cache_compact(const tm_cache* cache, void* blob, void* workspace, void* stream);

/* Synchronous: waits for `stream`, then reports the sticky flags and the
 * number of pages in use (either pointer may be null). */
tm_status tm_cache_check(const tm_cache* cache, const void* blob, int* flags, int* pages_used, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TM_ATTENTION_H */

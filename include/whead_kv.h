/*
 * whead_kv.h — C ABI of the paged KV cache held in 4 bits that stands beside the serial draft head (sm_103a).
 *
 * A draft walk returns gamma tokens; verifying them takes the target model's attention over what is cached, with
 * gamma + 1 query tokens a sequence, and afterwards the rejected tokens leave the cache and candidates are forked or
 * dropped. These calls hold that cache: whead_kv_append quantizes keys and values into pages, whead_kv_attend
 * reads them, whead_kv_compact keeps the accepted tokens of a block, whead_kv_fork lets sequences take over one
 * another's pages, whead_kv_read gives back the values that are held.
 *
 * Format. A value is code * s * g: an e2m1 code (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6; bit 3 is the sign), an e4m3
 * scale s for each 16 channels of a token, an fp32 scale g for each KV head (k_scale, v_scale; > 0, the caller's,
 * fixed for the cache's life). A page holds page_size tokens of every KV head. The pool is
 *   num_pages x kv_heads x (page_size / 16) groups of 18 * head_dim bytes,
 * a group being 16 tokens of one head, in the order in which a warp's lanes take them as operands of a 16 x 8 x 16
 * matrix product. With r the token in the group, g = r % 8, hi = r / 8, c the channel, b = c / 16, u = c % 16:
 *   keys' codes    byte (b/4)*512 + (4*g + u/4)*16 + (b%4)*4 + (u%4/2)*2 + hi, low nibble for even u
 *   keys' scales   byte 8*head_dim + g*(head_dim/8) + b*2 + hi
 *   values' codes  byte 9*head_dim + (b/4)*512 + (4*(u/2) + (r%8)/2)*16 + (b%4)*4 + hi*2 + u%2, low nibble for even r
 *   values' scales byte 17*head_dim + ((r%8)/2)*(head_dim/4) + b*4 + hi*2 + r%2
 *
 * Quantization of 16 channels x: s = E4M3(max|x| / (6 g)) to nearest even, saturated at 448; inv = 1 / (s g) in fp32;
 * each code is e2m1(x inv) to nearest even, saturated at 6. A NaN is held as zero, an infinity as the largest value.
 *
 * State, all int32 on the device: lens[max_seqs] (tokens held by each slot), refs[num_pages] (how many slots hold a
 * page; 0: free), tables[max_seqs x max_pages] (the slots' pages, -1 past their ends). An empty cache is all zeros, and
 * -1 in tables. Calls that need pages take the free ones of the lowest index, in the order of their entries and of
 * positions; pages that a call gives up are free for the next call. The last page of a slot, where it is not full, is
 * held by that slot alone: fork and compact copy it, so that append never writes a page that is shared.
 *
 * Conventions as in whead.h: device pointers, borrowed for the call; calls are asynchronous on kv->stream; return codes
 * are WHEAD_OK or WHEAD_ERR_*. Calls on one cache share its workspace and have to be ordered on one stream (or by events).
 * What only the device can see (a pool that runs out, a slot or position out of range) is reported by whead_kv_status:
 * such an append, compact or fork changes nothing at all, and an attend or read treats the slot as empty.
 * Two entries of one call must not name the same slot. No call allocates device memory; all can be captured in a graph.
 */
#ifndef WHEAD_KV_H_
#define WHEAD_KV_H_

#include "whead.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { WHEAD_KV_BF16 = 0, WHEAD_KV_F16 = 1, WHEAD_KV_F32 = 2 } whead_kv_dtype;

typedef struct {
  int32_t page_size;     /* tokens of a page: 16, 32, 64 or 128 */
  int32_t kv_heads;      /* 1..1024 */
  int32_t head_dim;      /* 64, 128 or 256 */
  int32_t max_seqs;      /* slots: 1..4096 */
  int32_t max_pages;     /* most pages of a slot; max_pages * page_size <= 2^31 - 1024 */
  int32_t num_pages;     /* pages of the pool */
  void* pool;            /* 16-byte aligned */
  int32_t* lens;
  int32_t* refs;
  int32_t* tables;
  const float* k_scale;  /* kv_heads fp32, > 0 */
  const float* v_scale;  /* kv_heads fp32, > 0 */
  void* workspace;       /* 256-byte aligned, whead_kv_workspace_bytes, zeroed before the first call */
  int64_t workspace_bytes;
  void* stream;          /* cudaStream_t; NULL = legacy default stream */
} whead_kv;

/* Bytes of one page, or WHEAD_ERR_UNSUPPORTED. */
int64_t whead_kv_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim);

/* Bytes of workspace for a cache of this shape (pointers are not looked at), or an error code. */
int64_t whead_kv_workspace_bytes(const whead_kv* kv);

/*
 * Appends tokens: entry i's are rows indptr[i] .. indptr[i+1] - 1 of k and v and go to the end of slot slots[i]
 * (slots NULL: slot i; indptr NULL: total / n tokens each). k and v: total x kv_heads x head_dim of `dtype`, channels
 * contiguous, the other strides in elements. Quantizes, takes pages as they are needed, sets lens.
 * Device errors: WHEAD_ERR_NO_PAGES (the pool or a table's row is full), WHEAD_ERR_INVALID_ARG.
 */
int whead_kv_append(const whead_kv* kv, const void* k, const void* v, int32_t dtype, int64_t k_token_stride,
                    int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t* indptr,
                    const int32_t* slots, int32_t n, int64_t total);

/*
 * The held values of `count` tokens from position start[i] >= 0 of each entry's slot, rounded once to `dtype`:
 * k_out, v_out: n x count x kv_heads x head_dim, contiguous, 16-byte aligned; zeros past a slot's length.
 */
int whead_kv_read(const whead_kv* kv, const int32_t* start, const int32_t* slots, int32_t n, int32_t count,
                  int32_t dtype, void* k_out, void* v_out);

typedef struct {
  const void* q;            /* total x heads x head_dim of `dtype`, channels contiguous */
  void* out;                /* total x heads x head_dim of `dtype`, contiguous, 16-byte aligned */
  float* lse;               /* total x heads, or NULL: log of the sum of exp of the scaled scores, -inf for none */
  const int32_t* indptr;    /* n + 1 offsets of the entries' query tokens, or NULL: total / n each */
  const int32_t* slots;     /* the entries' slots, or NULL: slot i */
  const uint64_t* tree;     /* NULL, or total x tree_words masks over an entry's own tokens (needs causal) */
  int64_t total;            /* query tokens */
  int64_t q_token_stride, q_head_stride; /* in elements */
  int32_t n;                /* entries */
  int32_t heads;            /* query heads, a multiple of kv_heads; head a reads KV head a / (heads / kv_heads) */
  int32_t max_q;            /* no entry may have more query tokens than this */
  int32_t dtype;            /* WHEAD_KV_BF16 or WHEAD_KV_F16, for q and out */
  int32_t causal;
  int32_t window;           /* 0, or the number of latest keys that a token sees (needs causal) */
  int32_t tree_words;       /* 64-bit words of a token's mask: 64 * tree_words >= max_q */
  float scale;              /* of the scores q . k */
} whead_kv_attend_args;

/*
 * Attention of each entry's query tokens over its slot's keys and values. With T query tokens and length L, query t
 * stands at position p = L - T + t, so that append comes before attend. It sees the keys j < L, and of those, with
 * causal, j <= p; with a window, j > p - window; with a tree, for j >= L - T, those whose bit j - (L - T) is set in its
 * mask. A query that sees none gives zeros and lse -inf. Scores, which may be of any finite size, maxima, exponentials and sums
 * are in fp32; the exponentials are rounded to f16 (2^-11 at most) where they meet the values.
 * Device errors: WHEAD_ERR_INVALID_ARG for an entry whose offsets are out of order or past total, or that has more than max_q
 * tokens (its rows of out and lse are not written, nor are rows that belong to no entry), and for a slot that is none.
 */
int whead_kv_attend(const whead_kv* kv, const whead_kv_attend_args* args);

/*
 * Keeps part of a block at a slot's end: of the tokens from position start[i] on, those at start[i] + keep[i][j],
 * j < count[i], move to start[i] + j; the length becomes start[i] + count[i] and pages past it lose this slot's
 * reference. keep: n x keep_width, each row's first count[i] offsets ascending and below lens - start; offsets
 * are at most WHEAD_KV_MAX_BLOCK - 1. count[i] = 0 cuts the slot at start[i] (NULL keep and count: for all). keep may be
 * NULL where keep_width is 0.
 * Device errors: WHEAD_ERR_NO_PAGES, WHEAD_ERR_INVALID_ARG.
 */
#define WHEAD_KV_MAX_BLOCK 256
int whead_kv_compact(const whead_kv* kv, const int32_t* start, const int32_t* keep, const int32_t* count,
                     const int32_t* slots, int32_t n, int32_t keep_width);

/*
 * Slot i takes over the sequence that slot parents[i] held before the call: i itself leaves it as it is, -1 empties
 * it. Full pages are shared, a partial last page is copied. parents: max_seqs int32.
 * Device errors: WHEAD_ERR_NO_PAGES, WHEAD_ERR_INVALID_ARG.
 */
int whead_kv_fork(const whead_kv* kv, const int32_t* parents);

/* Waits for the stream and returns WHEAD_OK or the first device-side error since the last whead_kv_status. */
int whead_kv_status(const whead_kv* kv);

#ifdef __cplusplus
}
#endif

#endif /* WHEAD_KV_H_ */

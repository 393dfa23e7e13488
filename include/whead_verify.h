/*
 * whead_verify.h — C ABI of what follows the target's forward pass in a verification step (sm_103a): what its logits say
 * about the drafts of a walk.
 *
 * whead_verify decides which drafts stay and draws the token after them; its counts are those that whead_kv_compact takes.
 * whead_logprobs gives log probabilities of given tokens, with the rows' entropy and top alternatives.
 *
 * Rows of logits lie in n x t x V (t = 1 for a plain list of rows), the V values of a row next to one another, the other
 * strides in elements and free. A row's distribution at temperature T is p(v) = exp(x_v / T - lse), lse = log sum_v exp(x_v / T):
 * logits of -inf are tokens that cannot be, any finite logit is taken as it is (the type's lowest value too). A row that holds NaN or
 * +inf has no distribution, nor has one of nothing but -inf; each call says what it gives for those.
 *
 * Conventions as in whead.h: device pointers, borrowed for the call; calls are asynchronous on `stream`; return codes are
 * WHEAD_OK or WHEAD_ERR_*. Calls share nothing but the workspace that they are given, allocate nothing and can be captured in a graph.
 * Sums, maxima and exponentials are in fp32.
 */
#ifndef WHEAD_VERIFY_H_
#define WHEAD_VERIFY_H_

#include "whead.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of logits. */
typedef enum { WHEAD_BF16 = 0, WHEAD_F16 = 1, WHEAD_F32 = 2 } whead_dtype;

#define WHEAD_MAX_TOP 32

typedef struct {
  const void* logits;      /* n x t x V of `dtype` */
  const int32_t* tokens;   /* n x t, contiguous, or NULL with logprob NULL */
  float* logprob;          /* n x t: log p(token); -inf for a token outside 0..V-1 */
  float* entropy;          /* n x t: -sum p log p; 0 for a row of nothing but -inf */
  float* lse;              /* n x t; -inf for a row of nothing but -inf */
  int32_t* top_tokens;     /* n x t x top, best first (equal logits: the lower token first); -1 past the tokens that can be */
  float* top_logprobs;     /* n x t x top; -inf past the tokens that can be */
  int64_t stride_n, stride_t;
  int64_t n, t;            /* n * t < 2^27 */
  int64_t V;               /* 1 <= V < 2^24 */
  double temperature;      /* > 0 */
  int32_t dtype;
  int32_t top;             /* 0..WHEAD_MAX_TOP */
  void* stream;            /* cudaStream_t; NULL = legacy default stream */
} whead_logprobs_args;

/* A row that holds NaN or +inf gives NaN for every number and -1 for every token. */
int whead_logprobs(const whead_logprobs_args* args);

#define WHEAD_MAX_DRAFTS 255

typedef struct {
  const void* target;      /* n x (gamma + 1) x V of target_dtype: row t says what follows the first t drafts */
  const void* draft;       /* n x gamma x V of draft_dtype: the logits that the drafts were drawn from; NULL: they were not drawn */
  const int32_t* tokens;   /* n x gamma drafts, contiguous */
  const int32_t* drafted;  /* n: how many of its gamma drafts an entry has (less than 0 counts as 0, more than gamma as gamma), or NULL: all */
  int32_t* said;           /* n x (gamma + 1): the drafts that stay, the token after them, -1 for the rest */
  int32_t* count;          /* n: 1 + how many drafts stay */
  int64_t target_stride_n, target_stride_t, draft_stride_n, draft_stride_t;
  int64_t n;               /* n * (2 gamma + 2) < 2^27 */
  int64_t V;               /* 1 <= V < 2^24 */
  int32_t gamma;           /* 0..WHEAD_MAX_DRAFTS */
  int32_t target_dtype, draft_dtype;
  uint32_t step;           /* the call's draws have the numbers step .. step + gamma, for all its entries: they only have to be fresh for `seed` */
  double temperature;      /* of the target: 0, or > 0 */
  double draft_temperature;/* > 0: of the drafts' logits */
  uint64_t seed;
  void* workspace;         /* 16-byte aligned, whead_verify_workspace_bytes; its contents do not matter */
  int64_t workspace_bytes;
  void* stream;
} whead_verify_args;

/*
 * Temperature 0: draft t stays if it is the target's largest logit (the lowest token of equal ones) and all before it stay; the token
 * after them is that of the first row whose draft does not stay, or of row gamma. `draft` is not looked at.
 * Above 0, with p the target's distribution and q the drafts' (without `draft`: all on the draft): draft t stays if all before it do and
 * U_t q(x_t) < p(x_t). In the first row whose draft does not stay the token after it is drawn from max(p - q, 0) (from p, where
 * rounding leaves nothing of that), in the row after the last draft from p; so that every token is one of the target's distribution.
 * It is the token of the largest p_v / E_v, E_v = -log U_v, equal ones: the lowest. p and q are exact but for fp32's sums and exponentials, some
 * 2^-20: what is decided by less than that (of p, not of p - q) may go either way, the same way whenever the same call is made.
 * U = ((w >> 9) + 0.5) 2^-23 from words of Philox4x32-10 with key `seed` and counters (v / 4, step + t, i, 1), word v % 4, for the token
 * after entry i's drafts in row t, and (0, step + t, i, 2), word 0, for draft t (sums modulo 2^32): apart from the walk's own, whose last
 * word is 0.
 * A draft that is no token of 0..V-1 does not stay, nor one whose row of `draft` has no distribution (the next token is then drawn
 * from p). In a row of `target` without a distribution no draft stays and the token after is -1.
 */
int64_t whead_verify_workspace_bytes(int64_t n, int32_t gamma);
int whead_verify(const whead_verify_args* args);

#ifdef __cplusplus
}
#endif

#endif /* WHEAD_VERIFY_H_ */

// verify_logprobs.cu — log probabilities of given tokens, entropy and top alternatives of rows of logits, in one pass over the logits.
//
// With d_v = (x_v - m) log2(e) / T, m the row's largest: s = sum 2^d, a = sum d 2^d; lse = m / T + ln s, log p(v) = ln 2 (d_v - log2 s),
// H = ln 2 (log2 s - a / s), whose two terms have one sign. Every thread has a running m of its own (verify_common.cuh).
//
// Alternatives. The pass keeps the largest value of every group (1 KB of the row) in shared memory. The `top` best
// tokens lie in the `top` groups that come first by (largest value, index): were one outside them, each of them would have a token that
// comes before it. So once the pass has ended, those groups are found, read again, and their values ranked: work that does
// not depend on the order of the logits, where lists kept in the pass would.
#include "verify_common.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

namespace whead_verify_impl {

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxRuns = 4224;  // largest values kept by a CTA: of groups, or of runs of 2^shift groups in rows of more (2^24 logits: shift 4)
constexpr int kCandidates = 512;

struct LogprobArgs {
  const void* logits;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_tokens;
  float* top_logprobs;
  int64_t stride_n, stride_t;
  int t, V, top, ctas, shift, runs;  // runs: room for largest values
  float c;
  double inverse;  // 1 / T
};

struct Shared {
  Sums part[kWarps];
  float part_top[kWarps];
  Sums mine;          // the CTA's, for the cluster
  float mine_top;
  int found;          // candidates
  int picked;         // what pick() found: how many keys, their indexes, the bound
  int order[WHEAD_MAX_TOP];
  uint32_t bound;
  int group[WHEAD_MAX_TOP];
  unsigned long long best[WHEAD_MAX_TOP];                          // the CTA's, in order: key, then the complement of the token; 0: none
  unsigned long long all[kMaxCluster * WHEAD_MAX_TOP];             // the cluster's
  unsigned long long candidate[kCandidates];
  uint32_t key[WHEAD_MAX_TOP * kGroup];                              // largest values of the picked groups' vectors, or of the picked runs' groups
};

// Of n keys in shared memory the `top` first by (key, index), by one warp: their indexes, ascending, into `list`, and how many they
// are. Returns a bound that all of them reach and none of those left out passes (0 where none is left out). Bit by bit, from the highest,
// the largest bound that `top` keys reach; ends early where exactly `top` do.
template <int BITS>
__device__ uint32_t pick(const uint32_t* keys, int n, int top, int* list, int* picked) {
  const int lane = threadIdx.x & 31;
  uint32_t bound = 0;
  int above = 0;  // keys above the bound, where it is one of them
  bool exact = n <= top;
  for (int bit = BITS - 1; bit >= 0 && !exact; --bit) {
    const uint32_t next = bound | 1u << bit;
    int count = 0;
    for (int i = lane; i < n; i += 32) count += keys[i] >= next;
    count = __reduce_add_sync(~0u, count);
    if (count >= top) bound = next;
    else above = count;
    exact = count == top;
  }
  int ties = exact ? n : top - above, out = 0;
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    const uint32_t key = i < n ? keys[i] : 0;
    const bool reach = i < n && key >= bound, tie = reach && !exact && key == bound;
    const unsigned tied = __ballot_sync(~0u, tie), before = (1u << lane) - 1;
    const bool take = reach && (!tie || __popc(tied & before) < ties);
    const unsigned taken = __ballot_sync(~0u, take);
    if (take) list[out + __popc(taken & before)] = i;
    out += __popc(taken);
    ties -= min(ties, __popc(tied));
  }
  if (lane == 0) *picked = out;
  __syncwarp();
  return bound;
}

template <int DT>
__device__ __forceinline__ void offer(Shared& s, const uint4& raw, int j, const Row& row, uint32_t bound) {
  constexpr int N = Type<DT>::kPer;
  float x[N];
  values_of<DT>(raw, x);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const uint32_t key = key_of<DT>(x[k]);
    if (key >= bound && key > Type<DT>::kNoneKey) {
      const int at = atomicAdd(&s.found, 1);
      if (at < kCandidates) s.candidate[at] = (unsigned long long)key << 32 | (uint32_t)~(uint32_t)(j * N + k - row.off);
    }
  }
}

template <int DT, bool TOP>
__global__ void __launch_bounds__(kThreads, 6) logprobs_rows(const __grid_constant__ LogprobArgs a) {
  after_previous();
  constexpr int BITS = Type<DT>::kKeyBits;
  __shared__ Shared s;
  extern __shared__ uint32_t runs[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / a.ctas, rank = blockIdx.x - r * a.ctas;
  const int i = r / a.t, t = r - i * a.t;
  const int64_t at = i * a.stride_n + t * a.stride_t;
  const Row row = row_at<DT>(a.logits, at, a.V);
  const int groups = row_groups<DT>(row), g0 = run_begin(groups, a.ctas, rank), g1 = run_begin(groups, a.ctas, rank + 1);
  const int n_runs = g1 > g0 ? ((g1 - 1) >> a.shift) - (g0 >> a.shift) + 1 : 0;
  if (TOP) {
    if (a.shift) {
      for (int k = tid; k < n_runs; k += kThreads) runs[k] = 0;
    }
    if (tid == 0) s.found = 0;
    if (tid < WHEAD_MAX_TOP) s.best[tid] = 0;
    __syncthreads();
  }
  int token = -1;
  float x_token = -INFINITY;
  if (rank == 0 && tid == 0 && a.tokens) {
    token = __ldg(a.tokens + r);
    if ((unsigned)token < (unsigned)a.V) x_token = load_one(a.logits, at + token, DT);
  }
  // ---- the pass
  Pass p;
  begin(p);
  over_groups<DT>(row, g0, g1, [&](int g, const uint4& v, const uint4& w) {
    const float high = fmaxf(largest<DT>(v), largest<DT>(w));
    take<DT, true>(p, v, w, high, a.c);
    if (TOP) {
      const float most = warp_max(high);
      if (lane == 0) {
        if (a.shift) atomicMax(&runs[(g >> a.shift) - (g0 >> a.shift)], key_of<DT>(most));
        else runs[g - g0] = __float_as_uint(most);
      }
    }
  });
  {
    float top;
    const Sums w = warp_joined(p, a.c, top);
    if (lane == 0) {
      s.part[warp] = w;
      s.part_top[warp] = top;
    }
  }
  __syncthreads();
  float top = s.part_top[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s.part_top[w]);
  Sums sums = moved(s.part[0], top, a.c);
#pragma unroll
  for (int w = 1; w < kWarps; ++w) {
    const Sums part = moved(s.part[w], top, a.c);
    sums.s += part.s;
    sums.a += part.a;
  }
  // ---- the CTA's best tokens
  if (TOP) {
    if (!a.shift) {
      for (int k = tid; k < n_runs; k += kThreads) runs[k] = key_of<DT>(__uint_as_float(runs[k]));
      __syncthreads();
    }
    auto choose = [&](const uint32_t* keys, int n) {
      if (warp == 0) {
        const uint32_t bound = pick<BITS>(keys, n, a.top, s.order, &s.picked);
        if (lane == 0) s.bound = bound;
      }
      __syncthreads();
    };
    auto key_at = [&](int j) { return key_of<DT>(largest<DT>(load_vector<DT>(row, j))); };
    // the groups
    choose(runs, n_runs);
    const int first = (g0 >> a.shift) << a.shift;
    if (tid < s.picked) s.group[tid] = first + (s.order[tid] << a.shift);
    __syncthreads();
    if (a.shift) {  // of the picked runs of groups
      const int n = s.picked << a.shift, mask = (1 << a.shift) - 1;
      for (int e = warp; e < n; e += kWarps) {
        const int g = s.group[e >> a.shift] + (e & mask);
        const bool mine = g >= g0 && g < g1;
        const uint32_t key = mine ? __reduce_max_sync(~0u, max(key_at(g * kGroup + lane), key_at(g * kGroup + 32 + lane))) : 0;
        if (lane == 0) s.key[e] = key;
      }
      __syncthreads();
      choose(s.key, n);
      const int g = tid < s.picked ? s.group[s.order[tid] >> a.shift] + (s.order[tid] & mask) : 0;
      __syncthreads();
      if (tid < s.picked) s.group[tid] = g;
      __syncthreads();
    }
    // their values that reach the bound, where that is one and they are not too many
    uint32_t bound = s.bound;
    const int picked = s.picked;
    if (bound > Type<DT>::kNoneKey) {
      for (int e = warp; e < 2 * picked; e += kWarps) {
        const int j = s.group[e / 2] * kGroup + e % 2 * 32 + lane;
        const uint4 raw = load_vector<DT>(row, j);
        if (key_of<DT>(largest<DT>(raw)) >= bound) offer<DT>(s, raw, j, row, bound);
      }
    }
    __syncthreads();
    if (bound <= Type<DT>::kNoneKey || s.found > kCandidates) {
      // the same step once more, with the groups' vectors in the groups' place: the best tokens lie in no more vectors than they are
      for (int e = tid; e < picked * kGroup; e += kThreads) s.key[e] = key_at(s.group[e / kGroup] * kGroup + e % kGroup);
      __syncthreads();
      if (tid == 0) s.found = 0;
      choose(s.key, picked * kGroup);
      bound = s.bound;
      if (tid < s.picked) {
        const int j = s.group[s.order[tid] / kGroup] * kGroup + s.order[tid] % kGroup;
        offer<DT>(s, load_vector<DT>(row, j), j, row, bound);
      }
      __syncthreads();
    }
    // ranked by counting those that come before
    const int found = s.found;
    for (int e = tid; e < found; e += kThreads) {
      const unsigned long long mine = s.candidate[e];
      int before = 0;
      for (int k = 0; k < found; ++k) before += s.candidate[k] > mine;
      if (before < a.top) s.best[before] = mine;
    }
    __syncthreads();
  }
  // ---- the cluster's parts
  if (a.ctas > 1) {
    cg::cluster_group cluster = cg::this_cluster();
    if (tid == 0) {
      s.mine = sums;
      s.mine_top = top;
    }
    cluster.sync();
    const int k = lane < a.ctas ? lane : 0;  // the same in every warp
    const float other = *cluster.map_shared_rank(&s.mine_top, k);
    Sums part = *cluster.map_shared_rank(&s.mine, k);
    if (lane >= a.ctas) part.s = 0.0f;
    top = other;
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    sums = moved(part, top, a.c);
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sums.s += __shfl_xor_sync(~0u, sums.s, o);
      sums.a += __shfl_xor_sync(~0u, sums.a, o);
    }
    if (TOP) {
      for (int e = tid; e < a.ctas * a.top; e += kThreads) s.all[e] = cluster.map_shared_rank(s.best, e / a.top)[e % a.top];
    }
    cluster.sync();  // nobody reads this CTA's shared memory after it
  }
  const float log_s = log2f(sums.s), k = top * a.c;
  const bool none = sums.s == 0.0f, bad = isnan(sums.s);
  auto log_p = [&](float x) {
    if (bad) return sums.s;
    if (none || x == -INFINITY) return -INFINITY;
    // a token at the type's lowest value keeps its finite log probability
    return plain(k) && plain(x * a.c) ? (__fmaf_rn(x, a.c, -k) - log_s) * kLn2 : (x - top) * (float)a.inverse - log_s * kLn2;
  };
  if (rank == 0 && tid == 0) {
    // m / T itself, and what k was rounded by
    const float off = plain(k) ? __fmaf_rn(top, a.c, -k) : 0.0f;
    if (a.lse) a.lse[r] = bad ? sums.s : none ? -INFINITY : (float)(top * a.inverse) + (log_s - off) * kLn2;
    if (a.entropy) a.entropy[r] = bad ? sums.s : none ? 0.0f : fmaxf((log_s - sums.a / sums.s) * kLn2, 0.0f);
    if (a.logprob) a.logprob[r] = log_p(x_token);
  }
  if (TOP) {
    int32_t* tokens = a.top_tokens + (int64_t)r * a.top;
    float* values = a.top_logprobs + (int64_t)r * a.top;
    auto put = [&](int place, unsigned long long e) {
      const bool is = e != 0 && !bad;
      tokens[place] = is ? (int32_t)~(uint32_t)e : -1;
      values[place] = is ? log_p(value_of<DT>((uint32_t)(e >> 32))) : bad ? sums.s : -INFINITY;
    };
    if (a.ctas == 1) {
      if (tid < a.top) put(tid, s.best[tid]);
    } else {
      __syncthreads();
      const int n = a.ctas * a.top;
      int live = 0;
      for (int e = warp; e < a.top; e += kWarps) {
        const unsigned long long mine = s.best[e];
        int before = 0;
        live = 0;
        for (int k = lane; k < n; k += 32) {
          before += s.all[k] > mine;
          live += s.all[k] != 0;
        }
        before = __reduce_add_sync(~0u, before);
        live = __reduce_add_sync(~0u, live);
        if (lane == 0 && mine != 0 && before < a.top) put(before, mine);
        if (lane == 0 && rank == 0 && e >= live) put(e, 0ull);
      }
    }
  }
}

template <int DT, bool TOP>
int launch(const LogprobArgs& a, int64_t rows, int device, cudaStream_t stream) {
  static std::atomic<bool> granted[kMaxDevices];
  return launch_clusters(logprobs_rows<DT, TOP>, rows, a.ctas, kThreads, TOP ? a.runs * 4 : 0, stream, granted, device, a);
}

}  // namespace

}  // namespace whead_verify_impl

using namespace whead_verify_impl;

extern "C" int whead_logprobs(const whead_logprobs_args* x) {
  if (!x || x->n < 0 || x->t < 0 || x->V < 1 || !is_dtype(x->dtype) || x->top < 0 || !good_temperature(x->temperature)) return WHEAD_ERR_INVALID_ARG;
  if (x->V >= 1 << 24 || x->top > WHEAD_MAX_TOP || (x->t > 0 && x->n > ((1 << 27) - 1) / x->t)) return WHEAD_ERR_UNSUPPORTED;
  const int64_t rows = x->n * x->t;
  if (rows == 0) return WHEAD_OK;
  if (!x->logits || !aligned(x->logits, dtype_size(x->dtype)) || (!x->tokens != !x->logprob)) return WHEAD_ERR_INVALID_ARG;
  if (!aligned(x->tokens, 4) || !aligned(x->logprob, 4) || !aligned(x->entropy, 4) || !aligned(x->lse, 4)) return WHEAD_ERR_INVALID_ARG;
  if (x->top && (!x->top_tokens || !x->top_logprobs || !aligned(x->top_tokens, 4) || !aligned(x->top_logprobs, 4))) return WHEAD_ERR_INVALID_ARG;
  int device = 0;
  const int sms = whead_kv_impl::device_sms(&device);
  if (sms < 1) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  LogprobArgs a{};
  a.logits = x->logits;
  a.tokens = x->tokens;
  a.logprob = x->logprob;
  a.entropy = x->entropy;
  a.lse = x->lse;
  a.top_tokens = x->top_tokens;
  a.top_logprobs = x->top_logprobs;
  a.stride_n = x->stride_n;
  a.stride_t = x->stride_t;
  a.t = (int)x->t;
  a.V = (int)x->V;
  a.top = x->top;
  a.inverse = 1.0 / x->temperature;
  a.c = (float)(1.4426950408889634 / x->temperature);
  const int64_t bytes = x->V * dtype_size(x->dtype);
  a.ctas = cluster_for(rows, bytes, sms);
  // most groups of a CTA: a row's, one more for its start anywhere, over the CTAs
  const int most = (int)((bytes / (kGroup * 16) + 2) / a.ctas + 1);
  while (((most >> a.shift) + 2) > kMaxRuns) ++a.shift;
  a.runs = (most >> a.shift) + 2;
  cudaStream_t stream = static_cast<cudaStream_t>(x->stream);
  switch (x->dtype) {
    case WHEAD_BF16: return a.top ? launch<WHEAD_BF16, true>(a, rows, device, stream) : launch<WHEAD_BF16, false>(a, rows, device, stream);
    case WHEAD_F16: return a.top ? launch<WHEAD_F16, true>(a, rows, device, stream) : launch<WHEAD_F16, false>(a, rows, device, stream);
    default: return a.top ? launch<WHEAD_F32, true>(a, rows, device, stream) : launch<WHEAD_F32, false>(a, rows, device, stream);
  }
}

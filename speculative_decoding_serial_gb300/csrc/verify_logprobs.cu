// verify_logprobs.cu — log probabilities of given tokens, entropy and top alternatives of rows of logits, in one pass over the logits.
//
// With d_v = (x_v - m) log2(e) / T, m the row's largest: s = sum 2^d, a = sum d 2^d; lse = m / T + ln s, log p(v) = ln 2 (d_v - log2 s),
// H = ln 2 (log2 s - a / s), whose two terms have one sign. Every thread has a running m of its own (verify_common.cuh).
//
// Alternatives. The CTA's threads make 64 parts of its values; the `top`-th of the parts' largest values is a bound that at least `top`
// values reach, and in rows without an order few more. The values that reach it are ranked by counting. Many rows: the pass keeps the
// largest value of every group (1 KB of the row) in shared memory, and the groups that reach the bound are read again; few rows:
// the CTA still holds its groups. Where more values reach the bound than there is room for, the groups with the best tokens are picked
// exactly (pick_candidates; one row 7 -> 21 us, 2,048 rows 122 -> 168 with 20 alternatives of sorted logits). None of this is part of the
// pass, whose work does not depend on the order of the logits.
//
// 4,096 rows of 151,936 bf16 logits: 182 us, the rate of a copy, without alternatives; 201 with the best one (6.2 TB/s; 69 % of the issue slots in use),
// 221 with 20: while a CTA picks it does not stream. 6 CTAs an SM of 40 registers: with 5 18 us more, with 8, which spill, 76. One row: 5.8 us with 5
// alternatives, 3.7 without: launch, copies, join, bound, ranking and the cluster's trade, a microsecond or less each.
#include "verify_common.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

namespace whead_verify_impl {

namespace {

namespace cg = cooperative_groups;

constexpr int kMaxRuns = 4224;  // largest values kept by a CTA: of groups, or of runs of 2^shift groups in rows of more (2^24 logits: shift 4)
static_assert(64 % kMaxCluster == 0, "");
constexpr int kFetchAhead = 16 * 1024;
constexpr int kListed = 128, kVectors = 96, kCandidates = kVectors * 8, kSubs = 64;

struct LogprobArgs {
  const void* logits;
  const int32_t* tokens;
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_tokens;
  float* top_logprobs;
  int64_t stride_n, stride_t;
  int t, V, top, ctas_shift, shift, runs, held;  // runs: room for largest values; held: for groups
  int ahead;                                     // CTAs that the device holds, where a row is one and there are more; else 0
  float c, inverse, inverse_low;                 // log2(e) / T, 1 / T, and what that was rounded by
};

struct RowShared {
  Sums part[16];          // the warps'
  Sums cluster[kMaxCluster];
};
struct TopShared {
  uint32_t bound;
  int found, listed, vectors;                                       // candidates, groups and vectors that reach the bound
  int list[kListed];
  alignas(16) uint32_t sub[kSubs];                                  // largest values of the CTA's parts
  alignas(16) uint32_t all[kSubs];                                  // of the row's
  int pushed;                                                       // numbers in `best`, in the cluster's first CTA
  uint4 vector[kVectors];
  int vector_at[kVectors];
  alignas(16) unsigned long long candidate[kCandidates];            // key, then the complement of the token
  alignas(16) unsigned long long best[kMaxCluster * WHEAD_MAX_TOP]; // the cluster's CTAs' best, in no order (one CTA: in order); 0: none
  // the way for rows where too many values reach the bound
  int picked;                                                       // what pick() found: how many keys, their indexes
  int order[WHEAD_MAX_TOP];
  int group[WHEAD_MAX_TOP];
  uint32_t key[WHEAD_MAX_TOP * kGroup];                             // largest values of the picked groups' vectors, or of the picked runs' groups
};
struct Nothing {};

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

// How many of n numbers in shared memory are greater.
__device__ __forceinline__ int greater(const unsigned long long* x, int n, unsigned long long than) {
  int count = 0, k = 0;
  for (; k + 8 <= n; k += 8) {
    ulonglong2 y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = *reinterpret_cast<const ulonglong2*>(x + k + 2 * i);
#pragma unroll
    for (int i = 0; i < 4; ++i) count += (y[i].x > than) + (y[i].y > than);
  }
  for (; k < n; ++k) count += x[k] > than;
  return count;
}

// Value e of vectors in shared memory.
template <int DT>
__device__ __forceinline__ float shared_one(const uint4* v, int e) {
  if constexpr (DT == WHEAD_F32) return reinterpret_cast<const float*>(v)[e];
  const unsigned short b = reinterpret_cast<const unsigned short*>(v)[e];
  return DT == WHEAD_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// Keeps a vector, if there is room.
__device__ __forceinline__ void keep(TopShared& s, const uint4& raw, int j) {
  const int at = atomicAdd(&s.vectors, 1);
  if (at < kVectors) {
    s.vector[at] = raw;
    s.vector_at[at] = j;
  }
}

// The way for a part of a row with too many values that reach the bound (many equal ones, or sorted ones): the groups that hold the best
// tokens by pick(), then their vectors likewise; the best tokens lie in no more vectors than they are. runs: the groups' largest values.
template <int DT, int THREADS>
__device__ __noinline__ void pick_candidates(TopShared& s, const uint32_t* runs, int n_runs, int g0, int g1, int shift, int top, Row row) {
  constexpr int BITS = Type<DT>::kKeyBits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto key_at = [&](int j) { return key_of<DT>(largest<DT>(load_vector<DT>(row, j))); };
  auto choose = [&](const uint32_t* keys, int n) {
    if (warp == 0) {
      const uint32_t bound = pick<BITS>(keys, n, top, s.order, &s.picked);
      if (lane == 0) s.bound = bound;
    }
    __syncthreads();
  };
  choose(runs, n_runs);
  if (tid < s.picked) s.group[tid] = ((g0 >> shift) + s.order[tid]) << shift;
  __syncthreads();
  if (shift) {  // of the picked runs of groups
    const int n = s.picked << shift, mask = (1 << shift) - 1;
    for (int e = warp; e < n; e += THREADS / 32) {
      const int g = s.group[e >> shift] + (e & mask);
      const bool mine = g >= g0 && g < g1;
      const uint32_t key = mine ? __reduce_max_sync(~0u, max(key_at(g * kGroup + lane), key_at(g * kGroup + 32 + lane))) : 0;
      if (lane == 0) s.key[e] = key;
    }
    __syncthreads();
    choose(s.key, n);
    const int g = tid < s.picked ? s.group[s.order[tid] >> shift] + (s.order[tid] & mask) : 0;
    __syncthreads();
    if (tid < s.picked) s.group[tid] = g;
    __syncthreads();
  }
  const int picked = s.picked;
  for (int e = tid; e < picked * kGroup; e += THREADS) s.key[e] = key_at(s.group[e / kGroup] * kGroup + e % kGroup);
  if (tid == 0) s.vectors = 0;
  __syncthreads();
  choose(s.key, picked * kGroup);
  if (tid < s.picked) {
    const int j = s.group[s.order[tid] / kGroup] * kGroup + s.order[tid] % kGroup;
    keep(s, load_vector<DT>(row, j), j);
  }
  if (tid == 0) s.bound = max(s.bound, Type<DT>::kNoneKey + 1);
  __syncthreads();
}

template <int DT, bool TOP, bool HELD>
__global__ void __launch_bounds__((Form<HELD>::kThreads), (Form<HELD>::kCtas)) logprobs_rows(const __grid_constant__ LogprobArgs a) {
  after_previous();
  constexpr int THREADS = Form<HELD>::kThreads, WARPS = THREADS / 32;
  __shared__ RowShared s;
  __shared__ std::conditional_t<TOP, TopShared, Nothing> top_shared;
  extern __shared__ __align__(16) uint4 held[];
  uint32_t* runs = reinterpret_cast<uint32_t*>(held + (HELD ? a.held * kGroup : 0));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x >> a.ctas_shift, ctas = 1 << a.ctas_shift, rank = blockIdx.x & (ctas - 1);
  const int i = a.t == 1 ? r : r / a.t, t = r - i * a.t;
  const int64_t at = i * a.stride_n + t * a.stride_t;
  const Row row = row_at<DT>(a.logits, at, a.V);
  const int groups = row_groups<DT>(row), g0 = run_begin(groups, a.ctas_shift, rank), g1 = run_begin(groups, a.ctas_shift, rank + 1);
  const int n_runs = g1 > g0 ? ((g1 - 1) >> a.shift) - (g0 >> a.shift) + 1 : 0;
  if constexpr (TOP) {
    if (tid == 0) {
      top_shared.found = top_shared.listed = top_shared.vectors = top_shared.pushed = 0;
      top_shared.bound = ~0u;
    }
    if (tid < kMaxCluster * WHEAD_MAX_TOP) top_shared.best[tid] = 0;
    if (!HELD && a.shift) {
      for (int k = tid; k < n_runs; k += THREADS) runs[k] = 0;
      __syncthreads();
    }
  }
  if (ctas > 1) cluster_arrive();  // before the loads: it waits for what is under way
  if (HELD) hold_groups<DT>(row, g0, g1, held);
  const int token = rank == 0 && a.tokens ? __ldg(a.tokens + r) : -1;
  // ---- the pass
  Pass p;
  begin(p);
  auto step = [&](int g, const uint4& v, const uint4& w) {
    const float high = fmaxf(largest<DT>(v), largest<DT>(w));
    take<DT, true>(p, v, w, high, a.c);
    if (TOP) {
      const float most = warp_max(high);
      if (lane == 0) {
        if (!HELD && a.shift) atomicMax(&runs[(g >> a.shift) - (g0 >> a.shift)], key_of<DT>(most));
        else runs[g - g0] = key_of<DT>(most);
      }
    }
  };
  if (HELD) over_held(g0, g1, held, step);
  else over_groups<DT>(row, g0, g1, step);
  // While this CTA joins and picks it reads nothing; the beginning of the row that comes in its place is fetched as far as L2 meanwhile (4,096
  // rows, top 1: 206 us without, 201 with 16 KB, 202 with 32, 206 with 64).
  if (!HELD && tid == 0 && a.ahead) {
    const unsigned next = blockIdx.x + a.ahead;
    if (next < gridDim.x) {
      const int ni = a.t == 1 ? next : next / a.t;
      const Row row = row_at<DT>(a.logits, ni * a.stride_n + ((int)next - ni * a.t) * a.stride_t, a.V);
      const char* from = row.base + (row.off ? 16 : 0);
      const int bytes = min(kFetchAhead, (a.V * Type<DT>::kSize - 16) & ~15);
      if (bytes > 0) asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(bytes) : "memory");
    }
  }
  {
    const Sums w = warp_joined(p, a.c);
    if (lane == 0) s.part[warp] = w;
  }
  if constexpr (TOP) {
    constexpr int SUB = THREADS / kSubs;
    uint32_t key = key_of<DT>(p.top);
#pragma unroll
    for (int o = 1; o < SUB; o <<= 1) key = max(key, __shfl_xor_sync(~0u, key, o));
    if (tid % SUB == 0) top_shared.sub[tid / SUB] = key;
  }
  __syncthreads();
  // ---- the CTA's best tokens
  if constexpr (TOP) {
    TopShared& ts = top_shared;
    // The CTA's values are in kSubs parts. The `top`-th of their largest values is one that `top` values reach, and on rows
    // without an order few more do. It is the lowest that fewer than `top` are greater than. For a long list a cluster's CTAs find one
    // bound for the row, by kSubs parts of it, which lets that many fewer values through; for a short list the trade takes longer than it
    // saves. One bound and bounds of their own, us, by the list's length: 1 x 151936 top 5 6.5, 6.1; top 8 6.5, 6.2; top 12 6.6, 6.5; top 20 6.6,
    // 7.2; top 32 6.9, 8.1. 17 x 151936: 7.9, 7.7; 7.9, 8.0; 7.9, 8.3; 8.0, 9.2; 8.3, 10.9. 64 x 248064: 16.1, 16.1; 16.2, 16.7; 16.4, 17.5; 16.6, 19.7; 17.2, 24.7.
    const uint32_t* sub = ts.sub;
    if (ctas > 1) cluster_wait();  // all have started
    if (ctas > 1 && a.top > 8) {
      const int each = kSubs >> a.ctas_shift;  // of this CTA's: every `ctas` parts are one
      if (tid < kSubs) {
        const int k = tid & (each - 1), to = tid >> (6 - a.ctas_shift);
        uint32_t high = 0;
        for (int e = 0; e < ctas; ++e) high = max(high, ts.sub[k * ctas + e]);
        *cg::this_cluster().map_shared_rank(&ts.all[rank * each + k], to) = high;
      }
      __syncwarp();
      cluster_arrive();
      cluster_wait();
      sub = ts.all;
    }
    if (tid < kSubs) {
      const uint32_t mine = sub[tid];
      int before = 0;
#pragma unroll
      for (int k = 0; k < kSubs; k += 4) {
        const uint4 y = *reinterpret_cast<const uint4*>(sub + k);
        before += (y.x > mine) + (y.y > mine) + (y.z > mine) + (y.w > mine);
      }
      const uint32_t low = __reduce_min_sync(~0u, before < a.top ? mine : ~0u);
      if (lane == 0) atomicMin(&ts.bound, low);
    }
    __syncthreads();
    uint32_t bound = max(ts.bound, Type<DT>::kNoneKey + 1);
    float least = value_of<DT>(bound);
    // the groups that reach it, and of those the vectors
    for (int k = tid; k < n_runs; k += THREADS)
      if (runs[k] >= bound) {
        const int place = atomicAdd(&ts.listed, 1);
        if (place < kListed) ts.list[place] = k;
      }
    __syncthreads();
    const int listed = ts.listed <= kListed ? ts.listed << a.shift : 0;
#pragma unroll 4
    for (int e = warp; e < 2 * listed; e += WARPS) {
      const int g = (((g0 >> a.shift) + ts.list[e / 2 >> a.shift]) << a.shift) + (e / 2 & ((1 << a.shift) - 1)), j = g * kGroup + e % 2 * 32 + lane;
      if (g >= g0 && g < g1) {
        const uint4 raw = HELD ? held[j - g0 * kGroup] : load_vector<DT>(row, j);
        if (largest<DT>(raw) >= least) keep(ts, raw, j);
      }
    }
    __syncthreads();
    if (ts.vectors > kVectors || ts.listed > kListed) {
      pick_candidates<DT, THREADS>(ts, runs, n_runs, g0, g1, a.shift, a.top, row);
      least = value_of<DT>(ts.bound);
    }
    // their values that reach it
    constexpr int N = Type<DT>::kPer;
    for (int e = tid; e < ts.vectors * N; e += THREADS) {
      const float x = shared_one<DT>(ts.vector, e);
      if (x >= least) ts.candidate[atomicAdd(&ts.found, 1)] = (unsigned long long)key_of<DT>(x) << 32 | (uint32_t)~(uint32_t)(ts.vector_at[e / N] * N + e % N - row.off);
    }
    __syncthreads();
    // ranked by counting those that come before
    const int found = ts.found;
    for (int e = tid; e < found; e += THREADS) {
      const unsigned long long mine = ts.candidate[e];
      const int before = greater(ts.candidate, found, mine);
      if (before < a.top) {
        if (ctas > 1) in_first(ts.best)[atomicAdd(in_first(&ts.pushed), 1)] = mine;
        else ts.best[before] = mine;
      }
    }
  } else if (ctas > 1) {
    cluster_wait();
  }
  // ---- the cluster's parts, in its first CTA
  const float x_token = (unsigned)token < (unsigned)a.V ? load_one(a.logits, at + token, DT) : -INFINITY;
  Sums sums;
  if (ctas > 1) {
    if (warp == 0) {
      sums = parts_joined(s.part[min(lane, WARPS - 1)], WARPS, a.c);
      if (lane == 0) *in_first(&s.cluster[rank]) = sums;
    }
    __syncwarp();
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    sums = parts_joined(s.cluster[min(lane, ctas - 1)], ctas, a.c);
  } else {
    if (TOP) __syncthreads();
    sums = parts_joined(s.part[min(lane, WARPS - 1)], WARPS, a.c);
  }
  const float top = sums.ref, log_s = log2f(sums.s), k = top * a.c, off = offset_of(top, a.c);
  const bool none = sums.s == 0.0f, bad = isnan(sums.s);
  auto log_p = [&](float x) {
    if (bad) return sums.s;
    if (none || x == -INFINITY) return -INFINITY;
    // a token at the type's lowest value keeps its finite log probability
    return plain(k) && plain(x * a.c) ? (__fmaf_rn(x, a.c, -k) - log_s) * kLn2 : (x - top) * a.inverse - (log_s - off) * kLn2;
  };
  if (tid == THREADS - 32) {  // not the warps that write alternatives
    // m / T itself, and what k was rounded by (0 where it is not formed)
    if (a.lse) a.lse[r] = bad ? sums.s : none ? -INFINITY : plain(k) ? __fmaf_rn(top, a.inverse, __fmaf_rn(top, a.inverse_low, (log_s - off) * kLn2)) : top * a.inverse + log_s * kLn2;
    if (a.entropy) a.entropy[r] = bad ? sums.s : none ? 0.0f : fmaxf((log_s - __fdividef(sums.a, sums.s)) * kLn2, 0.0f);
    if (a.logprob) a.logprob[r] = log_p(x_token);
  }
  if constexpr (TOP) {
    TopShared& ts = top_shared;
    const int n = ctas > 1 ? ts.pushed : a.top;  // at most a place a thread
    const unsigned long long mine = tid < n && !bad ? ts.best[tid] : 0ull;
    int before = tid;
    if (ctas > 1 && mine != 0) before = greater(ts.best, n, mine);
    const int live = __syncthreads_count(mine != 0);
    int32_t* tokens = a.top_tokens + (int64_t)r * a.top;
    float* values = a.top_logprobs + (int64_t)r * a.top;
    if (mine != 0 && before < a.top) {
      tokens[before] = (int32_t)~(uint32_t)mine;
      values[before] = log_p(value_of<DT>((uint32_t)(mine >> 32)));
    }
    if (tid >= live && tid < a.top) {
      tokens[tid] = -1;
      values[tid] = bad ? sums.s : -INFINITY;
    }
  }
}

template <int DT, bool TOP, bool HELD>
int launch(const LogprobArgs& a, int64_t rows, int device, cudaStream_t stream) {
  static std::atomic<bool> granted[kMaxDevices];
  return launch_clusters(logprobs_rows<DT, TOP, HELD>, rows, 1 << a.ctas_shift, Form<HELD>::kThreads, (HELD ? a.held * kGroup * 16 : 0) + (TOP ? a.runs * 4 : 0), stream, granted, device, a);
}
template <int DT>
int launch(const LogprobArgs& a, bool held, int64_t rows, int device, cudaStream_t stream) {
  if (held) return a.top ? launch<DT, true, true>(a, rows, device, stream) : launch<DT, false, true>(a, rows, device, stream);
  return a.top ? launch<DT, true, false>(a, rows, device, stream) : launch<DT, false, false>(a, rows, device, stream);
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
  a.inverse = (float)(1.0 / x->temperature);
  a.inverse_low = (float)(1.0 / x->temperature - a.inverse);
  a.c = (float)(1.4426950408889634 / x->temperature);
  const Division d = divide(rows, x->V * dtype_size(x->dtype), sms);
  a.ctas_shift = d.shift;
  a.held = d.groups;
  const int64_t room = (int64_t)sms * Form<false>::kCtas;
  a.ahead = !d.held && d.shift == 0 && rows > room ? (int)room : 0;
  while (((d.groups >> a.shift) + 2) > kMaxRuns) ++a.shift;
  a.runs = (d.groups >> a.shift) + 2;
  cudaStream_t stream = static_cast<cudaStream_t>(x->stream);
  switch (x->dtype) {
    case WHEAD_BF16: return launch<WHEAD_BF16>(a, d.held, rows, device, stream);
    case WHEAD_F16: return launch<WHEAD_F16>(a, d.held, rows, device, stream);
    default: return launch<WHEAD_F32>(a, d.held, rows, device, stream);
  }
}

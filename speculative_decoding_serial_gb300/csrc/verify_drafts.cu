// verify_drafts.cu — which drafts stay under the target's logits, and the token after them.
//
// Two kernels. The first takes every row of logits once: at temperature 0 its largest value's token, else its largest value and its sum of
// exponentials. The second, a cluster an entry, finds the first draft that does not stay and draws the token of that row: the largest of
// r_v / E_v with r = max(p - q, 0), E = -log U. Since E >= 1 - U, only a token with r_v / (1 - U) above the best so far needs its
// logarithm; 1 - U is known exactly from the word.
//
// What is near a border is settled in fp64: a draft whose U q and p differ by less than 2^-16 of p, and the two best tokens where they do.
#include "verify_common.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>

namespace whead_verify_impl {

namespace {

namespace cg = cooperative_groups;

constexpr float kNear = 0x1p-16f;
constexpr int kDrawThreads = 512, kDrawWarps = kDrawThreads / 32;

struct VerifyArgs {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* drafted;
  int32_t* said;
  int32_t* count;
  float2* stats;    // n x (gamma + 1) rows of the target, then n x gamma of the drafts: (largest, sum); at temperature 0 (token, -)
  int64_t target_stride_n, target_stride_t, draft_stride_n, draft_stride_t;
  int V, gamma, ctas_shift, held, target_dtype, draft_dtype;
  uint32_t step;
  int64_t n;
  float c, draft_c;              // log2(e) / T
  double inverse, draft_inverse; // 1 / T
  uint64_t seed;
};

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int i) { return a.drafted ? min(max(__ldg(a.drafted + i), 0), a.gamma) : a.gamma; }

// A part of a row's first largest value: the vector that holds it, and whether the part has NaN or +inf.
struct First {
  float top;
  int at, bad;
};
struct RowShared {
  Sums part[16];
  Sums cluster[kMaxCluster];
  First first[16];
  First first_cluster[kMaxCluster];
};

// Largest value and sum of a row, by a cluster.
template <int DT, bool HELD>
__device__ __forceinline__ void row_sums(const VerifyArgs& a, const Row& row, int rank, float c, float2* to, uint4* held, RowShared& s) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = row_groups<DT>(row), ctas = 1 << a.ctas_shift, g0 = run_begin(groups, a.ctas_shift, rank), g1 = run_begin(groups, a.ctas_shift, rank + 1);
  if (ctas > 1) cluster_arrive();  // before the loads: it waits for what is under way
  if (HELD) hold_groups<DT>(row, g0, g1, held);
  Pass p;
  begin(p);
  auto step = [&](int, const uint4& v, const uint4& w) { take<DT, false>(p, v, w, fmaxf(largest<DT>(v), largest<DT>(w)), c); };
  if (HELD) over_held(g0, g1, held, step);
  else over_groups<DT>(row, g0, g1, step);
  Sums q = warp_joined(p, c);
  if (lane == 0) s.part[warp] = q;
  __syncthreads();
  if (ctas > 1) {
    cluster_wait();
    if (warp == 0) {
      q = parts_joined(s.part, Form<HELD>::kWarps, c);
      if (lane == 0) *in_first(&s.cluster[rank]) = q;
    }
    __syncwarp();
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    if (warp == 0) q = parts_joined(s.cluster, ctas, c);
  } else if (warp == 0) {
    q = parts_joined(s.part, Form<HELD>::kWarps, c);
  }
  if (tid == 0) *to = make_float2(q.ref, q.s);
}

__device__ __forceinline__ First warp_first(First f) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(~0u, f.top, o);
    const int z = __shfl_xor_sync(~0u, f.at, o);
    if (y > f.top || (y == f.top && z < f.at)) {
      f.top = y;
      f.at = z;
    }
  }
  f.bad = __any_sync(~0u, f.bad);
  return f;
}

// Token of a row's largest value, by a cluster: the first vector that holds it, then its place there. -1 where the row has NaN, +inf or
// nothing but -inf.
template <int DT, bool HELD>
__device__ __forceinline__ void row_token(const VerifyArgs& a, const Row& row, int rank, float2* to, uint4* held, RowShared& s) {
  constexpr int N = Type<DT>::kPer, WARPS = Form<HELD>::kWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = row_groups<DT>(row), ctas = 1 << a.ctas_shift, g0 = run_begin(groups, a.ctas_shift, rank), g1 = run_begin(groups, a.ctas_shift, rank + 1);
  if (ctas > 1) cluster_arrive();  // before the loads: it waits for what is under way
  if (HELD) hold_groups<DT>(row, g0, g1, held);
  First f{-INFINITY, INT_MAX, 0};
  auto step = [&](int g, const uint4& v, const uint4& w) {
    const float first = largest_nan<DT>(v), high = max_nan(first, largest_nan<DT>(w));
    f.bad |= !(high < INFINITY);
    const int j = g * kGroup + (first == high ? lane : 32 + lane);
    if (high > f.top || (high == f.top && j < f.at)) {  // a row's first group may come last
      f.top = high;
      f.at = j;
    }
  };
  if (HELD) over_held(g0, g1, held, step);
  else over_groups<DT>(row, g0, g1, step);
  f = warp_first(f);
  if (lane == 0) s.first[warp] = f;
  __syncthreads();
  if (ctas > 1) cluster_wait();
  if (warp == 0) f = warp_first(s.first[lane & (WARPS - 1)]);
  if (ctas > 1) {
    if (tid == 0) *in_first(&s.first_cluster[rank]) = f;
    __syncwarp();
    cluster_arrive();
    if (rank != 0) return;
    cluster_wait();
    if (warp == 0) f = warp_first(s.first_cluster[lane < ctas ? lane : 0]);
  }
  if (tid == 0) {
    int token = -1;
    if (!f.bad && f.top > -INFINITY) {
      float x[N];
      values_of<DT>(load_vector<DT>(row, f.at), x);
#pragma unroll
      for (int k = N - 1; k >= 0; --k)
        if (x[k] == f.top) token = f.at * N + k - row.off;
    }
    *to = make_float2(__int_as_float(token), 0.0f);
  }
}

template <bool GREEDY, bool HELD>
__global__ void __launch_bounds__((Form<HELD>::kThreads), (Form<HELD>::kCtas)) verify_rows(const __grid_constant__ VerifyArgs a) {
  after_previous();
  __shared__ RowShared s;
  extern __shared__ __align__(16) uint4 held[];
  const int r = blockIdx.x >> a.ctas_shift, rank = blockIdx.x - (r << a.ctas_shift);
  const int targets = (int)a.n * (a.gamma + 1);
  const bool of_target = GREEDY || r < targets;
  const int each = of_target ? a.gamma + 1 : a.gamma, k = of_target ? r : r - targets;
  const int i = k / each, t = k - i * each;
  if (t >= drafts_of(a, i) + (of_target ? 1 : 0)) return;  // the whole cluster
  const void* p = of_target ? a.target : a.draft;
  const int64_t at = of_target ? i * a.target_stride_n + t * a.target_stride_t : i * a.draft_stride_n + t * a.draft_stride_t;
  const int dtype = of_target ? a.target_dtype : a.draft_dtype;
  const float c = of_target ? a.c : a.draft_c;
  float2* to = a.stats + r;
  auto go = [&](auto type) {
    constexpr int DT = decltype(type)::value;
    const Row row = row_at<DT>(p, at, a.V);
    if constexpr (GREEDY) row_token<DT, HELD>(a, row, rank, to, held, s);
    else row_sums<DT, HELD>(a, row, rank, c, to, held, s);
  };
  if (dtype == WHEAD_BF16) go(std::integral_constant<int, WHEAD_BF16>{});
  else if (dtype == WHEAD_F16) go(std::integral_constant<int, WHEAD_F16>{});
  else go(std::integral_constant<int, WHEAD_F32>{});
}

// One entry's row of `said`, and its count.
__device__ __forceinline__ void write_said(const VerifyArgs& a, int i, int stay, int next, int tid, int threads) {
  for (int t = tid; t <= a.gamma; t += threads) a.said[(int64_t)i * (a.gamma + 1) + t] = t < stay ? a.tokens[(int64_t)i * a.gamma + t] : t == stay ? next : -1;
  if (tid == 0) a.count[i] = stay + 1;
}

__global__ void __launch_bounds__(32) verify_greedy(const __grid_constant__ VerifyArgs a) {
  after_previous();
  const int i = blockIdx.x, lane = threadIdx.x, have = drafts_of(a, i);
  const float2* stats = a.stats + (int64_t)i * (a.gamma + 1);
  int stay = have;
  for (int base = 0; base < have; base += 32) {
    const int t = base + lane;
    const bool stops = t < have && (a.tokens[(int64_t)i * a.gamma + t] < 0 || __float_as_int(stats[t].x) != a.tokens[(int64_t)i * a.gamma + t]);
    const unsigned b = __ballot_sync(~0u, stops);
    if (b) {
      stay = base + __ffs(b) - 1;
      break;
    }
  }
  write_said(a, i, stay, __float_as_int(stats[stay].x), lane, 32);
}

// The best two tokens seen: keys r / E, of equal ones the lower token first; token -1: none.
struct Best {
  float k1, k2;
  int v1, v2;
};
__device__ __forceinline__ bool before(float k, int v, float k0, int v0) { return v >= 0 && (v0 < 0 || k > k0 || (k == k0 && v < v0)); }
__device__ __forceinline__ void add(Best& b, float k, int v) {
  if (before(k, v, b.k1, b.v1)) {
    b.k2 = b.k1;
    b.v2 = b.v1;
    b.k1 = k;
    b.v1 = v;
  } else if (before(k, v, b.k2, b.v2)) {
    b.k2 = k;
    b.v2 = v;
  }
}

struct DrawShared {
  int stay;
  Best part[kDrawWarps];
  Best mine[2];  // for the cluster, of the residual and of the target
};

__device__ __forceinline__ float uniform(uint32_t w) { return ((float)(w >> 9) + 0.5f) * 0x1p-23f; }

// Four logits from `at` on, of which `live` are there; `wide`: they can be read as one.
__device__ __forceinline__ void load_four_logits(const void* p, int64_t at, int dtype, bool wide, int live, float (&x)[4]) {
  if (wide && live >= 4) {
    if (dtype == WHEAD_F32) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + at));
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const unsigned short*>(p) + at));
      const float2 lo = whead_kv_impl::unpack16(v.x, dtype), hi = whead_kv_impl::unpack16(v.y, dtype);
      x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = k < live ? load_one(p, at + k, dtype) : -INFINITY;
  }
}

__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw(const __grid_constant__ VerifyArgs a) {
  after_previous();
  __shared__ DrawShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = 1 << a.ctas_shift, i = blockIdx.x >> a.ctas_shift, rank = blockIdx.x & (ctas - 1);
  const int have = drafts_of(a, i);
  const float2* p_stats = a.stats + (int64_t)i * (a.gamma + 1);
  const float2* q_stats = a.stats + a.n * (a.gamma + 1) + (int64_t)i * a.gamma;
  const int32_t* tokens = a.tokens + (int64_t)i * a.gamma;
  if (tid == 0) s.stay = have;
  __syncthreads();
  auto sound = [](float2 x) { return x.y > 0.0f && x.y < INFINITY; };
  if (tid < have) {
    const int x = tokens[tid];
    const float2 ps = p_stats[tid], qs = a.draft ? q_stats[tid] : make_float2(0.0f, 1.0f);
    bool stays = false;
    if ((unsigned)x < (unsigned)a.V && sound(ps) && sound(qs)) {
      const float xp = load_one(a.target, i * a.target_stride_n + tid * a.target_stride_t + x, a.target_dtype);
      const float xq = a.draft ? load_one(a.draft, i * a.draft_stride_n + tid * a.draft_stride_t + x, a.draft_dtype) : 0.0f;
      const float u = uniform(philox(make_uint4(0u, a.step + tid, (uint32_t)i, 2u), a.seed).x);
      const float p = ex2((xp - ps.x) * a.c) / ps.y, q = a.draft ? ex2((xq - qs.x) * a.draft_c) / qs.y : 1.0f;
      stays = u * q < p;
      if (fabsf(u * q - p) <= kNear * p || p < 1e-30f) {
        const double dp = exp(((double)xp - ps.x) * a.inverse) / ps.y, dq = a.draft ? exp(((double)xq - qs.x) * a.draft_inverse) / qs.y : 1.0;
        stays = u * dq < dp;
      }
    }
    if (!stays) atomicMin(&s.stay, tid);
  }
  __syncthreads();
  const int stay = s.stay;
  const float2 ps = p_stats[stay];
  const bool some = sound(ps), rejected = stay < have;
  const float2 qs = rejected && a.draft ? q_stats[stay] : make_float2(0.0f, 1.0f);
  const int drafted = rejected ? tokens[stay] : -1;
  const bool with_q = rejected && a.draft && sound(qs);  // a row q of logits to take off
  const int64_t p_at = i * a.target_stride_n + stay * a.target_stride_t, q_at = i * a.draft_stride_n + stay * a.draft_stride_t;
  const int p_size = a.target_dtype == WHEAD_F32 ? 4 : 2, q_size = a.draft_dtype == WHEAD_F32 ? 4 : 2;
  const bool p_wide = ((reinterpret_cast<uintptr_t>(a.target) + p_at * p_size) & (4 * p_size - 1)) == 0;
  const bool q_wide = with_q && ((reinterpret_cast<uintptr_t>(a.draft) + q_at * q_size) & (4 * q_size - 1)) == 0;
  const float p_inv = 1.0f / ps.y, q_inv = 1.0f / qs.y;
  Best all{0.0f, 0.0f, -1, -1};
  bool whole = !rejected;  // draw from p itself
  for (int turn = 0; some && turn < 2; ++turn) {
    Best best{0.0f, 0.0f, -1, -1};
    for (int g = rank * kDrawThreads + tid; g < (a.V + 3) / 4; g += ctas * kDrawThreads) {
      float x[4], y[4];
      load_four_logits(a.target, p_at + 4 * g, a.target_dtype, p_wide, a.V - 4 * g, x);
      if (with_q && !whole) load_four_logits(a.draft, q_at + 4 * g, a.draft_dtype, q_wide, a.V - 4 * g, y);
      const uint4 word = philox(make_uint4((uint32_t)g, a.step + stay, (uint32_t)i, 1u), a.seed);
      const uint32_t w[4] = {word.x, word.y, word.z, word.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float r = ex2((x[k] - ps.x) * a.c) * p_inv;
        if (!whole) {
          if (with_q) r -= ex2((y[k] - qs.x) * a.draft_c) * q_inv;
          else if (!a.draft && 4 * g + k == drafted) r = 0.0f;
        }
        const float rest = (float)(0x800000u - (w[k] >> 9)) - 0.5f;  // (1 - U) 2^23, exactly
        if (r > 0.0f && r * 8388736.0f > best.k1 * rest) add(best, r / -logf(uniform(w[k])), 4 * g + k);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const Best y{__shfl_xor_sync(~0u, best.k1, o), __shfl_xor_sync(~0u, best.k2, o), __shfl_xor_sync(~0u, best.v1, o), __shfl_xor_sync(~0u, best.v2, o)};
      add(best, y.k1, y.v1);
      add(best, y.k2, y.v2);
    }
    if (lane == 0) s.part[warp] = best;
    __syncthreads();
    for (int w = 0; w < kDrawWarps; ++w) {
      if (w == warp) continue;
      add(best, s.part[w].k1, s.part[w].v1);
      add(best, s.part[w].k2, s.part[w].v2);
    }
    all = best;
    if (ctas > 1) {
      cg::cluster_group cluster = cg::this_cluster();
      if (tid == 0) s.mine[turn] = best;
      cluster.sync();
      for (int k = 0; k < ctas; ++k) {
        if (k == rank) continue;
        const Best* y = cluster.map_shared_rank(&s.mine[turn], k);
        add(all, y->k1, y->v1);
        add(all, y->k2, y->v2);
      }
    } else {
      __syncthreads();
    }
    if (all.v1 >= 0 || whole) break;
    whole = true;  // rounding left nothing of p - q
  }
  if (ctas > 1) cg::this_cluster().sync();  // nobody reads this CTA's shared memory after it
  if (rank != 0) return;
  if (tid == 0) s.stay = all.v1;
  if (tid == 0 && all.v2 >= 0 && all.k1 - all.k2 <= kNear * all.k1) {
    auto key = [&](int v) {
      double r = exp(((double)load_one(a.target, p_at + v, a.target_dtype) - ps.x) * a.inverse) / ps.y;
      if (!whole && with_q) r -= exp(((double)load_one(a.draft, q_at + v, a.draft_dtype) - qs.x) * a.draft_inverse) / qs.y;
      const uint4 word = philox(make_uint4((uint32_t)v >> 2, a.step + stay, (uint32_t)i, 1u), a.seed);
      const uint32_t w = v & 2 ? (v & 1 ? word.w : word.z) : (v & 1 ? word.y : word.x);
      return r / -log((double)uniform(w));
    };
    const double k1 = key(all.v1), k2 = key(all.v2);
    if (k2 > k1 || (k2 == k1 && all.v2 < all.v1)) s.stay = all.v2;
  }
  __syncthreads();
  write_said(a, i, stay, some ? s.stay : -1, tid, kDrawThreads);
}

template <bool GREEDY, bool HELD>
int launch_rows(const VerifyArgs& a, int64_t rows, int device, cudaStream_t stream) {
  static std::atomic<bool> granted[kMaxDevices];
  return launch_clusters(verify_rows<GREEDY, HELD>, rows, 1 << a.ctas_shift, Form<HELD>::kThreads, HELD ? a.held * kGroup * 16 : 0, stream, granted, device, a);
}

int launch(const VerifyArgs& from, int device, int sms, cudaStream_t stream) {
  static std::atomic<bool> granted[kMaxDevices];
  VerifyArgs a = from;
  const bool greedy = a.inverse == 0.0;
  const int64_t rows = a.n * (a.gamma + 1) + (greedy || !a.draft ? 0 : a.n * a.gamma);
  const int64_t bytes = (int64_t)a.V * std::max(dtype_size(a.target_dtype), a.draft ? dtype_size(a.draft_dtype) : 0);
  const Division d = divide(rows, bytes, sms);
  a.ctas_shift = d.shift;
  a.held = d.groups;
  int rc;
  if (greedy) rc = d.held ? launch_rows<true, true>(a, rows, device, stream) : launch_rows<true, false>(a, rows, device, stream);
  else rc = d.held ? launch_rows<false, true>(a, rows, device, stream) : launch_rows<false, false>(a, rows, device, stream);
  if (rc != WHEAD_OK) return rc;
  if (greedy) return whead_kv_impl::launch_after(verify_greedy, dim3((unsigned)a.n), 32, 0, stream, a);
  a.ctas_shift = 0;
  while ((2 << a.ctas_shift) <= kMaxCluster && a.n << (a.ctas_shift + 1) <= (int64_t)sms * 3 && a.V >> (a.ctas_shift + 1) >= 4 * kDrawThreads) ++a.ctas_shift;
  return launch_clusters(verify_draw, a.n, 1 << a.ctas_shift, kDrawThreads, 0, stream, granted, device, a);
}

}  // namespace

}  // namespace whead_verify_impl

using namespace whead_verify_impl;

extern "C" int64_t whead_verify_workspace_bytes(int64_t n, int32_t gamma) {
  if (n < 0 || gamma < 0) return WHEAD_ERR_INVALID_ARG;
  if (gamma > WHEAD_MAX_DRAFTS || n > ((1 << 27) - 1) / (2 * gamma + 1)) return WHEAD_ERR_UNSUPPORTED;
  return whead_kv_impl::align256(n * (2 * gamma + 1) * (int64_t)sizeof(float2));
}

extern "C" int whead_verify(const whead_verify_args* x) {
  if (!x || x->V < 1 || !is_dtype(x->target_dtype) || !(x->temperature == 0 || good_temperature(x->temperature))) return WHEAD_ERR_INVALID_ARG;
  const int64_t need = whead_verify_workspace_bytes(x->n, x->gamma);
  if (need < 0) return (int)need;
  if (x->V >= 1 << 24) return WHEAD_ERR_UNSUPPORTED;
  const bool with_draft = x->draft && x->temperature > 0 && x->gamma > 0;
  if (with_draft && (!is_dtype(x->draft_dtype) || !good_temperature(x->draft_temperature) || !aligned(x->draft, dtype_size(x->draft_dtype)))) return WHEAD_ERR_INVALID_ARG;
  if (x->n == 0) return WHEAD_OK;
  if (!x->target || !x->said || !x->count || !x->workspace || (x->gamma > 0 && !x->tokens)) return WHEAD_ERR_INVALID_ARG;
  if (!aligned(x->target, dtype_size(x->target_dtype)) || !aligned(x->tokens, 4) || !aligned(x->drafted, 4) || !aligned(x->said, 4) || !aligned(x->count, 4) ||
      !aligned(x->workspace, 16) || x->workspace_bytes < need)
    return WHEAD_ERR_INVALID_ARG;
  int device = 0;
  const int sms = whead_kv_impl::device_sms(&device);
  if (sms < 1) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  VerifyArgs a{};
  a.target = x->target;
  a.draft = with_draft ? x->draft : nullptr;
  a.tokens = x->tokens;
  a.drafted = x->drafted;
  a.said = x->said;
  a.count = x->count;
  a.stats = static_cast<float2*>(x->workspace);
  a.target_stride_n = x->target_stride_n;
  a.target_stride_t = x->target_stride_t;
  a.draft_stride_n = x->draft_stride_n;
  a.draft_stride_t = x->draft_stride_t;
  a.V = (int)x->V;
  a.gamma = x->gamma;
  a.target_dtype = x->target_dtype;
  a.draft_dtype = x->draft_dtype;
  a.step = x->step;
  a.n = x->n;
  if (x->temperature > 0) {
    a.inverse = 1.0 / x->temperature;
    a.c = (float)(1.4426950408889634 / x->temperature);
  }
  if (with_draft) {
    a.draft_inverse = 1.0 / x->draft_temperature;
    a.draft_c = (float)(1.4426950408889634 / x->draft_temperature);
  }
  a.seed = x->seed;
  return launch(a, device, sms, static_cast<cudaStream_t>(x->stream));
}

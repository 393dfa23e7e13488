// verify_drafts.cu — which drafts stay under the target's logits, and the token after them.
//
// Two kernels. The first takes rows of logits: at temperature 0 their largest value's token, else their largest value and sum of
// exponentials, a CTA a part of a row. The second, for each entry, joins the parts, finds the first draft that does not stay and draws the
// token of that row: the largest of r_v / E_v with r = max(p - q, 0), E = -log U. Since E >= 1 - U, only a token with r_v / (1 - U)
// above the CTA's best so far needs its logarithm; 1 - U is known exactly from the word.
//
// Rows after the first draft that does not stay are not needed. Where there are more rows than the device takes at once, CTAs come in the order of
// the drafts' places, whoever finishes a place decides on its draft, and parts of later places that find
// theirs decided are left out. Results do not depend on how many are: whoever decides joins the same parts in the same order.
//
// What is near a border is settled in fp64: a draft whose U q and p differ by less than 2^-16 of p, and the two best tokens where their keys
// do. p and q are off by some 2^-20 in fp32, and p - q by p / (p - q) times that, so that keys of p - q are settled from 2^-9 on: drafts' rows as near
// to the target's as p - q = p / 1000. The sums of p and q stay those of fp32, and three keys so near to one another are not told apart.
//
// 64 entries of 16 drafts, 151,936 logits, bf16 and f32 for the drafts', a draft in five refused: rows 72 us (418 MB at 5.8 TB/s, of which 284 MB are
// needed: places that began before the one ahead was decided), drawing 27 us (176 issue slots for four tokens of a warp, Philox 86 of them; 256 CTAs on
// 304 places). 8 entries, greedy, f32: all rows, 14 us, 5.9 TB/s. One entry, bf16: rows 5 us, drawing 8, ten times four tokens a thread.
#include "verify_common.cuh"

#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

namespace whead_verify_impl {

namespace {

constexpr float kNear = 0x1p-16f;            // relative: what is settled in fp64
constexpr float kNearOfDifference = 0x1p-9f; // the same for keys of p - q; one draw in 512 or fewer is that near
constexpr int kDrawThreads = 512, kDrawWarps = kDrawThreads / 32;
constexpr int kMaxParts = 16;  // of a row

struct VerifyArgs {
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* drafted;
  int32_t* said;
  int32_t* count;
  float2* parts;     // n x (gamma + 1) x (target, draft) x parts: (largest, sum); at temperature 0 (largest or NaN, token)
  float* logit;      // n x (gamma + 1) x (target, draft): the draft's, NaN where it is no token
  int32_t* first;    // n: the first place whose draft is known not to stay; NULL: all rows are taken
  int32_t* arrived;  // n x (gamma + 1): parts of a place that are done
  int64_t target_stride_n, target_stride_t, draft_stride_n, draft_stride_t;
  int V, gamma, n, parts_shift, ctas_shift, held, target_dtype, draft_dtype;
  uint32_t step;
  float c, draft_c;              // log2(e) / T
  double inverse, draft_inverse; // 1 / T
  uint64_t seed;
};

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int i) { return a.drafted ? min(max(__ldg(a.drafted + i), 0), a.gamma) : a.gamma; }
__device__ __forceinline__ float2* parts_of(const VerifyArgs& a, int i, int t, int of_draft) {
  return a.parts + ((((int64_t)i * (a.gamma + 1) + t) * 2 + of_draft) << a.parts_shift);
}
__device__ __forceinline__ float uniform(uint32_t w) { return ((float)(w >> 9) + 0.5f) * 0x1p-23f; }

// A row's largest value m and sum of 2^((x - m) c), by a warp, from its parts; every lane gets them.
__device__ __forceinline__ float2 row_sums(const VerifyArgs& a, int i, int t, int of_draft) {
  const int lane = threadIdx.x & 31, n = 1 << a.parts_shift;
  const float2 x = __ldcg(parts_of(a, i, t, of_draft) + min(lane, n - 1));
  const float c = of_draft ? a.draft_c : a.c;
  const Sums s = parts_joined(Sums{x.x, x.y, 0.0f}, n, c);
  const float off = offset_of(s.ref, c);  // mostly so small that 1 - off ln 2 is nearer to 2^-off than the exponential's own rounding
  return make_float2(s.ref, fabsf(off) < 0x1p-12f ? __fmaf_rn(s.s, -off * kLn2, s.s) : s.s * ex2(-off));
}
// Whether a row has a distribution.
__device__ __forceinline__ bool sound(float2 x) { return x.y > 0.0f && x.y < INFINITY; }

// The token of a row's largest value, from its parts; -1 where the row has NaN, +inf or nothing but -inf.
__device__ __forceinline__ int row_token(const VerifyArgs& a, int i, int t) {
  const float2* part = parts_of(a, i, t, 0);
  float top = -INFINITY;
  int token = -1;
  bool bad = false;
  for (int k = 0; k < 1 << a.parts_shift; ++k) {
    const float2 x = __ldcg(part + k);
    bad |= !(x.x < INFINITY);
    if (x.x > top) {
      top = x.x;
      token = __float_as_int(x.y);
    }
  }
  return bad ? -1 : token;
}

// p and q of one token in 64 bits.
__device__ __noinline__ double probability64(float x, float2 stats, double inverse) { return exp(((double)x - stats.x) * inverse) / stats.y; }

// Whether draft t, whose logits are xp and xq, stays, given that all before it do.
__device__ __noinline__ bool draft_stays(const VerifyArgs& a, int i, int t, float xp, float xq, float2 ps, float2 qs) {
  if (isnan(xp) || !sound(ps) || !sound(qs)) return false;
  const float u = uniform(philox(make_uint4(0u, a.step + t, (uint32_t)i, 2u), a.seed).x);
  const float p = ex2((xp - ps.x) * a.c) / ps.y, q = a.draft ? ex2((xq - qs.x) * a.draft_c) / qs.y : 1.0f;
  if (fabsf(u * q - p) > kNear * p && p >= 1e-30f) return u * q < p;
  return u * (a.draft ? probability64(xq, qs, a.draft_inverse) : 1.0) < probability64(xp, ps, a.inverse);
}
__device__ __forceinline__ float* logit_of(const VerifyArgs& a, int i, int t, int of_draft) { return a.logit + ((int64_t)i * (a.gamma + 1) + t) * 2 + of_draft; }

// Values for `first` and `arrived` before the rows.
__global__ void __launch_bounds__(256) verify_begin(const __grid_constant__ VerifyArgs a) {
  after_previous();
  const int k = blockIdx.x * 256 + threadIdx.x;
  if (k < a.n) a.first[k] = INT_MAX;
  if (k < a.n * (a.gamma + 1)) a.arrived[k] = 0;
}

// A part of a row's first largest value: its vector, and whether the part has NaN or +inf.
struct First {
  float top;
  int at, bad;
};
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

struct RowShared {
  Sums part[16];
  First first[16];
  int last;
};

// One part of a row by a CTA; its first warp gets what `parts` holds.
template <int DT, bool GREEDY, bool HELD, typename F>
__device__ __forceinline__ float2 row_part(const VerifyArgs& a, const Row& row, int part, float c, uint4* held, RowShared& s, F after_pass) {
  constexpr int N = Type<DT>::kPer, WARPS = Form<HELD>::kWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = row_groups<DT>(row), g0 = run_begin(groups, a.parts_shift, part), g1 = run_begin(groups, a.parts_shift, part + 1);
  if (HELD) hold_groups<DT>(row, g0, g1, held);
  if constexpr (GREEDY) {
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
    f = warp_first(s.first[lane & (WARPS - 1)]);
    int token = -1;
    if (tid == 0 && !f.bad && f.top > -INFINITY) {
      float x[N];
      values_of<DT>(load_vector<DT>(row, f.at), x);
#pragma unroll
      for (int k = N - 1; k >= 0; --k)
        if (x[k] == f.top) token = f.at * N + k - row.off;
    }
    return make_float2(f.bad ? NAN : f.top, __int_as_float(token));
  } else {
    Pass p;
    begin(p);
    auto step = [&](int, const uint4& v, const uint4& w) { take<DT, false>(p, v, w, fmaxf(largest<DT>(v), largest<DT>(w)), c); };
    if (HELD) over_held(g0, g1, held, step);
    else over_groups<DT>(row, g0, g1, step);
    Sums q = warp_joined(p, c);
    if (lane == 0) s.part[warp] = q;
    after_pass();
    __syncthreads();
    q = parts_joined(s.part[min(lane, WARPS - 1)], WARPS, c);
    return make_float2(q.ref, q.s);
  }
}

template <bool GREEDY, bool HELD>
__global__ void __launch_bounds__((Form<HELD>::kThreads), (Form<HELD>::kCtas)) verify_rows(const __grid_constant__ VerifyArgs a) {
  after_previous();
  __shared__ RowShared s;
  extern __shared__ __align__(16) uint4 held[];
  const int tid = threadIdx.x, pair = a.draft ? 1 : 0;
  // parts of a row, then target and draft, then entries, then places
  const unsigned rest = blockIdx.x >> a.parts_shift;
  const int part = blockIdx.x & ((1 << a.parts_shift) - 1), of_draft = rest & pair, t = (rest >> pair) / a.n, i = (rest >> pair) - t * a.n;
  const int have = drafts_of(a, i);
  if (t + of_draft > have) return;
  const void* p = of_draft ? a.draft : a.target;
  const int dtype = of_draft ? a.draft_dtype : a.target_dtype;
  const float c = of_draft ? a.draft_c : a.c;
  if (a.first) {
    if (__syncthreads_or(tid == 0 && *(volatile const int32_t*)(a.first + i) < t)) return;
  }
  const int64_t at = of_draft ? i * a.draft_stride_n + t * a.draft_stride_t : i * a.target_stride_n + t * a.target_stride_t;
  const int x = t < have ? __ldg(a.tokens + (int64_t)i * a.gamma + t) : -1;
  // the draft's logit, by a thread of the second warp: what the first arrives with comes after a barrier
  auto logit = [&] {
    if (part == 0 && tid == 32) __stcg(logit_of(a, i, t, of_draft), (unsigned)x < (unsigned)a.V ? load_one(p, at + x, dtype) : NAN);
  };
  float2 mine;
  if (dtype == WHEAD_BF16) mine = row_part<WHEAD_BF16, GREEDY, HELD>(a, row_at<WHEAD_BF16>(p, at, a.V), part, c, held, s, logit);
  else if (dtype == WHEAD_F16) mine = row_part<WHEAD_F16, GREEDY, HELD>(a, row_at<WHEAD_F16>(p, at, a.V), part, c, held, s, logit);
  else mine = row_part<WHEAD_F32, GREEDY, HELD>(a, row_at<WHEAD_F32>(p, at, a.V), part, c, held, s, logit);
  if (tid >= 32) return;
  if (tid == 0) {
    __stcg(parts_of(a, i, t, of_draft) + part, mine);
    s.last = 0;
    if (a.first && t < have) {
      unsigned done;
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(done) : "l"(a.arrived + (int64_t)i * (a.gamma + 1) + t) : "memory");
      s.last = done + 1 == (1u + pair) << a.parts_shift;
    }
  }
  __syncwarp();
  if (!s.last) return;
  // the place is done: its draft is decided on
  bool stays;
  if constexpr (GREEDY) {
    stays = x >= 0 && row_token(a, i, t) == x;
  } else {
    const float2 ps = row_sums(a, i, t, 0), qs = pair ? row_sums(a, i, t, 1) : make_float2(0.0f, 1.0f);
    stays = draft_stays(a, i, t, __ldcg(logit_of(a, i, t, 0)), pair ? __ldcg(logit_of(a, i, t, 1)) : 0.0f, ps, qs);
  }
  if (tid == 0 && !stays) atomicMin(a.first + i, t);
}

// One entry's row of `said`, and its count.
__device__ __forceinline__ void write_said(const VerifyArgs& a, int i, int stay, int next, int tid, int threads) {
  for (int t = tid; t <= a.gamma; t += threads) a.said[(int64_t)i * (a.gamma + 1) + t] = t < stay ? a.tokens[(int64_t)i * a.gamma + t] : t == stay ? next : -1;
  if (tid == 0) a.count[i] = stay + 1;
}

// Temperature 0, an entry a CTA, a place a thread.
__global__ void __launch_bounds__(256) verify_greedy(const __grid_constant__ VerifyArgs a) {
  after_previous();
  __shared__ int stay, next;
  const int i = blockIdx.x, t = threadIdx.x, have = drafts_of(a, i);
  const int known = a.first ? min(a.first[i], have) : have;  // the rows up to here are done
  if (t == 0) stay = known;
  const int x = t < known ? a.tokens[(int64_t)i * a.gamma + t] : -1, token = t <= known ? row_token(a, i, t) : -1;
  __syncthreads();
  if (t < known && (x < 0 || token != x)) atomicMin(&stay, t);
  __syncthreads();
  if (t == stay) next = token;
  __syncthreads();
  write_said(a, i, stay, next, t, blockDim.x);
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
// Over a warp; every lane gets them. Keys are not negative, and such floats are ordered as their bits.
__device__ __forceinline__ Best warp_best(Best b) {
  const unsigned high = __reduce_max_sync(~0u, b.v1 >= 0 ? __float_as_uint(b.k1) : 0u);
  const int v = __reduce_min_sync(~0u, b.v1 >= 0 && __float_as_uint(b.k1) == high ? b.v1 : INT_MAX);
  const bool won = b.v1 == v;
  const float k2 = won ? b.k2 : b.k1;
  const int v2 = won ? b.v2 : b.v1;
  const unsigned next = __reduce_max_sync(~0u, v2 >= 0 ? __float_as_uint(k2) : 0u);
  const int w = __reduce_min_sync(~0u, v2 >= 0 && __float_as_uint(k2) == next ? v2 : INT_MAX);
  return Best{__uint_as_float(high), __uint_as_float(next), v == INT_MAX ? -1 : v, w == INT_MAX ? -1 : w};
}

struct DrawShared {
  int stay, next, known;
  float2 ps[WHEAD_MAX_DRAFTS + 1], qs[WHEAD_MAX_DRAFTS + 1];
  Best part[kDrawWarps];
  Best cluster[kMaxCluster];
};

// Four logits from `at` on, as they are; `wide`: they can be read as one.
template <int DT>
using Quad = std::conditional_t<DT == WHEAD_F32, uint4, uint2>;
template <int DT, bool WIDE>
__device__ __forceinline__ Quad<DT> load_quad(const void* p, int64_t at) {
  if constexpr (DT == WHEAD_F32) {
    const uint32_t* x = static_cast<const uint32_t*>(p) + at;
    if constexpr (WIDE) return __ldg(reinterpret_cast<const uint4*>(x));
    else return make_uint4(__ldg(x), __ldg(x + 1), __ldg(x + 2), __ldg(x + 3));
  } else {
    const unsigned short* x = static_cast<const unsigned short*>(p) + at;
    if constexpr (WIDE) return __ldg(reinterpret_cast<const uint2*>(x));
    else return make_uint2(__ldg(x) | (uint32_t)__ldg(x + 1) << 16, __ldg(x + 2) | (uint32_t)__ldg(x + 3) << 16);
  }
}
template <int DT>
__device__ __forceinline__ Quad<DT> no_quad() {
  constexpr uint32_t x = Type<DT>::kNone;
  if constexpr (DT == WHEAD_F32) return make_uint4(x, x, x, x);
  else return make_uint2(x, x);
}
// A row's last ones, fewer than four; -inf for the rest.
template <int DT>
__device__ __noinline__ Quad<DT> load_last(const void* p, int64_t at, int live) {
  uint32_t w[4];
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == WHEAD_F32) w[k] = k < live ? __ldg(static_cast<const uint32_t*>(p) + at + k) : Type<DT>::kNone;
    else w[k] = k < live ? (uint32_t)__ldg(static_cast<const unsigned short*>(p) + at + k) : Type<DT>::kNone & 0xFFFFu;
  }
  if constexpr (DT == WHEAD_F32) return make_uint4(w[0], w[1], w[2], w[3]);
  else return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
template <int DT>
__device__ __forceinline__ void quad_values(const Quad<DT>& v, float (&x)[4]) {
  if constexpr (DT == WHEAD_F32) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  } else {
    const float2 lo = whead_kv_impl::unpack16(v.x, DT), hi = whead_kv_impl::unpack16(v.y, DT);
    x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
  }
}

// The row that a token is drawn from.
struct DrawRow {
  int64_t p_at, q_at;
  float2 ps, qs;
  int stay, drafted;       // the draft that does not stay, -1: none
  bool q, wide;            // there is a row of the draft's to take off; quads can be read as one
};

// The best tokens of four at a time, from `from` on in steps; `whole`: of p itself, else of max(p - q, 0). Philox takes half of the issue
// slots, the exponentials as long on their own unit. A token that the bound does not rule out (a few dozen of a CTA) takes a loop of its own,
// so that its logarithm and division are there once and not eight times in the loop over all.
template <int PT, int QT, bool WIDE>
__device__ __forceinline__ Best draw(const VerifyArgs& a, const DrawRow& d, int i, int from, int step, bool whole, DrawShared& s) {
  constexpr int kTurn = 2;             // quads of a thread whose loads are under way at once
  constexpr int DT = QT < 0 ? PT : QT; // of the draft's row, where there is one
  Best best{0.0f, 0.0f, -1, -1};
  const float p_off = -log2f(d.ps.y), q_off = -log2f(d.qs.y);
  const bool with_q = QT >= 0 && d.q && !whole;
  const int quads = (a.V + 3) / 4, full = a.V / 4, taken = QT < 0 && !whole ? d.drafted : -1;
  constexpr float kBelow = 1.0f - 2.0f * kNearOfDifference;  // so that the keys that are settled with the best are not ruled out
  float known = 0.0f;  // kBelow times the CTA's best key, as far as this warp knows it
#pragma unroll 1
  for (int g0 = from; __any_sync(~0u, g0 < quads); g0 += kTurn * step) {
    Quad<PT> x[kTurn];
    Quad<DT> y[kTurn];
#pragma unroll
    for (int n = 0; n < kTurn; ++n) {
      const int g = g0 + n * step;
      if (g < full) {
        x[n] = load_quad<PT, WIDE>(a.target, d.p_at + 4 * g);
        if (with_q) y[n] = load_quad<DT, WIDE>(a.draft, d.q_at + 4 * g);
      } else if (g < quads) {
        x[n] = load_last<PT>(a.target, d.p_at + 4 * g, a.V - 4 * g);
        if (with_q) y[n] = load_last<DT>(a.draft, d.q_at + 4 * g, a.V - 4 * g);
      } else {
        x[n] = no_quad<PT>();
        y[n] = no_quad<DT>();
      }
    }
    float r[4 * kTurn];
    uint32_t w[4 * kTurn];
#pragma unroll
    for (int n = 0; n < kTurn; ++n) {
      const int g = g0 + n * step;
      const uint4 word = philox(make_uint4((uint32_t)g, a.step + d.stay, (uint32_t)i, 1u), a.seed);
      w[4 * n] = word.x; w[4 * n + 1] = word.y; w[4 * n + 2] = word.z; w[4 * n + 3] = word.w;
      float p[4];
      quad_values<PT>(x[n], p);
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = ex2(__fmaf_rn(p[k] - d.ps.x, a.c, p_off));
      if (with_q) {
        float q[4];
        quad_values<DT>(y[n], q);
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] -= ex2(__fmaf_rn(q[k] - d.qs.x, a.draft_c, q_off));
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) r[4 * n + k] = QT < 0 && taken == 4 * g + k ? 0.0f : p[k];
    }
    // E < (1 - U) / U: a key that is reached, before any is known. By a vote: every lane has read s.known for itself while others raise it, and
    // warp_max needs all lanes to come.
    if (__all_sync(~0u, known == 0.0f)) {
      float low = 0.0f;
#pragma unroll
      for (int e = 0; e < 4 * kTurn; ++e) {
        const float u = uniform(w[e]);
        low = fmaxf(low, r[e] * __fdividef(u, 1.0f - u));
      }
      known = warp_max(low) * kBelow;
    }
    // r / E <= r / (1 - U) and 1 - U > 2 - 2^-23 - f, f = 1 + (w >> 9) 2^-23
    auto over = [&](int e) { return __fmaf_rn(known, __uint_as_float(__funnelshift_r(w[e], 0x7Fu, 9)) - (2.0f - 0x1p-23f), r[e]); };
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < 4 * kTurn; ++e) most = fmaxf(most, over(e));
    if (__any_sync(~0u, most > 0.0f)) {
      unsigned may = 0;
#pragma unroll
      for (int e = 0; e < 4 * kTurn; ++e) may |= over(e) > 0.0f ? 1u << e : 0u;
      while (may) {
        const int e = __ffs(may) - 1;
        may &= may - 1;
        float re = 0.0f;
        uint32_t we = 0;
#pragma unroll
        for (int n = 0; n < 4 * kTurn; ++n)
          if (n == e) {
            re = r[n];
            we = w[n];
          }
        add(best, re / -logf(uniform(we)), 4 * (g0 + e / 4 * step) + e % 4);
      }
      __syncwarp();
      const float high = warp_max(best.k1);
      if ((threadIdx.x & 31) == 0) atomicMax(&s.known, __float_as_int(high));
      known = fmaxf(known, high * kBelow);
    }
    known = fmaxf(known, __int_as_float(*(volatile int*)&s.known) * kBelow);
  }
  return best;
}

// The best of a CTA, in its first warp.
__device__ __forceinline__ Best cta_best(Best b, DrawShared& s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  b = warp_best(b);
  if (lane == 0) s.part[warp] = b;
  __syncthreads();
  if (warp == 0) {
    b = lane < kDrawWarps ? s.part[lane] : Best{0.0f, 0.0f, -1, -1};
    b = warp_best(b);
  }
  return b;
}

// PT, QT: types of the target's and the draft's logits, QT -1: drafts without logits.
template <int PT, int QT>
__global__ void __launch_bounds__(kDrawThreads, 2) verify_draw(const __grid_constant__ VerifyArgs a) {
  after_previous();
  __shared__ DrawShared s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = 1 << a.ctas_shift, i = blockIdx.x >> a.ctas_shift, rank = blockIdx.x & (ctas - 1);
  const int have = drafts_of(a, i);
  const int known = a.first ? min(a.first[i], have) : have;  // the rows up to here are done
  const int32_t* tokens = a.tokens + (int64_t)i * a.gamma;
  if (ctas > 1) cluster_arrive();
  if (tid == 0) {
    s.stay = known;
    s.known = 0;
  }
  __syncthreads();
  // which drafts stay: where rows have been left out it is known already
  for (int t = a.first ? known + warp : warp; t <= known; t += kDrawWarps) {
    const float xp = __ldcg(logit_of(a, i, t, 0)), xq = a.draft ? __ldcg(logit_of(a, i, t, 1)) : 0.0f;
    const float2 ps = row_sums(a, i, t, 0), qs = t < have && a.draft ? row_sums(a, i, t, 1) : make_float2(0.0f, 1.0f);
    if (lane == 0) {
      s.ps[t] = ps;
      s.qs[t] = qs;
      if (t < known && !draft_stays(a, i, t, xp, xq, ps, qs)) atomicMin(&s.stay, t);
    }
  }
  __syncthreads();
  DrawRow d;
  d.stay = s.stay;
  d.ps = s.ps[d.stay];
  d.qs = s.qs[d.stay];
  const bool some = sound(d.ps), rejected = d.stay < have;
  d.drafted = rejected ? tokens[d.stay] : -1;
  d.q = rejected && a.draft && sound(d.qs);
  d.p_at = i * a.target_stride_n + d.stay * a.target_stride_t;
  d.q_at = i * a.draft_stride_n + d.stay * a.draft_stride_t;
  auto wide = [](const void* p, int64_t at, int size) { return ((reinterpret_cast<uintptr_t>(p) + at * size) & (4 * size - 1)) == 0; };
  d.wide = wide(a.target, d.p_at, Type<PT>::kSize) && (QT < 0 || !d.q || wide(a.draft, d.q_at, QT == WHEAD_F32 ? 4 : 2));
  bool whole = !rejected, alone = ctas == 1;
  Best best;
  while (true) {
    best = Best{0.0f, 0.0f, -1, -1};
    const int from = alone ? tid : rank * kDrawThreads + tid, step = alone ? kDrawThreads : ctas * kDrawThreads;
    if (some) best = d.wide ? draw<PT, QT, true>(a, d, i, from, step, whole, s) : draw<PT, QT, false>(a, d, i, from, step, whole, s);
    best = cta_best(best, s);
    if (!alone) {
      cluster_wait();  // all have started
      if (tid == 0) *in_first(&s.cluster[rank]) = best;
      __syncwarp();
      cluster_arrive();
      if (rank != 0) return;
      cluster_wait();
      if (warp == 0) best = warp_best(lane < ctas ? s.cluster[lane] : Best{0.0f, 0.0f, -1, -1});
      alone = true;
    }
    if (tid == 0) s.next = best.v1;
    __syncthreads();
    if (!some || whole || s.next >= 0) break;
    whole = true;  // rounding left nothing of p - q: from p, by this CTA
  }
  const bool difference = QT >= 0 && !whole && d.q;
  if (tid == 0 && best.v2 >= 0 && best.k1 - best.k2 <= (difference ? kNearOfDifference : kNear) * best.k1) {
    double key[2];
#pragma unroll 1
    for (int k = 0; k < 2; ++k) {
      const int v = k ? best.v2 : best.v1;
      double r = probability64(load_one(a.target, d.p_at + v, PT), d.ps, a.inverse);
      if (difference) r -= probability64(load_one(a.draft, d.q_at + v, QT), d.qs, a.draft_inverse);
      const uint4 word = philox(make_uint4((uint32_t)v >> 2, a.step + d.stay, (uint32_t)i, 1u), a.seed);
      const uint32_t w = v & 2 ? (v & 1 ? word.w : word.z) : (v & 1 ? word.y : word.x);
      key[k] = r / -log((double)uniform(w));
    }
    if (key[1] > key[0] || (key[1] == key[0] && best.v2 < best.v1)) s.next = best.v2;
  }
  __syncthreads();
  write_said(a, i, d.stay, s.next, tid, kDrawThreads);
}

template <bool GREEDY, bool HELD>
int launch_rows(const VerifyArgs& a, int64_t ctas, int device, cudaStream_t stream) {
  static std::atomic<bool> granted[kMaxDevices];
  return launch_clusters(verify_rows<GREEDY, HELD>, ctas, 1, Form<HELD>::kThreads, HELD ? a.held * kGroup * 16 : 0, stream, granted, device, a);
}

// Parts of a row, as a power of two: by the entries alone, so that the workspace's size does not depend on the device or on V.
int most_parts_shift(int64_t n) {
  int s = 4;
  while (s > 0 && n << s > 512) --s;
  return s;
}
static_assert(kMaxParts == 1 << 4, "");

struct Layout {
  int64_t logit, first, arrived, total;
};
Layout layout(int64_t n, int gamma) {
  const int64_t places = n * (gamma + 1);
  Layout l;
  l.logit = whead_kv_impl::align256((places * 2 << most_parts_shift(n)) * (int64_t)sizeof(float2));
  l.first = l.logit + whead_kv_impl::align256(places * 2 * 4);
  l.arrived = l.first + whead_kv_impl::align256(n * 4);
  l.total = l.arrived + whead_kv_impl::align256(places * 4);
  return l;
}

template <int PT, int QT>
int launch_draw(const VerifyArgs& a, int device, cudaStream_t stream) {
  static std::atomic<bool> granted[kMaxDevices];
  return launch_clusters(verify_draw<PT, QT>, a.n, 1 << a.ctas_shift, kDrawThreads, 0, stream, granted, device, a);
}
template <int PT>
int launch_draw(const VerifyArgs& a, int device, cudaStream_t stream) {
  if (!a.draft) return launch_draw<PT, -1>(a, device, stream);
  switch (a.draft_dtype) {
    case WHEAD_BF16: return launch_draw<PT, WHEAD_BF16>(a, device, stream);
    case WHEAD_F16: return launch_draw<PT, WHEAD_F16>(a, device, stream);
    default: return launch_draw<PT, WHEAD_F32>(a, device, stream);
  }
}

int launch(const VerifyArgs& from, int device, int sms, cudaStream_t stream) {
  VerifyArgs a = from;
  const bool greedy = a.inverse == 0.0;
  const int pair = a.draft ? 1 : 0;
  const int64_t places = (int64_t)a.n * (a.gamma + 1), bytes = (int64_t)a.V * std::max(dtype_size(a.target_dtype), pair ? dtype_size(a.draft_dtype) : 0);
  // parts of 16 KB or more, as many as there is room for (by the entries). 1 x 16 on 151,936, bf16: 14.1 us by parts of 16 or 32 KB, 15.2 by 64; 1 x 4
  // on 32,003 8.2 by 8 KB, 8.8 by 16, 9.6 by 32; 30 x 8 greedy, where 16 parts make a place half of the device, 21.8, by 8 parts 17.6.
  auto groups = [&](int shift) { return (int)(((bytes / (kGroup * 16) + 2) >> shift) + 1); };
  auto fits = [&](int shift) { return groups(shift) <= kHeldGroups && places << (pair + shift) <= (int64_t)sms * Form<true>::kCtas; };
  int shift = 0;
  while (shift < most_parts_shift(a.n) && bytes >> (shift + 1) >= 16384) ++shift;
  // parts held where all are there at once so, if need be in fewer parts
  int less = shift;
  while (less > 0 && !fits(less)) --less;
  const bool held = fits(less);
  a.parts_shift = held ? less : shift;
  int rc = WHEAD_OK;
  if (!held && a.gamma > 0 && ((int64_t)a.n << (pair + shift)) * 2 >= (int64_t)sms * Form<false>::kCtas) {
    // One place's parts take half of the device or more: what is decided in time is left out. (64 entries of 16 drafts, f32 drafts' logits,
    // a draft in five refused: 97 us, 200 without; 8 entries, greedy, f32, where a place takes a seventh: 19.0 us, 17.4 without.)
    rc = whead_kv_impl::launch_after(verify_begin, dim3((unsigned)((places + 255) / 256)), 256, 0, stream, a);
  } else {
    // no more parts than fill half of the device (8 entries, greedy: 4 parts a row 17.4 us, 16 parts 19.1)
    a.first = nullptr;
    while (!held && a.parts_shift > 0 && (places << (pair + a.parts_shift - 1)) * 2 >= (int64_t)sms * Form<false>::kCtas) --a.parts_shift;
  }
  const int64_t ctas = places << (pair + a.parts_shift);
  a.held = groups(a.parts_shift);
  if (rc != WHEAD_OK) return rc;
  if (greedy) rc = held ? launch_rows<true, true>(a, ctas, device, stream) : launch_rows<true, false>(a, ctas, device, stream);
  else rc = held ? launch_rows<false, true>(a, ctas, device, stream) : launch_rows<false, false>(a, ctas, device, stream);
  if (rc != WHEAD_OK) return rc;
  if (greedy) return whead_kv_impl::launch_after(verify_greedy, dim3((unsigned)a.n), (a.gamma + 32) / 32 * 32, 0, stream, a);
  // CTAs of an entry: up to three an SM, though two find room at once, and four quads a thread at least. Whole calls, by three and by two an SM: 40
  // entries of 4 drafts on 151,936 48.8 and 49.9 us, 48 56.1 and 53.6, 56 60.9 and 57.1, 64 alike, 80 83.5 and 87.4, 200 166.7 and 174.1. One
  // entry of 16,000: 8.7 us by four quads, 9.7 by eight, 10.6 by sixteen.
  a.ctas_shift = 0;
  while ((2 << a.ctas_shift) <= kMaxCluster && (int64_t)a.n << (a.ctas_shift + 1) <= (int64_t)sms * 3 && a.V >> (a.ctas_shift + 1) >= 4 * kDrawThreads) ++a.ctas_shift;
  switch (a.target_dtype) {
    case WHEAD_BF16: return launch_draw<WHEAD_BF16>(a, device, stream);
    case WHEAD_F16: return launch_draw<WHEAD_F16>(a, device, stream);
    default: return launch_draw<WHEAD_F32>(a, device, stream);
  }
}

}  // namespace

}  // namespace whead_verify_impl

using namespace whead_verify_impl;

extern "C" int64_t whead_verify_workspace_bytes(int64_t n, int32_t gamma) {
  if (n < 0 || gamma < 0) return WHEAD_ERR_INVALID_ARG;
  if (gamma > WHEAD_MAX_DRAFTS || n > ((1 << 27) - 1) / (2 * gamma + 2)) return WHEAD_ERR_UNSUPPORTED;
  return layout(n, gamma).total;
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
  const Layout l = layout(x->n, x->gamma);
  char* w = static_cast<char*>(x->workspace);
  VerifyArgs a{};
  a.target = x->target;
  a.draft = with_draft ? x->draft : nullptr;
  a.tokens = x->tokens;
  a.drafted = x->drafted;
  a.said = x->said;
  a.count = x->count;
  a.parts = reinterpret_cast<float2*>(w);
  a.logit = reinterpret_cast<float*>(w + l.logit);
  a.first = reinterpret_cast<int32_t*>(w + l.first);
  a.arrived = reinterpret_cast<int32_t*>(w + l.arrived);
  a.target_stride_n = x->target_stride_n;
  a.target_stride_t = x->target_stride_t;
  a.draft_stride_n = x->draft_stride_n;
  a.draft_stride_t = x->draft_stride_t;
  a.V = (int)x->V;
  a.gamma = x->gamma;
  a.target_dtype = x->target_dtype;
  a.draft_dtype = x->draft_dtype;
  a.step = x->step;
  a.n = (int)x->n;
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

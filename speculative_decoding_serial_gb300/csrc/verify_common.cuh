// verify_common.cuh — what the kernels over rows of logits share: vectors of logits, one pass over a part of a row, and the joining of its parts.
//
// A row of V logits is taken in vectors of 16 bytes, 64 of them (two a lane, 1 KB) being a group; a row's first and last
// vector may lie across its ends, since rows start anywhere. A cluster of CTAs has a row, each CTA a run of its groups.
#pragma once

#include "../../include/whead_verify.h"
#include "kv_common.cuh"

#include <cooperative_groups.h>

namespace whead_verify_impl {

using whead_kv_impl::after_previous;
using whead_kv_impl::aligned;
using whead_kv_impl::ex2;
using whead_kv_impl::kLn2;
using whead_kv_impl::kLog2e;
using whead_kv_impl::kMaxDevices;

constexpr int kGroup = 64;         // vectors of a group
constexpr int kMaxCluster = 8;     // clusters of 16 do not all find room at once: 17 rows of 608 KB take 16 us by them, 9 by clusters of 8

// Two forms of a CTA. For many rows: 256 threads, two groups a warp under way, the rest by the SM's other CTAs. For few rows: 512 threads that
// ask for their whole part of the row at once, by copies to shared memory, so that the call waits for memory once, not turn by turn; the
// loop over it is rolled, since code that runs once is fetched more slowly than it runs.
template <bool HELD>
struct Form {
  static constexpr int kThreads = HELD ? 512 : 256, kWarps = kThreads / 32;
  static constexpr int kCtas = HELD ? 2 : 6;
};
constexpr int kAhead = 2;       // groups of a warp under way
constexpr int kHeldGroups = 90; // of a CTA: two CTAs an SM

constexpr float kLowest = -3.402823466e38f;

// Types: values in a vector, and keys, whole numbers in the values' order (-0 counts as +0).
template <int DT>
struct Type {
  static constexpr int kPer = DT == WHEAD_F32 ? 4 : 8;
  static constexpr int kSize = DT == WHEAD_F32 ? 4 : 2;
  static constexpr int kKeyBits = DT == WHEAD_F32 ? 32 : 16;
  static constexpr uint32_t kNone = DT == WHEAD_F32 ? 0xFF800000u : DT == WHEAD_BF16 ? 0xFF80FF80u : 0xFC00FC00u;  // -inf, as a vector holds it
  static constexpr uint32_t kNoneKey = DT == WHEAD_F32 ? 0x007FFFFFu : DT == WHEAD_BF16 ? 0x007Fu : 0x03FFu;
};

template <int DT>
__device__ __forceinline__ uint32_t key_of(float x) {
  x += 0.0f;
  if constexpr (DT == WHEAD_F32) {
    const uint32_t b = __float_as_uint(x);
    return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
  } else {
    const uint32_t b = DT == WHEAD_BF16 ? __float_as_uint(x) >> 16 : (uint32_t)__half_as_ushort(__float2half_rn(x));
    return b & 0x8000u ? b ^ 0xFFFFu : b | 0x8000u;
  }
}
template <int DT>
__device__ __forceinline__ float value_of(uint32_t key) {
  if constexpr (DT == WHEAD_F32) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
  } else {
    const uint32_t b = key & 0x8000u ? key ^ 0x8000u : key ^ 0xFFFFu;
    return DT == WHEAD_BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half((unsigned short)b));
  }
}

__device__ __forceinline__ float load_one(const void* p, int64_t at, int dtype) {
  if (dtype == WHEAD_F32) return __ldg(static_cast<const float*>(p) + at);
  const unsigned short b = __ldg(static_cast<const unsigned short*>(p) + at);
  return dtype == WHEAD_BF16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// A row: where its first vector is (16-byte aligned, at or before its first value), how many values of it come before the row, and
// how many the row has.
struct Row {
  const char* base;
  int off, V;
};
template <int DT>
__device__ __forceinline__ Row row_at(const void* logits, int64_t at, int V) {
  const char* p = static_cast<const char*>(logits) + at * Type<DT>::kSize;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Row{reinterpret_cast<const char*>(a & ~(uintptr_t)15), (int)(a & 15) / Type<DT>::kSize, V};
}
template <int DT>
__device__ __forceinline__ int row_groups(const Row& r) { return (r.off + r.V + kGroup * Type<DT>::kPer - 1) / (kGroup * Type<DT>::kPer); }

__device__ __forceinline__ uint4 load16(const char* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// Vector j of a row; places outside the row hold -inf.
template <int DT>
__device__ __forceinline__ uint4 load_vector(const Row& r, int j) {
  constexpr int N = Type<DT>::kPer;
  const int first = j * N - r.off;
  if (first >= 0 && first + N <= r.V) return load16(r.base + (int64_t)j * 16);
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    w[k] = Type<DT>::kNone;
    if constexpr (DT == WHEAD_F32) {
      if ((unsigned)(first + k) < (unsigned)r.V) w[k] = __ldg(reinterpret_cast<const uint32_t*>(r.base) + (int64_t)j * 4 + k);
    } else {
      const unsigned short* p = reinterpret_cast<const unsigned short*>(r.base) + (int64_t)j * 8 + 2 * k;
      if ((unsigned)(first + 2 * k) < (unsigned)r.V) w[k] = (w[k] & 0xFFFF0000u) | __ldg(p);
      if ((unsigned)(first + 2 * k + 1) < (unsigned)r.V) w[k] = (w[k] & 0xFFFFu) | (uint32_t)__ldg(p + 1) << 16;
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DT>
__device__ __forceinline__ void values_of(const uint4& v, float (&x)[Type<DT>::kPer]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == WHEAD_F32) {
      x[k] = __uint_as_float(w[k]);
    } else if constexpr (DT == WHEAD_BF16) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    } else {
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      x[2 * k] = y.x;
      x[2 * k + 1] = y.y;
    }
  }
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The largest value of a vector, NaN left out.
template <int DT>
__device__ __forceinline__ float largest(const uint4& v) {
  if constexpr (DT == WHEAD_F32) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else if constexpr (DT == WHEAD_BF16) {
    auto as = [](const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const float2 m = __bfloat1622float2(__hmax2(__hmax2(as(v.x), as(v.y)), __hmax2(as(v.z), as(v.w))));
    return fmaxf(m.x, m.y);
  } else {
    auto as = [](const uint32_t& w) { return *reinterpret_cast<const __half2*>(&w); };
    const float2 m = __half22float2(__hmax2(__hmax2(as(v.x), as(v.y)), __hmax2(as(v.z), as(v.w))));
    return fmaxf(m.x, m.y);
  }
}

// The same, NaN if the vector holds one.
template <int DT>
__device__ __forceinline__ float largest_nan(const uint4& v) {
  if constexpr (DT == WHEAD_F32) {
    return max_nan(max_nan(__uint_as_float(v.x), __uint_as_float(v.y)), max_nan(__uint_as_float(v.z), __uint_as_float(v.w)));
  } else if constexpr (DT == WHEAD_BF16) {
    auto as = [](const uint32_t& w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const float2 m = __bfloat1622float2(__hmax2_nan(__hmax2_nan(as(v.x), as(v.y)), __hmax2_nan(as(v.z), as(v.w))));
    return max_nan(m.x, m.y);
  } else {
    auto as = [](const uint32_t& w) { return *reinterpret_cast<const __half2*>(&w); };
    const float2 m = __half22float2(__hmax2_nan(__hmax2_nan(as(v.x), as(v.y)), __hmax2_nan(as(v.z), as(v.w))));
    return max_nan(m.x, m.y);
  }
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
// A part's sums: s of 2^d and a of d 2^d, with d = x c - k, c = log2(e) / T, k = ref c rounded: one multiply-add, exact but for its own
// rounding, since k is what the sums refer to, whatever it was rounded from. From 2^23 on that rounding would be no small power of two any
// more (rows at the type's lowest value, temperatures near 0): there d is (x - ref) c, the difference formed before the product,
// which is right for any two finite logits.
struct Sums {
  float ref, s, a;
};
__device__ __forceinline__ bool plain(float k) { return fabsf(k) < 0x1p23f; }
// What a reference's k was rounded by: s is the sum of 2^((x - ref) c) times 2^off, off some 2^-24 of k, up to a quarter where k is near 2^23.
__device__ __forceinline__ float offset_of(float ref, float c) {
  const float k = __fmul_rn(ref, c);
  return plain(k) ? __fmaf_rn(ref, c, -k) : 0.0f;
}
// What d becomes less by when the reference goes from one value to another (at most 10,000: 2^-10000 is 0, and times 0 too). Where one of them has a
// k and the other none, the sums go from one way of referring to the other.
__device__ __forceinline__ float shift_of(float from, float to, float c) {
  const float k0 = __fmul_rn(from, c), k1 = __fmul_rn(to, c);  // as they are: not within a multiply-add
  return max_nan(plain(k0) && plain(k1) ? k0 - k1 : (from - to) * c + (offset_of(to, c) - offset_of(from, c)), -1e4f);
}
// The same sums for another reference. A part without a value has s = a = 0 and any reference.
__device__ __forceinline__ Sums moved(const Sums& p, float ref, float c) {
  if (p.s == 0.0f) return Sums{ref, 0.0f, 0.0f};
  const float d = shift_of(p.ref, ref, c), f = ex2(d);
  return Sums{ref, p.s * f, f == 0.0f ? 0.0f : (p.a + p.s * d) * f};
}

// One thread's way through its groups. The reference is raised when a group's largest value passes it by kSlack (in log2 units), so that
// most groups change nothing; sums then reach 2^kSlack times their number, and a, which loses kSlack units of 2^-24 when it is moved to the
// row's largest, costs the entropy 5e-7 at most.
constexpr float kSlack = 8.0f;
struct Pass {
  float ref, k, limit, top;
  bool careful;  // d may be -inf (then d 2^d would be NaN) or has to be formed from the difference
  bool masked;   // -inf has been met
  float2 s, a;
};
__device__ __forceinline__ void begin(Pass& p) {
  p.ref = p.limit = kLowest;
  p.k = p.top = -INFINITY;
  p.careful = true;
  p.masked = false;
  p.s = p.a = make_float2(0.0f, 0.0f);
}
template <int DT, bool ENTROPY, bool CAREFUL>
__device__ __forceinline__ void add_vector(Pass& p, const uint4& raw, float c) {
  constexpr int N = Type<DT>::kPer;
  float x[N];
  values_of<DT>(raw, x);
  const bool is_plain = plain(p.k);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float2 d;
    if (!CAREFUL || is_plain) d = fma2(make_float2(x[i], x[i + 1]), make_float2(c, c), make_float2(-p.k, -p.k));
    else d = mul2(add2(make_float2(x[i], x[i + 1]), make_float2(-p.ref, -p.ref)), make_float2(c, c));
    if (ENTROPY && CAREFUL) d = make_float2(max_nan(d.x, -200.0f), max_nan(d.y, -200.0f));
    const float2 e = make_float2(ex2(d.x), ex2(d.y));
    p.s = add2(p.s, e);
    if (ENTROPY) p.a = fma2(e, d, p.a);
  }
}
// Adds two vectors whose largest value is `high`. NaN and +inf end in s as NaN (+inf as its own reference: inf - inf). Values of -inf, or so
// far below the reference that d is -inf, add nothing, but would make a NaN: where a is NaN and s is not, the vectors are added once more
// with d cut off at -200, and so are the thread's later ones (cutting off always costs one instruction in six).
template <int DT, bool ENTROPY>
__device__ __forceinline__ void take(Pass& p, const uint4& v, const uint4& w, float high, float c) {
  p.top = fmaxf(p.top, high);
  if (high > p.limit) {
    const float d = shift_of(p.ref, high, c), f = ex2(d);
    if (ENTROPY) p.a = mul2(fma2(p.s, make_float2(d, d), p.a), make_float2(f, f));
    p.s = mul2(p.s, make_float2(f, f));
    p.ref = high;
    p.k = high * c;
    p.limit = high + kSlack / c;
    p.careful = p.masked || !plain(p.k);
  }
  if (!p.careful) {
    const float2 s = p.s, a = p.a;
    add_vector<DT, ENTROPY, false>(p, v, c);
    add_vector<DT, ENTROPY, false>(p, w, c);
    if (!ENTROPY) return;
    const float check = p.a.x + p.a.y;
    if (check == check) return;
    p.s = s;
    p.a = a;
    p.careful = p.masked = true;
  }
#pragma unroll 1
  for (int k = 0; k < 2; ++k) add_vector<DT, ENTROPY, true>(p, k ? w : v, c);
}

// Over the groups g0 .. g1 - 1 of a row, a warp a group, two vectors of each a lane: f(group, vector, vector). Groups inside the row are
// loaded without looking at its ends, several of them at a time.
template <int DT, typename F>
__device__ __forceinline__ void over_groups(const Row& row, int g0, int g1, F f) {
  constexpr int kWarps = Form<false>::kWarps;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inner0 = row.off ? 1 : 0, inner1 = (row.off + row.V) / (kGroup * Type<DT>::kPer);
  const int lo = max(g0, inner0), hi = min(g1, inner1);
  const char* at = row.base + ((int64_t)(lo + warp) * kGroup + lane) * 16;
  for (int g = lo + warp; g < hi; g += kWarps * kAhead, at += kWarps * kAhead * kGroup * 16) {
    uint4 v[kAhead], w[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (g + k * kWarps < hi) {
        v[k] = load16(at + k * kWarps * kGroup * 16);
        w[k] = load16(at + k * kWarps * kGroup * 16 + 512);
      }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (g + k * kWarps < hi) f(g + k * kWarps, v[k], w[k]);
  }
  // the groups across the row's ends
  if (warp >= 2) return;
  const int g = warp == 0 ? 0 : max(inner0, inner1);
  if (g >= g0 && g < g1 && (warp || inner0)) f(g, load_vector<DT>(row, g * kGroup + lane), load_vector<DT>(row, g * kGroup + 32 + lane));
}

// The other form: the groups to shared memory, group g at 64 (g - g0), all under way at once; and then over them. A thread
// takes what it has asked for itself, so that no barrier is needed before.
template <int DT>
__device__ __forceinline__ void hold_groups(const Row& row, int g0, int g1, uint4* held) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int inner0 = row.off ? 1 : 0, inner1 = (row.off + row.V) / (kGroup * Type<DT>::kPer);
#pragma unroll 2
  for (int g = g0 + warp; g < g1; g += Form<true>::kWarps) {
    uint4* to = held + (g - g0) * kGroup + lane;
    const int j = g * kGroup + lane;
    if (g >= inner0 && g < inner1) {
      const char* from = row.base + (int64_t)j * 16;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(whead_kv_impl::smem_u32(to)), "l"(from) : "memory");
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(whead_kv_impl::smem_u32(to + 32)), "l"(from + 512) : "memory");
    } else {
      to[0] = load_vector<DT>(row, j);
      to[32] = load_vector<DT>(row, j + 32);
    }
  }
}
template <typename F>
__device__ __forceinline__ void over_held(int g0, int g1, const uint4* held, F f) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 1
  for (int g = g0 + warp; g < g1; g += Form<true>::kWarps) f(g, held[(g - g0) * kGroup + lane], held[(g - g0) * kGroup + 32 + lane]);
}

// Largest of a warp's values, NaN left out.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Over a warp; every lane gets them.
__device__ __forceinline__ Sums warp_joined(const Pass& p, float c) {
  const float top = warp_max(p.top);
  Sums r = moved(Sums{p.ref, p.s.x + p.s.y, p.a.x + p.a.y}, top, c);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    r.s += __shfl_xor_sync(~0u, r.s, o);
    r.a += __shfl_xor_sync(~0u, r.a, o);
  }
  return r;
}
// Of n <= 16 parts, whose references are their largest values and of which lane k < n has the k-th, by a warp; every lane gets them.
__device__ __forceinline__ Sums parts_joined(Sums p, int n, float c) {
  const int lane = threadIdx.x & 31;
  const float top = warp_max(lane < n ? p.ref : -INFINITY);
  if (lane >= n) p.s = p.a = 0.0f;
  p = moved(p, top, c);
#pragma unroll
  for (int o = 8; o; o >>= 1) {
    p.s += __shfl_xor_sync(~0u, p.s, o);
    p.a += __shfl_xor_sync(~0u, p.a, o);
  }
  return Sums{top, __shfl_sync(~0u, p.s, 0), __shfl_sync(~0u, p.a, 0)};
}

// Runs of groups: CTA `rank` of 1 << ctas_shift has groups run_begin(rank) .. run_begin(rank + 1) - 1.
__device__ __forceinline__ int run_begin(int groups, int ctas_shift, int rank) { return (int)((unsigned)groups * (unsigned)rank >> ctas_shift); }

// A cluster's CTAs write what they have into the first one's shared memory: once when all have started, and the first goes on when all
// have written; the others need not wait for that.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
template <typename T>
__device__ __forceinline__ T* in_first(T* p) { return cooperative_groups::this_cluster().map_shared_rank(p, 0); }

// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11).
__device__ __forceinline__ uint4 philox(uint4 x, uint64_t seed) {
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    // products by halves: 86 cycles a warp and call on a scheduler that is full, with 64-bit products 112
    const uint32_t a = 0xD2511F53u * x.x, b = 0xCD9E8D57u * x.z;
    x = make_uint4(__umulhi(0xCD9E8D57u, x.z) ^ x.y ^ k0, b, __umulhi(0xD2511F53u, x.x) ^ x.w ^ k1, a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return x;
}

// ---------------------------------------------------------------- host

inline bool is_dtype(int dtype) { return dtype == WHEAD_BF16 || dtype == WHEAD_F16 || dtype == WHEAD_F32; }
inline int dtype_size(int dtype) { return dtype == WHEAD_F32 ? 4 : 2; }

// log2(e) / T in fp32 has to be a normal number.
inline bool good_temperature(double t) {
  const double c = 1.4426950408889634 / t;
  return t > 0 && c > 1.2e-38 && c < 3.4e38;
}

// Whether rows go by CTAs that hold their part, and how many CTAs a row has (a power of two), with most groups of a CTA.
struct Division {
  bool held;
  int shift, groups;
};
inline Division divide(int64_t rows, int64_t bytes, int sms) {
  // groups of a row, with one more for its start anywhere, over 1 << shift CTAs
  auto groups = [&](int shift) { return (int)(((bytes / (kGroup * 16) + 2) >> shift) + 1); };
  auto room = [&](int shift, int ctas) { return (1 << shift) <= kMaxCluster && (rows << shift) <= (int64_t)sms * ctas; };
  // held: as many CTAs as the row needs, then more while the device has room for them, down to 8 KB each (a row of 16 KB by one CTA 4.4 us, by
  // two 5.0, 40 such rows 4.6 and 5.4; rows of 64 KB by 8 KB a CTA 5.2, by 16 KB 5.6, by 32 KB 6.1)
  int s = 0;
  while ((1 << s) < kMaxCluster && groups(s) > kHeldGroups) ++s;
  if (groups(s) <= kHeldGroups && room(s, Form<true>::kCtas)) {
    while (room(s + 1, Form<true>::kCtas) && bytes >> (s + 1) >= 8192) ++s;
    return Division{true, s, groups(s)};
  }
  // streamed: as many as there is room for, down to 32 KB each (320 rows of 140 KB by two CTAs 17.4 us, by one 23.0; 120 of 300 KB by four
  // 17.6, by two 20.9; 320 rows of 64 KB would be faster by two of 32,000 bytes, 12.2 us, than by one, 13.8)
  s = 0;
  while (room(s + 1, Form<false>::kCtas) && bytes >> (s + 1) >= 32768) ++s;
  return Division{false, s, groups(s)};
}

constexpr int kMaxDynamic = 98 * 1024;  // shared memory that a launch may ask for

// A launch of `clusters` clusters of `ctas` CTAs, placed while the kernel before it in the stream still runs (it waits for its end).
template <typename... P, typename... A>
int launch_clusters(void (*kernel)(P...), int64_t clusters, int ctas, int threads, size_t smem, cudaStream_t stream, std::atomic<bool> (&granted)[kMaxDevices],
                    int device, A... args) {
  if (!granted[device].load(std::memory_order_relaxed)) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxDynamic) != cudaSuccess) {
      (void)cudaGetLastError();
      return WHEAD_ERR_CUDA;
    }
    granted[device].store(true, std::memory_order_relaxed);
  }
  cudaLaunchAttribute at[2]{};
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = (unsigned)ctas;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((unsigned)(clusters * ctas));
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = at;
  config.numAttrs = 2;
  if (cudaLaunchKernelEx(&config, kernel, P(args)...) != cudaSuccess) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  return WHEAD_OK;
}

}  // namespace whead_verify_impl

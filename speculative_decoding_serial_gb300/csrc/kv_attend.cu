// kv_attend.cu — attention over the 4-bit paged cache.
//
// For a row q and the visible keys k_j and values v_j of its KV head: o = sum_j p_j v_j / l, p_j = 2^(s_j - m),
// s_j = scale log2(e) q.k_j, l = sum_j p_j, lse = ln 2 (m + log2 l). m is any reference near the largest s; here it is a running
// one that is raised only when a score passes it by 2^kSlack, so that most tiles rescale nothing.
//
// Arithmetic. A held value without its head's fp32 factor is e2m1 x e4m3: 6 significant bits, at most 2688 and a multiple of
// 2^-10, so f16 holds it exactly, and the factor goes into the scores' scale (keys) and the output (values). A query
// row is scaled by a power of two to a largest value in [2^13, 2^14): bf16 and f16 rows then are f16 without rounding,
// but for parts below 2^-38 of the row's largest. Products are exact and their sums are fp32. p is rounded to f16 (2^-12
// relative, which is below the output's own rounding for bf16 and equal to it for f16); l sums what is not rounded.
#include "kv_schedule.cuh"

#include <algorithm>
#include <climits>
#include <cmath>

namespace whead_kv_impl {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = kWarps * 16;  // keys of a unit: 16 a warp
constexpr float kBias = 7.0f;       // m stands this far below the largest score at its setting: small p stay normal in f16
constexpr float kSlack = 15.0f;     // and is set anew when a score passes it by more: p <= 2^15
constexpr float kNoKey = -1e30f;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

template <int D, int NT>
struct Smem {
  uint2 q[NT][D / 16][32];        // query rows as operands: [8-row tile][16 channels][lane]
  float c[NT * 8];                // a row's factor from sums of products to scores in log2 units
  float o[NT * 8][D + 8];         // outputs of the CTA's warps, added up
  float m[kWarps][NT * 8];
  float l[kWarps][NT * 8];
  float row_m[NT * 8], row_l[NT * 8];
  SchedShared sched;
  int last;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) attend_rows(Cache c, AttendArgs a) {
  constexpr int NB = D / 16, ROWS = NT * 8;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D, NT>& s = *reinterpret_cast<Smem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const Start start = get_start<kThreads, kUnit>(c, a, ROWS, s.sched);
  if ((int)blockIdx.x >= start.ctas) return;
  long long cur = range_begin(start, blockIdx.x);
  const long long begin = cur, end = range_begin(start, blockIdx.x + 1);
  int item = start.item;
  long long item_at = start.at;
  while (cur < end) {
    const Tile tile = make_tile<kUnit>(c, a, item, ROWS);
    if (tile.units == 0) {
      ++item;
      continue;
    }
    const int h = (int)((cur - item_at) / tile.units);
    const long long head_at = item_at + (long long)h * tile.units;
    const int u0 = (int)(cur - head_at);
    const int u1 = (int)min((long long)tile.units, u0 + (end - cur));
    __syncthreads();
    // query rows
    for (int nt = warp; nt < NT; nt += kWarps) {
      const int row = tile.row0 + nt * 8 + g;
      const bool live = nt * 8 + g < tile.rows;
      const int64_t at = live ? (int64_t)(tile.first + row / a.group) * a.q_token_stride + (int64_t)(h * a.group + row % a.group) * a.q_head_stride : 0;
      float big = 0.0f;
      for (int b = 0; b < NB; ++b) {
        float x[4] = {};
        if (live) load_elems<4>(a.q, at + b * 16 + t * 4, a.dtype, a.wide_q, x);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
      }
      big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
      big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
      // 2^e <= big < 2^(e + 1), in the range whose powers of two are normal both ways
      const int e = min(max((int)((__float_as_uint(big) >> 23) & 255) - 127, -100), 100);
      const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23), down = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
      for (int b = 0; b < NB; ++b) {
        float x[4] = {};
        if (live) load_elems<4>(a.q, at + b * 16 + t * 4, a.dtype, a.wide_q, x);
        const __half2 lo = __floats2half2_rn(x[0] * up, x[1] * up), hi = __floats2half2_rn(x[2] * up, x[3] * up);
        s.q[nt][b][lane] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
      if (t == 0) s.c[nt * 8 + g] = down * (a.scale * c.k_scale[h] * kLog2e);
    }
    __syncthreads();
    float o[NT][NB][4];
    float m[NT][2], l[NT][2], f[NT][2];
    RowView view[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nt][e] = kNoKey;
        l[nt][e] = 0.0f;
        f[nt][e] = s.c[nt * 8 + 2 * t + e];
        view[nt][e] = row_view(a, tile, tile.row0 + nt * 8 + 2 * t + e);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][b][k] = 0.0f;
    }
    // keys that every row sees need no looking at masks
    const int t0 = tile.row0 / a.group, t1 = (tile.row0 + tile.rows - 1) / a.group, past = tile.len - tile.tokens;
    const int free_hi = a.tree ? min(past, a.causal ? past + t0 + 1 : tile.len) : a.causal ? min(past + t0 + 1, tile.len) : tile.len;
    const int free_lo = a.window ? max(past + t1 - a.window + 1, 0) : 0;
    const int32_t* table = c.tables + (int64_t)tile.slot * c.max_pages;
    for (int u = u0; u < u1; ++u) {
      const int key0 = (tile.unit0 + u) * kUnit + warp * 16;
      if (key0 >= tile.len) break;
      const uint8_t* gp = group_ptr<D>(c, table[key0 >> c.page_shift], h, key0);
      uint32_t kw[NB], ks[NB / 2], vw[NB], vs[NB];
#pragma unroll
      for (int i = 0; i < NB / 4; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(gp + i * 512) + lane);
        kw[4 * i] = x.x; kw[4 * i + 1] = x.y; kw[4 * i + 2] = x.z; kw[4 * i + 3] = x.w;
        const uint4 y = __ldg(reinterpret_cast<const uint4*>(gp + 9 * D + i * 512) + lane);
        vw[4 * i] = y.x; vw[4 * i + 1] = y.y; vw[4 * i + 2] = y.z; vw[4 * i + 3] = y.w;
        const uint2 z = __ldg(reinterpret_cast<const uint2*>(gp + 8 * D + g * 2 * NB) + i);
        ks[2 * i] = z.x; ks[2 * i + 1] = z.y;
        const uint4 w = __ldg(reinterpret_cast<const uint4*>(gp + 17 * D + t * 4 * NB) + i);
        vs[4 * i] = w.x; vs[4 * i + 1] = w.y; vs[4 * i + 2] = w.z; vs[4 * i + 3] = w.w;
      }
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < 4; ++k) sc[nt][k] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t x[4], s0, s1;
        e2m1x8_to_half2(kw[b], x);
        e4m3x4_to_half2(ks[b / 2], s0, s1);
        const uint32_t sb = b & 1 ? s1 : s0, sg = low2(sb), sh = high2(sb);
        x[0] = hmul2(x[0], sg);
        x[1] = hmul2(x[1], sh);
        x[2] = hmul2(x[2], sg);
        x[3] = hmul2(x[3], sh);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q = s.q[nt][b][lane];
          mma16816(sc[nt], x, q.x, q.y);
        }
      }
      const bool masked = key0 < free_lo || key0 + 16 > free_hi;
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[nt][k] *= f[nt][k & 1];
          if (masked && !sees(view[nt][k & 1], key0 + g + (k >> 1) * 8)) sc[nt][k] = -INFINITY;
          raise |= !(sc[nt][k] <= m[nt][k & 1] + kSlack);
        }
      }
      if (__any_sync(~0u, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float r[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = fmaxf(sc[nt][e], sc[nt][e + 2]);
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            const float now = x > m[nt][e] + kSlack ? x - kBias : m[nt][e];
            r[e] = ex2(m[nt][e] - now);
            m[nt][e] = now;
            l[nt][e] *= r[e];
          }
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nt][b][k] *= r[k & 1];
        }
      }
      uint32_t p[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          sc[nt][k] = ex2(sc[nt][k] - m[nt][k & 1]);
          l[nt][k & 1] += sc[nt][k];
        }
        const __half2 p0 = __floats2half2_rn(sc[nt][0], sc[nt][1]), p1 = __floats2half2_rn(sc[nt][2], sc[nt][3]);
        p[nt][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p0));
        p[nt][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p1));
      }
      // what lies past the length may be anything: its scales become zero, so that 0 x NaN does not arise
      uint32_t live = ~0u;
      if (key0 + 16 > tile.len) {
        live = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (key0 + 2 * t + (k & 1) + (k >> 1) * 8 < tile.len) live |= 0xFFu << (8 * k);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        uint32_t x[4], s0, s1;
        e2m1x8_to_half2(vw[b], x);
        e4m3x4_to_half2(vs[b] & live, s0, s1);
        x[0] = hmul2(x[0], s0);
        x[1] = hmul2(x[1], s0);
        x[2] = hmul2(x[2], s1);
        x[3] = hmul2(x[3], s1);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][b], x, p[nt][0], p[nt][1]);
      }
    }
    // the CTA's warps joined: one after the other they add their outputs, scaled to the common m
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], 16);
        if (g == 0) {
          s.m[warp][nt * 8 + 2 * t + e] = m[nt][e];
          s.l[warp][nt * 8 + 2 * t + e] = l[nt][e];
        }
      }
    __syncthreads();
    if (tid < ROWS) {
      float mm = s.m[0][tid];
      for (int w = 1; w < kWarps; ++w) mm = fmaxf(mm, s.m[w][tid]);
      float ll = 0.0f;
      for (int w = 0; w < kWarps; ++w) ll += s.l[w][tid] * ex2(s.m[w][tid] - mm);
      s.row_m[tid] = mm;
      s.row_l[tid] = ll;
    }
    __syncthreads();
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = nt * 8 + 2 * t + e;
            const float r = ex2(m[nt][e] - s.row_m[row]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              float2* to = reinterpret_cast<float2*>(&s.o[row][b * 16 + 2 * g]);
              float2 v = make_float2(o[nt][b][e] * r, o[nt][b][e + 2] * r);
              if (w) {
                const float2 x = *to;
                v.x += x.x;
                v.y += x.y;
              }
              *to = v;
            }
          }
      }
      __syncthreads();
    }
    const long long head_end = head_at + tile.units;
    const bool whole = u0 == 0 && u1 == tile.units;
    const int first_cta = whole ? 0 : range_owner(start, head_at), last_cta = whole ? 0 : range_owner(start, head_end - 1);
    constexpr int kPart = ROWS * (D + 2);
    if (!whole) {
      float* part = c.partial + (int64_t)(2 * blockIdx.x + (cur == begin ? 0 : 1)) * kPart;
      for (int x = tid; x < tile.rows * (D / 4); x += kThreads) {
        const int row = x / (D / 4), col = x % (D / 4) * 4;
        __stcg(reinterpret_cast<float4*>(part + 2 * ROWS + row * D + col), *reinterpret_cast<const float4*>(&s.o[row][col]));
      }
      if (tid < tile.rows) {
        __stcg(part + tid, s.row_m[tid]);
        __stcg(part + ROWS + tid, s.row_l[tid]);
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned parts = last_cta - first_cta + 1;
        const unsigned done = atomicAdd(&c.counters[first_cta], 1u);
        s.last = done + 1 == parts;
        if (s.last) c.counters[first_cta] = 0;
      }
      __syncthreads();
      __threadfence();
    }
    if (whole || s.last) {
      const float gv = c.v_scale[h];
      if (!whole) {
        if (tid < tile.rows) {
          float mm = kNoKey;
          for (int k = first_cta; k <= last_cta; ++k) {
            const bool in = k > first_cta || range_begin(start, k) == head_at;
            mm = fmaxf(mm, __ldcg(c.partial + (int64_t)(2 * k + (in ? 0 : 1)) * kPart + tid));
          }
          float ll = 0.0f;
          for (int k = first_cta; k <= last_cta; ++k) {
            const bool in = k > first_cta || range_begin(start, k) == head_at;
            const float* part = c.partial + (int64_t)(2 * k + (in ? 0 : 1)) * kPart;
            ll += __ldcg(part + ROWS + tid) * ex2(__ldcg(part + tid) - mm);
          }
          s.row_m[tid] = mm;
          s.row_l[tid] = ll;
        }
        __syncthreads();
      }
      for (int x = tid; x < tile.rows * (D / 4); x += kThreads) {
        const int row = x / (D / 4), col = x % (D / 4) * 4;
        float4 v;
        if (whole) {
          v = *reinterpret_cast<const float4*>(&s.o[row][col]);
        } else {
          v = make_float4(0.f, 0.f, 0.f, 0.f);
          const float mm = s.row_m[row];
          for (int k = first_cta; k <= last_cta; ++k) {
            const bool in = k > first_cta || range_begin(start, k) == head_at;
            const float* part = c.partial + (int64_t)(2 * k + (in ? 0 : 1)) * kPart;
            const float r = ex2(__ldcg(part + row) - mm);
            const float4 y = __ldcg(reinterpret_cast<const float4*>(part + 2 * ROWS + row * D + col));
            v.x += y.x * r; v.y += y.y * r; v.z += y.z * r; v.w += y.w * r;
          }
        }
        const float ll = s.row_l[row];
        const float r = ll != 0.0f ? gv / ll : 0.0f;
        const int grow = tile.row0 + row;
        const int64_t at = ((int64_t)(tile.first + grow / a.group) * a.heads + h * a.group + grow % a.group);
        if (ll == 0.0f) v = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + col) =
            make_uint2(pack16(v.x * r, v.y * r, a.dtype), pack16(v.z * r, v.w * r, a.dtype));
        if (a.lse && col == 0) a.lse[at] = ll == 0.0f ? -INFINITY : (s.row_m[row] + log2f(ll)) * kLn2;
      }
    }
    cur = head_at + u1;
    if (u1 == tile.units && h == c.kv_heads - 1) {
      item_at = cur;
      ++item;
    }
  }
}

template <int D, int NT>
int launch_rows(const HostCache& h, AttendArgs a, int max_q) {
  constexpr int ROWS = NT * 8;
  constexpr int smem = sizeof(Smem<D, NT>);
  static int per_sm = 0;
  if (per_sm == 0) {
    int n = 0;
    if (cudaFuncSetAttribute(attend_rows<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attend_rows<D, NT>, kThreads, smem) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      return WHEAD_ERR_CUDA;
    }
    per_sm = n;
  }
  const int64_t tiles = ((int64_t)max_q * a.group + ROWS - 1) / ROWS;
  if (tiles * a.n >= INT_MAX) return WHEAD_ERR_UNSUPPORTED;
  a.row_tiles = (int)tiles;
  int64_t ctas = std::min<int64_t>((int64_t)h.sms * std::min(per_sm, 4), kMaxCtas);
  ctas = std::min(ctas, h.c.partial_floats / (2 * ROWS * (D + 2)));
  a.planned = tiles * a.n > 4 * kThreads;
  if (a.planned) attend_plan<kUnit><<<1, 1024, 0, h.stream>>>(h.c, a, ROWS, (int)ctas);
  attend_rows<D, NT><<<(unsigned)ctas, kThreads, smem, h.stream>>>(h.c, a);
  return launch_status();
}

}  // namespace

}  // namespace whead_kv_impl

using namespace whead_kv_impl;

extern "C" int whead_kv_attend(const whead_kv* kv, const whead_kv_attend_args* x) {
  if (!kv || !x) return WHEAD_ERR_INVALID_ARG;
  if (x->n < 0 || x->n > kv->max_seqs || x->total < 0 || x->total >= INT_MAX || x->max_q < 0 || x->heads < 1) return WHEAD_ERR_INVALID_ARG;
  if (kv->kv_heads < 1 || x->heads % kv->kv_heads) return WHEAD_ERR_INVALID_ARG;
  if (x->dtype != WHEAD_KV_BF16 && x->dtype != WHEAD_KV_F16) return WHEAD_ERR_UNSUPPORTED;
  if (x->window < 0 || ((x->window || x->tree) && !x->causal) || !std::isfinite(x->scale)) return WHEAD_ERR_INVALID_ARG;
  if (x->tree && (x->tree_words < 1 || (int64_t)x->tree_words * 64 < x->max_q || !aligned(x->tree, 8))) return WHEAD_ERR_INVALID_ARG;
  HostCache h;
  if (x->n == 0 || x->total == 0) return x->total > 0 ? WHEAD_ERR_INVALID_ARG : host_cache(kv, &h);
  if (!x->q || !x->out || !aligned(x->q, 2) || !aligned(x->out, 16) || !aligned(x->lse, 4) || x->max_q < 1) return WHEAD_ERR_INVALID_ARG;
  if (!x->indptr && (x->total % x->n || x->total / x->n > x->max_q)) return WHEAD_ERR_INVALID_ARG;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  const int group = x->heads / kv->kv_heads;
  const int64_t rows = (int64_t)x->max_q * group;
  if (rows >= INT_MAX / 2) return WHEAD_ERR_UNSUPPORTED;
  AttendArgs a{x->q, x->out, x->lse, x->indptr, x->slots, reinterpret_cast<const unsigned long long*>(x->tree), x->total, x->q_token_stride,
               x->q_head_stride, x->n, x->heads, group, 1, x->dtype, x->causal, x->window, x->tree_words, x->scale, false, 0};
  a.wide_q = aligned(x->q, 8) && x->q_token_stride % 4 == 0 && x->q_head_stride % 4 == 0;
  const int nt = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  switch (kv->head_dim) {
    case 64: return nt == 1 ? launch_rows<64, 1>(h, a, x->max_q) : nt == 2 ? launch_rows<64, 2>(h, a, x->max_q) : launch_rows<64, 4>(h, a, x->max_q);
    case 128: return nt == 1 ? launch_rows<128, 1>(h, a, x->max_q) : nt == 2 ? launch_rows<128, 2>(h, a, x->max_q) : launch_rows<128, 4>(h, a, x->max_q);
    default: return nt == 1 ? launch_rows<256, 1>(h, a, x->max_q) : launch_rows<256, 2>(h, a, x->max_q);
  }
}

// kv_attend.cu — attention over the 4-bit paged cache.
//
// For a row q and the visible keys k_j and values v_j of its KV head: o = sum_j p_j v_j / l, p_j = 2^(s_j - m),
// s_j = scale log2(e) q.k_j, l = sum_j p_j, lse = ln 2 (m + log2 l). m is any reference near the largest s; here it is a running
// one that is raised only when a score passes it by kSlack, so that most tiles rescale nothing.
//
// This file: few rows of a KV head, on mma.sync. S^T = K Q^T and O^T = V^T P^T have the keys and the channels on the 16-row side and
// the query rows on the side of 8, so that one token's 4 rows waste half a tile and not three quarters; the groups of the cache lie in
// the operands' lane order. Bound by the cache's bytes where there are enough: 32 sequences on 2,000 to 32,768 keys, one token, 654 MB in
// 120 us, 5.5 TB/s, 82 % of the measured copy rate; what is missing is the spread of the CTAs' ends (93 to 119 us: the memory's
// share of an SM differs) and the issue slots, of which 61 % are in use, most of them for the unpacking. 16 on 300 to 8,200 keys (78 MB,
// 24 us, 3.3 TB/s) and below: a CTA's start, 4 us, and the joining of the parts. 256 channels, 4 heads a KV head: 16 on 300 to 8,200
// keys, one token, 83 MB in 28 us, 3.0 TB/s; with many rows every 16 unpack the keys again (2 x 512 tokens on 2,000 to 4,000 keys, 59 GFLOP
// in 283 us, 0.2 PFLOP/s; 8 x 17 on 900 to 6,100, 37 MB in 55 us).
//
// Arithmetic. A held value without its head's fp32 factor is e2m1 x e4m3: 6 significant bits, at most 2688 and a multiple of
// 2^-10, so f16 holds it exactly, and the factor goes into the scores' scale (keys) and the output (values). A query
// row is scaled by a power of two to a largest value in [2^13, 2^14): bf16 and f16 rows then are f16 without rounding,
// but for parts below 2^-38 of the row's largest. Products are exact and their sums are fp32. p is rounded to f16, the operand type of the
// product with the values (2^-11 relative at most: an eighth of the output's own rounding for bf16, as much for f16, whose outputs
// are off by 0.00028 of their norm for 0.00021 with p in fp32); l sums what is not rounded.
#include "kv_schedule.cuh"

#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>

namespace whead_kv_impl {

namespace {

constexpr float kBias = 7.0f;                // m stands this far below the largest score at its setting: small p stay normal in f16
constexpr float kSlack = 15.0f;              // and is set anew when a score passes it by more: p <= 2^15

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
  return r;
}

// What one CTA needs for D channels and 8 NT rows. Every warp has a ring of its own, with one or two groups (16 keys of one
// KV head each) a stage; red holds two warps' outputs while they are joined (rows 4 floats apart beyond D: a warp's stores
// then hit every bank once).
template <int D, int NT>
struct Shape {
  static constexpr int kRows = NT * 8;
  static constexpr int kHead = 512;
  static constexpr int kLoad = NT * D;  // a lane's output registers are a quarter of this
  static constexpr int kWarps = 4;
  static constexpr int kCtas = kLoad <= 128 ? 4 : kLoad == 256 ? 3 : 2;  // of an SM, by registers
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kGroups = D == 256 ? 1 : 2;  // of a stage
  static constexpr int kKeys = kGroups * 16;
  static constexpr int kUnit = kWarps * kKeys;
  static constexpr bool kQInRegs = kLoad <= 128;
  static constexpr int kGroup = 18 * D, kStage = kGroups * kGroup;
  static constexpr int kRed = 2 * kRows * (D + 4) * 4;
  static constexpr int kQ = kQInRegs ? 0 : NT * (D / 16) * 32 * 8;
  static constexpr int kFixed = (kHead + 2 * kWarps * kRows * 4 + kRows * 4 + kQ + kRed + 127) / 128 * 128;
  static constexpr int kRoom = (228 * 1024 / kCtas - 1024 - kFixed) / (kWarps * kStage);
  static constexpr int kStages = kRoom > 4 ? 4 : kRoom;
  static constexpr bool kTogether = kLoad <= 128 && kGroups == 2;  // a stage's groups worked on at once, for independent chains of products
  static constexpr int kBytes = kFixed + kStages * kWarps * kStage;
  static_assert(kStages >= 2, "the rings need two stages");
};

struct Head {  // the fixed head of shared memory
  SchedShared sched;
  unsigned long long full[4][4];
  int last;
};
static_assert(sizeof(Head) <= 512, "");

// A warp's way through a segment's groups and its ring. Lane 0 alone fetches; it has the next pages' numbers one copy ahead.
struct Fetch {
  const uint8_t* base;      // the pool at this KV head
  const int32_t* table;
  int next, end;            // units to fetch
  int key;                  // first key of the next stage
  int page, page1;          // its groups' pages (page1: where a page is one group)
  uint32_t slot;            // the next stage
};

__device__ __forceinline__ int page_of(const Cache& c, const int32_t* table, int key, int len) {
  if (key >= len) return 0;
  const int page = __ldg(table + (key >> c.page_shift));
  if ((unsigned)page < (unsigned)c.num_pages) return page;
  set_status(c, WHEAD_ERR_INTERNAL);
  return 0;
}

template <int D, int NT>
__device__ __forceinline__ void fetch_one(const Cache& c, int len, Fetch& f, uint32_t ring, uint32_t bars) {
  using S = Shape<D, NT>;
  if (f.next >= f.end) return;
  if ((threadIdx.x & 31) == 0) {
    const uint32_t bar = bars + f.slot * 8, dst = ring + f.slot * S::kStage;
    const int64_t page_bytes = (int64_t)c.kv_heads * (c.page_size >> 4) * S::kGroup;
    const uint8_t* src = f.base + f.page * page_bytes + ((f.key & (c.page_size - 1)) >> 4) * S::kGroup;
    const uint32_t bytes = S::kGroups == 2 && f.key + 16 < len ? 2 * S::kGroup : S::kGroup;  // a second group that holds no key stays out
    mbar_expect(bar, bytes);
    if (c.page_size > 16) {
      bulk_load(dst, src, bytes, bar);
    } else {
      bulk_load(dst, src, S::kGroup, bar);
      if (bytes > S::kGroup) bulk_load(dst + S::kGroup, f.base + f.page1 * page_bytes, S::kGroup, bar);
    }
    f.key = f.next + 1 < f.end ? f.key + S::kUnit : len;
    f.page = page_of(c, f.table, f.key, len);
    if (S::kGroups == 2 && c.page_size == 16) f.page1 = page_of(c, f.table, min(f.key, len - 16) + 16, len);
  }
  f.slot = f.slot + 1 == S::kStages ? 0 : f.slot + 1;
  ++f.next;
}

template <int D, int NT>
__global__ void __launch_bounds__((Shape<D, NT>::kThreads), (Shape<D, NT>::kCtas)) attend_rows(const __grid_constant__ Cache c, const __grid_constant__ AttendArgs a) {
  after_previous();
  using S = Shape<D, NT>;
  constexpr int NB = D / 16, ROWS = S::kRows, kWarps = S::kWarps, kConsumers = S::kThreads, kUnit = S::kUnit;
  extern __shared__ __align__(128) uint8_t smem[];
  Head& s = *reinterpret_cast<Head*>(smem);
  float* s_m = reinterpret_cast<float*>(smem + S::kHead);       // [warp][row]
  float* s_l = s_m + kWarps * ROWS;
  float* s_c = s_l + kWarps * ROWS;                          // a row's factor from sums of products to scores in log2 units
  uint2* s_q = reinterpret_cast<uint2*>(s_c + ROWS);         // query rows as operands: [8-row tile][16 channels][lane]
  float* red = reinterpret_cast<float*>(smem + S::kHead + 2 * kWarps * ROWS * 4 + ROWS * 4 + S::kQ);  // [2][row][D + 4]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint8_t* my_ring = smem + S::kFixed + warp * S::kStages * S::kStage;
  const uint32_t ring = smem_u32(my_ring), bars = smem_u32(&s.full[warp][0]);
  if (lane == 0) {
    for (int i = 0; i < S::kStages; ++i) mbar_init(bars + i * 8, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const Start start = get_start<S::kThreads, kUnit>(c, a, ROWS, s.sched);
  if (a.apart && tid == 0) put_record(c, 0, 0, 0, 0);
  if ((int)blockIdx.x >= start.ctas) return;
  long long cur = range_begin(start, blockIdx.x);
  const long long end = range_begin(start, blockIdx.x + 1);
  int item = start.item;
  long long item_at = start.at;
  uint32_t stage = 0, phase = 0;
  bool dead = false;
  Segment sg;
  Fetch fetch;
  fetch.slot = 0;

  // the segment that begins at unit `at`, and the first copies of this warp's groups; `fresh`: not the next head of the same tile
  long long next = cur;
  auto enter = [&](long long at, bool fresh) {
    if (fresh) {
      if (item == s.sched.item && s.sched.has_tile) {
        sg.tile = s.sched.tile;
      } else {
        while (true) {
          sg.tile = make_tile<kUnit>(c, a, item, ROWS);
          if (sg.tile.units > 0) break;
          ++item;
        }
      }
      const int past_item = (int)(at - item_at), each = sg.tile.units + kLead;
      sg.h = past_item / each;
      sg.head_at = item_at + (long long)sg.h * each;
    } else {
      ++sg.h;
      sg.head_at = at;
    }
    next = cut_segment(sg, at, end);
    fetch.base = c.pool + (int64_t)sg.h * (c.page_size >> 4) * S::kGroup;
    fetch.table = c.tables + (int64_t)sg.tile.slot * c.max_pages;
    fetch.next = sg.u0;
    // units in which this warp has any key
    fetch.end = min(sg.u1, max((sg.tile.len - warp * S::kKeys + kUnit - 1) / kUnit - sg.tile.unit0, sg.u0));
    if (dead) fetch.end = sg.u0;
    fetch.key = (sg.tile.unit0 + sg.u0) * kUnit + warp * S::kKeys;
    fetch.page = fetch.page1 = 0;
    if (fetch.next < fetch.end) {
      fetch.page = page_of(c, fetch.table, fetch.key, sg.tile.len);
      if (S::kGroups == 2 && c.page_size == 16) fetch.page1 = page_of(c, fetch.table, fetch.key + 16, sg.tile.len);
    }
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) fetch_one<D, NT>(c, sg.tile.len, fetch, ring, bars);
  };
  if (cur < end) enter(cur, true);

  while (cur < end && sg.u1 > sg.u0) {  // a range may end inside a lead
    const Segment now = sg;
    const Tile& tile = now.tile;
    const int h = now.h, u0 = now.u0, u1 = now.u1;
    int live_end = fetch.end;
    // query rows: from a power of two to f16, as operands
    const float k_scale = c.k_scale[h];
    uint2 q[S::kQInRegs ? NT : 1][S::kQInRegs ? NB : 1];
    float f[NT][2];
    if (!S::kQInRegs) named_sync<kConsumers>(1);
#pragma unroll
    for (int i = 0; i < (S::kQInRegs ? NT : (NT + kWarps - 1) / kWarps); ++i) {
      const int nt = S::kQInRegs ? i : i * kWarps + warp;
      if (nt < NT) {
        const int row = tile.row0 + nt * 8 + g;
        const bool live = nt * 8 + g < tile.rows;
        const int tok = row_token(a, row);
        const int64_t at = live ? (int64_t)(tile.first + tok) * a.q_token_stride + (int64_t)(h * a.group + row - tok * a.group) * a.q_head_stride : 0;
        // all of the row's loads before any of its values is looked at
        uint2 raw[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) raw[b] = live ? load_four(a.q, at + b * 16 + t * 4, a.wide_q) : make_uint2(0u, 0u);
        // the largest magnitude, by its bits: they are ordered like the values
        uint32_t top = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b) top = __vmaxu2(top, __vmaxu2(raw[b].x & 0x7FFF7FFFu, raw[b].y & 0x7FFF7FFFu));
        top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(~0u, top, 2));
        top = max(top & 0xFFFFu, top >> 16);
        // 2^e <= largest < 2^(e + 1) (an f16 below 2^-14 counts as one just there). Both powers of two are normal for every bf16 exponent
        // from -100 up; a row below counts as one there, where bf16's smallest step is still one that f16 holds.
        const int e = max(a.dtype == WHEAD_KV_BF16 ? (int)(top >> 7) - 127 : max((int)(top >> 10), 1) - 15, -100);
        const float up = __uint_as_float((uint32_t)(127 + 13 - e) << 23), down = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float2 lo = unpack16(raw[b].x, a.dtype), hi = unpack16(raw[b].y, a.dtype);
          const uint2 w = make_uint2(pack16(lo.x * up, lo.y * up, WHEAD_KV_F16), pack16(hi.x * up, hi.y * up, WHEAD_KV_F16));
          if constexpr (S::kQInRegs) q[i][b] = w;
          else s_q[(nt * NB + b) * 32 + lane] = w;
        }
        if constexpr (S::kQInRegs) {
          // the row's power of two first: it may be what the scale takes back
          f[i][0] = __shfl_sync(~0u, down, t * 8) * a.scale * k_scale * kLog2e;
          f[i][1] = __shfl_sync(~0u, down, t * 8 + 4) * a.scale * k_scale * kLog2e;
        } else if (t == 0) {
          s_c[nt * 8 + g] = down * a.scale * k_scale * kLog2e;
        }
      }
    }
    if constexpr (!S::kQInRegs) {
      named_sync<kConsumers>(1);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f[nt][0] = s_c[nt * 8 + 2 * t];
        f[nt][1] = s_c[nt * 8 + 2 * t + 1];
      }
    }
    float o[NT][NB][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = kNoKey;
      l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nt][b][k] = 0.0f;
    }
    // keys that every row sees need no looking at masks
    const int t0 = row_token(a, tile.row0), t1 = row_token(a, tile.row0 + tile.rows - 1), past = tile.len - tile.tokens;
    const int free_hi = a.tree ? min(past, past + t0 + 1) : a.causal ? min(past + t0 + 1, tile.len) : tile.len;
    const int free_lo = a.window ? window_begin(a, past + t1) : 0;
    // G neighbouring groups at a time, from key0 on
    auto work = [&](auto count, const uint8_t* gp, int key0) {
      constexpr int G = decltype(count)::value;
      float sc[G][NT][4];
#pragma unroll
      for (int i = 0; i < NB / 4; ++i) {
#pragma unroll
        for (int w = 0; w < G; ++w) {
          const uint4 kw = *reinterpret_cast<const uint4*>(gp + w * S::kGroup + i * 512 + lane * 16);
          const uint2 ks = *reinterpret_cast<const uint2*>(gp + w * S::kGroup + 8 * D + g * 2 * NB + i * 8);
          uint32_t sg4[4];
          e4m3x4_to_half2(ks.x, sg4[0], sg4[1]);
          e4m3x4_to_half2(ks.y, sg4[2], sg4[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x[4];
            e2m1x8_to_half2(j == 0 ? kw.x : j == 1 ? kw.y : j == 2 ? kw.z : kw.w, x);
            x[0] = hmul2_low(x[0], sg4[j]);
            x[1] = hmul2_high(x[1], sg4[j]);
            x[2] = hmul2_low(x[2], sg4[j]);
            x[3] = hmul2_high(x[3], sg4[j]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint2 y;
              if constexpr (S::kQInRegs) y = q[nt][i * 4 + j];
              else y = s_q[(nt * NB + i * 4 + j) * 32 + lane];
              if (i == 0 && j == 0) mma16816_first(sc[w][nt], x, y.x, y.y);
              else mma16816(sc[w][nt], x, y.x, y.y);
            }
          }
        }
      }
      // from sums of products to scores, rounded before the reference is taken off: the difference of a score and itself is then zero,
      // however large both are (in one multiply-add it would be the product's rounding, and p anything; 32 sequences on 2,000 to 32,768
      // keys took 119.4 us so, 119.9 now)
#pragma unroll
      for (int w = 0; w < G; ++w)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[w][nt][k] = __fmul_rn(sc[w][nt][k], f[nt][k & 1]);
#pragma unroll
      for (int w = 0; w < G; ++w) {
        if (key0 + w * 16 < free_lo || key0 + w * 16 + 16 > free_hi) {
          // what no row sees of the last group may be anything: its values' scales become zero, so that 0 x NaN does not arise
          if (key0 + w * 16 + 16 > tile.len) {
            uint8_t* vs = const_cast<uint8_t*>(gp + w * S::kGroup) + 17 * D;
            for (int k = lane; k < 16; k += 32)
              if (key0 + w * 16 + k >= tile.len)
                for (int b = 0; b < NB; ++b) vs[(k & 7) / 2 * 4 * NB + b * 4 + (k >> 3) * 2 + (k & 1)] = 0;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // before the stage's next copy
            __syncwarp();
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const RowView view = row_view(a, tile, tile.row0 + nt * 8 + 2 * t + e);
              if (!sees(view, key0 + w * 16 + g)) sc[w][nt][e] = -INFINITY;
              if (!sees(view, key0 + w * 16 + g + 8)) sc[w][nt][e + 2] = -INFINITY;
            }
        }
      }
      float d[G][NT][4], top = -INFINITY;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int w = 0; w < G; ++w)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            d[w][nt][k] = sc[w][nt][k] - m[nt][k & 1];
            top = fmaxf(top, d[w][nt][k]);
          }
      if (__any_sync(~0u, top > kSlack)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float r[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = -INFINITY;
#pragma unroll
            for (int w = 0; w < G; ++w) x = fmaxf(x, fmaxf(sc[w][nt][e], sc[w][nt][e + 2]));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
            x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            const float now = x > m[nt][e] + kSlack ? x - kBias : m[nt][e];
            r[e] = ex2(m[nt][e] - now);
            m[nt][e] = now;
            l[nt][e] *= r[e];
#pragma unroll
            for (int w = 0; w < G; ++w) {
              d[w][nt][e] = sc[w][nt][e] - now;
              d[w][nt][e + 2] = sc[w][nt][e + 2] - now;
            }
          }
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nt][b][k] *= r[k & 1];
        }
      }
      uint32_t p[G][NT][2];
#pragma unroll
      for (int w = 0; w < G; ++w)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            d[w][nt][k] = ex2(d[w][nt][k]);
            l[nt][k & 1] += d[w][nt][k];
          }
          const __half2 p0 = __floats2half2_rn(d[w][nt][0], d[w][nt][1]), p1 = __floats2half2_rn(d[w][nt][2], d[w][nt][3]);
          p[w][nt][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p0));
          p[w][nt][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p1));
        }
#pragma unroll
      for (int w = 0; w < G; ++w)
#pragma unroll
        for (int i = 0; i < NB / 4; ++i) {
          const uint4 vw = *reinterpret_cast<const uint4*>(gp + w * S::kGroup + 9 * D + i * 512 + lane * 16);
          const uint4 vs = *reinterpret_cast<const uint4*>(gp + w * S::kGroup + 17 * D + t * 4 * NB + i * 16);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t x[4], s0, s1;
            e2m1x8_to_half2(j == 0 ? vw.x : j == 1 ? vw.y : j == 2 ? vw.z : vw.w, x);
            e4m3x4_to_half2(j == 0 ? vs.x : j == 1 ? vs.y : j == 2 ? vs.z : vs.w, s0, s1);
            x[0] = hmul2(x[0], s0);
            x[1] = hmul2(x[1], s0);
            x[2] = hmul2(x[2], s1);
            x[3] = hmul2(x[3], s1);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][i * 4 + j], x, p[w][nt][0], p[w][nt][1]);
          }
        }
    };
#pragma unroll 1
    for (int u = u0; u < live_end; ++u) {
      const int key0 = (tile.unit0 + u) * kUnit + warp * S::kKeys;
      // a copy that does not come is reported; nothing more is fetched, and what is under way is still waited for
      if (!__all_sync(~0u, mbar_wait(bars + stage * 8, phase))) {
        set_status(c, WHEAD_ERR_TIMEOUT);
        dead = true;
        fetch.end = live_end = fetch.next;
      }
      const uint8_t* gp = my_ring + stage * S::kStage;
      if (S::kTogether && key0 + 16 < tile.len) {
        work(std::integral_constant<int, 2>{}, gp, key0);
      } else {
        work(std::integral_constant<int, 1>{}, gp, key0);
        if (!S::kTogether && S::kGroups == 2 && key0 + 16 < tile.len) work(std::integral_constant<int, 1>{}, gp + S::kGroup, key0 + 16);
      }
      __syncwarp();
      fetch_one<D, NT>(c, sg.tile.len, fetch, ring, bars);  // into the stage that has just been read
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    // the next segment's first copies come while this one is being joined
    const long long after = next;
    const bool item_done = u1 == tile.units && h == c.kv_heads - 1;
    if (item_done) {
      item_at = after;
      ++item;
    }
    if (after < end) enter(after, item_done);
    // ---- the warps' parts joined
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(~0u, l[nt][e], 16);
      }
    named_sync<kConsumers>(1);  // red and s_m of the segment before have been read
    const bool lower = warp < kWarps / 2;  // these add the others' outputs to their own
    auto red_at = [&](int row) { return red + ((warp & 1) * ROWS + row) * (D + 4) + 2 * g; };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * t + e;
        if (row < tile.rows) {
          if (g == 0) {
            s_m[warp * ROWS + row] = m[nt][e];
            s_l[warp * ROWS + row] = l[nt][e];
          }
          if (!lower) {
#pragma unroll
            for (int b = 0; b < NB; ++b) *reinterpret_cast<float2*>(red_at(row) + b * 16) = make_float2(o[nt][b][e], o[nt][b][e + 2]);
          }
        }
      }
    named_sync<kConsumers>(1);
    if (lower) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = nt * 8 + 2 * t + e;
          if (row < tile.rows) {
            const float other = s_m[(warp + 2) * ROWS + row];
            const float mm = fmaxf(fmaxf(m[nt][e], other), fmaxf(s_m[(warp ^ 1) * ROWS + row], s_m[((warp ^ 1) + 2) * ROWS + row]));
            const float r0 = ex2(m[nt][e] - mm), r1 = ex2(other - mm);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              float2* at = reinterpret_cast<float2*>(red_at(row) + b * 16);
              const float2 y = *at;
              *at = make_float2(o[nt][b][e] * r0 + y.x * r1, o[nt][b][e + 2] * r0 + y.y * r1);
            }
          }
        }
    }
    named_sync<kConsumers>(1);
    const bool whole = u0 == 0 && u1 == tile.units;
    constexpr int kPart = ROWS * (D + 2);
    float* part = c.partial + (int64_t)part_slot(start, now, blockIdx.x) * kPart;
    const float gv = c.v_scale[h];
    auto write_row = [&](int row, int col, float4 v, float mm, float ll) {
      const int grow = tile.row0 + row;
      const int tok = row_token(a, grow);
      const int64_t at = (int64_t)(tile.first + tok) * a.heads + h * a.group + grow - tok * a.group;
      const float r = ll != 0.0f ? gv / ll : 0.0f;
      if (ll == 0.0f) v = make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + col) =
          make_uint2(pack16(v.x * r, v.y * r, a.dtype), pack16(v.z * r, v.w * r, a.dtype));
      if (a.lse && col == 0) a.lse[at] = ll == 0.0f ? -INFINITY : (mm + log2f(ll)) * kLn2;
    };
    for (int x = tid; x < tile.rows * (D / 4); x += kConsumers) {
      const int row = x / (D / 4), col = x % (D / 4) * 4;
      float mm = kNoKey, ll = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * ROWS + row]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ll += s_l[w * ROWS + row] * ex2(s_m[w * ROWS + row] - mm);
      float4 v = *reinterpret_cast<const float4*>(red + row * (D + 4) + col);
      const float4 y = *reinterpret_cast<const float4*>(red + (ROWS + row) * (D + 4) + col);
      v.x += y.x; v.y += y.y; v.z += y.z; v.w += y.w;
      if (whole) {
        write_row(row, col, v, mm, ll);
      } else {
        __stcg(reinterpret_cast<float4*>(part + 2 * ROWS + row * D + col), v);
        if (col == 0) {
          __stcg(part + row, mm);
          __stcg(part + ROWS + row, ll);
        }
      }
    }
    if (!whole && a.apart) {
      if (tid == 0 && u0 == 0) put_record(c, item, h, last_owner(start, now) - (int)blockIdx.x + 1, part_slot(start, now, blockIdx.x));
    } else if (!whole) {
      // ---- an item's parts joined, by the last CTA to get here
      const int first_cta = first_owner(start, now), last_cta = last_owner(start, now);
      const int parts = last_cta - first_cta + 1;
      named_sync<kConsumers>(1);
      if (tid == 0) {  // its fence covers what the others wrote before the barrier
        unsigned done;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(done) : "l"(c.counters + first_cta) : "memory");
        s.last = done + 1 == (unsigned)parts;
        if (s.last) c.counters[first_cta] = 0;
      }
      named_sync<kConsumers>(1);
      if (s.last) {
        const int first_slot = part_slot(start, now, first_cta);
        auto part_at = [&](int k) { return c.partial + (int64_t)(k == 0 ? first_slot : 2 * (first_cta + k)) * kPart; };
#pragma unroll 1
        for (int x = tid; x < tile.rows * (D / 4); x += kConsumers) {
          const int row = x / (D / 4), col = x % (D / 4) * 4;
          float mm = kNoKey, ll = 0.0f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
          for (int k0 = 0; k0 < parts; k0 += 8) {  // eight parts' loads under way at once
            float pm[8], pl[8];
            float4 y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float* p = part_at(min(k0 + k, parts - 1));
              pm[k] = __ldcg(p + row);
              pl[k] = __ldcg(p + ROWS + row);
              y[k] = __ldcg(reinterpret_cast<const float4*>(p + 2 * ROWS + row * D + col));
            }
            float now = mm;
#pragma unroll
            for (int k = 0; k < 8; ++k) now = fmaxf(now, pm[k]);
            const float r0 = ex2(mm - now);
            mm = now;
            ll *= r0;
            v.x *= r0; v.y *= r0; v.z *= r0; v.w *= r0;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              if (k0 + k >= parts) break;
              const float r1 = ex2(pm[k] - mm);
              ll += pl[k] * r1;
              v.x += y[k].x * r1; v.y += y[k].y * r1; v.z += y[k].z * r1; v.w += y[k].w * r1;
            }
          }
          write_row(row, col, v, mm, ll);
        }
      }
    }
    cur = after;
  }
}

template <int D, int NT>
int launch_rows(const HostCache& h, AttendArgs a, int max_q) {
  using S = Shape<D, NT>;
  constexpr int kUnit = S::kUnit;
  static std::atomic<bool> granted[kMaxDevices];
  if (!grant_smem(attend_rows<D, NT>, S::kBytes, h, granted)) return WHEAD_ERR_CUDA;
  const int64_t tiles = ((int64_t)max_q * a.group + S::kRows - 1) / S::kRows;
  a.row_tiles = (int)tiles;
  int64_t ctas = std::min<int64_t>((int64_t)h.sms * S::kCtas, kMaxCtas);
  ctas = std::min(ctas, h.c.partial_floats / (2 * S::kRows * (D + 2)));
  a.planned = tiles * a.n > 4 * S::kThreads;
  a.small = tiles * a.n * h.c.kv_heads * ((int64_t)h.c.max_pages * h.c.page_size / kUnit + 2 + kLead) < INT_MAX;
  if (a.planned) {
    const int rc = launch_after(attend_plan<kUnit>, dim3(1), 1024, 0, h.stream, h.c, a, S::kRows, (int)ctas);
    if (rc != WHEAD_OK) return rc;
  }
  // The last CTA joins an item alone: up to 4 rows that is soon done (16 sequences of 4,096 keys 23 us, by a kernel of its own 28), for
  // more it is the longest part of the call (one sequence, 32 rows: 71 us, 22 by a kernel of its own; 16 sequences 50 and 44). Between 4
  // and 8 rows it depends on the parts of an item (1 sequence 24 and 17 us, 8 sequences 20 and 18, 16 sequences 25 and 26).
  const int64_t rows = (int64_t)max_q * a.group;
  a.apart = rows > 8 || (rows > 4 && tiles * a.n * h.c.kv_heads * 8 <= ctas);
  const int rc = launch_after(attend_rows<D, NT>, dim3((unsigned)ctas), S::kThreads, S::kBytes, h.stream, h.c, a);
  return rc == WHEAD_OK && a.apart ? launch_join<D, S::kRows, kUnit>(h, a, (int)ctas, max_q) : rc;
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
  if (!x->q || !x->out || !aligned(x->q, 2) || !aligned(x->out, 16) || !aligned(x->lse, 4) || !aligned(x->indptr, 4) || !aligned(x->slots, 4) || x->max_q < 1) return WHEAD_ERR_INVALID_ARG;
  if (!x->indptr && (x->total % x->n || x->total / x->n > x->max_q)) return WHEAD_ERR_INVALID_ARG;
  const int group = x->heads / kv->kv_heads;
  const int max_q = (int)std::min<int64_t>(x->max_q, x->total);
  const int64_t rows = (int64_t)max_q * group;
  const int tile = tile_rows(kv->head_dim, rows);
  if (rows >= INT_MAX / 2 || (rows + tile - 1) / tile * x->n > kMaxItems) return WHEAD_ERR_UNSUPPORTED;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  AttendArgs a{};
  a.q = x->q;
  a.out = x->out;
  a.lse = x->lse;
  a.indptr = x->indptr;
  a.slots = x->slots;
  a.tree = reinterpret_cast<const unsigned long long*>(x->tree);
  a.total = x->total;
  a.q_token_stride = x->q_token_stride;
  a.q_head_stride = x->q_head_stride;
  a.n = x->n;
  a.each = (int)(x->total / x->n);
  a.max_q = max_q;
  a.heads = x->heads;
  set_group(&a, group);
  a.row_tiles = 1;
  a.dtype = x->dtype;
  a.causal = x->causal;
  a.window = x->window;
  a.tree_words = x->tree_words;
  a.scale = x->scale;
  a.wide_q16 = aligned(x->q, 16) && x->q_token_stride % 8 == 0 && x->q_head_stride % 8 == 0;
  a.wide_q = aligned(x->q, 8) && x->q_token_stride % 4 == 0 && x->q_head_stride % 4 == 0;
  if (tile > 32) return launch_tiles(h, a, max_q);
  switch (kv->head_dim) {
    case 64: return tile == 8 ? launch_rows<64, 1>(h, a, max_q) : tile == 16 ? launch_rows<64, 2>(h, a, max_q) : launch_rows<64, 4>(h, a, max_q);
    case 128: return tile == 8 ? launch_rows<128, 1>(h, a, max_q) : tile == 16 ? launch_rows<128, 2>(h, a, max_q) : launch_rows<128, 4>(h, a, max_q);
    default: return tile == 8 ? launch_rows<256, 1>(h, a, max_q) : launch_rows<256, 2>(h, a, max_q);
  }
}

// kv_schedule.cuh — how an attention over the cache is divided over CTAs.
//
// The work is a list of items, one for each entry, tile of query rows and KV head. A row is a query token and one of the
// query heads of a KV head (row = token * group + head in the group), so that all rows of a tile read the same keys. An
// item is a run of units of UNIT keys, from the first that one of its rows sees to the last, but for those between the first keys that stay
// visible and a window. All units, laid end to end,
// are cut into as many equal ranges as there are CTAs: ragged lengths need no balancing, and a long sequence alone fills
// the device. Each item counts kLead units more than it has, ahead of its own: a CTA that goes on to another item spends some 9,000
// cycles on the joins, the query rows and the first copies, a unit 2,800 to 3,400 (16 sequences of 300 to 8,200 keys: with equal
// units the CTAs with two items ended at 26 us, those with one at 16). An item cut by a range's end leaves partial results (each
// row's running maximum, its sum and its output before the division) in the workspace. Few rows: the last CTA to finish one
// of an item's parts joins them; many rows: a second kernel does. Either way in the order of the keys, so that results do not
// depend on which CTA comes last.
#pragma once

#include "kv_common.cuh"

namespace whead_kv_impl {

constexpr int kLead = 3;

struct AttendArgs {
  const void* q;
  void* out;
  float* lse;
  const int32_t* indptr;
  const int32_t* slots;
  const unsigned long long* tree;
  int64_t total, q_token_stride, q_head_stride;
  int n, each, max_q, heads, group, group_shift, row_tiles, dtype, causal, window, tree_words;
  uint32_t group_mul;  // row / group = (row * group_mul >> 32 + row) >> group_shift, for rows below 2^31
  float scale;
  bool wide_q, wide_q16;  // query rows can be read 8, 16 bytes at a time
  int planned;  // the CTAs' starts are in the workspace
  int apart;    // a kernel of its own joins the parts (few rows; always so for many)
  int small;    // all units are less than 2^31
  int sinks;    // first keys that a window leaves visible, 0 without one (with SINKS, below)
  int early;    // their units
};

// The rows of a tile for entries of at most `rows` rows a KV head: up to 32 for the kernel of few rows (kv_attend_rows.cuh), above for that of many.
// Up to 32 rows the keys' bytes and their unpacking are the work, and the rows ride along in one pass; above, every 32 rows would
// unpack the keys again, and the tiles' products cost the same for 36 rows as for 128. 64 sequences on 8,192 keys, 8 KV heads, by rows
// and tiles: 32 rows 268 and 399 us, 36 rows 510 and 403; 16 on 4,096: 44 and 61, 80 and 54. Fewer rows have kernels of fewer registers: 4
// rows by the kernel for 32 take 254 us, by their own 113. 256 channels: 16 rows' outputs are what the registers hold.
inline int tile_rows(int head_dim, int64_t rows) {
  if (rows <= 8) return 8;
  if (rows <= 16 || head_dim == 256) return 16;
  return rows <= 32 ? 32 : rows <= 128 ? 128 : 256;
}
// Most items of a launch: whoever looks through them steps by up to 1024 beyond the last, in ints.
constexpr int64_t kMaxItems = INT32_MAX - 4096;

// Attention of few rows a KV head, in tiles of 8, 16 or 32 (kv_attend_rows.cuh), and of more (kv_attend_tiles.cuh; head_dim 64 or 128).
template <bool SINKS>
int launch_few(const struct HostCache& h, const AttendArgs& a, int max_q, int tile);
template <bool SINKS>
int launch_tiles(const struct HostCache& h, const AttendArgs& a, int max_q);

// One (entry, row tile): its rows and the units that they see.
struct Tile {
  int slot, len, tokens, first;  // first: row of q of the entry's first token
  int row0, rows;                // the tile's first row, and its rows
  int unit0, units;              // units of one KV head that are seen, and those that are left out before them (with SINKS: after the first keys')
};
// A tile's unit as a unit of the slot. SINKS: the call has first keys that stay visible. Its kernels are apart: one for both cost the others 2 to 4 %
// (32 sequences on 2,000 to 32,768 keys 120.6 us and 122.7, 8 x 17 tokens 31.3 and 32.7, prompts with a window 146 and 149).
template <bool SINKS>
__device__ __forceinline__ int unit_at(const AttendArgs& a, const Tile& t, int u) { return (!SINKS || u >= a.early ? t.unit0 : 0) + u; }

// The token of a row: division by the group, by multiplication with its reciprocal rounded up to 33 bits (Granlund and Montgomery, "Division
// by invariant integers using multiplication", 1994, figure 4.1). A division takes some 150 cycles of latency, and there are several
// before a CTA can load anything.
__device__ __forceinline__ int row_token(const AttendArgs& a, int row) {
  const uint32_t t = __umulhi(a.group_mul, (uint32_t)row);
  return (int)((t + (((uint32_t)row - t) >> (a.group_shift ? 1 : 0))) >> (a.group_shift ? a.group_shift - 1 : 0));
}
inline void set_group(AttendArgs* a, int group) {
  int l = 0;
  while ((1LL << l) < group) ++l;
  a->group = group;
  a->group_shift = l;
  a->group_mul = (uint32_t)(((1ULL << 32) * ((1ULL << l) - (uint64_t)group)) / (uint64_t)group + 1);
}

// The first key in the window of a token at this position. A position may be negative (more query tokens than keys) and a window as long
// as an int holds, so that their difference is formed only where it is not.
__device__ __forceinline__ int window_begin(const AttendArgs& a, int pos) { return pos >= a.window ? pos - a.window + 1 : 0; }

template <int UNIT, bool SINKS>
__device__ __forceinline__ Tile make_tile(const Cache& c, const AttendArgs& a, int item, int tile_rows) {
  Tile t;
  const int i = a.row_tiles == 1 ? item : item / a.row_tiles, m = item - i * a.row_tiles;
  t.slot = a.slots ? a.slots[i] : i;
  t.len = slot_len(c, t.slot);
  if (t.len == 0) t.slot = 0;
  if (a.indptr) {
    const int lo = a.indptr[i], hi = a.indptr[i + 1];
    const bool ok = lo >= 0 && hi >= lo && hi <= a.total && hi - lo <= a.max_q;  // the row tiles and the join's blocks are for max_q
    if (!ok) set_status(c, WHEAD_ERR_INVALID_ARG);
    t.first = ok ? lo : 0;
    t.tokens = ok ? hi - lo : 0;
  } else {
    t.tokens = a.each;
    t.first = t.tokens * i;
  }
  const int64_t all = (int64_t)t.tokens * a.group;
  const int64_t row0 = (int64_t)m * tile_rows;
  t.row0 = (int)row0;
  t.rows = (int)(all - row0 < 0 ? 0 : all - row0 < tile_rows ? all - row0 : tile_rows);
  t.unit0 = t.units = 0;
  if (t.rows == 0) return t;
  const int t0 = row_token(a, t.row0), t1 = row_token(a, t.row0 + t.rows - 1);
  int hi = t.len, lo = 0;
  if (a.causal) hi = min(max(t.len - t.tokens + t1 + 1, 0), t.len);
  if (a.window) lo = window_begin(a, t.len - t.tokens + t0);
  t.unit0 = lo / UNIT;
  if (SINKS) t.unit0 = max(t.unit0 - a.early, 0);
  t.units = max((hi + UNIT - 1) / UNIT - t.unit0, 1);  // at least one: somebody has to write the rows
  return t;
}

// What a tile counts for in the division of the work: all KV heads' units, and their leads.
__device__ __forceinline__ long long tile_cost(const Cache& c, const Tile& t) { return t.units ? (long long)(t.units + kLead) * c.kv_heads : 0; }

// The keys that a row sees: lo <= j < hi (with SINKS, j < sinks too), and the bits of its mask for j >= draft.
struct RowView {
  int lo, hi, draft;
  const unsigned long long* bits;
};

template <bool SINKS>
__device__ __forceinline__ RowView row_view(const AttendArgs& a, const Tile& t, int row) {
  RowView v{0, 0, 0x7FFFFFFF, nullptr};
  if (row >= t.row0 + t.rows) return v;
  const int tok = row_token(a, row);
  const int pos = t.len - t.tokens + tok;
  v.hi = a.causal ? min(pos + 1, t.len) : t.len;
  if (a.window) v.lo = window_begin(a, pos);
  if (a.tree) {
    v.draft = t.len - t.tokens;
    v.bits = a.tree + (int64_t)(t.first + tok) * a.tree_words;
  }
  return v;
}

template <bool SINKS>
__device__ __forceinline__ bool sees(const AttendArgs& a, const RowView& v, int j) {
  if ((j < v.lo && (!SINKS || j >= a.sinks)) || j >= v.hi) return false;
  if (j < v.draft) return true;
  const int u = j - v.draft;
  return (v.bits[u >> 6] >> (u & 63)) & 1;
}

// Where a CTA's range begins: the item, and the number of the item's first unit (of its lead).
struct Start {
  int item;
  int ctas;           // CTAs that have work: fewer than launched where there are fewer units
  long long at;       // number of the item's first unit (of all its KV heads)
  long long total;
};

__device__ __forceinline__ long long range_begin(const Start& s, int cta) { return s.total * cta / s.ctas; }
// the CTA whose range holds unit x
__device__ __forceinline__ int range_owner(const Start& s, long long x) { return (int)(((x + 1) * s.ctas - 1) / s.total); }

// A CTA's piece of one (tile, KV head): its units u0 .. u1 - 1, none where the range ends inside the lead. head_at: number of the lead's
// first unit.
struct Segment {
  Tile tile;
  int item, h, u0, u1;
  long long head_at;
};
// The piece of head h, whose lead begins at head_at, that a range from `at` to `end` holds; the range's rest begins where it ends.
__device__ __forceinline__ long long cut_segment(Segment& s, long long at, long long end) {
  const int from = (int)(at - s.head_at), to = (int)min((long long)(s.tile.units + kLead), end - s.head_at);
  s.u0 = max(from - kLead, 0);
  s.u1 = max(to - kLead, s.u0);
  return s.head_at + to;
}
// The CTAs that hold a head's units, and where the first of them keeps its partial result: in its first place if nothing of its
// range comes before this head.
__device__ __forceinline__ int first_owner(const Start& s, const Segment& g) { return range_owner(s, g.head_at + kLead); }
__device__ __forceinline__ int last_owner(const Start& s, const Segment& g) { return range_owner(s, g.head_at + kLead + g.tile.units - 1); }
__device__ __forceinline__ int part_slot(const Start& s, const Segment& g, int cta) { return 2 * cta + (range_begin(s, cta) >= g.head_at ? 0 : 1); }

// Sum of x over the threads before this one, and over all; `warps` words of shared memory.
template <int THREADS>
__device__ __forceinline__ long long scan64(long long x, long long* warps, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) warps[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const long long y = warps[w];
    if (w < warp) before += y;
    all += y;
  }
  total = all;
  return before + v - x;
}

struct SchedShared {
  long long warps[32];
  long long at;
  int item;
  int has_tile;  // tile is the item's
  Tile tile;
};

// This CTA's start, from the lengths themselves (few items).
template <int THREADS, int UNIT, bool SINKS>
__device__ __forceinline__ Start find_start(const Cache& c, const AttendArgs& a, int tile_rows, SchedShared& s) {
  const int items = a.n * a.row_tiles;
  Start r;
  if (items <= 32 && a.small) {
    // every warp finds the start for itself, a lane an item: no barrier before the CTA's first loads, and 32-bit sums
    const int lane = threadIdx.x & 31;
    Tile tile{};
    if (lane < items) tile = make_tile<UNIT, SINKS>(c, a, lane, tile_rows);
    const int mine = (int)tile_cost(c, tile);
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, sum, o);
      if (lane >= o) sum += y;
    }
    r.total = __shfl_sync(~0u, sum, 31);
    r.ctas = (int)min((long long)gridDim.x, r.total);
    r.item = 0;
    r.at = 0;
    if ((int)blockIdx.x >= r.ctas) return r;
    const int x = (int)range_begin(r, blockIdx.x);
    const int owner = __ffs(__ballot_sync(~0u, x < sum)) - 1;  // sums ascend, and an item without units adds none
    r.item = owner;
    r.at = __shfl_sync(~0u, sum - mine, owner);
    if (threadIdx.x == owner) {
      s.item = owner;
      s.tile = tile;
      s.has_tile = 1;
    }
    __syncthreads();
    return r;
  }
  r.total = 0;
  long long mine = 0, before = 0;
  Tile tile{};
  for (int base = 0; base < items; base += THREADS) {
    const int it = base + threadIdx.x;
    if (it < items) tile = make_tile<UNIT, SINKS>(c, a, it, tile_rows);
    mine = it < items ? tile_cost(c, tile) : 0;
    long long all;
    before = r.total + scan64<THREADS>(mine, s.warps, all);
    r.total += all;
  }
  r.ctas = (int)min((long long)gridDim.x, r.total);
  r.item = 0;
  r.at = 0;
  if ((int)blockIdx.x >= r.ctas) return r;
  const long long x = range_begin(r, blockIdx.x);
  if (items <= THREADS) {
    if (mine > 0 && before <= x && x < before + mine) {
      s.item = threadIdx.x;
      s.at = before;
      s.tile = tile;
      s.has_tile = 1;
    }
  } else {
    if (threadIdx.x == 0) s.has_tile = 0;
    long long sum = 0;
    for (int base = 0; base < items && sum <= x; base += THREADS) {
      const int it = base + threadIdx.x;
      mine = it < items ? tile_cost(c, make_tile<UNIT, SINKS>(c, a, it, tile_rows)) : 0;
      long long all;
      before = sum + scan64<THREADS>(mine, s.warps, all);
      if (mine > 0 && before <= x && x < before + mine) {
        s.item = it;
        s.at = before;
      }
      sum += all;
    }
  }
  __syncthreads();
  r.item = s.item;
  r.at = s.at;
  return r;
}

// The same for all CTAs of a launch, by one CTA, into the workspace (many items).
template <int UNIT, bool SINKS>
static __global__ void __launch_bounds__(1024, 1) attend_plan(const __grid_constant__ Cache c, const __grid_constant__ AttendArgs a, int tile_rows, int ctas) {
  after_previous();
  __shared__ long long warps[32];
  const int items = a.n * a.row_tiles;
  long long total = 0;
  for (int base = 0; base < items; base += 1024) {
    const int it = base + threadIdx.x;
    long long all;
    scan64<1024>(it < items ? tile_cost(c, make_tile<UNIT, SINKS>(c, a, it, tile_rows)) : 0, warps, all);
    total += all;
  }
  Start r;
  r.total = total;
  r.ctas = (int)min((long long)ctas, total);
  long long sum = 0;
  for (int base = 0; base < items; base += 1024) {
    const int it = base + threadIdx.x;
    const long long mine = it < items ? tile_cost(c, make_tile<UNIT, SINKS>(c, a, it, tile_rows)) : 0;
    long long all;
    const long long before = sum + scan64<1024>(mine, warps, all);
    sum += all;
    if (mine > 0) {
      int k = range_owner(r, before);
      if (range_begin(r, k) < before) ++k;
      for (; k < r.ctas && range_begin(r, k) < before + mine; ++k) {
        int32_t* to = c.starts + 4 * k;
        to[0] = it;
        *reinterpret_cast<long long*>(to + 2) = before;
      }
    }
  }
  if (threadIdx.x == 0) {
    c.ctl->pad = r.ctas;
    *reinterpret_cast<long long*>(&c.ctl->ticket[2]) = total;
  }
}

template <int THREADS, int UNIT, bool SINKS>
__device__ __forceinline__ Start get_start(const Cache& c, const AttendArgs& a, int tile_rows, SchedShared& s) {
  if (!a.planned) return find_start<THREADS, UNIT, SINKS>(c, a, tile_rows, s);
  if (threadIdx.x == 0) s.has_tile = 0;
  __syncthreads();
  Start r;
  r.ctas = c.ctl->pad;
  r.total = *reinterpret_cast<const long long*>(&c.ctl->ticket[2]);
  r.item = 0;
  r.at = 0;
  if ((int)blockIdx.x < r.ctas) {
    const int32_t* from = c.starts + 4 * blockIdx.x;
    r.item = from[0];
    r.at = *reinterpret_cast<const long long*>(from + 2);
  }
  return r;
}

// What a joining kernel has to do for the item that begins in this CTA's range and ends outside it: c.records + 4 CTA holds item, KV
// head, parts (none: 0) and the first part's place. Written by one thread, zeros first.
__device__ __forceinline__ void put_record(const Cache& c, int item, int h, int parts, int slot) {
  *reinterpret_cast<int4*>(c.records + 4 * blockIdx.x) = make_int4(item, h, parts, slot);
}

// Joins the parts of the items that are cut: block (k, z) the z-th `slice` rows of the item that begins in CTA k's range. Bound by
// latency, so four parts' loads are under way at once. A kernel of its own spreads this over the device: by the last CTA of each
// item it took 20 us of 84 (8 sequences, 68 rows, 5 parts), and 55 of 71 for one sequence (32 rows, 32 parts).
template <int D, int ROWS, int UNIT, bool SINKS>
__global__ void __launch_bounds__(128) join_parts(const __grid_constant__ Cache c, const __grid_constant__ AttendArgs a, int slice) {
  after_previous();
  const int4 record = __ldcg(reinterpret_cast<const int4*>(c.records) + blockIdx.x);
  const int parts = record.z;
  if (parts == 0) return;
  constexpr int kPart = ROWS * (D + 2), kLanes = D / 4, kAt = 128 / kLanes;
  const Tile tile = make_tile<UNIT, SINKS>(c, a, record.x, ROWS);
  const float gv = c.v_scale[record.y];
  auto part_at = [&](int k) { return c.partial + (int64_t)(k == 0 ? record.w : 2 * ((int)blockIdx.x + k)) * kPart; };
  const int col = threadIdx.x % kLanes * 4;
#pragma unroll 1
  for (int i = 0; i < slice; i += kAt) {
    const int row = blockIdx.y * slice + i + threadIdx.x / kLanes;
    if (row >= tile.rows) return;
    float m = kNoKey, l = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < parts; k0 += 4) {
      float pm[4], pl[4];
      float4 y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float* p = part_at(min(k0 + k, parts - 1));
        pm[k] = __ldcg(p + row);
        pl[k] = __ldcg(p + ROWS + row);
        y[k] = __ldcg(reinterpret_cast<const float4*>(p + 2 * ROWS + row * D + col));
      }
      float now = m;
#pragma unroll
      for (int k = 0; k < 4; ++k) now = fmaxf(now, pm[k]);
      const float r0 = ex2(m - now);
      m = now;
      l *= r0;
      v.x *= r0; v.y *= r0; v.z *= r0; v.w *= r0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k0 + k >= parts) break;
        const float r1 = ex2(pm[k] - m);
        l += pl[k] * r1;
        v.x += y[k].x * r1; v.y += y[k].y * r1; v.z += y[k].z * r1; v.w += y[k].w * r1;
      }
    }
    const int grow = tile.row0 + row;
    const int tok = row_token(a, grow);
    const int64_t at = (int64_t)(tile.first + tok) * a.heads + record.y * a.group + grow - tok * a.group;
    const float q = l != 0.0f ? gv / l : 0.0f;
    if (l == 0.0f) v = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + col) =
        make_uint2(pack16(v.x * q, v.y * q, a.dtype), pack16(v.z * q, v.w * q, a.dtype));
    if (a.lse && col == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// A block takes as many rows as its threads hold, and no second pass (one sequence of 4,096 keys, 256 rows: 35 us, with 16 rows a block
// 45). Where entries have several tiles there are blocks enough, most with nothing to join, and fewer are better (2 x 2048 tokens 299
// us, with 4 rows a block 300; one of 2048 on 512 keys 29 and 32).
template <int D, int ROWS, int UNIT, bool SINKS>
int launch_join(const HostCache& h, const AttendArgs& a, int ctas, int max_q) {
  const int64_t most = (int64_t)max_q * a.group, rows = most < ROWS ? most : ROWS;
  const int slice = most > 256 ? 16 : 512 / D;
  return launch_after(join_parts<D, ROWS, UNIT, SINKS>, dim3((unsigned)ctas, (unsigned)((rows + slice - 1) / slice)), 128, 0, h.stream, h.c, a, slice);
}

}  // namespace whead_kv_impl

// kv_attend_tiles.cu — attention over the 4-bit paged cache for many query rows: 128 rows a tile on the tensor cores' tcgen05
// instructions, with scores and outputs in tensor memory.
//
// The mathematics is kv_attend.cu's. A block is 128 keys. Four warps turn its codes into f16 tiles in shared memory, which TILES
// tiles of 128 rows then share; one thread issues the products S = Q K^T and O += P V; one warpgroup a tile reads S, a row a
// thread, and puts P where S was. The order of the products is PV(tile 0, block j), QK(tile 0, block j + 1), PV(tile 1, ...):
// one tile's softmax runs under the other's products. With one tile (at most 128 rows) two CTAs share an SM instead.
//
// Shared memory holds operands in rows of 128 bytes (64 f16), 8 rows to an atom of 1024 bytes, 16-byte chunks swizzled by the row.
// Channels 16 b + 8 s .. + 7 of a query row or key lie in chunk 4 s + b % 4 of the row, not 2 b + s: a warp's stores of a block's keys
// (8 bytes a lane, 4 lanes a key) then meet every bank once. Values lie with their channels as rows; row 16 b + i holds channel
// 16 b + 2 i for i < 8 and 16 b + 2 (i - 8) + 1 above, as the lanes have them.
#include "kv_schedule.cuh"

#include <algorithm>
#include <climits>

namespace whead_kv_impl {

namespace {

constexpr int kBlock = 128;      // keys
constexpr float kBias = 7.0f;    // as in kv_attend.cu
constexpr float kSlack = 15.0f;
constexpr float kNoKey = -1e30f;

template <int D, int TILES>
struct Shape {
  static constexpr int kRows = 128 * TILES;
  static constexpr int kBufs = TILES;                    // of key and value tiles
  static constexpr int kCtas = TILES == 1 ? 2 : 1;       // of an SM
  static constexpr int kSoft = 4 * TILES;                // softmax warps, then those that unpack, then the one that issues
  static constexpr int kUnpack = 4, kMine = 8 / kUnpack; // groups of a block that each of them takes
  static constexpr int kIssue = kSoft + kUnpack;
  static constexpr int kThreads = (kIssue + 1) * 32;
  static constexpr int kGroup = 18 * D;
  static constexpr int kQ = 128 * D * 2, kK = kBlock * D * 2, kV = D * kBlock * 2;
  static constexpr int kOffQ = 1024, kOffK = kOffQ + TILES * kQ, kOffV = kOffK + kBufs * kK;
  static constexpr int kBytes = kOffV + kBufs * kV + 1024;  // + alignment
  static constexpr int kCols = 256 * TILES;                 // of tensor memory: S of each tile, O of each tile
};

struct Head {
  SchedShared sched;
  unsigned long long k_full[2], k_free[2], v_full[2], v_free[2], s_full[2], p_full[2], o_full[2], q_full, drain;
  uint32_t tmem;
};
static_assert(sizeof(Head) <= 1024, "");

__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  // rows of 128 bytes, atoms of 8 rows 1024 bytes apart, 128-byte swizzle
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define KV_R32(x) "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), \
  "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), \
  "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), \
  "=r"(x[29]), "=r"(x[30]), "=r"(x[31])

// 32 columns of this warp's lanes
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&x)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
               "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];" : KV_R32(x) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load(uint32_t (&x)[32]) {
  // the registers are operands, so that no use of them moves before the wait
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]),
                 "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]), "+r"(x[16]), "+r"(x[17]), "+r"(x[18]),
                 "+r"(x[19]), "+r"(x[20]), "+r"(x[21]), "+r"(x[22]), "+r"(x[23]), "+r"(x[24]), "+r"(x[25]), "+r"(x[26]), "+r"(x[27]),
                 "+r"(x[28]), "+r"(x[29]) :: "memory");
  asm volatile("" : "+r"(x[30]), "+r"(x[31]));
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
                 "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]) : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&x)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
               "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
               ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
                 "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(x[16]), "r"(x[17]), "r"(x[18]), "r"(x[19]),
                 "r"(x[20]), "r"(x[21]), "r"(x[22]), "r"(x[23]), "r"(x[24]), "r"(x[25]), "r"(x[26]), "r"(x[27]), "r"(x[28]), "r"(x[29]),
                 "r"(x[30]), "r"(x[31]) : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n fma.rn.f32x2 d, a, b, c;\n"
      " mov.b64 {%0, %1}, d;\n}\n" : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The largest of a row's 128 scores, of those whose bits are set where MASKED (a code of its own: the bits cost more than the rest).
template <bool MASKED>
__device__ __forceinline__ float row_max(uint32_t st, const uint32_t (&seen)[4]) {
  float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    uint32_t x[32], y[32];
    tmem_load32(st + i * 32, x);
    tmem_load32(st + i * 32 + 32, y);
    tmem_wait_load(x);
    tmem_wait_load(y);
    if (MASKED) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        a0 = fmaxf(a0, (seen[i] >> k) & 1 ? __uint_as_float(x[k]) : -INFINITY);
        a1 = fmaxf(a1, (seen[i + 1] >> k) & 1 ? __uint_as_float(y[k]) : -INFINITY);
      }
      __syncwarp();
    } else {
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        a0 = max3(a0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        a1 = max3(a1, __uint_as_float(y[k]), __uint_as_float(y[k + 1]));
      }
    }
  }
  return fmaxf(a0, a1);
}

// Scores to p = 2^(score f - m), as f16 where the scores were; l: their sum.
template <bool MASKED>
__device__ __forceinline__ void row_exp(uint32_t st, const uint32_t (&seen)[4], float f, float m, float2& l) {
  const float2 f2 = make_float2(f, f), m2 = make_float2(-m, -m);
  float2 sum[2] = {l, make_float2(0.f, 0.f)};
  uint32_t x[2][32];
  tmem_load32(st, x[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t (&y)[32] = x[i & 1];
    tmem_wait_load(y);
    if (i < 3) tmem_load32(st + i * 32 + 32, x[(i + 1) & 1]);
    uint32_t p[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float2 d = fma2(make_float2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), f2, m2);
      d.x = ex2(d.x);
      d.y = ex2(d.y);
      if (MASKED) {
        if (!((seen[i] >> (2 * k)) & 1)) d.x = 0.0f;
        if (!((seen[i] >> (2 * k + 1)) & 1)) d.y = 0.0f;
      }
      sum[k & 1] = add2(sum[k & 1], d);
      p[k] = pack16(d.x, d.y, WHEAD_KV_F16);
    }
    if (MASKED) __syncwarp();
    tmem_store16(st + i * 16, p);  // over scores that have been read
  }
  l = add2(sum[0], sum[1]);
  tmem_wait_store();
}

// The keys key .. key + 31 that a row sees, as bits.
__device__ __forceinline__ uint32_t sees32(const AttendArgs& a, const RowView& v, int key) {
  uint32_t m = ~0u;
  if (key + 32 > v.hi) m = v.hi <= key ? 0u : (1u << (v.hi - key)) - 1u;
  if (key < v.lo) m &= v.lo - key >= 32 ? 0u : ~0u << (v.lo - key);
  if (v.bits != nullptr && key + 32 > v.draft && m) {
    const int u = key - v.draft;  // the first key's bit
    uint32_t b;
    if (u < 0) {
      b = (uint32_t)(v.bits[0] << -u) | ((1u << -u) - 1u);
    } else {
      const int w = u >> 6, s = u & 63;
      unsigned long long x = w < a.tree_words ? v.bits[w] >> s : 0ull;
      if (s > 32 && w + 1 < a.tree_words) x |= v.bits[w + 1] << (64 - s);
      b = (uint32_t)x;
    }
    m &= b;
  }
  return m;
}

struct Segment {
  Tile tile;
  int item, h, u0, u1;
  long long head_at;
};

// A CTA's way through its range; every role walks it for itself.
template <int D, int TILES>
struct Walk {
  long long cur, end, item_at;
  int item, n;  // n: blocks before this segment
  __device__ __forceinline__ bool next(const Cache& c, const AttendArgs& a, Segment& s) {
    if (cur >= end) return false;
    while (true) {
      s.tile = make_tile<kBlock>(c, a, item, Shape<D, TILES>::kRows);
      if (s.tile.units > 0) break;
      ++item;
    }
    s.item = item;
    const int past = (int)(cur - item_at);
    s.h = past / s.tile.units;
    s.u0 = past - s.h * s.tile.units;
    s.head_at = cur - s.u0;
    s.u1 = (int)min((long long)s.tile.units, s.u0 + (end - cur));
    cur = s.head_at + s.u1;
    if (s.u1 == s.tile.units && s.h == c.kv_heads - 1) {
      item_at = cur;
      ++item;
    }
    return true;
  }
};

// A wait that has run out is reported once; the role then goes on without waiting, on whatever is there, to its end.
__device__ __forceinline__ void await(const Cache& c, uint32_t bar, uint32_t parity, bool& dead) {
  if (!dead && !mbar_wait(bar, parity)) {
    set_status(c, WHEAD_ERR_TIMEOUT);
    dead = true;
  }
}

template <int D>
struct RawK {
  uint4 code[D / 64];
  uint2 scale[D / 64];
};
template <int D>
struct RawV {
  uint4 code[D / 64];
  uint4 scale[D / 64];
};

template <int D, int TILES>
__global__ void __launch_bounds__((Shape<D, TILES>::kThreads), (Shape<D, TILES>::kCtas)) attend_tiles(Cache c, AttendArgs a) {
  using S = Shape<D, TILES>;
  constexpr int NB = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Head& s = *reinterpret_cast<Head*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.k_full[i]), S::kUnpack);
      mbar_init(smem_u32(&s.k_free[i]), 1);
      mbar_init(smem_u32(&s.v_full[i]), S::kUnpack);
      mbar_init(smem_u32(&s.v_free[i]), 1);
      mbar_init(smem_u32(&s.s_full[i]), 1);
      mbar_init(smem_u32(&s.p_full[i]), 4);
      mbar_init(smem_u32(&s.o_full[i]), 1);
    }
    mbar_init(smem_u32(&s.q_full), S::kSoft);
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
  }
  const Start start = get_start<S::kThreads, kBlock>(c, a, S::kRows, s.sched);
  if ((int)blockIdx.x >= start.ctas) {
    if (tid == 0) *reinterpret_cast<int4*>(c.records + 4 * blockIdx.x) = make_int4(0, 0, 0, 0);
    return;
  }
  if (warp == S::kIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "n"(S::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s.tmem;
  Walk<D, TILES> walk{range_begin(start, blockIdx.x), range_begin(start, blockIdx.x + 1), start.at, start.item, 0};
  const long long begin = walk.cur;
  Segment sg;
  bool dead = false;

  if (warp == S::kIssue) {
    // ---- the thread that issues the products
    if (lane == 0) {
      constexpr uint32_t kQK = (1u << 4) | ((kBlock / 8u) << 17) | ((128u / 16u) << 24);  // fp32 from f16 x f16, both along k
      constexpr uint32_t kPV = (1u << 4) | ((D / 8u) << 17) | ((128u / 16u) << 24);
      const uint32_t q0 = smem_u32(smem + S::kOffQ), k0 = smem_u32(smem + S::kOffK), v0 = smem_u32(smem + S::kOffV);
      auto scores = [&](int t, int buf) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + t * 128, tile_desc(q0 + t * S::kQ + k / 4 * (128 * 128) + k % 4 * 32), tile_desc(k0 + buf * S::kK + k / 4 * (kBlock * 128) + k % 4 * 32),
                 kQK, k > 0);
      };
      auto outputs = [&](int t, int buf, bool add) {
#pragma unroll
        for (int k = 0; k < kBlock / 16; ++k)
          mma_ts(tmem + TILES * 128 + t * 128, tmem + t * 128 + k * 8, tile_desc(v0 + buf * S::kV + k / 4 * (D * 128) + k % 4 * 32), kPV, add || k > 0);
      };
      int n = 0, seg = 0;
      while (walk.next(c, a, sg)) {
        const int blocks = sg.u1 - sg.u0;
        await(c, smem_u32(&s.q_full), seg & 1, dead);
        await(c, smem_u32(&s.k_full[n % S::kBufs]), n / S::kBufs & 1, dead);
        if (dead) break;
        fence_after();
        for (int t = 0; t < TILES; ++t) {
          scores(t, n % S::kBufs);
          commit(smem_u32(&s.s_full[t]));
        }
        commit(smem_u32(&s.k_free[n % S::kBufs]));
        for (int j = 0; j < blocks && !dead; ++j, ++n) {
          const bool more = j + 1 < blocks;
          const int buf = n % S::kBufs, next = (n + 1) % S::kBufs;
          await(c, smem_u32(&s.v_full[buf]), n / S::kBufs & 1, dead);
          for (int t = 0; t < TILES; ++t) {
            await(c, smem_u32(&s.p_full[t]), n & 1, dead);
            if (dead) break;
            fence_after();
            outputs(t, buf, j > 0);
            if (t == TILES - 1) commit(smem_u32(&s.v_free[buf]));
            if (more) {
              if (t == 0) await(c, smem_u32(&s.k_full[next]), (n + 1) / S::kBufs & 1, dead);
              if (dead) break;
              fence_after();
              scores(t, next);
              commit(smem_u32(&s.s_full[t]));
              if (t == TILES - 1) commit(smem_u32(&s.k_free[next]));
            } else {
              commit(smem_u32(&s.o_full[t]));
            }
          }
        }
        if (dead) break;
        ++seg;
      }
      // nothing may be under way when the CTA gives its tensor memory back
      commit(smem_u32(&s.drain));
      mbar_wait(smem_u32(&s.drain), 0);
    }
    __syncwarp();
  } else if (warp >= S::kSoft) {
    // ---- codes to f16 tiles: groups w, w + kUnpack, .. of each block
    const int w = warp - S::kSoft, g = lane >> 2, t = lane & 3;
    const int64_t page_bytes = (int64_t)c.kv_heads * (c.page_size >> 4) * S::kGroup;
    int n = 0;
    while (walk.next(c, a, sg)) {
      const int32_t* table = c.tables + (int64_t)sg.tile.slot * c.max_pages;
      const uint8_t* base = c.pool + (int64_t)sg.h * (c.page_size >> 4) * S::kGroup;
      const int len = sg.tile.len, stop = min((sg.tile.unit0 + sg.u1) * kBlock, len);
      // codes come one block ahead of the tiles, the numbers of their pages two
      RawK<D> rk[S::kMine];
      RawV<D> rv[S::kMine];
      int page[S::kMine];
      auto look = [&](int u) {
#pragma unroll
        for (int i = 0; i < S::kMine; ++i) {
          const int key = u * kBlock + (w + S::kUnpack * i) * 16;
          page[i] = key < stop ? __ldg(table + (key >> c.page_shift)) : 0;
        }
      };
      auto group_at = [&](int i, int key) -> const uint8_t* {
        if ((unsigned)page[i] >= (unsigned)c.num_pages) {
          set_status(c, WHEAD_ERR_INTERNAL);
          page[i] = 0;
        }
        return base + page[i] * page_bytes + ((key & (c.page_size - 1)) >> 4) * S::kGroup;
      };
      auto fetch_k = [&](int u) {
#pragma unroll
        for (int i = 0; i < S::kMine; ++i) {
          const int key = u * kBlock + (w + S::kUnpack * i) * 16;
          if (key >= stop) continue;
          const uint8_t* gp = group_at(i, key);
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            rk[i].code[j] = __ldg(reinterpret_cast<const uint4*>(gp + j * 512) + lane);
            rk[i].scale[j] = __ldg(reinterpret_cast<const uint2*>(gp + 8 * D + g * 2 * NB) + j);
          }
        }
      };
      auto fetch_v = [&](int u) {
#pragma unroll
        for (int i = 0; i < S::kMine; ++i) {
          const int key = u * kBlock + (w + S::kUnpack * i) * 16;
          if (key >= stop) continue;
          const uint8_t* gp = group_at(i, key);
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            rv[i].code[j] = __ldg(reinterpret_cast<const uint4*>(gp + 9 * D + j * 512) + lane);
            rv[i].scale[j] = __ldg(reinterpret_cast<const uint4*>(gp + 17 * D + t * 4 * NB) + j);
          }
        }
      };
      const int first = sg.tile.unit0 + sg.u0;
      look(first);
      fetch_k(first);
      fetch_v(first);
      look(first + 1);
      for (int u = first; u < sg.tile.unit0 + sg.u1; ++u, ++n) {
        const int buf = n % S::kBufs;
        const uint32_t used = (n / S::kBufs - 1) & 1;
        if (n >= S::kBufs) await(c, smem_u32(&s.k_free[buf]), used, dead);
#pragma unroll
        for (int i = 0; i < S::kMine; ++i) {
          const int gi = w + S::kUnpack * i;
          if (u * kBlock + gi * 16 < len) {
            uint8_t* to = smem + S::kOffK + buf * S::kK + gi * 2048 + g * 128 + (t & 1) * 8;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const uint4 kw = rk[i].code[b / 4];
              uint32_t x[4], s0, s1;
              e2m1x8_to_half2(b % 4 == 0 ? kw.x : b % 4 == 1 ? kw.y : b % 4 == 2 ? kw.z : kw.w, x);
              e4m3x4_to_half2(b % 4 < 2 ? rk[i].scale[b / 4].x : rk[i].scale[b / 4].y, s0, s1);
              const uint32_t sc = b & 1 ? s1 : s0;
              uint8_t* at = to + b / 4 * (kBlock * 128) + ((((t >> 1) * 4 + b % 4) ^ g) << 4);
              *reinterpret_cast<uint2*>(at) = make_uint2(hmul2_low(x[0], sc), hmul2_low(x[2], sc));
              *reinterpret_cast<uint2*>(at + 1024) = make_uint2(hmul2_high(x[1], sc), hmul2_high(x[3], sc));
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.k_full[buf]));
        fetch_k(u + 1);
        if (n >= S::kBufs) await(c, smem_u32(&s.v_free[buf]), used, dead);
#pragma unroll
        for (int i = 0; i < S::kMine; ++i) {
          const int gi = w + S::kUnpack * i, key0 = u * kBlock + gi * 16;
          // what lies past the length may be anything: it becomes zero, so that 0 x NaN does not arise
          uint32_t live = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (key0 + 2 * t + (k & 1) + (k >> 1) * 8 < len) live |= 0xFFu << (8 * k);
          uint8_t* to = smem + S::kOffV + buf * S::kV + gi / 4 * (D * 128) + g * 128 + t * 4;
          const int c0 = (gi % 4 * 2 ^ g) << 4, c1 = ((gi % 4 * 2 + 1) ^ g) << 4;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint4 vw = rv[i].code[b / 4], vs = rv[i].scale[b / 4];
            uint32_t x[4], s0, s1;
            e2m1x8_to_half2(b % 4 == 0 ? vw.x : b % 4 == 1 ? vw.y : b % 4 == 2 ? vw.z : vw.w, x);
            e4m3x4_to_half2((b % 4 == 0 ? vs.x : b % 4 == 1 ? vs.y : b % 4 == 2 ? vs.z : vs.w) & live, s0, s1);
            uint8_t* at = to + b * 2048;
            *reinterpret_cast<uint32_t*>(at + c0) = hmul2(x[0], s0);
            *reinterpret_cast<uint32_t*>(at + 1024 + c0) = hmul2(x[1], s0);
            *reinterpret_cast<uint32_t*>(at + c1) = hmul2(x[2], s1);
            *reinterpret_cast<uint32_t*>(at + 1024 + c1) = hmul2(x[3], s1);
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.v_full[buf]));
        fetch_v(u + 1);
        look(u + 2);
      }
    }
  } else {
    // ---- softmax: a thread a row
    const int t = warp >> 2, sub = t * 128, r = sub + (warp & 3) * 32 + lane;  // row of the CTA's tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;                         // this warp's lanes of tensor memory (lane 32 w at bit 16)
    const uint32_t st = tmem + t * 128 + lanes, ot = tmem + TILES * 128 + t * 128 + lanes;
    int n = 0, seg = 0;
    while (walk.next(c, a, sg)) {
      const Tile tile = sg.tile;
      const int row = tile.row0 + r;
      const bool live = r < tile.rows;
      const int tok = row / a.group, head = sg.h * a.group + row % a.group;
      const bool idle = (warp & 3) * 32 + sub >= tile.rows;  // no row of this warp is one: its part of P may be anything
      float f;
      {
        // the warp's query rows, from a power of two to f16; a row is kPer lanes with 8 channels each, kAtOnce rows a load. The
        // sign of the scale goes into the rows, so that f is positive and scores need it only after their maximum is known.
        constexpr int kPer = D / 8, kAtOnce = 32 / kPer, kTurns = 32 / kAtOnce;
        const float to_log2 = a.scale * c.k_scale[sg.h] * kLog2e;
        const long long at = live ? (long long)(tile.first + tok) * a.q_token_stride + (long long)head * a.q_head_stride : -1;
        const int sub_lane = lane % kPer, sub_row = lane / kPer;
        const int b = sub_lane / 2, chunk = (sub_lane & 1) * 4 + b % 4;
        uint8_t* to = smem + S::kOffQ + t * S::kQ + (warp & 3) * 32 * 128 + b / 4 * (128 * 128);
        f = 0.0f;
#pragma unroll 1
        for (int i0 = 0; i0 < kTurns; i0 += 8) {
          uint4 x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const long long from = __shfl_sync(~0u, at, (i0 + i) * kAtOnce + sub_row);
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (from >= 0) {
              const uint2 lo = load_four(a.q, from + sub_lane * 8, a.wide_q), hi = load_four(a.q, from + sub_lane * 8 + 4, a.wide_q);
              x[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 y[4] = {unpack16(x[i].x, a.dtype), unpack16(x[i].y, a.dtype), unpack16(x[i].z, a.dtype), unpack16(x[i].w, a.dtype)};
            float big = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(y[k].x), fabsf(y[k].y)));
#pragma unroll
            for (int o = 1; o < kPer; o <<= 1) big = fmaxf(big, __shfl_xor_sync(~0u, big, o));
            // 2^e <= big < 2^(e + 1), in the range whose powers of two are normal both ways
            const int e = min(max((int)((__float_as_uint(big) >> 23) & 255) - 127, -100), 100);
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 13 - e) << 23), to_log2), down = __uint_as_float((uint32_t)(127 - 13 + e) << 23);
            uint32_t z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = pack16(y[k].x * up, y[k].y * up, WHEAD_KV_F16);
            const int mine = (i0 + i) * kAtOnce + sub_row;
            *reinterpret_cast<uint4*>(to + mine * 128 + ((chunk ^ (mine & 7)) << 4)) = make_uint4(z[0], z[1], z[2], z[3]);
            const float of = __shfl_sync(~0u, down, (lane % kAtOnce) * kPer);
            if (lane / kAtOnce == i0 + i) f = of * fabsf(to_log2);
          }
        }
        fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.q_full));
      }
      const RowView view = row_view(a, tile, row);
      const int w0 = (tile.row0 + sub) / a.group, w1 = (tile.row0 + max(min(sub + 128, tile.rows), sub + 1) - 1) / a.group, past = tile.len - tile.tokens;
      const int free_hi = a.tree ? min(past, past + w0 + 1) : a.causal ? min(past + w0 + 1, tile.len) : tile.len;
      const int free_lo = a.window ? max(past + w1 - a.window + 1, 0) : 0;
      float m = kNoKey;
      float2 l = make_float2(0.f, 0.f);
      for (int u = sg.u0; u < sg.u1; ++u, ++n) {
        const int key0 = (tile.unit0 + u) * kBlock;
        await(c, smem_u32(&s.s_full[t]), n & 1, dead);
        dead = __any_sync(~0u, dead);
        fence_after();
        if (idle) {
          fence_before();
          if (lane == 0) mbar_arrive(smem_u32(&s.p_full[t]));
          continue;
        }
        const bool masked = key0 < free_lo || key0 + kBlock > free_hi;
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};
        if (masked) {
#pragma unroll
          for (int i = 0; i < 4; ++i) seen[i] = sees32(a, view, key0 + 32 * i);
          __syncwarp();
        }
        float top = masked ? row_max<true>(st, seen) : row_max<false>(st, seen);
        top = top == -INFINITY ? top : top * f;  // -inf: nothing seen, whatever f is
        const bool raise = top > m + kSlack;
        if (__any_sync(~0u, raise)) {
          const float now = raise ? top - kBias : m, rr = ex2(m - now);
          m = now;
          l.x *= rr;
          l.y *= rr;
          if (u > sg.u0) {  // the products before this block's are done: its scores were issued after them
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t x[32];
              tmem_load32(ot + i * 32, x);
              tmem_wait_load(x);
#pragma unroll
              for (int k = 0; k < 32; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * rr);
              tmem_store32(ot + i * 32, x);
            }
          }
        }
        if (masked) row_exp<true>(st, seen, f, m, l);
        else row_exp<false>(st, seen, f, m, l);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.p_full[t]));
      }
      await(c, smem_u32(&s.o_full[t]), seg & 1, dead);
      dead = __any_sync(~0u, dead);
      ++seg;
      fence_after();
      const bool whole = sg.u0 == 0 && sg.u1 == tile.units;
      const float ll = l.x + l.y;
      constexpr int kPart = S::kRows * (D + 2);
      const int64_t out_row = (int64_t)(tile.first + tok) * a.heads + head;
      const float gv = c.v_scale[sg.h];
      float* part = c.partial + (int64_t)(2 * blockIdx.x + (sg.head_at + sg.u0 == begin ? 0 : 1)) * kPart;
      const float scale = whole ? (ll != 0.0f ? gv / ll : 0.0f) : 1.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t x[32];
        tmem_load32(ot + i * 32, x);
        tmem_wait_load(x);
#pragma unroll
        for (int b = 0; b < 2 && live; ++b) {  // 16 channels: column i and column 8 + i are channels 2i and 2i + 1
          float y[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[2 * k] = __uint_as_float(x[b * 16 + k]) * scale;
            y[2 * k + 1] = __uint_as_float(x[b * 16 + 8 + k]) * scale;
          }
          if (whole) {
            if (ll == 0.0f) {
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = 0.0f;
            }
            uint16_t* to = static_cast<uint16_t*>(a.out) + out_row * D + i * 32 + b * 16;
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              *reinterpret_cast<uint4*>(to + k) = make_uint4(pack16(y[k], y[k + 1], a.dtype), pack16(y[k + 2], y[k + 3], a.dtype),
                                                             pack16(y[k + 4], y[k + 5], a.dtype), pack16(y[k + 6], y[k + 7], a.dtype));
          } else {
            float* to = part + 2 * S::kRows + r * D + i * 32 + b * 16;
#pragma unroll
            for (int k = 0; k < 16; k += 4) __stcg(reinterpret_cast<float4*>(to + k), make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]));
          }
        }
        __syncwarp();
      }
      if (whole) {
        if (live && a.lse) a.lse[out_row] = ll == 0.0f ? -INFINITY : (m + log2f(ll)) * kLn2;
        continue;
      }
      if (live) {
        __stcg(part + r, m);
        __stcg(part + S::kRows + r, ll);
      }
    }
    // what the joining kernel has to do for the item that begins in this CTA's range and ends outside it
    if (tid == 0) {
      int4 record = make_int4(0, 0, 0, 0);
      if (sg.u0 == 0 && sg.u1 < sg.tile.units)
        record = make_int4(sg.item, sg.h, range_owner(start, sg.head_at + sg.tile.units - 1) - (int)blockIdx.x + 1,
                           2 * blockIdx.x + (sg.head_at == begin ? 0 : 1));
      *reinterpret_cast<int4*>(c.records + 4 * blockIdx.x) = record;
    }
  }
  // tensor memory goes back when every role is through with it
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == S::kIssue) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kCols) : "memory");
}

// Joins the parts of the items that are cut: block (k, z) rows 16 z .. of the item that begins in CTA k's range. A kernel of its own
// spreads this over the device: by the last CTA of each item it took 20 us of 84 (68 rows, 5 parts), here it takes 4.
template <int D, int ROWS>
__global__ void __launch_bounds__(128) join_parts(Cache c, AttendArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 record = __ldcg(reinterpret_cast<const int4*>(c.records) + blockIdx.x);
  const int parts = record.z;
  if (parts == 0) return;
  constexpr int kPart = ROWS * (D + 2), kLanes = D / 4, kAt = 128 / kLanes, kSlice = 16;
  const Tile tile = make_tile<kBlock>(c, a, record.x, ROWS);
  const float gv = c.v_scale[record.y];
  auto part_at = [&](int k) { return c.partial + (int64_t)(k == 0 ? record.w : 2 * ((int)blockIdx.x + k)) * kPart; };
  const int col = threadIdx.x % kLanes * 4;
#pragma unroll 1
  for (int i = 0; i < kSlice; i += kAt) {
    const int row = blockIdx.y * kSlice + i + threadIdx.x / kLanes;
    if (row >= tile.rows) return;
    float m = kNoKey, l = 0.0f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float* p = part_at(k);
      const float pm = __ldcg(p + row), pl = __ldcg(p + ROWS + row);
      const float4 y = __ldcg(reinterpret_cast<const float4*>(p + 2 * ROWS + row * D + col));
      const float now = fmaxf(m, pm), r0 = ex2(m - now), r1 = ex2(pm - now);
      m = now;
      l = l * r0 + pl * r1;
      v.x = v.x * r0 + y.x * r1; v.y = v.y * r0 + y.y * r1; v.z = v.z * r0 + y.z * r1; v.w = v.w * r0 + y.w * r1;
    }
    const int grow = tile.row0 + row;
    const int64_t at = (int64_t)(tile.first + grow / a.group) * a.heads + record.y * a.group + grow % a.group;
    const float q = l != 0.0f ? gv / l : 0.0f;
    if (l == 0.0f) v = make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at * D + col) =
        make_uint2(pack16(v.x * q, v.y * q, a.dtype), pack16(v.z * q, v.w * q, a.dtype));
    if (a.lse && col == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

template <int D, int TILES>
int launch(const HostCache& h, AttendArgs a, int max_q) {
  using S = Shape<D, TILES>;
  static bool granted = false;
  if (!granted) {
    if (cudaFuncSetAttribute(attend_tiles<D, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kBytes) != cudaSuccess) {
      (void)cudaGetLastError();
      return WHEAD_ERR_CUDA;
    }
    granted = true;
  }
  const int64_t tiles = ((int64_t)max_q * a.group + S::kRows - 1) / S::kRows;
  if (tiles * a.n >= INT_MAX) return WHEAD_ERR_UNSUPPORTED;
  a.row_tiles = (int)tiles;
  int64_t ctas = std::min<int64_t>((int64_t)h.sms * S::kCtas, kMaxCtas);
  ctas = std::min(ctas, h.c.partial_floats / (2 * S::kRows * (D + 2)));
  a.planned = tiles * a.n > 2 * S::kThreads;
  if (a.planned) attend_plan<kBlock><<<1, 1024, 0, h.stream>>>(h.c, a, S::kRows, (int)ctas);
  attend_tiles<D, TILES><<<(unsigned)ctas, S::kThreads, S::kBytes, h.stream>>>(h.c, a);
  // the joining kernel's blocks may be placed while the last CTAs still work; they wait for the grid before they read
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = dim3((unsigned)ctas, (unsigned)std::min<int64_t>(S::kRows / 16, ((int64_t)max_q * a.group + 15) / 16));
  config.blockDim = dim3(128);
  config.stream = h.stream;
  config.attrs = &early;
  config.numAttrs = 1;
  if (cudaLaunchKernelEx(&config, join_parts<D, S::kRows>, h.c, a) != cudaSuccess) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  return launch_status();
}

}  // namespace

int launch_tiles(const HostCache& h, const AttendArgs& a, int max_q) {
  const int64_t rows = (int64_t)max_q * a.group;
  if (h.c.head_dim == 64) return rows <= 128 ? launch<64, 1>(h, a, max_q) : launch<64, 2>(h, a, max_q);
  return rows <= 128 ? launch<128, 1>(h, a, max_q) : launch<128, 2>(h, a, max_q);
}

}  // namespace whead_kv_impl

// kv_attend_tiles.cu — attention over the 4-bit paged cache for many query rows: 128 rows a tile on the tensor cores' tcgen05
// instructions, with scores and outputs in tensor memory.
//
// The mathematics is kv_attend.cu's. A block is 128 keys. Eight warps turn its codes into f16 tiles in shared memory, which TILES
// tiles of 128 rows then share; two warps a tile issue the products, one S = Q K^T, one O += P V (one warp for both: its waits for
// the softmax held the next block's scores back); four warps a tile read S, a
// row a thread, and put P where S was. Tensor memory holds two S (128 columns each) beside the outputs. With one tile (at most 128
// rows) the next block's scores are there when a block's softmax ends. With two, a tile's S is one buffer: its next scores are
// issued by halves of 64 keys, each as soon as the product with P has read that half, and the softmax starts on the first (this and the two issuing
// warps: 2 prompts of 2,048 tokens 344 -> 300 us).
//
// What holds it back. Prompts: no unit is full (53 % of the issue slots, 46 % of the tensor pipe, 41 % of the ALU, 23 % of the
// exponentials); the roles wait for one another, the longest of them the softmax, one thread a row. At 128 keys a row and block its 128
// exponentials, as many differences, products, maxima, additions and half as many packings are some 650 issue slots of a warp; eight
// such warps and the eight that unpack share four schedulers. 2 x 2048 tokens on 4,100 and 6,200 keys, 32 query heads on 8: 303 us,
// 1.01 PFLOP/s, 53 % of the measured rate of large matrix products; 64 channels 227 us. Two threads a row (half the chain, but a
// trade of maxima and sums through shared memory for every block) and blocks of 64 keys (twice the barriers) were slower. For a few
// tokens a sequence (8 x 17, 31 MB: 30 us) what a CTA does once (tensor memory, query rows, the first blocks, its part for the joining)
// and the chain through one block: copy, unpack, QK, softmax, PV.
//
// Shared memory holds operands in rows of 128 bytes (64 f16), 8 rows to an atom of 1024 bytes, 16-byte chunks swizzled by the row.
// Channels 16 b + 8 s .. + 7 of a query row or key lie in chunk 4 s + b % 4 of the row, not 2 b + s: a warp's stores of a block's keys
// (8 bytes a lane, 4 lanes a key) then meet every bank once. Values lie with their channels as rows; row 16 b + i holds channel
// 16 b + 2 i for i < 8 and 16 b + 2 (i - 8) + 1 above, as the lanes have them.
#include "kv_schedule.cuh"

#include <algorithm>
#include <climits>
#include <type_traits>

namespace whead_kv_impl {

namespace {

constexpr int kBlock = 128;      // keys
constexpr float kBias = 7.0f;    // as in kv_attend.cu
constexpr float kSlack = 15.0f;

template <int D, int TILES>
struct Shape {
  static constexpr int kRows = 128 * TILES;
  static constexpr int kSBufs = 2 / TILES;               // score buffers of a tile
  static constexpr int kBufs = 2;                        // key and value tiles
  static constexpr int kSoft = 4 * TILES;                // softmax warps, then those that unpack, then two a tile that issue: QK, PV
  static constexpr int kUnpack = 8;                      // a group of each block to each
  static constexpr int kIssue = kSoft + kUnpack;
  static constexpr int kThreads = (kIssue + 2 * TILES) * 32;
  static constexpr int kGroup = 18 * D;
  static constexpr int kQ = 128 * D * 2, kK = kBlock * D * 2, kV = D * kBlock * 2;
  static constexpr int kOffWalk = 640;                   // the warps' places
  static constexpr int kOffQ = 3072, kOffK = kOffQ + TILES * kQ, kOffV = kOffK + kBufs * kK;
  static constexpr int kBytes = kOffV + kBufs * kV + 1024;  // + alignment
  static constexpr int kCols = 512;                         // of tensor memory: two S, then O of each tile
};

struct Head {
  SchedShared sched;
  unsigned long long k_full[2], k_free[2], v_full[2], v_free[2], s_full[4], p_full[4], pv_done[4], o_full[2], q_full[2], drain[4];
  uint32_t tmem;
};

__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
  // rows of 128 bytes, atoms of 8 rows 1024 bytes apart, 128-byte swizzle
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) | ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}

// Issued by the lane whose `leader` is not zero. The rest of the warp runs along, so that addresses and descriptors stay in uniform
// registers: under a branch for one lane, each product took a dozen moves and the issuing warp was the bottleneck.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add, uint32_t leader) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
               ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add, uint32_t leader) {
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader) : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar, uint32_t leader) {
  asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n"
               ::"r"(bar), "r"(leader) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16 columns of this warp's lanes; the registers are operands of the wait, so that no use of them moves before it
__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t (&x)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]),
                 "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]) : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_load(uint32_t (&x)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]), "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]),
                 "+r"(x[10]), "+r"(x[11]), "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15]) :: "memory");
}
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
               ::"r"(addr), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
                 "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]) : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// two fp32 operations in one instruction
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}\n"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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

// The largest of a row's 64 scores, of those whose bits are set where MASKED (a code of its own: the bits cost more than the rest).
template <bool MASKED>
__device__ __forceinline__ float row_max(uint32_t st, const uint32_t (&seen)[2]) {
  float a0 = -INFINITY, a1 = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x[16];
    tmem_load16(st + i * 16, x);
    tmem_wait_load(x);
    if (MASKED) {
#pragma unroll
      for (int k = 0; k < 16; ++k) a0 = fmaxf(a0, (seen[i / 2] >> (i % 2 * 16 + k)) & 1 ? __uint_as_float(x[k]) : -INFINITY);
      __syncwarp();
    } else {
#pragma unroll
      for (int k = 0; k < 16; k += 4) {
        a0 = max3(a0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
        a1 = max3(a1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
      }
    }
  }
  return fmaxf(a0, a1);
}

// p = 2^((x - ref) f) of a row's products x, as f16 pairs, their sum, and the largest x: one pass, on the guess that the reference still
// does. The reference is a product, or near one, and is taken off before the factor comes: the difference of x and itself is zero,
// however large the scores are. (2^(x f - m) in one multiply-add is off by the rounding of m = ref f: for scores past 2^24 p would be any
// power of two, or infinite. 2 prompts of 2,048 tokens took 300 us so and take 303, with a window of 1,024 135 and 141, with 64 channels
// 222 and 227.)
template <bool MASKED>
__device__ __forceinline__ float row_exp(uint32_t st, const uint32_t (&seen)[2], float f, float ref, float2& sum, uint32_t (&p)[2][16]) {
  const float2 f2 = make_float2(f, f), off = make_float2(-ref, -ref);
  float2 s0 = make_float2(0.f, 0.f), s1 = s0;
  float t0 = -INFINITY, t1 = -INFINITY;
  uint32_t ahead[2][16];
  tmem_load16(st, ahead[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 16 columns at a time: registers are short, and what spills misses the small L1
    uint32_t (&x)[16] = ahead[i & 1];
    tmem_wait_load(x);
    if (i < 3) tmem_load16(st + i * 16 + 16, ahead[(i + 1) & 1]);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float2 d = make_float2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
      if (MASKED) {
        d.x = (seen[i / 2] >> (i % 2 * 16 + 2 * k)) & 1 ? d.x : -INFINITY;
        d.y = (seen[i / 2] >> (i % 2 * 16 + 2 * k + 1)) & 1 ? d.y : -INFINITY;
      }
      if (k & 1) t1 = max3(t1, d.x, d.y);
      else t0 = max3(t0, d.x, d.y);
      d = mul2(add2(d, off), f2);
      d.x = ex2(d.x);
      d.y = ex2(d.y);
      if (k & 1) s1 = add2(s1, d);
      else s0 = add2(s0, d);
      p[i / 2][i % 2 * 8 + k] = pack16(d.x, d.y, WHEAD_KV_F16);
    }
    if (MASKED) __syncwarp();
  }
  sum = add2(s0, s1);
  return fmaxf(t0, t1);
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

// A CTA's way through its range. Every warp walks it for itself and keeps its place in shared memory, not in registers: those are
// short here, and what spills is read back from L2 (shared memory takes nearly all of L1).
struct Walk {
  long long cur, end, item_at;
  int next_item;
  Segment sg;
};

// The next segment, by a whole warp; false at the end.
template <int ROWS>
__device__ __forceinline__ bool next_segment(const Cache& c, const AttendArgs& a, Walk& w, const SchedShared& sched) {
  const long long cur = w.cur, end = w.end;
  if (cur >= end) return false;
  int item = w.next_item;
  Segment s;
  if (item == sched.item && sched.has_tile) {
    s.tile = sched.tile;
  } else {
    while (true) {
      s.tile = make_tile<kBlock>(c, a, item, ROWS);
      if (s.tile.units > 0) break;
      ++item;
    }
  }
  s.item = item;
  const long long item_at = w.item_at;
  const int past = (int)(cur - item_at), each = s.tile.units + kLead;
  s.h = past / each;
  s.head_at = item_at + (long long)s.h * each;
  const long long next = cut_segment(s, cur, end);
  if (s.u1 == s.u0) return false;  // a range may end inside a lead
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    w.sg = s;
    w.cur = next;
    const bool done = s.u1 == s.tile.units && s.h == c.kv_heads - 1;
    w.next_item = done ? item + 1 : item;
    if (done) w.item_at = next;
  }
  __syncwarp();
  return true;
}

static_assert(sizeof(Head) <= 640 && 640 + 20 * sizeof(Walk) <= 3072, "");

// A whole warp's wait. One that has run out is reported once; the warp then goes on without waiting, on whatever is there, to its end.
__device__ __forceinline__ void await(const Cache& c, uint32_t bar, uint32_t parity, bool& dead) {
  while (!dead && !__all_sync(~0u, mbar_try(bar, parity))) {
    if (!__all_sync(~0u, mbar_wait(bar, parity))) {
      set_status(c, WHEAD_ERR_TIMEOUT);
      dead = true;
    }
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
__global__ void __launch_bounds__((Shape<D, TILES>::kThreads), 1) attend_tiles(const __grid_constant__ Cache c, const __grid_constant__ AttendArgs a) {
  after_previous();
  using S = Shape<D, TILES>;
  constexpr int NB = D / 16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  Head& s = *reinterpret_cast<Head*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(~0u, tid >> 5, 0);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.k_full[i]), S::kUnpack);
      mbar_init(smem_u32(&s.k_free[i]), TILES);
      mbar_init(smem_u32(&s.v_full[i]), S::kUnpack);
      mbar_init(smem_u32(&s.v_free[i]), TILES);
      for (int h = 0; h < 2; ++h) {
        mbar_init(smem_u32(&s.s_full[2 * i + h]), 1);
        mbar_init(smem_u32(&s.p_full[2 * i + h]), 4);
        mbar_init(smem_u32(&s.pv_done[2 * i + h]), 1);
      }
      mbar_init(smem_u32(&s.o_full[i]), 1);
      mbar_init(smem_u32(&s.q_full[i]), 4);
      mbar_init(smem_u32(&s.drain[2 * i]), 1);
      mbar_init(smem_u32(&s.drain[2 * i + 1]), 1);
    }
    fence_mbar_init();
  }
  const Start start = get_start<S::kThreads, kBlock>(c, a, S::kRows, s.sched);
  if ((int)blockIdx.x >= start.ctas) {
    if (tid == 0) put_record(c, 0, 0, 0, 0);
    return;
  }
  if (warp == S::kIssue) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s.tmem)), "n"(S::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = __shfl_sync(~0u, s.tmem, 0);
  Walk& walk = reinterpret_cast<Walk*>(smem + S::kOffWalk)[warp];
  if (lane == 0) {
    walk.cur = range_begin(start, blockIdx.x);
    walk.end = range_begin(start, blockIdx.x + 1);
    walk.item_at = start.at;
    walk.sg.u0 = walk.sg.u1 = 0;
    walk.sg.tile.units = 0;
    walk.next_item = start.item;
  }
  __syncwarp();
  const Segment& sg = walk.sg;
  bool dead = false;

  if (warp >= S::kIssue) {
    // ---- a tile's products: QK by one warp, PV by another (each spends as long on its barriers and commits as on the products). With
    // two tiles there is one score buffer a tile: QK goes by half blocks, each as soon as the P there before has been taken, under the
    // other half's softmax. With one tile, whose next scores have a buffer of their own, whole blocks cost less: a product of 64 keys takes
    // 60 cycles, one of 128 keys 64 (two tiles, prompt chunk: 299 us by halves, 344 by blocks; one tile, 8 x 17 tokens: 34.8, 32.7).
    constexpr int kKeys = kBlock / TILES, kPieces = kBlock / kKeys;  // of a QK product
    constexpr uint32_t kQK = (1u << 4) | ((kKeys / 8u) << 17) | ((128u / 16u) << 24);  // fp32 from f16 x f16, both along k
    constexpr uint32_t kPV = (1u << 4) | ((D / 8u) << 17) | ((128u / 16u) << 24);
    const int t = (warp - S::kIssue) % TILES;
    const uint32_t leader = lane == 0;
    const uint64_t dq = tile_desc(smem_u32(smem + S::kOffQ) + t * S::kQ), dk = tile_desc(smem_u32(smem + S::kOffK)), dv = tile_desc(smem_u32(smem + S::kOffV));
    const uint32_t s_col = tmem + t * S::kSBufs * kBlock, o_col = tmem + 256 + t * 128;
    int n = 0, seg = 0;
    if (warp < S::kIssue + TILES) {
      while (next_segment<S::kRows>(c, a, walk, s.sched)) {
        const int last = n + __shfl_sync(~0u, sg.u1 - sg.u0, 0);
        await(c, smem_u32(&s.q_full[t]), seg & 1, dead);
#pragma unroll 1
        for (; n < last; ++n) {
          const int buf = n % S::kBufs, sb = n % S::kSBufs, half0 = (t * S::kSBufs + sb) * 2;
          await(c, smem_u32(&s.k_full[buf]), n / S::kBufs & 1, dead);
          const uint64_t db = dk + (uint64_t)(buf * (S::kK >> 4));
#pragma unroll
          for (int h = 0; h < kPieces; ++h) {
            if (n >= S::kSBufs) await(c, smem_u32(&s.pv_done[half0 + 2 / kPieces * (h + 1) - 1]), (n / S::kSBufs - 1) & 1, dead);
            fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_ss(s_col + sb * kBlock + h * 64, dq + (k / 4 * (128 * 128) + k % 4 * 32) / 16, db + (h * 64 * 128 + k / 4 * (kBlock * 128) + k % 4 * 32) / 16, kQK, k > 0, leader);
            commit(smem_u32(&s.s_full[half0 + h]), leader);
            if (kPieces == 1) commit(smem_u32(&s.s_full[half0 + 1]), leader);
          }
          commit(smem_u32(&s.k_free[buf]), leader);
        }
        ++seg;
      }
    } else {
      while (next_segment<S::kRows>(c, a, walk, s.sched)) {
        const int first = n, last = n + __shfl_sync(~0u, sg.u1 - sg.u0, 0);
#pragma unroll 1
        for (; n < last; ++n) {
          const int buf = n % S::kBufs, sb = n % S::kSBufs, half0 = (t * S::kSBufs + sb) * 2;
          await(c, smem_u32(&s.v_full[buf]), n / S::kBufs & 1, dead);
          const uint64_t db = dv + (uint64_t)(buf * (S::kV >> 4));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            await(c, smem_u32(&s.p_full[half0 + h]), n / S::kSBufs & 1, dead);
            fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(o_col, s_col + sb * kBlock + h * 64 + k * 8, db + (h * (D * 128) + k * 32) / 16, kPV, n > first || h + k > 0, leader);
            commit(smem_u32(&s.pv_done[half0 + h]), leader);
          }
          commit(smem_u32(&s.v_free[buf]), leader);
        }
        commit(smem_u32(&s.o_full[t]), leader);
      }
    }
    // nothing may be under way when the CTA gives its tensor memory back
    __syncwarp();
    const uint32_t drain = smem_u32(&s.drain[warp - S::kIssue]);
    commit(drain, leader);
    mbar_wait(drain, 0);
    __syncwarp();
  } else if (warp >= S::kSoft) {
    // ---- codes to f16 tiles: group w of each block
    const int w = warp - S::kSoft, g = lane >> 2, t = lane & 3;
    const int64_t page_bytes = (int64_t)c.kv_heads * (c.page_size >> 4) * S::kGroup;
    int n = 0;
    while (next_segment<S::kRows>(c, a, walk, s.sched)) {
      const int32_t* table = c.tables + (int64_t)sg.tile.slot * c.max_pages;
      const uint8_t* base = c.pool + (int64_t)sg.h * (c.page_size >> 4) * S::kGroup;
      const int len = sg.tile.len, stop = min((sg.tile.unit0 + sg.u1) * kBlock, len);
      // codes come one block ahead of the tiles, the numbers of their pages two
      RawK<D> rk;
      RawV<D> rv;
      int page;
      auto look = [&](int u) {
        const int key = u * kBlock + w * 16;
        page = key < stop ? __ldg(table + (key >> c.page_shift)) : 0;
      };
      auto group_at = [&](int key) -> const uint8_t* {
        if ((unsigned)page >= (unsigned)c.num_pages) {
          set_status(c, WHEAD_ERR_INTERNAL);
          page = 0;
        }
        return base + page * page_bytes + ((key & (c.page_size - 1)) >> 4) * S::kGroup;
      };
      auto fetch_k = [&](int u) {
        const int key = u * kBlock + w * 16;
        if (key >= stop) return;
        const uint8_t* gp = group_at(key);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          rk.code[j] = __ldg(reinterpret_cast<const uint4*>(gp + j * 512) + lane);
          rk.scale[j] = __ldg(reinterpret_cast<const uint2*>(gp + 8 * D + g * 2 * NB) + j);
        }
      };
      auto fetch_v = [&](int u) {
        const int key = u * kBlock + w * 16;
        if (key >= stop) return;
        const uint8_t* gp = group_at(key);
#pragma unroll
        for (int j = 0; j < D / 64; ++j) {
          rv.code[j] = __ldg(reinterpret_cast<const uint4*>(gp + 9 * D + j * 512) + lane);
          rv.scale[j] = __ldg(reinterpret_cast<const uint4*>(gp + 17 * D + t * 4 * NB) + j);
        }
      };
      const int end = sg.tile.unit0 + sg.u1;
      int u = sg.tile.unit0 + sg.u0;
      look(u);
      fetch_k(u);
      fetch_v(u);
      look(u + 1);
      for (; u < end; ++u, ++n) {
        const int buf = n % S::kBufs, key0 = u * kBlock + w * 16;
        const uint32_t used = (n / S::kBufs - 1) & 1;
        if (n >= S::kBufs) await(c, smem_u32(&s.k_free[buf]), used, dead);
        if (key0 < len) {
          uint8_t* to = smem + S::kOffK + buf * S::kK + w * 2048 + g * 128 + (t & 1) * 8;
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint4 kw = rk.code[b / 4];
            uint32_t x[4], s0, s1;
            e2m1x8_to_half2(b % 4 == 0 ? kw.x : b % 4 == 1 ? kw.y : b % 4 == 2 ? kw.z : kw.w, x);
            e4m3x4_to_half2(b % 4 < 2 ? rk.scale[b / 4].x : rk.scale[b / 4].y, s0, s1);
            const uint32_t sc = b & 1 ? s1 : s0;
            uint8_t* at = to + b / 4 * (kBlock * 128) + ((((t >> 1) * 4 + b % 4) ^ g) << 4);
            *reinterpret_cast<uint2*>(at) = make_uint2(hmul2_low(x[0], sc), hmul2_low(x[2], sc));
            *reinterpret_cast<uint2*>(at + 1024) = make_uint2(hmul2_high(x[1], sc), hmul2_high(x[3], sc));
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.k_full[buf]));
        fetch_k(u + 1);
        if (n >= S::kBufs) await(c, smem_u32(&s.v_free[buf]), used, dead);
        // what lies past the length may be anything: it becomes zero, so that 0 x NaN does not arise
        uint32_t live = ~0u;
        if (key0 + 16 > len) {
          live = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (key0 + 2 * t + (i & 1) + (i >> 1) * 8 < len) live |= 0xFFu << (8 * i);
          __syncwarp();
        }
        uint8_t* to = smem + S::kOffV + buf * S::kV + w / 4 * (D * 128) + g * 128 + t * 4;
        const int c0 = ((w % 4 * 2) ^ g) << 4, c1 = ((w % 4 * 2 + 1) ^ g) << 4;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint4 vw = rv.code[b / 4], vs = rv.scale[b / 4];
          uint32_t x[4], s0, s1;
          e2m1x8_to_half2(b % 4 == 0 ? vw.x : b % 4 == 1 ? vw.y : b % 4 == 2 ? vw.z : vw.w, x);
          e4m3x4_to_half2((b % 4 == 0 ? vs.x : b % 4 == 1 ? vs.y : b % 4 == 2 ? vs.z : vs.w) & live, s0, s1);
          uint8_t* at = to + b * 2048;
          *reinterpret_cast<uint32_t*>(at + c0) = hmul2(x[0], s0);
          *reinterpret_cast<uint32_t*>(at + 1024 + c0) = hmul2(x[1], s0);
          *reinterpret_cast<uint32_t*>(at + c1) = hmul2(x[2], s1);
          *reinterpret_cast<uint32_t*>(at + 1024 + c1) = hmul2(x[3], s1);
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
    const int t = warp >> 2, quarter = warp & 3, sub = t * 128;
    const int r = sub + quarter * 32 + lane;           // row of the CTA's tile
    const uint32_t lanes = (uint32_t)quarter << 21;    // this warp's lanes of tensor memory (lane 32 w at bit 16)
    const uint32_t ot = tmem + 256 + t * 128 + lanes;
    int n = 0, seg = 0;
    while (next_segment<S::kRows>(c, a, walk, s.sched)) {
      const Tile& tile = sg.tile;
      const bool idle = quarter * 32 + sub >= tile.rows;  // no row of this warp is one: its part of P may be anything
      float f;
      {
        // The thread's query row, from a power of two to f16. All of its loads are under way before it looks at one. (Rows fetched by bulk
        // or asynchronous copies took 4,500 cycles to ask for: those are issued lane by lane.) The sign of the scale goes into the
        // row, so that f is positive and scores need it only after their maximum is known.
        const float k_scale = c.k_scale[sg.h];
        const int row = tile.row0 + r, tok = row_token(a, row);
        uint4 x[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < tile.rows) {
          const uint16_t* src = static_cast<const uint16_t*>(a.q) + (long long)(tile.first + tok) * a.q_token_stride + (long long)(sg.h * a.group + row - tok * a.group) * a.q_head_stride;
          if (a.wide_q16) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) x[i] = __ldg(reinterpret_cast<const uint4*>(src) + i);
          } else {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              const uint2 lo = load_four(src, i * 8, a.wide_q), hi = load_four(src, i * 8 + 4, a.wide_q);
              x[i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
          }
        }
        // the largest magnitude, by its bits: they are ordered like the values
        uint32_t big = 0, also = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          big = __vmaxu2(big, __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu));
          also = __vmaxu2(also, __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
        }
        big = __vmaxu2(big, also);
        big = max(big & 0xFFFFu, big >> 16);
        // 2^e <= largest < 2^(e + 1), from -100 up, as in kv_attend.cu; the row's power of two first: it may be what the scale takes back
        const int e = max(a.dtype == WHEAD_KV_BF16 ? (int)(big >> 7) - 127 : max((int)(big >> 10), 1) - 15, -100);
        const float factor = __uint_as_float((uint32_t)(127 - 13 + e) << 23) * a.scale * k_scale * kLog2e;
        const float up = copysignf(__uint_as_float((uint32_t)(127 + 13 - e) << 23), factor);
        f = fmaxf(fabsf(factor), 1e-30f);  // positive: products stay below 2^34, so that scores of less are zero all the same
        uint8_t* to = smem + S::kOffQ + t * S::kQ + (quarter * 32 + lane) * 128;
        auto put = [&](auto bf16) {
          constexpr int kType = decltype(bf16)::value ? WHEAD_KV_BF16 : WHEAD_KV_F16;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {  // 8 channels: block i / 2, half i % 2
            uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = unpack16(w[k], kType);
              w[k] = pack16(y.x * up, y.y * up, WHEAD_KV_F16);
            }
            *reinterpret_cast<uint4*>(to + i / 8 * (128 * 128) + (((i % 2 * 4 + i / 2 % 4) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        };
        if (a.dtype == WHEAD_KV_BF16) put(std::true_type{});
        else put(std::false_type{});
        fence_async();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.q_full[t]));
      }
      int free_lo, free_hi;  // keys that all rows of the tile see
      {
        const int w0 = row_token(a, tile.row0 + sub), w1 = row_token(a, tile.row0 + max(min(sub + 128, tile.rows), sub + 1) - 1), past = tile.len - tile.tokens;
        const int hi = a.tree ? min(past, past + w0 + 1) : a.causal ? min(past + w0 + 1, tile.len) : tile.len;
        const int lo = a.window ? window_begin(a, past + w1) : 0;
        free_hi = hi;
        free_lo = lo;
      }
      bool fresh = true;  // some row of the warp has no reference yet
      float ref = kNoKey;  // in units of the products; m = ref f
      const float bias = __fdividef(kBias, f);
      float2 l = make_float2(0.f, 0.f);
      for (int u = sg.u0; u < sg.u1; ++u, ++n) {
        const int key0 = (tile.unit0 + u) * kBlock;
        // these barriers belong to the half of the score buffer: with one of each a tile, two blocks' scores could be turned into
        // P before the issuing warp has looked for the first, and it would miss that phase
        const int sb = t * S::kSBufs + n % S::kSBufs;
        // half a block at a time, each with its own P over its own scores: the first half's products run under the second's softmax
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          await(c, smem_u32(&s.s_full[2 * sb + h]), n / S::kSBufs & 1, dead);
          fence_after();
          if (idle) {
            fence_before();
            if (lane == 0) mbar_arrive(smem_u32(&s.p_full[2 * sb + h]));
            continue;
          }
          const uint32_t st = tmem + sb * kBlock + h * 64 + lanes;
          const int key = key0 + h * 64;
          const bool masked = key < free_lo || key + 64 > free_hi;
          uint32_t seen[2] = {~0u, ~0u};
          if (masked) {
            const RowView view = row_view(a, tile, tile.row0 + r);
            seen[0] = sees32(a, view, key);
            seen[1] = sees32(a, view, key + 32);
            __syncwarp();
          }
          if (fresh) {  // a row's first keys: its reference is their maximum
            const float top = masked ? row_max<true>(st, seen) : row_max<false>(st, seen);
            if (ref == kNoKey && top > kNoKey) ref = top - bias;
            fresh = __any_sync(~0u, ref == kNoKey);
          }
          uint32_t p[2][16];
          float2 sum;
          const float top = masked ? row_exp<true>(st, seen, f, ref, sum, p) : row_exp<false>(st, seen, f, ref, sum, p);
          const bool over = (top - ref) * f > kSlack;
          if (__any_sync(~0u, over)) {  // some p came out too large: the reference goes up, what there is comes down, once more
            const float now = over ? top - bias : ref, rr = over ? ex2((ref - now) * f) : 1.0f;
            ref = now;
            l.x *= rr;
            l.y *= rr;
            if (u > sg.u0 || h > 0) {  // after the products of the half before
              const int nb = h ? n : n - 1;
              await(c, smem_u32(&s.pv_done[(t * S::kSBufs + nb % S::kSBufs) * 2 + (h ^ 1)]), nb / S::kSBufs & 1, dead);
              fence_after();
#pragma unroll 1
              for (int i = 0; i < D / 16; ++i) {
                uint32_t x[16];
                tmem_load16(ot + i * 16, x);
                tmem_wait_load(x);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __float_as_uint(__uint_as_float(x[k]) * rr);
                tmem_store16(ot + i * 16, x);
              }
            }
            masked ? row_exp<true>(st, seen, f, ref, sum, p) : row_exp<false>(st, seen, f, ref, sum, p);
          }
          l = add2(l, sum);
          tmem_store16(st, p[0]);  // over the scores
          tmem_store16(st + 16, p[1]);
          tmem_wait_store();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.p_full[2 * sb + h]));
        }
      }
      await(c, smem_u32(&s.o_full[t]), seg & 1, dead);
      ++seg;
      fence_after();
      const int row = tile.row0 + r;
      const bool live = r < tile.rows;
      const int tok = row_token(a, row), head = sg.h * a.group + row - tok * a.group;
      const bool whole = sg.u0 == 0 && sg.u1 == tile.units;
      const float m = __fmul_rn(ref, f);
      // a part's m is rounded: what that took from it goes into its sums, up to what they bear (past that the reference is the score of
      // one of the keys, and every part's the same for the same score)
      const float back = whole ? 1.0f : ex2(fminf(fmaxf(__fmaf_rn(ref, f, -m), -16.0f), 16.0f));
      const float ll = (l.x + l.y) * back;
      constexpr int kPart = S::kRows * (D + 2);
      const int64_t out_row = (int64_t)(tile.first + tok) * a.heads + head;
      const float gv = c.v_scale[sg.h];
      float* part = c.partial + (int64_t)part_slot(start, sg, blockIdx.x) * kPart;
      const float scale = whole ? (ll != 0.0f ? gv / ll : 0.0f) : back;
#pragma unroll 1
      for (int i = 0; i < D / 16; ++i) {
        uint32_t x[16];
        tmem_load16(ot + i * 16, x);
        tmem_wait_load(x);
        if (live) {  // 16 channels: columns k and 8 + k are channels 2k and 2k + 1
          float y[16];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[2 * k] = __uint_as_float(x[k]) * scale;
            y[2 * k + 1] = __uint_as_float(x[8 + k]) * scale;
          }
          if (whole) {
            if (ll == 0.0f) {
#pragma unroll
              for (int k = 0; k < 16; ++k) y[k] = 0.0f;
            }
            uint16_t* to = static_cast<uint16_t*>(a.out) + out_row * D + i * 16;
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              *reinterpret_cast<uint4*>(to + k) = make_uint4(pack16(y[k], y[k + 1], a.dtype), pack16(y[k + 2], y[k + 3], a.dtype),
                                                             pack16(y[k + 4], y[k + 5], a.dtype), pack16(y[k + 6], y[k + 7], a.dtype));
          } else {
            float* to = part + 2 * S::kRows + r * D + i * 16;
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
        __stcg(part + r, ll == 0.0f ? kNoKey : m);
        __stcg(part + S::kRows + r, ll);
      }
    }
    // what the joining kernel has to do for the item that begins in this CTA's range and ends outside it
    if (tid == 0) {
      const bool cut = sg.u0 == 0 && sg.u1 > 0 && sg.u1 < sg.tile.units;
      put_record(c, sg.item, sg.h, cut ? last_owner(start, sg) - (int)blockIdx.x + 1 : 0, cut ? part_slot(start, sg, blockIdx.x) : 0);
    }
  }
  // tensor memory goes back when every role is through with it
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == S::kIssue) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kCols) : "memory");
}

template <int D, int TILES>
int launch(const HostCache& h, AttendArgs a, int max_q) {
  using S = Shape<D, TILES>;
  static std::atomic<bool> granted[kMaxDevices];
  if (!grant_smem(attend_tiles<D, TILES>, S::kBytes, h, granted)) return WHEAD_ERR_CUDA;
  const int64_t tiles = ((int64_t)max_q * a.group + S::kRows - 1) / S::kRows;
  a.row_tiles = (int)tiles;
  int64_t ctas = std::min<int64_t>((int64_t)h.sms, kMaxCtas);
  ctas = std::min(ctas, h.c.partial_floats / (2 * S::kRows * (D + 2)));
  a.planned = tiles * a.n > 2 * S::kThreads;
  a.small = tiles * a.n * h.c.kv_heads * ((int64_t)h.c.max_pages * h.c.page_size / kBlock + 2 + kLead) < INT_MAX;
  int rc = WHEAD_OK;
  if (a.planned) rc = launch_after(attend_plan<kBlock>, dim3(1), 1024, 0, h.stream, h.c, a, S::kRows, (int)ctas);
  if (rc == WHEAD_OK) rc = launch_after(attend_tiles<D, TILES>, dim3((unsigned)ctas), S::kThreads, S::kBytes, h.stream, h.c, a);
  if (rc != WHEAD_OK) return rc;
  return launch_join<D, S::kRows, kBlock>(h, a, (int)ctas, max_q);
}

}  // namespace

int launch_tiles(const HostCache& h, const AttendArgs& a, int max_q) {
  // Two tiles share the unpacked keys where there are rows for both (64 sequences on 8,192 keys, 256 rows: 468 us, one tile a CTA 811); one
  // has its scores a block ahead (128 rows: 419 us, in a CTA for two 424; 16 on 4,096 keys 36 rows 62 and 67).
  const bool one = tile_rows(h.c.head_dim, (int64_t)max_q * a.group) == 128;
  if (h.c.head_dim == 64) return one ? launch<64, 1>(h, a, max_q) : launch<64, 2>(h, a, max_q);
  return one ? launch<128, 1>(h, a, max_q) : launch<128, 2>(h, a, max_q);
}

}  // namespace whead_kv_impl

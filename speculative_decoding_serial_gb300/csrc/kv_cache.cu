// kv_cache.cu — the 4-bit paged KV cache's host checks and the kernels that write and move it: append, read, compact, fork.
#include "kv_common.cuh"

#include <algorithm>
#include <climits>

namespace whead_kv_impl {

namespace {

struct Layout {
  int64_t seq_a, seq_b, region, fresh, rows, counters, starts, records, partial, total;
  int64_t floats;
};

Layout layout(const whead_kv& k, int sms) {
  Layout l{};
  int64_t at = 256;
  auto take = [&](int64_t bytes) { const int64_t r = at; at = align256(at + bytes); return r; };
  l.counters = take(4LL * kMaxCtas);
  l.seq_a = take(4LL * (k.max_seqs + 1));
  l.seq_b = take(4LL * (k.max_seqs + 1));
  l.region = take(4LL * k.max_seqs * 2 * kRegionPages);
  l.fresh = take(4LL * k.num_pages);
  l.rows = take(4LL * k.max_seqs * k.max_pages);
  l.starts = take(16LL * kMaxCtas);
  l.records = take(16LL * kMaxCtas);
  l.floats = partial_floats(k.head_dim, sms);
  l.partial = take(4LL * l.floats);
  l.total = at;
  return l;
}

int check_shape(const whead_kv& k) {
  if (k.page_size != 16 && k.page_size != 32 && k.page_size != 64 && k.page_size != 128) return WHEAD_ERR_UNSUPPORTED;
  if (k.head_dim != 64 && k.head_dim != 128 && k.head_dim != 256) return WHEAD_ERR_UNSUPPORTED;
  if (k.kv_heads < 1 || k.max_seqs < 1 || k.max_pages < 1 || k.num_pages < 1) return WHEAD_ERR_INVALID_ARG;
  if (k.kv_heads > 1024 || k.max_seqs > 4096) return WHEAD_ERR_UNSUPPORTED;
  // positions are ints, and the attention forms those of up to three blocks of 128 keys past a slot's end
  if ((int64_t)k.max_pages * k.page_size > INT_MAX - 1023 || (int64_t)k.max_seqs * k.max_pages >= INT_MAX) return WHEAD_ERR_UNSUPPORTED;
  return WHEAD_OK;
}

}  // namespace

int device_sms(int* device) {
  static std::atomic<int> cached[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  *device = dev;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

int host_cache(const whead_kv* kv, HostCache* out) {
  if (!kv) return WHEAD_ERR_INVALID_ARG;
  const int rc = check_shape(*kv);
  if (rc != WHEAD_OK) return rc;
  if (!kv->pool || !kv->lens || !kv->refs || !kv->tables || !kv->k_scale || !kv->v_scale || !kv->workspace)
    return WHEAD_ERR_INVALID_ARG;
  if (!aligned(kv->pool, 16) || !aligned(kv->workspace, 256) || !aligned(kv->lens, 4) || !aligned(kv->refs, 4) ||
      !aligned(kv->tables, 4) || !aligned(kv->k_scale, 4) || !aligned(kv->v_scale, 4))
    return WHEAD_ERR_INVALID_ARG;
  out->sms = device_sms(&out->device);
  if (out->sms < 1) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  const Layout l = layout(*kv, out->sms);
  if (kv->workspace_bytes < l.total) return WHEAD_ERR_INVALID_ARG;
  char* w = static_cast<char*>(kv->workspace);
  Cache& c = out->c;
  c.pool = static_cast<uint8_t*>(kv->pool);
  c.lens = kv->lens;
  c.refs = kv->refs;
  c.tables = kv->tables;
  c.k_scale = kv->k_scale;
  c.v_scale = kv->v_scale;
  c.page_size = kv->page_size;
  c.page_shift = kv->page_size == 16 ? 4 : kv->page_size == 32 ? 5 : kv->page_size == 64 ? 6 : 7;
  c.kv_heads = kv->kv_heads;
  c.head_dim = kv->head_dim;
  c.max_seqs = kv->max_seqs;
  c.max_pages = kv->max_pages;
  c.num_pages = kv->num_pages;
  c.ctl = reinterpret_cast<Ctl*>(w);
  c.seq_a = reinterpret_cast<int32_t*>(w + l.seq_a);
  c.seq_b = reinterpret_cast<int32_t*>(w + l.seq_b);
  c.region = reinterpret_cast<int32_t*>(w + l.region);
  c.fresh = reinterpret_cast<int32_t*>(w + l.fresh);
  c.rows = reinterpret_cast<int32_t*>(w + l.rows);
  c.counters = reinterpret_cast<unsigned*>(w + l.counters);
  c.starts = reinterpret_cast<int32_t*>(w + l.starts);
  c.records = reinterpret_cast<int32_t*>(w + l.records);
  c.partial = reinterpret_cast<float*>(w + l.partial);
  c.partial_floats = l.floats;
  out->stream = static_cast<cudaStream_t>(kv->stream);
  return WHEAD_OK;
}

namespace {

// ---------------------------------------------------------------- planning: one CTA of kPlan threads

constexpr int kPlan = 1024;

struct PlanShared {
  int warp[32];
  int carry;
  int found;
  int bad;
};

// Exclusive sum of x over the CTA's threads, and the total.
__device__ __forceinline__ int block_scan(int x, PlanShared& s, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(~0u, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) s.warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = lane < (int)(blockDim.x >> 5) ? s.warp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(~0u, w, o);
      if (lane >= o) w += y;
    }
    s.warp[lane] = w;
  }
  __syncthreads();
  total = s.warp[(blockDim.x >> 5) - 1];
  return v - x + (warp ? s.warp[warp - 1] : 0);
}

// The `need` free pages of lowest index into c.fresh; how many there are (at most need).
__device__ int find_free(const Cache& c, int need, PlanShared& s) {
  int have = 0;
  for (int base = 0; base < c.num_pages && have < need; base += kPlan * 4) {
    const int at = base + threadIdx.x * 4;
    int free[4], n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      free[k] = at + k < c.num_pages && c.refs[at + k] == 0;
      n += free[k];
    }
    int total;
    int rank = have + block_scan(n, s, total);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (free[k]) {
        if (rank < need) c.fresh[rank] = at + k;
        ++rank;
      }
    }
    have += total;
  }
  __syncthreads();
  return have < need ? have : need;
}

__device__ __forceinline__ int pages_of(const Cache& c, int len) { return (int)(((int64_t)len + c.page_size - 1) >> c.page_shift); }

// A planning kernel's verdict: on an error the call's later kernels do nothing.
__device__ __forceinline__ void verdict(const Cache& c, int code) {
  if (threadIdx.x == 0) {
    c.ctl->abort = code != 0;
    if (code) set_status(c, code);
  }
}

__device__ __forceinline__ int entry_slot(const int32_t* slots, int i) { return slots ? slots[i] : i; }

// ---------------------------------------------------------------- append

struct AppendArgs {
  const void* k;
  const void* v;
  int dtype;
  int64_t kt, kh, vt, vh;
  const int32_t* indptr;
  const int32_t* slots;
  int n;
  int64_t total;
  bool wide_k, wide_v;
};

// Where an entry's tokens are; a bad range or slot gives count -1.
__device__ __forceinline__ void append_entry(const Cache& c, const AppendArgs& a, int i, int& slot, int64_t& first, int& count) {
  slot = entry_slot(a.slots, i);
  int64_t end;
  if (a.indptr) {
    first = a.indptr[i];
    end = a.indptr[i + 1];
  } else {
    const int64_t each = a.total / a.n;
    first = each * i;
    end = first + each;
  }
  count = (unsigned)slot >= (unsigned)c.max_seqs || first < 0 || end < first || end > a.total ? -1 : (int)(end - first);
}

// One group that an append writes, as the writing kernel needs it: one load away, instead of a search and four dependent loads in every
// CTA (26,968 tokens of 8 heads of 128 channels: this and the scales worked out once took the writing from 109 to 47 us).
struct __align__(16) AppendGroup {
  int page;    // of the pool
  int place;   // of the group in the page, the first new token in bits 8.., the one past the last in bits 16..
  int64_t row; // of k, v: the group's first token
};

// The last of n ascending sums that is at most x.
__device__ __forceinline__ int find_sum(const int32_t* sums, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Lengths, pages and tables for an append, and the groups it writes; seq_a: each entry's length before, seq_b: sums of the groups it
// touches.
__global__ void __launch_bounds__(kPlan, 1) append_plan(Cache c, AppendArgs a) {
  after_previous();
  __shared__ PlanShared s;
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  int need = 0, groups = 0;
  for (int base = 0; base < a.n; base += kPlan) {
    const int i = base + threadIdx.x;
    int pages = 0, g = 0;
    if (i < a.n) {
      int slot, count;
      int64_t first;
      append_entry(c, a, i, slot, first, count);
      const int len = count < 0 ? 0 : c.lens[slot];
      const int64_t now = (int64_t)len + count;
      if (count < 0 || len < 0) {
        atomicMin(&s.bad, WHEAD_ERR_INVALID_ARG);
      } else if (now > (int64_t)c.max_pages * c.page_size) {
        atomicMin(&s.bad, WHEAD_ERR_NO_PAGES);
      } else {
        pages = pages_of(c, (int)now) - pages_of(c, len);
        g = count ? (int)(((now + 15) >> 4) - (len >> 4)) : 0;
      }
      c.seq_a[i] = len;
    }
    int total;
    const int at = block_scan(g, s, total);
    if (i < a.n) c.seq_b[i] = groups + at;
    groups += total;
    block_scan(pages, s, total);
    need += total;
  }
  if (threadIdx.x == 0) c.ctl->total = groups;
  __syncthreads();
  int bad = s.bad;
  if (!bad && need > 0 && find_free(c, need, s) < need) bad = WHEAD_ERR_NO_PAGES;
  verdict(c, bad);
  if (bad) return;
  int taken = 0;
  for (int base = 0; base < a.n; base += kPlan) {
    const int i = base + threadIdx.x;
    int slot = 0, count = 0, len = 0, had = 0, pages = 0;
    int64_t first;
    if (i < a.n) {
      append_entry(c, a, i, slot, first, count);
      len = c.seq_a[i];
      had = pages_of(c, len);
      pages = pages_of(c, len + count) - had;
      c.lens[slot] = len + count;
    }
    if (need > 0) {
      int total;
      const int at = taken + block_scan(pages, s, total);
      taken += total;
      // the entries' pages, a warp for each entry at a time
      const int lane = threadIdx.x & 31;
      for (unsigned left = __ballot_sync(~0u, pages > 0); left; left &= left - 1) {
        const int l = __ffs(left) - 1;
        const int p = __shfl_sync(~0u, pages, l), sl = __shfl_sync(~0u, slot, l), h = __shfl_sync(~0u, had, l), f = __shfl_sync(~0u, at, l);
#pragma unroll 4
        for (int j = lane; j < p; j += 32) {
          const int page = c.fresh[f + j];
          c.tables[(int64_t)sl * c.max_pages + h + j] = page;
          c.refs[page] = 1;
        }
      }
    }
  }
  __syncthreads();
  AppendGroup* to = reinterpret_cast<AppendGroup*>(c.partial);
  for (int x = threadIdx.x; x < groups; x += kPlan) {
    const int i = find_sum(c.seq_b, a.n, x);  // entries without groups share their sum with the next one: the last of them holds x
    int slot, count;
    int64_t first;
    append_entry(c, a, i, slot, first, count);
    const int len = c.seq_a[i];
    const int pos0 = ((len >> 4) + (x - c.seq_b[i])) << 4;
    AppendGroup g;
    g.page = c.tables[(int64_t)slot * c.max_pages + (pos0 >> c.page_shift)];
    g.place = ((pos0 & (c.page_size - 1)) >> 4) | max(len - pos0, 0) << 8 | min(len + count - pos0, 16) << 16;
    g.row = first + pos0 - len;
    to[x] = g;
  }
}

// One block of 16 channels' scale byte and the factor 1 / (s g) that its codes are formed with. The maximum passes over a NaN beside
// numbers; of nothing but NaN it is one, and counts as zero: a NaN scale would reach every row whose masks hide the token.
__device__ __forceinline__ uint32_t block_scale(float amax, float g, float& inv) {
  const float r = __fdiv_rn(fmaxf(amax, 0.0f), __fmul_rn(6.0f, g));
  const uint32_t byte = __nv_cvt_float_to_fp8(r, __NV_SATFINITE, __NV_E4M3);
  inv = __frcp_rn(__fmul_rn(e4m3_to_float((uint8_t)byte), g));
  return byte;
}

__device__ __forceinline__ float scaled(float x, float inv) {
  const float y = __fmul_rn(x, inv);
  return y == y ? y : 0.0f;
}

// Largest of N values over the lanes that differ in the bits BIT, BIT / 2, .. (log2(N / 2) of them); each lane ends with two of the
// N: those of its number in these bits, the first of them in x[0].
template <int N, int BIT>
__device__ __forceinline__ void max_scatter(float (&x)[N]) {
  if constexpr (N > 2) {
    const bool up = (threadIdx.x & BIT) != 0;
    float half[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const float send = up ? x[i] : x[N / 2 + i];
      half[i] = fmaxf(up ? x[N / 2 + i] : x[i], __shfl_xor_sync(~0u, send, BIT));
    }
    max_scatter<N / 2, BIT / 2>(half);
    x[0] = half[0];
    x[1] = half[1];
  }
}

// A warp quantizes 64 channels of the keys, or of the values, of the new tokens of one group of one head; a CTA has all of the
// group's. Its loads are all under way before the first is used (one loop over the blocks took 27 us for a single token: its stores kept
// the next block's loads back). A group's owner is the only writer of its words, so the codes of two tokens that share a byte
// do not race; what an owner does not write of a word it reads first. Bound by latency for single tokens. Prompts: 26,968
// tokens, 8 heads of 128 channels, 141.5 MB of inputs and groups in 47 us, 3.0 TB/s, 45 % of the measured copy rate: a short CTA a
// group and head loads, works and stores in turn, and what others have under way does not fill the gaps.
template <int D, int DTYPE>
__global__ void __launch_bounds__(D) append_write(const __grid_constant__ Cache c, const __grid_constant__ AppendArgs a) {
  constexpr int NB = D / 16;
  after_previous();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, chunk = part >> 1;  // 64 channels; even parts: keys
  if (c.ctl->abort) return;
  const int total = c.ctl->total;
  for (int x = blockIdx.x; x < total; x += gridDim.x) {
    const int4 what = __ldcg(reinterpret_cast<const int4*>(c.partial) + x);  // an AppendGroup
    if (!is_page(c, what.x)) continue;                                       // a table that is not this cache's
    const int lo = what.y >> 8 & 0xFF, hi = what.y >> 16;                    // new tokens of the group: lo .. hi - 1
    const bool whole = lo == 0 && hi == 16;
    const int64_t row0 = (int64_t)((uint64_t)(uint32_t)what.z | (uint64_t)(uint32_t)what.w << 32);  // row of k, v of the group's first token
    if ((part & 1) == 0) {
      // this lane's tokens g and g + 8, four channels of each block
      const bool in0 = g >= lo && g < hi, in1 = g + 8 >= lo && g + 8 < hi;
      const int64_t ch = (int64_t)h * a.kh + chunk * 64 + t * 4;
      RawElems<DTYPE, 4> raw[4][2] = {};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (in0) load_raw(a.k, (row0 + g) * a.kt + ch + b * 16, a.wide_k, raw[b][0]);
        if (in1) load_raw(a.k, (row0 + g + 8) * a.kt + ch + b * 16, a.wide_k, raw[b][1]);
      }
      uint8_t* gp = group_ptr<D>(c, what.x, h, (what.y & 0xFF) << 4);
      uint4* codes = reinterpret_cast<uint4*>(gp + chunk * 512) + lane;
      uint16_t* scales = reinterpret_cast<uint16_t*>(gp + 8 * D + g * 2 * NB + chunk * 8) + t;  // of block t: tokens g, g + 8
      uint4 old = make_uint4(0, 0, 0, 0);
      if (!whole) old = *codes;
      const float gk = c.k_scale[h];
      // the four lanes of a token share its blocks' scales: lane t works out block t's, for tokens g and g + 8
      float v[4][2][4], top[8], inv[2];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        raw_values(raw[i / 2][i % 2], v[i / 2][i % 2]);
        const float (&x)[4] = v[i / 2][i % 2];
        top[i] = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
      }
      max_scatter<8, 2>(top);
      const uint32_t s0 = block_scale(top[0], gk, inv[0]), s1 = block_scale(top[1], gk, inv[1]);
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float i0 = __shfl_sync(~0u, inv[0], g * 4 + b), i1 = __shfl_sync(~0u, inv[1], g * 4 + b);
        w[b] = e2m1x2_from_float(scaled(v[b][0][0], i0), scaled(v[b][0][1], i0)) |
               e2m1x2_from_float(scaled(v[b][1][0], i1), scaled(v[b][1][1], i1)) << 8 |
               e2m1x2_from_float(scaled(v[b][0][2], i0), scaled(v[b][0][3], i0)) << 16 |
               e2m1x2_from_float(scaled(v[b][1][2], i1), scaled(v[b][1][3], i1)) << 24;
      }
      const uint32_t mine = (in0 ? 0x00FF00FFu : 0u) | (in1 ? 0xFF00FF00u : 0u);
      *codes = make_uint4((w[0] & mine) | (old.x & ~mine), (w[1] & mine) | (old.y & ~mine), (w[2] & mine) | (old.z & ~mine), (w[3] & mine) | (old.w & ~mine));
      if (whole) {
        *scales = (uint16_t)(s0 | s1 << 8);
      } else {
        if (in0) reinterpret_cast<uint8_t*>(scales)[0] = (uint8_t)s0;
        if (in1) reinterpret_cast<uint8_t*>(scales)[1] = (uint8_t)s1;
      }
    } else {
      // this lane's tokens 2t, 2t + 1, 2t + 8, 2t + 9, two channels of each block
      bool in[4];
      uint32_t mine = 0;
      RawElems<DTYPE, 2> raw[4][4] = {};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = 2 * t + (k & 1) + (k >> 1) * 8;
        in[k] = r >= lo && r < hi;
        if (in[k]) {
          mine |= 0x0F0Fu << ((k & 1) * 4 + (k >> 1) * 16);
#pragma unroll
          for (int b = 0; b < 4; ++b) load_raw(a.v, (row0 + r) * a.vt + (int64_t)h * a.vh + chunk * 64 + b * 16 + g * 2, a.wide_v, raw[b][k]);
        }
      }
      uint8_t* gp = group_ptr<D>(c, what.x, h, (what.y & 0xFF) << 4);
      uint4* codes = reinterpret_cast<uint4*>(gp + 9 * D + chunk * 512) + lane;
      uint16_t* scales = reinterpret_cast<uint16_t*>(gp + 17 * D + t * 4 * NB + chunk * 16) + g;  // bytes 2g, 2g + 1 of [block][token]
      uint4 old = make_uint4(0, 0, 0, 0);
      if (!whole) old = *codes;
      const float gv = c.v_scale[h];
      // the eight lanes of a token pair share its 16 scales: lane g works out two, block g / 2's for tokens 2t + 8 (g % 2) and the one after
      float v[4][4][2], top[16], inv[2];
#pragma unroll
      for (int i = 0; i < 16; ++i) raw_values(raw[i / 4][i % 4], v[i / 4][i % 4]);
#pragma unroll
      for (int i = 0; i < 16; ++i) top[i] = fmaxf(fabsf(v[i / 4][i % 4][0]), fabsf(v[i / 4][i % 4][1]));
      max_scatter<16, 16>(top);
      const uint32_t s0 = block_scale(top[0], gv, inv[0]), s1 = block_scale(top[1], gv, inv[1]);
      uint32_t w[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        float i4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) i4[k] = __shfl_sync(~0u, inv[k & 1], (b * 2 + (k >> 1)) * 4 + t);
        w[b] = 0;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          w[b] |= e2m1x2_from_float(scaled(v[b][0][e], i4[0]), scaled(v[b][1][e], i4[1])) << (e * 8) |
                  e2m1x2_from_float(scaled(v[b][2][e], i4[2]), scaled(v[b][3][e], i4[3])) << (e * 8 + 16);
      }
      *codes = make_uint4((w[0] & mine) | (old.x & ~mine), (w[1] & mine) | (old.y & ~mine), (w[2] & mine) | (old.z & ~mine), (w[3] & mine) | (old.w & ~mine));
      if (whole) {
        *scales = (uint16_t)(s0 | s1 << 8);
      } else {
        const bool high = (g & 1) != 0;
        if (high ? in[2] : in[0]) reinterpret_cast<uint8_t*>(scales)[0] = (uint8_t)s0;
        if (high ? in[3] : in[1]) reinterpret_cast<uint8_t*>(scales)[1] = (uint8_t)s1;
      }
    }
  }
}

// ---------------------------------------------------------------- read

struct ReadArgs {
  const int32_t* start;
  const int32_t* slots;
  int n, count, dtype;
  void* k;
  void* v;
};

__device__ __forceinline__ void store4(void* p, int64_t i, int dtype, const float (&x)[4]) {
  if (dtype == WHEAD_KV_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x[0], x[1], x[2], x[3]);
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(pack16(x[0], x[1], dtype), pack16(x[2], x[3], dtype));
}
__device__ __forceinline__ void store2(void* p, int64_t i, int dtype, float x, float y) {
  if (dtype == WHEAD_KV_F32)
    *reinterpret_cast<float2*>(static_cast<float*>(p) + i) = make_float2(x, y);
  else
    *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p) + i) = pack16(x, y, dtype);
}

// A warp takes 64 channels of the keys, or of the values, of one group of one head apart and writes those of its tokens that are asked
// for; a CTA has all of a group. Bound by the bytes that it writes.
template <int D>
__global__ void __launch_bounds__(D) read_kernel(const __grid_constant__ Cache c, const __grid_constant__ ReadArgs a) {
  constexpr int NB = D / 16;
  after_previous();
  const int lane = threadIdx.x & 31, part = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int h = blockIdx.y, chunk = part >> 1;
  const int per = (a.count + 30) / 16;  // groups that `count` tokens can touch, whatever the first one's place
  const int i = (int)(blockIdx.x / (unsigned)per);
  const int slot = entry_slot(a.slots, i);
  int len = slot_len(c, slot);
  int start = a.start[i];
  if (start < 0) {
    set_status(c, WHEAD_ERR_INVALID_ARG);
    start = 0;
    len = 0;
  }
  const int64_t pos0 = ((int64_t)(start >> 4) + (blockIdx.x - (unsigned)i * per)) << 4;
  const int64_t end = (int64_t)start + a.count;
  if (pos0 >= end) return;
  const bool held = pos0 < len;
  const uint8_t* gp = held ? group_ptr<D>(c, c.tables[(int64_t)slot * c.max_pages + (pos0 >> c.page_shift)], h, (int)pos0) : nullptr;
  const int64_t out0 = ((int64_t)i * a.count + (pos0 - start)) * c.kv_heads + h;  // row of the group's first token
  if ((part & 1) == 0) {
    uint4 code = make_uint4(0, 0, 0, 0);
    uint2 scale = make_uint2(0, 0);
    if (held) {
      code = *(reinterpret_cast<const uint4*>(gp + chunk * 512) + lane);
      scale = *reinterpret_cast<const uint2*>(gp + 8 * D + g * 2 * NB + chunk * 8);
    }
    const float gk = c.k_scale[h];
#pragma unroll
    for (int hi = 0; hi < 2; ++hi) {
      const int64_t pos = pos0 + g + hi * 8;
      if (pos < start || pos >= end) continue;
      const bool live = pos < len;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t x[4];
        e2m1x8_to_half2(b == 0 ? code.x : b == 1 ? code.y : b == 2 ? code.z : code.w, x);
        const float s = __fmul_rn(e4m3_to_float((uint8_t)((b < 2 ? scale.x : scale.y) >> ((b % 2 * 2 + hi) * 8))), gk);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x[hi])), q = __half22float2(*reinterpret_cast<const __half2*>(&x[hi + 2]));
        const float y[4] = {live ? p.x * s : 0.0f, live ? p.y * s : 0.0f, live ? q.x * s : 0.0f, live ? q.y * s : 0.0f};
        store4(a.k, (out0 + (int64_t)(g + hi * 8) * c.kv_heads) * D + chunk * 64 + b * 16 + t * 4, a.dtype, y);
      }
    }
  } else {
    uint4 code = make_uint4(0, 0, 0, 0), scale = code;
    if (held) {
      code = *(reinterpret_cast<const uint4*>(gp + 9 * D + chunk * 512) + lane);
      scale = *reinterpret_cast<const uint4*>(gp + 17 * D + t * 4 * NB + chunk * 16);
    }
    const float gv = c.v_scale[h];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = 2 * t + (k & 1) + (k >> 1) * 8;
      const int64_t pos = pos0 + r;
      if (pos < start || pos >= end) continue;
      const bool live = pos < len;
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t x[4];
        e2m1x8_to_half2(b == 0 ? code.x : b == 1 ? code.y : b == 2 ? code.z : code.w, x);
        const uint32_t sw = b == 0 ? scale.x : b == 1 ? scale.y : b == 2 ? scale.z : scale.w;
        const float s = __fmul_rn(e4m3_to_float((uint8_t)(sw >> ((k >> 1) * 16 + (k & 1) * 8))), gv);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x[(k >> 1) * 2])), q = __half22float2(*reinterpret_cast<const __half2*>(&x[(k >> 1) * 2 + 1]));
        store2(a.v, (out0 + (int64_t)r * c.kv_heads) * D + chunk * 64 + b * 16 + g * 2, a.dtype, live ? ((k & 1) ? p.y : p.x) * s : 0.0f,
               live ? ((k & 1) ? q.y : q.x) * s : 0.0f);
      }
    }
  }
}

// ---------------------------------------------------------------- compact

// a block's 256 tokens reach into 17 groups, and a copied page has up to 7 more before them
constexpr int kMoveGroups = WHEAD_KV_MAX_BLOCK / 16 + 1 + 7;
constexpr int kMoveTokens = kMoveGroups * 16;

struct CompactArgs {
  const int32_t* start;
  const int32_t* keep;
  const int32_t* count;
  const int32_t* slots;
  int n, width;
};

struct CompactEntry {
  int slot, start, count, len, stay;
  bool ok;
};

// An entry with its first kept tokens that are in place already counted, by a whole warp.
__device__ __forceinline__ CompactEntry compact_entry(const Cache& c, const CompactArgs& a, int i) {
  const int lane = threadIdx.x & 31;
  CompactEntry e;
  e.slot = entry_slot(a.slots, i);
  e.start = a.start[i];
  e.count = a.count ? a.count[i] : 0;
  e.stay = 0;
  e.ok = (unsigned)e.slot < (unsigned)c.max_seqs;
  e.len = e.ok ? c.lens[e.slot] : 0;
  if (e.start < 0 || e.start > e.len || e.count < 0 || e.count > a.width || e.len > (int64_t)c.max_pages * c.page_size) e.ok = false;
  if (!e.ok) return e;
  bool bad = false;
  int stay = 0;
  for (int base = 0; base < e.count; base += 32) {
    const int j = base + lane;
    int k = -1, before = -1;
    if (j < e.count) {
      k = a.keep[(int64_t)i * a.width + j];
      before = j ? a.keep[(int64_t)i * a.width + j - 1] : -1;
      bad |= k <= before || k >= WHEAD_KV_MAX_BLOCK || k >= e.len - e.start || before < -1;
    }
    stay += __popc(__ballot_sync(~0u, j < e.count && k == j));
  }
  e.stay = stay;
  e.ok = !__any_sync(~0u, bad);
  return e;
}

// Tables, lengths and references after a compact, by one CTA: which pages are free, and which are the lowest, is one scan of all
// references. Bound by the latency of its steps (5.6 us for 8 blocks of 17, plan and move; 12.6 for 64 of 33). region: the pages that each entry's block lay in and those that it lies in.
__global__ void __launch_bounds__(kPlan, 1) compact_plan(Cache c, CompactArgs a) {
  after_previous();
  __shared__ PlanShared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  // the entries' pages that are shared and will be written
  for (int i = warp; i < a.n; i += kPlan / 32) {
    const CompactEntry e = compact_entry(c, a, i);
    if (!e.ok) {
      if (lane == 0) atomicMin(&s.bad, WHEAD_ERR_INVALID_ARG);
      continue;
    }
    const int lo = (e.start + e.stay) >> c.page_shift, hi = pages_of(c, e.start + e.count);
    int shared = 0;
    for (int base = lo; base < hi; base += 32) {
      const int p = base + lane;
      const int page = p < hi ? c.tables[(int64_t)e.slot * c.max_pages + p] : -1;
      shared += __popc(__ballot_sync(~0u, (unsigned)page < (unsigned)c.num_pages && c.refs[page] > 1));
    }
    if (lane == 0) c.seq_a[i] = shared;
  }
  __syncthreads();
  int bad = s.bad;
  int need = 0;
  if (!bad) {
    for (int base = 0; base < a.n; base += kPlan) {
      const int i = base + threadIdx.x;
      int total;
      const int at = block_scan(i < a.n ? c.seq_a[i] : 0, s, total);
      if (i < a.n) c.seq_b[i] = need + at;
      need += total;
    }
    __syncthreads();
    if (need > 0 && find_free(c, need, s) < need) bad = WHEAD_ERR_NO_PAGES;
  }
  verdict(c, bad);
  if (bad) return;
  // which pages are shared is decided for all entries before any reference changes
  for (int i = warp; i < a.n; i += kPlan / 32) {
    const CompactEntry e = compact_entry(c, a, i);
    const int first = e.start >> c.page_shift, lo = (e.start + e.stay) >> c.page_shift, hi = pages_of(c, e.start + e.count);
    int at = c.seq_b[i];
    for (int base = first; base < first + kRegionPages; base += 32) {
      const int p = base + lane;
      const bool in = p < first + kRegionPages && p < c.max_pages;
      const int page = in ? c.tables[(int64_t)e.slot * c.max_pages + p] : -1;
      const bool copy = in && p >= lo && p < hi && (unsigned)page < (unsigned)c.num_pages && c.refs[page] > 1;
      const unsigned m = __ballot_sync(~0u, copy);
      if (p < first + kRegionPages) {
        c.region[(int64_t)i * 2 * kRegionPages + p - first] = page;
        c.region[((int64_t)i * 2 + 1) * kRegionPages + p - first] = copy ? c.fresh[at + __popc(m & ((1u << lane) - 1u))] : page;
      }
      at += __popc(m);
    }
  }
  __syncthreads();
  for (int i = warp; i < a.n; i += kPlan / 32) {
    const CompactEntry e = compact_entry(c, a, i);
    const int first = e.start >> c.page_shift, hi = pages_of(c, e.start + e.count), had = pages_of(c, e.len);
    __syncwarp();
    for (int p = first + lane; p < had; p += 32) {
      int32_t* at = &c.tables[(int64_t)e.slot * c.max_pages + p];
      const int old = *at;
      const int now = p >= hi ? -1 : p - first < kRegionPages ? c.region[((int64_t)i * 2 + 1) * kRegionPages + p - first] : old;
      if (now == old) continue;
      *at = now;
      if ((unsigned)old < (unsigned)c.num_pages) atomicSub(&c.refs[old], 1);
      if (now >= 0) c.refs[now] = 1;
    }
    if (lane == 0) {
      c.seq_a[i] = e.stay;
      c.lens[e.slot] = e.start + e.count;
    }
  }
}

// One CTA moves one entry's kept tokens of one head. All groups that tokens come from are in shared memory before the
// first one is written, so a group may be source and target. Bound by latency: 64 blocks of 33 tokens are 12 MB.
template <int D>
__global__ void __launch_bounds__(128) compact_move(Cache c, CompactArgs a) {
  after_previous();
  constexpr int NB = D / 16, kGroup = 18 * D;
  extern __shared__ __align__(16) uint8_t smem[];
  if (c.ctl->abort) return;
  const int i = blockIdx.x, h = blockIdx.y;
  const int start = a.start[i], count = a.count ? a.count[i] : 0, stay = c.seq_a[i];
  const int first = start >> c.page_shift;
  const int32_t* before = c.region + (int64_t)i * 2 * kRegionPages;
  const int32_t* after = before + kRegionPages;
  const int end = start + count;
  if (end == 0) return;
  // groups to write: from the first moved token on, and the whole of a page that is copied
  int lo = (start + stay) >> 4;
  const int lo_page = (start + stay) >> c.page_shift;
  const int gpp = c.page_size >> 4;
  const bool copied = lo_page - first < kRegionPages && lo_page < pages_of(c, end) && before[lo_page - first] != after[lo_page - first];
  if (copied) lo = lo_page * gpp;
  const int hi = (end + 15) >> 4;
  if (lo >= hi || (stay == count && !copied)) return;
  // source groups: from lo to the last kept token's
  const int last = count ? (start + max(a.keep[(int64_t)i * a.width + count - 1], 0)) >> 4 : hi - 1;
  const int ng = max(last, hi - 1) - lo + 1;
  int* from = reinterpret_cast<int*>(smem);  // token map, then the groups
  uint8_t* groups = smem + kMoveTokens * 4;
  for (int x = threadIdx.x; x < (hi - lo) * 16; x += blockDim.x) {
    const int pos = lo * 16 + x, j = pos - start;
    from[x] = (j >= stay && j < count ? start + a.keep[(int64_t)i * a.width + j] : pos) - lo * 16;
  }
  for (int x = threadIdx.x; x < ng * (kGroup / 16); x += blockDim.x) {
    const int gr = lo + x / (kGroup / 16), off = x % (kGroup / 16);
    const int page = before[gr / gpp - first];
    reinterpret_cast<uint4*>(groups)[x] = is_page(c, page) ? reinterpret_cast<const uint4*>(group_ptr<D>(c, page, h, gr * 16))[off] : make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  for (int y = threadIdx.x >> 5; y < hi - lo; y += blockDim.x >> 5) {
    const int page = after[(lo + y) / gpp - first];
    if (!is_page(c, page)) continue;
    uint8_t* out = group_ptr<D>(c, page, h, (lo + y) * 16);
    const int* m = from + y * 16;
    const int k0 = m[g], k1 = m[g + 8];
    const int v[4] = {m[2 * t], m[2 * t + 1], m[2 * t + 8], m[2 * t + 9]};
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int word = (b / 4) * 128 + (b % 4);
      auto key = [&](int r) {
        const uint32_t w = reinterpret_cast<const uint32_t*>(groups + (r >> 4) * kGroup)[word + ((r & 7) * 4 + t) * 4];
        return (r & 8) ? (w >> 8) & 0x00FF00FFu : w & 0x00FF00FFu;
      };
      reinterpret_cast<uint32_t*>(out)[word + lane * 4] = key(k0) | key(k1) << 8;
      uint32_t w = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = v[k];
        const uint32_t u = reinterpret_cast<const uint32_t*>(groups + (r >> 4) * kGroup + 9 * D)[word + (g * 4 + (r & 7) / 2) * 4];
        w |= ((u >> ((r & 1) * 4 + ((r >> 3) & 1) * 16)) & 0x0F0Fu) << ((k & 1) * 4 + (k >> 1) * 16);
      }
      reinterpret_cast<uint32_t*>(out + 9 * D)[word + lane * 4] = w;
    }
    for (int x = lane; x < 16 * NB; x += 32) {
      const int r = x / NB, b = x % NB, f = m[r];
      const uint8_t* src = groups + (f >> 4) * kGroup;
      out[8 * D + (r & 7) * 2 * NB + b * 2 + (r >> 3)] = src[8 * D + (f & 7) * 2 * NB + b * 2 + ((f >> 3) & 1)];
      out[17 * D + ((r & 7) >> 1) * 4 * NB + b * 4 + (r >> 3) * 2 + (r & 1)] =
          src[17 * D + ((f & 7) >> 1) * 4 * NB + b * 4 + ((f >> 3) & 1) * 2 + (f & 1)];
    }
  }
}

// ---------------------------------------------------------------- fork

// Three kernels: who needs a page, and which; new rows and copied pages beside the old rows, which other slots may still read;
// then the new rows in place. Bound by the latency of the three (7.2 us for 8 slots on 2,000 tokens, 10.6 us for 128 on 12,000, of
// which the copied pages' bytes are 2 at most).

// Which slots get a copy of a partial last page, and the page: seq_a[i] = that page or -1.
__global__ void __launch_bounds__(kPlan, 1) fork_plan(Cache c, const int32_t* parents) {
  after_previous();
  __shared__ PlanShared s;
  if (threadIdx.x == 0) s.bad = 0;
  __syncthreads();
  int need = 0;
  for (int base = 0; base < c.max_seqs; base += kPlan) {
    const int i = base + threadIdx.x;
    int copy = 0;
    if (i < c.max_seqs) {
      const int p = parents[i];
      const int64_t most = (int64_t)c.max_pages * c.page_size;
      const int own = c.lens[i];
      if (p < -1 || p >= c.max_seqs || own < 0 || own > most) {
        atomicMin(&s.bad, WHEAD_ERR_INVALID_ARG);
      } else if (p >= 0 && p != i) {
        const int len = c.lens[p];
        if (len < 0 || len > most) atomicMin(&s.bad, WHEAD_ERR_INVALID_ARG);
        else copy = (len & (c.page_size - 1)) != 0;
      }
    }
    int total;
    const int at = block_scan(copy, s, total);
    if (i < c.max_seqs) c.seq_a[i] = copy ? need + at : -1;
    need += total;
  }
  __syncthreads();
  int bad = s.bad;
  if (!bad && need > 0 && find_free(c, need, s) < need) bad = WHEAD_ERR_NO_PAGES;
  verdict(c, bad);
  if (bad) return;
  for (int i = threadIdx.x; i < c.max_seqs; i += kPlan)
    if (c.seq_a[i] >= 0) c.seq_a[i] = c.fresh[c.seq_a[i]];
}

// The slots' new rows and lengths (into the workspace: other slots may still read the old ones), the partial pages' copies.
// gridDim.y CTAs share a slot's copy; the first of them does its row.
__global__ void __launch_bounds__(256) fork_copy(Cache c, const int32_t* parents) {
  after_previous();
  if (c.ctl->abort) return;
  const int i = blockIdx.x;
  const int p = parents[i];
  if (p == i) return;
  const int len = p >= 0 ? c.lens[p] : 0;
  const int fresh = c.seq_a[i];
  if (blockIdx.y == 0) {
    const int pages = pages_of(c, len);
    for (int k = threadIdx.x; k < c.max_pages; k += blockDim.x)
      c.rows[(int64_t)i * c.max_pages + k] = k >= pages ? -1 : k == pages - 1 && fresh >= 0 ? fresh : c.tables[(int64_t)p * c.max_pages + k];
    if (threadIdx.x == 0) c.seq_b[i] = len;
  }
  if (fresh >= 0) {
    const int page = c.tables[(int64_t)p * c.max_pages + (len >> c.page_shift)];
    if ((unsigned)page >= (unsigned)c.num_pages) {
      if (threadIdx.x == 0) set_status(c, WHEAD_ERR_INTERNAL);
      return;
    }
    const int64_t bytes = (int64_t)c.kv_heads * (c.page_size >> 4) * 18 * c.head_dim;
    const uint4* src = reinterpret_cast<const uint4*>(c.pool + page * bytes);
    uint4* dst = reinterpret_cast<uint4*>(c.pool + fresh * bytes);
    for (int64_t k = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; k < bytes / 16; k += (int64_t)gridDim.y * blockDim.x) dst[k] = src[k];
  }
}

__global__ void __launch_bounds__(256) fork_apply(Cache c, const int32_t* parents) {
  after_previous();
  if (c.ctl->abort) return;
  const int i = blockIdx.x;
  const int p = parents[i];
  if (p == i) return;
  const int had = pages_of(c, c.lens[i]);
  const int now = c.seq_b[i], pages = pages_of(c, now);
  for (int k = threadIdx.x; k < c.max_pages; k += blockDim.x) {
    int32_t* at = &c.tables[(int64_t)i * c.max_pages + k];
    const int old = *at, page = c.rows[(int64_t)i * c.max_pages + k];
    if (k < had && (unsigned)old < (unsigned)c.num_pages) atomicSub(&c.refs[old], 1);
    if (k < pages && (unsigned)page < (unsigned)c.num_pages) atomicAdd(&c.refs[page], 1);
    *at = page;
  }
  __syncthreads();
  if (threadIdx.x == 0) c.lens[i] = now;
}

}  // namespace

}  // namespace whead_kv_impl

using namespace whead_kv_impl;

namespace {
template <int D>
int launch_write(const HostCache& h, const AppendArgs& a, dim3 grid) {
  return a.dtype == WHEAD_KV_BF16  ? launch_after(append_write<D, WHEAD_KV_BF16>, grid, D, 0, h.stream, h.c, a)
         : a.dtype == WHEAD_KV_F16 ? launch_after(append_write<D, WHEAD_KV_F16>, grid, D, 0, h.stream, h.c, a)
                                   : launch_after(append_write<D, WHEAD_KV_F32>, grid, D, 0, h.stream, h.c, a);
}

template <int D>
int launch_move(const HostCache& h, const CompactArgs& a) {
  const int smem = kMoveTokens * 4 + kMoveGroups * 18 * D;
  static std::atomic<bool> granted[kMaxDevices];
  if (!grant_smem(compact_move<D>, smem, h, granted)) return WHEAD_ERR_CUDA;
  return launch_after(compact_move<D>, dim3(a.n, h.c.kv_heads), 128, smem, h.stream, h.c, a);
}
}  // namespace

extern "C" {

int64_t whead_kv_page_bytes(int32_t page_size, int32_t kv_heads, int32_t head_dim) {
  whead_kv k{};
  k.page_size = page_size;
  k.kv_heads = kv_heads;
  k.head_dim = head_dim;
  k.max_seqs = k.max_pages = k.num_pages = 1;
  const int rc = check_shape(k);
  return rc != WHEAD_OK ? rc : (int64_t)kv_heads * (page_size / 16) * 18 * head_dim;
}

int64_t whead_kv_workspace_bytes(const whead_kv* kv) {
  if (!kv) return WHEAD_ERR_INVALID_ARG;
  const int rc = check_shape(*kv);
  if (rc != WHEAD_OK) return rc;
  int device;
  const int sms = device_sms(&device);
  if (sms < 1) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  return layout(*kv, sms).total;
}

int whead_kv_append(const whead_kv* kv, const void* k, const void* v, int32_t dtype, int64_t k_token_stride,
                    int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t* indptr,
                    const int32_t* slots, int32_t n, int64_t total) {
  if (n < 0 || total < 0 || dtype < WHEAD_KV_BF16 || dtype > WHEAD_KV_F32) return WHEAD_ERR_INVALID_ARG;
  if (!kv || n > kv->max_seqs || total >= INT_MAX) return WHEAD_ERR_INVALID_ARG;
  if (n == 0 || total == 0) {
    HostCache h;
    return n == 0 && total > 0 ? WHEAD_ERR_INVALID_ARG : host_cache(kv, &h);
  }
  if (!k || !v || (!indptr && total % n) || (indptr && !aligned(indptr, 4)) || (slots && !aligned(slots, 4))) return WHEAD_ERR_INVALID_ARG;
  const uintptr_t e = dtype == WHEAD_KV_F32 ? 4 : 2;
  if (!aligned(k, e) || !aligned(v, e)) return WHEAD_ERR_INVALID_ARG;
  HostCache h;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  AppendArgs a{k, v, dtype, k_token_stride, k_head_stride, v_token_stride, v_head_stride, indptr, slots, n, total, false, false};
  a.wide_k = aligned(k, 4 * e) && k_token_stride % 4 == 0 && k_head_stride % 4 == 0;
  a.wide_v = aligned(v, 2 * e) && v_token_stride % 2 == 0 && v_head_stride % 2 == 0;
  const int64_t groups = std::min(total / 16 + 2 * (int64_t)n, total);  // most that the tokens can touch
  if (groups > h.c.partial_floats / 4) return WHEAD_ERR_UNSUPPORTED;    // more than the workspace can list: some 20 million tokens of 64 channels
  const int st = launch_after(append_plan, dim3(1), kPlan, 0, h.stream, h.c, a);
  if (st != WHEAD_OK) return st;
  const dim3 grid((unsigned)std::min<int64_t>(groups, 65535 * 4), kv->kv_heads);
  return kv->head_dim == 64 ? launch_write<64>(h, a, grid) : kv->head_dim == 128 ? launch_write<128>(h, a, grid) : launch_write<256>(h, a, grid);
}

int whead_kv_read(const whead_kv* kv, const int32_t* start, const int32_t* slots, int32_t n, int32_t count, int32_t dtype,
                  void* k_out, void* v_out) {
  if (!kv || n < 0 || n > kv->max_seqs || count < 0 || dtype < WHEAD_KV_BF16 || dtype > WHEAD_KV_F32) return WHEAD_ERR_INVALID_ARG;
  HostCache h;
  if (n == 0 || count == 0) return host_cache(kv, &h);
  if (!start || !k_out || !v_out || !aligned(start, 4) || !aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return WHEAD_ERR_INVALID_ARG;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  const int64_t groups = (int64_t)n * ((count + 30LL) / 16);
  if (count > INT_MAX - 64 || groups >= INT_MAX) return WHEAD_ERR_UNSUPPORTED;
  const ReadArgs a{start, slots, n, count, dtype, k_out, v_out};
  const dim3 grid((unsigned)groups, kv->kv_heads);
  return kv->head_dim == 64    ? launch_after(read_kernel<64>, grid, 64, 0, h.stream, h.c, a)
         : kv->head_dim == 128 ? launch_after(read_kernel<128>, grid, 128, 0, h.stream, h.c, a)
                               : launch_after(read_kernel<256>, grid, 256, 0, h.stream, h.c, a);
}

int whead_kv_compact(const whead_kv* kv, const int32_t* start, const int32_t* keep, const int32_t* count, const int32_t* slots,
                     int32_t n, int32_t keep_width) {
  if (!kv || n < 0 || n > kv->max_seqs || keep_width < 0 || keep_width > WHEAD_KV_MAX_BLOCK) return WHEAD_ERR_INVALID_ARG;
  HostCache h;
  if (n == 0) return host_cache(kv, &h);
  if (!start || (keep && !count) || (!keep && keep_width > 0)) return WHEAD_ERR_INVALID_ARG;  // an empty keep may have no address
  if (!aligned(start, 4) || !aligned(keep, 4) || !aligned(count, 4) || !aligned(slots, 4)) return WHEAD_ERR_INVALID_ARG;
  int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  const CompactArgs a{start, keep, count, slots, n, keep_width};
  rc = launch_after(compact_plan, dim3(1), kPlan, 0, h.stream, h.c, a);
  if (rc != WHEAD_OK) return rc;
  return kv->head_dim == 64 ? launch_move<64>(h, a) : kv->head_dim == 128 ? launch_move<128>(h, a) : launch_move<256>(h, a);
}

int whead_kv_fork(const whead_kv* kv, const int32_t* parents) {
  if (!kv || !parents || !aligned(parents, 4)) return WHEAD_ERR_INVALID_ARG;
  HostCache h;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  int st = launch_after(fork_plan, dim3(1), kPlan, 0, h.stream, h.c, parents);
  if (st != WHEAD_OK) return st;
  const int64_t bytes = (int64_t)kv->kv_heads * (kv->page_size / 16) * 18 * kv->head_dim;
  st = launch_after(fork_copy, dim3(kv->max_seqs, (unsigned)std::min<int64_t>(8, (bytes + 16383) / 16384)), 256, 0, h.stream, h.c, parents);
  if (st != WHEAD_OK) return st;
  return launch_after(fork_apply, dim3(kv->max_seqs), 256, 0, h.stream, h.c, parents);
}

int whead_kv_status(const whead_kv* kv) {
  HostCache h;
  const int rc = host_cache(kv, &h);
  if (rc != WHEAD_OK) return rc;
  int st = 0;
  if (cudaMemcpyAsync(&st, &h.c.ctl->status, sizeof st, cudaMemcpyDeviceToHost, h.stream) != cudaSuccess ||
      cudaStreamSynchronize(h.stream) != cudaSuccess) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  if (st != 0 && (cudaMemsetAsync(&h.c.ctl->status, 0, sizeof st, h.stream) != cudaSuccess ||
                  cudaStreamSynchronize(h.stream) != cudaSuccess)) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  return st;
}

}  // extern "C"

// kv_common.cuh — what the 4-bit paged KV cache's kernels share: the cache as kernels see it, the workspace's layout,
// conversions of its number formats, and the attention's division of work over CTAs.
#pragma once

#include "../../include/whead_kv.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace whead_kv_impl {

constexpr int kMaxCtas = 2048;        // most CTAs of an attend launch (partial results, counters)
constexpr int kRegionPages = WHEAD_KV_MAX_BLOCK / 16 + 1;  // pages that a block's tokens can lie in
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoKey = -3.402823466e38f;  // a running maximum before the first key: fp32's lowest, so that every score may follow it

// Workspace: the control words, then per-slot arrays, then the attention's counters and partial results.
struct Ctl {
  int status;  // first device-side error
  int abort;   // set by a planning kernel: the call's later kernels do nothing
  int total;   // groups of an append
  int pad;
  unsigned ticket[4];
};

struct Cache {
  uint8_t* pool;
  int32_t* lens;
  int32_t* refs;
  int32_t* tables;
  const float* k_scale;
  const float* v_scale;
  int page_size, page_shift, kv_heads, head_dim, max_seqs, max_pages, num_pages;
  Ctl* ctl;
  int32_t* seq_a;   // max_seqs + 1
  int32_t* seq_b;   // max_seqs + 1
  int32_t* region;  // max_seqs x 2 x kRegionPages: pages of a block before and after
  int32_t* fresh;   // num_pages: free pages found
  int32_t* rows;    // max_seqs x max_pages: tables after a fork
  unsigned* counters;   // kMaxCtas
  int32_t* starts;      // kMaxCtas x 4
  int32_t* records;     // kMaxCtas x 4: what a joining kernel has to do
  float* partial;
  int64_t partial_floats;
};

__host__ __device__ inline int64_t align256(int64_t x) { return (x + 255) & ~(int64_t)255; }

// Floats of partial results: two for each CTA (a CTA's range of work begins inside one item and ends inside another). The most
// rows an SM has under way: 256, by one CTA of two tiles; the kernel for few rows has up to four CTAs of 32.
inline int64_t partial_floats(int head_dim, int sms) { return (int64_t)sms * 2 * 256 * (head_dim + 2); }

// ---------------------------------------------------------------- number formats

// the two e2m1 values of each byte of w as f16 pairs (low nibble in the low half)
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

// the four e4m3 values of w as two f16 pairs
__device__ __forceinline__ void e4m3x4_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi) : "r"(w));
}

// byte of e2m1 codes: lo in the low nibble; nearest even, saturating
__device__ __forceinline__ uint32_t e2m1x2_from_float(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 b;\n cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n mov.b32 %0, {b, 0, 0, 0};\n}\n" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ float e4m3_to_float(uint8_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(b, __NV_E4M3)));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// products with one half of s (an operand modifier: no instruction of its own)
__device__ __forceinline__ uint32_t hmul2_low(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul2_high(uint32_t a, uint32_t s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(*reinterpret_cast<const __half2*>(&s)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// N consecutive elements from i on, in two steps, so that many loads can be under way before the first is looked at: the elements as
// they are, and their values. `wide`: the address is a multiple of their size.
template <int DTYPE, int N>
struct RawElems {
  uint32_t w[DTYPE == WHEAD_KV_F32 ? N : N / 2];
};
template <int DTYPE, int N>
__device__ __forceinline__ void load_raw(const void* p, int64_t i, bool wide, RawElems<DTYPE, N>& r) {
  constexpr int W = DTYPE == WHEAD_KV_F32 ? N : N / 2;
  const char* at = static_cast<const char*>(p) + i * (DTYPE == WHEAD_KV_F32 ? 4 : 2);
  if (wide) {
    if constexpr (W == 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(at));
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    } else if constexpr (W == 2) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(at));
      r.w[0] = v.x; r.w[1] = v.y;
    } else {
      r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(at));
    }
  } else if constexpr (DTYPE == WHEAD_KV_F32) {
#pragma unroll
    for (int k = 0; k < N; ++k) r.w[k] = __ldg(reinterpret_cast<const uint32_t*>(at) + k);
  } else {
    const unsigned short* x = reinterpret_cast<const unsigned short*>(at);
#pragma unroll
    for (int k = 0; k < N / 2; ++k) r.w[k] = __ldg(x + 2 * k) | (uint32_t)__ldg(x + 2 * k + 1) << 16;
  }
}
template <int DTYPE, int N>
__device__ __forceinline__ void raw_values(const RawElems<DTYPE, N>& r, float (&x)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if constexpr (DTYPE == WHEAD_KV_F32) x[k] = __uint_as_float(r.w[k]);
    else if constexpr (DTYPE == WHEAD_KV_BF16) x[k] = __uint_as_float(k & 1 ? r.w[k / 2] & 0xFFFF0000u : r.w[k / 2] << 16);
    else x[k] = __half2float(__ushort_as_half((unsigned short)(r.w[k / 2] >> (k & 1) * 16)));
  }
}

// four consecutive elements of a 16-bit type from i on, as they are; `wide`: the address is a multiple of 8
__device__ __forceinline__ uint2 load_four(const void* p, int64_t i, bool wide) {
  const uint16_t* x = static_cast<const uint16_t*>(p) + i;
  if (wide) return __ldg(reinterpret_cast<const uint2*>(x));
  return make_uint2(x[0] | (uint32_t)x[1] << 16, x[2] | (uint32_t)x[3] << 16);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, int dtype) {
  if (dtype == WHEAD_KV_BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, int dtype) {
  if (dtype == WHEAD_KV_BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ---------------------------------------------------------------- copies and barriers

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// Waits for the phase of this parity to complete, for at most two seconds; false when it did not.
static __device__ __noinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity) {
  unsigned long long t0, t1;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  do {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try(bar, parity)) return true;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
  } while (t1 - t0 < 2000000000ull);
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity) {
  return mbar_try(bar, parity) || mbar_try(bar, parity) || mbar_wait_slow(bar, parity);
}
__device__ __forceinline__ void fence_mbar_init() { asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory"); }

// `bytes` (a multiple of 16) from global to shared memory, both 16-byte aligned; counted by the barrier
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar) : "memory");
}

template <int THREADS>
__device__ __forceinline__ void named_sync(int id) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(THREADS) : "memory");
}

// ---------------------------------------------------------------- the cache

__device__ __forceinline__ void set_status(const Cache& c, int code) { atomicCAS(&c.ctl->status, 0, code); }

// Whether a table's entry is a page of the pool; reported where it is not.
__device__ __forceinline__ bool is_page(const Cache& c, int page) {
  if ((unsigned)page < (unsigned)c.num_pages) return true;
  set_status(c, WHEAD_ERR_INTERNAL);
  return false;
}

// Group `pos / 16` of head h in a slot's page, to read: pages out of range read page 0. Who writes asks is_page first.
template <int D>
__device__ __forceinline__ uint8_t* group_ptr(const Cache& c, int page, int h, int pos) {
  if (!is_page(c, page)) page = 0;
  const int in_page = (pos & (c.page_size - 1)) >> 4;
  return c.pool + (((int64_t)page * c.kv_heads + h) * (c.page_size >> 4) + in_page) * (18 * D);
}

// A slot's length, 0 (and an error) for what is not a slot.
__device__ __forceinline__ int slot_len(const Cache& c, int slot) {
  if ((unsigned)slot >= (unsigned)c.max_seqs) {
    set_status(c, WHEAD_ERR_INVALID_ARG);
    return 0;
  }
  const int len = c.lens[slot];
  const int64_t most = (int64_t)c.max_pages * c.page_size;
  if (len < 0 || len > most) {
    set_status(c, WHEAD_ERR_INTERNAL);
    return 0;
  }
  return len;
}

// ---------------------------------------------------------------- host

struct HostCache {
  Cache c;
  cudaStream_t stream;
  int device, sms;
};

// Checks a whead_kv and lays its workspace out; WHEAD_OK or an error.
int host_cache(const whead_kv* kv, HostCache* out);
int device_sms(int* device);  // SMs of the current device, 0 on an error

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// ---------------------------------------------------------------- launches

// Every kernel of the cache may be placed while the one before it in the stream still runs. It lets the next one be placed as soon
// as all of its own CTAs are, and waits for the one before it to end before it looks at anything: that hides most of the time
// between two kernels, which counts where a call is two or three small ones (a fork, three kernels, and the reading of what it
// wrote: 16.7 us where a kernel waits but does not let the next one go early, 15.7 so). A chain stays in order: a kernel that has
// ended has waited for all before it.
__device__ __forceinline__ void after_previous() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets a kernel have more than 48 KB of shared memory, once on each device; `granted`: a static of the kernel's own.
constexpr int kMaxDevices = 64;
template <typename K>
bool grant_smem(K* kernel, int bytes, const HostCache& h, std::atomic<bool> (&granted)[kMaxDevices]) {
  if (granted[h.device].load(std::memory_order_relaxed)) return true;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    (void)cudaGetLastError();
    return false;
  }
  granted[h.device].store(true, std::memory_order_relaxed);
  return true;
}

template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config{};
  config.gridDim = grid;
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &early;
  config.numAttrs = 1;
  if (cudaLaunchKernelEx(&config, kernel, P(args)...) != cudaSuccess) {
    (void)cudaGetLastError();
    return WHEAD_ERR_CUDA;
  }
  return WHEAD_OK;
}

}  // namespace whead_kv_impl

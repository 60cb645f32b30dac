// Shared by the paged key-value cache kernels: sizes, the request scan, and
// the launchers that page_api.cu calls.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace mova {

constexpr int kHeadDim = 128;
constexpr int kMaxRequests = 4096;
constexpr int kMaxGroup = 16;    // query heads per KV head
constexpr int kMaxCtas = 592;    // of an attention or score kernel
constexpr int kMaxWorkers = kMaxCtas * 4;  // warps of an attention kernel
constexpr int kNoBad = 0x7fffffff;
// Floats of a partial result per query head: 128 outputs, a maximum and a sum,
// and two that keep every partial result 16-byte aligned.  The outputs of the
// G heads come first, then the maxima, then the sums.
constexpr int kPartRow = kHeadDim + 4;

// Parts of the workspace.  `part` holds two partial results per worker.
struct PageWs {
  StatusBlock* sb;
  int32_t* bad;     // (kMaxCtas) first bad request seen by each CTA (kNoBad: none)
  int32_t* prefix;  // (B + 1) tiles of one KV head before each request
  float* part;
  unsigned long long* keys;  // select: (B, kv_heads, max_pages) sortable scores
  size_t bytes;
};

// What the kernels know of the cache.  Strides in elements.
struct PageArgs {
  const void* k;
  const void* v;
  long long k_stride, v_stride;  // page to page
  const float* k_scale;
  const float* v_scale;
  int num_pages, kv, shift;  // page_size = 1 << shift
  const int32_t* table;
  long long table_stride;
  int max_pages;
  const int32_t* lens;
  int B;
};

// Exclusive prefix sum over the requests, by the whole CTA: pre[0..B] in
// shared memory, count(b) evaluated once per request.  Ends with a barrier.
template <int kThreads, typename T, typename F>
__device__ __forceinline__ void request_scan(int B, T* pre, F count) {
  __shared__ T warp_sum[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  T carry = 0;
  for (int base = 0; base < B; base += kThreads) {
    const int b = base + tid;
    const T c = b < B ? count(b) : T(0);
    T incl = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    T before = carry, all = carry;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const T s = warp_sum[w];
      if (w < warp) before += s;
      all += s;
    }
    if (b < B) pre[b] = before + incl - c;
    carry = all;
    __syncthreads();
  }
  if (tid == 0) pre[B] = carry;
  __syncthreads();
}

// As request_scan, of two counts per request at once; sums in 64 bits, stored
// clipped to kClip (more than any count of pages or tokens that is used).
constexpr int kClip = 0x7fffffff;
template <int kThreads, typename F>
__device__ __forceinline__ void request_scan2(int B, int2* pre, F count) {
  __shared__ long long warp_sum[2][kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long carry1 = 0, carry2 = 0;
  auto clip = [](long long x) { return static_cast<int>(x > kClip ? kClip : x); };
  for (int base = 0; base < B; base += kThreads) {
    const int b = base + tid;
    long long c1 = 0, c2 = 0;
    if (b < B) count(b, c1, c2);
    long long i1 = c1, i2 = c2;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u1 = __shfl_up_sync(0xffffffffu, i1, o), u2 = __shfl_up_sync(0xffffffffu, i2, o);
      if (lane >= o) i1 += u1, i2 += u2;
    }
    if (lane == 31) warp_sum[0][warp] = i1, warp_sum[1][warp] = i2;
    __syncthreads();
    long long before1 = carry1, before2 = carry2;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const long long s1 = warp_sum[0][w], s2 = warp_sum[1][w];
      if (w < warp) before1 += s1, before2 += s2;
      carry1 += s1, carry2 += s2;
    }
    if (b < B) pre[b] = make_int2(clip(before1 + i1 - c1), clip(before2 + i2 - c2));
    __syncthreads();
  }
  if (tid == 0) pre[B] = make_int2(clip(carry1), clip(carry2));
  __syncthreads();
}

// The last b in [0, B) with pre[b] <= x (pre[0] = 0 <= x < pre[B]).
template <typename T>
__device__ __forceinline__ int request_of(const T* pre, int B, T x) {
  int lo = 0, hi = B;  // pre[lo] <= x < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int clamp_len(int len, int max_pages, int shift) {
  const long long cap = static_cast<long long>(max_pages) << shift;
  return len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
}

// c (16 x 8, fp32) += a (16 x 16) b (16 x 8), both bf16 or both fp16 (kHalf).
template <bool kHalf>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (!kHalf)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Two E4M3 values (low 16 bits of x, or high) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t x) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Prepares `kern` for its launches, once per device: `bytes` of dynamic shared
// memory, and the SM's memory split all to shared memory unless `carveout` says
// otherwise.  Kernels chained by programmatic dependent launch overlap, and an SM
// changes its split only when idle: a kernel with another split keeps the next
// one's CTAs off.
template <typename K>
cudaError_t prepare_kernel(K kern, size_t bytes, bool (&done)[64], int carveout = cudaSharedmemCarveoutMaxShared) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, carveout);
  if (err == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return err;
}

struct MapArgs {
  const int32_t *cached, *added;
  int B;
  int32_t* table;
  long long table_stride;
  int max_pages;
  const int32_t* free_pages;
  int n_free;
  const int32_t* taken;
  int shift, num_pages, T;
  int32_t *lens, *starts, *slots, *positions, *taken_out;
  StatusBlock* sb;
};
cudaError_t launch_page_map(const MapArgs& a, cudaStream_t stream);

cudaError_t launch_page_write(const void* k, const void* v, mova_dtype dt, long long k_stride, long long v_stride,
                              const int32_t* slots, int T, const mova_pages& p, StatusBlock* sb, cudaStream_t stream);
cudaError_t launch_page_bounds(const PageArgs& a, mova_dtype dt, const int32_t* cached, void* lo, void* hi,
                               StatusBlock* sb, cudaStream_t stream);
cudaError_t launch_page_attend(const void* q, long long q_stride, int G, const PageArgs& a, mova_dtype dt, float scale,
                               const int32_t* picked, int top, void* o, float* lse, const PageWs& ws,
                               cudaStream_t stream);
cudaError_t launch_page_select(const void* q, long long q_stride, int G, const PageArgs& a, mova_dtype dt,
                               const void* lo, const void* hi, int top, int32_t* picked, const PageWs& ws,
                               cudaStream_t stream);

}  // namespace mova

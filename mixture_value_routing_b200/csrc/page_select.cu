// The cache pages worth reading for a query, by per-page key bounds.
//
//   score(page) = max over the KV head's query heads h of
//                 sum_d q[h, d] * (q[h, d] < 0 ? lo[page, d] : hi[page, d])
//
// and, of the request's full pages, the `top - 1` greatest (ties: the lower
// page number), with the last page always, in ascending order.
//
// Scores: a warp takes 32 / NH pages at a time (NH heads, padded to 4, 8 or
// 16); a lane holds 4 dimensions of the queries in fp64 and accumulates one
// sum per (page, head), 32 of them, which 31 exchanges reduce and spread over
// the lanes at once.  fp64 because neighbouring scores decide what is read:
// with fp32 sums the choice would depend on their order.  2 x 128 elements
// are read for 128 G fp64 FMAs, a ratio at which the fp64 pipes and memory
// are about level for G = 4.  Scores are stored as unsigned integers in the
// same order (NaN greatest, -0 = +0).
//
// Selection: one CTA per (request, KV head) finds the K-th greatest score by
// radix search: the digits start below the bits that the least and the
// greatest score share, so two or three passes of 11 bits settle it; then one
// scan places the selected pages in order.  No atomics decide an order.
#include <math.h>

#include "paged.cuh"

namespace mova {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
constexpr int kScorePerSm = 4;
constexpr int kTopThreads = 512;
constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;

using u64 = unsigned long long;

__device__ __forceinline__ void load4(const float* p, double (&d)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, double (&d)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
  d[0] = a.x, d[1] = a.y, d[2] = b.x, d[3] = b.y;
}
__device__ __forceinline__ void load4(const uint8_t* p, double (&d)[4]) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(u >> (8 * i)), __NV_E4M3)));
}

// An unsigned integer in the order of the scores; 0 is below all of them.
__device__ __forceinline__ u64 sortable(double s) {
  if (s != s) return ~0ULL;
  const u64 b = static_cast<u64>(__double_as_longlong(s + 0.0));  // -0 + 0 = +0
  return (b >> 63) ? ~b : (b | (1ULL << 63));
}

struct SelectArgs {
  PageArgs a;
  const void* q;
  long long q_stride;
  int G, top;
  const void* lo;
  const void* hi;
  u64* keys;  // (B, kv, max_pages)
  int32_t* bad;
  int32_t* picked;
};

__device__ __forceinline__ int pages_of(const PageArgs& a, int b) {
  const int len = clamp_len(a.lens[b], a.max_pages, a.shift);
  return (len + (1 << a.shift) - 1) >> a.shift;
}

template <typename Q, typename E, int NH>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelectArgs s) {
  constexpr int kPages = 32 / NH;
  extern __shared__ int pre[];
  __shared__ int sm_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = s.a.B, kv = s.a.kv;
  if (tid == 0) sm_bad = kNoBad;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  request_scan<kScoreThreads>(B, pre, [&](int b) {
    const int len = s.a.lens[b];
    if (clamp_len(len, s.a.max_pages, s.a.shift) != len) atomicMin(&sm_bad, b);
    const int n = pages_of(s.a, b);
    return n > s.top ? (n - 1 + kPages - 1) / kPages : 0;
  });
  const int U = kv * pre[B], W = gridDim.x * kScoreWarps, w = blockIdx.x * kScoreWarps + warp;
  const int u0 = static_cast<int>(static_cast<long long>(w) * U / W);
  const int u1 = static_cast<int>(static_cast<long long>(w + 1) * U / W);
  double q[NH][4];
  int row = -1, b = 0, h = 0, tiles = 1, first = 0, pages = 0;
  for (int u = u0; u < u1; ++u) {
    if (row < 0 || u - first == tiles) {  // the next (request, KV head)
      b = request_of(pre, B, u / kv);
      tiles = pre[b + 1] - pre[b];
      h = (u - kv * pre[b]) / tiles;
      first = kv * pre[b] + h * tiles;
      row = b * kv + h;
      pages = pages_of(s.a, b) - 1;
      const Q* src = static_cast<const Q*>(s.q) + b * s.q_stride + static_cast<long long>(h) * s.G * kHeadDim + 4 * lane;
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (n < s.G) {
          load4(src + n * kHeadDim, q[n]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) q[n][i] = 0.0;
        }
      }
    }
    const int page0 = (u - first) * kPages;
    int id = -1;
    if (lane < kPages && page0 + lane < pages) {
      id = s.a.table[b * s.a.table_stride + page0 + lane];
      if (id < 0 || id >= s.a.num_pages) {
        id = -1;
        atomicMin(&sm_bad, b);
      }
    }
    double sum[32];
#pragma unroll
    for (int p = 0; p < kPages; ++p) {
      const int at = __shfl_sync(0xffffffffu, id, p);
      double lo[4] = {0.0, 0.0, 0.0, 0.0}, hi[4] = {0.0, 0.0, 0.0, 0.0};
      if (at >= 0) {
        const long long off = (static_cast<long long>(at) * kv + h) * kHeadDim + 4 * lane;
        load4(static_cast<const E*>(s.lo) + off, lo);
        load4(static_cast<const E*>(s.hi) + off, hi);
      }
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        double x = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fma(q[n][i], q[n][i] < 0.0 ? lo[i] : hi[i], x);
        sum[p * NH + n] = x;
      }
    }
    // Lane i ends with the whole warp's sum of value i.
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool upper = lane & o;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const double give = upper ? sum[i] : sum[i + o], keep = upper ? sum[i + o] : sum[i];
        sum[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    const int p = lane / NH, n = lane % NH;
    const bool there = __shfl_sync(0xffffffffu, id, p) >= 0;
    u64 key = there && n < s.G ? sortable(sum[0]) : 0ULL;
#pragma unroll
    for (int o = 1; o < NH; o <<= 1) {
      const u64 other = __shfl_xor_sync(0xffffffffu, key, o);
      key = other > key ? other : key;
    }
    if (n == 0 && page0 + p < pages) s.keys[static_cast<long long>(row) * s.a.max_pages + page0 + p] = key;
  }
  __syncthreads();
  if (tid == 0) s.bad[blockIdx.x] = sm_bad;
}

__device__ __forceinline__ u64 warp_min(u64 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 y = __shfl_xor_sync(0xffffffffu, x, o);
    x = y < x ? y : x;
  }
  return x;
}

// Exclusive prefix sum of x over the CTA; *all receives the total.  One
// barrier before and after, so calls may follow one another.
__device__ __forceinline__ int cta_scan(int x, int* all) {
  __shared__ int sums[kTopThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kTopThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    total += sums[w];
  }
  *all = total;
  return before + incl - x;
}

__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectArgs s, int score_ctas, StatusBlock* sb) {
  __shared__ int hist[kBins];
  __shared__ u64 sm_min[kTopThreads / 32], sm_max[kTopThreads / 32];
  __shared__ int sm_bin, sm_above, sm_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && warp == 0) {
    int bad = kNoBad;
    for (int i = lane; i < score_ctas; i += 32) bad = min(bad, s.bad[i]);
    bad = __reduce_min_sync(0xffffffffu, bad);
    if (lane == 0) {
      sb->code = bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
      sb->detail = bad == kNoBad ? 0 : bad;
    }
  }
  const int b = blockIdx.x / s.a.kv;
  const int n = pages_of(s.a, b), top = s.top;
  int32_t* out = s.picked + static_cast<long long>(blockIdx.x) * top;
  if (n <= top) {
    for (int i = tid; i < top; i += kTopThreads) out[i] = i < n ? i : -1;
    return;
  }
  if (tid == 0) out[top - 1] = n - 1;
  if (top == 1) return;
  const int N = n - 1;
  const u64* keys = s.keys + static_cast<long long>(blockIdx.x) * s.a.max_pages;

  u64 least = ~0ULL, most_inv = ~0ULL;  // the greatest, as the least complement
#pragma unroll 4
  for (int i = tid; i < N; i += kTopThreads) {
    const u64 k = keys[i];
    least = k < least ? k : least;
    most_inv = ~k < most_inv ? ~k : most_inv;
  }
  least = warp_min(least);
  most_inv = warp_min(most_inv);
  if (lane == 0) sm_min[warp] = least, sm_max[warp] = most_inv;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTopThreads / 32; ++w) {
    least = sm_min[w] < least ? sm_min[w] : least;
    most_inv = sm_max[w] < most_inv ? sm_max[w] : most_inv;
  }
  const u64 most = ~most_inv;
  int bits = least == most ? 0 : 64 - __clzll(static_cast<long long>(least ^ most));  // still open below
  u64 prefix = bits == 64 ? 0ULL : most >> bits;
  int need = top - 1;  // to take from the keys that share the prefix
  bool all = false;    // every one of them
  while (bits > 0 && !all) {
    const int width = bits < kDigit ? bits : kDigit, sh = bits - width;
    for (int i = tid; i < kBins; i += kTopThreads) hist[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = tid; i < N; i += kTopThreads) {
      const u64 k = keys[i];
      if (bits == 64 || (k >> bits) == prefix) atomicAdd(&hist[static_cast<int>(k >> sh) & ((1 << width) - 1)], 1);
    }
    __syncthreads();
    // Thread i holds the bins below kBins - 4 i, from the top.
    constexpr int kPer = kBins / kTopThreads;
    int c[kPer], mine = 0, total;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = hist[kBins - 1 - (tid * kPer + j)];
      mine += c[j];
    }
    int above = cta_scan(mine, &total);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (above < need && need <= above + c[j]) sm_bin = kBins - 1 - (tid * kPer + j), sm_above = above, sm_in = c[j];
      above += c[j];
    }
    __syncthreads();
    prefix = (prefix << width) | static_cast<u64>(sm_bin);
    need -= sm_above;
    all = need == sm_in;
    bits = sh;
    __syncthreads();
  }
  // Each thread a contiguous run of pages: counts, one scan, and out.
  const int run = (N + kTopThreads - 1) / kTopThreads;
  const int i0 = min(N, tid * run), i1 = min(N, i0 + run);
  int more = 0, same = 0, total;
  for (int i = i0; i < i1; ++i) {
    const u64 k = bits == 64 ? 0ULL : keys[i] >> bits;
    more += k > prefix;
    same += k == prefix;
  }
  const int more0 = cta_scan(more, &total);
  const int same0 = cta_scan(same, &total);
  int at = more0, eq = same0;
  for (int i = i0; i < i1; ++i) {
    const u64 k = bits == 64 ? 0ULL : keys[i] >> bits;
    const bool gt = k > prefix, take = gt || (k == prefix && (all || eq < need));
    if (take) out[at + min(eq, need)] = i;
    at += gt;
    eq += k == prefix;
  }
}

template <typename Q, typename E, int NH>
cudaError_t launch_score(const SelectArgs& s, int ctas, cudaStream_t stream) {
  return launch_pdl(page_score_kernel<Q, E, NH>, dim3(ctas), dim3(kScoreThreads),
                    static_cast<size_t>(s.a.B + 1) * 4, stream, s);
}
template <typename Q, typename E>
cudaError_t launch_score(const SelectArgs& s, int ctas, cudaStream_t stream) {
  if (s.G <= 4) return launch_score<Q, E, 4>(s, ctas, stream);
  if (s.G <= 8) return launch_score<Q, E, 8>(s, ctas, stream);
  return launch_score<Q, E, 16>(s, ctas, stream);
}

}  // namespace

cudaError_t launch_page_select(const void* q, long long q_stride, int G, const PageArgs& a, mova_dtype dt,
                               const void* lo, const void* hi, int top, int32_t* picked, const PageWs& ws,
                               cudaStream_t stream) {
  const SelectArgs s{a, q, q_stride, G, top, lo, hi, ws.keys, ws.bad, picked};
  const long long most = (static_cast<long long>(a.B) * a.kv * a.max_pages + kScoreWarps - 1) / kScoreWarps;
  long long ctas = sm_count() * static_cast<long long>(kScorePerSm);
  if (ctas > kMaxWorkers) ctas = kMaxWorkers;
  if (ctas > most) ctas = most < 1 ? 1 : most;
  const int n = static_cast<int>(ctas);
  cudaError_t err;
  if (dt == MOVA_F32) err = launch_score<float, float>(s, n, stream);
  else if (dt == MOVA_BF16) err = launch_score<__nv_bfloat16, __nv_bfloat16>(s, n, stream);
  else err = launch_score<__nv_bfloat16, uint8_t>(s, n, stream);
  if (err != cudaSuccess) return err;
  return launch_pdl(page_top_kernel, dim3(a.B * a.kv), dim3(kTopThreads), 0, stream, s, n, ws.sb);
}

}  // namespace mova

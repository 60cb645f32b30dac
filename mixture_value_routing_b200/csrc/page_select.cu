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

// Four consecutive elements, as stored and in fp64.
template <typename E> struct Four;
template <> struct Four<float> {
  using Raw = uint4;
  static __device__ __forceinline__ void get(const Raw& u, double (&d)[4]) {
    d[0] = __uint_as_float(u.x), d[1] = __uint_as_float(u.y), d[2] = __uint_as_float(u.z), d[3] = __uint_as_float(u.w);
  }
};
template <> struct Four<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ void get(const Raw& u, double (&d)[4]) {
    d[0] = __uint_as_float(u.x << 16), d[1] = __uint_as_float(u.x & 0xffff0000u);
    d[2] = __uint_as_float(u.y << 16), d[3] = __uint_as_float(u.y & 0xffff0000u);
  }
};
template <> struct Four<uint8_t> {
  using Raw = uint32_t;
  static __device__ __forceinline__ void get(const Raw& u, double (&d)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      d[i] = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<uint8_t>(u >> (8 * i)), __NV_E4M3)));
  }
};

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
      typename Four<Q>::Raw raw[NH];
#pragma unroll
      for (int n = 0; n < NH; ++n)
        raw[n] = *reinterpret_cast<const typename Four<Q>::Raw*>(src + (n < s.G ? n : 0) * kHeadDim);
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        Four<Q>::get(raw[n], q[n]);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[n][i] = q[n][i] + 0.0;  // -0 counts as 0: its sign bit picks no bound
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
    // All pages' bounds are on their way before the first is used; a page that
    // is none reads page 0 and is dropped below.
    typename Four<E>::Raw raw_lo[kPages], raw_hi[kPages];
#pragma unroll
    for (int p = 0; p < kPages; ++p) {
      const int at = max(0, __shfl_sync(0xffffffffu, id, p));
      const long long off = (static_cast<long long>(at) * kv + h) * kHeadDim + 4 * lane;
      raw_lo[p] = *reinterpret_cast<const typename Four<E>::Raw*>(static_cast<const E*>(s.lo) + off);
      raw_hi[p] = *reinterpret_cast<const typename Four<E>::Raw*>(static_cast<const E*>(s.hi) + off);
    }
    double sum[32];
#pragma unroll
    for (int p = 0; p < kPages; ++p) {
      double lo[4], hi[4];
      Four<E>::get(raw_lo[p], lo);
      Four<E>::get(raw_hi[p], hi);
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        double x = 0.0;
#pragma unroll
        for (int i = 0; i < 4; ++i) x = fma(q[n][i], __double2hiint(q[n][i]) < 0 ? lo[i] : hi[i], x);
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

// Exclusive prefix sum of x over the CTA.  `sums` is the caller's alone.
__device__ __forceinline__ int cta_scan(int x, int (&sums)[kTopThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int before = 0;
#pragma unroll
  for (int w = 0; w < kTopThreads / 32; ++w)
    if (w < warp) before += sums[w];
  return before + incl - x;
}

// The keys of one (request, KV head): thread t holds keys t + i * kTopThreads,
// the first kHeld of them in registers, the rest (long requests) in memory.
constexpr int kHeld = 16;
struct Keys {
  const u64* from;
  int N;
  u64 held[kHeld];
  __device__ __forceinline__ Keys(const u64* p, int n) : from(p), N(n) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int at = threadIdx.x + i * kTopThreads;
      held[i] = at < N ? from[at] : 0ULL;
    }
  }
  template <typename F> __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (static_cast<int>(threadIdx.x) + i * kTopThreads < N) f(held[i]);
    for (int at = threadIdx.x + kHeld * kTopThreads; at < N; at += kTopThreads) f(from[at]);
  }
};

__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectArgs s, int score_ctas, StatusBlock* sb) {
  __shared__ int hist[kBins];
  __shared__ u64 sm_min[kTopThreads / 32], sm_max[kTopThreads / 32];
  __shared__ int sums[kTopThreads / 32], sums2[kTopThreads / 32];
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
  const Keys keys(s.keys + static_cast<long long>(blockIdx.x) * s.a.max_pages, N);

  u64 least = ~0ULL, most_inv = ~0ULL;  // the greatest, as the least complement
  keys.each([&](u64 k) {
    least = k < least ? k : least;
    most_inv = ~k < most_inv ? ~k : most_inv;
  });
  least = warp_min(least);
  most_inv = warp_min(most_inv);
  if (lane == 0) sm_min[warp] = least, sm_max[warp] = most_inv;
  for (int i = tid; i < kBins; i += kTopThreads) hist[i] = 0;
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
    keys.each([&](u64 k) {
      if (bits == 64 || (k >> bits) == prefix) atomicAdd(&hist[static_cast<int>(k >> sh) & ((1 << width) - 1)], 1);
    });
    __syncthreads();
    // Thread i holds the bins below kBins - 4 i, from the top.
    constexpr int kPer = kBins / kTopThreads;
    int c[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = hist[kBins - 1 - (tid * kPer + j)];
      mine += c[j];
    }
    int above = cta_scan(mine, sums);  // its barrier: every bin has been read
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (above < need && need <= above + c[j]) sm_bin = kBins - 1 - (tid * kPer + j), sm_above = above, sm_in = c[j];
      above += c[j];
      hist[kBins - 1 - (tid * kPer + j)] = 0;  // for the next digit
    }
    __syncthreads();
    prefix = (prefix << width) | static_cast<u64>(sm_bin);
    need -= sm_above;
    all = need == sm_in;
    bits = sh;
    __syncthreads();
  }
  // Places, in page order: kTopThreads pages at a time.
  int base_more = 0, base_same = 0;
  for (int at0 = 0, i = 0; at0 < N; at0 += kTopThreads, ++i) {
    const int at = at0 + tid;
    u64 k = 0ULL;
    if (i < kHeld) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (j == i) k = keys.held[j];
    } else if (at < N) {
      k = keys.from[at];
    }
    k >>= bits;
    const bool more = at < N && k > prefix, same = at < N && k == prefix;
    const unsigned m = __ballot_sync(0xffffffffu, more), e = __ballot_sync(0xffffffffu, same);
    const unsigned below = (1u << lane) - 1;
    if (lane == 0) sums[warp] = __popc(m), sums2[warp] = __popc(e);
    __syncthreads();
    int more_at = base_more + __popc(m & below), same_at = base_same + __popc(e & below);
#pragma unroll
    for (int w = 0; w < kTopThreads / 32; ++w) {
      const int x = sums[w], y = sums2[w];
      if (w < warp) more_at += x, same_at += y;
      base_more += x, base_same += y;
    }
    if (more || (same && (all || same_at < need))) out[more_at + min(same_at, need)] = at;
    __syncthreads();
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

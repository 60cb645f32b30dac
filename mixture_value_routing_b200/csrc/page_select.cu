// The cache pages worth reading for a query, by per-page key bounds.
//
//   score(page) = max over the KV head's query heads h of
//                 sum_d q[h, d] * (q[h, d] < 0 ? lo[page, d] : hi[page, d])
//
// and, of the request's full pages, the `top - 1` greatest (ties: the lower
// page number), with the last page always, in ascending order.
//
// Scores: the formula is q+ . hi + q- . lo with q split by sign, a product of
// (heads) x (2 * 128) by (2 * 128) x (pages).  Neighbouring scores decide what is
// read, so the choice is that of fp64 scores: with fp32 ones it would depend on
// the order of their sums.  fp32 pages are scored in fp64 (matrix instructions
// m8n8k4, 8 heads by 8 pages), which the fp64 rate bounds.  bf16 and E4M3 pages
// are screened first, in fp32 by mma.m16n8k16 with a bound on each score's
// error, as fast as their bounds can be read; the selection scores again in
// fp64 the few pages whose side of the border the errors leave open (262144
// tokens in 4 rows: about a dozen of 4095 pages a row).
//
// Selection: one CTA per (request, KV head) finds the K-th greatest score, by a
// histogram of the screened scores, or by radix search of fp64 ones from below
// the bits that the least and the greatest share.  Latency bounds it: a warp
// owns a contiguous run of pages, so that placing them in order needs one
// barrier.  No atomics decide an order.
//
// Measured, both kernels: 4 rows of 262144 tokens in pages of 64, 4 KV heads (34
// MB of bounds): 18 us, 25 with all scores in fp64; one row of 524288 tokens in
// pages of 16, 8 heads (134 MB): 53 us, 97 in fp64.  The error bound goes by the
// greatest bound of a page, and the border's width by the greatest error of a row:
// 57 us with bounds of one size, 78 with four channels 20 larger, but 1.6 ms, all
// scored in fp64 by the selection, where one page's bounds are 2^8 times as large,
// where 2048 pages are taken of those with the four channels, or where all bounds
// are equal (4096 pages: 0.27 ms).
#include <math.h>

#include <algorithm>

#include "paged.cuh"

namespace mova {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
// CTAs of the score kernel an SM: by the registers of its NT tiles of heads.
constexpr int score_per_sm(int NT) { return NT == 1 ? 3 : 2; }
constexpr int kDigit = 8;
constexpr int kBins = 1 << kDigit;

using u64 = unsigned long long;

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

__device__ __forceinline__ double value(float x) { return x; }

__device__ __forceinline__ int pages_of(const PageArgs& a, int b) {
  const int len = clamp_len(a.lens[b], a.max_pages, a.shift);
  return (len + (1 << a.shift) - 1) >> a.shift;
}

// c (8 heads x 8 pages) += a (8 heads x 4 dimensions) b (4 dimensions x 8 pages).
__device__ __forceinline__ void mma884(double (&c)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
               : "+d"(c[0]), "+d"(c[1]) : "d"(a), "d"(b));
}

// The dimensions of a lane (t = lane & 3) come in chunks of 16 stored bytes:
// chunk i holds dimensions (t + 4 i) * kPer + {0 .. kPer - 1}.
template <typename E> struct Chunk {
  static constexpr int kPer = 16 / sizeof(E);
  static constexpr int kCount = kHeadDim / kPer / 4;
};

// Where a batch of pages lies: its request, its first page, and the full pages
// of the request, which are read again only for another request.
struct At { int b = -1, page0 = 0, pages = 0; };
__device__ __forceinline__ At locate(const PageArgs& a, const int* pre, At r, int u, int batch) {
  if (r.b < 0 || u >= pre[r.b + 1]) {
    r.b = request_of(pre, a.B, u);
    r.pages = pages_of(a, r.b) - 1;
  }
  r.page0 = (u - pre[r.b]) * batch;
  return r;
}
// What warp w of W does for KV head h: batches [u0, u1) of them all.  Warps in a
// row have the heads in turn, then the heads' next shares.
struct Share { int u0, u1; };
__device__ __forceinline__ Share share_of_head(int U, int kv, int h, int w, int W) {
  const int shares = W >= kv ? (W - h + kv - 1) / kv : 1, j = w / kv;
  return Share{static_cast<int>(static_cast<long long>(j) * U / shares),
               static_cast<int>(static_cast<long long>(j + 1) * U / shares)};
}
// Page `i` of a batch as a page number, -1 if it is none.
__device__ __forceinline__ int look_up(const PageArgs& a, const At& r, int i, int* bad) {
  if (r.page0 + i >= r.pages) return -1;
  const int id = a.table[r.b * a.table_stride + r.page0 + i];
  if (id >= 0 && id < a.num_pages) return id;
  atomicMin(bad, r.b);
  return -1;
}
// Prefix of the batches of the requests that have a choice of pages.
__device__ __forceinline__ void scan_batches(const SelectArgs& s, int* pre, int batch, int* bad) {
  request_scan<kScoreThreads>(s.a.B, pre, [&](int b) {
    const int len = s.a.lens[b];
    if (clamp_len(len, s.a.max_pages, s.a.shift) != len) atomicMin(bad, b);
    const int n = pages_of(s.a, b);
    return n > s.top ? (n - 1 + batch - 1) / batch : 0;
  });
}

// ---- fp32 pages: scores in fp64 ---------------------------------------------------

// NT: tiles of 8 heads.
template <int NT>
__global__ void __launch_bounds__(kScoreThreads, score_per_sm(NT)) page_score_kernel(const SelectArgs s) {
  using C = Chunk<float>;
  constexpr int kWords = C::kCount * 4;  // a lane's bounds
  constexpr int kPages = 8;              // of one batch
  extern __shared__ int pre[];
  __shared__ int sm_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kv = s.a.kv, G = s.G;
  if (tid == 0) sm_bad = kNoBad;
  pdl_wait();
  __syncthreads();
  scan_batches(s, pre, kPages, &sm_bad);
  const int W = gridDim.x * kScoreWarps, w = blockIdx.x * kScoreWarps + warp;

  // This lane's first bounds in page `id`; a page that is none reads page 0, and
  // its score is dropped.
  auto offset = [&](int h, int id) {
    return (static_cast<long long>(max(id, 0)) * kv + h) * kHeadDim + t * C::kPer;
  };
  float lo[kWords], hi[kWords];
  auto load = [&](long long off, int i) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(s.lo) + off + i * 4 * C::kPer);
    const float4 y = *reinterpret_cast<const float4*>(static_cast<const float*>(s.hi) + off + i * 4 * C::kPer);
    lo[4 * i] = x.x, lo[4 * i + 1] = x.y, lo[4 * i + 2] = x.z, lo[4 * i + 3] = x.w;
    hi[4 * i] = y.x, hi[4 * i + 1] = y.y, hi[4 * i + 2] = y.z, hi[4 * i + 3] = y.w;
  };

  float q[NT][kWords];
  for (int h = w % kv; h < kv; h += W) {
    const auto [u0, u1] = share_of_head(pre[s.a.B], kv, h, w, W);
    // Bounds are loaded one batch ahead, page numbers two.
    At at, next, later;
    int id = -1, next_id = -1, later_id = -1, row = -1;
    if (u0 < u1) {
      at = locate(s.a, pre, at, u0, kPages);
      id = look_up(s.a, at, g, &sm_bad);
      if (u0 + 1 < u1) {
        next = locate(s.a, pre, at, u0 + 1, kPages);
        next_id = look_up(s.a, next, g, &sm_bad);
      }
      const long long off = offset(h, id);
#pragma unroll
      for (int i = 0; i < C::kCount; ++i) load(off, i);
    }
    for (int u = u0; u < u1; ++u) {
      const bool more = u + 1 < u1;
      if (u + 2 < u1) {
        later = locate(s.a, pre, next, u + 2, kPages);
        later_id = look_up(s.a, later, g, &sm_bad);
      }
      if (at.b * kv + h != row) {
        row = at.b * kv + h;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int head = min(n * 8 + g, G - 1);  // rows past the last head repeat it and are dropped
          const float* src = static_cast<const float*>(s.q) + at.b * s.q_stride +
                             (static_cast<long long>(h) * G + head) * kHeadDim + t * C::kPer;
#pragma unroll
          for (int i = 0; i < C::kCount; ++i) {
            const float4 x = *reinterpret_cast<const float4*>(src + i * 4 * C::kPer);
            q[n][4 * i] = x.x, q[n][4 * i + 1] = x.y, q[n][4 * i + 2] = x.z, q[n][4 * i + 3] = x.w;
          }
        }
      }
      // Four sums of 16 products of 4 dimensions each, so that products need not
      // wait for one another; a chunk's registers take the next pages' bounds as
      // soon as it is used.
      double c[NT][4][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) c[n][x][0] = c[n][x][1] = 0.0;
      const long long next_off = more ? offset(h, next_id) : 0;
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const double dl = lo[k], dh = hi[k];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const double d = q[n][k];
          mma884(c[n][2 * (k & 1)], d < 0.0 ? 0.0 : d, dh);
          mma884(c[n][2 * (k & 1) + 1], d < 0.0 ? d : 0.0, dl);
        }
        if (more && (k & 3) == 3) load(next_off, k >> 2);
      }
      // This lane: heads g (+ 8), pages 2 t and 2 t + 1.
      u64 key[2] = {0ULL, 0ULL};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        double sum[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) sum[x] = (c[n][0][x] + c[n][1][x]) + (c[n][2][x] + c[n][3][x]);
        const bool here = n * 8 + g < G;
        // NaN may come of an infinite bound that the query's sign does not use
        // (0 * inf): those scores are formed again without it.
        unsigned odd = __ballot_sync(0xffffffffu, here && (sum[0] != sum[0] || sum[1] != sum[1]));
        while (odd != 0u) {
          const int from = __ffs(odd) - 1, head = n * 8 + (from >> 2);
          odd &= odd - 1;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int p = max(0, __shfl_sync(0xffffffffu, id, (2 * (from & 3) + x) * 4));
            const long long off = (static_cast<long long>(p) * kv + h) * kHeadDim + 4 * lane;
            const float* src = static_cast<const float*>(s.q) + at.b * s.q_stride +
                               (static_cast<long long>(h) * G + head) * kHeadDim + 4 * lane;
            double v = 0.0;
            for (int i = 0; i < 4; ++i) {
              const double d = src[i];
              v = fma(d, value(static_cast<const float*>(d < 0.0 ? s.lo : s.hi)[off + i]), v);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == from && sum[x] != sum[x]) sum[x] = v;
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const u64 mine = here ? sortable(sum[x]) : 0ULL;
          key[x] = mine > key[x] ? mine : key[x];
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          const u64 other = __shfl_xor_sync(0xffffffffu, key[x], o);
          key[x] = other > key[x] ? other : key[x];
        }
        const int p = 2 * t + x;
        const bool there = __shfl_sync(0xffffffffu, id, p * 4) >= 0;
        if (g == 0 && at.page0 + p < at.pages)
          s.keys[static_cast<long long>(row) * s.a.max_pages + at.page0 + p] = there ? key[x] : 0ULL;
      }
      at = next, next = later;
      id = next_id, next_id = later_id;
    }
  }
  pdl_trigger();
  __syncthreads();
  if (tid == 0) s.bad[blockIdx.x] = sm_bad;
}

// ---- bf16 and E4M3 pages: scores screened in fp32 ------------------------------------

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The operand words of one loaded word of bounds: itself (two bf16), or two
// words of two fp16 (four E4M3); and the greatest magnitude of such a word and
// another's, NaN if either has one.
template <typename E> struct Bound;
template <> struct Bound<__nv_bfloat16> {
  static constexpr int kWords = 1;
  static __device__ __forceinline__ uint32_t get(uint32_t w, int) { return w; }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t w) {
    w &= 0x7fff7fffu;
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&w));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float widest(uint32_t a) {
    return max_nan(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
};
template <> struct Bound<uint8_t> {
  static constexpr int kWords = 2;
  static __device__ __forceinline__ uint32_t get(uint32_t w, int i) { return i == 0 ? e4m3_lo(w) : e4m3_hi(w); }
  static __device__ __forceinline__ uint32_t most(uint32_t a, uint32_t w) {
    w &= 0x7fff7fffu;
    const __half2 r = __hmax2_nan(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&w));
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  static __device__ __forceinline__ float widest(uint32_t a) {
    const __half2 h = *reinterpret_cast<const __half2*>(&a);
    return max_nan(__low2float(h), __high2float(h));
  }
};

// Rounding of a screened score, relative to sum |q_d| max |bound_d|.  256
// products, exact, are added in fp32 in 16 steps whose roundings are at most
// 2^-22 of the sums' magnitudes each on the tensor cores: below 2^-17 with the
// additions within a step; q in fp16 (E4M3) adds 2^-18.  Taken ten times as large.
constexpr float kScreenError = 0x1p-13f;
// No sum of products that are below this in all can leave fp32's range, nor a score
// with its error the range in which the selection steps; others are not screened.
constexpr float kScreenMost = 0x1p126f;

// NT: tiles of 8 heads.  16 pages (rows) by 8 heads (columns): a lane loads 16
// bytes a time of pages g and g + 8, whose words are row operands as they are
// (E4M3: as fp16), and has q ordered to match, its positive and negative parts
// apart for the upper and the lower bounds.
template <typename E, int NT>
__global__ void __launch_bounds__(kScoreThreads, score_per_sm(NT)) page_screen_kernel(const SelectArgs s) {
  using C = Chunk<E>;
  constexpr bool kHalf = sizeof(E) == 1;
  constexpr int kPages = 16;
  extern __shared__ int pre[];
  __shared__ int sm_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int kv = s.a.kv, G = s.G;
  if (tid == 0) sm_bad = kNoBad;
  pdl_wait();
  __syncthreads();
  scan_batches(s, pre, kPages, &sm_bad);
  const int W = gridDim.x * kScoreWarps, w = blockIdx.x * kScoreWarps + warp;

  uint32_t pos[NT][16], neg[NT][16];  // two elements of q each: steps of 16 dimensions, two words a step
  float factor[NT][2], reach = 0.0f;  // from a sum to a score, columns 2 t and 2 t + 1; sum |q_d|, the largest head's
  int row = -1;
  // Bounds of pages g and g + 8; a page that is none reads page 0, and its score is dropped.
  uint4 raw[2][C::kCount][2];  // lower and upper bounds
  auto offset = [&](int h, int id) {
    return (static_cast<long long>(max(id, 0)) * kv + h) * kHeadDim + t * C::kPer;
  };
  auto load = [&](int bound, int i, long long off0, long long off1) {
    const E* from = static_cast<const E*>(bound == 0 ? s.lo : s.hi) + i * 4 * C::kPer;
    raw[bound][i][0] = *reinterpret_cast<const uint4*>(from + off0);
    raw[bound][i][1] = *reinterpret_cast<const uint4*>(from + off1);
  };
  for (int h = w % kv; h < kv; h += W) {
    const auto [u0, u1] = share_of_head(pre[s.a.B], kv, h, w, W);
    // Bounds are loaded one batch ahead, page numbers two.
    At at, next, later;
    int id0 = -1, id1 = -1, next0 = -1, next1 = -1, later0 = -1, later1 = -1;
    if (u0 < u1) {
      at = locate(s.a, pre, at, u0, kPages);
      id0 = look_up(s.a, at, g, &sm_bad), id1 = look_up(s.a, at, g + 8, &sm_bad);
      if (u0 + 1 < u1) {
        next = locate(s.a, pre, at, u0 + 1, kPages);
        next0 = look_up(s.a, next, g, &sm_bad), next1 = look_up(s.a, next, g + 8, &sm_bad);
      }
#pragma unroll
      for (int i = 0; i < C::kCount; ++i) {
        load(0, i, offset(h, id0), offset(h, id1));
        load(1, i, offset(h, id0), offset(h, id1));
      }
    }
    for (int u = u0; u < u1; ++u) {
      const bool more = u + 1 < u1;
      if (u + 2 < u1) {
        later = locate(s.a, pre, next, u + 2, kPages);
        later0 = look_up(s.a, later, g, &sm_bad), later1 = look_up(s.a, later, g + 8, &sm_bad);
      }
      if (at.b * kv + h != row) {
        row = at.b * kv + h;
        reach = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int head = n * 8 + g;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(s.q) + at.b * s.q_stride +
                                     (static_cast<long long>(h) * G + min(head, G - 1)) * kHeadDim + t * C::kPer;
          uint32_t words[16];
#pragma unroll
          for (int i = 0; i < C::kCount; ++i)
#pragma unroll
            for (int v = 0; v < 4 / C::kCount; ++v) {
              const uint4 x = *reinterpret_cast<const uint4*>(src + i * 4 * C::kPer + v * 8);
              uint32_t* to = &words[(i * (4 / C::kCount) + v) * 4];
              to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
            }
          float sum = 0.0f, big = 0.0f;
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float a = fabsf(__uint_as_float(words[x] << 16)), b = fabsf(__uint_as_float(words[x] & 0xffff0000u));
            sum += a + b;
            big = fmaxf(big, fmaxf(a, b));
          }
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
          }
          float up = 1.0f;
          if constexpr (kHalf) {
            // As in the attention: a power of two takes the row's largest element to [1, 2).
            int e = static_cast<int>(__float_as_uint(big) >> 23);
            e = e < 1 ? 127 : (e > 253 ? 253 : e);
            const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
            up = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
            for (int x = 0; x < 16; ++x)
              words[x] = pack_f16(__uint_as_float(words[x] << 16) * down, __uint_as_float(words[x] & 0xffff0000u) * down);
          }
          factor[n][0] = __shfl_sync(0xffffffffu, up, (2 * t) * 4);
          factor[n][1] = __shfl_sync(0xffffffffu, up, (2 * t + 1) * 4);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const uint32_t sign = ((words[x] >> 15) & 0x00010001u) * 0xffffu;  // halves below zero
            pos[n][x] = words[x] & ~sign;
            neg[n][x] = words[x] & sign;
          }
          reach = max_nan(reach, head < G ? sum : 0.0f);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) reach = max_nan(reach, __shfl_xor_sync(0xffffffffu, reach, o));
      }
      float c[NT][2][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 8; ++x) c[n][x >> 2][x & 3] = 0.0f;
      uint32_t most0 = 0u, most1 = 0u;  // the greatest magnitudes, pages g and g + 8
      // A chunk's registers take the next pages' bounds as soon as it is used.
      const long long next_off0 = offset(h, next0), next_off1 = offset(h, next1);
#pragma unroll
      for (int i = 0; i < C::kCount; ++i)
#pragma unroll
        for (int bound = 0; bound < 2; ++bound) {
          const uint32_t x[4] = {raw[bound][i][0].x, raw[bound][i][0].y, raw[bound][i][0].z, raw[bound][i][0].w};
          const uint32_t y[4] = {raw[bound][i][1].x, raw[bound][i][1].y, raw[bound][i][1].z, raw[bound][i][1].w};
          // Two operand words make a step of 16 dimensions.
#pragma unroll
          for (int k = 0; k < 2 * Bound<E>::kWords; ++k) {
            uint32_t a[2][2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const int word = (2 * k + z) / Bound<E>::kWords, part = (2 * k + z) % Bound<E>::kWords;
              a[0][z] = Bound<E>::get(x[word], part);
              a[1][z] = Bound<E>::get(y[word], part);
              most0 = Bound<E>::most(most0, a[0][z]);
              most1 = Bound<E>::most(most1, a[1][z]);
            }
            const int step = i * 2 * Bound<E>::kWords + k;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t* q = bound == 0 ? neg[n] : pos[n];
              mma16816<kHalf>(c[n][bound], a[0][0], a[1][0], a[0][1], a[1][1], q[2 * step], q[2 * step + 1]);
            }
          }
          if (more) load(bound, i, next_off0, next_off1);
        }
      // Columns 2 t and 2 t + 1 of rows g and g + 8: the best head of each page.
      float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float v = (c[n][0][x] + c[n][1][x]) * factor[n][x & 1];
          if (n * 8 + 2 * t + (x & 1) < G) best[x >> 1] = max_nan(best[x >> 1], v);
        }
      float wide[2] = {Bound<E>::widest(most0), Bound<E>::widest(most1)};
#pragma unroll
      for (int o = 1; o < 4; o <<= 1)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          best[x] = max_nan(best[x], __shfl_xor_sync(0xffffffffu, best[x], o));
          wide[x] = max_nan(wide[x], __shfl_xor_sync(0xffffffffu, wide[x], o));
        }
      if (t < 2) {
        const int page = at.page0 + g + 8 * t;
        const float far = t == 0 ? wide[0] : wide[1];
        const float error = reach * far < kScreenMost ? fmaf(kScreenError * reach, far, 0x1p-100f) : INFINITY;
        const float2 out = (t == 0 ? id0 : id1) < 0 ? make_float2(0.0f, -1.0f)
                                                    : make_float2(t == 0 ? best[0] : best[1], error);
        if (page < at.pages)
          reinterpret_cast<float2*>(s.keys)[static_cast<long long>(row) * s.a.max_pages + page] = out;
      }
      at = next, next = later;
      id0 = next0, id1 = next1, next0 = later0, next1 = later1;
    }
  }
  pdl_trigger();
  __syncthreads();
  if (tid == 0) s.bad[blockIdx.x] = sm_bad;
}

// ---- Selection -------------------------------------------------------------------------

__device__ __forceinline__ u64 warp_min(u64 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const u64 y = __shfl_xor_sync(0xffffffffu, x, o);
    x = y < x ? y : x;
  }
  return x;
}

constexpr int kHeld = 16;  // keys of a thread in registers; a long request's others are read again

// Radix search among 32-bit values for the `need` greatest: each(f) calls f for
// every value of this thread, whose upper `bits` are searched.  Returns how
// many of them are left open; *prefix the bits above those that the least of
// the greatest has, *need how many to take of the values with that prefix,
// *all whether those are all there are.  hist: one zeroed row for each digit.
// Every warp reads the counts and comes to the same answer, so a digit costs
// one barrier.
template <typename Each>
__device__ __forceinline__ int radix_search(Each each, int bits, int (*hist)[kBins], uint32_t* prefix, int* need,
                                            bool* all) {
  const int lane = threadIdx.x & 31;
  *prefix = 0;
  *all = false;
  for (int digit = 0; bits > 0 && !*all; ++digit) {
    const int width = min(bits, kDigit), low = bits - width;
    const uint32_t mask = (1u << width) - 1, above_mask = bits == 32 ? 0u : ~0u << bits;
    const uint32_t want = bits == 32 ? 0u : *prefix << bits;
    each([&](uint32_t v) {
      if ((v & above_mask) == want) atomicAdd(&hist[digit][(v >> low) & mask], 1);
    });
    __syncthreads();
    // Lane i holds the kPer bins below kBins - kPer * i, from the top.
    constexpr int kPer = kBins / 32;
    const int top_bin = kBins - 1 - lane * kPer;
    int c[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = hist[digit][top_bin - j];
      mine += c[j];
    }
    int above = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, above, o);
      if (lane >= o) above += up;
    }
    above -= mine;
    int bin = 0, left = 0, in = 0;
    bool here = false;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (above < *need && *need <= above + c[j]) here = true, bin = top_bin - j, left = *need - above, in = c[j];
      above += c[j];
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    bin = __shfl_sync(0xffffffffu, bin, from);
    *need = __shfl_sync(0xffffffffu, left, from);
    *all = *need == __shfl_sync(0xffffffffu, in, from);
    *prefix = (*prefix << width) | static_cast<uint32_t>(bin);
    bits = low;
  }
  return bits;
}

// What the selection kernels share in shared memory.
template <int kThreads> struct TopShared {
  int hist[2 * 32 / kDigit][kBins];
  u64 least[kThreads / 32], most[kThreads / 32];
  int2 count[kThreads / 32];
};

// The `need` greatest of N sortable scores (ties: the lower page), as page
// numbers in ascending order.  sh.hist is zero, and not again afterwards.
template <int kTopThreads>
__device__ __forceinline__ void top_of(const u64* keys, int N, int need, int32_t* out, TopShared<kTopThreads>& sh) {
  constexpr int kTopWarps = kTopThreads / 32, kDigits = 32 / kDigit;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Each warp has a contiguous run of `span` stripes of 32 pages.
  const int span = (N + kTopThreads - 1) / kTopThreads, first = warp * span * 32 + lane;

  // The least and the greatest score: above the bits in which they differ, all agree.
  u64 held[kHeld], least = ~0ULL, most_inv = ~0ULL;  // the greatest, as the least complement
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = i < span && first + 32 * i < N ? keys[first + 32 * i] : 0ULL;
  // Calls f(key, i) for every key i of this thread that is not held; loads eight
  // at a time.
  auto others = [&](auto f) {
    constexpr int kAhead = 8;
    for (int i0 = kHeld; i0 < span; i0 += kAhead) {
      u64 k[kAhead];
#pragma unroll
      for (int x = 0; x < kAhead; ++x) {
        const int at = first + 32 * (i0 + x);
        k[x] = i0 + x < span && at < N ? keys[at] : 0ULL;
      }
#pragma unroll
      for (int x = 0; x < kAhead; ++x)
        if (i0 + x < span) f(k[x], i0 + x);
    }
  };
  auto see = [&](u64 k) {
    least = k < least ? k : least;
    most_inv = ~k < most_inv ? ~k : most_inv;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (i >= span) break;
    if (first + 32 * i < N) see(held[i]);
  }
  others([&](u64 k, int i) {
    if (first + 32 * i < N) see(k);
  });
  least = warp_min(least);
  most_inv = warp_min(most_inv);
  if (lane == 0) sh.least[warp] = least, sh.most[warp] = most_inv;
  __syncthreads();
  least = warp_min(sh.least[lane % kTopWarps]);
  most_inv = warp_min(sh.most[lane % kTopWarps]);
  const u64 differ = least ^ ~most_inv;
  const int open = differ == 0 ? 0 : 64 - __clzll(static_cast<long long>(differ));

  // The upper 32 of the open bits settle it, unless scores agree in all of
  // them; then the rest does, and equal scores go by page number.
  const int up = max(1, open);
  auto upper = [&](u64 k) { return static_cast<uint32_t>((k << (64 - up)) >> 32); };
  const uint32_t rest = open > 32 ? (open == 64 ? ~0u : (1u << (open - 32)) - 1) : 0u;
  uint32_t v[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) v[i] = upper(held[i]);
  bool all;
  uint32_t p1, p2 = 0;
  const int r1 = radix_search(
      [&](auto f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          if (i >= span) break;
          if (first + 32 * i < N) f(v[i]);
        }
        others([&](u64 k, int i) {
          if (first + 32 * i < N) f(upper(k));
        });
      },
      open == 0 ? 0 : 32, sh.hist, &p1, &need, &all);
  const bool second = open > 32 && !all;
  int r2 = 0;
  if (second)
    r2 = radix_search(
        [&](auto f) {
          for (int i = 0; i < span; ++i) {
            if (first + 32 * i >= N) continue;
            const u64 k = keys[first + 32 * i];
            if (upper(k) == p1) f(static_cast<uint32_t>(k) & rest);
          }
        },
        open - 32, sh.hist + kDigits, &p2, &need, &all);

  // Whether key i of this thread is above the threshold (1), at it (2), or neither.
  auto place = [&](int i, uint32_t value) {
    if (first + 32 * i >= N) return 0;
    uint32_t x = open == 0 ? 0u : value >> r1, p = p1;
    if (second && x == p) x = (static_cast<uint32_t>(keys[first + 32 * i]) & rest) >> r2, p = p2;
    return x > p ? 1 : x == p ? 2 : 0;
  };
  // The warps' counts, one barrier, and out, in page order.
  int2 mine = make_int2(0, 0);
  auto count = [&](int at) {
    mine.x += __popc(__ballot_sync(0xffffffffu, at == 1));
    mine.y += __popc(__ballot_sync(0xffffffffu, at == 2));
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (i >= span) break;
    count(place(i, v[i]));
  }
  others([&](u64 k, int i) { count(place(i, upper(k))); });
  if (lane == 0) sh.count[warp] = mine;
  __syncthreads();
  int more = 0, same = 0;
  for (int w = 0; w < warp; ++w) more += sh.count[w].x, same += sh.count[w].y;
  const unsigned below = (1u << lane) - 1;
  auto write = [&](int i, int at) {
    const unsigned m = __ballot_sync(0xffffffffu, at == 1), e = __ballot_sync(0xffffffffu, at == 2);
    const int more_at = more + __popc(m & below), same_at = same + __popc(e & below);
    if (at == 1 || (at == 2 && (all || same_at < need))) out[more_at + min(same_at, need)] = first + 32 * i;
    more += __popc(m);
    same += __popc(e);
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    if (i >= span) break;
    write(i, place(i, v[i]));
  }
  others([&](u64 k, int i) { write(i, place(i, upper(k))); });
}

// The status of a selection, from what the score kernel's CTAs saw.  One warp.
__device__ __forceinline__ void write_status(const int32_t* seen, int ctas, StatusBlock* sb) {
  const int lane = threadIdx.x & 31;
  int bad = kNoBad;
  for (int i = lane; i < ctas; i += 32) bad = min(bad, seen[i]);
  bad = __reduce_min_sync(0xffffffffu, bad);
  if (lane == 0) {
    sb->code = bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
    sb->detail = bad == kNoBad ? 0 : bad;
  }
}

// Rows that need no choice: writes them and returns 0.  Else the row's pages, the
// last of which is written.
template <int kThreads> __device__ __forceinline__ int few_pages(const SelectArgs& s, int32_t* out) {
  const int n = pages_of(s.a, blockIdx.x / s.a.kv), top = s.top;
  if (n <= top) {
    for (int i = threadIdx.x; i < top; i += kThreads) out[i] = i < n ? i : -1;
    return 0;
  }
  if (threadIdx.x == 0) out[top - 1] = n - 1;
  return top == 1 ? 0 : n;
}

// From fp64 scores (fp32 pages).
template <int kThreads>
__global__ void __launch_bounds__(kThreads) page_top_kernel(const SelectArgs s, int score_ctas, StatusBlock* sb) {
  __shared__ TopShared<kThreads> sh;
  const int tid = threadIdx.x;
  for (int i = tid; i < static_cast<int>(sizeof(sh.hist) / 4); i += kThreads) (&sh.hist[0][0])[i] = 0;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {  // not a row's: a row would end a microsecond later
    if (tid < 32) write_status(s.bad, score_ctas, sb);
    return;
  }
  int32_t* out = s.picked + static_cast<long long>(blockIdx.x) * s.top;
  const int n = few_pages<kThreads>(s, out);
  if (n > 0)
    top_of<kThreads>(s.keys + static_cast<long long>(blockIdx.x) * s.a.max_pages, n - 1, s.top - 1, out, sh);
}

// Four stored elements as fp32, exactly.
__device__ __forceinline__ float4 four(const __nv_bfloat16* from) {
  const uint2 w = *reinterpret_cast<const uint2*>(from);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u));
}
__device__ __forceinline__ float4 four(const uint8_t* from) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(from), lo = e4m3_lo(w), hi = e4m3_hi(w);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x, a.y, b.x, b.y);
}

// fp64 score of a page, in sortable form; by one warp, the same in every lane.
// Eight lanes have a head, so that four heads go at a time.
template <typename E>
__device__ __forceinline__ u64 exact_score(const SelectArgs& s, int b, int h, int page) {
  const int lane = threadIdx.x & 31, dim = 4 * (lane & 7);
  const int id = s.a.table[b * s.a.table_stride + page];
  if (id < 0 || id >= s.a.num_pages) return 0ULL;
  const long long off = (static_cast<long long>(id) * s.a.kv + h) * kHeadDim + dim;
  const __nv_bfloat16* q =
      static_cast<const __nv_bfloat16*>(s.q) + b * s.q_stride + static_cast<long long>(h) * s.G * kHeadDim + dim;
  float4 lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    lo[i] = four(static_cast<const E*>(s.lo) + off + 32 * i);
    hi[i] = four(static_cast<const E*>(s.hi) + off + 32 * i);
  }
  u64 best = 0ULL;
#pragma unroll 1
  for (int head0 = 0; head0 < s.G; head0 += 4) {
    const int head = min(head0 + (lane >> 3), s.G - 1);  // past the last, that one again
    double v[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 d = four(q + head * kHeadDim + 32 * i);
      v[0] = fma(static_cast<double>(d.x), static_cast<double>(d.x < 0.0f ? lo[i].x : hi[i].x), v[0]);
      v[1] = fma(static_cast<double>(d.y), static_cast<double>(d.y < 0.0f ? lo[i].y : hi[i].y), v[1]);
      v[2] = fma(static_cast<double>(d.z), static_cast<double>(d.z < 0.0f ? lo[i].z : hi[i].z), v[2]);
      v[3] = fma(static_cast<double>(d.w), static_cast<double>(d.w < 0.0f ? lo[i].w : hi[i].w), v[3]);
    }
    double sum = (v[0] + v[1]) + (v[2] + v[3]);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const u64 key = sortable(sum);
    best = key > best ? key : best;
  }
#pragma unroll
  for (int o = 8; o < 32; o <<= 1) {
    const u64 other = __shfl_xor_sync(0xffffffffu, best, o);
    best = other > best ? other : best;
  }
  return best;
}

// Sum over the block of x in the threads before this one, and *total of all.
// sums: one int a warp; a barrier before it is used again.
template <int kThreads> __device__ __forceinline__ int block_before(int x, int* sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int up = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += y;
  }
  if (lane == 31) sums[warp] = up;
  __syncthreads();
  const int of = lane < kThreads / 32 ? sums[lane] : 0;
  *total = __reduce_add_sync(0xffffffffu, of);
  return __reduce_add_sync(0xffffffffu, lane < warp ? of : 0) + up - x;
}

__device__ __forceinline__ uint32_t sortable32(float s) {
  const uint32_t b = __float_as_uint(s + 0.0f);
  return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_sortable(uint32_t v) { return __uint_as_float(v >> 31 ? v & 0x7fffffffu : ~v); }

constexpr int kStored = 32768;  // scores of a row in shared memory; a longer row's others are read again

// From screened scores (bf16 and E4M3 pages).  With e the largest error bound of
// the row and the K-th greatest fp32 score in [x, y], the K-th greatest fp64
// score lies in [x - e, y + e]: a page above y + 2 e is among the K greatest, one
// below x - 2 e is not, and the few between are scored again in fp64.  One
// histogram of kSteps equal steps from the least to the greatest score gives
// [x, y]: no score is beyond 2^13 e by the definition of e, so a step is at most
// 8 e, and mostly less than one.  Where more than kUnsure pages lie between, a
// score or a bound is not finite, or pages are missing, all pages are scored
// again: exact, but slow (above).
//
// The loops are left rolled where they can be: a CTA runs each once, so their
// instructions come from memory, and unrolled 16 times over registers, with a
// radix search, this kernel took twice the time (32768 pages: 50 us against 27).
template <typename E, int kThreads>
__global__ void __launch_bounds__(kThreads) page_pick_kernel(const SelectArgs s, int score_ctas, StatusBlock* sb) {
  constexpr int kWarps = kThreads / 32, kUnsure = 512, kSteps = 2048, kPer = kSteps / kThreads;
  extern __shared__ float score[];
  __shared__ union {
    TopShared<kThreads> top;
    struct {
      int hist[kSteps];
      u64 key[kUnsure];
      int page[kUnsure];
    } pick;
  } sh;
  __shared__ int sums[kWarps], counts[kWarps];
  __shared__ int sm_unsure, sm_odd, sm_step;
  __shared__ uint32_t sm_least, sm_most, sm_error;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kSteps; i += kThreads) sh.pick.hist[i] = 0;
  if (tid == 0) sm_unsure = sm_odd = 0, sm_least = ~0u, sm_most = sm_error = 0u;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == gridDim.x - 1) {
    if (warp == 0) write_status(s.bad, score_ctas, sb);
    return;
  }
  int32_t* out = s.picked + static_cast<long long>(blockIdx.x) * s.top;
  const int n = few_pages<kThreads>(s, out);
  if (n == 0) return;
  const int N = n - 1, K = s.top - 1, b = blockIdx.x / s.a.kv, h = blockIdx.x - b * s.a.kv;
  u64* keys = s.keys + static_cast<long long>(blockIdx.x) * s.a.max_pages;
  float2* screened = reinterpret_cast<float2*>(keys);

  // The scores; a page that is none has -inf.
  uint32_t least = ~0u, most = 0u, error = 0u;
  int real = 0;
  bool odd = false;
#pragma unroll 4
  for (int i = tid; i < N; i += kThreads) {
    const float2 x = screened[i];
    const bool none = x.y < 0.0f;
    if (!none) {
      odd |= !(fabsf(x.x) < INFINITY) || !(x.y < INFINITY);
      const uint32_t y = sortable32(x.x);
      least = min(least, y), most = max(most, y), error = max(error, __float_as_uint(x.y));
      ++real;
    }
    if (i < kStored) score[i] = none ? -INFINITY : x.x;
  }
  auto score_of = [&](int i) {
    if (i < kStored) return score[i];
    const float2 x = screened[i];
    return x.y < 0.0f ? -INFINITY : x.x;
  };
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  error = __reduce_max_sync(0xffffffffu, error);
  real = __reduce_add_sync(0xffffffffu, real);
  odd = __any_sync(0xffffffffu, odd);
  if (lane == 0) counts[warp] = real;
  __syncthreads();
  if (lane == 0) {
    atomicMin(&sm_least, least);
    atomicMax(&sm_most, most);
    atomicMax(&sm_error, error);
    if (odd) sm_odd = 1;
  }
  __syncthreads();
  const float low = from_sortable(sm_least), e = __uint_as_float(sm_error), range = from_sortable(sm_most) - low;
  real = __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[lane] : 0);
  bool again = sm_odd != 0 || real < K || !(range < INFINITY);

  // 0: not among the K greatest; 1: among them; 2: unsure.
  float from = 0.0f, above = 0.0f;
  auto side_of = [&](float z) { return z < from || z == -INFINITY ? 0 : z > above ? 1 : 2; };
  // Each warp has a contiguous run of stripes of 32 pages.
  const int stripes = (N + 31) >> 5, span = (stripes + kWarps - 1) / kWarps;
  const int run0 = warp * span, run1 = min(run0 + span, stripes);
  if (!again) {
    const bool flat = range <= e;  // one step
    const float scale = flat ? 0.0f : (kSteps - 1) / range, step = flat ? range : range / (kSteps - 1);
    // Steps from the greatest score down: monotone, as each rounding is.
#pragma unroll 4
    for (int i = tid; i < N; i += kThreads) {
      const float z = score_of(i);
      if (z != -INFINITY) atomicAdd(&sh.pick.hist[kSteps - 1 - min(static_cast<int>((z - low) * scale), kSteps - 1)], 1);
    }
    __syncthreads();
    int c[kPer], mine = 0, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = sh.pick.hist[tid * kPer + i];
      mine += c[i];
    }
    int before = block_before<kThreads>(mine, sums, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if (before < K && K <= before + c[i]) sm_step = kSteps - 1 - (tid * kPer + i);
      before += c[i];
    }
    __syncthreads();
    // The step's ends are off by roundings of 2^-23 of the range and of `low`, below 2^-8 e.
    from = low + sm_step * step - 2.1f * e;
    above = low + (sm_step + 1) * step + 2.1f * e;

    int sure = 0;
    for (int st = run0; st < run1; ++st) {
      const int i = 32 * st + lane, at = i < N ? side_of(score_of(i)) : 0;
      sure += at == 1;
      if (at == 2) {
        const int place = atomicAdd(&sm_unsure, 1);
        if (place < kUnsure) sh.pick.page[place] = i;
      }
    }
    sure = __reduce_add_sync(0xffffffffu, sure);
    if (lane == 0) counts[warp] = sure;
    __syncthreads();
    again = sm_unsure > kUnsure;
  }
  if (again) {
    // Every page in fp64, over the screened scores.
    __syncthreads();
    for (int i = tid; i < static_cast<int>(sizeof(sh.top.hist) / 4); i += kThreads) (&sh.top.hist[0][0])[i] = 0;
    for (int page = warp; page < N; page += kWarps) {
      const u64 key = exact_score<E>(s, b, h, page);
      if (lane == 0) keys[page] = key;
    }
    __syncthreads();
    top_of<kThreads>(keys, N, K, out, sh.top);
    return;
  }
  // Of the unsure all, or the greatest in fp64: their scores become inf, the others' -inf.
  const int unsure = sm_unsure, need = K - __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[lane] : 0);
  if (need < unsure)
    for (int i = warp; i < unsure; i += kWarps) {
      const u64 key = exact_score<E>(s, b, h, sh.pick.page[i]);
      if (lane == 0) sh.pick.key[i] = key;
    }
  __syncthreads();
  if (tid < unsure) {
    const int page = sh.pick.page[tid];
    int before = 0;
    if (need < unsure) {
      const u64 mine = sh.pick.key[tid];
      for (int j = 0; j < unsure; ++j)
        before += sh.pick.key[j] > mine || (sh.pick.key[j] == mine && sh.pick.page[j] < page);
    }
    const bool in = before < need;
    if (page < kStored) score[page] = in ? INFINITY : -INFINITY;
    else screened[page] = make_float2(in ? INFINITY : -INFINITY, 0.0f);
    if (in) atomicAdd(&counts[(page >> 5) / span], 1);
  }
  __syncthreads();
  int at = __reduce_add_sync(0xffffffffu, lane < warp ? counts[lane] : 0);  // a place for each, in page order
  for (int st = run0; st < run1; ++st) {
    const int i = 32 * st + lane;
    const bool in = i < N && side_of(score_of(i)) == 1;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (in) out[at + __popc(m & ((1u << lane) - 1))] = i;
    at += __popc(m);
  }
}

// Score kernel, then selection; Score and Top: the kernels; stored: scores that
// Top has in shared memory.
template <typename Score, typename Top>
cudaError_t launch_pair(Score score, Top top, int threads, int stored, const SelectArgs& s, int NT, StatusBlock* sb,
                        bool (&score_done)[64], bool (&top_done)[64], cudaStream_t stream) {
  // The score kernels' loads in flight have their place in L1, which is given all it can have
  // (134 MB of bounds: 54 us for the selection against 65).
  cudaError_t err = prepare_kernel(score, (kMaxRequests + 1) * 4, score_done, cudaSharedmemCarveoutMaxL1);
  if (err == cudaSuccess) err = prepare_kernel(top, stored * 4, top_done);
  if (err != cudaSuccess) return err;
  const long long most = (static_cast<long long>(s.a.B) * s.a.kv * s.a.max_pages + kScoreWarps - 1) / kScoreWarps;
  const long long fit = std::min<long long>(static_cast<long long>(sm_count()) * score_per_sm(NT), kMaxCtas);
  const int ctas = static_cast<int>(std::max(1LL, std::min(fit, most)));
  err = launch_pdl(score, dim3(ctas), dim3(kScoreThreads), static_cast<size_t>(s.a.B + 1) * 4, stream, s);
  if (err != cudaSuccess) return err;
  const size_t held = static_cast<size_t>(std::min(s.a.max_pages, stored)) * 4;
  return launch_pdl(top, dim3(s.a.B * s.a.kv + 1), dim3(threads), held, stream, s, ctas, sb);
}
template <int NT, int kThreads>
cudaError_t launch_f32(const SelectArgs& s, StatusBlock* sb, cudaStream_t stream) {
  static bool done[2][64] = {};
  return launch_pair(page_score_kernel<NT>, page_top_kernel<kThreads>, kThreads, 0, s, NT, sb, done[0], done[1], stream);
}
template <typename E, int NT, int kThreads>
cudaError_t launch_screened(const SelectArgs& s, StatusBlock* sb, cudaStream_t stream) {
  static bool done[2][64] = {};
  return launch_pair(page_screen_kernel<E, NT>, page_pick_kernel<E, kThreads>, kThreads, kStored, s, NT, sb, done[0],
                     done[1], stream);
}
// Twice the threads where a row may have more scores than 512 hold (at 64 registers a
// thread, so the selection spills 16 to 32 bytes).
template <int NT>
cudaError_t launch_select(const SelectArgs& s, mova_dtype dt, StatusBlock* sb, cudaStream_t stream) {
  const bool few = s.a.max_pages <= 512 * kHeld;
  if (dt == MOVA_F32) return few ? launch_f32<NT, 512>(s, sb, stream) : launch_f32<NT, 1024>(s, sb, stream);
  if (dt == MOVA_BF16)
    return few ? launch_screened<__nv_bfloat16, NT, 512>(s, sb, stream)
               : launch_screened<__nv_bfloat16, NT, 1024>(s, sb, stream);
  return few ? launch_screened<uint8_t, NT, 512>(s, sb, stream) : launch_screened<uint8_t, NT, 1024>(s, sb, stream);
}

}  // namespace

cudaError_t launch_page_select(const void* q, long long q_stride, int G, const PageArgs& a, mova_dtype dt,
                               const void* lo, const void* hi, int top, int32_t* picked, const PageWs& ws,
                               cudaStream_t stream) {
  const SelectArgs s{a, q, q_stride, G, top, lo, hi, ws.keys, ws.bad, picked};
  return G <= 8 ? launch_select<1>(s, dt, ws.sb, stream) : launch_select<2>(s, dt, ws.sb, stream);
}

}  // namespace mova

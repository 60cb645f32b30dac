// The cache pages worth reading for a query, by per-page key bounds.
//
//   score(page) = max over the KV head's query heads h of
//                 sum_d q[h, d] * (q[h, d] < 0 ? lo[page, d] : hi[page, d])
//
// and, of the request's full pages, the `top - 1` greatest (ties: the lower
// page number), with the last page always, in ascending order.
//
// Scores: the formula is q+ . hi + q- . lo with q split by sign, a product of
// (heads) x (2 * 128) by (2 * 128) x (pages).  A warp takes 8 pages at a time
// and forms it with fp64 matrix instructions (m8n8k4): 8 heads by 8 pages, the
// pages' bounds as loaded, 16 bytes a lane, whose dimensions q's registers
// match.  fp64 because neighbouring scores decide what is read: with fp32 sums
// the choice would depend on their order.  Products of the parts are exact for
// bf16 and E4M3 bounds.  Scores are stored as unsigned integers in the same
// order (NaN greatest, -0 = +0).
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
constexpr int kScorePerSm = 2;
constexpr int kPages = 8;  // of one batch
constexpr int kTopThreads = 512;
constexpr int kDigit = 11;
constexpr int kBins = 1 << kDigit;

using u64 = unsigned long long;

// One 32-bit word of stored elements in fp64.
template <typename E> struct Word;
template <> struct Word<float> {
  static constexpr int kPer = 1;
  static __device__ __forceinline__ void get(uint32_t u, double (&d)[1]) { d[0] = __uint_as_float(u); }
};
template <> struct Word<__nv_bfloat16> {
  static constexpr int kPer = 2;
  static __device__ __forceinline__ void get(uint32_t u, double (&d)[2]) {
    d[0] = __uint_as_float(u << 16), d[1] = __uint_as_float(u & 0xffff0000u);
  }
};
template <> struct Word<uint8_t> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ void get(uint32_t u, double (&d)[4]) {
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

__device__ __forceinline__ double value(float x) { return x; }
__device__ __forceinline__ double value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ double value(uint8_t x) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3))); }

__device__ __forceinline__ int pages_of(const PageArgs& a, int b) {
  const int len = clamp_len(a.lens[b], a.max_pages, a.shift);
  return (len + (1 << a.shift) - 1) >> a.shift;
}

// c (8 heads x 8 pages) += a (8 heads x 4 dimensions) b (4 dimensions x 8 pages).
__device__ __forceinline__ void mma884(double (&c)[2], double a, double b) {
  asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
               : "+d"(c[0]), "+d"(c[1]) : "d"(a), "d"(b));
}

// The dimensions of this lane (t = lane & 3) come in chunks of 16 stored bytes:
// chunk i holds dimensions (t + 4 i) * kPer + {0 .. kPer - 1}.
template <typename E> struct Chunk {
  static constexpr int kPer = 16 / sizeof(E);
  static constexpr int kCount = kHeadDim / kPer / 4;
};

// NT: tiles of 8 heads.  One tile's q stays in registers in fp64, split by
// sign; two tiles' q stays as loaded and is converted for each batch of pages.
template <typename Q, typename E, int NT>
__global__ void __launch_bounds__(kScoreThreads, 2) page_score_kernel(const SelectArgs s) {
  using C = Chunk<E>;
  constexpr int kWords = C::kCount * 4;                       // 32-bit words of a lane's bounds
  constexpr int kQWords = 32 / Word<Q>::kPer;                 // and of its 32 elements of q
  constexpr int kQVec = kQWords / C::kCount / 4;              // 16-byte loads of q per chunk
  extern __shared__ int pre[];
  __shared__ int sm_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int B = s.a.B, kv = s.a.kv, G = s.G;
  if (tid == 0) sm_bad = kNoBad;
  pdl_wait();
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

  // Where a batch of pages lies: its request and KV head, and its first page.
  struct At { int b, h, page0, pages; };
  auto locate = [&](int u) {
    At r;
    r.b = request_of(pre, B, u / kv);
    const int tiles = pre[r.b + 1] - pre[r.b], rem = u - kv * pre[r.b];
    r.h = rem / tiles;
    r.page0 = (rem - r.h * tiles) * kPages;
    r.pages = pages_of(s.a, r.b) - 1;
    return r;
  };
  // Page g of a batch as a page number, -1 if it is none.
  auto look_up = [&](const At& r) {
    if (r.page0 + g >= r.pages) return -1;
    const int id = s.a.table[r.b * s.a.table_stride + r.page0 + g];
    if (id >= 0 && id < s.a.num_pages) return id;
    atomicMin(&sm_bad, r.b);
    return -1;
  };
  // A page that is none reads page 0; its score is dropped.
  auto load = [&](const At& r, int id, uint32_t (&lo)[kWords], uint32_t (&hi)[kWords]) {
    const long long off = (static_cast<long long>(max(id, 0)) * kv + r.h) * kHeadDim + t * C::kPer;
    const E* pl = static_cast<const E*>(s.lo) + off;
    const E* ph = static_cast<const E*>(s.hi) + off;
#pragma unroll
    for (int i = 0; i < C::kCount; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(pl + i * 4 * C::kPer);
      const uint4 y = *reinterpret_cast<const uint4*>(ph + i * 4 * C::kPer);
      lo[4 * i] = x.x, lo[4 * i + 1] = x.y, lo[4 * i + 2] = x.z, lo[4 * i + 3] = x.w;
      hi[4 * i] = y.x, hi[4 * i + 1] = y.y, hi[4 * i + 2] = y.z, hi[4 * i + 3] = y.w;
    }
  };

  uint32_t q_raw[NT][kQWords];
  double q_pos[NT == 1 ? 32 : 1], q_neg[NT == 1 ? 32 : 1];
  uint32_t lo[kWords], hi[kWords];
  At at{}, next{};
  int id = -1, next_id = -1, row = -1;
  if (u0 < u1) {
    at = locate(u0);
    id = look_up(at);
    load(at, id, lo, hi);
  }
  for (int u = u0; u < u1; ++u) {
    const bool more = u + 1 < u1;
    if (more) {
      next = locate(u + 1);
      next_id = look_up(next);
    }
    if (at.b * kv + at.h != row) {
      row = at.b * kv + at.h;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int head = min(n * 8 + g, G - 1);  // rows past the last head repeat it and are dropped
        const Q* src = static_cast<const Q*>(s.q) + at.b * s.q_stride +
                       (static_cast<long long>(at.h) * G + head) * kHeadDim + t * C::kPer;
#pragma unroll
        for (int i = 0; i < C::kCount; ++i)
#pragma unroll
          for (int v = 0; v < kQVec; ++v) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + i * 4 * C::kPer + v * (16 / sizeof(Q)));
            uint32_t* to = &q_raw[n][(i * kQVec + v) * 4];
            to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
          }
      }
      if constexpr (NT == 1) {
#pragma unroll
        for (int x = 0; x < kQWords; ++x) {
          double d[Word<Q>::kPer];
          Word<Q>::get(q_raw[0][x], d);
#pragma unroll
          for (int y = 0; y < Word<Q>::kPer; ++y) {
            const bool neg = d[y] < 0.0;
            q_pos[x * Word<Q>::kPer + y] = neg ? 0.0 : d[y];
            q_neg[x * Word<Q>::kPer + y] = neg ? d[y] : 0.0;
          }
        }
      }
    }
    // Four sums of 16 products of 4 dimensions each, so that products need not
    // wait for one another.
    double c[NT][4][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) c[n][x][0] = c[n][x][1] = 0.0;
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      double dl[Word<E>::kPer], dh[Word<E>::kPer];
      Word<E>::get(lo[x], dl);
      Word<E>::get(hi[x], dh);
#pragma unroll
      for (int y = 0; y < Word<E>::kPer; ++y) {
        const int k = x * Word<E>::kPer + y;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          double pos, neg;
          if constexpr (NT == 1) {
            pos = q_pos[k], neg = q_neg[k];
          } else {
            double d[Word<Q>::kPer];
            Word<Q>::get(q_raw[n][k / Word<Q>::kPer], d);
            const double v = d[k % Word<Q>::kPer];
            pos = v < 0.0 ? 0.0 : v, neg = v < 0.0 ? v : 0.0;
          }
          mma884(c[n][2 * (k & 1)], pos, dh[y]);
          mma884(c[n][2 * (k & 1) + 1], neg, dl[y]);
        }
      }
    }
    if (more) load(next, next_id, lo, hi);
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
          const long long off = (static_cast<long long>(p) * kv + at.h) * kHeadDim + 4 * lane;
          const Q* src = static_cast<const Q*>(s.q) + at.b * s.q_stride +
                         (static_cast<long long>(at.h) * G + head) * kHeadDim + 4 * lane;
          double v = 0.0;
          for (int i = 0; i < 4; ++i) {
            const double d = value(src[i]);
            v = fma(d, d < 0.0 ? value(static_cast<const E*>(s.lo)[off + i]) : value(static_cast<const E*>(s.hi)[off + i]), v);
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
    at = next;
    id = next_id;
  }
  pdl_trigger();
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

constexpr int kHeld = 16;  // keys of a thread in registers; a long request's others are read again
constexpr int kTopWarps = kTopThreads / 32;

struct TopShared {
  int hist[kBins];
  int sums[kTopWarps];
  int bin, above, in;
};

// Radix search among 32-bit values, `bits` of them open, for the `need`
// greatest: each(f) calls f for every value of this thread.  Returns how many
// low bits are left open; *prefix the bits above them that the least of the
// greatest has, *need how many to take of the values with that prefix, *all
// whether those are all there are.  hist is zero before and after.
template <typename Each>
__device__ __forceinline__ int radix_search(Each each, int bits, TopShared& sh, uint32_t* prefix, int* need, bool* all) {
  *prefix = 0;
  *all = false;
  while (bits > 0 && !*all) {
    const int width = bits < kDigit ? bits : kDigit, low = bits - width;
    const uint32_t mask = (1u << width) - 1, above_mask = bits == 32 ? 0u : ~0u << bits, want = bits == 32 ? 0u : *prefix << bits;
    each([&](uint32_t v) {
      if ((v & above_mask) == want) atomicAdd(&sh.hist[(v >> low) & mask], 1);
    });
    __syncthreads();
    // Thread i holds the bins below kBins - 4 i, from the top.
    constexpr int kPer = kBins / kTopThreads;
    const int top_bin = kBins - 1 - static_cast<int>(threadIdx.x) * kPer;
    int c[kPer], mine = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      c[j] = sh.hist[top_bin - j];
      mine += c[j];
    }
    int above = cta_scan(mine, sh.sums);  // its barrier: every bin has been read
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (above < *need && *need <= above + c[j]) sh.bin = top_bin - j, sh.above = above, sh.in = c[j];
      above += c[j];
      sh.hist[top_bin - j] = 0;
    }
    __syncthreads();
    *prefix = (*prefix << width) | static_cast<uint32_t>(sh.bin);
    *need -= sh.above;
    *all = *need == sh.in;
    bits = low;
    __syncthreads();
  }
  return bits;
}

__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectArgs s, int score_ctas, StatusBlock* sb) {
  __shared__ TopShared sh;
  __shared__ u64 sm_min[kTopWarps], sm_max[kTopWarps];
  __shared__ unsigned counts[kHeld * kTopWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kBins; i += kTopThreads) sh.hist[i] = 0;
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

  // The least and the greatest score: above the bits in which they differ, all agree.
  u64 held[kHeld], least = ~0ULL, most_inv = ~0ULL;  // the greatest, as the least complement
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    const int at = tid + i * kTopThreads;
    held[i] = at < N ? keys[at] : 0ULL;
  }
  auto see = [&](u64 k) {
    least = k < least ? k : least;
    most_inv = ~k < most_inv ? ~k : most_inv;
  };
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (tid + i * kTopThreads < N) see(held[i]);
  for (int at = tid + kHeld * kTopThreads; at < N; at += kTopThreads) see(keys[at]);
  least = warp_min(least);
  most_inv = warp_min(most_inv);
  if (lane == 0) sm_min[warp] = least, sm_max[warp] = most_inv;
  __syncthreads();
  least = warp_min(sm_min[lane % kTopWarps]);
  most_inv = warp_min(sm_max[lane % kTopWarps]);
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
  int need = top - 1;
  bool all;
  uint32_t p1, p2 = 0;
  const int r1 = radix_search(
      [&](auto f) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
          if (tid + i * kTopThreads < N) f(v[i]);
        for (int at = tid + kHeld * kTopThreads; at < N; at += kTopThreads) f(upper(keys[at]));
      },
      open == 0 ? 0 : 32, sh, &p1, &need, &all);
  const bool second = open > 32 && !all;
  int r2 = 0;
  if (second)
    r2 = radix_search(
        [&](auto f) {
          for (int at = tid; at < N; at += kTopThreads) {
            const u64 k = keys[at];
            if (upper(k) == p1) f(static_cast<uint32_t>(k) & rest);
          }
        },
        open - 32, sh, &p2, &need, &all);

  // Places, in page order, kHeld stripes of kTopThreads pages at a time: the
  // counts of every (stripe, warp), one scan of them, and out.  A count holds
  // the greater ones in its low half, the equal ones in its high half.
  const unsigned below = (1u << lane) - 1;
  int base_more = 0, base_same = 0;
  for (int at0 = 0; at0 < N; at0 += kHeld * kTopThreads) {
    unsigned ranks[kHeld];  // of this thread within (stripe, warp), and its two flags
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      ranks[i] = 0;
      if (at0 + i * kTopThreads < N) {
        const int at = at0 + i * kTopThreads + tid;
        bool more = false, same = false;
        if (at < N) {
          const uint32_t x = open == 0 ? 0u : (at0 == 0 ? v[i] : upper(keys[at])) >> (r1 & 31);
          more = x > p1;
          same = x == p1;
          if (second && same) {
            const uint32_t y = (static_cast<uint32_t>(keys[at]) & rest) >> r2;
            more = y > p2;
            same = y == p2;
          }
        }
        const unsigned m = __ballot_sync(0xffffffffu, more), e = __ballot_sync(0xffffffffu, same);
        if (lane == 0) counts[i * kTopWarps + warp] = __popc(m) | (__popc(e) << 16);
        ranks[i] = __popc(m & below) | (__popc(e & below) << 8) | (more ? 1u << 16 : 0u) | (same ? 1u << 17 : 0u);
      } else if (lane == 0) {
        counts[i * kTopWarps + warp] = 0;
      }
    }
    __syncthreads();
    static_assert(kHeld * kTopWarps <= kTopThreads, "one count per thread");
    const unsigned mine = tid < kHeld * kTopWarps ? counts[tid] : 0u;
    const unsigned before = static_cast<unsigned>(cta_scan(static_cast<int>(mine), sh.sums));
    if (tid < kHeld * kTopWarps) counts[tid] = before;
    if (tid == kHeld * kTopWarps - 1) sh.above = static_cast<int>(before + mine);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (ranks[i] >> 16) {
        const unsigned c = counts[i * kTopWarps + warp];
        const int more_at = base_more + static_cast<int>((c & 0xffffu) + (ranks[i] & 0xffu));
        const int same_at = base_same + static_cast<int>((c >> 16) + ((ranks[i] >> 8) & 0xffu));
        if ((ranks[i] >> 16 & 1u) || all || same_at < need) out[more_at + min(same_at, need)] = at0 + i * kTopThreads + tid;
      }
    }
    base_more += sh.above & 0xffff;
    base_same += static_cast<int>(static_cast<unsigned>(sh.above) >> 16);
    __syncthreads();
  }
}

template <typename Q, typename E, int NT>
cudaError_t launch_score_t(const SelectArgs& s, int ctas, cudaStream_t stream) {
  static bool done[64] = {false};
  const cudaError_t err = prepare_kernel(page_score_kernel<Q, E, NT>, (kMaxRequests + 1) * 4, done);
  if (err != cudaSuccess) return err;
  return launch_pdl(page_score_kernel<Q, E, NT>, dim3(ctas), dim3(kScoreThreads), static_cast<size_t>(s.a.B + 1) * 4,
                    stream, s);
}
template <typename Q, typename E>
cudaError_t launch_score(const SelectArgs& s, int ctas, cudaStream_t stream) {
  return s.G <= 8 ? launch_score_t<Q, E, 1>(s, ctas, stream) : launch_score_t<Q, E, 2>(s, ctas, stream);
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
  static bool done[64] = {false};
  if (err == cudaSuccess) err = prepare_kernel(page_top_kernel, 0, done);
  if (err != cudaSuccess) return err;
  return launch_pdl(page_top_kernel, dim3(a.B * a.kv), dim3(kTopThreads), 0, stream, s, n, ws.sb);
}

}  // namespace mova

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
// greatest score share, so three or four passes of 8 bits settle it.  Latency
// bounds it (a few thousand scores, in registers): a warp owns a contiguous run
// of pages, so the passes and the placing in order need one barrier each.  No
// atomics decide an order.
#include <math.h>

#include "paged.cuh"

namespace mova {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kScoreWarps = kScoreThreads / 32;
// CTAs of the score kernel an SM: by the registers of its NT tiles of heads.
constexpr int score_per_sm(int NT) { return NT == 1 ? 3 : 2; }
constexpr int kPages = 8;  // of one batch
constexpr int kDigit = 8;
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

// An element of q as it stays in registers, and its positive and negative part
// in fp64.  bf16: the upper word of the fp64 value, whose lower word is zero;
// fp32: as it is, converted at each use.
template <typename Q> struct Part;
template <> struct Part<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t keep(double d) { return static_cast<uint32_t>(__double2hiint(d)); }
  static __device__ __forceinline__ void get(uint32_t w, double& pos, double& neg) {
    const int sign = static_cast<int>(w) >> 31;  // all ones below zero
    pos = __hiloint2double(static_cast<int>(w) & ~sign, 0);
    neg = __hiloint2double(static_cast<int>(w) & sign, 0);
  }
};
template <> struct Part<float> {
  static __device__ __forceinline__ uint32_t keep(double d) { return __float_as_uint(static_cast<float>(d)); }
  static __device__ __forceinline__ void get(uint32_t w, double& pos, double& neg) {
    const int sign = static_cast<int>(w) >> 31;
    const double d = __uint_as_float(w);
    pos = __hiloint2double(__double2hiint(d) & ~sign, __double2loint(d) & ~sign);
    neg = __hiloint2double(__double2hiint(d) & sign, __double2loint(d) & sign);
  }
};

// NT: tiles of 8 heads.
template <typename Q, typename E, int NT>
__global__ void __launch_bounds__(kScoreThreads, score_per_sm(NT)) page_score_kernel(const SelectArgs s) {
  using C = Chunk<E>;
  constexpr int kWords = C::kCount * 4;                          // 32-bit words of a lane's bounds
  constexpr int kQVec = 32 / Word<Q>::kPer / C::kCount / 4;      // 16-byte loads of q per chunk
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
  // This lane's first bounds in page `id`; a page that is none reads page 0, and
  // its score is dropped.
  auto offset = [&](const At& r, int id) {
    return (static_cast<long long>(max(id, 0)) * kv + r.h) * kHeadDim + t * C::kPer;
  };
  uint32_t lo[kWords], hi[kWords];
  auto load = [&](long long off, int i) {
    const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const E*>(s.lo) + off + i * 4 * C::kPer);
    const uint4 y = *reinterpret_cast<const uint4*>(static_cast<const E*>(s.hi) + off + i * 4 * C::kPer);
    lo[4 * i] = x.x, lo[4 * i + 1] = x.y, lo[4 * i + 2] = x.z, lo[4 * i + 3] = x.w;
    hi[4 * i] = y.x, hi[4 * i + 1] = y.y, hi[4 * i + 2] = y.z, hi[4 * i + 3] = y.w;
  };

  uint32_t q[NT][32];
  At at{}, next{};
  int id = -1, next_id = -1, row = -1;
  if (u0 < u1) {
    at = locate(u0);
    id = look_up(at);
    const long long off = offset(at, id);
#pragma unroll
    for (int i = 0; i < C::kCount; ++i) load(off, i);
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
            const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              double d[Word<Q>::kPer];
              Word<Q>::get(words[y], d);
#pragma unroll
              for (int z = 0; z < Word<Q>::kPer; ++z)
                q[n][((i * kQVec + v) * 4 + y) * Word<Q>::kPer + z] = Part<Q>::keep(d[z]);
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
    // Conversions run a word ahead of the products, whose latency they have; a
    // chunk's registers take the next pages' bounds as soon as it is used.
    const long long next_off = more ? offset(next, next_id) : 0;
    double dl[2][Word<E>::kPer], dh[2][Word<E>::kPer];
    Word<E>::get(lo[0], dl[0]);
    Word<E>::get(hi[0], dh[0]);
#pragma unroll
    for (int x = 0; x < kWords; ++x) {
      if (x + 1 < kWords) {
        Word<E>::get(lo[x + 1], dl[(x + 1) & 1]);
        Word<E>::get(hi[x + 1], dh[(x + 1) & 1]);
      }
#pragma unroll
      for (int y = 0; y < Word<E>::kPer; ++y) {
        const int k = x * Word<E>::kPer + y;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          double pos, neg;
          Part<Q>::get(q[n][k], pos, neg);
          mma884(c[n][2 * (k & 1)], pos, dh[x & 1][y]);
          mma884(c[n][2 * (k & 1) + 1], neg, dl[x & 1][y]);
        }
      }
      if (more && (x & 3) == 3) load(next_off, x >> 2);
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

template <int kTopThreads>
__global__ void __launch_bounds__(kTopThreads) page_top_kernel(const SelectArgs s, int score_ctas, StatusBlock* sb) {
  constexpr int kTopWarps = kTopThreads / 32;
  constexpr int kDigits = 32 / kDigit;
  __shared__ int hist[2 * kDigits][kBins];
  __shared__ u64 sm_min[kTopWarps], sm_max[kTopWarps];
  __shared__ int2 sm_count[kTopWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < 2 * kDigits * kBins; i += kTopThreads) (&hist[0][0])[i] = 0;
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
        for (int i = 0; i < kHeld; ++i) {
          if (i >= span) break;
          if (first + 32 * i < N) f(v[i]);
        }
        others([&](u64 k, int i) {
          if (first + 32 * i < N) f(upper(k));
        });
      },
      open == 0 ? 0 : 32, hist, &p1, &need, &all);
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
        open - 32, hist + kDigits, &p2, &need, &all);

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
  if (lane == 0) sm_count[warp] = mine;
  __syncthreads();
  int more = 0, same = 0;
  for (int w = 0; w < warp; ++w) more += sm_count[w].x, same += sm_count[w].y;
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

template <int kTopThreads>
cudaError_t launch_top(const SelectArgs& s, int score_ctas, StatusBlock* sb, cudaStream_t stream) {
  static bool done[64] = {false};
  const cudaError_t err = prepare_kernel(page_top_kernel<kTopThreads>, 0, done);
  if (err != cudaSuccess) return err;
  return launch_pdl(page_top_kernel<kTopThreads>, dim3(s.a.B * s.a.kv), dim3(kTopThreads), 0, stream, s, score_ctas, sb);
}

}  // namespace

cudaError_t launch_page_select(const void* q, long long q_stride, int G, const PageArgs& a, mova_dtype dt,
                               const void* lo, const void* hi, int top, int32_t* picked, const PageWs& ws,
                               cudaStream_t stream) {
  const SelectArgs s{a, q, q_stride, G, top, lo, hi, ws.keys, ws.bad, picked};
  const long long most = (static_cast<long long>(a.B) * a.kv * a.max_pages + kScoreWarps - 1) / kScoreWarps;
  long long ctas = static_cast<long long>(sm_count()) * score_per_sm(G <= 8 ? 1 : 2);
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  if (ctas > most) ctas = most < 1 ? 1 : most;
  const int n = static_cast<int>(ctas);
  cudaError_t err;
  if (dt == MOVA_F32) err = launch_score<float, float>(s, n, stream);
  else if (dt == MOVA_BF16) err = launch_score<__nv_bfloat16, __nv_bfloat16>(s, n, stream);
  else err = launch_score<__nv_bfloat16, uint8_t>(s, n, stream);
  if (err != cudaSuccess) return err;
  // Twice the threads where a row may have more scores than 512 hold.
  return a.max_pages > 512 * kHeld ? launch_top<1024>(s, n, ws.sb, stream) : launch_top<512>(s, n, ws.sb, stream);
}

}  // namespace mova

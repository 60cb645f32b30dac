// Attention of one new token per request over a paged key-value cache.
//
//   o[b, h] = sum_i p_i v_i / sum_i p_i,   p_i = exp(scale * q[b, h] . k_i)
//
// over the request's tokens, or over those of given pages.  Per cached token
// and KV head the kernel reads 2 x 128 elements and does 4 * 128 * G
// operations, G <= 16: far below the tensor cores' rate at any G, so the
// bytes of K and V bound it and every step below serves the memory stream.
//
// Split.  The keys of all rows -- a row is a (request, KV head) -- are laid out
// in one line of units, row by row, and each of the resident workers takes an
// equal, contiguous share; empty units stand for what a row's end costs.
// Lengths are known on the device only, so every CTA scans them itself.  A worker that covers a row alone writes its output; where
// several share one, each leaves a partial result (running maximum, sum, and
// unnormalised output) and the second kernel joins them in the order of the
// keys.  A worker has at most two partial results, its first and its last, so
// the workspace does not grow with the batch.  A worker is a CTA, whose four
// warps take a tile of each unit (16 keys of bf16, 32 of E4M3, 8 of fp32) and
// join where a row ends; or, where there are many rows, which may be short, a
// warp alone, as the joining costs more than a short row.  Rows that cannot be
// long are instead a cluster's each, where they are few, or a warp's, without
// scan, partial results or second kernel.
//
// Stream.  Each warp has a ring of 8 KB stages (K and V of one tile) that it
// fills with 16-byte asynchronous copies, one or two tiles ahead and across
// rows, so the stream does not stop where a softmax ends.  Page numbers are
// looked up 32 tiles at a time, one per lane.  Tokens past the end and pages
// that are none are filled with zeros and their scores set to -inf.
//
// Mathematics.  bf16: S^T = K q^T and O^T = V^T P^T on mma.m16n8k16, keys (or
// dimensions) as the 16 rows and query heads as the 8 columns, so that G <= 8
// heads need one column tile; one mma takes 16 keys, which tcgen05's
// 128-row tiles would need 8 tiles of one page table for.  Scores, maxima,
// sums and outputs are fp32.  P enters the second product as two bf16 terms
// (p = hi + lo, relative error 2^-16): one term would add an error as large
// as the output's own rounding.  E4M3: K, V become fp16 exactly; q is scaled
// by a power of two to [1, 2) at its largest element and rounded to fp16
// (exact for elements down to 2^-14 of the largest); P in fp16, 2^15 times as
// large (kLift), so that weights down to 2^-29 of a warp's greatest keep 2^-11
// against the output's 2^-8, and only those below 2^-40 count as none.  The sum
// of the weights is fp32 and as much larger.  fp32, up to 4 query heads a KV head: plain FMAs, whose
// rate is enough for 8 bytes per token, head and dimension.  fp32, more heads:
// the FMAs and their operands from shared memory would bound it (16 heads: 470
// us for 1.1 GB), so every fp32 number is split exactly into three bf16 parts
// and six products of parts are formed by mma (217 us; up to 8 heads, two parts
// at a time in the rows that heads leave free, 169 us); there an infinite key or
// value shows as NaN.
//
// Measured, of 6459 GB/s: bf16 16 requests to 32768 tokens, 775 MB: 124 us,
// 97%; 64 x 4096 tokens, 1.1 GB: 168.6 us, 99% with 4 heads, 92% with 16; E4M3
// 64 requests to 8192, 463 MB: 79 us, 91%; fp32 32 x 4096: 164 us, 101% with 4
// heads, 98% with 7, 77% with 16.  8 requests to 500 tokens: 6.3 us, the latency of a launch
// and four dependent loads.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"

namespace mova {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 128;
constexpr int kMaxCluster = 8;
constexpr int kWarps = kThreads / 32;
constexpr int kStageBytes = 8192;  // K and V of one warp's tile
constexpr int kRingAlign = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// fp32 pages by FMAs (up to 4 query heads a KV head) or by matrix products of
// bf16 parts; bf16 pages; E4M3 pages.
enum Mode { kF32 = 0, kB16 = 1, kE8 = 2, kF32Parts = 3 };
template <int M> constexpr bool kIsF32 = M == kF32 || M == kF32Parts;

template <int M> struct Tile;  // of one warp
template <> struct Tile<kF32> { using E = float;         static constexpr int keys = 8;  static constexpr int groups = 1; static constexpr int stages = 2; };
template <> struct Tile<kF32Parts> : Tile<kF32> {};
template <> struct Tile<kB16> { using E = __nv_bfloat16; static constexpr int keys = 16; static constexpr int groups = 1; static constexpr int stages = 3; };
template <> struct Tile<kE8>  { using E = uint8_t;       static constexpr int keys = 32; static constexpr int groups = 2; static constexpr int stages = 2; };

struct AttendArgs {
  PageArgs a;
  const void* q;
  long long q_stride;
  int G;
  float scale;
  const int32_t* picked;
  int top;
  void* o;
  float* lse;
  int32_t* bad;
  int32_t* prefix;
  float* part;
  int extra;  // empty units that follow each row's
};

// Units of request b: of its tokens, or of the picked pages' places.
__device__ __forceinline__ int places_of(const AttendArgs& s, int len) {
  if (s.picked == nullptr) return len;
  const int pages = (len + (1 << s.a.shift) - 1) >> s.a.shift;
  return (pages < s.top ? pages : s.top) << s.a.shift;
}

__device__ __forceinline__ void cp16_zfill(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}
// 2^x for x <= 15 (or NaN), relative error 2^-22; below 2^-126 it is 0.
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The factor of all weights, their sums and outputs: for fp16 weights the greatest
// power of two that fp16 holds, else 1.  Outputs are quotients, so it shows in
// the logarithm of a sum only.
template <int M> constexpr float kLift = M == kE8 ? 0x1p15f : 1.0f;
template <int M> __device__ __forceinline__ float log_sum(float m, float l) {
  return (m + log2f(l * (1.0f / kLift<M>))) * kLn2;
}
// The maximum to subtract: 0 while nothing has been seen.
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.0f : m; }

// One warp's softmax state for up to NT x 8 heads (mma) or NT heads (FMAs).
// mma: column heads nt * 8 + 2 * (lane & 3) + {0, 1}; FMAs: all heads.
template <int M, int NT> struct State {
  float o[M == kF32 ? 1 : 8][NT][4];
  float m[NT][2], l[NT][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (M == kF32 ? 1 : 8); ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[i][n][c] = 0.0f;
#pragma unroll
    for (int n = 0; n < NT; ++n) m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.0f;
  }
};

// The query heads of one KV head as mma column operands, and the factor from
// a raw product to a base-2 exponent for this thread's columns.
template <int M, int NT> struct Query {
  uint32_t b[8][NT][2];
  float f[NT][2];
};

template <int M, int NT>
__device__ __forceinline__ void load_query(Query<M, NT>& r, const __nv_bfloat16* q, int G, float scale, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int head = n * 8 + g;
    const __nv_bfloat16* row = q + head * kHeadDim;
    if constexpr (M == kB16) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r.b[k][n][0] = head < G ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 2 * t) : 0u;
        r.b[k][n][1] = head < G ? *reinterpret_cast<const uint32_t*>(row + 16 * k + 2 * t + 8) : 0u;
      }
      r.f[n][0] = r.f[n][1] = scale;
    } else {
      uint2 raw[8];
      float big = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        raw[k] = head < G ? *reinterpret_cast<const uint2*>(row + 16 * k + 4 * t) : make_uint2(0u, 0u);
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[k].x));
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[k].y));
        big = fmaxf(fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
      }
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // Power of two 2^e <= big; an infinite or subnormal row keeps a factor in range.
      int e = static_cast<int>(__float_as_uint(big) >> 23);
      e = e < 1 ? 127 : (e > 253 ? 253 : e);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[k].x));
        const float2 y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[k].y));
        r.b[k][n][0] = pack_f16(x.x * down, x.y * down);
        r.b[k][n][1] = pack_f16(y.x * down, y.y * down);
      }
      r.f[n][0] = scale * __shfl_sync(0xffffffffu, up, (2 * t) * 4);
      r.f[n][1] = scale * __shfl_sync(0xffffffffu, up, (2 * t + 1) * 4);
    }
  }
}

// Softmax of H x 16 keys' scores (rows g, g + 8 of each fragment): updates the
// state, and returns P^T as the second product's column operand.
template <int M, int NT, int H>
__device__ __forceinline__ void softmax(State<M, NT>& st, const float (&s)[H][NT][4], const Query<M, NT>& q,
                                        const int (&valid)[H], int lane, uint32_t (&p)[H][NT][2],
                                        uint32_t (&plo)[H][NT][2]) {
  const int g = lane >> 2;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float x[H][4], top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[h][c] = (c < 2 ? g : g + 8) < valid[h] ? s[h][n][c] * q.f[n][c & 1] : -INFINITY;
        top[c & 1] = fmaxf(top[c & 1], x[h][c]);
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], o));
      top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], o));
    }
    if (__any_sync(0xffffffffu, top[0] > st.m[n][0] || top[1] > st.m[n][1])) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float m = fmaxf(st.m[n][c], top[c]);
        const float a = ex2(st.m[n][c] - ref_of(m));
        st.m[n][c] = m;
        st.l[n][c] *= a;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          st.o[i][n][c] *= a;
          st.o[i][n][c + 2] *= a;
        }
      }
    }
    const float ref[2] = {ref_of(st.m[n][0]), ref_of(st.m[n][1])};
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        x[h][c] -= ref[c & 1];
        if constexpr (M == kE8) x[h][c] += 15.0f;  // after the difference, so that no rounding passes 2^15
        x[h][c] = ex2(x[h][c]);
      }
      st.l[n][0] += x[h][0] + x[h][2];
      st.l[n][1] += x[h][1] + x[h][3];
      if constexpr (M == kB16) {
        // hi: the upper 16 bits (p truncated); lo: the rest, kept above zero so that
        // an infinite value's products with both have one sign.
        float lo[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          lo[c] = fmaxf(x[h][c] - __uint_as_float(__float_as_uint(x[h][c]) & 0xffff0000u), x[h][c] * 0x1p-24f);
        p[h][n][0] = transpose8x8(__byte_perm(__float_as_uint(x[h][0]), __float_as_uint(x[h][1]), 0x7632));
        p[h][n][1] = transpose8x8(__byte_perm(__float_as_uint(x[h][2]), __float_as_uint(x[h][3]), 0x7632));
        plo[h][n][0] = transpose8x8(pack_bf16(lo[0], lo[1]));
        plo[h][n][1] = transpose8x8(pack_bf16(lo[2], lo[3]));
      } else {
        p[h][n][0] = transpose8x8(pack_f16(x[h][0], x[h][1]));
        p[h][n][1] = transpose8x8(pack_f16(x[h][2], x[h][3]));
      }
    }
  }
}

// One tile of 16 bf16 keys: K rows of 256 bytes at `kt`, V rows at `vt`,
// 16-byte chunk c of row r at place c ^ (r & 7).
template <int NT>
__device__ __forceinline__ void tile_b16(State<kB16, NT>& st, const Query<kB16, NT>& q, uint32_t kt, uint32_t vt,
                                         int valid, int lane) {
  const int r8 = lane & 7;
  float s[2][NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[0][n][c] = s[1][n][c] = 0.0f;
  // Rows are 256-byte aligned, so the swizzled chunk is an exclusive or away.
  const uint32_t krow = kt + (r8 + (lane & 8)) * 256 + (((lane >> 4) ^ r8) << 4);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t a[4];
    ldsm4(a, krow ^ (k << 5));
#pragma unroll
    for (int n = 0; n < NT; ++n) mma16816<false>(s[k & 1][n], a[0], a[1], a[2], a[3], q.b[k][n][0], q.b[k][n][1]);
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[0][n][c] += s[1][n][c];
  uint32_t p[1][NT][2], plo[1][NT][2];
  const float (&sum)[1][NT][4] = reinterpret_cast<const float (&)[1][NT][4]>(s);
  const int valids[1] = {valid};
  softmax<kB16, NT, 1>(st, sum, q, valids, lane, p, plo);
  const uint32_t vrow = vt + (r8 + ((lane >> 4) << 3)) * 256 + ((((lane >> 3) & 1) ^ r8) << 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t a[4];
    ldsm4t(a, vrow ^ (i << 5));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mma16816<false>(st.o[i][n], a[0], a[1], a[2], a[3], p[0][n][0], p[0][n][1]);
      mma16816<false>(st.o[i][n], a[0], a[1], a[2], a[3], plo[0][n][0], plo[0][n][1]);
    }
  }
}

// One tile of 32 E4M3 keys: rows of 128 bytes, chunk c of row r at c ^ (r & 7).
// A 32-bit word of a row fragment holds dimensions 16 c + 4 t + {0..3} of row
// g: the first two are the product's k = 2t, 2t + 1, the others k = 2t + 8,
// 2t + 9 (load_query orders q alike).  A transposed V fragment holds
// dimensions 16 c + 2 g + {0, 1} of keys 2t, 2t + 1: the even dimension is
// row g of the output tile, the odd one row g + 8.
template <int NT>
__device__ __forceinline__ void tile_e8(State<kE8, NT>& st, const Query<kE8, NT>& q, uint32_t kt, uint32_t vt,
                                        int valid0, int valid1, int lane) {
  const int r8 = lane & 7;
  float s[2][NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[0][n][c] = s[1][n][c] = 0.0f;
  // Matrices: rows 0-7, 8-15 (first 16 keys), 16-23, 24-31 (second), one chunk.
  const uint32_t krow = kt + lane * 128 + (r8 << 4);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    uint32_t a[4];
    ldsm4(a, krow ^ (k << 4));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a0 = e4m3_lo(a[2 * h]), a1 = e4m3_lo(a[2 * h + 1]);
      const uint32_t a2 = e4m3_hi(a[2 * h]), a3 = e4m3_hi(a[2 * h + 1]);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816<true>(s[h][n], a0, a1, a2, a3, q.b[k][n][0], q.b[k][n][1]);
    }
  }
  uint32_t p[2][NT][2], none[2][NT][2];
  const int valids[2] = {valid0, valid1};
  softmax<kE8, NT, 2>(st, s, q, valids, lane, p, none);
  const uint32_t vrow = vt + lane * 128 + (r8 << 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t a[4];
    ldsm4t(a, vrow ^ (i << 4));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t x = __byte_perm(a[2 * h], 0, 0x3120), y = __byte_perm(a[2 * h + 1], 0, 0x3120);
      const uint32_t a0 = e4m3_lo(x), a1 = e4m3_hi(x), a2 = e4m3_lo(y), a3 = e4m3_hi(y);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma16816<true>(st.o[i][n], a0, a1, a2, a3, p[h][n][0], p[h][n][1]);
    }
  }
}

// fp32 rows are 512 bytes, chunk c of row r at place c ^ f32_swizzle(r): four
// chunks of two neighbouring rows, and two of every second row, then lie in
// different banks.
__host__ __device__ constexpr int f32_swizzle(int r) { return ((r >> 1 & 3) << 1) ^ ((r & 1) << 2); }

// One tile of 8 fp32 keys, by FMAs.  Scores: four lanes per key, 32 dimensions
// each; then each lane holds dimensions 4 * lane + {0..3} of the output.  NT
// heads.
template <int NT>
__device__ __forceinline__ void tile_f32(State<kF32, NT>& st, const float* q, float scale, const char* kt,
                                         const char* vt, int valid, int lane) {
  const int key = lane >> 2, part = lane & 3;
  float s[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) s[n] = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = part + 4 * i;
    const float4 k = *reinterpret_cast<const float4*>(kt + key * 512 + ((c ^ f32_swizzle(key)) << 4));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 x = *reinterpret_cast<const float4*>(q + n * kHeadDim + 4 * c);
      s[n] = fmaf(k.w, x.w, fmaf(k.z, x.z, fmaf(k.y, x.y, fmaf(k.x, x.x, s[n]))));
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    s[n] += __shfl_xor_sync(0xffffffffu, s[n], 1);
    s[n] += __shfl_xor_sync(0xffffffffu, s[n], 2);
    const float x = key < valid ? s[n] * scale : -INFINITY;
    float top = x;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m = fmaxf(st.m[n][0], top);
    const float a = ex2(st.m[n][0] - ref_of(m));
    st.m[n][0] = m;
    s[n] = ex2(x - ref_of(m));
    st.l[n][0] = st.l[n][0] * a + s[n];
#pragma unroll
    for (int c = 0; c < 4; ++c) st.o[0][n][c] *= a;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float4 v = *reinterpret_cast<const float4*>(vt + j * 512 + ((lane ^ f32_swizzle(j)) << 4));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float p = __shfl_sync(0xffffffffu, s[n], 4 * j);
      st.o[0][n][0] = fmaf(p, v.x, st.o[0][n][0]);
      st.o[0][n][1] = fmaf(p, v.y, st.o[0][n][1]);
      st.o[0][n][2] = fmaf(p, v.z, st.o[0][n][2]);
      st.o[0][n][3] = fmaf(p, v.w, st.o[0][n][3]);
    }
  }
}

// Three bf16 numbers whose sum is x exactly (8 + 8 + 8 significand bits, each
// truncated), as the upper halves of fp32 words.
__device__ __forceinline__ void split3(float x, uint32_t (&p)[3]) {
  p[0] = __float_as_uint(x) & 0xffff0000u;
  const float r = x - __uint_as_float(p[0]);
  p[1] = __float_as_uint(r) & 0xffff0000u;
  p[2] = __float_as_uint(r - __uint_as_float(p[1]));
}
// The parts of two numbers, packed.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&p)[3]) {
  uint32_t a[3], b[3];
  split3(x, a);
  split3(y, b);
#pragma unroll
  for (int i = 0; i < 3; ++i) p[i] = __byte_perm(a[i], b[i], 0x7632);
}

// fp32 by parts: heads g and g + 8 (NT = 2) of the rows of S = q K^T and
// O = P V.  Output tile 4 c + j holds dimensions 32 c + 4 n + j in column n, so
// a lane's columns 2 t and 2 t + 1 of tiles 4 c .. 4 c + 3 are dimensions
// 32 c + 8 t .. + 7.  NT = 1: rows g + 8 have what the second part of P gives.
template <int NT> struct State<kF32Parts, NT> {
  float o[16][4];
  float m[2], l[2];
  __device__ __forceinline__ float at(int tile, int i) const { return NT > 1 ? o[tile][i] : o[tile][i] + o[tile][i + 2]; }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.0f;
    m[0] = m[1] = -INFINITY, l[0] = l[1] = 0.0f;
  }
};
template <int NT> struct Query<kF32Parts, NT> {
  uint32_t a[3][8][2 * NT];  // parts; steps of 16 dimensions; row operand words of heads g (and g + 8)
};
template <int NT>
__device__ __forceinline__ void load_query_parts(Query<kF32Parts, NT>& r, const float* q, int G, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int head = n * 8 + g;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float4 x = head < G ? *reinterpret_cast<const float4*>(q + head * kHeadDim + 16 * k + 4 * t)
                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      uint32_t p[3], s[3];
      split3(x.x, x.y, p);
      split3(x.z, x.w, s);
#pragma unroll
      for (int i = 0; i < 3; ++i) r.a[i][k][n] = p[i], r.a[i][k][NT + n] = s[i];
    }
  }
}

// One tile of 8 fp32 keys by matrix products: with every fp32 number the sum of
// three bf16 parts, a product keeps the six pairs of parts down to 2^-16 of it
// (what is left out is below 2^-23).  A lane's four loaded dimensions 4 t ..
// 4 t + 3 of a step of 16 are the step's k = 2t, 2t + 1, 2t + 8, 2t + 9.
template <int NT>
__device__ __forceinline__ void tile_f32_parts(State<kF32Parts, NT>& st, const Query<kF32Parts, NT>& q, float scale,
                                               const char* kt, const char* vt, int valid, int lane) {
  const int g = lane >> 2, t = lane & 3;
  // Several sums, as a product waits for the one before it in its sum.
  constexpr int kSums = NT > 1 ? 3 : 4;
  float s[kSums][4];
#pragma unroll
  for (int i = 0; i < kSums; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(kt + g * 512 + (((4 * k + t) ^ f32_swizzle(g)) << 4));
    uint32_t lo[3], hi[3];
    split3(x.x, x.y, lo);
    split3(x.z, x.w, hi);
    if constexpr (NT > 1) {
      // By the size of the pairs.
#pragma unroll
      for (int sum = 2; sum >= 0; --sum)
#pragma unroll
        for (int i = 0; i <= sum; ++i)
          mma16816<false>(s[sum], q.a[i][k][0], q.a[i][k][NT - 1], q.a[i][k][NT], q.a[i][k][2 * NT - 1], lo[sum - i],
                          hi[sum - i]);
    } else {
      // The rows that no head has take the second part of q.
      mma16816<false>(s[3], q.a[2][k][0], 0u, q.a[2][k][1], 0u, lo[0], hi[0]);
#pragma unroll
      for (int i = 2; i >= 0; --i)
        mma16816<false>(s[i], q.a[0][k][0], q.a[1][k][0], q.a[0][k][1], q.a[1][k][1], lo[i], hi[i]);
    }
  }
  // Score of keys 2 t + c, head g + 8 r: the small pairs first.
  auto score = [&](int r, int c) {
    if constexpr (NT > 1)
      return (s[2][2 * r + c] + s[1][2 * r + c]) + s[0][2 * r + c];
    else
      return ((((s[2][2 + c] + s[3][c]) + s[2][c]) + s[1][2 + c]) + (s[0][2 + c] + s[1][c])) + s[0][c];
  };
  uint32_t p[NT][3];  // parts of P: heads g (and g + 8), keys 2t, 2t + 1
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    float x[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) x[c] = 2 * t + c < valid ? score(r, c) * scale : -INFINITY;
    float top = fmaxf(x[0], x[1]);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float m = fmaxf(st.m[r], top);
    if (__any_sync(0xffffffffu, m > st.m[r])) {
      const float a = ex2(st.m[r] - ref_of(m));
      st.l[r] *= a;
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int c = NT > 1 ? 2 * r : 0; c < (NT > 1 ? 2 * r + 2 : 4); ++c) st.o[i][c] *= a;
    }
    st.m[r] = m;
#pragma unroll
    for (int c = 0; c < 2; ++c) x[c] = ex2(x[c] - ref_of(m));
    st.l[r] += x[0] + x[1];
    split3(x[0], x[1], p[r]);
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(vt + 2 * t * 512 + (((8 * c + g) ^ f32_swizzle(2 * t)) << 4));
    const float4 y = *reinterpret_cast<const float4*>(vt + (2 * t + 1) * 512 + (((8 * c + g) ^ f32_swizzle(2 * t + 1)) << 4));
    const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t v[3];
      split3(xs[j], ys[j], v);
      // Two pairs of parts at a time, one in each half of the 16 keys' places; and
      // with the second part of P in the rows that no head has, four.
      if constexpr (NT > 1) {
        mma16816<false>(st.o[4 * c + j], p[0][0], p[1][0], p[0][1], p[1][1], v[2], v[1]);
        mma16816<false>(st.o[4 * c + j], p[0][2], p[1][2], p[0][0], p[1][0], v[0], v[1]);
        mma16816<false>(st.o[4 * c + j], p[0][1], p[1][1], p[0][0], p[1][0], v[0], v[0]);
      } else {
        mma16816<false>(st.o[4 * c + j], p[0][2], 0u, p[0][0], 0u, v[0], v[2]);
        mma16816<false>(st.o[4 * c + j], p[0][0], p[0][1], p[0][0], p[0][1], v[0], v[1]);
      }
    }
  }
}

// A worker is a team of kTeam warps, and its unit of work kTeam tiles in a row,
// one for each warp.  Units that a worker has at least: a lone warp as many as
// it has in flight, so that a short row is not cut into more parts than its
// latency repays.
template <int M, int kTeam> constexpr int kLeast = kTeam > 1 ? 1 : Tile<M>::stages;

// Units of each worker, U in all (the last that has any may have fewer): worker
// w begins at unit w * share, so every worker between a row's first and last
// leaves a partial result.  Whole numbers of units, so that rows of one length
// are cut alike, and often at their ends (8 requests of 500 tokens: 8.7 us, 10.3
// in equal fractions of the units; long ones the same either way).
template <int M, int kTeam> __device__ __forceinline__ int share_of(int ctas, int U) {
  const int workers = ctas * (kWarps / kTeam);
  return max(kLeast<M, kTeam>, (U + workers - 1) / workers);
}

// Dynamic shared memory: the rings, each worker's fp32 queries (NT heads), the prefix.
template <int M, int NT, int kTeam>
__host__ __device__ constexpr size_t attend_smem(int B) {
  return kRingAlign + kWarps * Tile<M>::stages * kStageBytes +
         (M == kF32 ? kWarps / kTeam * NT * kHeadDim * 4 : 0) + static_cast<size_t>(B + 1) * 4;
}

// CTAs of an SM, by registers: as many as shared memory allows for the stages, or
// two where the state of 16 heads or of fp32 parts needs the registers.
template <int M, int NT> __host__ __device__ constexpr int ctas_per_sm() {
  return M == kF32 || (M == kE8 && NT == 1) ? 3 : 2;
}

// Where a warp turns its outputs round, head's dimension d lies at
// d ^ turn_swizzle(head): the four heads that it stores at once use different banks.
__device__ __forceinline__ int turn_swizzle(int head) { return ((head >> 1) & 3) << 3; }

// Four consecutive outputs of one head.
template <int M> __device__ __forceinline__ void store_out(void* o, long long at, const float4& v) {
  if constexpr (kIsF32<M>)
    *reinterpret_cast<float4*>(static_cast<float*>(o) + at) = v;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(o) + at) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
}

// What a cluster's CTAs share at the end: unnormalised outputs, then maxima and sums.
template <int M, int NT> constexpr int kMineFloats = (M == kF32 ? NT : 8 * NT) * kPartRow;

// The status of a call without a second kernel, by one cluster of its own: every
// length, and every table entry that the other clusters look up.
__device__ __forceinline__ void check_pages(const AttendArgs& s, StatusBlock* sb, int* sm_bad) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), tid = threadIdx.x, threads = cluster.num_blocks() * kThreads;
  const int B = s.a.B, kv = s.a.kv, shift = s.a.shift, width = s.picked == nullptr ? s.a.max_pages : s.top;
  int bad = kNoBad;
  for (int b = rank * kThreads + tid; b < B; b += threads) {
    const int len = s.a.lens[b];
    if (clamp_len(len, s.a.max_pages, shift) != len) bad = min(bad, b);
  }
  const int rows = s.picked == nullptr ? B : B * kv;
#pragma unroll 4
  for (int i = rank * kThreads + tid; i < rows * width; i += threads) {
    const int row = i / width, place = i - row * width, b = s.picked == nullptr ? row : row / kv;
    const int pages = (clamp_len(s.a.lens[b], s.a.max_pages, shift) + (1 << shift) - 1) >> shift;
    const int page = place >= pages ? -1 : s.picked == nullptr ? place : s.picked[i];
    if (page >= 0 && page < pages) {
      const int id = s.a.table[b * s.a.table_stride + page];
      if (id < 0 || id >= s.a.num_pages) bad = min(bad, b);
    }
  }
  bad = __reduce_min_sync(0xffffffffu, bad);
  cluster.sync();  // rank 0 has set its word
  if ((tid & 31) == 0 && bad != kNoBad) atomicMin(cluster.map_shared_rank(sm_bad, 0), bad);
  cluster.sync();
  if (rank == 0 && tid == 0) {
    sb->code = *sm_bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
    sb->detail = *sm_bad == kNoBad ? 0 : *sm_bad;
  }
}

// NT: mma column tiles of 8 heads, or fp32 heads.  kOwn: a cluster has one row,
// its CTAs equal shares of it, and joins them itself (a team), or a warp has one
// (kTeam = 1); the first cluster sees to the status, sb.
template <int M, int NT, int kTeam, bool kOwn>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<M, NT>()) page_attend_kernel(const AttendArgs s, StatusBlock* sb) {
  using E = typename Tile<M>::E;
  using Out = typename std::conditional<kIsF32<M>, float, __nv_bfloat16>::type;
  constexpr int kKeys = Tile<M>::keys;
  constexpr int kUnit = kTeam * kKeys;
  constexpr int kGroups = Tile<M>::groups;
  constexpr int kStages = Tile<M>::stages;
  constexpr int kRow = kHeadDim * sizeof(E);      // bytes of a key
  constexpr int kChunks = kRow / 16;
  extern __shared__ char smem_raw[];
  __shared__ float sm_m[kWarps][kMaxGroup], sm_l[kWarps][kMaxGroup];
  __shared__ float4 sm_f[kTeam > 1 ? kMaxGroup : 1];
  __shared__ float sm_sum[kTeam > 1 ? kMaxGroup : 1];
  __shared__ int sm_valid[kWarps][kStages][2];
  __shared__ int sm_bad;

  // The ring's rows are aligned to their size (tile_b16, tile_e8 count on it).
  char* smem = smem_raw + ((kRingAlign - (smem_u32(smem_raw) & (kRingAlign - 1))) & (kRingAlign - 1));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = s.G, kv = s.a.kv, B = s.a.B, shift = s.a.shift;
  char* ring_base = smem + warp * (kStages * kStageBytes);
  float* q_all = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);
  float* q_sm = q_all + (M == kF32 ? warp / kTeam * NT * kHeadDim : 0);
  int* pre = reinterpret_cast<int*>(q_all + (M == kF32 ? kWarps / kTeam * NT * kHeadDim : 0));

  float* mine = reinterpret_cast<float*>(pre);  // kOwn

  if (tid == 0) sm_bad = kNoBad;
  pdl_wait();
  int w = 0, u0, count, row_b = 0, row_h = 0, row_tiles = 0;
  if constexpr (kOwn) {
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = cluster.block_rank(), size = cluster.num_blocks(), id = blockIdx.x / size - 1;
    if (id < 0) {
      __syncthreads();
      check_pages(s, sb, &sm_bad);
      return;
    }
    const int row = kTeam > 1 ? id : (id * size + rank) * kWarps + warp;
    if (kTeam == 1 && row >= B * kv) return;
    row_b = row / kv, row_h = row - row_b * kv;
    row_tiles = (places_of(s, clamp_len(s.a.lens[row_b], s.a.max_pages, shift)) + kUnit - 1) / kUnit;
    u0 = kTeam > 1 ? rank * row_tiles / size : 0;
    count = kTeam > 1 ? (rank + 1) * row_tiles / size - u0 : row_tiles;
  } else {
    __syncthreads();
    request_scan<kThreads>(B, pre, [&](int b) {
      const int len = s.a.lens[b], use = clamp_len(len, s.a.max_pages, shift);
      if (use != len) atomicMin(&sm_bad, b);
      const int tiles = (places_of(s, use) + kUnit - 1) / kUnit;
      return tiles == 0 ? 0 : tiles + s.extra;
    });
    const int U = kv * pre[B];
    if (blockIdx.x == 0)
      for (int b = tid; b <= B; b += kThreads) s.prefix[b] = pre[b];
    const int share = share_of<M, kTeam>(gridDim.x, U);
    w = (blockIdx.x * kWarps + warp) / kTeam;
    u0 = min(w * share, U), count = min(share, U - u0);
  }

  // Page lookup of 32 tiles: lane i that of this warp's tile in unit `at + i`,
  // with the row (request, KV head) that it belongs to.
  int t_page[kGroups], t_row[kGroups], t_valid[kGroups], t_owner = -1;
  auto look_up = [&](int at) {
    const int i = at + lane;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) t_page[j] = t_row[j] = t_valid[j] = 0;
    t_owner = -1;
    if (i >= count) return;
    const int u = u0 + i;
    int b = row_b, h = row_h, tile = u;
    if constexpr (!kOwn) {
      b = request_of(pre, B, u / kv);
      const int units = pre[b + 1] - pre[b], rem = u - kv * pre[b];
      h = rem / units;
      tile = rem - h * units;
      if (tile >= units - s.extra) return;  // an empty unit: nothing valid, and no row's
    }
    const int len = clamp_len(s.a.lens[b], s.a.max_pages, shift);
    t_owner = b * kv + h;
#pragma unroll
    for (int j = 0; j < kGroups; ++j) {
      const int place = tile * kUnit + warp % kTeam * kKeys + 16 * j;
      const int in = place & ((1 << shift) - 1);
      int page = place >> shift;
      if (s.picked != nullptr) {
        const int pages = (len + (1 << shift) - 1) >> shift;
        const int listed = page < s.top && page < pages
                               ? s.picked[(static_cast<long long>(b) * kv + h) * s.top + page] : -1;
        page = listed < pages ? listed : -1;
      }
      int valid = page < 0 ? 0 : len - ((page << shift) + in);
      valid = valid < 0 ? 0 : (valid > 16 ? 16 : valid);
      if (valid > 0) {
        const int id = s.a.table[b * s.a.table_stride + page];
        if (id < 0 || id >= s.a.num_pages) {
          atomicMin(&sm_bad, b);
          valid = 0;
        } else {
          t_page[j] = id;
          t_row[j] = (h << shift) + in;
        }
      }
      t_valid[j] = valid;
    }
  };
  // The query rows of (request, KV head) number `owner`, in elements.
  auto q_at = [&](int owner) {
    return (owner / kv) * s.q_stride + static_cast<long long>(owner % kv) * G * kHeadDim;
  };
  const uint32_t ring = smem_u32(ring_base);
  const char* k_base = static_cast<const char*>(s.a.k);
  const char* v_base = static_cast<const char*>(s.a.v);
  constexpr int kRowsPer = 32 / kChunks;               // rows of one warp-wide copy
  constexpr int kCopies = kKeys / kGroups / kRowsPer;  // of K, and of V, per group
  constexpr int kPeriod = 8 / kRowsPer;  // copies after which the swizzle repeats
  const int lane_off = (lane / kChunks) * kRow + (lane % kChunks) * 16;
  uint32_t swz[kPeriod];
#pragma unroll
  for (int x = 0; x < kPeriod; ++x) {
    const int r = x * kRowsPer + lane / kChunks, c = lane % kChunks;
    swz[x] = r * kRow + ((kIsF32<M> ? c ^ f32_swizzle(r) : c ^ (r & 7)) << 4);
  }
  // Starts the copies of tile i (of this warp) into its stage.  Where a new row
  // begins, its queries are called into the cache: they are needed with its keys.
  int ahead = -1;
  auto issue = [&](int i) {
    if ((i & 31) == 0) look_up(i);
    if (i < count) {
      const int owner = __shfl_sync(0xffffffffu, t_owner, i & 31);
      if (!kOwn && owner < 0) {
        cp_commit();
        return;
      }
      if (owner != ahead) {
        ahead = owner;
        const int line = lane * 128;
        if (line < G * kHeadDim * (kIsF32<M> ? 4 : 2)) {
          const char* at = static_cast<const char*>(s.q) + q_at(owner) * (kIsF32<M> ? 4 : 2) + line;
          asm volatile("prefetch.global.L1 [%0];" ::"l"(at));
        }
      }
      const int stage = i % kStages;
      const uint32_t dst = ring + stage * kStageBytes;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) {
        const long long page = __shfl_sync(0xffffffffu, t_page[j], i & 31);
        const long long row = __shfl_sync(0xffffffffu, t_row[j], i & 31);
        const int valid = __shfl_sync(0xffffffffu, t_valid[j], i & 31);
        const char* ks = k_base + (page * s.a.k_stride + row * kHeadDim) * static_cast<long long>(sizeof(E));
        const char* vs = v_base + (page * s.a.v_stride + row * kHeadDim) * static_cast<long long>(sizeof(E));
        if (lane == 0) sm_valid[warp][stage][j] = valid;
        const uint32_t to = dst + j * 16 * kRow;
        if (valid >= kKeys / kGroups) {
#pragma unroll
          for (int x = 0; x < kCopies; ++x) {
            const uint32_t at = to + swz[x % kPeriod] + (x / kPeriod) * (kPeriod * kRowsPer * kRow);
            cp16(at, ks + lane_off + x * kRowsPer * kRow);
            cp16(at + kStageBytes / 2, vs + lane_off + x * kRowsPer * kRow);
          }
        } else {
#pragma unroll
          for (int x = 0; x < kCopies; ++x) {
            const bool in = x * kRowsPer + lane / kChunks < valid;
            const uint32_t at = to + swz[x % kPeriod] + (x / kPeriod) * (kPeriod * kRowsPer * kRow);
            const int off = in ? lane_off + x * kRowsPer * kRow : 0;
            cp16_zfill(at, ks + off, in ? 16 : 0);
            cp16_zfill(at + kStageBytes / 2, vs + off, in ? 16 : 0);
          }
        }
      }
    }
    cp_commit();
  };

  if (count > 0) {
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
    int b = row_b, tiles = row_tiles, h = row_h, t = u0;
    const int extra = kOwn ? 0 : s.extra;
    if constexpr (!kOwn) {
      b = request_of(pre, B, u0 / kv);
      const int units = pre[b + 1] - pre[b];
      tiles = units - extra;
      h = (u0 - kv * pre[b]) / units;
      t = u0 - kv * pre[b] - h * units;
    }
    State<M, NT> st;
    Query<M, M == kF32 ? 1 : NT> q;
    bool fresh = true, whole = t == 0;
    for (int i = 0; i < count; ++i) {
      if (!kOwn && t >= tiles) {  // an empty unit
        issue(i + kStages - 1);
        if (++t == tiles + extra) {
          fresh = whole = true;
          t = 0;
          if (i + 1 < count && ++h == kv) {
            h = 0;
            do ++b; while (pre[b + 1] == pre[b]);
            tiles = pre[b + 1] - pre[b] - extra;
          }
        }
        continue;
      }
      if (fresh) {
        st.clear();
        const long long at = q_at(b * kv + h);
        if constexpr (M == kF32) {
          const float* src = static_cast<const float*>(s.q) + at;
          for (int x = kTeam > 1 ? tid : lane; x < NT * kHeadDim / 4; x += kTeam > 1 ? kThreads : 32)
            reinterpret_cast<float4*>(q_sm)[x] =
                4 * x < G * kHeadDim ? reinterpret_cast<const float4*>(src)[x] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if constexpr (kTeam > 1) __syncthreads();
        } else if constexpr (M == kF32Parts) {
          load_query_parts<NT>(q, static_cast<const float*>(s.q) + at, G, lane);
        } else {
          const float k_scale = M == kE8 && s.a.k_scale != nullptr ? s.a.k_scale[h] : 1.0f;
          load_query<M, NT>(q, static_cast<const __nv_bfloat16*>(s.q) + at, G, s.scale * kLog2e * k_scale, lane);
        }
        fresh = false;
      }
      cp_wait<kStages - 2>();
      __syncwarp();  // the tile (and q_sm) is there; every lane has done with the tile before
      issue(i + kStages - 1);
      const int stage = i % kStages;
      const uint32_t kt = ring + stage * kStageBytes, vt = kt + kStageBytes / 2;
      char* tile = ring_base + stage * kStageBytes;
      if constexpr (M == kB16) {
        tile_b16<NT>(st, q, kt, vt, sm_valid[warp][stage][0], lane);
      } else if constexpr (M == kE8) {
        tile_e8<NT>(st, q, kt, vt, sm_valid[warp][stage][0], sm_valid[warp][stage][1], lane);
      } else if constexpr (M == kF32Parts) {
        tile_f32_parts<NT>(st, q, s.scale * kLog2e, tile, tile + kStageBytes / 2, sm_valid[warp][stage][0], lane);
      } else {
        tile_f32<NT>(st, q_sm, s.scale * kLog2e, tile, tile + kStageBytes / 2, sm_valid[warp][stage][0], lane);
      }
      const bool row_end = t + 1 == tiles;
      if (row_end || i + 1 == count) {
        // The row is done, or what this worker has of it.  Each warp lays its
        // outputs where the tile it has just used was (at most 16 heads x 512
        // bytes; the next copies into that stage start later), to be read back by
        // head: by a warp alone four dimensions a lane, by a team joined.
        const bool done = kOwn ? kTeam == 1 : whole && row_end;
        float* part = kOwn ? mine : s.part + (static_cast<size_t>(w) * 2 + (whole ? 1 : 0)) * (G * kPartRow);
        const long long row = static_cast<long long>(b) * kv + h;
        const float v_scale = M == kE8 && s.a.v_scale != nullptr ? s.a.v_scale[h] : 1.0f;
        float* turn = reinterpret_cast<float*>(tile);
        auto note = [&](int head, float m, float l) {
          if (done) {
            if (s.lse != nullptr) s.lse[row * G + head] = log_sum<M>(m, l);
          } else {
            part[G * kHeadDim + head] = m, part[G * (kHeadDim + 1) + head] = l;
          }
        };
        // Warp alone: lane l puts dimensions 4 l .. 4 l + 3.
        auto put = [&](int head, float m, float l, float4 v) {
          const float f = done ? v_scale / l : v_scale;
          v = l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
          if (done)
            store_out<M>(s.o, (row * G + head) * kHeadDim + 4 * lane, v);
          else
            *reinterpret_cast<float4*>(part + head * kHeadDim + 4 * lane) = v;
          if (lane == 0) note(head, m, l);
        };
        auto put_all = [&] {
          __syncwarp();
          for (int head = 0; head < G; ++head)
            put(head, sm_m[warp][head], sm_l[warp][head],
                *reinterpret_cast<const float4*>(&turn[head * kHeadDim + ((4 * lane) ^ turn_swizzle(head))]));
        };
        __syncwarp();  // every lane has read the tile
        if constexpr (M == kF32) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float l = st.l[n][0];  // the four lanes of a key hold the same
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const float4 v = make_float4(st.o[0][n][0], st.o[0][n][1], st.o[0][n][2], st.o[0][n][3]);
            if (n < G) {
              if constexpr (kTeam == 1) {
                put(n, st.m[n][0], l, v);
              } else {
                if (lane == 0) sm_m[warp][n] = st.m[n][0], sm_l[warp][n] = l;
                *reinterpret_cast<float4*>(&turn[n * kHeadDim + ((4 * lane) ^ turn_swizzle(n))]) = v;
              }
            }
          }
        } else if constexpr (M == kF32Parts) {
          const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float l = st.l[n];
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            const int head = n * 8 + g;
            if (head < G) {
              if (t4 == 0) sm_m[warp][head] = st.m[n], sm_l[warp][head] = l;
              float* to = &turn[head * kHeadDim];
              const int z = turn_swizzle(head);
#pragma unroll
              for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  *reinterpret_cast<float4*>(&to[(32 * c + 8 * t4 + 4 * x) ^ z]) =
                      make_float4(st.at(4 * c, 2 * n + x), st.at(4 * c + 1, 2 * n + x), st.at(4 * c + 2, 2 * n + x),
                                  st.at(4 * c + 3, 2 * n + x));
            }
          }
          if constexpr (kTeam == 1) put_all();
        } else {
          const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float l = st.l[n][c];
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
              const int head = n * 8 + 2 * t4 + c;
              if (head < G) {
                if (g == 0) sm_m[warp][head] = st.m[n][c], sm_l[warp][head] = l;
                float* to = &turn[head * kHeadDim];
                const int z = turn_swizzle(head);
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                  if constexpr (M == kE8) {
                    *reinterpret_cast<float2*>(&to[(16 * x + 2 * g) ^ z]) = make_float2(st.o[x][n][c], st.o[x][n][c + 2]);
                  } else {
                    to[(16 * x + g) ^ z] = st.o[x][n][c];
                    to[(16 * x + g + 8) ^ z] = st.o[x][n][c + 2];
                  }
                }
              }
            }
          if constexpr (kTeam == 1) put_all();
        }
        if constexpr (kTeam == 1) {
          __syncwarp();  // q_sm, sm_m and sm_l are free again
        } else {
          // A thread a head for the factors, then a thread a dimension for the outputs.
          const float* all = reinterpret_cast<const float*>(smem + stage * kStageBytes);
          constexpr int kNext = kStages * kStageBytes / 4;  // from one warp's stage to the next's
          static_assert(kTeam == 4, "a head's factors are one float4");
          __syncthreads();
          if (tid < G) {
            float m = -INFINITY, f[kTeam], l = 0.0f;
#pragma unroll
            for (int x = 0; x < kTeam; ++x) m = fmaxf(m, sm_m[x][tid]);
#pragma unroll
            for (int x = 0; x < kTeam; ++x) {
              f[x] = ex2(sm_m[x][tid] - ref_of(m));
              l = fmaf(sm_l[x][tid], f[x], l);
            }
            sm_f[tid] = make_float4(f[0], f[1], f[2], f[3]);
            sm_sum[tid] = l;
            note(tid, m, l);
          }
          __syncthreads();
#pragma unroll 4
          for (int head = 0; head < G; ++head) {
            const float4 f = sm_f[head];
            const float l = sm_sum[head];
            const float* at = all + head * kHeadDim + (tid ^ turn_swizzle(head));
            float o = at[0] * f.x;
            o = fmaf(at[kNext], f.y, o);
            o = fmaf(at[2 * kNext], f.z, o);
            o = fmaf(at[3 * kNext], f.w, o);
            o = l == 0.0f ? 0.0f : o * v_scale;
            if (done)
              static_cast<Out*>(s.o)[(row * G + head) * kHeadDim + tid] = from_f32<Out>(l == 0.0f ? 0.0f : o / l);
            else
              part[head * kHeadDim + tid] = o;
          }
          __syncthreads();
        }
        fresh = whole = true;
        if (row_end && extra == 0) {
          t = -1;
          if (i + 1 < count && ++h == kv) {
            h = 0;
            do ++b; while (pre[b + 1] == pre[b]);
            tiles = pre[b + 1] - pre[b];
          }
        }
      }
      ++t;
    }
    cp_wait<0>();
  }
  if constexpr (kOwn && kTeam == 1) {
    if (count == 0) {
      const long long row = static_cast<long long>(row_b) * kv + row_h;
      for (int head = 0; head < G; ++head) {
        store_out<M>(s.o, (row * G + head) * kHeadDim + 4 * lane, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
        if (lane == 0 && s.lse != nullptr) s.lse[row * G + head] = -INFINITY;
      }
    }
    pdl_trigger();
    return;
  }
  if constexpr (kOwn) {
    // The cluster's CTAs take the heads in turn, a thread a dimension.
    cg::cluster_group cluster = cg::this_cluster();
    const int size = cluster.num_blocks();
    if (count == 0)
      for (int head = 0; head < G; ++head) {
        mine[head * kHeadDim + tid] = 0.0f;
        if (tid == 0) mine[G * kHeadDim + head] = -INFINITY, mine[G * (kHeadDim + 1) + head] = 0.0f;
      }
    cluster.sync();
    const long long row = static_cast<long long>(row_b) * kv + row_h;
    for (int head = cluster.block_rank(); head < G; head += size) {
      float pm[kMaxCluster], pl[kMaxCluster], po[kMaxCluster], m = -INFINITY, l = 0.0f, o = 0.0f;
#pragma unroll
      for (int x = 0; x < kMaxCluster; ++x) {
        pm[x] = -INFINITY, pl[x] = po[x] = 0.0f;
        if (x < size) {
          const float* part = cluster.map_shared_rank(mine, x);
          pm[x] = part[G * kHeadDim + head];
          pl[x] = part[G * (kHeadDim + 1) + head];
          po[x] = part[head * kHeadDim + tid];
        }
        m = fmaxf(m, pm[x]);
      }
#pragma unroll
      for (int x = 0; x < kMaxCluster; ++x) {
        const float f = ex2(pm[x] - ref_of(m));
        l = fmaf(pl[x], f, l);
        o = fmaf(po[x], f, o);
      }
      static_cast<Out*>(s.o)[(row * G + head) * kHeadDim + tid] = from_f32<Out>(l == 0.0f ? 0.0f : o / l);
      if (tid == 0 && s.lse != nullptr) s.lse[row * G + head] = log_sum<M>(m, l);
    }
    pdl_trigger();
    cluster.sync();  // nobody leaves while its part may be read
    return;
  }
  // Only now: CTAs of the join that wait on an SM from the start cost this
  // kernel a third of its rate (118 us against 83 for 463 MB of E4M3 pages).
  pdl_trigger();
  __syncthreads();
  if (tid == 0) s.bad[blockIdx.x] = sm_bad;
}

// Joins the partial results of each (request, KV head) that several workers
// share, in the order of its keys; writes zeros where there is no token; and
// the status.  A warp takes one query head, four dimensions a lane, four parts'
// maxima, sums and outputs at once.  kSplit = 1: a CTA holds a warp for each
// head; otherwise kSplit warps share the one head of a CTA, warp g taking
// every kSplit-th four parts from the g-th, and are joined at the end.
template <int M, int kTeam, int kSplit>
__global__ void __launch_bounds__(kSplit > 1 ? 32 * kSplit : 32 * kMaxGroup)
page_join_kernel(const AttendArgs s, int ctas, StatusBlock* sb) {
  constexpr int kAhead = 4;
  __shared__ float4 sm_o[kSplit][kSplit > 1 ? 32 : 1];
  __shared__ float sm_m[kSplit], sm_l[kSplit];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = s.G, kv = s.a.kv, B = s.a.B;
  const int head = kSplit > 1 ? blockIdx.y : warp, group = kSplit > 1 ? warp : 0;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / kv, h = blockIdx.x - b * kv;
  const int p0 = s.prefix[b], units = s.prefix[b + 1] - p0, tiles = units - s.extra, U = kv * s.prefix[B];
  if (blockIdx.x == 0 && blockIdx.y == 0 && warp == 0) {
    int bad = kNoBad;
    for (int i = lane; i < ctas; i += 32) bad = min(bad, s.bad[i]);
    bad = __reduce_min_sync(0xffffffffu, bad);
    if (lane == 0) {
      sb->code = bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
      sb->detail = bad == kNoBad ? 0 : bad;
    }
  }
  const long long at = static_cast<long long>(blockIdx.x) * G + head;
  auto write = [&](const float4& v, float lse) {
    store_out<M>(s.o, at * kHeadDim + 4 * lane, v);
    if (s.lse != nullptr && lane == 0) s.lse[at] = lse;
  };
  if (units == 0) {
    if (group == 0) write(make_float4(0.0f, 0.0f, 0.0f, 0.0f), -INFINITY);
    return;
  }
  const int share = share_of<M, kTeam>(ctas, U), u0 = kv * p0 + h * units;
  const int w0 = u0 / share, parts = (u0 + tiles - 1) / share - w0 + 1;
  if (parts == 1) return;
  const int size = G * kPartRow;
  // Worker w0 begins this row (its second place), the others continue it.
  const float* part0 = s.part + static_cast<size_t>(w0) * 2 * size;
  float m = -INFINITY, l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto scale = [&](float a) { l *= a, acc.x *= a, acc.y *= a, acc.z *= a, acc.w *= a; };
  auto add = [&](float pl, const float4& po, float f) {
    l = fmaf(pl, f, l);
    acc.x = fmaf(po.x, f, acc.x), acc.y = fmaf(po.y, f, acc.y);
    acc.z = fmaf(po.z, f, acc.z), acc.w = fmaf(po.w, f, acc.w);
  };
  for (int i0 = group * kAhead; i0 < parts; i0 += kSplit * kAhead) {
    float pm[kAhead], pl[kAhead];
    float4 po[kAhead];
#pragma unroll
    for (int x = 0; x < kAhead; ++x) {
      if (i0 + x < parts) {
        const float* part = part0 + (2 * (i0 + x) + (i0 + x == 0 ? 1 : 0)) * size;
        pm[x] = part[G * kHeadDim + head];
        pl[x] = part[G * (kHeadDim + 1) + head];
        po[x] = *reinterpret_cast<const float4*>(part + head * kHeadDim + 4 * lane);
      } else {
        pm[x] = -INFINITY, pl[x] = 0.0f, po[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
    float top = m;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) top = fmaxf(top, pm[x]);
    scale(ex2(m - ref_of(top)));
    m = top;
#pragma unroll
    for (int x = 0; x < kAhead; ++x) add(pl[x], po[x], ex2(pm[x] - ref_of(m)));
  }
  if constexpr (kSplit > 1) {
    sm_o[group][lane] = acc;
    if (lane == 0) sm_m[group] = m, sm_l[group] = l;
    __syncthreads();
    if (group != 0) return;
    float top = m;
#pragma unroll
    for (int x = 1; x < kSplit; ++x) top = fmaxf(top, sm_m[x]);
    scale(ex2(m - ref_of(top)));
    m = top;
#pragma unroll
    for (int x = 1; x < kSplit; ++x) add(sm_l[x], sm_o[x][lane], ex2(sm_m[x] - ref_of(m)));
  }
  write(make_float4(l == 0.0f ? 0.0f : acc.x / l, l == 0.0f ? 0.0f : acc.y / l, l == 0.0f ? 0.0f : acc.z / l,
                    l == 0.0f ? 0.0f : acc.w / l),
        log_sum<M>(m, l));
}

// Shared memory of an SM to count on, and what a CTA takes of it beyond the dynamic: at
// most 1 KB of static memory, and 1 KB that the system keeps.
constexpr size_t kSmShared = 227 << 10, kCtaReserve = 2048;

// Rows from which warps work alone.  Measured alone and in teams, where the table
// could hold 131072 tokens a request: bf16, 2048 rows of 100 tokens 28.1 and 32.7
// us, 8192 (4096 requests) 140 and 203, 1024 of up to 1000 45.3 and 45.5, of 500 50.7
// and 47.4; 512 of 500 30.1 and 28.2, of 4096 170 and 165; E4M3, 1024 of up to 1000
// 28.8 and 30.4; fp32 83 and 80.
constexpr int kAloneRows = 1024;

// Tokens of a row that may be attended, by the host's knowledge.
long long row_tokens(const AttendArgs& s) {
  const long long pages = s.picked == nullptr ? s.a.max_pages : std::min(s.top, s.a.max_pages);
  return pages << s.a.shift;
}

// A launch of clusters of `size` CTAs.
struct ClusterLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  ClusterLaunch(long long clusters, int size, size_t smem, cudaStream_t stream) {
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
  }
};

template <int M, int NT, int kTeam>
cudaError_t launch_clusters(const AttendArgs& s, StatusBlock* sb, cudaStream_t stream, long long clusters, int size,
                            size_t smem) {
  auto kern = page_attend_kernel<M, NT, kTeam, true>;
  static bool done[64] = {false};
  cudaError_t err = prepare_kernel(kern, smem, done);
  if (err != cudaSuccess) return err;
  const ClusterLaunch launch(clusters, size, smem, stream);
  note_launch();
  return cudaLaunchKernelEx(&launch.cfg, kern, s, sb);
}

// Clusters of 2^i CTAs that are resident at once: fewer than the SMs' CTAs make, as a
// cluster lies in one group of SMs.  Asked for once per device.
template <int M, int NT>
int resident_clusters(int i, size_t smem) {
  static int known[64][4] = {};  // and one more; 0: not asked yet
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (known[dev][i] == 0) {
    auto kern = page_attend_kernel<M, NT, kWarps, true>;
    static bool done[64] = {false};
    ClusterLaunch launch(1, 1 << i, smem, nullptr);
    launch.cfg.numAttrs = 1;
    int n = 0;
    if (prepare_kernel(kern, smem, done) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &launch.cfg) != cudaSuccess) {
      cudaGetLastError();  // not the next caller's
      return 0;
    }
    known[dev][i] = n + 1;
  }
  return known[dev][i] - 1;
}

// One launch, a cluster to a row: for calls that have few rows, all of whose
// clusters are resident (35 bf16 rows of 1000 tokens: 7.4 us in clusters of 4, 10.6
// in clusters of 8, of which 33 are), and whose rows cannot be long.  It saves the second
// launch and the partial results' way through memory, about 2.5 us and as much
// of the host's time, and loses where lengths differ, as one cluster may then
// have what all would share.  So a CTA has at most kOwnBytes, which a full grid, two
// CTAs an SM, reads in 12 us; twice that of picked pages, of which every long row
// has the same number; but of fp32 pages, whose products take longer, not that, and
// half where the clusters leave SMs free.
// Measured, one launch and two: bf16, 8 KV heads, 8 requests of 250 tokens 5.6
// and 8.6 us, 8 of 2000 14.9 and 18.8, 1 of 4000 8.8 and 10.3, 1 of 8000 13.0
// and 12.2; fp32, 4 of 2000 16.7 and 19.4, 1 of 2000 with one KV head 10.7 and
// 7.4, 5 to 3001 with 7 heads a KV head 18 and 14.  Picked pages of 64, bf16: 8 rows
// of 64 pages 9.0 and 9.6, 32 of 64 15.1 and 19.8, 32 of 96 20.0 and 24.7, 16 of 128
// (kOwnBytes twice) 16.9 and 18.4; E4M3: 8 of 64 7.8 and 9.4, 16 of 128 14.0 and
// 15.8, but 16 of 256 (twice) 22.1 and 20.3; fp32, 8 of 16 7.5 and 9.3.  Clusters of 16 gained 0.7 us
// for one request of 4000 and lost 0.8 for one of 500.  False: the call is not
// one for it.
constexpr long long kOwnBytes = 256 << 10;
template <int M, int NT>
bool launch_own(const AttendArgs& s, StatusBlock* sb, cudaStream_t stream, cudaError_t* err) {
  constexpr int kUnit = kWarps * Tile<M>::keys, kKeyBytes = 2 * kHeadDim * sizeof(typename Tile<M>::E);
  constexpr size_t kSmem = attend_smem<M, NT, kWarps>(0) + kMineFloats<M, NT> * 4;
  static_assert(ctas_per_sm<M, NT>() * (kSmem + kCtaReserve) <= kSmShared, "as many CTAs as are counted on an SM");
  const long long rows = static_cast<long long>(s.a.B) * s.a.kv, units = (row_tokens(s) + kUnit - 1) / kUnit;
  int size = 1;
  for (int i = 1; i < 4 && size < units && rows < resident_clusters<M, NT>(i, kSmem); ++i) size *= 2;
  const long long own = kIsF32<M> ? (rows * size < sm_count() ? kOwnBytes / 2 : kOwnBytes)
                                  : (s.picked != nullptr ? 2 * kOwnBytes : kOwnBytes);
  // What one cluster checks for the status, 32 table entries a thread at most.
  const long long entries = s.picked == nullptr ? static_cast<long long>(s.a.B) * s.a.max_pages : rows * s.top;
  if ((size == 1 && rows >= resident_clusters<M, NT>(0, kSmem)) || (units + size - 1) / size * kUnit * kKeyBytes > own ||
      entries > size * kThreads * 32)
    return false;
  *err = launch_clusters<M, NT, kWarps>(s, sb, stream, rows + 1, size, kSmem);
  return true;
}

// One launch, a warp to a row: where clusters would not all be resident and rows
// cannot be long.  CTAs come and go, so that many short rows need no scan of the
// lengths (whose place in shared memory leaves one CTA an SM for 4096 requests),
// no partial results and no second kernel.  A row may have kWarpBytes, which the
// warps of a full grid, eight an SM, read in 24 us; twice that of 1024 rows or more,
// where the last rows are a small part of the time, but not of fp32, whose rows
// take longer.  Measured, one launch and two: bf16 8192 rows of 100 tokens 82 and
// 140 us as 4096 requests, 80 and 86 as 1024; of 20 43 and 71; 512 of 200 14.7 and
// 17.7; 1024 of 400 37 and 42; 640 to 500 26 and 22; E4M3 1024 of 200 14 and 19, of
// 400 23 and 27, 4096 of 400 76 and 80, but 2048, a few more than the 1776 warps that
// run at once, of 300 40 and 37, of 400 49 and 45; fp32 8192 of 100 162 and 162, 2048
// of 200 98 and 78.  False: the call is not one for it.
constexpr long long kWarpBytes = 128 << 10;
template <int M, int NT>
bool launch_warps(const AttendArgs& s, StatusBlock* sb, cudaStream_t stream, cudaError_t* err) {
  constexpr int kKeyBytes = 2 * kHeadDim * sizeof(typename Tile<M>::E);
  const long long rows = static_cast<long long>(s.a.B) * s.a.kv;
  const long long entries = s.picked == nullptr ? static_cast<long long>(s.a.B) * s.a.max_pages : rows * s.top;
  const long long most = rows >= kAloneRows && !kIsF32<M> ? 2 * kWarpBytes : kWarpBytes;
  if (row_tokens(s) * kKeyBytes > most || entries > kMaxCluster * kThreads * 64) return false;
  constexpr int kRows = kMaxCluster * kWarps;
  *err = launch_clusters<M, NT, 1>(s, sb, stream, (rows + kRows - 1) / kRows + 1, kMaxCluster,
                                   attend_smem<M, NT, 1>(0));
  return true;
}
template <int M, int NT, int kTeam>
cudaError_t launch_attend_t(const AttendArgs& s, StatusBlock* sb, cudaStream_t stream) {
  auto kern = page_attend_kernel<M, NT, kTeam, false>;
  static bool done[64] = {false};
  cudaError_t err = prepare_kernel(kern, attend_smem<M, NT, kTeam>(kMaxRequests), done);
  if (err != cudaSuccess) return err;
  const size_t smem = attend_smem<M, NT, kTeam>(s.a.B);
  // All CTAs are resident at once, as each takes an equal share.  The prefix of many
  // requests takes the place of rings: bf16 has one CTA an SM from 3904 requests on (3800
  // of 100 tokens 60 us, 4000 83; of 500 177 for 3800, 232 for 4096), E4M3 two from 2410
  // on (2300 of 500 68 us, 2500 80), fp32 with up to 4 heads two from 363 on where warps
  // work alone.
  const int per_sm = std::max(1, std::min(ctas_per_sm<M, NT>(), static_cast<int>(kSmShared / (smem + kCtaReserve))));
  constexpr int kCta = kWarps * kLeast<M, kTeam> * Tile<M>::keys;  // tokens that keep a CTA busy
  const long long most = static_cast<long long>(s.a.B) * s.a.kv * ((row_tokens(s) + kCta - 1) / kCta);
  const int ctas = static_cast<int>(std::max(1LL, std::min({static_cast<long long>(sm_count()) * per_sm, most,
                                                             static_cast<long long>(kMaxCtas)})));
  err = launch_pdl(kern, dim3(ctas), dim3(kThreads), smem, stream, s, sb);
  if (err != cudaSuccess) return err;
  // Few rows have many parts each, and leave SMs free: a CTA per head, of four
  // warps, or of sixteen from 8 parts a row on.  Measured, 16, 4 and 1 warps: one row
  // of 65536 tokens with 16 heads, 296 parts, 20.3, 25.5 and 55.6 us; 16 rows of 32768
  // with 4, 18 parts, 48.2, 48.8 and 50.0; 32 of 20000, 9 parts, 57.3, 56.2 and 57.3.
  const int rows = s.a.B * s.a.kv;
  if (static_cast<long long>(rows) * s.G <= 4LL * sm_count()) {
    if (ctas * (kWarps / kTeam) >= 8 * rows) {
      static bool wide_done[64] = {false};
      err = prepare_kernel(page_join_kernel<M, kTeam, 16>, 0, wide_done);
      if (err != cudaSuccess) return err;
      return launch_pdl(page_join_kernel<M, kTeam, 16>, dim3(rows, s.G), dim3(32 * 16), 0, stream, s, ctas, sb);
    }
    static bool split_done[64] = {false};
    err = prepare_kernel(page_join_kernel<M, kTeam, 4>, 0, split_done);
    if (err != cudaSuccess) return err;
    return launch_pdl(page_join_kernel<M, kTeam, 4>, dim3(rows, s.G), dim3(32 * 4), 0, stream, s, ctas, sb);
  }
  static bool join_done[64] = {false};
  err = prepare_kernel(page_join_kernel<M, kTeam, 1>, 0, join_done);
  if (err != cudaSuccess) return err;
  return launch_pdl(page_join_kernel<M, kTeam, 1>, dim3(rows), dim3(32 * s.G), 0, stream, s, ctas, sb);
}

// What ending a row and starting the next costs a worker, in units: rows are laid
// out that much longer, so that a worker with many short rows has fewer tokens.
// Measured, without and with: bf16, 512 rows of up to 4096 tokens, 4 heads 78.5
// and 76.8 us (2: 77.1), 16 heads 100 and 82.7 (1: 92, 2: 85, 8: 82); fp32, 256
// rows, 7 heads 94 and 81 (1: 86, 4: 82), 16 heads 129 and 106 (2: 107, 8: 111).
// Rows of one length take the same time either way.
int row_cost(int G) { return G <= 4 ? 1 : G <= 8 ? 2 : 4; }

template <int M, int NT>
cudaError_t launch_attend(const AttendArgs& s, StatusBlock* sb, cudaStream_t stream) {
  cudaError_t err = cudaSuccess;
  if (launch_own<M, NT>(s, sb, stream, &err)) return err;
  if (launch_warps<M, NT>(s, sb, stream, &err)) return err;
  return static_cast<long long>(s.a.B) * s.a.kv >= kAloneRows ? launch_attend_t<M, NT, 1>(s, sb, stream)
                                                              : launch_attend_t<M, NT, kWarps>(s, sb, stream);
}

}  // namespace

cudaError_t launch_page_attend(const void* q, long long q_stride, int G, const PageArgs& a, mova_dtype dt, float scale,
                               const int32_t* picked, int top, void* o, float* lse, const PageWs& ws,
                               cudaStream_t stream) {
  const int extra = static_cast<long long>(a.B) * a.kv < (1 << 26) ? row_cost(G) : 0;
  const AttendArgs s{a, q, q_stride, G, scale, picked, top, o, lse, ws.bad, ws.prefix, ws.part, extra};
  if (dt == MOVA_F32) {
    if (G <= 4) return launch_attend<kF32, 4>(s, ws.sb, stream);
    if (G <= 8) return launch_attend<kF32Parts, 1>(s, ws.sb, stream);
    return launch_attend<kF32Parts, 2>(s, ws.sb, stream);
  }
  if (dt == MOVA_BF16) {
    if (G <= 8) return launch_attend<kB16, 1>(s, ws.sb, stream);
    return launch_attend<kB16, 2>(s, ws.sb, stream);
  }
  if (G <= 8) return launch_attend<kE8, 1>(s, ws.sb, stream);
  return launch_attend<kE8, 2>(s, ws.sb, stream);
}

}  // namespace mova

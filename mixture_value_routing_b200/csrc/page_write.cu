// Writing new tokens into cache pages, and the pages' key bounds.
//
// page_write: cache[slot / page_size, h, slot % page_size, :] = k[t, h, :] (v
// alike), converted to the pages' type; E4M3 as round(k / scale), the quotient
// formed in fp32 (IEEE division) and clamped to +-448.  Each element is read
// and written once: a copy, bound by memory (16384 tokens of 8 bf16 heads, 134
// MB: 22.8 us, 5.9 TB/s; loads and stores marked as streams, 25.2 us without
// and with smaller CTAs; fp32, 269 MB: 43.3 us, 6.2 TB/s).  E4M3, 101 MB, takes 23.5
// us, 4.3 TB/s: at 64 registers a thread to the others' 32 it has half as many warps
// an SM.  A warp takes one token's keys or
// values -- kv_heads * 128 elements, contiguous on the input side and 128 at a
// time in the cache -- with 16-byte loads that do not wait for the slot.
//
// page_bounds: lo / hi[page, h, d] = min / max over the page's keys, for pages
// that the step filled: page_size * 128 elements read for 256 written, bound
// by memory.  Four warps share a (page, head), 16 keys each (E4M3: 64) in flight at
// once, in packed 16-bit minima and maxima, and join in shared memory, one barrier a
// page.  737 pages of 64 keys, 8 heads: fp32, 199 MB, 33.5 us, bf16 18.4, E4M3, 50
// MB, 13.3; the first 4 us are the scan of the requests, the table and the first keys.
#include <math.h>

#include "paged.cuh"

namespace mova {

namespace {

// A 16-byte load of data that is read once.  Not a read-only (.nc) load, and no
// pointer here is __restrict__: the kernel before this one on the stream may
// have written the data while this one was already launched.
__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], %5;"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p), "l"(evict_first_policy()) : "memory");
  return r;
}

constexpr int kWriteSmall = 1024;  // CTAs of 512 threads from this many tokens on, 256 below

// x / scale as IEEE division rounds it, from r, the rounded reciprocal of scale:
// a quotient and one correction by its exact remainder (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// 1990, theorem on division), for |x| < 2^60 and scale from 2^-60 to 2^40.
// Signs of zeros come out as the division's; quotients too small for the
// theorem are 0 in E4M3 either way.
__device__ __forceinline__ float quotient(float x, float scale, float r) {
  const float q = x * r;
  return fmaf(-fmaf(q, scale, -x), r, q);
}

// One unit of a thread: the 16-byte loads whose elements fill 16 bytes of the cache.
template <typename In, typename Out> struct Unit {
  static constexpr int kPer = 16 / sizeof(Out);             // elements
  static constexpr int kLoads = sizeof(In) / sizeof(Out);   // 16-byte loads
  uint4 x[kLoads];
  __device__ __forceinline__ void load(const In* p) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x[i] = load_once(p + i * (16 / sizeof(In)));
  }
  __device__ __forceinline__ void store(Out* p, float scale) const {
    if constexpr (sizeof(Out) > 1)
      __stcs(reinterpret_cast<uint4*>(p), x[0]);
    else
      __stcs(reinterpret_cast<uint4*>(p), quantised(scale));
  }
  // 16 bf16 elements over the scale, as E4M3.
  __device__ __forceinline__ uint4 quantised(float scale) const {
    const uint32_t w[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
    uint32_t big = scale > 0x1p-60f && scale < 0x1p40f ? 0u : 1u;  // outside quotient()'s range
#pragma unroll
    for (int i = 0; i < 8; ++i) big |= ((w[i] & 0x7f807f80u) + 0x22802280u) & 0x80008000u;  // exponents from 60 on
    const float r = __frcp_rn(scale);
    uint32_t out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
      out[i] = __nv_cvt_float2_to_fp8x2(make_float2(quotient(lo, scale, r), quotient(hi, scale, r)), __NV_SATFINITE,
                                        __NV_E4M3);
    }
    if (big != 0u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xffff0000u);
        out[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(lo, scale), __fdiv_rn(hi, scale)), __NV_SATFINITE,
                                          __NV_E4M3);
      }
    }
    return make_uint4(out[0] | (out[1] << 16), out[2] | (out[3] << 16), out[4] | (out[5] << 16),
                      out[6] | (out[7] << 16));
  }
};

template <typename In, typename Out, int kThreads>
__global__ void __launch_bounds__(kThreads)
page_write_kernel(const In* k, const In* v, long long k_stride, long long v_stride,
                  const int32_t* slots, int T, Out* kc, Out* vc,
                  long long kp_stride, long long vp_stride, const float* k_scale, const float* v_scale, int kv,
                  int shift, int num_slots, int lanes, StatusBlock* sb) {
  using U = Unit<In, Out>;
  constexpr int kPer = U::kPer;
  constexpr int kUnroll = 4 / U::kLoads;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x == gridDim.x - 1) {
    // The last CTA only looks the slots over and writes the status.
    __shared__ int bad;
    if (tid == 0) bad = kNoBad;
    __syncthreads();
    int mine = kNoBad;
#pragma unroll 8
    for (int t = tid; t < T; t += kThreads) {
      const int slot = slots[t];
      if (slot < -1 || slot >= num_slots) mine = min(mine, t);
    }
    if (mine != kNoBad) atomicMin(&bad, mine);
    __syncthreads();
    if (tid == 0) {
      sb->code = bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
      sb->detail = bad == kNoBad ? 0 : bad;
    }
    return;
  }
  // `lanes` (8, 16 or 32) threads per (token, keys or values).
  const long long unit = (static_cast<long long>(blockIdx.x) * kThreads + tid) / lanes;
  const int lane = tid % lanes;
  const int t = static_cast<int>(unit >> 1);
  if (t >= T) return;
  const bool is_v = unit & 1;
  const In* src = is_v ? v + t * v_stride : k + t * k_stride;
  Out* cache = is_v ? vc : kc;
  const float* scale = is_v ? v_scale : k_scale;
  const int chunks = kv * (kHeadDim / kPer);
  const int slot = slots[t];
  const bool ok = slot >= 0 && slot < num_slots;
  const long long base =
      ok ? (slot >> shift) * (is_v ? vp_stride : kp_stride) + static_cast<long long>(slot & ((1 << shift) - 1)) * kHeadDim
         : 0;
  for (int c0 = lane; c0 < chunks; c0 += lanes * kUnroll) {
    U x[kUnroll];
    float f[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * lanes;
      f[i] = 1.0f;
      if (c < chunks) {
        x[i].load(src + c * kPer);
        if (sizeof(Out) == 1 && scale != nullptr) f[i] = scale[c / (kHeadDim / kPer)];
      }
    }
    if (!ok) return;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * lanes;
      if (c < chunks) {
        const int h = c / (kHeadDim / kPer), d = (c % (kHeadDim / kPer)) * kPer;
        x[i].store(cache + base + (static_cast<long long>(h) << shift) * kHeadDim + d, f[i]);
      }
    }
  }
}

template <typename In, typename Out, int kThreads>
cudaError_t launch_write_t(const void* k, const void* v, long long k_stride, long long v_stride, const int32_t* slots,
                           int T, const mova_pages& p, int shift, StatusBlock* sb, cudaStream_t stream) {
  const int units = p.kv_heads * (kHeadDim / Unit<In, Out>::kPer);
  const int lanes = units >= 32 ? 32 : units >= 16 ? 16 : 8;
  const long long blocks = (2LL * T * lanes + kThreads - 1) / kThreads;
  return launch_pdl(page_write_kernel<In, Out, kThreads>, dim3(static_cast<unsigned>(blocks + 1)), dim3(kThreads), 0,
                    stream, static_cast<const In*>(k), static_cast<const In*>(v), k_stride, v_stride, slots, T,
                    static_cast<Out*>(p.k), static_cast<Out*>(p.v), p.k_page_stride, p.v_page_stride, p.k_scale,
                    p.v_scale, p.kv_heads, shift, p.num_pages << shift, lanes, sb);
}

// Measured for 16384 tokens of 8 heads, bf16, before stores were marked as streams:
// 23.5 us with 512 threads, 25.2 with 256, 27.1 with 1024; for 64 tokens 2.3, 1.9
// and 3.1.
template <typename In, typename Out, typename... Args>
cudaError_t launch_write(int T, Args... args) {
  return T < kWriteSmall ? launch_write_t<In, Out, 256>(args...) : launch_write_t<In, Out, 512>(args...);
}

// ---- Bounds --------------------------------------------------------------------

constexpr int kBoundThreads = 128;
constexpr int kBoundPerSm = 8;

// Least and greatest of packed elements, NaN if either operand is NaN.
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }
template <typename T> __device__ __forceinline__ T from_u32(uint32_t v) { return *reinterpret_cast<T*>(&v); }

// Bounds of one 16-byte chunk of a key: kWords 32-bit words of packed fp32,
// bf16 or (for E4M3, exactly) fp16.  store: the words that a lane keeps.
template <typename E> struct Range;
template <> struct Range<float> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void load(const uint4& u, uint32_t (&w)[4]) { w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w; }
  static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
  }
  static __device__ __forceinline__ uint32_t greatest(uint32_t a, uint32_t b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
  }
  static __device__ __forceinline__ void store(float* p, const uint32_t (&w)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <> struct Range<__nv_bfloat16> {
  static constexpr int kWords = 4;
  static __device__ __forceinline__ void load(const uint4& u, uint32_t (&w)[4]) { w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w; }
  static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
    return as_u32(__hmin2_nan(from_u32<__nv_bfloat162>(a), from_u32<__nv_bfloat162>(b)));
  }
  static __device__ __forceinline__ uint32_t greatest(uint32_t a, uint32_t b) {
    return as_u32(__hmax2_nan(from_u32<__nv_bfloat162>(a), from_u32<__nv_bfloat162>(b)));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const uint32_t (&w)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
};
template <> struct Range<uint8_t> {
  static constexpr int kWords = 8;
  static __device__ __forceinline__ void load(const uint4& u, uint32_t (&w)[8]) {
    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[i] = as_u32(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(in[i >> 1] >> (16 * (i & 1))), __NV_E4M3)));
  }
  static __device__ __forceinline__ uint32_t least(uint32_t a, uint32_t b) {
    return as_u32(__hmin2_nan(from_u32<__half2>(a), from_u32<__half2>(b)));
  }
  static __device__ __forceinline__ uint32_t greatest(uint32_t a, uint32_t b) {
    return as_u32(__hmax2_nan(from_u32<__half2>(a), from_u32<__half2>(b)));
  }
  static __device__ __forceinline__ void store(uint8_t* p, const uint32_t (&w)[8]) {
    const uint32_t a = __nv_cvt_halfraw2_to_fp8x2(from_u32<__half2_raw>(w[0]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_halfraw2_to_fp8x2(from_u32<__half2_raw>(w[1]), __NV_SATFINITE, __NV_E4M3);
    *reinterpret_cast<uint32_t*>(p) = a | (b << 16);
  }
};

template <typename E>
__global__ void __launch_bounds__(kBoundThreads)
page_bounds_kernel(const PageArgs a, const int32_t* cached, E* lo, E* hi,
                   StatusBlock* sb) {
  using R = Range<E>;
  constexpr int kPer = 16 / sizeof(E);
  constexpr int kCols = kHeadDim / kPer;  // 16-byte chunks of a key
  constexpr int kRows = 32 / kCols;       // keys of one warp-wide load
  // Keys of a warp.  E4M3: 64, where 16 took 16.0 us for 50 MB and 64 takes 12.8.
  constexpr int kTake = sizeof(E) == 1 ? 64 : 16;
  constexpr int kLoads = 16 / kRows;
  constexpr int kWarps = kBoundThreads / 32;
  constexpr int kKept = R::kWords / kRows;  // words of a lane once the warp's rows are joined
  __shared__ uint32_t red[2][kWarps][2][kKept][32];
  extern __shared__ int pre[];
  __shared__ int bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) bad = kNoBad;
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  auto first_page = [&](int b) {
    const int c = cached[b];
    return (c < 0 ? 0 : c) >> a.shift;
  };
  request_scan<kBoundThreads>(a.B, pre, [&](int b) {
    const int len = a.lens[b], use = clamp_len(len, a.max_pages, a.shift);
    if (use != len || cached[b] < 0) atomicMin(&bad, b);
    const int n = (use >> a.shift) - first_page(b);
    return n < 0 ? 0 : n;
  });
  const int items = pre[a.B];
  auto page_of = [&](int item, int* b) {
    *b = request_of(pre, a.B, item);
    return a.table[*b * a.table_stride + first_page(*b) + item - pre[*b]];
  };
  if (blockIdx.x == gridDim.x - 1) {
    // The last CTA only looks the pages over and writes the status.
    for (int i = tid; i < items; i += kBoundThreads) {
      int b;
      const int page = page_of(i, &b);
      if (page < 0 || page >= a.num_pages) atomicMin(&bad, b);
    }
    __syncthreads();
    if (tid == 0) {
      sb->code = bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
      sb->detail = bad == kNoBad ? 0 : bad;
    }
    return;
  }
  // A warp reads kTake keys of one (page, head), or of a long page a quarter, so
  // that a CTA takes whole pages: `share` warps each, 4 / share at a time.
  const int share = max(1, min(kWarps, (1 << a.shift) / kTake)), rows = (1 << a.shift) / share;
  const int part = warp & (share - 1), lane_pair = warp / share, pairs = kWarps / share;  // powers of two
  const int col = lane % kCols, row0 = lane / kCols;
  // First of the elements of the chunk whose bounds this lane comes to hold.
  int kept0 = 0;
#pragma unroll
  for (int o = kCols, n = kPer / 2; o < 32; o <<= 1, n /= 2) kept0 += lane & o ? n : 0;
  const int work = items * a.kv, CTAs = gridDim.x - 1;  // work: below 2^30, as the entry point has checked
  const int x0 = static_cast<int>(static_cast<long long>(blockIdx.x) * work / CTAs);
  const int x1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * work / CTAs);
  int t_page = -1, t_head = 0;  // of (page, head) number 32 n + lane from x0
  for (int x = x0, i = 0, round = 0; x < x1; x += pairs, i += pairs, ++round) {
    const int buf = round & 1;
    if ((i & 31) == 0) {
      int b;
      t_page = -1;
      if (x + lane < x1) {
        const int item = (x + lane) / a.kv;
        t_page = page_of(item, &b);
        t_head = x + lane - item * a.kv;
        if (t_page >= a.num_pages) t_page = -1;
      }
    }
    const int page = __shfl_sync(0xffffffffu, t_page, (i + lane_pair) & 31);  // -1 past x1
    const int h = __shfl_sync(0xffffffffu, t_head, (i + lane_pair) & 31);
    uint32_t l[R::kWords], u[R::kWords];
    if (page >= 0) {
      const E* src = static_cast<const E*>(a.k) + page * a.k_stride +
                     ((static_cast<long long>(h) << a.shift) + part * rows + row0) * kHeadDim + col * kPer;
      bool first = true;
#pragma unroll 4
      for (int r = 0; r < rows; r += 16) {
        uint4 raw[kLoads];
#pragma unroll
        for (int y = 0; y < kLoads; ++y) raw[y] = load_once(src + (r + y * kRows) * kHeadDim);
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          uint32_t v[R::kWords];
          R::load(raw[y], v);
#pragma unroll
          for (int j = 0; j < R::kWords; ++j) {
            l[j] = y == 0 && first ? v[j] : R::least(l[j], v[j]);
            u[j] = y == 0 && first ? v[j] : R::greatest(u[j], v[j]);
          }
        }
        first = false;
      }
      // Joins the kRows keys that a load holds: a lane hands on half its words and
      // keeps the other half, so each ends with kKept words of its chunk.
#pragma unroll
      for (int o = kCols, n = R::kWords / 2; o < 32; o <<= 1, n /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int j = 0; j < n; ++j) {
          const uint32_t lo_give = upper ? l[j] : l[j + n], lo_keep = upper ? l[j + n] : l[j];
          const uint32_t hi_give = upper ? u[j] : u[j + n], hi_keep = upper ? u[j + n] : u[j];
          l[j] = R::least(lo_keep, __shfl_xor_sync(0xffffffffu, lo_give, o));
          u[j] = R::greatest(hi_keep, __shfl_xor_sync(0xffffffffu, hi_give, o));
        }
      }
    }
    const int writer = round & (share - 1);  // the warps of a page take turns
    if (share > 1) {
      // One barrier a round: the other buffer is read until the next one.
      if (page >= 0 && part != writer) {
#pragma unroll
        for (int j = 0; j < kKept; ++j) red[buf][warp][0][j][lane] = l[j], red[buf][warp][1][j][lane] = u[j];
      }
      __syncthreads();
    }
    if (page >= 0 && part == writer) {
      for (int y = 1; y < share; ++y) {
        const int from = lane_pair * share + ((part + y) & (share - 1));
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
          l[j] = R::least(l[j], red[buf][from][0][j][lane]);
          u[j] = R::greatest(u[j], red[buf][from][1][j][lane]);
        }
      }
      const long long out = (static_cast<long long>(page) * a.kv + h) * kHeadDim + col * kPer + kept0;
      R::store(lo + out, l);
      R::store(hi + out, u);
    }
  }
}

template <typename E>
cudaError_t launch_bounds_t(const PageArgs& a, const int32_t* cached, void* lo, void* hi, StatusBlock* sb,
                            cudaStream_t stream) {
  const long long most = static_cast<long long>(a.B) * a.max_pages * a.kv;
  const long long grid = static_cast<long long>(sm_count()) * kBoundPerSm;
  return launch_pdl(page_bounds_kernel<E>, dim3(static_cast<unsigned>((most < grid ? most : grid) + 1)),
                    dim3(kBoundThreads), static_cast<size_t>(a.B + 1) * 4, stream, a, cached, static_cast<E*>(lo),
                    static_cast<E*>(hi), sb);
}

}  // namespace

cudaError_t launch_page_write(const void* k, const void* v, mova_dtype dt, long long k_stride, long long v_stride,
                              const int32_t* slots, int T, const mova_pages& p, StatusBlock* sb, cudaStream_t stream) {
  int shift = 0;
  while ((1 << shift) < p.page_size) ++shift;
  (void)dt;
  if (p.dtype == MOVA_F32)
    return launch_write<float, float>(T, k, v, k_stride, v_stride, slots, T, p, shift, sb, stream);
  if (p.dtype == MOVA_BF16)
    return launch_write<__nv_bfloat16, __nv_bfloat16>(T, k, v, k_stride, v_stride, slots, T, p, shift, sb, stream);
  return launch_write<__nv_bfloat16, uint8_t>(T, k, v, k_stride, v_stride, slots, T, p, shift, sb, stream);
}

cudaError_t launch_page_bounds(const PageArgs& a, mova_dtype dt, const int32_t* cached, void* lo, void* hi,
                               StatusBlock* sb, cudaStream_t stream) {
  if (dt == MOVA_F32) return launch_bounds_t<float>(a, cached, lo, hi, sb, stream);
  if (dt == MOVA_BF16) return launch_bounds_t<__nv_bfloat16>(a, cached, lo, hi, sb, stream);
  return launch_bounds_t<uint8_t>(a, cached, lo, hi, sb, stream);
}

}  // namespace mova

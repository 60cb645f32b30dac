// Writing new tokens into cache pages, and the pages' key bounds.
//
// page_write: cache[slot / page_size, h, slot % page_size, :] = k[t, h, :] (v
// alike), converted to the pages' type; E4M3 as round(k / scale), the quotient
// formed in fp32 (IEEE division) and clamped to +-448.  Each element is read
// and written once: a copy, bound by memory (16384 tokens of 8 bf16 heads, 134
// MB: 22.7 us, 5.9 TB/s; loads and stores marked as streams, 25.2 us without
// and with smaller CTAs).  A warp takes one token's keys or
// values -- kv_heads * 128 elements, contiguous on the input side and 128 at a
// time in the cache -- with 16-byte loads that do not wait for the slot.
//
// page_bounds: lo / hi[page, h, d] = min / max over the page's keys, for pages
// that the step filled: page_size * 128 elements read for 256 written, bound
// by memory.  Four warps share a (page, head), 16 keys each in flight at once, in
// packed 16-bit minima and maxima, and join in shared memory, one barrier a page.
#include <math.h>

#include "paged.cuh"

namespace mova {

namespace {

constexpr int kWriteSmall = 1024;  // CTAs of 512 threads from this many tokens on, 256 below

template <typename In> constexpr int per_chunk() { return 16 / sizeof(In); }

__device__ __forceinline__ uint8_t to_e4m3(float x, float scale) {
  const float y = __fdiv_rn(x, scale);
  return __nv_cvt_float_to_fp8(y, __NV_SATFINITE, __NV_E4M3);
}

// Stores one 16-byte input chunk at element `at` of the cache.
__device__ __forceinline__ void store_chunk(float* cache, long long at, const uint4& x, float) {
  __stcs(reinterpret_cast<uint4*>(cache + at), x);
}
__device__ __forceinline__ void store_chunk(__nv_bfloat16* cache, long long at, const uint4& x, float) {
  __stcs(reinterpret_cast<uint4*>(cache + at), x);
}
__device__ __forceinline__ void store_chunk(uint8_t* cache, long long at, const uint4& x, float scale) {
  const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&x);
  uint32_t out[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    out[i >> 2] |= static_cast<uint32_t>(to_e4m3(__bfloat162float(e[i]), scale)) << (8 * (i & 3));
  __stcs(reinterpret_cast<uint2*>(cache + at), make_uint2(out[0], out[1]));
}

template <typename In, typename Out, int kThreads>
__global__ void __launch_bounds__(kThreads)
page_write_kernel(const In* __restrict__ k, const In* __restrict__ v, long long k_stride, long long v_stride,
                  const int32_t* __restrict__ slots, int T, Out* __restrict__ kc, Out* __restrict__ vc,
                  long long kp_stride, long long vp_stride, const float* k_scale, const float* v_scale, int kv,
                  int shift, int num_slots, int lanes, StatusBlock* sb) {
  constexpr int kPer = per_chunk<In>();
  constexpr int kUnroll = 4;
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
  // `lanes` (16 or 32) threads per (token, keys or values).
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
    uint4 x[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * lanes;
      if (c < chunks) x[i] = ld_stream_u4(src + c * kPer);
    }
    if (!ok) return;
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const int c = c0 + i * lanes;
      if (c < chunks) {
        const int h = c / (kHeadDim / kPer), d = (c % (kHeadDim / kPer)) * kPer;
        const float s = scale == nullptr ? 1.0f : scale[h];
        store_chunk(cache, base + (static_cast<long long>(h) << shift) * kHeadDim + d, x[i], s);
      }
    }
  }
}

template <typename In, typename Out, int kThreads>
cudaError_t launch_write_t(const void* k, const void* v, long long k_stride, long long v_stride, const int32_t* slots,
                           int T, const mova_pages& p, int shift, StatusBlock* sb, cudaStream_t stream) {
  const int lanes = p.kv_heads * (kHeadDim / per_chunk<In>()) >= 32 ? 32 : 16;
  const long long blocks = (2LL * T * lanes + kThreads - 1) / kThreads;
  return launch_pdl(page_write_kernel<In, Out, kThreads>, dim3(static_cast<unsigned>(blocks + 1)), dim3(kThreads), 0,
                    stream, static_cast<const In*>(k), static_cast<const In*>(v), k_stride, v_stride, slots, T,
                    static_cast<Out*>(p.k), static_cast<Out*>(p.v), p.k_page_stride, p.v_page_stride, p.k_scale,
                    p.v_scale, p.kv_heads, shift, p.num_pages << shift, lanes, sb);
}

// Measured for 16384 tokens of 8 heads, bf16: 23.5 us with 512 threads, 25.2
// with 256, 27.1 with 1024 (plain stores); for 64 tokens 2.3, 1.9 and 3.1.
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
// bf16 or (for E4M3, exactly) fp16.
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
  static __device__ __forceinline__ uint4 store(const uint32_t (&w)[4]) { return make_uint4(w[0], w[1], w[2], w[3]); }
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
  static __device__ __forceinline__ uint4 store(const uint32_t (&w)[4]) { return make_uint4(w[0], w[1], w[2], w[3]); }
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
  static __device__ __forceinline__ uint4 store(const uint32_t (&w)[8]) {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = __nv_cvt_halfraw2_to_fp8x2(from_u32<__half2_raw>(w[2 * i]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_halfraw2_to_fp8x2(from_u32<__half2_raw>(w[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      out[i] = lo | (hi << 16);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
};

template <typename E>
__global__ void __launch_bounds__(kBoundThreads)
page_bounds_kernel(const PageArgs a, const int32_t* __restrict__ cached, E* __restrict__ lo, E* __restrict__ hi,
                   StatusBlock* sb) {
  using R = Range<E>;
  constexpr int kPer = 16 / sizeof(E);
  constexpr int kCols = kHeadDim / kPer;  // 16-byte chunks of a key
  constexpr int kRows = 32 / kCols;       // keys of one warp-wide load
  constexpr int kLoads = 16 / kRows;      // of 16 keys, in flight at once
  constexpr int kWarps = kBoundThreads / 32;
  __shared__ uint32_t red[2][kWarps][2][R::kWords][kCols];
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
  // A warp reads 16 keys of one (page, head), or of a long page a quarter, so
  // that a CTA takes whole pages: `share` warps each, 4 / share at a time.
  const int share = min(kWarps, (1 << a.shift) >> 4), rows = (1 << a.shift) / share;
  const int part = warp % share, lane_pair = warp / share, pairs = kWarps / share;
  const int col = lane % kCols, row0 = lane / kCols;
  const int work = items * a.kv, CTAs = gridDim.x - 1;  // work: below 2^30, as the entry point has checked
  const int x0 = static_cast<int>(static_cast<long long>(blockIdx.x) * work / CTAs);
  const int x1 = static_cast<int>(static_cast<long long>(blockIdx.x + 1) * work / CTAs);
  int t_page = -1;  // page of (page, head) number 32 n + lane from x0
  for (int x = x0, i = 0, buf = 0; x < x1; x += pairs, i += pairs, buf ^= 1) {
    if ((i & 31) == 0) {
      int b;
      t_page = x + lane < x1 ? page_of((x + lane) / a.kv, &b) : -1;
      if (t_page >= a.num_pages) t_page = -1;
    }
    const int page = __shfl_sync(0xffffffffu, t_page, (i + lane_pair) & 31);  // -1 past x1
    uint32_t l[R::kWords], u[R::kWords];
    const int h = static_cast<unsigned>(x + lane_pair) % a.kv;
    if (page >= 0) {
      const E* src = static_cast<const E*>(a.k) + page * a.k_stride +
                     ((static_cast<long long>(h) << a.shift) + part * rows + row0) * kHeadDim + col * kPer;
      for (int r = 0; r < rows; r += kRows * kLoads) {
        uint4 raw[kLoads];
#pragma unroll
        for (int y = 0; y < kLoads; ++y) raw[y] = ld_stream_u4(src + (r + y * kRows) * kHeadDim);
#pragma unroll
        for (int y = 0; y < kLoads; ++y) {
          uint32_t v[R::kWords];
          R::load(raw[y], v);
#pragma unroll
          for (int j = 0; j < R::kWords; ++j) {
            l[j] = y == 0 && r == 0 ? v[j] : R::least(l[j], v[j]);
            u[j] = y == 0 && r == 0 ? v[j] : R::greatest(u[j], v[j]);
          }
        }
      }
#pragma unroll
      for (int o = kCols; o < 32; o <<= 1)
#pragma unroll
        for (int j = 0; j < R::kWords; ++j) {
          l[j] = R::least(l[j], __shfl_xor_sync(0xffffffffu, l[j], o));
          u[j] = R::greatest(u[j], __shfl_xor_sync(0xffffffffu, u[j], o));
        }
    }
    const int writer = i / pairs % share;  // the warps of a page take turns
    if (share > 1) {
      // One barrier a round: the other buffer is read until the next one.
      if (page >= 0 && lane < kCols && part != writer) {
#pragma unroll
        for (int j = 0; j < R::kWords; ++j) red[buf][warp][0][j][lane] = l[j], red[buf][warp][1][j][lane] = u[j];
      }
      __syncthreads();
    }
    if (page >= 0 && lane < kCols && part == writer) {
      for (int y = 1; y < share; ++y) {
        const int from = lane_pair * share + (part + y) % share;
#pragma unroll
        for (int j = 0; j < R::kWords; ++j) {
          l[j] = R::least(l[j], red[buf][from][0][j][lane]);
          u[j] = R::greatest(u[j], red[buf][from][1][j][lane]);
        }
      }
      const long long out = (static_cast<long long>(page) * a.kv + h) * kHeadDim + col * kPer;
      *reinterpret_cast<uint4*>(lo + out) = R::store(l);
      *reinterpret_cast<uint4*>(hi + out) = R::store(u);
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

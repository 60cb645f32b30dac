// C ABI entry points of the paged key-value cache: argument checks, workspace
// layout, and the enqueueing of the kernels on the caller's stream.
#include <stddef.h>
#include <stdio.h>

#include "paged.cuh"

namespace mova {

namespace {

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
bool aligned(const void* p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
bool elem_size(mova_dtype dt, long long* out) {
  *out = dt == MOVA_F32 ? 4 : dt == MOVA_BF16 ? 2 : 1;
  return dt == MOVA_F32 || dt == MOVA_BF16 || dt == MOVA_E4M3;
}

mova_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MOVA_OK;
  fprintf(stderr, "mova: CUDA error %s\n", cudaGetErrorString(e));
  return MOVA_ERR_CUDA;
}

// The smallest workspace: the status word alone.
constexpr size_t kStatusBytes = 256;

mova_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
  return ws == nullptr || !aligned(ws, 256) || ws_bytes < need ? MOVA_ERR_INVALID_ARG : MOVA_OK;
}

// A call of no tokens or requests does nothing but say so in the workspace, if
// it has one.
mova_status empty_call(void* ws, size_t ws_bytes, void* stream) {
  static_assert(MOVA_OK == 0, "the status is set by a memset");
  if (ws == nullptr) return MOVA_OK;
  const mova_status st = check_ws(ws, ws_bytes, kStatusBytes);
  if (st != MOVA_OK) return st;
  return from_cuda(cudaMemsetAsync(ws, 0, offsetof(StatusBlock, num_active), static_cast<cudaStream_t>(stream)));
}

int shift_of(int page_size) {
  for (int s = 4; s <= 8; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

mova_status check_batch(int B, int max_pages, int kv) {
  if (B < 0 || max_pages <= 0 || kv <= 0) return MOVA_ERR_INVALID_ARG;
  return B > kMaxRequests ? MOVA_ERR_UNSUPPORTED : MOVA_OK;
}

mova_status check_heads(int kv, int H) {
  if (kv <= 0 || H <= 0) return MOVA_ERR_INVALID_ARG;
  return H % kv != 0 || H / kv > kMaxGroup ? MOVA_ERR_UNSUPPORTED : MOVA_OK;
}

// The cache's description; dense strides filled in.
mova_status read_pages(const mova_pages* p, mova_pages* out) {
  if (p == nullptr) return MOVA_ERR_INVALID_ARG;
  *out = *p;
  long long es;
  if (!elem_size(p->dtype, &es)) return MOVA_ERR_UNSUPPORTED;
  if (p->num_pages <= 0 || p->kv_heads <= 0 || p->page_size <= 0) return MOVA_ERR_INVALID_ARG;
  if (shift_of(p->page_size) < 0) return MOVA_ERR_UNSUPPORTED;
  if (static_cast<long long>(p->num_pages) * p->page_size >= (1LL << 31)) return MOVA_ERR_UNSUPPORTED;
  const long long dense = static_cast<long long>(p->kv_heads) * p->page_size * kHeadDim;
  for (long long* s : {&out->k_page_stride, &out->v_page_stride}) {
    if (*s == 0) *s = dense;
    if (*s < dense || *s > (1LL << 40) || (*s * es) % 16 != 0) return MOVA_ERR_INVALID_ARG;
  }
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->k_scale, 4) || !aligned(p->v_scale, 4))
    return MOVA_ERR_INVALID_ARG;
  if (p->dtype != MOVA_E4M3) out->k_scale = out->v_scale = nullptr;
  return MOVA_OK;
}

bool io_fits(mova_dtype io, mova_dtype pages) {
  return pages == MOVA_F32 ? io == MOVA_F32 : io == MOVA_BF16;
}

// Tokens (or requests) `stride` elements apart, each of `width`; 0: dense.
mova_status read_stride(long long* stride, long long width, mova_dtype dt) {
  long long es;
  elem_size(dt, &es);
  if (*stride == 0) *stride = width;
  return *stride < width || *stride > (1LL << 40) || (*stride * es) % 16 != 0 ? MOVA_ERR_INVALID_ARG : MOVA_OK;
}

// The requests' tables and lengths, with the limits on their sizes.
mova_status read_table(const mova_pages& p, const int32_t* table, long long table_stride, int max_pages,
                       const int32_t* lens, int B, PageArgs* out) {
  mova_status st = check_batch(B, max_pages, p.kv_heads);
  if (st != MOVA_OK) return st;
  const long long tokens = static_cast<long long>(max_pages) * p.page_size;
  if (tokens > (1LL << 30)) return MOVA_ERR_UNSUPPORTED;
  if (static_cast<double>(tokens) * B * p.kv_heads >= static_cast<double>(1LL << 33)) return MOVA_ERR_UNSUPPORTED;
  if (table_stride == 0) table_stride = max_pages;
  if (table_stride < max_pages || table_stride > (1LL << 40)) return MOVA_ERR_INVALID_ARG;
  if (B > 0 && (!table || !lens || !aligned(table, 4) || !aligned(lens, 4))) return MOVA_ERR_INVALID_ARG;
  *out = PageArgs{p.k,      p.v,         p.k_page_stride, p.v_page_stride,        p.k_scale, p.v_scale,
                  p.num_pages, p.kv_heads, shift_of(p.page_size), table, table_stride, max_pages, lens, B};
  return MOVA_OK;
}

PageWs layout(void* base, int B, int max_pages, int kv, int H) {
  char* b = static_cast<char*>(base);
  size_t o = 0;
  PageWs w{};
  w.sb = reinterpret_cast<StatusBlock*>(b);
  o += kStatusBytes;
  w.bad = reinterpret_cast<int32_t*>(b + o);
  o += align256(kMaxCtas * sizeof(int32_t));
  w.prefix = reinterpret_cast<int32_t*>(b + o);
  o += align256(static_cast<size_t>(B + 1) * sizeof(int32_t));
  // The scores are gone before the attention that follows writes partial results.
  w.part = reinterpret_cast<float*>(b + o);
  w.keys = reinterpret_cast<unsigned long long*>(b + o);
  const size_t part = static_cast<size_t>(kMaxWorkers) * 2 * (H / kv) * kPartRow * sizeof(float);
  const size_t keys = static_cast<size_t>(B) * kv * max_pages * sizeof(unsigned long long);
  o += align256(part > keys ? part : keys);
  w.bytes = o;
  return w;
}

}  // namespace
}  // namespace mova

using namespace mova;

extern "C" {

size_t mova_page_workspace_size(int B, int max_pages, int kv_heads, int H) {
  if (check_batch(B, max_pages, kv_heads) != MOVA_OK || check_heads(kv_heads, H) != MOVA_OK) return 0;
  if (static_cast<double>(max_pages) * B * kv_heads >= static_cast<double>(1LL << 30)) return 0;
  return layout(nullptr, B, max_pages, kv_heads, H).bytes;
}

mova_status mova_page_map(const int32_t* cached, const int32_t* added, int B, int32_t* table, long long table_stride,
                          int max_pages, const int32_t* free_pages, int n_free, const int32_t* taken, int page_size,
                          int num_pages, int T, int32_t* lens, int32_t* starts, int32_t* slots, int32_t* positions,
                          int32_t* taken_out, void* ws, size_t ws_bytes, void* stream) {
  mova_status st = check_batch(B, max_pages, 1);
  if (st != MOVA_OK) return st;
  if (page_size <= 0 || num_pages <= 0 || T < 0 || n_free < 0) return MOVA_ERR_INVALID_ARG;
  const int shift = shift_of(page_size);
  if (shift < 0 || static_cast<long long>(num_pages) * page_size >= (1LL << 31)) return MOVA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page_size > (1LL << 30)) return MOVA_ERR_UNSUPPORTED;
  if (table_stride == 0) table_stride = max_pages;
  if (table_stride < max_pages || table_stride > (1LL << 40)) return MOVA_ERR_INVALID_ARG;
  if (!starts || !taken || !taken_out || (n_free > 0 && !free_pages)) return MOVA_ERR_INVALID_ARG;
  if (B > 0 && (!cached || !added || !table || !lens)) return MOVA_ERR_INVALID_ARG;
  if (T > 0 && (!slots || !positions)) return MOVA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(cached), static_cast<const void*>(added),
                        static_cast<const void*>(table), static_cast<const void*>(lens),
                        static_cast<const void*>(starts), static_cast<const void*>(taken),
                        static_cast<const void*>(taken_out), static_cast<const void*>(free_pages),
                        static_cast<const void*>(slots), static_cast<const void*>(positions)})
    if (!aligned(p, 4)) return MOVA_ERR_INVALID_ARG;
  st = check_ws(ws, ws_bytes, kStatusBytes);
  if (st != MOVA_OK) return st;
  const MapArgs a{cached, added, B,     table, table_stride, max_pages, free_pages, n_free,    taken,
                  shift,  num_pages, T, lens,  starts,       slots,     positions,  taken_out, static_cast<StatusBlock*>(ws)};
  return from_cuda(launch_page_map(a, static_cast<cudaStream_t>(stream)));
}

mova_status mova_page_write(const void* k, const void* v, mova_dtype dt, long long k_stride, long long v_stride,
                            const int32_t* slots, int T, const mova_pages* pages, void* ws, size_t ws_bytes,
                            void* stream) {
  mova_pages p;
  mova_status st = read_pages(pages, &p);
  if (st != MOVA_OK) return st;
  if (!io_fits(dt, p.dtype)) return MOVA_ERR_UNSUPPORTED;
  if (T < 0) return MOVA_ERR_INVALID_ARG;
  if (T == 0) return empty_call(ws, ws_bytes, stream);
  const long long width = static_cast<long long>(p.kv_heads) * kHeadDim;
  if ((st = read_stride(&k_stride, width, dt)) != MOVA_OK || (st = read_stride(&v_stride, width, dt)) != MOVA_OK)
    return st;
  if (!k || !v || !slots || !p.k || !p.v || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4))
    return MOVA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, kStatusBytes)) != MOVA_OK) return st;
  return from_cuda(launch_page_write(k, v, dt, k_stride, v_stride, slots, T, p, static_cast<StatusBlock*>(ws),
                                     static_cast<cudaStream_t>(stream)));
}

mova_status mova_page_bounds(const mova_pages* pages, const int32_t* table, long long table_stride, int max_pages,
                             const int32_t* cached, const int32_t* lens, int B, void* k_lo, void* k_hi, void* ws,
                             size_t ws_bytes, void* stream) {
  mova_pages p;
  PageArgs a;
  mova_status st = read_pages(pages, &p);
  if (st == MOVA_OK) st = read_table(p, table, table_stride, max_pages, lens, B, &a);
  if (st != MOVA_OK) return st;
  if (B == 0) return empty_call(ws, ws_bytes, stream);
  if (!p.k || !cached || !k_lo || !k_hi || !aligned(cached, 4) || !aligned(k_lo, 16) || !aligned(k_hi, 16))
    return MOVA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, kStatusBytes)) != MOVA_OK) return st;
  return from_cuda(launch_page_bounds(a, p.dtype, cached, k_lo, k_hi, static_cast<StatusBlock*>(ws),
                                      static_cast<cudaStream_t>(stream)));
}

mova_status mova_page_attend(const void* q, mova_dtype q_dt, long long q_stride, int H, const mova_pages* pages,
                             const int32_t* table, long long table_stride, int max_pages, const int32_t* lens, int B,
                             float scale, const int32_t* picked, int top, void* o, float* lse, void* ws,
                             size_t ws_bytes, void* stream) {
  mova_pages p;
  PageArgs a;
  mova_status st = read_pages(pages, &p);
  if (st == MOVA_OK) st = check_heads(p.kv_heads, H);
  if (st == MOVA_OK) st = read_table(p, table, table_stride, max_pages, lens, B, &a);
  if (st != MOVA_OK) return st;
  if (!io_fits(q_dt, p.dtype)) return MOVA_ERR_UNSUPPORTED;
  if (picked == nullptr ? top != 0 : top < 1) return MOVA_ERR_INVALID_ARG;
  if (B == 0) return empty_call(ws, ws_bytes, stream);
  if ((st = read_stride(&q_stride, static_cast<long long>(H) * kHeadDim, q_dt)) != MOVA_OK) return st;
  if (!q || !o || !p.k || !p.v || !aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(picked, 4))
    return MOVA_ERR_INVALID_ARG;
  const PageWs w = layout(ws, B, max_pages, p.kv_heads, H);
  if ((st = check_ws(ws, ws_bytes, w.bytes)) != MOVA_OK) return st;
  return from_cuda(launch_page_attend(q, q_stride, H / p.kv_heads, a, p.dtype, scale, picked, top, o, lse, w,
                                      static_cast<cudaStream_t>(stream)));
}

mova_status mova_page_select(const void* q, mova_dtype q_dt, long long q_stride, int H, const mova_pages* pages,
                             const void* k_lo, const void* k_hi, const int32_t* table, long long table_stride,
                             int max_pages, const int32_t* lens, int B, int top, int32_t* picked, void* ws,
                             size_t ws_bytes, void* stream) {
  mova_pages p;
  PageArgs a;
  mova_status st = read_pages(pages, &p);
  if (st == MOVA_OK) st = check_heads(p.kv_heads, H);
  if (st == MOVA_OK) st = read_table(p, table, table_stride, max_pages, lens, B, &a);
  if (st != MOVA_OK) return st;
  if (!io_fits(q_dt, p.dtype)) return MOVA_ERR_UNSUPPORTED;
  if (top < 1) return MOVA_ERR_INVALID_ARG;
  if (B == 0) return empty_call(ws, ws_bytes, stream);
  if ((st = read_stride(&q_stride, static_cast<long long>(H) * kHeadDim, q_dt)) != MOVA_OK) return st;
  if (!q || !k_lo || !k_hi || !picked || !aligned(q, 16) || !aligned(k_lo, 16) || !aligned(k_hi, 16) ||
      !aligned(picked, 4))
    return MOVA_ERR_INVALID_ARG;
  const PageWs w = layout(ws, B, max_pages, p.kv_heads, H);
  if ((st = check_ws(ws, ws_bytes, w.bytes)) != MOVA_OK) return st;
  return from_cuda(launch_page_select(q, q_stride, H / p.kv_heads, a, p.dtype, k_lo, k_hi, top, picked, w,
                                      static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

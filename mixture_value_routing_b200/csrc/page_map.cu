// Page tables and slot maps of one step, from request lengths.
//
//   need[b]   = ceil((cached + added) / page) - ceil(cached / page)
//   pages     taken from the free list in request order (exclusive scan of need)
//   starts    exclusive scan of added
//   slot(i)   = page(b, pos / page_size) * page_size + pos % page_size,
//               pos = cached[b] + i - starts[b], b the request of token i
//
// 8 bytes per request in, 8 bytes per new token out: latency bounds it, so it
// is one launch, of one cluster of up to 8 CTAs.  Every CTA scans all
// requests (at most 4096, in shared memory) and takes its share of the new
// pages and tokens, finding a token's request by binary search.  A token in a
// new page reads the free list, not the table, so no CTA waits for another's
// table entries.  The cluster meets before the end, so that taken_out (which may be
// `taken`) and the status are written after every CTA has read and checked.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace mova {

namespace {

constexpr int kMapMaxCluster = 8;
// Tokens per CTA at which another CTA joins: four per thread.
constexpr int kMapTokensPerCta = 4096;

// kCluster: a cluster of several CTAs; otherwise one CTA, launched without one.
template <int kThreads, bool kCluster>
__global__ void __launch_bounds__(kThreads) page_map_kernel(const MapArgs a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) char smem[];
  __shared__ int sm_bad, sm_used;
  long long* starts = reinterpret_cast<long long*>(smem);
  long long* pre = starts + a.B + 1;
  int* cached = reinterpret_cast<int*>(pre + a.B + 1);
  int* added = cached + a.B;
  const int tid = threadIdx.x;
  const int rank = kCluster ? static_cast<int>(blockIdx.x) : 0, CTAs = kCluster ? static_cast<int>(gridDim.x) : 1;
  const int page_size = 1 << a.shift;
  if (tid == 0) sm_bad = kNoBad, sm_used = 0;
  // Rank 0's sm_bad is set before another CTA reduces into it.
  if constexpr (kCluster) cg::this_cluster().sync();
  pdl_wait();
  pdl_trigger();
  const int taken = a.taken[0];
  const bool taken_ok = taken >= 0 && taken <= a.n_free;
  const long long avail = taken_ok ? a.n_free - taken : 0;
  const long long cap = static_cast<long long>(a.max_pages) << a.shift;
  auto pages = [&](long long tokens) { return (tokens + page_size - 1) >> a.shift; };
  auto fits = [&](int c, int n) { return c >= 0 && n >= 0 && static_cast<long long>(c) + n <= cap; };

  request_scan2<kThreads>(a.B, starts, pre, [&](int b, long long& tokens, long long& need) {
    const int c = a.cached[b], n = a.added[b];
    cached[b] = c;
    added[b] = n;
    tokens = n < 0 ? 0 : n;
    need = fits(c, n) ? pages(static_cast<long long>(c) + n) - pages(c) : 0LL;
  });
  // Whether request b gets its pages; its share of the free list is [pre[b], pre[b + 1]).
  auto granted = [&](int b) {
    return fits(cached[b], added[b]) && (pre[b + 1] == pre[b] || pre[b + 1] <= avail);
  };
  for (int b = tid; b < a.B; b += kThreads) {
    const bool ok = granted(b);
    if (!ok || starts[b + 1] > a.T) atomicMin(&sm_bad, b);
    // The last request within the free pages: what is handed out.
    if (pre[b + 1] <= avail && (b + 1 == a.B || pre[b + 2] > avail)) sm_used = static_cast<int>(pre[b + 1]);
    if (rank == 0) a.lens[b] = ok ? cached[b] + added[b] : max(cached[b], 0);
  }
  if (rank == 0)
    for (int b = tid; b <= a.B; b += kThreads)
      a.starts[b] = static_cast<int>(starts[b] > 0x7fffffff ? 0x7fffffff : starts[b]);
  __syncthreads();
  const int used = sm_used;
  const int all = CTAs * kThreads, me = rank * kThreads + tid;
  for (int x = me; x < used; x += all) {
    const int b = request_of(pre, a.B, static_cast<long long>(x));
    const long long j = pages(cached[b]) + x - pre[b];
    a.table[b * a.table_stride + j] = a.free_pages[taken + x];
  }
  const long long total = starts[a.B];
  for (long long i = me; i < a.T; i += all) {
    int slot = -1, pos = -1;
    if (i < total) {
      const int b = request_of(starts, a.B, i);
      const int c = cached[b];
      if (granted(b)) {
        pos = static_cast<int>(c + i - starts[b]);
        const int j = pos >> a.shift, have = static_cast<int>(pages(c));
        const int page = j < have ? a.table[b * a.table_stride + j] : a.free_pages[taken + pre[b] + j - have];
        if (page >= 0 && page < a.num_pages)
          slot = (page << a.shift) + (pos & (page_size - 1));
        else
          atomicMin(&sm_bad, b);
      }
    }
    a.slots[i] = slot;
    a.positions[i] = pos;
  }
  __syncthreads();
  if constexpr (kCluster) {
    cg::cluster_group cluster = cg::this_cluster();
    if (rank != 0 && tid == 0) atomicMin(cluster.map_shared_rank(&sm_bad, 0), sm_bad);
    cluster.sync();
  }
  if (rank == 0 && tid == 0) {
    a.taken_out[0] = taken + used;
    a.sb->code = sm_bad == kNoBad ? MOVA_OK : MOVA_ERR_DEVICE_CHECK;
    a.sb->detail = sm_bad == kNoBad ? 0 : sm_bad;
  }
}

template <int kThreads, bool kCluster>
cudaError_t launch_map_t(const MapArgs& a, int ctas, cudaStream_t stream) {
  static bool done[64] = {false};
  auto kern = page_map_kernel<kThreads, kCluster>;
  constexpr size_t kMost = (kMaxRequests + 1) * 16 + kMaxRequests * 8;
  cudaError_t err = prepare_kernel(kern, kMost, done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.B + 1) * 16 + static_cast<size_t>(a.B) * 8;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = kCluster ? 2 : 1;
  note_launch();
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_page_map(const MapArgs& a, cudaStream_t stream) {
  int ctas = 1;
  while (ctas < kMapMaxCluster && a.T > ctas * kMapTokensPerCta) ctas *= 2;
  if (ctas > 1) return launch_map_t<1024, true>(a, ctas, stream);
  return a.B <= 256 && a.T <= 1024 ? launch_map_t<256, false>(a, 1, stream) : launch_map_t<1024, false>(a, 1, stream);
}

}  // namespace mova

// Page tables and slot maps of one step, from request lengths.
//
//   need[b]   = ceil((cached + added) / page) - ceil(cached / page)
//   pages     taken from the free list in request order (exclusive scan of need)
//   starts    exclusive scan of added
//   slot(i)   = page(b, pos / page_size) * page_size + pos % page_size,
//               pos = cached[b] + i - starts[b], b the request of token i
//
// 8 bytes per request in, 8 bytes per new token out: latency bounds it, so it
// is one launch, of one cluster of up to 8 CTAs.  Measured: 64 requests of a token
// each 3.2 us; 256 requests and 46590 new tokens 11.2, as a thread searches the
// requests of five or six tokens one after another; 4096 requests and 15210 tokens
// 22.7, as the scan and the checks go through the requests in four steps and a search
// takes twelve.  Every CTA scans all
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
  // Of each request: {tokens before it in the step, pages of the step before
  // it} (both clipped to kClip), and {cached tokens, pages it has, first entry
  // of the free list that is its own (-1: refused)}.
  int2* before = reinterpret_cast<int2*>(smem);                            // (B + 1)
  int* cached = reinterpret_cast<int*>(before + a.B + 1);
  int* have = cached + a.B;
  int* own = have + a.B;
  const int tid = threadIdx.x;
  const int rank = kCluster ? static_cast<int>(blockIdx.x) : 0, CTAs = kCluster ? static_cast<int>(gridDim.x) : 1;
  const int page_size = 1 << a.shift;
  if (tid == 0) sm_bad = kNoBad, sm_used = 0;
  // Rank 0's sm_bad is set before another CTA reduces into it.
  if constexpr (kCluster) cg::this_cluster().sync();
  pdl_wait();
  pdl_trigger();
  const int taken = a.taken[0];
  const int avail = taken >= 0 && taken <= a.n_free ? min(a.n_free - taken, kClip - 1) : 0;
  const long long cap = static_cast<long long>(a.max_pages) << a.shift;

  request_scan2<kThreads>(a.B, before, [&](int b, long long& tokens, long long& need) {
    const int c = a.cached[b], n = a.added[b];
    const bool fits = c >= 0 && n >= 0 && static_cast<long long>(c) + n <= cap;
    cached[b] = c;
    have[b] = fits ? (c + page_size - 1) >> a.shift : -1;
    tokens = n < 0 ? 0 : n;
    need = fits ? ((c + n + page_size - 1) >> a.shift) - have[b] : 0;
  });
  for (int b = tid; b < a.B; b += kThreads) {
    const int end = before[b + 1].y, c = cached[b], n = a.added[b];
    const bool ok = have[b] >= 0 && (((c + n + page_size - 1) >> a.shift) == have[b] || end <= avail);
    own[b] = ok ? max(taken, 0) + before[b].y : -1;
    if (!ok || before[b + 1].x > a.T) atomicMin(&sm_bad, b);
    // The last request within the free pages: what is handed out.
    if (end <= avail && (b + 1 == a.B || before[b + 2].y > avail)) sm_used = end;
    if (rank == 0) a.lens[b] = ok ? c + n : max(c, 0);
  }
  if (rank == 0)
    for (int b = tid; b <= a.B; b += kThreads) a.starts[b] = before[b].x;
  __syncthreads();
  const int used = sm_used;
  const int all = CTAs * kThreads, me = rank * kThreads + tid;
  // The last request with at most x before it, by the chosen count.
  auto find = [&](int x, bool by_page) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((by_page ? before[mid].y : before[mid].x) <= x) lo = mid; else hi = mid;
    }
    return lo;
  };
  for (int x = me; x < used; x += all) {
    const int b = find(x, true);
    a.table[b * a.table_stride + have[b] + x - before[b].y] = a.free_pages[taken + x];
  }
  const int total = before[a.B].x;
  for (long long i64 = me; i64 < a.T; i64 += all) {
    const int i = static_cast<int>(i64);
    int slot = -1, pos = -1;
    if (i < total) {
      const int b = find(i, false);
      const int first = own[b];
      if (first >= 0) {
        pos = cached[b] + i - before[b].x;
        const int j = pos >> a.shift;
        const int page = j < have[b] ? a.table[b * a.table_stride + j] : a.free_pages[first + j - have[b]];
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
  constexpr size_t kMost = (kMaxRequests + 1) * 8 + kMaxRequests * 12;
  cudaError_t err = prepare_kernel(kern, kMost, done);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(a.B + 1) * 8 + static_cast<size_t>(a.B) * 12;
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

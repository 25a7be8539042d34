// K11: upkeep of a paged cache: resize (allocate, give back, copy on write), fork and compact.
//
// State: page_table [nseq, max_pages] (entry -1: no page) and refs [num_pages], the number of
// table entries that name each page; a page is free when its count is 0.  Free pages are always
// taken lowest first and in the order (sequence, slot), so results do not depend on timing.
//
// resize and compact need ranks among the free (or live) pages: one cluster of CTAs counts its
// slices of refs, adds the lower slices' counts over distributed shared memory and writes the
// list of pages in order (latency-bound: 4 B a page, read twice).  A second, wide kernel then
// rewrites the table and copies page contents (HBM-bound: a copied byte is read and written once).
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "misa.h"
#include "paged.cuh"

namespace misa {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanCtas = 8;       // the largest portable cluster
constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kCopyBytes = kApplyThreads * 16 * kCopyUnroll;   // piece of a page that a block copies

// Scratch of resize and compact (256-aligned regions).
struct PlanScratch {
  int* head;      // [8]: copies, n_live, whether the call goes ahead
  int* list;      // [num_pages]: resize: the lowest free pages; compact: the holes below n_live
  int* list2;     // [num_pages]: resize: holders of a page that grow; compact: live pages from
                  // n_live on, at their rank among the live ones
  int* map;       // [num_pages]: resize: the last holder that grows; compact: where a page goes
  int* first;     // [nseq]: rank of the first page that a sequence takes
  int* cow;       // [nseq]: page to copy, -1: none
  int* cow_seq;   // [nseq]: the sequences that copy, in order
};

size_t plan_scratch(int nseq, int num_pages, void* base, PlanScratch* s) {
  size_t at = 0;
  char* b = static_cast<char*>(base);
  auto take = [&](size_t n) {
    int* p = reinterpret_cast<int*>(b + at);
    at += align256(n * sizeof(int));
    return p;
  };
  PlanScratch x;
  x.head = take(8);
  x.list = take(num_pages);
  x.list2 = take(num_pages);
  x.map = take(num_pages);
  x.first = take(nseq);
  x.cow = take(nseq);
  x.cow_seq = take(nseq);
  if (s) *s = x;
  return at;
}

// Exclusive prefix sum over the block's threads (kPlanThreads); *total: the sum.  Barriers at
// both ends, so s_scan may be used again at once.
__device__ __forceinline__ int block_scan(int x, int* s_scan, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int y = s_scan[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    s_scan[lane] = y;
  }
  __syncthreads();
  const int before = (warp ? s_scan[warp - 1] : 0) + inc - x;
  *total = s_scan[31];
  __syncthreads();
  return before;
}

// What a sequence's lengths ask for.  `ok` false: a length out of range, the row stays as it is.
struct Span {
  int oldp, newp, tail;   // pages before and after; slot of a partly filled last page of a
                          // sequence that grows (-1: none)
  bool ok;
  __device__ __forceinline__ Span(int o, int x, int page_size, int max_pages) {
    const int cap = max_pages * page_size;
    ok = o >= 0 && x >= 0 && o <= cap && x <= cap;
    oldp = ok ? (o + page_size - 1) / page_size : 0;
    newp = ok ? (x + page_size - 1) / page_size : 0;
    tail = ok && x > o && o % page_size ? o / page_size : -1;
  }
};

// Number of CTA-slice pages that are free (FREE) or live, summed over the block.
template <bool FREE>
__device__ __forceinline__ int count_slice(const int32_t* __restrict__ refs, int lo, int hi,
                                           int* s_scan) {
  int n = 0;
  for (int p = lo + threadIdx.x; p < hi; p += kPlanThreads) n += (refs[p] > 0) != FREE;
  int total;
  block_scan(n, s_scan, &total);
  return total;
}

__global__ void __launch_bounds__(kPlanThreads)
    resize_plan_kernel(const int32_t* __restrict__ table, const int32_t* refs,
                       const int32_t* __restrict__ old_len, const int32_t* __restrict__ new_len,
                       int nseq, int max_pages, int num_pages, int page_size, int32_t* out_refs,
                       PlanScratch s, int* status) {
  __shared__ int s_scan[32];
  __shared__ int s_free, s_need;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int slice = (num_pages + kPlanCtas - 1) / kPlanCtas;
  const int lo = min(num_pages, rank * slice), hi = min(num_pages, lo + slice);
  const int n_free = count_slice<true>(refs, lo, hi, s_scan);
  if (tid == 0) s_free = n_free;

  if (rank == 0) {
    // pages whose last token's sequence grows: how many such sequences hold it, and the last
    auto tail_page = [&](int n, const Span& sp) {
      if (sp.tail < 0) return -1;
      const int p = table[(int64_t)n * max_pages + sp.tail];
      return (unsigned)p < (unsigned)num_pages ? p : -1;
    };
    for (int n = tid; n < nseq; n += kPlanThreads) {
      const int p = tail_page(n, Span(old_len[n], new_len[n], page_size, max_pages));
      if (p >= 0) {
        s.list2[p] = 0;
        s.map[p] = -1;
      }
    }
    __syncthreads();
    for (int n = tid; n < nseq; n += kPlanThreads) {
      const int p = tail_page(n, Span(old_len[n], new_len[n], page_size, max_pages));
      if (p >= 0) {
        atomicAdd(s.list2 + p, 1);
        atomicMax(s.map + p, n);
      }
    }
    __syncthreads();
    int need = 0, copies = 0;
    for (int n0 = 0; n0 < nseq; n0 += kPlanThreads) {
      const int n = n0 + tid;
      int want = 0, page = -1;
      if (n < nseq) {
        const Span sp(old_len[n], new_len[n], page_size, max_pages);
        const int p = tail_page(n, sp);
        if (!sp.ok || (sp.tail >= 0 && p < 0)) set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
        if (p >= 0) {
          const int holders = refs[p];
          if (holders > 1 && !(__ldcg(s.list2 + p) >= holders && __ldcg(s.map + p) == n)) page = p;
        }
        want = max(0, sp.newp - sp.oldp) + (page >= 0);
      }
      int sum, ncow;
      const int before = block_scan(want, s_scan, &sum);
      const int at = block_scan(page >= 0, s_scan, &ncow);
      if (n < nseq) {
        s.first[n] = need + before;
        s.cow[n] = page;
        if (page >= 0) s.cow_seq[copies + at] = n;
      }
      need += sum;
      copies += ncow;
    }
    if (tid == 0) {
      s_need = need;
      s.head[0] = copies;
    }
  }
  cluster.sync();
  const int need = *cluster.map_shared_rank(&s_need, 0);
  int before = 0, total = 0;
  for (int r = 0; r < kPlanCtas; ++r) {
    const int f = *cluster.map_shared_rank(&s_free, r);
    if (r < rank) before += f;
    total += f;
  }
  const bool go = need <= total;
  if (rank == 0 && tid == 0) {
    s.head[2] = go;
    if (!go) set_status(status, MISA_ERR_OUT_OF_PAGES);
  }
  const bool copy_refs = out_refs != refs;
  for (int p0 = lo; p0 < hi && (copy_refs || (go && before < need)); p0 += kPlanThreads) {
    const int p = p0 + tid;
    const int r = p < hi ? refs[p] : 1;
    if (copy_refs && p < hi) out_refs[p] = r;
    int n;
    const int at = before + block_scan(r <= 0, s_scan, &n);
    if (go && r <= 0 && at < need) s.list[at] = p;
    before += n;
  }
  cluster.sync();   // no CTA leaves while another reads its shared memory
}

// One piece of a page, by the whole block.  src and dst: pages.
__device__ __forceinline__ void copy_piece(const PagePools& pools, int pool, int src, int dst,
                                           int piece) {
  const uint32_t bytes = pools.page_bytes[pool];
  const uint32_t at = (uint32_t)piece * kCopyBytes;
  if (at >= bytes) return;
  const uint4* from =
      reinterpret_cast<const uint4*>(pools.base[pool] + (size_t)src * bytes + at) + threadIdx.x;
  uint4* to = reinterpret_cast<uint4*>(pools.base[pool] + (size_t)dst * bytes + at) + threadIdx.x;
  const int n = (int)(min(bytes - at, (uint32_t)kCopyBytes) / 16) - (int)threadIdx.x;
  uint4 x[kCopyUnroll];
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (u * kApplyThreads < n) x[u] = __ldcs(from + u * kApplyThreads);
#pragma unroll
  for (int u = 0; u < kCopyUnroll; ++u)
    if (u * kApplyThreads < n) to[u * kApplyThreads] = x[u];
}

__global__ void __launch_bounds__(kApplyThreads)
    resize_apply_kernel(const int32_t* table, const int32_t* __restrict__ old_len,
                        const int32_t* __restrict__ new_len, int nseq, int max_pages,
                        int num_pages, int page_size, const __grid_constant__ PagePools pools,
                        int pieces, int32_t* out_table, int32_t* out_refs, PlanScratch s,
                        int* status) {
  pdl_prologue();
  const bool go = s.head[2] != 0;
  const int64_t entries = (int64_t)nseq * max_pages;
  for (int64_t i = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x; i < entries;
       i += (int64_t)gridDim.x * kApplyThreads) {
    const int n = (int)(i / max_pages), c = (int)(i - (int64_t)n * max_pages);
    const int was = table[i];
    const Span sp(old_len[n], new_len[n], page_size, max_pages);
    int now = was;
    if (go && sp.ok) {
      const int page = s.cow[n];
      if (c >= max(sp.oldp, sp.newp)) {
        now = -1;
      } else if (c >= sp.oldp) {
        now = s.list[s.first[n] + (page >= 0) + (c - sp.oldp)];
        out_refs[now] = 1;
      } else if (c >= sp.newp || (page >= 0 && c == sp.tail)) {
        if ((unsigned)was < (unsigned)num_pages)
          atomicSub(out_refs + was, 1);
        else
          set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
        now = -1;
        if (c < sp.newp) {
          now = s.list[s.first[n]];
          out_refs[now] = 1;
        }
      }
    }
    if (now != was || out_table != table) out_table[i] = now;
  }
  if (!go || pools.n == 0) return;
  const int64_t per = (int64_t)pools.n * pieces, work = s.head[0] * per;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int n = s.cow_seq[i / per], x = (int)(i % per);
    copy_piece(pools, x / pieces, s.cow[n], s.list[s.first[n]], x % pieces);
  }
}

__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const int32_t* refs, int num_pages, int32_t* out_refs, int32_t* n_live_out,
                        PlanScratch s) {
  __shared__ int s_scan[32];
  __shared__ int s_live, s_holes;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int slice = (num_pages + kPlanCtas - 1) / kPlanCtas;
  const int lo = min(num_pages, rank * slice), hi = min(num_pages, lo + slice);
  const int live = count_slice<false>(refs, lo, hi, s_scan);
  if (tid == 0) {
    s_live = live;
    s_holes = 0;
  }
  cluster.sync();
  int before = 0, n_live = 0;
  for (int r = 0; r < kPlanCtas; ++r) {
    const int f = *cluster.map_shared_rank(&s_live, r);
    if (r < rank) before += f;
    n_live += f;
  }
  // hole i below n_live goes to list[i]; the live page of rank i from n_live on to list2[i]
  int holes = 0;
  for (int p0 = lo; p0 < hi; p0 += kPlanThreads) {
    const int p = p0 + tid;
    const int r = p < hi ? refs[p] : 0;
    int n;
    const int at = before + block_scan(r > 0, s_scan, &n);
    before += n;
    if (p < hi) {
      if (out_refs != refs) out_refs[p] = r;
      if (p < n_live && r <= 0) {
        s.list[p - at] = p;
        ++holes;
      }
      if (p >= n_live) {
        if (r > 0) s.list2[at] = p;
        s.map[p] = -1;
      }
    }
  }
  int sum;
  block_scan(holes, s_scan, &sum);
  if (tid == 0) s_holes = sum;
  cluster.sync();
  int moves = 0;
  for (int r = 0; r < kPlanCtas; ++r) moves += *cluster.map_shared_rank(&s_holes, r);
  for (int i = rank * kPlanThreads + tid; i < moves; i += kPlanCtas * kPlanThreads) {
    const int src = __ldcg(s.list2 + n_live - moves + i), dst = __ldcg(s.list + i);
    s.map[src] = dst;
    out_refs[dst] = refs[src];
    out_refs[src] = 0;
  }
  if (rank == 0 && tid == 0) {
    s.head[0] = moves;
    s.head[1] = n_live;
    if (n_live_out) *n_live_out = n_live;
  }
  cluster.sync();
}

__global__ void __launch_bounds__(kApplyThreads)
    compact_apply_kernel(const int32_t* table, int64_t entries, int num_pages,
                         const __grid_constant__ PagePools pools, int pieces, int32_t* out_table,
                         PlanScratch s, int* status) {
  pdl_prologue();
  const int moves = s.head[0], n_live = s.head[1];
  for (int64_t i = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x; i < entries;
       i += (int64_t)gridDim.x * kApplyThreads) {
    const int was = table[i];
    int now = was;
    if (was < -1 || was >= num_pages) {
      set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
    } else if (was >= n_live) {
      now = s.map[was];
      if (now < 0) {   // the table names a page that refs says is free
        set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
        now = was;
      }
    }
    if (now != was || out_table != table) out_table[i] = now;
  }
  if (pools.n == 0) return;
  const int64_t per = (int64_t)pools.n * pieces, work = moves * per;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int m = (int)(i / per), x = (int)(i % per);
    copy_piece(pools, x / pieces, s.list2[n_live - moves + m], s.list[m], x % pieces);
  }
}

// Row n takes the entries of row parent[n] of `table`; the counts of the pages it lets go of and
// takes follow (entries that stay the same touch no count).  out_refs holds the counts before.
__global__ void __launch_bounds__(kApplyThreads)
    fork_kernel(const int32_t* __restrict__ table, const int32_t* __restrict__ parent, int nseq,
                int max_pages, int num_pages, int32_t* __restrict__ out_table, int32_t* out_refs,
                int* status) {
  pdl_prologue();
  const int64_t entries = (int64_t)nseq * max_pages;
  for (int64_t i = (int64_t)blockIdx.x * kApplyThreads + threadIdx.x; i < entries;
       i += (int64_t)gridDim.x * kApplyThreads) {
    const int n = (int)(i / max_pages), c = (int)(i - (int64_t)n * max_pages);
    int from = parent[n];
    if (from < -1 || from >= nseq) {
      set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
      from = n;
    }
    const int was = table[i];
    const int now = from < 0 ? -1 : table[(int64_t)from * max_pages + c];
    if (was < -1 || was >= num_pages) set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
    if (now != was) {
      if ((unsigned)now < (unsigned)num_pages) atomicAdd(out_refs + now, 1);
      if ((unsigned)was < (unsigned)num_pages) atomicSub(out_refs + was, 1);
    }
    out_table[i] = now;
  }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_plan(void (*kernel)(KArgs...), cudaStream_t st, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPlanCtas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPlanCtas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

int pieces_of(const PagePools& pools) {
  int most = 1;
  for (int i = 0; i < pools.n; ++i) {
    const int n = (int)((pools.page_bytes[i] + (int64_t)kCopyBytes - 1) / kCopyBytes);
    if (n > most) most = n;
  }
  return most;
}

// Blocks of the wide kernels: the table's entries and at most `copies` page copies, eight blocks
// per SM (148) at most.
int apply_grid(int64_t entries, int64_t copies, const PagePools& pools, int pieces) {
  int64_t n = (entries + kApplyThreads - 1) / kApplyThreads;
  const int64_t c = copies * pools.n * pieces;
  if (c > n) n = c;
  return (int)(n < 148 * 8 ? n : 148 * 8);
}

}  // namespace

size_t pages_ws_bytes(int nseq, int num_pages) { return plan_scratch(nseq, num_pages, nullptr, nullptr); }

cudaError_t launch_pages_resize(const int32_t* table, const int32_t* refs, const int32_t* old_len,
                                const int32_t* new_len, int nseq, int max_pages, int num_pages,
                                int page_size, const PagePools& pools, int32_t* out_table,
                                int32_t* out_refs, void* scratch, int* status, cudaStream_t st) {
  PlanScratch s;
  plan_scratch(nseq, num_pages, scratch, &s);
  cudaError_t e = launch_plan(resize_plan_kernel, st, table, refs, old_len, new_len, nseq,
                              max_pages, num_pages, page_size, out_refs, s, status);
  if (e != cudaSuccess) return e;
  const int pieces = pieces_of(pools);
  const int grid = apply_grid((int64_t)nseq * max_pages, nseq, pools, pieces);
  return launch_pdl(resize_apply_kernel, dim3(grid), dim3(kApplyThreads), 0, st, table, old_len,
                    new_len, nseq, max_pages, num_pages, page_size, pools, pieces, out_table,
                    out_refs, s, status);
}

cudaError_t launch_pages_fork(const int32_t* table, const int32_t* refs, const int32_t* parent,
                              int nseq, int max_pages, int num_pages, int32_t* out_table,
                              int32_t* out_refs, void* scratch, int* status, cudaStream_t st) {
  const size_t table_bytes = (size_t)nseq * max_pages * sizeof(int32_t);
  if (out_refs != refs) {
    const cudaError_t e = cudaMemcpyAsync(out_refs, refs, (size_t)num_pages * sizeof(int32_t),
                                          cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
  }
  if (out_table == table) {   // rows read one another: in place they read a copy
    const cudaError_t e =
        cudaMemcpyAsync(scratch, table, table_bytes, cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
    table = static_cast<const int32_t*>(scratch);
  }
  const int64_t entries = (int64_t)nseq * max_pages;
  const int64_t blocks = (entries + kApplyThreads - 1) / kApplyThreads;
  return launch_pdl(fork_kernel, dim3((unsigned)(blocks < 148 * 8 ? blocks : 148 * 8)),
                    dim3(kApplyThreads), 0, st, table, parent, nseq, max_pages, num_pages,
                    out_table, out_refs, status);
}

cudaError_t launch_pages_compact(const int32_t* table, const int32_t* refs, int nseq,
                                 int max_pages, int num_pages, const PagePools& pools,
                                 int32_t* out_table, int32_t* out_refs, int32_t* n_live,
                                 void* scratch, int* status, cudaStream_t st) {
  PlanScratch s;
  plan_scratch(0, num_pages, scratch, &s);
  cudaError_t e = launch_plan(compact_plan_kernel, st, refs, num_pages, out_refs, n_live, s);
  if (e != cudaSuccess) return e;
  const int pieces = pieces_of(pools);
  const int64_t entries = (int64_t)nseq * max_pages;
  const int grid = apply_grid(entries, num_pages / 2, pools, pieces);
  return launch_pdl(compact_apply_kernel, dim3(grid), dim3(kApplyThreads), 0, st, table, entries,
                    num_pages, pools, pieces, out_table, s, status);
}

}  // namespace misa

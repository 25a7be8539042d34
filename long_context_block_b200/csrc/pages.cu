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

#include <climits>
#include <utility>

#include "internal.h"
#include "misa.h"
#include "paged.cuh"

namespace misa {
namespace {

namespace cg = cooperative_groups;
using paged::Divide;

constexpr int kPlanCtas = 8;       // the largest portable cluster
constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int kForkUnroll = 4;
// Tables that one cluster rewrites: larger ones want every SM.
constexpr int kSmallEntries = kPlanCtas * kPlanThreads * kForkUnroll;
constexpr int kSmallPages = 1 << 17;
constexpr int kCopyBytes = kApplyThreads * 16 * kCopyUnroll;   // piece of a page that a block copies

// Scratch of resize and compact (256-aligned regions).
struct PlanScratch {
  int* head;      // [8]: page copies; compact: n_live; resize: whether the call goes ahead
  int* list;      // [num_pages]: resize: the lowest free pages; compact: the holes below n_live
  int* list2;     // [num_pages]: resize: holders of a page that grow; compact: live pages from
                  // n_live on, at their rank among the live ones
  int* map;       // [num_pages]: resize: the last holder that grows; compact: the rank of a live
                  // page from n_live on, -1 of a free one
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

// A slice's pages in tiles of kTile: bit p of the tile's words says whether the page is live
// (refs > 0).  Pages behind the slice count as live (FREE) or free, so that no list takes them.
constexpr int kTile = kPlanThreads * 32;

template <bool FREE>
__device__ __forceinline__ void load_bits(const int32_t* refs, int lo, int hi, int32_t* out_refs,
                                          uint32_t* s_bits) {
  const int lane = threadIdx.x & 31;
  const int words = (min(hi - lo, kTile) + 31) / 32;
#pragma unroll 4
  for (int w = threadIdx.x >> 5; w < words; w += kPlanThreads / 32) {
    const int p = lo + w * 32 + lane;
    const int r = p < hi ? refs[p] : FREE;
    if (out_refs != refs && p < hi) out_refs[p] = r;
    const uint32_t live = __ballot_sync(0xffffffffu, r > 0);
    if (lane == 0) s_bits[w] = live;
  }
  if ((int)threadIdx.x >= words) s_bits[threadIdx.x] = FREE ? 0xffffffffu : 0u;
  __syncthreads();
}

// Pages of the slice that are free (FREE) or live.  out_refs receives the counts where it is
// another buffer; the last tile's bits stay in s_bits.
template <bool FREE>
__device__ __forceinline__ int count_slice(const int32_t* refs, int lo, int hi, int32_t* out_refs,
                                           uint32_t* s_bits, int* s_scan) {
  int n = 0;
  for (int t = lo; t < hi; t += kTile) {
    load_bits<FREE>(refs, t, hi, out_refs, s_bits);
    n += __popc(FREE ? ~s_bits[threadIdx.x] : s_bits[threadIdx.x]);
    __syncthreads();
  }
  int total;
  block_scan(n, s_scan, &total);
  return total;
}

// Calls f(page, is it free (FREE) or live, rank) for every page of the slice, ranks counted from
// `before`, until they reach `stop`; a warp's lanes have 32 neighbouring pages.
template <bool FREE, typename F>
__device__ __forceinline__ void rank_slice(const int32_t* refs, int lo, int hi, int before,
                                           int stop, uint32_t* s_bits, int* s_at, int* s_scan,
                                           F f) {
  const int lane = threadIdx.x & 31;
  for (int t = lo; t < hi && before < stop; t += kTile) {
    if (hi - lo > kTile) load_bits<FREE>(refs, t, hi, const_cast<int32_t*>(refs), s_bits);
    int n;
    const uint32_t mine = FREE ? ~s_bits[threadIdx.x] : s_bits[threadIdx.x];
    s_at[threadIdx.x] = before + block_scan(__popc(mine), s_scan, &n);
    __syncthreads();
    const int words = (min(hi - t, kTile) + 31) / 32;
    for (int w = threadIdx.x >> 5; w < words; w += kPlanThreads / 32) {
      const uint32_t bits = FREE ? ~s_bits[w] : s_bits[w];
      const int p = t + w * 32 + lane;
      if (p < hi) f(p, (bits >> lane) & 1u, s_at[w] + __popc(bits & ((1u << lane) - 1u)));
    }
    __syncthreads();
    before += n;
  }
}

// What the calls of one resize share.
struct ResizeArgs {
  const int32_t* table;
  const int32_t* refs;
  const int32_t* old_len;
  const int32_t* new_len;
  int32_t* out_table;
  int32_t* out_refs;
  int* status;
  int nseq, max_pages, num_pages, page_size;
  Divide by_row;   // division by max_pages
  PlanScratch s;
};

// The table's entries from `first` on, `step` apart, and the counts of the pages they let go of
// and take.  kForkUnroll entries at a time, whose lookups are in flight together.
__device__ __forceinline__ void resize_entries(const ResizeArgs& a, bool go, int first, int step) {
  const int entries = a.nseq * a.max_pages;
  for (int64_t i0 = first; i0 < entries; i0 += (int64_t)step * kForkUnroll) {
    int was[kForkUnroll], o[kForkUnroll], x[kForkUnroll], cow[kForkUnroll], at[kForkUnroll],
        col[kForkUnroll];
#pragma unroll
    for (int u = 0; u < kForkUnroll; ++u) {
      const int64_t i = i0 + (int64_t)u * step;
      if (i >= entries) break;
      const int n = a.by_row((int)i);
      col[u] = (int)i - n * a.max_pages;
      was[u] = a.table[i];
      o[u] = a.old_len[n];
      x[u] = a.new_len[n];
      cow[u] = a.s.cow[n];
      at[u] = a.s.first[n];
    }
#pragma unroll
    for (int u = 0; u < kForkUnroll; ++u) {
      const int64_t i = i0 + (int64_t)u * step;
      if (i >= entries) break;
      const Span sp(o[u], x[u], a.page_size, a.max_pages);
      int now = was[u];
      if (go && sp.ok) {
        const int c = col[u];
        const bool copy = cow[u] >= 0;
        if (c >= max(sp.oldp, sp.newp)) {
          now = -1;
        } else if (c >= sp.oldp) {
          now = a.s.list[at[u] + copy + (c - sp.oldp)];
          a.out_refs[now] = 1;
        } else if (c >= sp.newp || (copy && c == sp.tail)) {
          if ((unsigned)was[u] < (unsigned)a.num_pages)
            atomicSub(a.out_refs + was[u], 1);
          else
            set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
          now = -1;
          if (c < sp.newp) {
            now = a.s.list[at[u]];
            a.out_refs[now] = 1;
          }
        }
      }
      if (now != was[u] || a.out_table != a.table) a.out_table[i] = now;
    }
  }
}

// APPLY: the cluster rewrites the table too (a small table, no pools), so that one launch does it.
template <bool APPLY>
__global__ void __launch_bounds__(kPlanThreads, 1) resize_plan_kernel(const ResizeArgs a) {
  __shared__ int s_scan[32];
  __shared__ uint32_t s_bits[kPlanThreads];
  __shared__ int s_at[kPlanThreads];
  __shared__ int s_free, s_need;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const PlanScratch& s = a.s;
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  // CTA 0 sees what the sequences want while the others count the free pages of their slices
  const int slice = (a.num_pages + kPlanCtas - 2) / (kPlanCtas - 1);
  const int lo = rank == 0 ? 0 : min(a.num_pages, (rank - 1) * slice);
  const int hi = rank == 0 ? 0 : min(a.num_pages, lo + slice);
  if (rank > 0) {
    const int n_free = count_slice<true>(a.refs, lo, hi, a.out_refs, s_bits, s_scan);
    if (tid == 0) s_free = n_free;
  } else {
    if (tid == 0) s_free = 0;
    // what sequence n wants: `want` pages, without the copy of a last page that others hold;
    // that page (-1: none)
    auto look = [&](int n, int& want, int& page) {
      want = 0;
      page = -1;
      if (n >= a.nseq) return;
      const Span sp(a.old_len[n], a.new_len[n], a.page_size, a.max_pages);
      want = max(0, sp.newp - sp.oldp);
      if (!sp.ok) set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
      if (sp.tail < 0) return;
      const int p = a.table[(int64_t)n * a.max_pages + sp.tail];
      if ((unsigned)p >= (unsigned)a.num_pages)
        set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
      else if (a.refs[p] > 1)
        page = p;
    };
    int want, page;
    bool any = false;
    for (int n = tid; n < a.nseq; n += kPlanThreads) {
      look(n, want, page);
      if (page >= 0) {
        any = true;
        s.list2[page] = 0;
        s.map[page] = -1;
      }
    }
    const bool one = a.nseq <= kPlanThreads;   // what look() said is still at hand
    if (tid >= a.nseq) {
      want = 0;
      page = -1;
    }
    if (__syncthreads_or(any)) {   // how many of its holders grow, and the last of them
      for (int n = tid; n < a.nseq; n += kPlanThreads) {
        if (!one) look(n, want, page);
        if (page >= 0) {
          atomicAdd(s.list2 + page, 1);
          atomicMax(s.map + page, n);
        }
      }
      __syncthreads();
    }
    int need = 0, copies = 0;
    for (int n0 = 0; n0 < a.nseq; n0 += kPlanThreads) {
      const int n = n0 + tid;
      if (!one) look(n, want, page);
      if (page >= 0) {
        if (__ldcg(s.list2 + page) >= a.refs[page] && __ldcg(s.map + page) == n)
          page = -1;   // the last of its holders, who all grow, keeps it
        else
          ++want;
      }
      int sum, ncow = 0, at = 0;
      const int before = block_scan(want, s_scan, &sum);
      if (__syncthreads_or(page >= 0)) at = block_scan(page >= 0, s_scan, &ncow);
      if (n < a.nseq) {
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
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int f = *cluster.map_shared_rank(&s_free, r);
    if (r < rank) before += f;
    total += f;
  }
  const bool go = need <= total;
  if (rank == 0 && tid == 0) {
    s.head[2] = go;
    if (!go) set_status(a.status, MISA_ERR_OUT_OF_PAGES);
  }
  if (go)
    rank_slice<true>(a.refs, lo, hi, before, need, s_bits, s_at, s_scan,
                     [&](int p, bool free, int at) {
                       if (free && at < need) s.list[at] = p;
                     });
  cluster.sync();   // the list is complete, and no CTA reads another's shared memory any more
  if constexpr (APPLY) {
    resize_entries(a, go, rank * kPlanThreads + tid, kPlanCtas * kPlanThreads);
  }
}

// Copies of pages, a piece (kCopyBytes of one page in one pool) per block and step; page_of(m,
// &src, &dst) tells copy m's pages.  The next piece's loads are in flight while one is stored.
template <typename F>
__device__ __forceinline__ void copy_pages(const PagePools& pools, int pieces, int copies,
                                           F page_of) {
  const int64_t per = (int64_t)pools.n * pieces, work = copies * per;
  uint4 x[2][kCopyUnroll];
  uint4* to[2];
  int left[2];   // 16-byte words from this thread's first one to the piece's end
  auto load = [&](int64_t i, int b) {
    left[b] = 0;
    if (i >= work) return;
    const int m = (int)(i / per), y = (int)(i - m * per), pool = y / pieces;
    const uint32_t bytes = pools.page_bytes[pool], at = (uint32_t)(y - pool * pieces) * kCopyBytes;
    if (at >= bytes) return;
    int src, dst;
    page_of(m, &src, &dst);
    unsigned char* base = pools.base[pool] + at;
    const uint4* from = reinterpret_cast<const uint4*>(base + (size_t)src * bytes) + threadIdx.x;
    to[b] = reinterpret_cast<uint4*>(base + (size_t)dst * bytes) + threadIdx.x;
    left[b] = (int)(min(bytes - at, (uint32_t)kCopyBytes) / 16) - (int)threadIdx.x;
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (u * kApplyThreads < left[b]) x[b][u] = __ldcs(from + u * kApplyThreads);
  };
  auto store = [&](int b) {
#pragma unroll
    for (int u = 0; u < kCopyUnroll; ++u)
      if (u * kApplyThreads < left[b]) __stcs(to[b] + u * kApplyThreads, x[b][u]);
  };
  load(blockIdx.x, 0);
  for (int64_t i = blockIdx.x; i < work; i += 2 * (int64_t)gridDim.x) {
    load(i + gridDim.x, 1);
    store(0);
    load(i + 2 * (int64_t)gridDim.x, 0);
    store(1);
  }
}

__global__ void __launch_bounds__(kApplyThreads, 4)
    resize_apply_kernel(const ResizeArgs a, const __grid_constant__ PagePools pools, int pieces) {
  pdl_prologue();
  const bool go = a.s.head[2] != 0;
  resize_entries(a, go, blockIdx.x * kApplyThreads + threadIdx.x, gridDim.x * kApplyThreads);
  if (go && pools.n > 0)
    copy_pages(pools, pieces, a.s.head[0], [&](int m, int* src, int* dst) {
      const int n = a.s.cow_seq[m];
      *src = a.s.cow[n];
      *dst = a.s.list[a.s.first[n]];
    });
}

__global__ void __launch_bounds__(kPlanThreads, 1)
    compact_plan_kernel(const int32_t* refs, int num_pages, int32_t* out_refs, int32_t* n_live_out,
                        PlanScratch s) {
  __shared__ int s_scan[32];
  __shared__ uint32_t s_bits[kPlanThreads];
  __shared__ int s_at[kPlanThreads];
  __shared__ int s_live, s_holes;
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
  const int slice = (num_pages + kPlanCtas - 1) / kPlanCtas;
  const int lo = min(num_pages, rank * slice), hi = min(num_pages, lo + slice);
  const int live = count_slice<false>(refs, lo, hi, out_refs, s_bits, s_scan);
  if (tid == 0) {
    s_live = live;
    s_holes = 0;
    if (rank == 0) s.head[0] = 0;
  }
  cluster.sync();
  int before = 0, n_live = 0;
#pragma unroll
  for (int r = 0; r < kPlanCtas; ++r) {
    const int f = *cluster.map_shared_rank(&s_live, r);
    if (r < rank) before += f;
    n_live += f;
  }
  auto token = cluster.barrier_arrive();   // this CTA reads no other's shared memory any more
  int holes = 0;
  rank_slice<false>(refs, lo, hi, before, INT_MAX, s_bits, s_at, s_scan,
                    [&](int p, bool is_live, int at) {
                      if (p >= n_live) {
                        if (is_live) s.list2[at] = p;
                        s.map[p] = is_live ? at : -1;
                      } else if (!is_live) {
                        s.list[p - at] = p;
                        ++holes;
                      }
                    });
  if (holes) atomicAdd(&s_holes, holes);
  __syncthreads();
  if (tid == 0) {
    if (s_holes) atomicAdd(s.head, s_holes);
    if (rank == 0) {
      s.head[1] = n_live;
      if (n_live_out) *n_live_out = n_live;
    }
  }
  cluster.barrier_wait(std::move(token));
}

__global__ void __launch_bounds__(kApplyThreads, 4)
    compact_apply_kernel(const int32_t* table, const int32_t* refs, int entries, int num_pages,
                         const __grid_constant__ PagePools pools, int pieces, int32_t* out_table,
                         int32_t* out_refs, PlanScratch s, int* status) {
  pdl_prologue();
  const int moves = s.head[0], n_live = s.head[1];
  const int stay = n_live - moves;   // live pages below n_live
  for (int m = blockIdx.x * kApplyThreads + threadIdx.x; m < moves;
       m += gridDim.x * kApplyThreads) {
    const int src = s.list2[stay + m];
    out_refs[s.list[m]] = refs[src];
    out_refs[src] = 0;
  }
  for (int i = blockIdx.x * kApplyThreads + threadIdx.x; i < entries;
       i += gridDim.x * kApplyThreads) {
    const int was = table[i];
    int now = was;
    if (was < -1 || was >= num_pages) {
      set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
    } else if (was >= n_live) {
      const int at = s.map[was];
      if (at >= 0)
        now = s.list[at - stay];
      else   // the table names a page that refs says is free
        set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
    }
    if (now != was || out_table != table) out_table[i] = now;
  }
  if (pools.n > 0)
    copy_pages(pools, pieces, moves, [&](int m, int* src, int* dst) {
      *src = s.list2[stay + m];
      *dst = s.list[m];
    });
}

struct ForkArgs {
  const int32_t* table;
  const int32_t* parent;
  int32_t* out_table;
  int32_t* out_refs;
  int* status;
  int nseq, max_pages, num_pages, entries;
  Divide by_row;   // division by max_pages
};

// Entry i = n * max_pages + c before and after: row n takes the entries of row parent[n].
__device__ __forceinline__ void fork_read(const ForkArgs& a, int i, int& was, int& now) {
  const int n = a.by_row(i);
  int from = a.parent[n];
  if (from < -1 || from >= a.nseq) {
    set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
    from = n;
  }
  was = a.table[i];
  now = from < 0 ? -1 : a.table[i + (from - n) * a.max_pages];
}

// The counts follow; an entry that stays the same touches none.
__device__ __forceinline__ void fork_count(const ForkArgs& a, int was, int now) {
  if (was < -1 || was >= a.num_pages) set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
  if (now != was) {
    if ((unsigned)now < (unsigned)a.num_pages) atomicAdd(a.out_refs + now, 1);
    if ((unsigned)was < (unsigned)a.num_pages) atomicSub(a.out_refs + was, 1);
  }
}

// A table of at most kPlanCtas * kPlanThreads * kForkUnroll entries by one cluster: everything is
// read (and refs copied) before anything is written, so that it also works in place.
__global__ void __launch_bounds__(kPlanThreads, 1)
    fork_small_kernel(const ForkArgs a, const int32_t* refs) {
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int at = (int)cluster.block_rank() * kPlanThreads + threadIdx.x;
  constexpr int kStep = kPlanCtas * kPlanThreads;
  int was[kForkUnroll], now[kForkUnroll];
#pragma unroll
  for (int u = 0; u < kForkUnroll; ++u)
    if (at + u * kStep < a.entries) fork_read(a, at + u * kStep, was[u], now[u]);
  if (a.out_refs != refs)
    for (int p = at; p < a.num_pages; p += kStep) a.out_refs[p] = refs[p];
  cluster.sync();
#pragma unroll
  for (int u = 0; u < kForkUnroll; ++u)
    if (at + u * kStep < a.entries) {
      fork_count(a, was[u], now[u]);
      a.out_table[at + u * kStep] = now[u];
    }
}

// Any table, V entries (of one row) a thread and step.  The counts bound it: an entry that changes
// costs two atomic updates at random places, 0.75 M of each 4 us (1024 rows of 2048 entries, half
// of the rows changing: 9 us without the counts).
template <int V>
__global__ void __launch_bounds__(kApplyThreads) fork_kernel(const ForkArgs a) {
  pdl_prologue();
  const int words = a.entries / V, step = gridDim.x * kApplyThreads;
  for (int w = blockIdx.x * kApplyThreads + threadIdx.x; w < words; w += step) {
    const int i = w * V, n = a.by_row(i);
    int from = a.parent[n];
    if (from < -1 || from >= a.nseq) {
      set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
      from = n;
    }
    int was[V], now[V];
    if constexpr (V == 4) {
      *reinterpret_cast<int4*>(was) = *reinterpret_cast<const int4*>(a.table + i);
      if (from == n)
        *reinterpret_cast<int4*>(now) = *reinterpret_cast<const int4*>(was);
      else if (from < 0)
        *reinterpret_cast<int4*>(now) = make_int4(-1, -1, -1, -1);
      else
        *reinterpret_cast<int4*>(now) =
            *reinterpret_cast<const int4*>(a.table + i + (from - n) * a.max_pages);
      *reinterpret_cast<int4*>(a.out_table + i) = *reinterpret_cast<const int4*>(now);
    } else {
      was[0] = a.table[i];
      now[0] = from < 0 ? -1 : a.table[i + (from - n) * a.max_pages];
      a.out_table[i] = now[0];
    }
#pragma unroll
    for (int v = 0; v < V; ++v) fork_count(a, was[v], now[v]);
  }
}

// 32-bit words from one buffer to another, neither overlapping the other; V = 4: 16-byte aligned.
template <int V>
__global__ void __launch_bounds__(kApplyThreads)
    copy_words_kernel(const int32_t* __restrict__ from, int32_t* __restrict__ to, int n) {
  pdl_prologue();
  const int step = gridDim.x * kApplyThreads, first = blockIdx.x * kApplyThreads + threadIdx.x;
  if constexpr (V == 4) {
#pragma unroll 4
    for (int i = first; i < n / 4; i += step)
      reinterpret_cast<int4*>(to)[i] = reinterpret_cast<const int4*>(from)[i];
    if (first < n % 4) to[n / 4 * 4 + first] = from[n / 4 * 4 + first];
  } else {
    for (int i = first; i < n; i += step) to[i] = from[i];
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
int apply_grid(int64_t entries, int64_t copies, const PagePools* pools, int pieces) {
  int64_t n = (entries + kApplyThreads - 1) / kApplyThreads;
  const int64_t c = pools ? copies * pools->n * pieces : 0;
  if (c > n) n = c;
  return (int)(n < 148 * 8 ? n : 148 * 8);
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

cudaError_t copy_words(const int32_t* from, int32_t* to, int n, cudaStream_t st) {
  const bool wide = n >= 4 && aligned16(from) && aligned16(to);
  return launch_pdl(wide ? copy_words_kernel<4> : copy_words_kernel<1>,
                    dim3(apply_grid(wide ? n / 4 : n, 0, nullptr, 0)), dim3(kApplyThreads), 0, st,
                    from, to, n);
}

}  // namespace

size_t pages_ws_bytes(int nseq, int num_pages) { return plan_scratch(nseq, num_pages, nullptr, nullptr); }

// A large table that changes in place is read from a copy.
size_t fork_ws_bytes(int nseq, int max_pages, int num_pages) {
  const int64_t entries = (int64_t)nseq * max_pages;
  return entries <= kSmallEntries && num_pages <= kSmallPages ? 0 : align256(entries * 4);
}

cudaError_t launch_pages_resize(const int32_t* table, const int32_t* refs, const int32_t* old_len,
                                const int32_t* new_len, int nseq, int max_pages, int num_pages,
                                int page_size, const PagePools& pools, int32_t* out_table,
                                int32_t* out_refs, void* scratch, int* status, cudaStream_t st) {
  ResizeArgs a = {table,  refs, old_len,   new_len,   out_table, out_refs,
                  status, nseq, max_pages, num_pages, page_size, Divide::by(max_pages)};
  plan_scratch(nseq, num_pages, scratch, &a.s);
  const int entries = nseq * max_pages;
  if (pools.n == 0 && entries <= kSmallEntries)
    return launch_plan(resize_plan_kernel<true>, st, a);
  const cudaError_t e = launch_plan(resize_plan_kernel<false>, st, a);
  if (e != cudaSuccess) return e;
  const int pieces = pieces_of(pools);
  return launch_pdl(resize_apply_kernel, dim3(apply_grid(entries, nseq, &pools, pieces)),
                    dim3(kApplyThreads), 0, st, a, pools, pieces);
}

cudaError_t launch_pages_fork(const int32_t* table, const int32_t* refs, const int32_t* parent,
                              int nseq, int max_pages, int num_pages, int32_t* out_table,
                              int32_t* out_refs, void* scratch, int* status, cudaStream_t st) {
  ForkArgs a = {table,     parent,    out_table,        out_refs,              status, nseq,
                max_pages, num_pages, nseq * max_pages, Divide::by(max_pages)};
  if (a.entries <= kSmallEntries && num_pages <= kSmallPages)
    return launch_plan(fork_small_kernel, st, a, refs);
  cudaError_t e = cudaSuccess;
  if (out_refs != refs) e = copy_words(refs, out_refs, num_pages, st);
  if (e == cudaSuccess && out_table == table) {   // rows read one another: in place, from a copy
    e = copy_words(table, static_cast<int32_t*>(scratch), a.entries, st);
    a.table = static_cast<const int32_t*>(scratch);
  }
  if (e != cudaSuccess) return e;
  const bool wide = max_pages % 4 == 0 && aligned16(a.table) && aligned16(out_table);
  return launch_pdl(wide ? fork_kernel<4> : fork_kernel<1>,
                    dim3(apply_grid(a.entries / (wide ? 4 : 1), 0, nullptr, 0)),
                    dim3(kApplyThreads), 0, st, a);
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
  const int entries = nseq * max_pages;
  return launch_pdl(compact_apply_kernel, dim3(apply_grid(entries, num_pages / 2, &pools, pieces)),
                    dim3(kApplyThreads), 0, st, table, refs, entries, num_pages, pools, pieces,
                    out_table, out_refs, s, status);
}

}  // namespace misa

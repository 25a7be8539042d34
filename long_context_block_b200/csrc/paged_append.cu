// K10: the keys and values of new tokens copied into their pages of the cache: row (n, t) goes to
// token pos[n, t] of sequence n.  HBM-bound: every byte is read once and written once.  A thread
// moves U 16-byte pieces: their loads, the position and the page entry are all in flight before
// the first store.  U = 4 with streaming stores: 40.4 us for the 241 MB of four prompt chunks (5.97
// TB/s, 91% of the measured copy rate; U = 2 44.6, U = 8 53.0, plain stores 41.9 us).  A decode
// step's few rows take U = 1 and plain stores, as the attention after it reads them: 1.6 us for 32
// rows of 8 heads, a launch.
#include <cuda_runtime.h>

#include "internal.h"
#include "misa.h"
#include "paged.cuh"

namespace misa {
namespace {

using namespace paged;

constexpr int kAppendThreads = 256;

// blockIdx.y: 0 keys, 1 values.  `per_row`: 16-byte pieces of a row.
template <int U>
__global__ void __launch_bounds__(kAppendThreads, 6)
    paged_append_kernel(const uint4* __restrict__ k_new, const uint4* __restrict__ v_new,
                        const int32_t* __restrict__ pos, const int32_t* __restrict__ table, int T,
                        int64_t pieces, int per_row, int num_pages, int page_size, Divide by_page,
                        int max_pages,
                        uint4* __restrict__ k_cache, uint4* __restrict__ v_cache, int* status) {
  pdl_prologue();
  const uint4* src = blockIdx.y ? v_new : k_new;
  uint4* dst = blockIdx.y ? v_cache : k_cache;
  const int64_t base = (int64_t)blockIdx.x * (kAppendThreads * U);
  const int row0 = (int)(base / per_row);
  const int rem = (int)(base - (int64_t)row0 * per_row);
  uint4 x[U];
  int row[U];
  int c[U], p[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = rem + u * kAppendThreads + (int)threadIdx.x;
    row[u] = row0 + at / per_row;
    c[u] = at % per_row;
    p[u] = -1;
    if (base + u * kAppendThreads + (int)threadIdx.x < pieces) {
      x[u] = __ldcs(src + base + u * kAppendThreads + threadIdx.x);
      p[u] = last_token(pos, row[u], max_pages * page_size, status);
      // a position past the table's last page has no place: skipped, not clamped onto another
      if (p[u] != pos[row[u]]) p[u] = -1;
    }
  }
  int at[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    at[u] = p[u] < 0 ? -1
                     : cache_row(table + (int64_t)(row[u] / T) * max_pages, p[u], page_size, by_page, num_pages, status);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (at[u] >= 0) {
      uint4* to = dst + (int64_t)at[u] * per_row + c[u];
      if (U > 1)
        __stcs(to, x[u]);
      else
        *to = x[u];
    }
}

}  // namespace

cudaError_t launch_paged_append(const void* k_new, const void* v_new, const int32_t* pos,
                                const int32_t* page_table, int nseq, int T, int row_bytes,
                                int num_pages, int page_size, int max_pages, void* k_cache,
                                void* v_cache, int* status, cudaStream_t st) {
  const int per_row = row_bytes / 16;
  const int64_t pieces = (int64_t)nseq * T * per_row;
  // one piece a thread until every SM has two blocks' worth, then four
  const bool wide = pieces > 148 * 2 * kAppendThreads;
  const int64_t per_block = kAppendThreads * (wide ? 4 : 1);
  const int64_t blocks = (pieces + per_block - 1) / per_block;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(wide ? paged_append_kernel<4> : paged_append_kernel<1>,
                    dim3((unsigned)blocks, 2), dim3(kAppendThreads), 0, st,
                    static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), pos,
                    page_table, T, pieces, per_row, num_pages, page_size, Divide::by(page_size), max_pages,
                    static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), status);
}

}  // namespace misa

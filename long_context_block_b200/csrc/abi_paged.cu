// C ABI of the paged key-value cache: argument validation and the launches of each entry point.
// Declarations and contracts: include/misa.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "internal.h"
#include "misa.h"
#include "misa_testing.h"

using namespace misa;

namespace {

#define MISA_TRY(expr)            \
  do {                            \
    const int _s = (expr);        \
    if (_s != MISA_OK) return _s; \
  } while (0)

int cuda_status(cudaError_t e) { return e == cudaSuccess ? MISA_OK : MISA_ERR_CUDA; }

// Token counts and row ids are 32-bit in the kernels.
constexpr int64_t kMaxSpan = int64_t(1) << 30;

int check_table(int nseq, int max_pages, int num_pages) {
  if (nseq < 1 || max_pages < 1 || num_pages < 1) return MISA_ERR_INVALID_ARG;
  if (num_pages > kMaxSpan || (int64_t)nseq * max_pages > kMaxSpan) return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

int check_cache(int dtype, int nseq, int T, int Hkv, int d, int num_pages, int page_size,
                int max_pages) {
  if (nseq < 1 || T < 1 || Hkv < 1 || d < 1 || page_size < 1) return MISA_ERR_INVALID_ARG;
  if (dtype != MISA_DTYPE_BF16 && dtype != MISA_DTYPE_FP16) return MISA_ERR_INVALID_ARG;
  MISA_TRY(check_table(nseq, max_pages, num_pages));
  if ((d != 64 && d != 128) || Hkv > (1 << 16) || (int64_t)nseq * T >= INT32_MAX ||
      (int64_t)max_pages * page_size > kMaxSpan ||
      (int64_t)num_pages * page_size > INT32_MAX)
    return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

int check_heads(int nseq, int T, int Hq, int Hkv, int topk) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv || topk < 0) return MISA_ERR_INVALID_ARG;
  if ((int64_t)nseq * T >= INT32_MAX || (int64_t)nseq * T * Hq >= INT32_MAX || topk > kMaxSpan)
    return MISA_ERR_UNSUPPORTED;
  return MISA_OK;
}

int check_scratch(void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return MISA_OK;
  if (ws_bytes < need) return MISA_ERR_WORKSPACE_TOO_SMALL;
  return check_dev(ws, need, 256);
}

struct Buffer {
  const void* p;   // null: none
  size_t bytes;
};

bool overlap(const Buffer& x, const Buffer& y) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x.p), b = reinterpret_cast<uintptr_t>(y.p);
  return a != 0 && b != 0 && a < b + y.bytes && b < a + x.bytes;
}

// What is written must not overlap what another buffer holds.
int check_apart(std::initializer_list<Buffer> written, std::initializer_list<Buffer> read) {
  for (const Buffer* x = written.begin(); x != written.end(); ++x) {
    for (const Buffer* y = x + 1; y != written.end(); ++y)
      if (overlap(*x, *y)) return MISA_ERR_INVALID_ARG;
    for (const Buffer& y : read)
      if (overlap(*x, y)) return MISA_ERR_INVALID_ARG;
  }
  return MISA_OK;
}

// An input that the output may take the place of: none where it does.
Buffer unless(const void* out, const Buffer& in) {
  return {out == in.p ? nullptr : in.p, in.bytes};
}

// The buffers of an upkeep call; x, y: its own inputs, nseq ints each.
struct Upkeep {
  const int32_t *table, *refs, *x, *y;
  const int32_t *out_table, *out_refs, *n_live, *status;
  const void* ws;
};

int check_upkeep(int op, const Upkeep& u, int nseq, int max_pages, int num_pages, size_t ws_bytes,
                 const PagePools* pools) {
  const size_t tb = (size_t)nseq * max_pages * 4, rb = (size_t)num_pages * 4, nb = (size_t)nseq * 4;
  const size_t need = misa_pages_workspace_size(op, nseq, max_pages, num_pages);
  MISA_TRY(check_dev(u.table, tb, 4));
  MISA_TRY(check_dev(u.refs, rb, 4));
  MISA_TRY(check_dev(u.out_table, tb, 4));
  MISA_TRY(check_dev(u.out_refs, rb, 4));
  MISA_TRY(check_opt(u.n_live, 4, 4));
  MISA_TRY(check_opt(u.status, 4, 4));
  MISA_TRY(check_scratch(const_cast<void*>(u.ws), ws_bytes, need));
  const Buffer table = {u.table, tb}, refs = {u.refs, rb}, x = {u.x, nb}, y = {u.y, nb};
  const Buffer out_table = {u.out_table, tb}, out_refs = {u.out_refs, rb}, n_live = {u.n_live, 4};
  const Buffer status = {u.status, 4}, ws = {need ? u.ws : nullptr, need};
  MISA_TRY(check_apart({out_table, out_refs, n_live, status, ws},
                       {unless(u.out_table, table), unless(u.out_refs, refs), x, y}));
  for (int i = 0; pools && i < pools->n; ++i)
    MISA_TRY(check_apart({{pools->base[i], (size_t)num_pages * pools->page_bytes[i]}},
                         {table, refs, x, y, out_table, out_refs, n_live, status, ws}));
  return MISA_OK;
}

int take_pools(void* const* pools, const int64_t* page_bytes, int npools, int num_pages,
               PagePools* out) {
  if (npools < 0 || (npools > 0 && (pools == nullptr || page_bytes == nullptr)))
    return MISA_ERR_INVALID_ARG;
  if (npools > MISA_MAX_POOLS) return MISA_ERR_UNSUPPORTED;
  out->n = npools;
  for (int i = 0; i < npools; ++i) {
    if (page_bytes[i] < 16 || page_bytes[i] % 16) return MISA_ERR_INVALID_ARG;
    if (page_bytes[i] > kMaxSpan) return MISA_ERR_UNSUPPORTED;
    MISA_TRY(check_dev(pools[i], (size_t)num_pages * page_bytes[i], 16));
    out->base[i] = static_cast<unsigned char*>(pools[i]);
    out->page_bytes[i] = (uint32_t)page_bytes[i];
  }
  Buffer all[MISA_MAX_POOLS];
  for (int i = 0; i < npools; ++i) all[i] = {pools[i], (size_t)num_pages * page_bytes[i]};
  std::sort(all, all + npools, [](const Buffer& x, const Buffer& y) { return x.p < y.p; });
  for (int i = 1; i < npools; ++i)
    if (overlap(all[i - 1], all[i])) return MISA_ERR_INVALID_ARG;
  return MISA_OK;
}

}  // namespace

extern "C" {

size_t misa_paged_attention_workspace_size(int nseq, int T, int Hq, int Hkv, int d, int page_size,
                                           int max_pages, int topk) {
  if (nseq < 1 || T < 1 || (d != 64 && d != 128) || page_size < 1 || max_pages < 1) return 0;
  if (check_heads(nseq, T, Hq, Hkv, topk) != MISA_OK) return 0;
  PagedAttn p = {};
  p.nseq = nseq;
  p.T = T;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.d = d;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.topk = topk;
  return paged_attn_ws_bytes(p);
}

static int paged_attention(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* page_table, const int32_t* pos, const int32_t* idx,
                           int dtype, int nseq, int T, int Hq, int Hkv, int d, int num_pages,
                           int page_size, int max_pages, int topk, float scale, void* out,
                           float* lse, int32_t* device_status, void* ws, size_t ws_bytes,
                           void* stream, const WaitProbe* probe) {
  MISA_TRY(check_cache(dtype, nseq, T, Hkv, d, num_pages, page_size, max_pages));
  MISA_TRY(check_heads(nseq, T, Hq, Hkv, topk));
  if ((idx != nullptr) != (topk > 0) || !std::isfinite(scale)) return MISA_ERR_INVALID_ARG;
  const size_t rows = (size_t)nseq * T;
  const size_t pool = (size_t)num_pages * page_size * Hkv * d * 2;
  MISA_TRY(check_dev(q, rows * Hq * d * 2, 16));
  MISA_TRY(check_dev(k_cache, pool, 16));
  MISA_TRY(check_dev(v_cache, pool, 16));
  MISA_TRY(check_dev(page_table, (size_t)nseq * max_pages * 4, 4));
  MISA_TRY(check_dev(pos, rows * 4, 4));
  MISA_TRY(check_opt(idx, rows * topk * 4, 4));
  MISA_TRY(check_dev(out, rows * Hq * d * 2, 16));
  MISA_TRY(check_opt(lse, rows * Hq * 4, 4));
  MISA_TRY(check_opt(device_status, 4, 4));
  PagedAttn p = {q,    k_cache, v_cache, page_table, pos, idx,       out,       lse,       dtype,
                 nseq, T,       Hq,      Hkv,        d,   num_pages, page_size, max_pages, topk,
                 scale, probe};
  if (probe && !paged_attn_tc(p)) return MISA_ERR_UNSUPPORTED;
  const size_t need = paged_attn_ws_bytes(p);
  MISA_TRY(check_scratch(ws, ws_bytes, need));
  const Buffer queries = {q, rows * Hq * d * 2}, result = {out, queries.bytes};
  const Buffer sums = {lse, rows * Hq * 4}, scratch = {need ? ws : nullptr, need};
  const Buffer status = {device_status, 4};
  MISA_TRY(check_apart({result, sums, scratch, status},
                       {{k_cache, pool}, {v_cache, pool}, {page_table, (size_t)nseq * max_pages * 4},
                        {pos, rows * 4}, {idx, rows * topk * 4}, unless(out, queries)}));
  if (q == out) MISA_TRY(check_apart({sums, scratch, status}, {queries}));
  return cuda_status(launch_paged_attn(p, ws, device_status, (cudaStream_t)stream));
}

int misa_paged_attention(const void* q, const void* k_cache, const void* v_cache,
                         const int32_t* page_table, const int32_t* pos, const int32_t* idx,
                         int dtype, int nseq, int T, int Hq, int Hkv, int d, int num_pages,
                         int page_size, int max_pages, int topk, float scale, void* out,
                         float* lse, int32_t* device_status, void* ws, size_t ws_bytes,
                         void* stream) {
  return paged_attention(q, k_cache, v_cache, page_table, pos, idx, dtype, nseq, T, Hq, Hkv, d,
                         num_pages, page_size, max_pages, topk, scale, out, lse, device_status,
                         ws, ws_bytes, stream, nullptr);
}

int misa_testing_paged_attention_wait_expiry(
    const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
    const int32_t* pos, const int32_t* idx, int dtype, int nseq, int T, int Hq, int Hkv, int d,
    int num_pages, int page_size, int max_pages, int topk, float scale, void* out, float* lse,
    int32_t* device_status, void* ws, size_t ws_bytes, long long wait_cycles, int skip_tile,
    void* stream) {
  if (wait_cycles < 1000 || wait_cycles > 4000000000LL || skip_tile < -1)
    return MISA_ERR_INVALID_ARG;
  WaitProbe probe;
  probe.wait_cycles = wait_cycles;
  probe.skip_tile = skip_tile;
  return paged_attention(q, k_cache, v_cache, page_table, pos, idx, dtype, nseq, T, Hq, Hkv, d,
                         num_pages, page_size, max_pages, topk, scale, out, lse, device_status,
                         ws, ws_bytes, stream, &probe);
}

int misa_paged_append(const void* k_new, const void* v_new, const int32_t* pos,
                      const int32_t* page_table, int dtype, int nseq, int T, int Hkv, int d,
                      int num_pages, int page_size, int max_pages, void* k_cache, void* v_cache,
                      int32_t* device_status, void* stream) {
  MISA_TRY(check_cache(dtype, nseq, T, Hkv, d, num_pages, page_size, max_pages));
  const size_t rows = (size_t)nseq * T;
  const size_t pool = (size_t)num_pages * page_size * Hkv * d * 2;
  MISA_TRY(check_dev(k_new, rows * Hkv * d * 2, 16));
  MISA_TRY(check_dev(v_new, rows * Hkv * d * 2, 16));
  MISA_TRY(check_dev(pos, rows * 4, 4));
  MISA_TRY(check_dev(page_table, (size_t)nseq * max_pages * 4, 4));
  MISA_TRY(check_dev(k_cache, pool, 16));
  MISA_TRY(check_dev(v_cache, pool, 16));
  MISA_TRY(check_opt(device_status, 4, 4));
  MISA_TRY(check_apart({{k_cache, pool}, {v_cache, pool}, {device_status, 4}},
                       {{page_table, (size_t)nseq * max_pages * 4}, {pos, rows * 4}}));
  return cuda_status(launch_paged_append(k_new, v_new, pos, page_table, nseq, T, Hkv * d * 2,
                                         num_pages, page_size, max_pages, k_cache, v_cache,
                                         device_status, (cudaStream_t)stream));
}

size_t misa_pages_workspace_size(int op, int nseq, int max_pages, int num_pages) {
  if (check_table(nseq, max_pages, num_pages) != MISA_OK) return 0;
  switch (op) {
    case MISA_OP_PAGES_RESIZE:
    case MISA_OP_PAGES_COMPACT:
      return pages_ws_bytes(nseq, num_pages);
    case MISA_OP_PAGES_FORK:
      return fork_ws_bytes(nseq, max_pages, num_pages);
    default:
      return 0;
  }
}

int misa_pages_resize(const int32_t* page_table, const int32_t* refs, const int32_t* old_len,
                      const int32_t* new_len, int nseq, int max_pages, int num_pages,
                      int page_size, void* const* pools, const int64_t* page_bytes, int npools,
                      int32_t* out_table, int32_t* out_refs, int32_t* device_status, void* ws,
                      size_t ws_bytes, void* stream) {
  MISA_TRY(check_table(nseq, max_pages, num_pages));
  if (page_size < 1) return MISA_ERR_INVALID_ARG;
  if ((int64_t)max_pages * page_size > kMaxSpan) return MISA_ERR_UNSUPPORTED;
  MISA_TRY(check_dev(old_len, (size_t)nseq * 4, 4));
  MISA_TRY(check_dev(new_len, (size_t)nseq * 4, 4));
  PagePools pp;
  MISA_TRY(take_pools(pools, page_bytes, npools, num_pages, &pp));
  MISA_TRY(check_upkeep(MISA_OP_PAGES_RESIZE,
                        {page_table, refs, old_len, new_len, out_table, out_refs, nullptr,
                         device_status, ws},
                        nseq, max_pages, num_pages, ws_bytes, &pp));
  return cuda_status(launch_pages_resize(page_table, refs, old_len, new_len, nseq, max_pages,
                                         num_pages, page_size, pp, out_table, out_refs, ws,
                                         device_status, (cudaStream_t)stream));
}

int misa_pages_fork(const int32_t* page_table, const int32_t* refs, const int32_t* parent,
                    int nseq, int max_pages, int num_pages, int32_t* out_table,
                    int32_t* out_refs, int32_t* device_status, void* ws, size_t ws_bytes,
                    void* stream) {
  MISA_TRY(check_table(nseq, max_pages, num_pages));
  MISA_TRY(check_dev(parent, (size_t)nseq * 4, 4));
  MISA_TRY(check_upkeep(MISA_OP_PAGES_FORK,
                        {page_table, refs, parent, nullptr, out_table, out_refs, nullptr,
                         device_status, ws},
                        nseq, max_pages, num_pages, ws_bytes, nullptr));
  return cuda_status(launch_pages_fork(page_table, refs, parent, nseq, max_pages, num_pages,
                                       out_table, out_refs, ws, device_status,
                                       (cudaStream_t)stream));
}

int misa_pages_compact(const int32_t* page_table, const int32_t* refs, int nseq, int max_pages,
                       int num_pages, void* const* pools, const int64_t* page_bytes, int npools,
                       int32_t* out_table, int32_t* out_refs, int32_t* n_live,
                       int32_t* device_status, void* ws, size_t ws_bytes, void* stream) {
  MISA_TRY(check_table(nseq, max_pages, num_pages));
  PagePools pp;
  MISA_TRY(take_pools(pools, page_bytes, npools, num_pages, &pp));
  MISA_TRY(check_upkeep(MISA_OP_PAGES_COMPACT,
                        {page_table, refs, nullptr, nullptr, out_table, out_refs, n_live,
                         device_status, ws},
                        nseq, max_pages, num_pages, ws_bytes, &pp));
  return cuda_status(launch_pages_compact(page_table, refs, nseq, max_pages, num_pages, pp,
                                          out_table, out_refs, n_live, ws, device_status,
                                          (cudaStream_t)stream));
}

}  // extern "C"

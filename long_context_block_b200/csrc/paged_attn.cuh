// What the kernels of the paged attention share: arguments, row blocks, the cut of all items'
// units into equal ranges and the join of partials.
#pragma once

#include <cmath>

#include "internal.h"
#include "misa.h"
#include "paged.cuh"

namespace misa {
namespace paged {

// Units that starting on an item costs, when ranges are cut (about 3 us; 32 ragged sequences of up
// to 8192 tokens, where one range held ten short items: 92 against 103 us without).
constexpr int kItemCost = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  const int32_t* table;
  const int32_t* pos;
  const int32_t* idx;
  void* out;
  float* lse;
  int* status;
  float* part_o;   // [2 * kMaxCtas][RB][D]
  float2* part_ml; // [2 * kMaxCtas][RB]  (maximum in the log2 domain, sum)
  int2* split;     // [kMaxCtas]: item that starts in this CTA and ends in another (-1: none),
                   // and the CTA it ends in
  int nseq, T, Hq, Hkv, G, num_pages, page_size, max_pages, topk;
  int nb;          // row blocks: per sequence (prefix form) or per query (selected form)
  float scale2;    // |scale| log2 e, or 1 with queries of zeros
  uint32_t q_flip; // sign bits of a query's word to flip (scale < 0)
  uint32_t q_keep; // bits of a query's word to keep (none: scale = 0)
  Divide by_page;  // division by page_size
};

// An entry is a row block: of a sequence's T * G rows (prefix form, r = t * G + g) or of one
// query's G rows (selected form).
template <int RB, bool SEL>
struct Entry {
  int n, row0, rows;
  __device__ __forceinline__ Entry(const AttnArgs& a, int e) {
    const int nq = e / a.nb, b = e - nq * a.nb;
    if (SEL) {
      n = nq / a.T;
      row0 = (nq - n * a.T) * a.G + b * RB;
      rows = min(RB, a.G - b * RB);
    } else {
      n = nq;
      row0 = b * RB;
      rows = min(RB, a.T * a.G - row0);
    }
  }
  // tokens the entry walks over
  __device__ __forceinline__ int tokens(const AttnArgs& a) const {
    if (SEL) return a.topk;
    int last = -1;
    for (int t = row0 / a.G; t <= (row0 + rows - 1) / a.G; ++t)
      last = max(last, last_token(a.pos, (int64_t)n * a.T + t, a.max_pages * a.page_size,
                                  a.status));
    return last + 1;
  }
};

// One output position: 4 elements of a row, from its sum of weights and weighted values.
template <typename E, int D>
__device__ __forceinline__ void finish(const AttnArgs& a, int n, int rr, int hk, int c,
                                       const float4& acc, float mm, float ll) {
  const int t = rr / a.G, g = rr - t * a.G;
  const int64_t head = ((int64_t)n * a.T + t) * a.Hq + hk * a.G + g;
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  uint2 y;
  y.x = pack2<E>(acc.x * inv, acc.y * inv);
  y.y = pack2<E>(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(static_cast<E*>(a.out) + head * D + c) = y;
  if (a.lse && c == 0) a.lse[head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// Adds a part (maximum pm, sum pl, weighted values x) under the joint maximum mm.
__device__ __forceinline__ void add_part(float4& acc, float& ll, float mm, float pm, float pl,
                                         const float4& x) {
  const float f = pm == mm ? 1.f : exp2_approx(pm - (mm == -INFINITY ? 0.f : mm));
  ll += pl * f;
  acc.x += x.x * f;
  acc.y += x.y * f;
  acc.z += x.z * f;
  acc.w += x.w * f;
}

// The share of one CTA of NT threads in all items' units.  An item of u units costs kItemCost + u:
// the cost of starting on it (lookups, filling the ring) comes first.  Ranges of equal cost, one
// for each of the first nc CTAs.
template <int RB, bool SEL, int UNIT, int NT>
struct Range {
  long long x, x1, total, off;   // position, end, sum of all costs; from the start of entry e to x
  int e, nc;

  struct Shared {
    long long sum[NT / 32], off;
    int e;
  };
  // A piece of one item: units uo .. uo + take - 1 of `units`.
  struct Segment {
    int e, hk, uo, take, units, ntok;
    int last_cta;   // of the item
  };

  static __device__ __forceinline__ int units_of(int ntok) {
    return max(1, (ntok + UNIT - 1) / UNIT);
  }

  // Every thread of the CTA; false: no share.
  __device__ __forceinline__ bool cut(const AttnArgs& a, Shared& sh) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ne = (SEL ? a.nseq * a.T : a.nseq) * a.nb;
    const int chunk = (ne + NT - 1) / NT;
    const int per = SEL ? (kItemCost + units_of(a.topk)) * a.Hkv : 0;   // cost of an entry
    auto cost_of = [&](int i) {
      return (kItemCost + units_of(Entry<RB, SEL>(a, i).tokens(a))) * a.Hkv;
    };
    long long mine = 0, before = 0;
    total = (long long)ne * per;
    if (!SEL) {
      for (int i = tid * chunk; i < min(ne, (tid + 1) * chunk); ++i) mine += cost_of(i);
      long long inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sh.sum[warp] = inc;
      __syncthreads();
      before = inc - mine;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += sh.sum[w];
        total += sh.sum[w];
      }
    }
    nc = (int)min((long long)gridDim.x, total);
    const int cta = blockIdx.x;
    if (cta >= nc) return false;
    x = cta * total / nc;
    x1 = (cta + 1) * total / nc;
    if constexpr (SEL) {
      e = (int)(x / per);
      off = x - (long long)e * per;
    } else {
      if (x >= before && x < before + mine) {
        off = x - before;
        e = tid * chunk;
        for (int n = cost_of(e); off >= n; n = cost_of(e)) {
          off -= n;
          ++e;
        }
        sh.e = e;
        sh.off = off;
      }
      __syncthreads();
      e = sh.e;
      off = sh.off;
    }
    return true;
  }

  // The next piece that holds units; false: none.
  __device__ __forceinline__ bool next(const AttnArgs& a, Segment& s) {
    while (x < x1) {
      s.e = e;
      s.ntok = Entry<RB, SEL>(a, e).tokens(a);
      s.units = units_of(s.ntok);
      const int cost = kItemCost + s.units;
      s.hk = (int)(off / cost);
      const int at = (int)(off - (long long)s.hk * cost);
      const int go = (int)min((long long)(cost - at), x1 - x);
      s.uo = max(0, at - kItemCost);
      s.take = max(0, at + go - kItemCost) - s.uo;
      // position y of all costs lies in CTA floor(((y + 1) nc - 1) / total); y: the last unit
      s.last_cta = (int)(((x - at + cost) * nc - 1) / total);
      x += go;
      off += go;
      if (off == (long long)cost * a.Hkv) {
        ++e;
        off = 0;
      }
      if (s.take > 0) return true;
    }
    return false;
  }
};

// Joins the partials of the items that several CTAs share, in CTA order: block (c, y) the rows
// kJoinRows y .. of the item that starts in CTA c.  A few KB per item: latency-bound, so a row's
// parts are dealt out to kJoinGroups groups of threads.
constexpr int kJoinRows = 2, kJoinGroups = 4, kJoinBatch = 8;

template <typename E, int D, int RB, bool SEL>
__global__ void __launch_bounds__(kJoinRows* kJoinGroups*(D / 4))
    paged_join_kernel(const AttnArgs a) {
  constexpr int LANES = D / 4;
  __shared__ float4 s_acc[kJoinRows * kJoinGroups][LANES];
  __shared__ float2 s_ml[kJoinRows * kJoinGroups];
  pdl_prologue();
  const int cta = blockIdx.x;
  const int2 sp = a.split[cta];
  if (sp.x < 0) return;
  const int e = sp.x / a.Hkv, hk = sp.x - e * a.Hkv;
  const Entry<RB, SEL> en(a, e);
  const int team = threadIdx.x / LANES, lane = threadIdx.x - team * LANES, c = lane * 4;
  const int group = team % kJoinGroups;
  for (int r0 = blockIdx.y * kJoinRows; r0 < en.rows; r0 += gridDim.y * kJoinRows) {
  const int r = r0 + team / kJoinGroups;
  // parts: slot 2 cta + 1, then slot 2 p of the CTAs p up to sp.y; this group's: every fourth
  float mm = -INFINITY, ll = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = cta + group; r < en.rows && p0 <= sp.y; p0 += kJoinGroups * kJoinBatch) {
    float2 part[kJoinBatch];
    float4 vals[kJoinBatch];
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {   // all reads at once
      const int p = p0 + i * kJoinGroups, slot = p == cta ? 2 * p + 1 : 2 * p;
      part[i] = make_float2(-INFINITY, 0.f);
      if (p <= sp.y) {
        part[i] = a.part_ml[slot * RB + r];
        vals[i] = *reinterpret_cast<const float4*>(a.part_o + ((int64_t)slot * RB + r) * D + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kJoinBatch; ++i) {
      if (p0 + i * kJoinGroups > sp.y) break;
      const float2 ml = part[i];
      const float up = fmaxf(mm, ml.x);
      const float f = mm == up ? 1.f : exp2_approx(mm - up);
      ll *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
      mm = up;
      add_part(acc, ll, mm, ml.x, ml.y, vals[i]);
    }
  }
  s_acc[team][lane] = acc;
  if (lane == 0) s_ml[team] = make_float2(mm, ll);
  __syncthreads();
  if (group == 0 && r < en.rows) {
#pragma unroll
  for (int g = 1; g < kJoinGroups; ++g) mm = fmaxf(mm, s_ml[team + g].x);
  ll = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int g = 0; g < kJoinGroups; ++g)
    add_part(acc, ll, mm, s_ml[team + g].x, s_ml[team + g].y, s_acc[team + g][lane]);
  finish<E, D>(a, en.n, en.row0 + r, hk, c, acc, mm, ll);
  }
  __syncthreads();
  }
}

// ---------------------------------------------------------------- host side
// Query rows that share an item's tokens.
inline int attn_rows(const PagedAttn& p) {
  return p.topk > 0 ? p.Hq / p.Hkv : p.T * (p.Hq / p.Hkv);
}

// Scratch of equal ranges over `ctas` CTAs with row blocks of rb rows: two partials per CTA.
inline size_t attn_ws_bytes(int ctas, int rb, int d) {
  return align256((size_t)2 * ctas * rb * d * sizeof(float)) +
         align256((size_t)2 * ctas * rb * sizeof(float2)) + align256(ctas * sizeof(int2));
}

inline AttnArgs attn_args(const PagedAttn& p, void* scratch, int ctas, int rb, int* status) {
  AttnArgs a = {};
  a.q = p.q;
  a.k = p.k_cache;
  a.v = p.v_cache;
  a.table = p.page_table;
  a.pos = p.pos;
  a.idx = p.idx;
  a.out = p.out;
  a.lse = p.lse;
  a.status = status;
  char* w = static_cast<char*>(scratch);
  a.part_o = reinterpret_cast<float*>(w);
  w += align256((size_t)2 * ctas * rb * p.d * sizeof(float));
  a.part_ml = reinterpret_cast<float2*>(w);
  w += align256((size_t)2 * ctas * rb * sizeof(float2));
  a.split = reinterpret_cast<int2*>(w);
  a.nseq = p.nseq;
  a.T = p.T;
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.G = p.Hq / p.Hkv;
  a.num_pages = p.num_pages;
  a.page_size = p.page_size;
  a.max_pages = p.max_pages;
  a.topk = p.topk;
  a.scale2 = p.scale == 0.f ? 1.f : std::fabs(p.scale) * kLog2e;
  a.q_flip = p.scale < 0.f ? 0x80008000u : 0u;
  a.q_keep = p.scale == 0.f ? 0u : 0xffffffffu;
  a.by_page = Divide::by(p.page_size);
  return a;
}

template <typename E, int D, int RB, bool SEL>
cudaError_t launch_join(const AttnArgs& a, int ctas, int rows, cudaStream_t st) {
  int y = (rows + kJoinRows - 1) / kJoinRows;
  if (y > 16) y = 16;
  return launch_pdl(paged_join_kernel<E, D, RB, SEL>, dim3(ctas, y),
                    dim3(kJoinRows * kJoinGroups * (D / 4)), 0, st, a);
}

}  // namespace paged
}  // namespace misa

// What the kernels of the paged attention share: arguments, row blocks, the cut of all items'
// units into equal ranges and the join of partials.
#pragma once

#include <climits>
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
  int ctas;        // of the kernel that leaves the partials
  int whole;       // an item for every group of CTAs, none is split
  int side;        // row blocks that neighbouring CTAs walk side by side: nb, or 1 (one by one)
  float scale2;    // |scale| log2 e, or 1 with queries of zeros
  long long wait_cycles;   // bound of every wait (tensor-core form)
  int skip_tile;           // tests only: a tile of CTA 0 whose keys never come, -1: none
  uint32_t q_flip; // sign bits of a query's word to flip (scale < 0)
  uint32_t q_keep; // bits of a query's word to keep (none: scale = 0)
  Divide by_page;  // division by page_size
};

// Tokens that the longest of the prefixes of queries t0 .. t1 of sequence n holds.  By one thread,
// eight reads at once, or by a converged warp.
__device__ __forceinline__ int longest(const AttnArgs& a, int n, int t0, int t1) {
  const int cap = a.max_pages * a.page_size;
  const int32_t* pos = a.pos + (int64_t)n * a.T;
  int last = -1;
  for (int t = t0; t <= t1; t += 8) {
    int p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = pos[min(t + i, t1)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (p[i] < -1 || p[i] >= cap) set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
      last = max(last, min(p[i], cap - 1));
    }
  }
  return last + 1;
}
__device__ __forceinline__ int longest_warp(const AttnArgs& a, int n, int t0, int t1) {
  const int cap = a.max_pages * a.page_size;
  int last = -1;
  for (int t = t0 + (threadIdx.x & 31); t <= t1; t += 32)
    last = max(last, last_token(a.pos, (int64_t)n * a.T + t, cap, a.status));
  return __reduce_max_sync(0xffffffffu, last) + 1;
}

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
  // tokens the entry walks over (a converged warp)
  __device__ __forceinline__ int tokens(const AttnArgs& a) const {
    if (SEL) return a.topk;
    return longest_warp(a, n, row0 / a.G, (row0 + rows - 1) / a.G);
  }
};

// Tokens tok0 .. tok1 - 1 of a prefix entry for one key-value head.
struct Part {
  int n, row0, rows, hk, tok0, tok1;
};

// The last token that every row sees, of the rows that see tok0 (what the others gather is never
// used); with step and at, the least of one thread's share of them.
__device__ __forceinline__ int seen_by_all(const AttnArgs& a, const Part& p, int step, int at) {
  int least = INT_MAX;
  for (int t = p.row0 / a.G + at; t <= (p.row0 + p.rows - 1) / a.G; t += step) {
    const int last = last_token(a.pos, (int64_t)p.n * a.T + t, a.max_pages * a.page_size, nullptr);
    if (last >= p.tok0) least = min(least, last);
  }
  return least;
}

// One output position: 4 elements of a row, from its sum of weights and weighted values.
template <typename E, int D>
__device__ __forceinline__ void finish(const AttnArgs& a, int n, int rr, int hk, int c,
                                       const float4& acc, float mm, float ll) {
  const int t = rr / a.G, g = rr - t * a.G;
  const int64_t head = ((int64_t)n * a.T + t) * a.Hq + hk * a.G + g;
  if (Weights<E>::beyond(mm)) ll = NAN;
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  uint2 y;
  y.x = pack2<E>(acc.x * inv, acc.y * inv);
  y.y = pack2<E>(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(static_cast<E*>(a.out) + head * D + c) = y;
  if (a.lse && c == 0) a.lse[head] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * kLn2;
}

// Adds a part (maximum pm, sum pl, weighted values x) under the joint maximum mm.  A part that saw
// nothing (sum 0) adds nothing: its products may be NaN where another row's tokens were.
__device__ __forceinline__ void add_part(float4& acc, float& ll, float mm, float pm, float pl,
                                         const float4& x) {
  if (pl == 0.f) return;
  const float f = pm == mm ? 1.f : exp2_approx(pm - mm);
  ll += pl * f;
  acc.x += x.x * f;
  acc.y += x.y * f;
  acc.z += x.z * f;
  acc.w += x.w * f;
}

// A draft's later tokens lie in the same tiles as those that its earlier queries see, with weight 0
// for them, but 0 times a NaN or infinite value is NaN.  So such values of tokens that not every
// row of the block sees are set to 0 in shared memory, which tokens they were is kept (Dropped), and
// afterwards they are looked up in the cache and added to the rows that see them: a weight is
// positive, and any positive weight gives the same sum.
//
// Dropped holds a bit for every bucket of a segment's tokens, so that only these are read again: one
// value between two queries 32768 tokens apart costs 32 tokens, not 32768 (which took longer than
// the tensor-core form's waits in a test with short ones).
struct Dropped {
  static constexpr int kBuckets = 1024;
  uint32_t bits[kBuckets / 32];
  static __device__ __forceinline__ int shift(int tokens) {   // 2^shift tokens to a bucket
    return max(0, 22 - __clz(tokens - 1));
  }
  __device__ __forceinline__ void clear(int thread) {
    if (thread < kBuckets / 32) bits[thread] = 0u;
  }
  __device__ __forceinline__ void add(int at, int tokens) {   // token `at` of a segment's
    const int b = at >> shift(tokens);
    atomicOr(&bits[b >> 5], 1u << (b & 31));
  }
};

// What the dropped values add to a row, in 64 neighbouring columns: +inf (bit x of plus[i]: column
// 32 i + x), -inf, or NaN where both are.
struct NonFinite {
  uint32_t plus[2], minus[2];
  __device__ __forceinline__ float at(int c) const {
    const bool p = (plus[c >> 5] >> (c & 31)) & 1u, m = (minus[c >> 5] >> (c & 31)) & 1u;
    return p && m ? NAN : p ? INFINITY : m ? -INFINITY : 0.f;
  }
};

// By a converged warp, a lane per row r (`mine`: the row exists and has a sum): columns c0 ..
// c0 + nc - 1, at most 64.
template <typename E, int D>
__device__ __forceinline__ NonFinite non_finite(const AttnArgs& a, Part p, const Dropped& dropped,
                                             int r, bool mine, int c0, int nc) {
  constexpr int U = 4;   // tokens whose values are read at once
  const int lane = threadIdx.x & 31, cap = a.max_pages * a.page_size, shift = Dropped::shift(p.tok1 - p.tok0);
  const int last =
      mine ? last_token(a.pos, (int64_t)p.n * a.T + (p.row0 + r) / a.G, cap, nullptr) : -1;
  const int seen = __reduce_min_sync(0xffffffffu, seen_by_all(a, p, 32, lane));
  NonFinite f = {{0u, 0u}, {0u, 0u}};
  uint32_t word = 0;
  for (int w = 0; w < Dropped::kBuckets / 32 || word != 0;) {
    if (word == 0) {
      word = dropped.bits[w++];
      continue;
    }
    const int b = 32 * (w - 1) + __ffs(word) - 1;
    word &= word - 1u;
    const int end = p.tok0 + min((b + 1) << shift, p.tok1 - p.tok0);
    for (int s0 = max(p.tok0 + (b << shift), seen + 1); s0 < end; s0 += 32) {
      const int row = s0 + lane < end
                          ? cache_row(a.table + (int64_t)p.n * a.max_pages, s0 + lane, a.page_size,
                                      a.by_page, a.num_pages, nullptr)
                          : -1;
      const int n = min(32, end - s0);
      for (int j = 0; j < n; j += U) {
        float x[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int at = __shfl_sync(0xffffffffu, row, (j + u) & 31);
          const E* v = static_cast<const E*>(a.v) + ((int64_t)max(at, 0) * a.Hkv + p.hk) * D + c0;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            x[u][i] = j + u < n && at >= 0 && lane + 32 * i < nc ? to_f32(v[lane + 32 * i]) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t plus =
                __ballot_sync(0xffffffffu, isnan(x[u][i]) || x[u][i] == INFINITY);
            const uint32_t minus =
                __ballot_sync(0xffffffffu, isnan(x[u][i]) || x[u][i] == -INFINITY);
            if (s0 + j + u <= last) {
              f.plus[i] |= plus;
              f.minus[i] |= minus;
            }
          }
      }
    }
  }
  return f;
}

// The same, added to the half of row r that begins at column c0 and lies at `to`, of type E (narrow)
// or fp32.  Not inlined, as its code slows down short calls: 0.5 us of 10 us.
template <typename E, int D>
__device__ __noinline__ void add_non_finite(const AttnArgs& a, Part p, const Dropped& dropped, int r,
                                            bool mine, int c0, void* to, bool narrow) {
  const NonFinite f = non_finite<E, D>(a, p, dropped, r, mine, c0, D / 2);
  for (int c = 0; c < D / 2; ++c) {
    const float x = f.at(c);
    if (x == 0.f) continue;
    if (narrow) {
      E* y = static_cast<E*>(to) + c;
      *y = from_f32<E>(to_f32(*y) + x);
    } else {
      static_cast<float*>(to)[c] += x;
    }
  }
}

// The share of one CTA of NT threads in all items' units.  An item of u units costs kItemCost + u:
// the cost of starting on it (lookups, filling the ring) comes first.  Ranges of equal cost, one
// for each of the first nc groups of a.side CTAs, whose CTAs take a row block each: they read the
// same tokens at the same time, so that the second reads come from L2 (two blocks of 256 drafted
// rows over 32 x 32768 tokens: 542 MB of DRAM reads, 1085 MB when each block was an item of its
// own).
template <int RB, bool SEL, int UNIT, int NT>
struct Range {
  long long x, x1, total;   // position, end, sum of all costs
  int e, hk, at, nc;        // e: counts entries, or groups of a.side entries; at: from the start of
                            // the item (e, hk) to x
  int ntok;                 // tokens of e; -1: not looked up yet

  struct Shared {
    long long sum[NT / 32], off;
    int e, first, ntok[NT];
  };
  // A piece of one item: units uo .. uo + take - 1 of `units`.
  struct Segment {
    int e, hk, uo, take, units, ntok;
    int last_cta;   // of an item that starts here and ends in another CTA
  };

  static __device__ __forceinline__ int units_of(int ntok) {
    return max(1, (ntok + UNIT - 1) / UNIT);
  }
  // Sequence and queries of the entries of group e (prefix form).
  struct Queries {
    int n, t0, t1;
  };
  static __device__ __forceinline__ Queries queries_of(const AttnArgs& a, int e) {
    if (a.side > 1) return {e, 0, a.T - 1};
    const Entry<RB, SEL> en(a, e);
    return {en.n, en.row0 / a.G, (en.row0 + en.rows - 1) / a.G};
  }
  // Tokens that they walk over (a converged warp).
  static __device__ __forceinline__ int tokens_of(const AttnArgs& a, int e) {
    if (SEL) return a.topk;
    const Queries q = queries_of(a, e);
    return longest_warp(a, q.n, q.t0, q.t1);
  }
  // Cost of group e.
  static __device__ __forceinline__ long long cost_of(const AttnArgs& a, int ntok) {
    return (long long)(kItemCost + units_of(ntok)) * a.Hkv;
  }

  // Every thread of the CTA; false: no share.
  __device__ __forceinline__ bool cut(const AttnArgs& a, Shared& sh) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ne = (SEL ? a.nseq * a.T : a.nseq) * (a.nb / a.side);
    if (a.whole) {   // gridDim.x = side * entries * Hkv
      const int item = blockIdx.x / a.side;
      e = item / a.Hkv;
      ntok = tokens_of(a, e);
      total = x1 = kItemCost + units_of(ntok);
      hk = item - e * a.Hkv;
      at = 0;
      x = 0;
      nc = 1;
      return true;
    }
    const int chunk = (ne + NT - 1) / NT;   // entries of a thread
    const long long per = SEL ? cost_of(a, a.topk) : 0;
    long long mine = 0, before = 0, off;
    int tokens = 0;   // of this thread's last entry
    total = ne * per;
    if (!SEL) {
      // With few queries a thread reads its entries' positions, eight at once; with many the
      // warps read an entry's together, dealt out to all warps and four entries at once (a warp
      // that took its lanes' entries one by one spent 0.6 us on each: 20 us of 62 us for 32
      // sequences of 16 queries).
      const bool alone = a.T <= 8 || (chunk > 1 && a.T <= 32);
      for (int j = 0; j < chunk; ++j) {
        const int i = tid * chunk + j;
        if (alone) {
          if (i < ne) {
            const Queries q = queries_of(a, i);
            tokens = longest(a, q.n, q.t0, q.t1);
            mine += cost_of(a, tokens);
          }
          continue;
        }
        constexpr int W = NT / 32, U = 4;
        const int cap = a.max_pages * a.page_size;
        for (int k0 = warp; k0 < NT && k0 * chunk + j < ne; k0 += U * W) {
          int last[U];
          Queries q[U];
          int most = 0;
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int k = k0 + u * W, x = k * chunk + j;
            last[u] = -1;
            q[u] = {0, 0, -1};
            if (k < NT && x < ne) q[u] = queries_of(a, x);
            most = max(most, q[u].t1 - q[u].t0 + 1);
          }
          for (int t = lane; t < most; t += 32) {
            int p[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
              p[u] = q[u].t0 + t <= q[u].t1 ? a.pos[(int64_t)q[u].n * a.T + q[u].t0 + t] : -1;
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (p[u] < -1 || p[u] >= cap) set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
              last[u] = max(last[u], min(p[u], cap - 1));
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int k = k0 + u * W, most_u = __reduce_max_sync(0xffffffffu, last[u]) + 1;
            if (lane == 0 && k < NT) sh.ntok[k] = most_u;
          }
        }
        __syncthreads();
        tokens = sh.ntok[tid];
        if (i < ne) mine += cost_of(a, tokens);
        __syncthreads();
      }
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
    nc = (int)min((long long)(gridDim.x / a.side), total);
    const int cta = blockIdx.x / a.side;
    if (cta >= nc) return false;
    x = cta * total / nc;
    x1 = (cta + 1) * total / nc;
    if constexpr (SEL) {
      e = (int)(x / per);
      off = x - (long long)e * per;
      ntok = a.topk;
    } else {
      if (x >= before && x < before + mine) {
        off = x - before;
        e = tid * chunk;
        while (chunk > 1) {
          const Queries q = queries_of(a, e);
          tokens = longest(a, q.n, q.t0, q.t1);
          const long long n = cost_of(a, tokens);
          if (off < n) break;
          off -= n;
          ++e;
        }
        sh.e = e;
        sh.off = off;
        sh.first = tokens;
      }
      __syncthreads();
      e = sh.e;
      off = sh.off;
      ntok = sh.first;
    }
    const int cost = kItemCost + units_of(ntok);
    hk = (int)(off / cost);
    at = (int)(off - (long long)hk * cost);
    return true;
  }

  // The next piece that holds units; false: none.  By converged warps.
  __device__ __forceinline__ bool next(const AttnArgs& a, Segment& s) {
    while (x < x1) {
      const int block = blockIdx.x % a.side;
      if (ntok < 0) ntok = tokens_of(a, e);
      s.e = e * a.side + block;
      s.hk = hk;
      s.ntok = ntok;
      s.units = units_of(ntok);
      const int cost = kItemCost + s.units, go = (int)min((long long)(cost - at), x1 - x);
      s.uo = max(0, at - kItemCost);
      s.take = max(0, at + go - kItemCost) - s.uo;
      s.last_cta = 0;
      // position y of all costs lies in group floor(((y + 1) nc - 1) / total); y: the last unit
      if (s.uo == 0 && at + go < cost)
        s.last_cta = (int)(((x - at + cost) * nc - 1) / total) * a.side + block;
      x += go;
      at += go;
      if (at == cost) {
        at = 0;
        if (++hk == a.Hkv) {
          hk = 0;
          ++e;
          if (!SEL) ntok = -1;
        }
      }
      if (s.take > 0) return true;
    }
    return false;
  }
};

// Joins the partials of the items that several CTAs share, in CTA order: block (x, y) rows of the
// x-th item that starts in one CTA and ends in another.  A few KB per item, so latency-bound:
// every team of D / 4 threads reads up to kJoinBatch parts at once, and a row with more parts
// gets up to kJoinTeams teams.
constexpr int kJoinTeams = 8, kJoinBatch = 4;

template <typename E, int D, int RB, bool SEL>
__global__ void __launch_bounds__(kJoinTeams*(D / 4)) paged_join_kernel(const AttnArgs a) {
  constexpr int LANES = D / 4;
  __shared__ float4 s_acc[kJoinTeams][LANES];
  __shared__ float2 s_ml[kJoinTeams];
  __shared__ int s_count[kJoinTeams * LANES / 32], s_cta;
  pdl_prologue();
  const bool direct = (int)gridDim.x == a.ctas;   // a block for every CTA
  if (threadIdx.x == 0) s_cta = direct && a.split[blockIdx.x].x >= 0 ? (int)blockIdx.x : -1;
  if (direct) __syncthreads();
  for (int base = 0, before = 0; !direct && base < a.ctas; base += blockDim.x) {
    const int i = base + threadIdx.x;
    const bool starts = i < a.ctas && a.split[i].x >= 0;
    const uint32_t votes = __ballot_sync(0xffffffffu, starts);
    if ((threadIdx.x & 31) == 0) s_count[threadIdx.x >> 5] = __popc(votes);
    __syncthreads();
    int rank = before + __popc(votes & ((1u << (threadIdx.x & 31)) - 1u));
    for (int w = 0; w < kJoinTeams * LANES / 32; ++w) {
      if (w < (int)(threadIdx.x >> 5)) rank += s_count[w];
      before += s_count[w];
    }
    if (starts && rank == (int)blockIdx.x) s_cta = i;
    __syncthreads();
  }
  const int cta = s_cta;
  if (cta < 0) return;
  const int2 sp = a.split[cta];
  const int e = sp.x / a.Hkv, hk = sp.x - e * a.Hkv;
  const Entry<RB, SEL> en(a, e);
  const int team = threadIdx.x / LANES, lane = threadIdx.x - team * LANES, c = lane * 4;
  const int parts = (sp.y - cta) / a.side + 1;   // a.side CTAs apart
  const int groups = parts > 16 ? 8 : parts > 8 ? 4 : parts > 4 ? 2 : 1;   // teams of a row
  const int group = team % groups, rows = kJoinTeams / groups;
  for (int r0 = blockIdx.y * rows; r0 < en.rows; r0 += gridDim.y * rows) {
    const int r = r0 + team / groups;
    float mm = -INFINITY, ll = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // part 0 is slot 2 cta + 1, part k slot 2 (cta + k side); a team's are `groups` apart
    for (int k0 = group; r < en.rows && k0 < parts; k0 += groups * kJoinBatch) {
      float2 part[kJoinBatch];
      float4 vals[kJoinBatch];
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) {   // all reads at once
        const int k = k0 + i * groups, slot = k == 0 ? 2 * cta + 1 : 2 * (cta + k * a.side);
        part[i] = make_float2(-INFINITY, 0.f);
        vals[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k < parts) {
          part[i] = a.part_ml[slot * RB + r];
          vals[i] = *reinterpret_cast<const float4*>(a.part_o + ((int64_t)slot * RB + r) * D + c);
        }
      }
      float up = mm;
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) up = fmaxf(up, part[i].x);
      const float f = mm == up ? 1.f : exp2_approx(mm - up);   // 0 before the first part
      ll *= f;
      acc.x *= f;
      acc.y *= f;
      acc.z *= f;
      acc.w *= f;
      mm = up;
#pragma unroll
      for (int i = 0; i < kJoinBatch; ++i) add_part(acc, ll, mm, part[i].x, part[i].y, vals[i]);
    }
    if (groups > 1) {
      s_acc[team][lane] = acc;
      if (lane == 0) s_ml[team] = make_float2(mm, ll);
      __syncthreads();
      if (group == 0) {
        for (int g = 1; g < groups; ++g) mm = fmaxf(mm, s_ml[team + g].x);
        ll = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int g = 0; g < groups; ++g)
          add_part(acc, ll, mm, s_ml[team + g].x, s_ml[team + g].y, s_acc[team + g][lane]);
      }
      __syncthreads();
    }
    if (group == 0 && r < en.rows) finish<E, D>(a, en.n, en.row0 + r, hk, c, acc, mm, ll);
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
  a.nb = (attn_rows(p) + rb - 1) / rb;
  a.side = 1;
  a.whole = 0;
  a.wait_cycles = p.test_probe ? p.test_probe->wait_cycles : 4000000000LL;   // about 2 s
  a.skip_tile = p.test_probe ? p.test_probe->skip_tile : -1;
  return a;
}

template <typename E, int D, int RB, bool SEL>
cudaError_t launch_join(AttnArgs a, int ctas, int64_t items, int rows, cudaStream_t st) {
  a.ctas = ctas;
  // Few rows: a block for every CTA and row, most of which end at once.  Many rows: only blocks for
  // the items that can be split, which find theirs first (about 1 us); eight blocks an SM.
  int x = ctas, y = rows;
  if ((int64_t)x * y > 148 * 16) {
    if (items < ctas) x = (int)items;
    y = 148 * 8 / x;
    if (y > rows) y = rows;
  }
  return launch_pdl(paged_join_kernel<E, D, RB, SEL>, dim3(x, y),
                    dim3(kJoinTeams * (D / 4)), 0, st, a);
}

}  // namespace paged
}  // namespace misa

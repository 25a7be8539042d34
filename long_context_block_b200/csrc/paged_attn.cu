// K9: attention of new tokens over a paged key-value cache, the consumer of the indexer's
// token selection (Eqs. 2, 10): for query row (n, t) and head j,
//   z[s] = scale * q[j] . k[s],   out[j] = sum_s 2^((z[s] - m) log2 e) v[s] / sum_s 2^(...),
// over the query's prefix or over the tokens of its idx row.
//
// Memory-bound: a token costs 4 d bytes per key-value head and 4 d G flops (G query heads share
// it), far below the 250 flop/B at which this card's tensor cores would bound it.  So the kernel
// is built to keep bytes in flight: every warp owns a ring of key-value tiles in shared memory
// that it fills itself (cp.async, 16 bytes a lane) and reads itself, and no barrier stands in the
// loop.  A warp holds the item's up-to-16 MT query rows, so that the heads of a group (and the
// queries of a draft) share each loaded tile, and keeps the running maximum, sum and output in
// registers; the CTA's warps are joined at the end of a segment.
//
// Split, two ways:
//   - shared items (paged_attn_cluster_kernel): one thread-block cluster per item (row block x
//     key-value head) whose CTAs take equal parts of its tokens and join over distributed shared
//     memory: one launch, no scratch.
//   - equal ranges (paged_attn_kernel): the units (64 or 128 tokens) of all items are laid end to
//     end and cut into one equal range per CTA, whatever the lengths are.  An item that spans
//     CTAs leaves fp32 partials (at most two per CTA), joined by paged_join_kernel.
// Both join in a fixed order, so results do not depend on timing.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "misa.h"
#include "paged_attn.cuh"

namespace misa {
namespace {

using namespace paged;
namespace cg = cooperative_groups;

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;
// Two CTAs per SM (148 SMs): also what bounds the partials, so the workspace does not depend on
// the lengths.
constexpr int kMaxCtas = 296;
constexpr int kMaxCluster = 8;     // the largest portable cluster
// CTAs of larger clusters than pairs that are resident at once: a cluster stays within one group
// of SMs, which leaves 264 to 284 of the 296 places (cudaOccupancyMaxActiveClusters, sizes 3 - 8).
constexpr int kClusterCtas = 256;

template <int D, int MT>
struct Shape {
  static constexpr int RB = 16 * MT;      // query rows of an item
  static constexpr int KT = 2048 / D;     // tokens of a warp's tile
  static constexpr int UNIT = kWarps * KT;
  static constexpr int ROWB = D * 2;      // bytes of a key or value row
  static constexpr int CH = ROWB / 16;    // 16-byte chunks of a row
  static constexpr int TILE = KT * ROWB;  // bytes of a key (or value) tile
  static constexpr int RING = kWarps * kStages * 2 * TILE;
  static constexpr int OSTR = D + 8;      // row stride of the join buffer (no bank conflicts)
  static constexpr int SMEM = RING + RB * ROWB;
  static_assert(kWarps * RB * OSTR * 4 <= RING, "the join buffer lies in the ring");
};

// What the dropped values add, by the whole CTA: a warp takes a quarter of the columns of all rows,
// and a row's go to its part of the largest weights.  Not inlined: as add_non_finite.
template <typename E, int D, int RB, int OSTR>
__device__ __noinline__ void add_to_parts(const AttnArgs& a, Part p, const Dropped& dropped,
                                          float* s_o, const float2 (*s_ml)[RB]) {
  constexpr int C = D / kWarps;
  static_assert(C <= 32 && RB <= 32, "a lane per column, a lane per row");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const NonFinite f = non_finite<E, D>(a, p, dropped, lane, lane < p.rows, warp * C, C);
  for (int r = 0; r < p.rows; ++r) {
    NonFinite x = {};
    x.plus[0] = __shfl_sync(0xffffffffu, f.plus[0], r);
    x.minus[0] = __shfl_sync(0xffffffffu, f.minus[0], r);
    if (lane >= C || x.at(lane) == 0.f) continue;
    int w = 0;
    for (int y = 1; y < kWarps; ++y)
      if (s_ml[y][r].x > s_ml[w][r].x) w = y;
    s_o[(w * RB + r) * OSTR + warp * C + lane] += x.at(lane);
  }
}

// Tokens tok0 .. tok1 - 1 of entry `en` (of the prefix, or slots of its idx row) for key-value
// head hk, by the whole CTA.  Leaves each warp's part in shared memory: weighted values at
// smem (rows of OSTR floats, warp-major), maximum and sum in s_ml.
template <typename E, int D, int MT, bool SEL>
__device__ __forceinline__ void attend(const AttnArgs& a, const Entry<16 * MT, SEL>& en, int hk,
                                       int tok0, int tok1, unsigned char* smem,
                                       float2 (*s_ml)[16 * MT], Dropped& dropped) {   // cleared
  using S = Shape<D, MT>;
  constexpr int RB = S::RB, KT = S::KT, UNIT = S::UNIT, ROWB = S::ROWB, CH = S::CH,
                TILE = S::TILE;
  constexpr int NT = KT / 8;              // 8-token columns of a score tile
  constexpr int DN = D / 8;               // 8-wide columns of the output
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  unsigned char* s_q = smem + S::RING;
  const uint32_t ring = sm100::smem_u32(smem) + warp * (kStages * 2 * TILE);
  const uint32_t qbase = sm100::smem_u32(s_q);
  const int cap = a.max_pages * a.page_size;
  const int32_t* pages = a.table + (int64_t)en.n * a.max_pages;
  const int64_t sel_row = (int64_t)en.n * a.T + en.row0 / a.G;   // selected form: the query
  const int32_t* ids = SEL ? a.idx + sel_row * a.topk : nullptr;

  // ---- tile i of this warp starts at token tok0 + (i * kWarps + warp) * KT
  const int first = tok0 + warp * KT;
  const int ntile = first < tok1 ? (tok1 - first + UNIT - 1) / UNIT : 0;
  // What a lane looks up for its token of a tile is read ahead of its use, a tile per step:
  // the token id (selected form), then its page entry, then the copy.
  auto token = [&](int i) -> int {
    const int s = first + i * UNIT + lane;
    if (lane >= KT || i >= ntile || s >= tok1) return -1;
    return SEL ? __ldg(ids + s) : s;
  };
  int last_sel = -1;
  auto page_of = [&](int tok, int& page, int& in_page) {
    page = in_page = -1;
    if (SEL && (tok < -1 || tok > last_sel)) {
      set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
      tok = -1;
    }
    if (tok < 0) return;
    const int i = a.by_page(tok);
    page = __ldg(pages + i);
    in_page = tok - i * a.page_size;
  };
  const char* kb = static_cast<const char*>(a.k) + hk * ROWB + (lane % CH) * 16;
  const char* vb = static_cast<const char*>(a.v) + hk * ROWB + (lane % CH) * 16;
  const int64_t tstride = (int64_t)a.Hkv * ROWB;
  // copy the tile whose page entries the lanes hold; returns the tokens that are there
  auto issue = [&](int i, int page, int in_page) -> uint32_t {
    int row = -1;
    if (in_page >= 0) {
      if ((unsigned)page < (unsigned)a.num_pages)
        row = page * a.page_size + in_page;
      else
        set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
    }
    const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
    if (live) {
      const uint32_t dst = ring + (i % kStages) * (2 * TILE);
      constexpr int PER = 32 / CH;   // rows of one warp-wide copy
#pragma unroll
      for (int j = 0; j < KT / PER; ++j) {
        const int r = j * PER + lane / CH;
        const int src = __shfl_sync(0xffffffffu, row, r);
        const bool ok = src >= 0;
        const int64_t at = ok ? src * tstride : 0;
        const uint32_t d = dst + r * ROWB + (((lane % CH) ^ (r & 7)) << 4);
        cp_async16_or_zero(d, kb + at, ok);
        cp_async16_or_zero(d + TILE, vb + at, ok);
      }
    }
    cp_async_commit();
    return live;
  };
  // The first tiles' lookups go together, so that they cost one latency per step, not per tile.
  int tok[kStages];
#pragma unroll
  for (int i = 0; i < kStages; ++i) tok[i] = token(i);
  if (SEL) last_sel = last_token(a.pos, sel_row, cap, a.status);
  int pages_at[kStages], in_pages[kStages];
#pragma unroll
  for (int i = 0; i < kStages; ++i) page_of(tok[i], pages_at[i], in_pages[i]);
  int page = pages_at[kStages - 1], in_page = in_pages[kStages - 1], tok_next = token(kStages);
  uint32_t live[kStages];
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) live[i] = issue(i, pages_at[i], in_pages[i]);

  // ---- the query rows, zero behind the last one, while the first tiles are on their way
  {
    const E* q = static_cast<const E*>(a.q);
    for (int i = tid; i < RB * CH; i += kThreads) {
      const int r = i / CH, c = i - r * CH;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (r < en.rows) {
        const int rr = en.row0 + r, t = rr / a.G, g = rr - t * a.G;
        x = *reinterpret_cast<const uint4*>(
            q + (((int64_t)en.n * a.T + t) * a.Hq + hk * a.G + g) * D + c * 8);
        x.x = (x.x ^ a.q_flip) & a.q_keep;
        x.y = (x.y ^ a.q_flip) & a.q_keep;
        x.z = (x.z ^ a.q_flip) & a.q_keep;
        x.w = (x.w ^ a.q_flip) & a.q_keep;
      }
      *reinterpret_cast<uint4*>(s_q + r * ROWB + ((c ^ (r & 7)) << 4)) = x;
    }
  }
  // last visible token of this thread's rows
  int lim[2 * MT];
  int lim_min = cap, seen = cap;   // seen: of the rows that see tok0, the least
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    const int r = (lane >> 2) + 8 * i;
    lim[i] = cap;
    if (!SEL && r < en.rows) {
      lim[i] = last_token(a.pos, (int64_t)en.n * a.T + (en.row0 + r) / a.G, cap, nullptr);
      lim_min = min(lim_min, lim[i]);
      if (lim[i] >= tok0) seen = min(seen, lim[i]);
    }
  }
  if (!SEL) seen = __reduce_min_sync(0xffffffffu, seen);
  bool drop = false;   // NaN or infinite values were left out
  __syncthreads();

  float o[MT][DN][4];
  float m[2 * MT], l[2 * MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < DN; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[mt][i][x] = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  uint32_t qf[MT == 1 ? D / 16 : 1][4];
  const int arow = (lane & 7) + ((lane >> 3) & 1) * 8;
  if constexpr (MT == 1) {
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      ldmatrix4(qf[kk], qbase + arow * ROWB + (((2 * kk + (lane >> 4)) ^ (lane & 7)) << 4));
  }

  for (int i = 0; i < ntile; ++i) {
    cp_async_wait<kStages - 2>();
    __syncwarp();
    live[kStages - 1] = issue(i + kStages - 1, page, in_page);
    page_of(tok_next, page, in_page);
    tok_next = token(i + kStages + 1);
    const uint32_t ok = live[0];
#pragma unroll
    for (int j = 0; j + 1 < kStages; ++j) live[j] = live[j + 1];
    if (ok == 0) continue;
    const uint32_t kt = ring + (i % kStages) * (2 * TILE), vt = kt + TILE;

    float s[MT][NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < NT; ++x) s[mt][x][0] = s[mt][x][1] = s[mt][x][2] = s[mt][x][3] = 0.f;
    const int brow = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t qa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if constexpr (MT == 1) {
#pragma unroll
          for (int x = 0; x < 4; ++x) qa[mt][x] = qf[kk][x];
        } else {
          ldmatrix4(qa[mt], qbase + (mt * 16 + arow) * ROWB +
                                (((2 * kk + (lane >> 4)) ^ (lane & 7)) << 4));
        }
      }
#pragma unroll
      for (int p = 0; p < NT / 2; ++p) {
        uint32_t b[4];
        ldmatrix4(b, kt + (p * 16 + brow) * ROWB +
                         (((2 * kk + ((lane >> 3) & 1)) ^ (lane & 7)) << 4));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816<E>(s[mt][2 * p], qa[mt], b[0], b[1]);
          mma16816<E>(s[mt][2 * p + 1], qa[mt], b[2], b[3]);
        }
      }
    }

    // what a row does not see is -inf
    const int s0 = first + i * UNIT;
    const uint32_t full = KT == 32 ? 0xffffffffu : (1u << KT) - 1u;
    if (!SEL && min(s0 + KT, tok1) - 1 > seen) {   // values of tokens that some rows do not see
      for (int r = max(seen + 1 - s0, 0) + lane / CH; r < min(KT, tok1 - s0); r += 32 / CH) {
        uint4* at = reinterpret_cast<uint4*>(smem + (vt - sm100::smem_u32(smem)) + r * ROWB +
                                             (((lane % CH) ^ (r & 7)) << 4));
        uint4 x = *at;
        if (drop_non_finite<E>(x)) {
          *at = x;
          dropped.add(s0 + r - tok0, tok1 - tok0);
          drop = true;
        }
      }
      __syncwarp();
    }
    if (ok != full || (!SEL && s0 + KT - 1 > lim_min)) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int c = x * 8 + (lane & 3) * 2 + (y & 1);
            const bool see = ((ok >> c) & 1u) && (SEL || s0 + c <= lim[2 * mt + (y >> 1)]);
            if (!see) s[mt][x][y] = -INFINITY;
          }
    }
    // the running maximum is kept in the log2 domain: m = max of the scores * scale2 (> 0), in fp16
    // less the exponent that the largest weight gets
    float mx[2 * MT];
    bool up = false;
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {
      float t = -INFINITY;
#pragma unroll
      for (int x = 0; x < NT; ++x)
        t = fmaxf(t, fmaxf(s[r >> 1][x][(r & 1) * 2], s[r >> 1][x][(r & 1) * 2 + 1]));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
      t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
      mx[r] = fmaxf(m[r], Weights<E>::reference(t, a.scale2, Weights<E>::kTop));
      up |= mx[r] > m[r];
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) {
        const float f = mx[r] == m[r] ? 1.f : exp2_approx(m[r] - mx[r]);
        m[r] = mx[r];
        l[r] *= f;
#pragma unroll
        for (int x = 0; x < DN; ++x) {
          o[r >> 1][x][(r & 1) * 2] *= f;
          o[r >> 1][x][(r & 1) * 2 + 1] *= f;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {
      const float base = m[r] == -INFINITY ? 0.f : -m[r];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float& p = s[r >> 1][x][(r & 1) * 2 + y];
          p = exp2_approx(fmaf(p, a.scale2, base));
          l[r] += p;
        }
    }
    const int vrow = (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
    for (int ks = 0; ks < NT / 2; ++ks) {
      uint32_t pa[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        pa[mt][0] = pack2<E>(s[mt][2 * ks][0], s[mt][2 * ks][1]);
        pa[mt][1] = pack2<E>(s[mt][2 * ks][2], s[mt][2 * ks][3]);
        pa[mt][2] = pack2<E>(s[mt][2 * ks + 1][0], s[mt][2 * ks + 1][1]);
        pa[mt][3] = pack2<E>(s[mt][2 * ks + 1][2], s[mt][2 * ks + 1][3]);
      }
#pragma unroll
      for (int p = 0; p < DN / 2; ++p) {
        uint32_t b[4];
        ldmatrix4_trans(b, vt + (ks * 16 + vrow) * ROWB +
                               (((2 * p + (lane >> 4)) ^ (lane & 7)) << 4));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma16816<E>(o[mt][2 * p], pa[mt], b[0], b[1]);
          mma16816<E>(o[mt][2 * p + 1], pa[mt], b[2], b[3]);
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();   // every warp is done with its ring

  float* s_o = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int r = 0; r < 2 * MT; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    const int row = (lane >> 2) + 8 * r;
    if ((lane & 3) == 0) s_ml[warp][row] = make_float2(m[r], l[r]);
#pragma unroll
    for (int x = 0; x < DN; ++x)
      *reinterpret_cast<float2*>(s_o + (warp * RB + row) * S::OSTR + x * 8 + (lane & 3) * 2) =
          make_float2(o[r >> 1][x][(r & 1) * 2], o[r >> 1][x][(r & 1) * 2 + 1]);
  }
  if (SEL) {
    __syncthreads();
  } else if (__syncthreads_or(drop)) {
    add_to_parts<E, D, RB, S::OSTR>(a, {en.n, en.row0, en.rows, hk, tok0, tok1}, dropped, s_o, s_ml);
    __syncthreads();
    dropped.clear(tid);
  }
}

// The CTA's sum over its warps at row r, elements c .. c + 3.
template <int D, int MT>
__device__ __forceinline__ float4 warp_sum(const unsigned char* smem,
                                           const float2 (*s_ml)[16 * MT], int r, int c, float& mm,
                                           float& ll) {
  using S = Shape<D, MT>;
  const float* s_o = reinterpret_cast<const float*>(smem);
  mm = -INFINITY;
  ll = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_ml[w][r].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w)
    add_part(acc, ll, mm, s_ml[w][r].x, s_ml[w][r].y,
             *reinterpret_cast<const float4*>(s_o + (w * S::RB + r) * S::OSTR + c));
  return acc;
}

template <typename E, int D, int MT, bool SEL>
__global__ void __launch_bounds__(kThreads, 2)
paged_attn_cluster_kernel(const __grid_constant__ AttnArgs a) {
  using S = Shape<D, MT>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float2 s_ml[kWarps][S::RB];
  __shared__ float2 s_part[S::RB];
  __shared__ Dropped s_dropped;
  if (!SEL) s_dropped.clear(threadIdx.x);
  pdl_prologue();
  cg::cluster_group cluster = cg::this_cluster();
  const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int item = blockIdx.x / size, hk = item % a.Hkv;
  const Entry<S::RB, SEL> en(a, item / a.Hkv);
  const int ntok = en.tokens(a);
  const int64_t units = (ntok + S::UNIT - 1) / S::UNIT;
  const int tok0 = (int)(rank * units / size) * S::UNIT;
  const int tok1 = min(ntok, (int)((rank + 1) * units / size) * S::UNIT);
  attend<E, D, MT, SEL>(a, en, hk, tok0, tok1, smem, s_ml, s_dropped);
  float* s_o = reinterpret_cast<float*>(smem);
  const int work = en.rows * (D / 4);
  if (size > 1) {   // this CTA's sum takes the place of its first warp's part
    for (int i = threadIdx.x; i < work; i += kThreads) {
      const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
      float mm, ll;
      const float4 acc = warp_sum<D, MT>(smem, s_ml, r, c, mm, ll);
      *reinterpret_cast<float4*>(s_o + r * S::OSTR + c) = acc;
      if (c == 0) s_part[r] = make_float2(mm, ll);
    }
    cluster.sync();
  }
  for (int i = rank * kThreads + threadIdx.x; i < work; i += size * kThreads) {
    const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
    float mm = -INFINITY, ll = 0.f;
    float4 acc;
    if (size > 1) {
      float2 ml[kMaxCluster];
      float4 x[kMaxCluster];
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)   // all reads at once
        if (p < size) {
          ml[p] = cluster.map_shared_rank(s_part, p)[r];
          x[p] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(s_o, p) + r * S::OSTR + c);
        }
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)
        if (p < size) mm = fmaxf(mm, ml[p].x);
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < kMaxCluster; ++p)
        if (p < size) add_part(acc, ll, mm, ml[p].x, ml[p].y, x[p]);
    } else {
      acc = warp_sum<D, MT>(smem, s_ml, r, c, mm, ll);
    }
    finish<E, D>(a, en.n, en.row0 + r, hk, c, acc, mm, ll);
  }
  if (size > 1) cluster.sync();   // no CTA leaves while another reads its shared memory
}

template <typename E, int D, int MT, bool SEL>
__global__ void __launch_bounds__(kThreads, 2)
paged_attn_kernel(const __grid_constant__ AttnArgs a) {
  using S = Shape<D, MT>;
  constexpr int RB = S::RB, UNIT = S::UNIT;
  using R = Range<RB, SEL, UNIT, kThreads>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ float2 s_ml[kWarps][RB];
  __shared__ typename R::Shared s_range;
  __shared__ Dropped s_dropped;
  const int cta = blockIdx.x;
  if (!SEL) s_dropped.clear(threadIdx.x);
  pdl_prologue();
  R range;
  typename R::Segment sg;
  int2 split = make_int2(-1, 0);
  if (range.cut(a, s_range))
    while (range.next(a, sg)) {
      const Entry<RB, SEL> en(a, sg.e);
      const int hk = sg.hk, tok0 = sg.uo * UNIT;
      const int tok1 = min(sg.ntok, (sg.uo + sg.take) * UNIT);
      attend<E, D, MT, SEL>(a, en, hk, tok0, tok1, smem, s_ml, s_dropped);
      const bool whole = sg.take == sg.units;
      const int slot = 2 * cta + (sg.uo == 0 ? 1 : 0);
      for (int i = threadIdx.x; i < en.rows * (D / 4); i += kThreads) {
        const int r = i / (D / 4), c = (i - r * (D / 4)) * 4;
        float mm, ll;
        const float4 acc = warp_sum<D, MT>(smem, s_ml, r, c, mm, ll);
        if (whole) {
          finish<E, D>(a, en.n, en.row0 + r, hk, c, acc, mm, ll);
        } else {
          *reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * RB + r) * D + c) = acc;
          if (c == 0) a.part_ml[slot * RB + r] = make_float2(mm, ll);
        }
      }
      __syncthreads();   // the buffers are free for the next segment
      if (!whole && sg.uo == 0) split = make_int2(sg.e * a.Hkv + hk, sg.last_cta);
    }
  if (threadIdx.x == 0) a.split[cta] = split;
}

// CTAs that share an item: 0 for equal ranges.  The longest item there can be decides, as the
// lengths are known on the device only: one sequence of 777 tokens takes 6.2 us under a table of its
// own width, 9.0 us under one for 131072 tokens.
//   Time of a unit (32 KB) per CTA: 1.48 us where all 296 CTAs stream (the memory's rate), 0.9 us
//   where few do (latency).  Shared items pay full waves of CTAs and a last, partial one; equal
//   ranges pay the average and about 3 us for the join: 64 items of 2048 selected tokens 17.7
//   against 20.7 us, 360 items (two waves, the second a fifth full) 84 against 72 us.
//   In the prefix form the lengths may differ, and a long sequence among short ones keeps its
//   cluster alone, so 16 units a CTA are the most: 8 sequences of up to 4096 tokens (16 units) 25.4
//   against 29.4 us when equally long and 19.8 against 17.0 us when ragged, of up to 8192 (32
//   units) 44.0 against 49.3 and 32.1 against 19.7 us.
int cluster_size(const PagedAttn& p) {
  const int rows = attn_rows(p), rb = rows > 16 ? 32 : 16, unit = kWarps * (2048 / p.d);
  const int64_t items =
      (int64_t)p.nseq * (p.topk > 0 ? p.T : 1) * ((rows + rb - 1) / rb) * p.Hkv;
  const int64_t span = p.topk > 0 ? p.topk : (int64_t)p.max_pages * p.page_size;
  const int64_t units = (span + unit - 1) / unit;
  int64_t c = (2 * items > kClusterCtas ? kMaxCtas : kClusterCtas) / items;
  if (c > kMaxCluster) c = kMaxCluster;
  if (c > units) c = units;
  if (c < 1) c = 1;
  const int64_t steps = (units + c - 1) / c;   // units of a CTA
  if (p.topk == 0 && steps > 16) return 0;
  const int64_t full = items * c / kMaxCtas, rest = items * c % kMaxCtas;
  const double last = rest == 0 ? 0.0 : std::fmax(0.9, 1.48 * rest / kMaxCtas);
  const double shared = (double)steps * (1.48 * full + last);
  const double ranges = (double)items * units * 1.48 / kMaxCtas + 3.0;
  return shared <= ranges ? (int)c : 0;
}

// Whether the tensor-core form (paged_attn_tc.cu) runs: for more rows on a token than a warp
// holds, but for little work the clusters of this file are quicker, as they need no join.  Measured
// at 64 rows, clusters against tensor cores.  Units of a cluster's CTA: 4 (32 sequences of 1024
// tokens, one key-value head) 15.3 against 18.2 us, (8 x 2048 selected tokens) 13.6 against 14.5 us;
// 8 (one sequence of 4096 tokens, 8 key-value heads) 19.9 against 16.4 us, (32 x 2048 selected)
// 21.5 against 19.7 us, (8 sequences of 1024 tokens, 8 heads) 23.5 against 23.8 us.  Units in all:
// 8192 (8 sequences of 4096 tokens, 8 heads) 66.6 against 39.2 us.  Up to four tiles an item stays
// with one CTA, without a join, and 512 units are enough: 8 sequences of 256 tokens 15.6 against
// 11.6 us.
bool use_tc(const PagedAttn& p) {
  const int rows = attn_rows(p);
  if (rows <= 32) return false;
  const int64_t heads = (int64_t)p.nseq * (p.topk > 0 ? p.T : 1) * p.Hkv;
  const int64_t span = p.topk > 0 ? p.topk : (int64_t)p.max_pages * p.page_size;
  const int64_t unit = kWarps * (2048 / p.d);
  const int64_t units = (span + unit - 1) / unit, work = heads * ((rows + 31) / 32) * units;
  const int64_t tiles = (span + 127) / 128;
  if (tiles == 1) return true;
  if (tiles <= 4 && heads * ((rows + 127) / 128) <= 148) return work >= 512;
  const int c = cluster_size(p);
  return c == 0 || work > 2048 || (units + c - 1) / c >= 8;
}

template <typename E, int D, int MT, bool SEL>
cudaError_t launch_variant(const PagedAttn& p, AttnArgs a, cudaStream_t st) {
  using S = Shape<D, MT>;
  const int rows = attn_rows(p);
  const int64_t items = (int64_t)p.nseq * (SEL ? p.T : 1) * a.nb * p.Hkv;
  const int size = cluster_size(p);
  const auto kernel =
      size ? paged_attn_cluster_kernel<E, D, MT, SEL> : paged_attn_kernel<E, D, MT, SEL>;
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (err != cudaSuccess) return err;
  if (size) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * size));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = S::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
  }
  const int64_t span = SEL ? p.topk : (int64_t)p.max_pages * p.page_size;
  const int64_t units = (span + S::UNIT - 1) / S::UNIT;   // of the longest item there can be
  const int grid = (int)(items * units < kMaxCtas ? items * units : kMaxCtas);
  err = launch_pdl(kernel, dim3(grid), dim3(kThreads), S::SMEM, st, a);
  if (err != cudaSuccess || units == 1) return err;
  return launch_join<E, D, S::RB, SEL>(a, grid, items, rows < S::RB ? rows : S::RB, st);
}

template <typename E, int D>
cudaError_t launch_type(const PagedAttn& p, const AttnArgs& a, cudaStream_t st) {
  const bool two = attn_rows(p) > 16;
  if (p.topk > 0)
    return two ? launch_variant<E, D, 2, true>(p, a, st) : launch_variant<E, D, 1, true>(p, a, st);
  return two ? launch_variant<E, D, 2, false>(p, a, st) : launch_variant<E, D, 1, false>(p, a, st);
}

}  // namespace

bool paged_attn_tc(const PagedAttn& p) { return use_tc(p); }

size_t paged_attn_ws_bytes(const PagedAttn& p) {
  if (use_tc(p)) return paged_attn_tc_ws_bytes(p);
  if (cluster_size(p)) return 0;
  return attn_ws_bytes(kMaxCtas, attn_rows(p) > 16 ? 32 : 16, p.d);
}

cudaError_t launch_paged_attn(const PagedAttn& p, void* scratch, int* status, cudaStream_t st) {
  if (use_tc(p)) return launch_paged_attn_tc(p, scratch, status, st);
  const AttnArgs a = attn_args(p, scratch, kMaxCtas, attn_rows(p) > 16 ? 32 : 16, status);
  if (p.dtype == MISA_DTYPE_BF16)
    return p.d == 128 ? launch_type<__nv_bfloat16, 128>(p, a, st)
                      : launch_type<__nv_bfloat16, 64>(p, a, st);
  return p.d == 128 ? launch_type<__half, 128>(p, a, st) : launch_type<__half, 64>(p, a, st);
}

}  // namespace misa

// K9 for many query rows per key-value head: the paged attention on the fifth-generation tensor
// cores.  Drafts of several tokens, wide groups and single key-value heads put more than 32 rows
// (queries x heads of a group) on each loaded token, where warp-level matrix steps bound the
// kernel (about 190 TFLOP/s).
//
// One CTA per SM, roles by warp:
//   warps 0 - 7   two threads per query row, half of a tile's tokens each: scores from tensor
//                 memory, running maximum and sum, weights to shared memory as the second
//                 product's operand; the output at the end
//   warps 8 - 11  gather the tiles (128 tokens): page entries, then keys and values with 16-byte
//                 asynchronous copies into the 128-byte-swizzled operand layout
//   warp 12       one thread issues the products: S = Q K^T (two buffers, so that the next tile's
//                 scores are made while this one's weights are) and O += P V, both with fp32 sums
//                 in tensor memory
// The running maximum moves only when a row's scores exceed it by more than 2^8, so that O, which
// stays in tensor memory, is rescaled a few times per item at most; any reference gives the same
// quotient.  Ranges and partials as in paged_attn.cu.  All waits are bounded; where one runs out
// the CTA reports MISA_ERR_DEVICE_TIMEOUT, lets its copies and products end and frees its tensor
// memory.
#include <cuda_runtime.h>

#include <climits>

#include "internal.h"
#include "misa.h"
#include "paged_attn.cuh"

namespace misa {
namespace {

using namespace paged;
using namespace sm100;

constexpr int kRows = 128;       // query rows of an item
constexpr int kTile = 128;       // tokens of a tile
constexpr int kSoftWarps = 8, kLoadWarps = 4;
constexpr int kCols = kTile / 2;   // tokens of a tile that a thread has the weights of
constexpr int kThreads = 32 * (kSoftWarps + kLoadWarps + 1);
constexpr int kTcCtas = 148;     // one per SM
constexpr int kLiveDepth = 8;
constexpr long long kWaitCycles = 4000000000LL;   // about 2 s at the top SM clock
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 2 * kTile;            // S at columns 0 and 128

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                 // operand tiles are 64 columns wide
  static constexpr int kHalf = 128 * 128;                // 128 rows of 128 bytes
  static constexpr int kTileBytes = kHalves * kHalf;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kQ = kV + kStages * kTileBytes;
  static constexpr int kP = kQ + kTileBytes;             // 128 rows x 128 tokens
  static constexpr int kLive = kP + 2 * kHalf;           // [kLiveDepth][4] words
  static constexpr int kBars = kLive + kLiveDepth * 16;
  // kfull, kfree, vfull, vfree [kStages], sfull, sfree [2], pfull, odone, qfull, drain,
  // live [kLiveDepth], pair [4]
  static constexpr int kNumBars = 4 * kStages + 4 + 4 + kLiveDepth + 4;
  static constexpr int kBytes = kBars + kNumBars * 8 + 1024;   // 1 KB alignment of the base
  static_assert(kBytes <= 227 * 1024, "shared memory");
};

// Descriptor of an operand whose 128-byte rows run along its M or N dimension (V: a row per token,
// the token is the reduced dimension), 128-byte swizzle: groups of 8 rows 1024 bytes apart,
// further 64 columns `cols64` bytes away.
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t addr, uint32_t cols64) {
  uint64_t d = 0;
  d |= (uint64_t)((addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(cols64 >> 4) << 16;              // leading byte offset
  d |= (uint64_t)(1024u >> 4) << 32;               // stride byte offset
  d |= (uint64_t)1 << 46;                          // descriptor version for sm_100
  d |= (uint64_t)2 << 61;                          // swizzle mode: 128-byte
  return d;
}

// Instruction descriptor of kind::f16, fp32 sums; b_mn: B's rows run along N.
template <typename E>
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N, bool b_mn) {
  const uint32_t type = sizeof(E) == 2 && IsBf16<E>::value ? 1u : 0u;
  return (1u << 4) | (type << 7) | (type << 10) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

#define MISA_R32(r)                                                                         \
  r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7], r[8], r[9], r[10], r[11], r[12], r[13],   \
      r[14], r[15], r[16], r[17], r[18], r[19], r[20], r[21], r[22], r[23], r[24], r[25],   \
      r[26], r[27], r[28], r[29], r[30], r[31]

// 32 fp32 columns of the warp's 32 tensor-memory lanes, a lane per thread; the wait comes apart,
// so that several loads are in flight.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// Waits for the thread's tensor-memory loads; the values pass through, so that no use of them
// moves before the wait.
__device__ __forceinline__ void tmem_ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"f"(
          v[0]),
      "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
      "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
      "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]),
      "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]),
      "f"(v[30]), "f"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Weights rise above 1 up to this factor (log2) before the running maximum follows.
constexpr float kSlack = 8.f;

template <typename E, int D, bool SEL>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_tc_kernel(const AttnArgs a) {
  using C = Cfg<D>;
  using R = Range<kRows, SEL, kTile, kThreads>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ typename R::Shared s_range;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float s_pair[2][2][kRows];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t *kfull = bars, *kfree = kfull + C::kStages, *vfull = kfree + C::kStages,
           *vfree = vfull + C::kStages, *sfull = vfree + C::kStages, *sfree = sfull + 2,
           *pfull = sfree + 2, *odone = pfull + 1, *qfull = odone + 1, *drain = qfull + 1,
           *live = drain + 1, *pair = live + kLiveDepth;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  volatile int* abort_flag = &s_abort;

  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&kfull[i], 32 * kLoadWarps);
      mbar_init(&kfree[i], 1);
      mbar_init(&vfull[i], 32 * kLoadWarps);
      mbar_init(&vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], 32 * kSoftWarps);
    }
    mbar_init(pfull, 32 * kSoftWarps);
    mbar_init(odone, 1);
    mbar_init(qfull, 32 * kSoftWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < kLiveDepth; ++i) mbar_init(&live[i], kLoadWarps);
    for (int i = 0; i < 4; ++i) mbar_init(&pair[i], 2);
    fence_barrier_init();
  }
  if (warp == kSoftWarps + kLoadWarps) tmem_alloc(&s_tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  pdl_prologue();

  R range;
  typename R::Segment sg;
  const bool share = range.cut(a, s_range);
  int2 split = make_int2(-1, 0);
  auto wait = [&](uint64_t* bar, int phase) {
    return mbar_wait(bar, phase & 1, abort_flag, a.status, kWaitCycles);
  };
  // a whole warp's wait: lane 0 polls, all lanes agree on the outcome
  auto warp_wait = [&](uint64_t* bar, int phase) {
    int r = 1;
    if (lane == 0) r = wait(bar, phase);
    r = __shfl_sync(0xffffffffu, r, 0);
    __syncwarp();
    return r != 0;
  };
  int g = 0;        // tiles before this segment, in every role
  bool ok = true;

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------ scores to weights, output
    // Warps w and w + 4 have the same rows (a warp reaches the 32 tensor-memory lanes of its
    // number modulo 4) and each half of the columns.
    const int row = tid % kRows, half = warp / 4, quad = warp % 4;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    int swaps = 0;
    // max or sum over the row's two threads; x of the partner, or false
    auto swap = [&](float x, float& other) {
      float(*buf)[kRows] = s_pair[swaps & 1];
      buf[half][row] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pair[quad]);
      if (!warp_wait(&pair[quad], swaps++)) return false;
      other = buf[half ^ 1][row];
      return true;
    };
    while (share && ok && range.next(a, sg)) {
      const Entry<kRows, SEL> en(a, sg.e);
      const int tok0 = sg.uo * kTile, tok1 = min(sg.ntok, (sg.uo + sg.take) * kTile);
      const int n = (tok1 - tok0 + kTile - 1) / kTile;
      const bool mine = row < en.rows, warp_live = quad * 32 < en.rows;
      const int rr = en.row0 + row, t = mine ? rr / a.G : 0;
      float m = -INFINITY, l = 0.f;
      if (n > 0) {
        // the row of Q; the products of the segment before have ended (their scores are here)
        const uint4* q = reinterpret_cast<const uint4*>(
            static_cast<const E*>(a.q) +
            (((int64_t)en.n * a.T + t) * a.Hq + sg.hk * a.G + (rr - t * a.G)) * D);
        unsigned char* dst = smem + C::kQ + row * 128;
#pragma unroll
        for (int c0 = 0; c0 < D / 16; ++c0) {
          const int c = half * (D / 16) + c0;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (mine) {
            x = q[c];
            x.x = (x.x ^ a.q_flip) & a.q_keep;
            x.y = (x.y ^ a.q_flip) & a.q_keep;
            x.z = (x.z ^ a.q_flip) & a.q_keep;
            x.w = (x.w ^ a.q_flip) & a.q_keep;
          }
          *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kHalf + (((c & 7) ^ (row & 7)) << 4)) = x;
        }
        fence_proxy_async_smem();
        mbar_arrive(qfull);
      }
      int lim = INT_MAX;
      if (!SEL && mine)
        lim = last_token(a.pos, (int64_t)en.n * a.T + t, a.max_pages * a.page_size, nullptr);
      for (int i = 0; i < n; ++i) {
        const int gi = g + i, buf = gi & 1;
        if (!(ok = warp_wait(&sfull[buf], gi >> 1))) break;
        tc_fence_after();
        float s[kCols];
        if (warp_live) {
#pragma unroll
          for (int c = 0; c < kCols; c += 32)
            tmem_ld32(lanes + buf * kTile + half * kCols + c, s + c);
#pragma unroll
          for (int c = 0; c < kCols; c += 32) tmem_ld_wait(s + c);
        }
        if (!(ok = warp_wait(&live[gi % kLiveDepth], gi / kLiveDepth))) break;
        const uint2 there = *reinterpret_cast<const uint2*>(smem + C::kLive +
                                                            (gi % kLiveDepth) * 16 + half * 8);
        tc_fence_before();
        mbar_arrive(&sfree[buf]);
        if (warp_live) {
          const int s0 = tok0 + i * kTile + half * kCols;
          if ((there.x & there.y) != 0xffffffffu || (!SEL && s0 + kCols - 1 > lim)) {
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (!(((c < 32 ? there.x : there.y) >> (c & 31)) & 1u) || (!SEL && s0 + c > lim))
                s[c] = -INFINITY;
          }
          float mx[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) mx[c] = s[c];
#pragma unroll
          for (int c = 4; c < kCols; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
          float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2, other;
          if (!(ok = swap(top, other))) break;
          top = fmaxf(top, other);
          if (__any_sync(0xffffffffu, top > m + kSlack)) {
            const float up = fmaxf(m, top), f = up == m ? 1.f : exp2_approx(m - up);
            m = up;
            l *= f;
            if (i > 0) {
              if (!(ok = warp_wait(odone, gi - 1))) break;
              tc_fence_after();
#pragma unroll 1
              for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
                float o[32];
                tmem_ld32(lanes + kTmemO + c, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= f;
                tmem_st32(lanes + kTmemO + c, o);
              }
              tmem_st_wait();
            }
          }
          const float base = m == -INFINITY ? 0.f : -m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            s[c] = exp2_approx(fmaf(s[c], a.scale2, base));
            sum[c & 3] += s[c];
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        }
        // the weights' buffer is free once the product before has ended
        if (i > 0 && !(ok = warp_wait(odone, gi - 1))) break;
        if (warp_live) {
          unsigned char* dst = smem + C::kP + half * C::kHalf + row * 128;
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c) {
            const float* p = s + c * 8;
            *reinterpret_cast<uint4*>(dst + ((c ^ (row & 7)) << 4)) =
                make_uint4(pack2<E>(p[0], p[1]), pack2<E>(p[2], p[3]), pack2<E>(p[4], p[5]),
                           pack2<E>(p[6], p[7]));
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(pfull);
      }
      if (!ok) break;
      if (n > 0 && !(ok = warp_wait(odone, g + n - 1))) break;
      tc_fence_after();
      const bool whole = sg.take == sg.units;
      const int slot = 2 * cta + (sg.uo == 0 ? 1 : 0);
      if (warp_live) {
        float other;
        if (!(ok = swap(l, other))) break;
        l += other;
        const int gq = rr - t * a.G;
        const int64_t head = ((int64_t)en.n * a.T + t) * a.Hq + sg.hk * a.G + gq;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
        for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 32) {
          float o[32];
          __syncwarp();
          if (n > 0) {
            tmem_ld32(lanes + kTmemO + c, o);
            tmem_ld_wait(o);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0.f;
          }
          if (mine && whole) {
            uint4* to = reinterpret_cast<uint4*>(static_cast<E*>(a.out) + head * D + c);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const float* p = o + x * 8;
              to[x] = make_uint4(pack2<E>(p[0] * inv, p[1] * inv), pack2<E>(p[2] * inv, p[3] * inv),
                                 pack2<E>(p[4] * inv, p[5] * inv), pack2<E>(p[6] * inv, p[7] * inv));
            }
          } else if (mine) {
            float4* to =
                reinterpret_cast<float4*>(a.part_o + ((int64_t)slot * kRows + row) * D + c);
#pragma unroll
            for (int x = 0; x < 8; ++x)
              to[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        }
        if (mine && half == 0) {
          if (!whole)
            a.part_ml[slot * kRows + row] = make_float2(m, l);
          else if (a.lse)
            a.lse[head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      tc_fence_before();   // the loads of O come before the next segment's products
      if (!whole && sg.uo == 0) split = make_int2(sg.e * a.Hkv + sg.hk, sg.last_cta);
      g += n;
    }
  } else if (warp < kSoftWarps + kLoadWarps) {
    // ------------------------------------------------------------ tiles
    const int w = warp - kSoftWarps;
    constexpr int CH = D / 8, PER = 32 / CH;   // 16-byte chunks of a row, rows of a warp-wide copy
    const int c = lane % CH;
    const uint32_t smem0 = smem_u32(smem) + (c >> 3) * C::kHalf;
    const int cap = a.max_pages * a.page_size;
    while (share && ok && range.next(a, sg)) {
      const Entry<kRows, SEL> en(a, sg.e);
      const int tok0 = sg.uo * kTile, tok1 = min(sg.ntok, (sg.uo + sg.take) * kTile);
      const int n = (tok1 - tok0 + kTile - 1) / kTile;
      const int32_t* pages = a.table + (int64_t)en.n * a.max_pages;
      const int64_t sel_row = (int64_t)en.n * a.T + en.row0 / a.G;
      const int32_t* ids = SEL ? a.idx + sel_row * a.topk : nullptr;
      auto token = [&](int i) -> int {
        const int s = tok0 + i * kTile + w * 32 + lane;
        if (i >= n || s >= tok1) return -1;
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
        const int p = a.by_page(tok);
        page = __ldg(pages + p);
        in_page = tok - p * a.page_size;
      };
      const char* kb = static_cast<const char*>(a.k) + (int64_t)sg.hk * (D * 2) + c * 16;
      const char* vb = static_cast<const char*>(a.v) + (int64_t)sg.hk * (D * 2) + c * 16;
      const int64_t tstride = (int64_t)a.Hkv * (D * 2);
      const int tok_a = token(0);
      int tok_b = token(1), page, in_page;
      if (SEL) last_sel = last_token(a.pos, sel_row, cap, a.status);
      page_of(tok_a, page, in_page);
      for (int i = 0; i < n; ++i) {
        const int gi = g + i, st = gi % C::kStages, ph = gi / C::kStages;
        int src = -1;
        if (in_page >= 0) {
          if ((unsigned)page < (unsigned)a.num_pages)
            src = page * a.page_size + in_page;
          else
            set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
        }
        page_of(tok_b, page, in_page);
        tok_b = token(i + 2);
        const uint32_t there = __ballot_sync(0xffffffffu, src >= 0);
        auto copy = [&](const char* from, uint32_t base) {
#pragma unroll
          for (int j = 0; j < 32 / PER; ++j) {
            const int in = j * PER + lane / CH;
            const int x = __shfl_sync(0xffffffffu, src, in);
            const int r = w * 32 + in;
            cp_async16_or_zero(smem0 + base + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                               from + (x >= 0 ? x * tstride : 0), x >= 0);
          }
        };
        if (!(ok = warp_wait(&kfree[st], ph ^ 1))) break;
        if (lane == 0) {
          *reinterpret_cast<uint32_t*>(smem + C::kLive + (gi % kLiveDepth) * 16 + w * 4) = there;
          mbar_arrive(&live[gi % kLiveDepth]);
        }
        copy(kb, C::kK + st * C::kTileBytes);
        cp_async_mbar_arrive(&kfull[st]);
        if (!(ok = warp_wait(&vfree[st], ph ^ 1))) break;
        copy(vb, C::kV + st * C::kTileBytes);
        cp_async_mbar_arrive(&vfull[st]);
      }
      g += n;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");   // this CTA's copies land before it ends
  } else if (lane == 0) {
    // ------------------------------------------------------------ products
    constexpr uint32_t id_s = idesc_f32<E>(kRows, kTile, false);
    constexpr uint32_t id_o = idesc_f32<E>(kRows, D, true);
    const uint32_t smem0 = smem_u32(smem);
    int seg = 0;
    while (share && ok && range.next(a, sg)) {
      const int tok0 = sg.uo * kTile, tok1 = min(sg.ntok, (sg.uo + sg.take) * kTile);
      const int n = (tok1 - tok0 + kTile - 1) / kTile;
      if (n == 0) continue;
      if (!(ok = wait(qfull, seg++))) break;
      auto scores = [&](int gi) {
        const int st = gi % C::kStages, buf = gi & 1;
        if (!wait(&kfull[st], gi / C::kStages)) return false;
        if (gi >= 2 && !wait(&sfree[buf], (gi >> 1) - 1)) return false;
        tc_fence_after();
        fence_proxy_async_smem();   // the tile was written by cp.async
        const uint32_t k = smem0 + C::kK + st * C::kTileBytes, q = smem0 + C::kQ;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t at = (x >> 2) * C::kHalf + (x & 3) * 32;
          mma_bf16(tmem + buf * kTile, desc_kmajor_sw128(q + at), desc_kmajor_sw128(k + at), id_s,
                   x > 0);
        }
        mma_commit(&kfree[st]);
        mma_commit(&sfull[buf]);
        return true;
      };
      if (!(ok = scores(g))) break;
      for (int i = 0; i < n; ++i) {
        const int gi = g + i, st = gi % C::kStages;
        if (i + 1 < n && !(ok = scores(gi + 1))) break;
        if (!(ok = wait(&vfull[st], gi / C::kStages))) break;
        if (!(ok = wait(pfull, gi))) break;
        tc_fence_after();
        fence_proxy_async_smem();
        const uint32_t v = smem0 + C::kV + st * C::kTileBytes, p = smem0 + C::kP;
#pragma unroll
        for (int x = 0; x < kTile / 16; ++x)
          mma_bf16(tmem + kTmemO, desc_kmajor_sw128(p + (x >> 2) * C::kHalf + (x & 3) * 32),
                   desc_mnmajor_sw128(v + x * 2048, C::kHalf), id_o, i > 0 || x > 0);
        mma_commit(&vfree[st]);
        mma_commit(odone);
      }
      g += n;
    }
    mma_commit(drain);   // completes once every product issued above has
    const long long t0 = clock64();
    while (!mbar_try_wait_suspend(drain, 0, kSuspendNs))
      if (clock64() - t0 > kWaitCycles) {
        set_status(a.status, MISA_ERR_DEVICE_TIMEOUT);
        break;
      }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftWarps + kLoadWarps) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
  if (tid == 0) a.split[cta] = split;
}

template <typename E, int D, bool SEL>
cudaError_t launch_variant(const PagedAttn& p, AttnArgs a, cudaStream_t st) {
  using C = Cfg<D>;
  const auto kernel = paged_attn_tc_kernel<E, D, SEL>;
  cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (err != cudaSuccess) return err;
  const int rows = attn_rows(p);
  a.nb = (rows + kRows - 1) / kRows;
  const int64_t items = (int64_t)p.nseq * (SEL ? p.T : 1) * a.nb * p.Hkv;
  const int64_t span = SEL ? p.topk : (int64_t)p.max_pages * p.page_size;
  const int64_t units = (span + kTile - 1) / kTile;   // of the longest item there can be
  const int grid = (int)(items * units < kTcCtas ? items * units : kTcCtas);
  err = launch_pdl(kernel, dim3(grid), dim3(kThreads), C::kBytes, st, a);
  if (err != cudaSuccess || units == 1) return err;
  return launch_join<E, D, kRows, SEL>(a, grid, rows < kRows ? rows : kRows, st);
}

}  // namespace

size_t paged_attn_tc_ws_bytes(const PagedAttn& p) { return attn_ws_bytes(kTcCtas, kRows, p.d); }

cudaError_t launch_paged_attn_tc(const PagedAttn& p, void* scratch, int* status, cudaStream_t st) {
  const AttnArgs a = attn_args(p, scratch, kTcCtas, kRows, status);
  const bool bf16 = p.dtype == MISA_DTYPE_BF16, sel = p.topk > 0;
  if (p.d == 128) {
    if (bf16)
      return sel ? launch_variant<__nv_bfloat16, 128, true>(p, a, st)
                 : launch_variant<__nv_bfloat16, 128, false>(p, a, st);
    return sel ? launch_variant<__half, 128, true>(p, a, st)
               : launch_variant<__half, 128, false>(p, a, st);
  }
  if (bf16)
    return sel ? launch_variant<__nv_bfloat16, 64, true>(p, a, st)
               : launch_variant<__nv_bfloat16, 64, false>(p, a, st);
  return sel ? launch_variant<__half, 64, true>(p, a, st)
             : launch_variant<__half, 64, false>(p, a, st);
}

}  // namespace misa

// K9 for many query rows per key-value head: the paged attention on the fifth-generation tensor
// cores.  Drafts of several tokens, wide groups and single key-value heads put more than 32 rows
// (queries x heads of a group) on each loaded token, where warp-level matrix steps bound the
// kernel (about 190 TFLOP/s).
//
// One CTA per SM, roles by warp:
//   warps 0 - 3, 4 - 7   the weights of the first and of the second 64 tokens of a tile, a thread
//                 per query row: scores from tensor memory, running maximum and sum, weights back
//                 to tensor memory (over the scores) as the second product's operand.  The two
//                 groups keep a maximum, a sum and an output of their own, joined at the end, so
//                 that nothing is exchanged in between; two score buffers keep the next tile's
//                 scores ready
//   warps 8, 9 and 10, 11   gather the tiles of keys and of values: page entries, then 16-byte
//                 asynchronous copies into the 128-byte-swizzled operand layout; the warps of the
//                 values also fetch the queries, but those of the first segment
//   warp 12       one thread issues the products S = Q K^T and O += P V, fp32 sums in tensor memory
// A group's maximum moves only when a row's scores exceed it by more than 2^8 (fp16: 2^4), so that
// O, which stays in tensor memory, is rescaled a few times per item at most; any reference gives the
// same quotient (the conditional rescaling published for attention on this architecture).  Ranges and partials as in paged_attn.cu.  All waits are bounded; where one runs out
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
constexpr int kThreads = 32 * (kSoftWarps + kLoadWarps + 1);
constexpr int kTcCtas = 148;     // one per SM
constexpr int kWholeUnits = 4;   // tiles up to which an item stays with one CTA: no join
constexpr int kLiveDepth = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 2 * kTile;            // S at columns 0 and 128, then the groups' O

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;                 // operand tiles are 64 columns wide
  static constexpr int kHalf = 128 * 128;                // 128 rows of 128 bytes
  static constexpr int kTileBytes = kHalves * kHalf;
  // keys are wanted two tiles before their values are
  static constexpr int kKStages = D == 128 ? 3 : 5, kVStages = D == 128 ? 2 : 4;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kKStages * kTileBytes;
  static constexpr int kQ = kV + kVStages * kTileBytes;
  static constexpr int kLive = kQ + kTileBytes;          // [kLiveDepth][4] words
  static constexpr int kBars = kLive + kLiveDepth * 16;
  // kfull, kfree [kKStages], vfull, vfree [kVStages], sfull [2], pfull [2][2], qfirst, qfull, qfree,
  // odone, joined, ofree, drain, live [kLiveDepth]
  static constexpr int kNumBars = 2 * kKStages + 2 * kVStages + 6 + 7 + kLiveDepth;
  static constexpr int kBytes = kBars + kNumBars * 8 + 1024;   // 1 KB alignment of the base
  static_assert(kBytes <= 224 * 1024, "shared memory");
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

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(
          v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
// True in one lane of a converged warp, the same one each time (tcgen05.commit tracks the products
// of the thread that issues it).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// D[tmem] (+)= A[tmem] * B[smem desc]: A's rows are the lanes, two 16-bit elements a column.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 bytes (a sector) to global memory at once; 32-byte aligned.
__device__ __forceinline__ void store32(void* to, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Weights rise above the maximum's up to this factor (log2) before the running maximum follows.
// In fp16 the slack is taken from the room for small weights (Weights), so it is smaller there: 16
// drafted queries of 16 heads over 32 x 8192 tokens 61.3 us (61.6 us with 2^8, 63.4 us with 2^2).
template <typename E>
constexpr float kSlack = Weights<E>::kFp16 ? 4.f : 8.f;

template <typename E, int D, bool SEL>
__global__ void __launch_bounds__(kThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ AttnArgs a) {
  using C = Cfg<D>;
  using R = Range<kRows, SEL, kTile, kThreads>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ typename R::Shared s_range;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ float2 s_ml[2][2][kRows];   // [segment parity][group][row]
  // values of this segment that not every row sees were NaN or infinite and left out; their tokens
  __shared__ int s_non_finite;
  __shared__ Dropped s_dropped;
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t *kfull = bars, *kfree = kfull + C::kKStages, *vfull = kfree + C::kKStages,
           *vfree = vfull + C::kVStages, *sfull = vfree + C::kVStages, *pfull = sfull + 2,
           *qfirst = pfull + 4, *qfull = qfirst + 1, *qfree = qfull + 1, *odone = qfree + 1,
           *joined = odone + 1, *ofree = joined + 1, *drain = ofree + 1, *live = drain + 1;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  volatile int* abort_flag = &s_abort;

  if (!SEL) s_dropped.clear(tid);
  if (tid == 0) {
    s_abort = s_non_finite = 0;
    for (int i = 0; i < C::kKStages; ++i) {
      mbar_init(&kfull[i], 32 * kLoadWarps / 2);
      mbar_init(&kfree[i], 1);
    }
    for (int i = 0; i < C::kVStages; ++i) {
      mbar_init(&vfull[i], 32 * kLoadWarps / 2);
      mbar_init(&vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sfull[i], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&pfull[i], 32 * kSoftWarps / 2);
    mbar_init(qfirst, 32 * kSoftWarps);
    mbar_init(qfull, 32 * kLoadWarps / 2);
    mbar_init(qfree, 1);
    mbar_init(odone, 1);
    mbar_init(joined, 32 * kSoftWarps);
    mbar_init(ofree, 32 * kSoftWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < kLiveDepth; ++i) mbar_init(&live[i], kLoadWarps / 2);
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
  // A whole warp's bounded wait: every lane polls, and all leave the loop together.  (With lane 0
  // polling alone the warp stayed diverged behind a wait that had to wait, at 0.2 us for every
  // later shuffle: 3.3 us a tile instead of 2.0 us.)  A barrier's phases are waited for one by one
  // by every waiter, so that its parity is never ambiguous.
  auto warp_wait = [&](uint64_t* bar, int phase) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1))) return true;
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait_suspend(bar, phase & 1, kSuspendNs))) {
      const bool late = clock64() - t0 > a.wait_cycles;
      if (__any_sync(0xffffffffu, late || *abort_flag)) {
        if (late) {
          *abort_flag = 1;
          set_status(a.status, MISA_ERR_DEVICE_TIMEOUT);
        }
        return false;
      }
    }
    return true;
  };
  auto scaled = [&](uint4 x) {   // a query's elements, with the scale's sign
    x.x = (x.x ^ a.q_flip) & a.q_keep;
    x.y = (x.y ^ a.q_flip) & a.q_keep;
    x.z = (x.z ^ a.q_flip) & a.q_keep;
    x.w = (x.w ^ a.q_flip) & a.q_keep;
    return x;
  };
  int g = 0;        // tiles before this segment, in every role
  int seg = 0;      // segments with tiles before this one
  bool ok = true;

  if (warp < kSoftWarps) {
    // ------------------------------------------------------------ scores to weights, output
    const int group = warp / 4, row = tid % kRows;   // a warp reaches the 32 tensor-memory lanes
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);   // of its number modulo 4
    const uint32_t to = lanes + kTmemO + group * D;
    while (share && ok && range.next(a, sg)) {
      const Entry<kRows, SEL> en(a, sg.e);
      const int tok0 = sg.uo * kTile, tok1 = min(sg.ntok, (sg.uo + sg.take) * kTile);
      const int n = (tok1 - tok0 + kTile - 1) / kTile;
      const bool mine = row < en.rows, warp_live = warp % 4 * 32 < en.rows;
      const int rr = en.row0 + row, t = mine ? rr / a.G : 0;
      float m = -INFINITY, l = 0.f;
      if (n > 0 && seg == 0) {   // half of the row of Q; of later segments a loader does it
        const uint4* q = reinterpret_cast<const uint4*>(
            static_cast<const E*>(a.q) +
            (((int64_t)en.n * a.T + t) * a.Hq + sg.hk * a.G + (rr - t * a.G)) * D);
        unsigned char* dst = smem + C::kQ + row * 128;
        uint4 x[D / 16];
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          x[i] = mine ? q[group * (D / 16) + i] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const int c = group * (D / 16) + i;
          *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kHalf + (((c & 7) ^ (row & 7)) << 4)) =
              scaled(x[i]);
        }
        fence_proxy_async_smem();
        mbar_arrive(qfirst);
      }
      int lim = INT_MAX;
      if (!SEL && mine)
        lim = last_token(a.pos, (int64_t)en.n * a.T + t, a.max_pages * a.page_size, nullptr);
      for (int i = 0; i < n; ++i) {
        const int gi = g + i, buf = gi & 1;
        const uint32_t ts = lanes + buf * kTile + group * 64;
        bool behind = i > 0;   // the product of the tile before is still to be waited for
        if (!(ok = warp_wait(&sfull[buf], gi >> 1))) break;
        tc_fence_after();
        if (!(ok = warp_wait(&live[gi % kLiveDepth], gi / kLiveDepth))) break;
        if (warp_live) {
          const uint2 there = *reinterpret_cast<const uint2*>(
              smem + C::kLive + (gi % kLiveDepth) * 16 + group * 8);
          const int s0 = tok0 + i * kTile + group * 64;
          float s[64];
          tmem_ld32(ts, s);
          tmem_ld32(ts + 32, s + 32);
          tmem_ld_wait(s);
          tmem_ld_wait(s + 32);
          if ((there.x & there.y) != 0xffffffffu || (!SEL && s0 + 63 > lim)) {
#pragma unroll
            for (int c = 0; c < 64; ++c)   // what the row does not see is -inf
              if (!(((c < 32 ? there.x : there.y) >> (c & 31)) & 1u) || (!SEL && s0 + c > lim))
                s[c] = -INFINITY;
          }
          float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int c = 4; c < 64; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
          const float top =
              Weights<E>::reference(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), a.scale2,
                                    Weights<E>::kTop - kSlack<E>);
          if (__any_sync(0xffffffffu, top > __fadd_rd(m, kSlack<E>))) {   // the maximum moves, O with it
            const float up = fmaxf(m, top), f = up == m ? 1.f : exp2_approx(m - up);
            m = up;
            l *= f;
            if (behind) {
              if (!(ok = warp_wait(odone, gi - 1))) break;
              behind = false;
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(to + c, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int x = 0; x < 32; ++x) o[x] *= f;
                tmem_st32(to + c, o);
              }
            }
          }
          const float base = m == -INFINITY ? 0.f : -m;
          float sum[4] = {0.f, 0.f, 0.f, 0.f};
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const float x = exp2_approx(fmaf(s[c], a.scale2, base));
            const float y = exp2_approx(fmaf(s[c + 1], a.scale2, base));
            sum[c & 2] += x;
            sum[(c & 2) + 1] += y;
            p[c / 2] = pack2<E>(x, y);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_st32(ts, p);   // two weights to a column, over the scores
          tmem_st_wait();
        }
        if (behind && !(ok = warp_wait(odone, gi - 1))) break;
        tc_fence_before();
        mbar_arrive(&pfull[2 * buf + group]);
      }
      if (!ok) break;
      const bool whole = sg.take == sg.units;
      const int slot = 2 * cta + (sg.uo == 0 ? 1 : 0);
      float f[2] = {0.f, 0.f};   // factors of the groups' outputs
      if (n > 0) {
        s_ml[seg & 1][group][row] = make_float2(m, l);
        mbar_arrive(joined);
        if (!(ok = warp_wait(joined, seg)) || !(ok = warp_wait(odone, g + n - 1))) break;
        tc_fence_after();
        const float2 x[2] = {s_ml[seg & 1][0][row], s_ml[seg & 1][1][row]};
        m = fmaxf(x[0].x, x[1].x);
        l = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          // a group that saw nothing of the row adds nothing, whatever its products came to
          if (x[k].y == 0.f) continue;
          f[k] = x[k].x == m ? 1.f : exp2_approx(x[k].x - m);
          l += x[k].y * f[k];
        }
        if (whole && Weights<E>::beyond(m)) l = f[0] = f[1] = NAN;
      }
      if (warp_live) {
        const int64_t head = ((int64_t)en.n * a.T + t) * a.Hq + sg.hk * a.G + (rr - t * a.G);
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
        const bool wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;   // the caller's: 16 at least
#pragma unroll 1
        for (int c = group * (D / 2); c < (group + 1) * (D / 2); c += 32) {
          float o[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) o[x] = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (n > 0) {
              float y[32];
              __syncwarp();
              tmem_ld32(lanes + kTmemO + k * D + c, y);
              tmem_ld_wait(y);
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (f[k] != 0.f) o[x] = fmaf(y[x], f[k] * inv, o[x]);
            }
          if (mine && whole) {
            uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<E*>(a.out) + head * D + c);
#pragma unroll
            for (int x = 0; x < 32; x += 16) {
              uint32_t y[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) y[z] = pack2<E>(o[x + 2 * z], o[x + 2 * z + 1]);
              if (wide) {
                store32(out + x / 2, y);
              } else {
                reinterpret_cast<uint4*>(out + x / 2)[0] = make_uint4(y[0], y[1], y[2], y[3]);
                reinterpret_cast<uint4*>(out + x / 2)[1] = make_uint4(y[4], y[5], y[6], y[7]);
              }
            }
          } else if (mine) {
            float* out = a.part_o + ((int64_t)slot * kRows + row) * D + c;
#pragma unroll
            for (int x = 0; x < 32; x += 8)
              store32(out + x, reinterpret_cast<const uint32_t*>(o + x));
          }
        }
        if (!SEL && n > 0 && *static_cast<volatile int*>(&s_non_finite)) {
          const int c = group * (D / 2);
          void* to = whole ? static_cast<void*>(static_cast<E*>(a.out) + head * D + c)
                           : a.part_o + ((int64_t)slot * kRows + row) * D + c;
          add_non_finite<E, D>(a, {en.n, en.row0, en.rows, sg.hk, tok0, tok1}, s_dropped, row,
                               mine && l != 0.f, c, to, whole);
        }
        if (mine && group == 0) {
          if (!whole)
            a.part_ml[slot * kRows + row] = make_float2(m, l);
          else if (a.lse)
            a.lse[head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
      }
      if (n > 0) {   // the next segment's products may write O
        tc_fence_before();
        mbar_arrive(ofree);
        ++seg;
      }
      if (!whole && sg.uo == 0) split = make_int2(sg.e * a.Hkv + sg.hk, sg.last_cta);
      g += n;
    }
  } else if (warp < kSoftWarps + kLoadWarps) {
    // ------------------------------------------------------------ tiles
    const int w = (warp - kSoftWarps) & 1;             // which 64 tokens of a tile
    const bool vals = warp >= kSoftWarps + 2;          // values, or keys
    constexpr int CH = D / 8, PER = 32 / CH;   // 16-byte chunks of a row, rows of a warp-wide copy
    constexpr int STEPS = 64 / PER;
    const int c = lane % CH;
    const int stages = vals ? C::kVStages : C::kKStages;
    uint64_t *full = vals ? vfull : kfull, *free = vals ? vfree : kfree;
    const uint32_t ring = smem_u32(smem) + (vals ? C::kV : C::kK) + (c >> 3) * C::kHalf;
    const int cap = a.max_pages * a.page_size;
    int st = 0, ph = 0;   // stage and its use
    while (share && ok && range.next(a, sg)) {
      const Entry<kRows, SEL> en(a, sg.e);
      const int tok0 = sg.uo * kTile, tok1 = min(sg.ntok, (sg.uo + sg.take) * kTile);
      const int n = (tok1 - tok0 + kTile - 1) / kTile;
      const int32_t* pages = a.table + (int64_t)en.n * a.max_pages;
      const int64_t sel_row = (int64_t)en.n * a.T + en.row0 / a.G;
      const int32_t* ids = SEL ? a.idx + sel_row * a.topk : nullptr;
      // a lane looks up two tokens of a tile, x and x + 32: the id, a tile ahead the page entry
      auto token = [&](int i, int x) -> int {
        const int s = tok0 + i * kTile + w * 64 + x * 32 + lane;
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
      const char* from = static_cast<const char*>(vals ? a.v : a.k) +
                         (int64_t)sg.hk * (D * 2) + c * 16;
      const int tstride = a.Hkv * (D * 2);   // at most 2^16 heads
      int tok[2] = {token(0, 0), token(0, 1)}, next[2] = {token(1, 0), token(1, 1)};
      int page[2], in_page[2];
      if (SEL) last_sel = last_token(a.pos, sel_row, cap, a.status);
#pragma unroll
      for (int x = 0; x < 2; ++x) page_of(tok[x], page[x], in_page[x]);
      if (vals && n > 0 && seg > 0) {
        // The query rows, as soon as the last scores of the segment before are there: their
        // weights, their product and the output follow meanwhile.  From the output to the next
        // scores 1.5 to 2 us; 5.5 us when the warps of the weights loaded them after the output.
        // (By the warps of the keys they held up the next keys.)
        if (!(ok = warp_wait(qfree, seg - 1))) break;
        int row[2];   // of the two rows that a lane looks up
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = w * 64 + x * 32 + lane, rr = en.row0 + r, t = rr / a.G;
          row[x] = r < en.rows ? t * a.Hq + (rr - t * a.G) : -1;
        }
        const char* q = static_cast<const char*>(a.q) +
                        ((int64_t)en.n * a.T * a.Hq + sg.hk * a.G) * (D * 2) + c * 16;
        const uint32_t dst = smem_u32(smem) + C::kQ + (c >> 3) * C::kHalf;
#pragma unroll
        for (int j = 0; j < STEPS; ++j) {
          const int in = j * PER + lane / CH, r = w * 64 + in;
          const int x = __shfl_sync(0xffffffffu, row[j * PER / 32], in & 31);
          cp_async16_or_zero(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                             q + (int64_t)max(x, 0) * (D * 2), x >= 0);
        }
        if (a.q_flip != 0 || a.q_keep != 0xffffffffu) {   // a scale below zero, or zero
          asm volatile("cp.async.wait_all;" ::: "memory");
          for (int j = 0; j < STEPS; ++j) {
            const int r = w * 64 + j * PER + lane / CH;
            uint4* at = reinterpret_cast<uint4*>(smem + C::kQ + (c >> 3) * C::kHalf + r * 128 +
                                                 (((c & 7) ^ (r & 7)) << 4));
            *at = scaled(*at);
          }
          fence_proxy_async_smem();
          mbar_arrive(qfull);
        } else {
          cp_async_mbar_arrive(qfull);
        }
      }
      for (int i = 0; i < n; ++i) {
        const int gi = g + i;
        int src[2];
        uint32_t there[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          src[x] = -1;
          if (in_page[x] >= 0) {
            if ((unsigned)page[x] < (unsigned)a.num_pages)
              src[x] = page[x] * a.page_size + in_page[x];
            else
              set_status(a.status, MISA_ERR_BAD_DEVICE_INPUT);
          }
          there[x] = __ballot_sync(0xffffffffu, src[x] >= 0);
          page_of(next[x], page[x], in_page[x]);
          next[x] = token(i + 2, x);
        }
        if (!(ok = warp_wait(&free[st], ph ^ 1))) break;
        if (!vals && lane == 0) {
          *reinterpret_cast<uint2*>(smem + C::kLive + (gi % kLiveDepth) * 16 + w * 8) =
              make_uint2(there[0], there[1]);
          mbar_arrive(&live[gi % kLiveDepth]);
        }
        const uint32_t dst = ring + st * C::kTileBytes;
        if (vals || gi != a.skip_tile || cta != 0) {   // always, but in a test
#pragma unroll
          for (int j = 0; j < STEPS; ++j) {
            const int in = j * PER + lane / CH;   // of the warp's 64 tokens
            const int x = __shfl_sync(0xffffffffu, src[j * PER / 32], in & 31);
            const int r = w * 64 + in;
            cp_async16_or_zero(dst + r * 128 + (((c & 7) ^ (r & 7)) << 4),
                               from + (int64_t)max(x, 0) * tstride, x >= 0);
          }
          cp_async_mbar_arrive(&full[st]);
        }
        if (++st == stages) {
          st = 0;
          ph ^= 1;
        }
      }
      g += n;
      if (n > 0) ++seg;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");   // this CTA's copies land before it ends
  } else {
    // ------------------------------------------------------------ products
    // The warp stays together; one elected lane issues.
    constexpr uint32_t id_s = idesc_f32<E>(kRows, kTile, false);
    constexpr uint32_t id_o = idesc_f32<E>(kRows, D, true);
    // operand descriptors; a step within the operands adds to the start address (16-byte units)
    const uint32_t smem0 = smem_u32(smem);
    const uint64_t q0 = desc_kmajor_sw128(smem0 + C::kQ), k0 = desc_kmajor_sw128(smem0 + C::kK),
                   v0 = desc_mnmajor_sw128(smem0 + C::kV, C::kHalf);
    auto scores = [&](int gi, bool last) {
      const int st = gi % C::kKStages, buf = gi & 1;
      if (!warp_wait(&kfull[st], gi / C::kKStages)) return false;
      tc_fence_after();
      fence_proxy_async_smem();   // the tile was written by cp.async
      const uint64_t k = k0 + st * (C::kTileBytes >> 4);
      if (elect_one()) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const uint32_t at = ((x >> 2) * C::kHalf + (x & 3) * 32) >> 4;
          mma_bf16(tmem + buf * kTile, q0 + at, k + at, id_s, x > 0);
        }
        mma_commit(&kfree[st]);
        mma_commit(&sfull[buf]);
        if (last) mma_commit(qfree);
      }
      __syncwarp();
      return true;
    };
    while (share && ok && range.next(a, sg)) {
      const int tok0 = sg.uo * kTile, tok1 = min(sg.ntok, (sg.uo + sg.take) * kTile);
      const int n = (tok1 - tok0 + kTile - 1) / kTile;
      if (n == 0) continue;
      const Entry<kRows, SEL> en(a, sg.e);
      int seen = INT_MAX;
      if (!SEL)
        seen = seen_by_all(a, {en.n, en.row0, en.rows, sg.hk, tok0, tok1}, 32, lane);
      if (!(ok = seg == 0 ? warp_wait(qfirst, 0) : warp_wait(qfull, seg - 1))) break;
      if (!(ok = scores(g, n == 1)) || (n > 1 && !(ok = scores(g + 1, n == 2)))) break;
      if (seg > 0 && !(ok = warp_wait(ofree, seg - 1))) break;
      if (!SEL && s_non_finite) {   // the segment before is through with them
        __syncwarp();
        s_dropped.clear(lane);
        s_non_finite = 0;
        __syncwarp();
      }
      if (!SEL) seen = __reduce_min_sync(0xffffffffu, seen);
      for (int i = 0; i < n; ++i) {
        const int gi = g + i, st = gi % C::kVStages, buf = gi & 1;
        if (!(ok = warp_wait(&vfull[st], gi / C::kVStages))) break;
        const int s0 = tok0 + i * kTile, s1 = min(s0 + kTile, tok1);
        // Values of tokens that some rows do not see, before the product reads them.  Here, as this
        // warp waits for them anyway: a loader that looked at its own copies stood still until
        // they had landed (70 us instead of 65 us for 32 sequences of 16 x 4 rows, 8 key-value
        // heads, 1024 tokens), and the warps of the weights took 67 us.
        if (!SEL && s1 - 1 > seen) {
          unsigned char* tile = smem + C::kV + st * C::kTileBytes;
          bool drop = false;
          for (int x = max(seen + 1 - s0, 0) * (D / 8) + lane; x < (s1 - s0) * (D / 8); x += 32) {
            const int r = x / (D / 8), c = x % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(tile + (c >> 3) * C::kHalf + r * 128 +
                                                 (((c & 7) ^ (r & 7)) << 4));
            uint4 y = *at;
            if (drop_non_finite<E>(y)) {
              *at = y;
              s_dropped.add(s0 + r - tok0, tok1 - tok0);
              drop = true;
            }
          }
          if (drop) s_non_finite = 1;
          __threadfence_block();
          fence_proxy_async_smem();
          __syncwarp();
        }
        const uint64_t v = v0 + st * (C::kTileBytes >> 4);
        // The groups' weights are waited for apart: of two warps on a scheduler one is ahead by
        // its exponentials, and so one computes while the other waits.
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!(ok = warp_wait(&pfull[2 * buf + k], gi >> 1))) break;
          tc_fence_after();
          fence_proxy_async_smem();
          if (elect_one()) {
#pragma unroll
            for (int x = 0; x < 4; ++x)   // 16 tokens each
              mma_bf16_ts(tmem + kTmemO + k * D, tmem + buf * kTile + k * 64 + x * 8,
                          v + (((k * 4 + x) * 2048) >> 4), id_o, i > 0 || x > 0);
            if (k == 1) {
              mma_commit(&vfree[st]);
              mma_commit(odone);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        if (i + 2 < n && !(ok = scores(gi + 2, i + 3 == n))) break;   // over the weights just used
      }
      if (!ok) break;
      g += n;
      ++seg;
    }
    if (elect_one()) mma_commit(drain);   // completes once every product issued above has
    __syncwarp();
    const long long t0 = clock64();
    while (!__all_sync(0xffffffffu, mbar_try_wait_suspend(drain, 0, kSuspendNs)))
      if (__any_sync(0xffffffffu, clock64() - t0 > a.wait_cycles)) {
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
  // side by side where that leaves few CTAs over (16 and more of 148 are the tenth)
  if (a.nb <= kTcCtas && kTcCtas % a.nb < 16) a.side = a.nb;
  const int64_t items = (int64_t)p.nseq * (SEL ? p.T : 1) * (a.nb / a.side) * p.Hkv;
  const int64_t span = SEL ? p.topk : (int64_t)p.max_pages * p.page_size;
  const int64_t units = (span + kTile - 1) / kTile;   // of the longest item there can be
  const int64_t most = kTcCtas / a.side;
  a.whole = items <= most && units <= kWholeUnits;
  const int grid = (int)(a.whole ? items : items * units < most ? items * units : most) * a.side;
  err = launch_pdl(kernel, dim3(grid), dim3(kThreads), C::kBytes, st, a);
  if (err != cudaSuccess || a.whole || units == 1) return err;
  return launch_join<E, D, kRows, SEL>(a, grid, items * a.side, rows < kRows ? rows : kRows, st);
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

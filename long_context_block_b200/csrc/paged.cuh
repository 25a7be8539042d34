// Helpers shared by the paged-cache kernels: 16-bit element types, page lookups, warp-level
// matrix steps and asynchronous row copies.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "common.cuh"
#include "sm100.cuh"

namespace misa {
namespace paged {

// n / d of 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d), (umulhi(n, mul) + n) >> l for
// mul = floor(2^32 (2^l - d) / d) + 1 (Granlund and Montgomery).
struct Divide {
  uint32_t mul, shift;
  static Divide by(int divisor) {
    const uint32_t d = (uint32_t)divisor;
    Divide x = {0, 0};
    while ((uint64_t(1) << x.shift) < d) ++x.shift;
    x.mul = (uint32_t)((((uint64_t(1) << x.shift) - d) << 32) / d + 1);
    return x;
  }
  __device__ __forceinline__ int operator()(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
};

template <typename E>
struct IsBf16 {
  static constexpr bool value = false;
};
template <>
struct IsBf16<__nv_bfloat16> {
  static constexpr bool value = true;
};

// Two fp32 values rounded to the 16-bit type, `lo` in the lower half.
template <typename E>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
template <typename O>
__device__ __forceinline__ O from_f32(float x) { return O(x); }

// c (16 x 8, fp32) += a (16 x 16) * b (16 x 8), operands in the 16-bit type.
template <typename E>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4],
                                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4],
                                                 uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 bytes global -> shared memory, asynchronously; `live` false writes zeros and reads nothing.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool live) {
  const uint32_t n = live ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(n)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sets the elements of a word (two 16-bit values) that are NaN or infinite to 0; true if any was.
template <typename E>
__device__ __forceinline__ bool drop_non_finite(uint32_t& x) {
  constexpr uint32_t kExp = IsBf16<E>::value ? 0x7f80u : 0x7c00u;
  const bool lo = (x & kExp) == kExp, hi = ((x >> 16) & kExp) == kExp;
  if (lo) x &= 0xffff0000u;
  if (hi) x &= 0x0000ffffu;
  return lo || hi;
}
template <typename E>
__device__ __forceinline__ bool drop_non_finite(uint4& x) {
  const bool a = drop_non_finite<E>(x.x), b = drop_non_finite<E>(x.y), c = drop_non_finite<E>(x.z),
             d = drop_non_finite<E>(x.w);
  return a || b || c || d;
}

// 2^x; the result's relative error is at most 2^-22.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A softmax weight is rounded to the 16-bit type for its product with V, as the matrix instruction
// takes both factors in one type.  bf16 has fp32's exponents.  fp16 counts in steps of 2^-24 below
// 2^-14, so there a row's reference m is taken below its largest score, which scales weights and sum
// alike and leaves the quotient.  With the largest weight at 2^11 to 2^15, those down to 2^-25 of it
// keep fp16's precision, and those below 2^-36 of it vanish (2^-14 and 2^-25 with the largest at 1).
//
// A weight's exponent is s scale2 - m in one rounding, m the largest score's product, rounded too.
// So a row's largest weight is off by a factor 2^x, x up to half a step of m (2^-4 where m is 2^20,
// log2 domain).  m is rounded upward where that counts (beyond 2^20; in fp16, which ends at 2^16,
// always): the weights then get smaller, by up to 2^-8 where m is 2^26 and 2^-64 where it is 2^30,
// but none overflows.  That is as much as fp16 and bf16 take.  Beyond, the largest weight may vanish,
// so a row whose largest score is beyond is NaN (finish); scores so far below a row's largest weigh
// nothing.
template <typename E>
struct Weights {
  static constexpr bool kFp16 = !IsBf16<E>::value;
  static constexpr float kTop = kFp16 ? 15.f : 0.f;   // log2 of the largest weight there can be
  // magnitude of a row's largest score: 2^26, 2^30
  static constexpr float kLargest = kFp16 ? 67108864.f : 1073741824.f;
  // What a row's exponents are taken from (log2 domain): its largest score `top`, in fp16 less `up`.
  static __device__ __forceinline__ float reference(float top, float scale2, float up) {
    const float above = __fmul_ru(top, scale2);
    if constexpr (kFp16) return __fadd_ru(above, -up);
    return fabsf(above) > 1048576.f ? above : top * scale2;
  }
  // Whether a row of reference m in the end is past that (-inf: no score).
  static __device__ __forceinline__ bool beyond(float m) {
    return fabsf(m) > kLargest && m != -INFINITY;
  }
};

// Last token a query sees: pos[row] in [-1, cap); -1 sees nothing.  A value outside is
// reported and clamped.
__device__ __forceinline__ int last_token(const int32_t* __restrict__ pos, int64_t row, int cap,
                                          int* status) {
  int p = pos[row];
  if (p < -1 || p >= cap) {
    set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
    p = p < -1 ? -1 : cap - 1;
  }
  return p;
}

// Cache row (page * page_size + offset) of token `s` of a sequence whose pages are `pages`;
// -1 (reported) when the page entry names no page of the pool.  The pool holds fewer than 2^31
// rows.
__device__ __forceinline__ int cache_row(const int32_t* __restrict__ pages, int s, int page_size,
                                         const Divide& by_page, int num_pages, int* status) {
  const int i = by_page(s);
  const int page = __ldg(pages + i);
  if ((unsigned)page >= (unsigned)num_pages) {
    set_status(status, MISA_ERR_BAD_DEVICE_INPUT);
    return -1;
  }
  return page * page_size + (s - i * page_size);
}

}  // namespace paged
}  // namespace misa

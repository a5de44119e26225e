// swa_paged_mask.cuh — which keys a row of a tree of drafted tokens sees, and
// the values of an 8-bit cache, on the device.
#pragma once
#include "swa_device.cuh"
#include "swa_paged.h"

namespace swa {

// Accesses to shared memory by 32-bit addresses: after the alignment of its base
// the compiler no longer knows where a pointer points, and generic accesses wait
// for more.
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ int lds_s8(uint32_t addr) {
  int v;
  asm volatile("ld.shared.s8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Position of token i of the chunk.  A depth outside the chunk counts as the nearest inside.
template <bool X = true>
__device__ __forceinline__ int token_position(const ArgsOf<X>& a, const PagedItem& w, int kv_len, int i) {
  int at = i;
  if constexpr (X) {
    if (a.tree && a.depth) {
      const int64_t t = w.q_start + i;
      at = in_bounds(t, 1, a.n_depth, a.err) ? min(max(a.depth[t], 0), w.q_len - 1) : 0;
    }
  }
  return kv_len - w.q_len + at;
}

// Bits [c, c + 32) of the row of token i of a tree, as bits 0..31; those outside
// [0, q_len) are 0.
__device__ __forceinline__ uint32_t tree_bits(const PagedArgs& a, const PagedItem& w, int i, int c) {
  const int n = w.q_len - c;
  if (n <= 0 || c <= -32) return 0u;
  const int64_t e = (w.q_start + i) * a.tree_row;
  const int words = (w.q_len + 31) >> 5, x = c >> 5, sh = c & 31;
  const uint32_t lo = x >= 0 && in_bounds(e + x, 1, a.n_tree, a.err) ? a.tree[e + x] : 0u;
  const uint32_t hi = sh != 0 && x + 1 < words && in_bounds(e + x + 1, 1, a.n_tree, a.err) ? a.tree[e + x + 1] : 0u;
  const uint32_t bits = __funnelshift_r(lo, hi, sh);
  return n < 32 ? bits & ((1u << n) - 1u) : bits;
}

// ------------------------------------------------------- 8-bit values --
// A code of the e4m3 format (sign, 4 exponent bits of bias 7, 3 mantissa bits)
// and its row's exponent e stand for code 2^e, which the 16-bit types hold
// exactly over the exponents that a row may have.
//
// The conversion instruction gives a pair of codes as fp16, exactly.  What reads a
// row back multiplies by 2^e (fp16), or by 2^(e + 112) after moving the fp16 bits
// to the places of a bf16, whose exponents' bias is 112 higher.  That takes 3 to 4
// integer instructions a pair, at half the rate of others, and so the kernel of
// few query rows multiplies in fp16 whatever the type of q (swa_paged_rows_e4m3.cu).

// 2^(112 + e) as bf16 bits, or 2^e as fp16 bits; NaN for an exponent above the most.
template <bool F16>
__device__ __forceinline__ uint32_t exp_factor(int e) {
  if (e > kExpMost) return F16 ? 0x7E00u : 0x7FC0u;
  if constexpr (F16) {
    e = max(e, kExpLeastF16);
    return e < -14 ? 0x0200u : static_cast<uint32_t>(e + 15) << 10;
  } else {
    return static_cast<uint32_t>(max(e, kExpLeastBf16) + 239) << 7;
  }
}
// 2^e in fp32, NaN above kExpMost (e not below the least).
__device__ __forceinline__ float exp_f32(int e) {
  return e > kExpMost ? __int_as_float(0x7FC00000) : __int_as_float((e + 127) << 23);
}
// Elementwise product of two pairs.
template <bool F16>
__device__ __forceinline__ uint32_t mul2(uint32_t x, uint32_t y) {
  uint32_t r;
  if constexpr (F16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// The pair of codes in the low two bytes of x as fp16.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x) {
  uint32_t r;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(x));
  return r;
}
// Codes `at` of x (low half) and of y (high half).
__device__ __forceinline__ uint32_t codes_of(uint32_t x, uint32_t y, int at) {
  return codes_f16(__byte_perm(x, y, static_cast<uint32_t>(at | (4 + at) << 4)));
}
// The values of the four codes of x, times the factor that exp_factor gives.
template <bool F16>
__device__ __forceinline__ uint2 values4(uint32_t x, uint32_t factor) {
  uint32_t lo = codes_f16(x), hi = codes_f16(x >> 16);
  if constexpr (!F16) {  // 5 exponent bits and 3 of the mantissa, 3 places lower (a NaN stays one or becomes 480)
    lo = ((lo & 0x7FFF7FFFu) >> 3 & 0x0FFF0FFFu) | (lo & 0x80008000u);
    hi = ((hi & 0x7FFF7FFFu) >> 3 & 0x0FFF0FFFu) | (hi & 0x80008000u);
  }
  return make_uint2(mul2<F16>(lo, factor), mul2<F16>(hi, factor));
}
// The power of two that brings a row of magnitude `top` (bits of |x|) to [2^14, 2^15),
// as far as 2^100 goes: its fp16 values then lose nothing of a bf16's 8 bits
// down to 2^-29 of the largest.  A row of zeros stays.
__device__ __forceinline__ int row_shift(uint32_t top) {
  const int e = static_cast<int>(top >> 23) - 127;
  return top == 0 ? 0 : min(14 - e, 100);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }  // |e| <= 126

}  // namespace swa

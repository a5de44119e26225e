// swa_paged_mask.cuh — which keys a row of a tree of drafted tokens sees, and
// the values of an 8-bit cache, on the device.
#pragma once
#include "swa_device.cuh"
#include "swa_paged.h"

namespace swa {

// Position of token i of the chunk.  A depth outside the chunk counts as the nearest inside.
__device__ __forceinline__ int token_position(const PagedArgs& a, const PagedItem& w, int kv_len, int i) {
  int at = i;
  if (a.tree && a.depth) {
    const int64_t t = w.q_start + i;
    at = in_bounds(t, 1, a.n_depth, a.err) ? min(max(a.depth[t], 0), w.q_len - 1) : 0;
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
// bf16: the code's exponent and mantissa bits, moved to the low exponent bits
// and the high mantissa bits of a bf16, are the code's value times 2^-120 (the
// formats' biases differ by 120; subnormals too, whose rule is the same); a
// multiplication by 2^(120 + e) gives the value.  fp16: the conversion
// instruction gives the code's value, and a multiplication by 2^e the rest.

// 2^(120 + e) as bf16 bits, or 2^e as fp16 bits; NaN for an exponent above the most.
template <bool F16>
__device__ __forceinline__ uint32_t exp_factor(int e) {
  if (e > kExpMost) return F16 ? 0x7E00u : 0x7FC0u;
  if constexpr (F16) {
    e = max(e, kExpLeastF16);
    return e < -14 ? 0x0200u : static_cast<uint32_t>(e + 15) << 10;
  } else {
    return static_cast<uint32_t>(max(e, kExpLeastBf16) + 247) << 7;
  }
}
// Elementwise product of two pairs.
template <bool F16>
__device__ __forceinline__ uint32_t mul2(uint32_t x, uint32_t y) {
  uint32_t r;
  if constexpr (F16) asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  else asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// bf16: the pair of codes in bytes 1 and 3 of x, times 2^-120.
__device__ __forceinline__ uint32_t codes_high(uint32_t x) {
  return ((x & 0x7F007F00u) >> 4) | (x & 0x80008000u);
}
// fp16: the pair of codes in the low two bytes of x.
__device__ __forceinline__ uint32_t codes_f16(uint32_t x) {
  uint32_t r;
  asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(x));
  return r;
}
// Codes a (low half) and b (high half) of bytes `at` of x and y, as a pair; not yet times 2^e.
template <bool F16>
__device__ __forceinline__ uint32_t codes_of(uint32_t x, uint32_t y, int at) {
  if constexpr (F16) return codes_f16(__byte_perm(x, y, static_cast<uint32_t>(at | (4 + at) << 4)));
  else return codes_high(__byte_perm(x, y, static_cast<uint32_t>(at << 4 | (4 + at) << 12)));
}
// The four codes of x in order: pairs (0, 1) and (2, 3).
template <bool F16>
__device__ __forceinline__ void codes4(uint32_t x, uint32_t& p01, uint32_t& p23) {
  if constexpr (F16) {
    p01 = codes_f16(x);
    p23 = codes_f16(x >> 16);
  } else {
    p01 = codes_high(__byte_perm(x, 0, 0x1000));
    p23 = codes_high(__byte_perm(x, 0, 0x3020));
  }
}

}  // namespace swa

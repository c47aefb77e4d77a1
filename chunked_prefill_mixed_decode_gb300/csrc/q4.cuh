// The 4-bit K/V page: layout, encoding and decoding, shared by the kernels
// that write, read back and attend over a 4-bit cache.
//
// Encoding.  A cached row of one token and KV head is cut into groups of 32
// consecutive elements.  With a = max |x| of a group,
//     s = r5(a / 7),    code = rint(x / s) in -7..7,    value = s * code,
// where r5 rounds the fp32 quotient to five significant bits (nearest, ties
// to even).  A code has at most three significant bits (or is a power of
// two), so s * code has at most eight: every value a page can hold is exactly
// a bf16, and tensor-core operands made from it carry no further rounding.
// Rounding the scale to nearest rather than up costs no clipping: |x / s| <=
// 7 (1 + 1/32) still rounds to 7, half a step away at most.
//
// Layout.  Page `pg` of KV head `h` is the 18 D-byte block at
// ((pg * H_kv) + h) * 18 D, with NG = D / 32 groups to a row:
//     K codes   [16 rows][D / 2 bytes]
//     V codes   [16 rows][D / 2 bytes]
//     K scales  [16 rows][NG] bf16
//     V scales  [16 rows][NG] bf16
// A nibble holds code + 8.  Element d = 32 g + 8 t + e (group g, quarter t,
// e < 8) of a row sits, counted in nibbles from the row's start, at
//     K:  (t NG + g) 8 + (e odd) 4 + e / 2
//     V:  ((2 t + (e odd)) NG + g) 4 + e / 2
// Tokens never share a byte, so an append writes whole bytes.  Either order
// makes (w >> 4 i) & 0x000f000f a pair that an MMA fragment wants: for K the
// neighbouring elements (2 i, 2 i + 1) of quarter t, whose 4 NG bytes one lane
// loads at once; for V, after a byte permute joins the words of two tokens,
// element 2 i + odd of both tokens.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace {

constexpr int kQ4Page = 16;
constexpr int kQ4Group = 32;

__host__ __device__ constexpr int q4_block_bytes(int D) { return 18 * D; }

template <int D>
struct Q4 {
  static constexpr int NG = D / kQ4Group;
  static constexpr int ROW = D / 2;  // code bytes of a row
  static constexpr int V_OFF = kQ4Page * ROW;
  static constexpr int KS_OFF = 2 * kQ4Page * ROW;
  static constexpr int VS_OFF = KS_OFF + kQ4Page * NG * 2;
  static constexpr int BYTES = q4_block_bytes(D);
  static_assert(VS_OFF + kQ4Page * NG * 2 == BYTES, "block layout");
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Scale of a group whose largest magnitude is `a` (finite): zero where a / 7
// is below the smallest normal number (the whole group is then stored as
// zeros), and held to the largest scale whose codes stay finite in bf16.
__device__ __forceinline__ float q4_scale(float a) {
  const float r = __fdiv_rn(a, 7.f);
  if (!(r >= 1.17549435e-38f)) return 0.f;
  uint32_t u = __float_as_uint(r);
  u = (u + 0x3ffffu + ((u >> 19) & 1u)) & ~0x7ffffu;
  return fminf(__uint_as_float(u), 1.125f * 4.2535295865117308e37f);  // 1.125 * 2^125
}

// Code + 8 of x for a group of scale s, r = 1 / s rounded (0 for s = 0): rint of
// x / s without a division.  With x = X 2^e (X < 256) and s = m 2^f (m in
// 16..31), a quotient q of at most 7.25 that is not exactly halfway between two
// codes is |2 X - m (2 n + 1) 2^j| / (2 m 2^j) >= q / (2 X) > 2^-10 away from
// halfway.  x r is off by 2^-22 relative at most, so rounding it to a multiple of
// 2^-11 (adding and subtracting 6144) restores the exact halfway points and moves
// nothing across one; the last addition rounds to a whole number, ties to even.
__device__ __forceinline__ uint32_t q4_nibble(float x, float r) {
  const float q = __fadd_rn(__fmaf_rn(x, r, 6144.f), -6144.f);
  return __float_as_uint(__fadd_rn(q, 12582920.f)) & 15u;  // 1.5 * 2^23 + 8
}

// ---- decoding

// Nibbles i and i + 4 of a code word as the bf16 pair 128 + nibble (the nibble
// lands in the low mantissa bits of 128): one shift and one three-input logic
// instruction for two values.
__device__ __forceinline__ uint32_t q4_pair128(uint32_t w, int i) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w >> (4 * i)), "r"(0x000f000fu), "r"(0x43004300u));
  return r;
}

// The same pair as codes (nibble - 8), exact.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, int i) {
  const uint32_t r = q4_pair128(w, i), c = 0x43084308u;  // 136
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&r), *reinterpret_cast<const __nv_bfloat162*>(&c));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// A pair of values, scale * code, from s2 = (s, s): any scale.  The product plus
// zero: a scale of zero gives +0 whatever the codes (-8 in a row never written).
__device__ __forceinline__ uint32_t q4_pair_times(uint32_t w, int i, uint32_t s2) {
  const uint32_t r = q4_pair(w, i), zero = 0u;
  const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&r), *reinterpret_cast<const __nv_bfloat162*>(&s2),
                                   *reinterpret_cast<const __nv_bfloat162*>(&zero));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// A quarter of the same pair from s2 and c2 = -6 s2: with the nibble n higher in
// the mantissa the operand is 4 + n / 4, and
//     (4 + n / 4) s - 6 s = s (n - 8) / 4
// is one fused multiply-add.  6 s is exact (6 = 3 * 2 and s has five bits) and
// finite for every scale, which 24 s for whole values would not be from 2^123.4 on;
// the result fits in eight bits, so the single rounding changes nothing.
__device__ __forceinline__ uint32_t q4_quarter_pair(uint32_t w, int i, uint32_t s2, uint32_t c2) {
  uint32_t r;
  const uint32_t m = i == 0 ? w << 3 : w >> (4 * i - 3);
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(m), "r"(0x00780078u), "r"(0x40804080u));
  const __nv_bfloat162 d = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&r), *reinterpret_cast<const __nv_bfloat162*>(&s2),
                                   *reinterpret_cast<const __nv_bfloat162*>(&c2));
  return *reinterpret_cast<const uint32_t*>(&d);
}

__device__ __forceinline__ uint32_t q4_minus_6(uint32_t s2) {
  const uint32_t m6 = 0xc0c0c0c0u;
  const __nv_bfloat162 d = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&s2), *reinterpret_cast<const __nv_bfloat162*>(&m6));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// N words of global memory, 4 N-byte aligned
template <int N>
__device__ __forceinline__ void ldg_words(const uint8_t* src, uint32_t* dst) {
  if constexpr (N == 4) {
    const uint4 x = __ldg(reinterpret_cast<const uint4*>(src));
    dst[0] = x.x; dst[1] = x.y; dst[2] = x.z; dst[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(src));
    dst[0] = x.x; dst[1] = x.y;
  } else {
    dst[0] = __ldg(reinterpret_cast<const uint32_t*>(src));
  }
}

// Half h (0 low, 1 high) of `a` below the same half of `b`.
__device__ __forceinline__ uint32_t join_halves(uint32_t a, uint32_t b, int h) {
  return __byte_perm(a, b, h == 0 ? 0x5410 : 0x7632);
}

}  // namespace

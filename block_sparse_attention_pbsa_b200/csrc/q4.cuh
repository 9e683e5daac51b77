// The 4-bit cache block: layout and number format shared by the kernels that write and read it.
//
// A slot of one head holds 64 tokens (BT) of K and V.  A token's K (and, apart from it, its V) has
// one scale s and one minimum m, both bf16, and a 4-bit code c per channel; the value held is
// s*c + m.  With lo = min x and hi = max x over the channels,
//   m = the largest bf16 <= lo,  s = the smallest bf16 >= (hi - m)/15 (at least 2^-126; 0 if hi = m),
//   c = round((x - m)/s), 0 .. 15:
// s and m are rounded outward so that no channel is clipped, and s*c is exact in fp32, so a value
// read back carries one rounding.  |value - x| <= s/2 (up to the fp32 roundings of the quotient).
//
// Layout of a slot (bytes; D = 128: 8704, D = 64: 4608), chosen so that a warp's mma.sync A
// fragments are whole 16-byte (8-byte at D = 64) shared-memory reads without bank conflicts, and
// so that one bulk copy brings K, V, scales and minima:
//   K codes  [64 tokens][D/2 bytes]: 32-bit word w of a token holds channels 8w .. 8w+7, channel
//            8w + 2i in nibble i and 8w + 2i + 1 in nibble i + 4, so (word >> 4i) & 0x000F000F is a
//            pair of neighbouring channels in the two halves of a register.
//   K (s, m) [64] pairs of bf16 (s in the low half).
//   V codes  pairs along tokens, as the second product contracts over tokens: units of 16 tokens,
//            [unit u][half ph][g 0..7][j 0..3][D/8 bytes], tokens 16u + 8ph + 2j (low half words) and
//            + 1 (high half words); 32-bit word w holds channels (D/8) g + 4w + n in nibble n of
//            each half word.
//   V (s, m) [64] pairs of bf16.
// The K half and the V half of a slot are equally long and can be copied apart.
#pragma once
#include "common.cuh"

namespace pbsa {

// What rounds to infinity in bf16: half a step above its largest number (2^128 - 2^120), and more.  Held values end below,
// or 0 * infinity would put NaN into rows that do not see the token.
constexpr float Q4_PAST = 0x1.ffp127f;

template <int D>
struct Q4 {
  static constexpr int CODE = BT * D / 2;          // bytes of K (or V) codes of a slot
  static constexpr int HALF = CODE + BT * 4;       // K, or V, with its scales and minima
  static constexpr int OFF_KS = CODE;
  static constexpr int OFF_V = HALF;
  static constexpr int OFF_VS = HALF + CODE;
  static constexpr int BYTES = 2 * HALF;
  static constexpr int KROW = D / 2;               // bytes of a token's K codes
  static constexpr int UNIT = 16 * D / 2;          // bytes of V codes of 16 tokens
  static constexpr int LANE = D / 8;               // bytes of one thread's fragment words
  static constexpr int WORDS = D / 32;             // ... in 32-bit words
  // byte of token row's half words of channel group g (D/8 channels) inside the V codes; word w is
  // 4w bytes further
  __host__ __device__ static constexpr int v_at(int row, int g) {
    return (row >> 4) * UNIT + ((row >> 3) & 1) * (UNIT / 2) + (g * 4 + ((row >> 1) & 3)) * LANE + (row & 1) * 2;
  }
};

// As mbar_wait, for waits that are expected to last: the thread is parked by the hardware for up to 20 us at a
// time instead of polling, which would take issue slots from the warps that have work.
__device__ __forceinline__ bool mbar_wait_parked(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    if (ok) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

// min and max that return NaN if either operand is NaN
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
// x - (the bf16 nearest x): what the next term of a split into bf16 terms holds
__device__ __forceinline__ float bf16_rest(float x) { return x - __bfloat162float(__float2bfloat16_rn(x)); }
// the neighbouring bf16 on the asked side, as fp32 bits
__device__ __forceinline__ float bf16_down(float x) {
  uint32_t u = __float_as_uint(x);
  if (u & 0x80000000u) u += 0xFFFFu;   // a negative number moves away from zero unless it is a bf16
  return __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ float bf16_up_pos(float x) {   // x >= 0
  return __uint_as_float((__float_as_uint(x) + 0xFFFFu) & 0xFFFF0000u);
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// nibbles i and i + 4 of a word as the bf16 pair (128 + low, 128 + high): a code or-ed into the
// mantissa of 128.0 (7 mantissa bits, so the units place is the last bit)
template <int I>
__device__ __forceinline__ uint32_t nibble_pair(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(r) : "r"(w >> (4 * I)));   // (a & b) | c
  return r;
}
// ... minus 136: the codes centred, -8 .. 7, exact
__device__ __forceinline__ uint32_t centred(uint32_t pair) {
  uint32_t r;
  asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(pair), "r"(0x43084308u));
  return r;
}

}  // namespace pbsa

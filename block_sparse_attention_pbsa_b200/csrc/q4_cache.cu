// Tokens into the 4-bit cache (append) and blocks of it back into dense block pools (expand).
//
// append: for token t with slot_map[t] = slot*64 + row >= 0 and each head, the K and V vectors are
// quantised as q4.cuh defines and written to (head, slot, row).  One thread holds 8 neighbouring
// channels (one or two 16-byte loads); the 16 (D = 64: 8) threads of a vector find its minimum and
// maximum by shuffles, and a warp holds the K and the V of a token and head together, so that a
// token whose K or V is not finite can be marked as one: its K scale and minimum become NaN (every
// query that attends it then yields NaN) and its V zero, which keeps NaN out of the rows that
// do not attend it.
// expand: s*c + m of every token of the listed slots, rounded once to the pools' type, in the
// layout of the block pools that pbsa_attend reads.
//
// Both are bound by HBM: append reads 2*D*sizeof(T) bytes and writes D + 8 per (token, head).
#include "internal.h"
#include "q4.cuh"

namespace pbsa {
namespace {

struct AppendParams {
  const void *k, *v;
  long long k_ld, v_ld;   // elements from one token to the next
  int T, H;
  const int* slot_map;
  uint8_t* pool;
  int pool_slots;
  void* ws;
};

// 8 neighbouring channels as they lie in memory.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  float4 a, b;
  __device__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ void load(const float* p) {
    a = __ldg(reinterpret_cast<const float4*>(p));
    b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ void values(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  // least and greatest of the vector that `N` neighbouring threads hold (NaN if any is)
  template <int N>
  __device__ void range(float& lo, float& hi) const {
    float x[8];
    values(x);
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) { lo = min_nan(lo, x[i]); hi = max_nan(hi, x[i]); }
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
      lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
  }
};
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
  __device__ void load(const __nv_bfloat16* p) { a = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ void values(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = lo_bf16(w[i]); x[2 * i + 1] = hi_bf16(w[i]); }
  }
  // as above, two at a time: (least, -greatest) travel as one pair of bf16, both taken by minima
  template <int N>
  __device__ void range(float& lo, float& hi) const {
    const uint32_t least = min2_nan(min2_nan(a.x, a.y), min2_nan(a.z, a.w)), n = 0x80008000u;
    const uint32_t most = min2_nan(min2_nan(a.x ^ n, a.y ^ n), min2_nan(a.z ^ n, a.w ^ n));
    uint32_t r = min2_nan(__byte_perm(least, most, 0x5410), __byte_perm(least, most, 0x7632));
#pragma unroll
    for (int o = 1; o < N; o <<= 1) r = min2_nan(r, __shfl_xor_sync(0xffffffffu, r, o));
    lo = lo_bf16(r);
    hi = -hi_bf16(r);
  }
};

// round(x) in the low bits of the result, which carries a constant above them (0 <= x < 2^21, ties to even)
__device__ __forceinline__ uint32_t rounded_bits(float x) { return __float_as_uint(__fadd_rn(x, 12582912.f)); }
// four codes as nibbles: multiply-adds on the rounded floats' bits, the constant taken off at the end
__device__ __forceinline__ uint32_t four(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return a + 16u * b + 256u * c + 4096u * d - 4369u * 0x4B400000u;
}

constexpr int AP_THREADS = 256;

// U neighbouring tokens of a head at once: their slots and then their values are in flight together, and the two
// tokens that share V's words are mostly written as one
template <typename T, int D, int U>
__global__ void __launch_bounds__(AP_THREADS) append_q4_kernel(const AppendParams p) {
  constexpr int LPV = D / 8;            // threads of a vector
  constexpr int PAIRS = 32 / (2 * LPV);  // (token, head) pairs of a warp
  using Q = Q4<D>;
  const int lane = threadIdx.x & 31;
  const int l = lane % LPV, part = (lane / LPV) & 1, sub = lane / (2 * LPV);
  const int runs = (p.T + U - 1) / U;                 // of U neighbouring tokens
  const long long items = (long long)runs * p.H;
  const long long warps = (long long)gridDim.x * (AP_THREADS / 32);
  // every lane of a warp runs the same iterations (shuffles); items past the end are only not written
  for (long long base = ((long long)blockIdx.x * (AP_THREADS / 32) + (threadIdx.x >> 5)) * PAIRS; base < items;
       base += warps * PAIRS) {
    const long long it = base + sub;
    const bool in = it < items;
    const int run = in ? (int)(it / p.H) : 0, h = in ? (int)(it - (long long)run * p.H) : 0;
    int at[U];
    Eight<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = in && run * U + u < p.T ? __ldg(p.slot_map + run * U + u) : -1;
    const T* src = static_cast<const T*>(part ? p.v : p.k) + (long long)run * U * (part ? p.v_ld : p.k_ld) + (long long)h * D + 8 * l;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool ok = at[u] >= 0 && at[u] < p.pool_slots * BT;
      if (!ok && at[u] != -1) {
        if (l == 0 && part == 0) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, at[u], K_Q4_APPEND);
        at[u] = -1;
      }
      x[u].zero();
      if (ok) x[u].load(src + u * (part ? p.v_ld : p.k_ld));
    }
    uint32_t lower[U], upper[U];   // K: a word's even and odd channels; V: channels 0 .. 3 and 4 .. 7
    uint32_t sm[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lo, hi, v[8];
      x[u].template range<LPV>(lo, hi);
      x[u].values(v);
      const float m = bf16_down(lo);
      const float span = __fsub_rn(hi, m);
      float s = bf16_up_pos(__fmul_rn(span, 1.0f / 15.0f));
      s = span == 0.f ? 0.f : fmaxf(s, 1.17549435e-38f);
      // (NaN compares false: fmaxf would drop it, so the operands are tested themselves)
      const bool bad = !(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY && fabsf(m) < INFINITY && s < INFINITY);
      const unsigned votes = __ballot_sync(0xffffffffu, bad);
      const unsigned pair = (2 * LPV == 32 ? 0xffffffffu : ((1u << (2 * LPV)) - 1u)) << (sub * 2 * LPV);
      const bool poison = (votes & pair) != 0;
      const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
      // no code is above 15: s >= (hi - m) / 15 (1 - 2^-23), and 15.5 is far off
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = rounded_bits(__fmul_rn(__fsub_rn(v[i], m), inv));
      lower[u] = part ? four(c[0], c[1], c[2], c[3]) : four(c[0], c[2], c[4], c[6]);
      upper[u] = part ? four(c[4], c[5], c[6], c[7]) : four(c[1], c[3], c[5], c[7]);
      sm[u] = (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xFFFF0000u);
      if (poison) {
        lower[u] = upper[u] = 0u;
        sm[u] = part ? 0u : 0x7FC07FC0u;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (at[u] < 0) continue;
      const int slot = at[u] / BT, row = at[u] % BT;
      uint8_t* blk = p.pool + ((size_t)h * p.pool_slots + slot) * Q::BYTES;
      if (l == 0) *reinterpret_cast<uint32_t*>(blk + (part ? Q::OFF_VS : Q::OFF_KS) + 4 * row) = sm[u];
      if (part == 0) {
        *reinterpret_cast<uint32_t*>(blk + row * Q::KROW + 4 * l) = lower[u] | upper[u] << 16;
        continue;
      }
      // 8 channels are half words of words (8l % (D/8)) / 4 and the next of group 8l / (D/8); the two tokens of a word
      // are written together where both are here
      uint8_t* dst = blk + Q::OFF_V + Q::v_at(row, (8 * l) / (D / 8)) + ((8 * l) % (D / 8));
      if (u + 1 < U && (row & 1) == 0 && at[u + 1 < U ? u + 1 : u] == at[u] + 1) {
        *reinterpret_cast<uint32_t*>(dst) = lower[u] | lower[u + 1 < U ? u + 1 : u] << 16;
        *reinterpret_cast<uint32_t*>(dst + 4) = upper[u] | upper[u + 1 < U ? u + 1 : u] << 16;
      } else if (u == 0 || (row & 1) == 0 || at[u > 0 ? u - 1 : 0] != at[u] - 1) {
        *reinterpret_cast<uint16_t*>(dst) = (uint16_t)lower[u];
        *reinterpret_cast<uint16_t*>(dst + 4) = (uint16_t)upper[u];
      }
    }
  }
}

struct ExpandParams {
  const uint8_t* pool;
  int pool_slots, H, n;
  const int* src_slot;
  void *k_out, *v_out;
  void* ws;
};

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

constexpr int EX_THREADS = 256;

template <typename T, int D>
__global__ void __launch_bounds__(EX_THREADS) expand_q4_kernel(const ExpandParams p) {
  using Q = Q4<D>;
  const int i = blockIdx.x, h = blockIdx.y;
  const int slot = __ldg(p.src_slot + i);
  if (slot < 0 || slot >= p.pool_slots) {
    if (slot != -1 && threadIdx.x == 0) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot, K_Q4_EXPAND);
    return;
  }
  const uint8_t* blk = p.pool + ((size_t)h * p.pool_slots + slot) * Q::BYTES;
  const size_t out = ((size_t)h * p.n + i) * BT * D;
  T* ko = static_cast<T*>(p.k_out) + out;
  T* vo = static_cast<T*>(p.v_out) + out;
  // K: word w of a token is its channels 8w ..
#pragma unroll
  for (int e = threadIdx.x; e < BT * D / 8; e += EX_THREADS) {
    const int row = e / (D / 8);
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(blk) + e);
    const uint32_t sm = __ldg(reinterpret_cast<const uint32_t*>(blk + Q::OFF_KS) + row);
    const float s = lo_bf16(sm), m = hi_bf16(sm);
    float x[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      x[2 * q] = fmaf(s, (float)((w >> (4 * q)) & 15u), m);
      x[2 * q + 1] = fmaf(s, (float)((w >> (4 * q + 16)) & 15u), m);
    }
    store8(ko + (size_t)e * 8, x);
  }
  // V: two words hold 8 channels of a pair of tokens
  for (int e = threadIdx.x; e < BT / 2 * (D / 8); e += EX_THREADS) {
    const int c8 = e % (D / 8), pr = e / (D / 8);   // channels 8 c8 .., tokens 2 pr and 2 pr + 1
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(blk + Q::OFF_V + Q::v_at(2 * pr, (8 * c8) / (D / 8)) +
                                                         (8 * c8) % (D / 8)));
    const uint2 sm = __ldg(reinterpret_cast<const uint2*>(blk + Q::OFF_VS) + pr);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const float s = lo_bf16(b ? sm.y : sm.x), m = hi_bf16(b ? sm.y : sm.x);
      float x[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        x[q] = fmaf(s, (float)((w.x >> (4 * q + 16 * b)) & 15u), m);
        x[q + 4] = fmaf(s, (float)((w.y >> (4 * q + 16 * b)) & 15u), m);
      }
      store8(vo + (size_t)(2 * pr + b) * D + 8 * c8, x);
    }
  }
}

template <typename T, int D, int U>
cudaError_t append_u(const AppendParams& p, cudaStream_t st) {
  constexpr int PAIRS = 32 / (D / 4);
  const long long warps = ((long long)((p.T + U - 1) / U) * p.H + PAIRS - 1) / PAIRS;
  const long long ctas = (warps + AP_THREADS / 32 - 1) / (AP_THREADS / 32);
  append_q4_kernel<T, D, U><<<(unsigned)(ctas < 148 * 8 ? ctas : 148 * 8), AP_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t append_t(const AppendParams& p, cudaStream_t st) {
  // a few items are spread over warps, many are loaded four at a time
  return (long long)p.T * p.H < 16384 ? append_u<T, D, 1>(p, st) : append_u<T, D, 4>(p, st);
}

}  // namespace

size_t q4_block_bytes(int d) { return d == 128 ? Q4<128>::BYTES : Q4<64>::BYTES; }

cudaError_t launch_append_q4(int H, int d, int dtype, const void* k, long long k_ld, const void* v, long long v_ld,
                             int T, const int* slot_map, void* pool, int pool_slots, void* ws, cudaStream_t st) {
  const AppendParams p = {k, v, k_ld, v_ld, T, H, slot_map, static_cast<uint8_t*>(pool), pool_slots, ws};
  if (dtype == PBSA_BF16) return d == 128 ? append_t<__nv_bfloat16, 128>(p, st) : append_t<__nv_bfloat16, 64>(p, st);
  return d == 128 ? append_t<float, 128>(p, st) : append_t<float, 64>(p, st);
}

cudaError_t launch_expand_q4(int H, int d, int dtype, const void* pool, int pool_slots, const int* src_slot, int n,
                             void* k_out, void* v_out, void* ws, cudaStream_t st) {
  const ExpandParams p = {static_cast<const uint8_t*>(pool), pool_slots, H, n, src_slot, k_out, v_out, ws};
  const dim3 grid(n, H);
  if (dtype == PBSA_BF16) {
    if (d == 128) expand_q4_kernel<__nv_bfloat16, 128><<<grid, EX_THREADS, 0, st>>>(p);
    else expand_q4_kernel<__nv_bfloat16, 64><<<grid, EX_THREADS, 0, st>>>(p);
  } else {
    if (d == 128) expand_q4_kernel<float, 128><<<grid, EX_THREADS, 0, st>>>(p);
    else expand_q4_kernel<float, 64><<<grid, EX_THREADS, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace pbsa

// Tokens into the 4-bit cache (append) and blocks of it back into dense block pools (expand).
//
// append: for token t with slot_map[t] = slot*64 + row >= 0 and each head, the K and V vectors are
// quantised as q4.cuh defines and written to (head, slot, row).  One thread holds 16 neighbouring
// channels (two or four 16-byte loads); the 8 (D = 64: 4) threads of a vector find its minimum and
// maximum by shuffles, and a warp holds the K and the V of a token and head together, so that a
// token whose K or V is not finite, or would be read back as such, can be marked: its K scale and minimum become NaN
// (every query that attends it then yields NaN) and its V zero, which keeps NaN out of the rows that do not attend it.
// expand: s*c + m of every token of the listed slots, rounded to fp32 and, where that is the pools' type, from there to
// bf16, in the layout of the block pools that pbsa_attend reads.
//
// append reads 2*D*sizeof(T) bytes and writes D + 8 per (token, head): 36 MB, 5.5 us, for 4608 tokens of 12
// heads, which take 10.1 us (3.6 TB/s).  It is bound by issue: about 130 warp instructions a token and head, most
// of them per thread (range, scale, addresses), which is why a thread holds as many channels as one
// group of V's layout.  With 8 channels a thread they were 216, and 15.2 us.
// expand moves the same bytes the other way in 6.1-6.3 us (5.7-5.9 TB/s), bound by HBM.
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

// 16 neighbouring channels as they lie in memory.
template <typename T>
struct Sixteen;
template <>
struct Sixteen<float> {
  float4 a[4];
  __device__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __ldg(reinterpret_cast<const float4*>(p) + i);
  }
  __device__ void values(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[4 * i] = a[i].x; x[4 * i + 1] = a[i].y; x[4 * i + 2] = a[i].z; x[4 * i + 3] = a[i].w; }
  }
  // least and greatest of the vector that `N` neighbouring threads hold (NaN if any is)
  template <int N>
  __device__ void range(float& lo, float& hi) const {
    float x[16];
    values(x);
    lo = hi = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) { lo = min_nan(lo, x[i]); hi = max_nan(hi, x[i]); }
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
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <>
struct Sixteen<__nv_bfloat16> {
  uint4 a, b;
  __device__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
  __device__ void load(const __nv_bfloat16* p) {
    a = __ldg(reinterpret_cast<const uint4*>(p));
    b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ void values(float (&x)[16]) const {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) { x[2 * i] = lo_bf16(w[i]); x[2 * i + 1] = hi_bf16(w[i]); }
  }
  // as above, two at a time: (least, -greatest) travel as one pair of bf16, both taken by minima
  template <int N>
  __device__ void range(float& lo, float& hi) const {
    const uint32_t least = min2_nan(min2_nan(min2_nan(a.x, a.y), min2_nan(a.z, a.w)), min2_nan(min2_nan(b.x, b.y), min2_nan(b.z, b.w)));
    const uint32_t most = max2_nan(max2_nan(max2_nan(a.x, a.y), max2_nan(a.z, a.w)), max2_nan(max2_nan(b.x, b.y), max2_nan(b.z, b.w))) ^ 0x80008000u;
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

constexpr int AP_THREADS = 64;   // (256: the 64 tokens of a decode step take 2.7 us instead of 2.3)

// U neighbouring tokens of a head at once: their slots and then their values are in flight together, and the two
// tokens that share V's words are mostly written as one
template <typename T, int D, int U>
__global__ void __launch_bounds__(AP_THREADS) append_q4_kernel(const AppendParams p) {
  constexpr int LPV = D / 16;            // threads of a vector
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
    Sixteen<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = in && run * U + u < p.T ? __ldg(p.slot_map + run * U + u) : -1;
    const T* src = static_cast<const T*>(part ? p.v : p.k) + (long long)run * U * (part ? p.v_ld : p.k_ld) + (long long)h * D + 16 * l;
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
    uint32_t code[U][4];   // K: even and odd channels of a word, then of the next; V: channels 0 .. 3, 4 .. 7, ...
    uint32_t sm[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float lo, hi, v[16];
      x[u].template range<LPV>(lo, hi);
      x[u].values(v);
      const float m = bf16_down(lo);
      const float span = __fsub_rn(hi, m);
      float s = bf16_up_pos(__fmul_rn(span, 1.0f / 15.0f));
      s = span == 0.f ? 0.f : fmaxf(s, 1.17549435e-38f);
      // (NaN compares false: fmaxf would drop it, so the operands are tested themselves.  15 s + m bounds the values held.)
      const bool bad = !(fabsf(lo) < INFINITY && fabsf(hi) < INFINITY && fabsf(m) < INFINITY && fmaf(15.f, s, m) < Q4_PAST);
      const unsigned votes = __ballot_sync(0xffffffffu, bad);
      const unsigned pair = (2 * LPV == 32 ? 0xffffffffu : ((1u << (2 * LPV)) - 1u)) << (sub * 2 * LPV);
      const bool poison = (votes & pair) != 0;
      const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
      // no code is above 15: s >= (hi - m) / 15 (1 - 2^-23), and 15.5 is far off
      uint32_t c[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) c[i] = rounded_bits(__fmul_rn(__fsub_rn(v[i], m), inv));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 8 * (i >> 1) + (i & 1);
        code[u][i] = part ? four(c[4 * i], c[4 * i + 1], c[4 * i + 2], c[4 * i + 3]) : four(c[e], c[e + 2], c[e + 4], c[e + 6]);
      }
      sm[u] = (__float_as_uint(s) >> 16) | (__float_as_uint(m) & 0xFFFF0000u);
      if (poison) {
        code[u][0] = code[u][1] = code[u][2] = code[u][3] = 0u;
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
        *reinterpret_cast<uint2*>(blk + row * Q::KROW + 8 * l) =
            make_uint2(code[u][0] | code[u][1] << 16, code[u][2] | code[u][3] << 16);
        continue;
      }
      // 16 channels are half words of four words, in one group of D/8 channels or in two; the two tokens of a word
      // are written together where both are here
      constexpr int GROUPS = 128 / D, PER = 4 / GROUPS;   // groups of the channels, words of each
      uint8_t* dst = blk + Q::OFF_V + Q::v_at(row, l * GROUPS);
      const uint32_t(&mine)[4] = code[u], (&next)[4] = code[u + 1 < U ? u + 1 : u];
      if (u + 1 < U && (row & 1) == 0 && at[u + 1 < U ? u + 1 : u] == at[u] + 1) {
        if (GROUPS == 1) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(mine[0] | next[0] << 16, mine[1] | next[1] << 16, mine[2] | next[2] << 16,
                                                      mine[3] | next[3] << 16);
        } else {
          *reinterpret_cast<uint2*>(dst) = make_uint2(mine[0] | next[0] << 16, mine[1] | next[1] << 16);
          *reinterpret_cast<uint2*>(dst + 4 * Q::LANE) = make_uint2(mine[2] | next[2] << 16, mine[3] | next[3] << 16);
        }
      } else if (u == 0 || (row & 1) == 0 || at[u > 0 ? u - 1 : 0] != at[u] - 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint16_t*>(dst + i / PER * 4 * Q::LANE + i % PER * 4) = (uint16_t)mine[i];
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
  constexpr int PAIRS = 32 / (D / 8);
  const long long warps = ((long long)((p.T + U - 1) / U) * p.H + PAIRS - 1) / PAIRS;
  const long long ctas = (warps + AP_THREADS / 32 - 1) / (AP_THREADS / 32);
  append_q4_kernel<T, D, U><<<(unsigned)(ctas < 148 * 32 ? ctas : 148 * 32), AP_THREADS, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t append_t(const AppendParams& p, cudaStream_t st) {
  // Few items are spread over as many warps as there are, many go in pairs.  Singly and in pairs, bf16 of D = 128: 512
  // items 2.3 and 2.6 us, 2048 2.9 and 2.6, 4096 3.4 and 2.9, 16384 6.6 and 4.3, 55296 15.1 and 10.0; fp32 of D = 128,
  // the last to gain: 2048 2.7 and 2.7, 3072 2.9 and 3.1, 4096 3.1 and 3.1, 8192 4.2 and 3.9, 16384 6.7 and 5.1.
  return (long long)p.T * p.H < 4096 ? append_u<T, D, 1>(p, st) : append_u<T, D, 2>(p, st);
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

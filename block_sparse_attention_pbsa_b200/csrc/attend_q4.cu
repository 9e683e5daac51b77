// Attention of the requests' queries over the 4-bit cache: the form for few query rows (single
// tokens, a few tokens, shared heads), and fp32.
//
//   x_j = scale * q . k_j,  o = sum_j 2^(x_j c - M) v_j / sum_j 2^(x_j c - M),  c = log2 e
// with k_j = s_j c_j + m_j held as 4-bit codes c_j, so that
//   q . k_j = s_j (q . c_j) + m_j sum(q),   sum_j p_j v_j = sum_j (p_j s_j)(c_j - 8) + sum_j p_j (m_j + 8 s_j):
// the two products run on the codes themselves, which bf16 holds exactly, and the scales and minima
// enter in fp32 (scores) or with p (rounded once to bf16, like any p that feeds a bf16 product).
//
// Few rows: every cached byte is used a few times only, so the aim is to read the cache once, at the
// memory's rate, and to spend less issue time on unpacking than the bytes take.  The tensor
// instruction is mma.sync m16n8k16, whose A operand comes from registers: keys (or value channels)
// are the 16 rows, query rows the 8 columns, and the codes go from shared memory through a shift
// and a lop3 straight into A fragments.  (tcgen05 reads A from TMEM or shared memory: a code
// would be written back once before it is used, and 128 rows would hold 8.)
//  * Work: the line of attend_q4.cuh.  A tile that crosses CTAs is written as partial (o, maximum, sum) per piece, and
//    a second kernel, launched as a programmatic dependent, joins the pieces in order.  At most one tile starts
//    in a CTA and ends in a later one, so a CTA has two places for pieces.  Nothing carries over from call to call.
//  * A producer warp brings whole slots (8704 bytes: K, V, scales) with one bulk copy each into a ring of three pairs;
//    four warps take 16 tokens of each slot, with a running maximum and sum of their own, joined
//    in shared memory at a tile's end.  The reference maximum moves only when a score exceeds it by
//    2^8, which one vote per 16 tokens detects.
//  * Scores come out with keys as rows; their transposition into the second product's B operand is one
//    movmatrix per 8 keys.
//  * fp32: q, and p s, are split into three bf16 terms (24 bits); the codes are exact, so the three
//    products are fp32 products.
// A slot id outside the pool is recorded and its block skipped.  Waits are bounded; on expiry the
// error is recorded, copies in flight are waited for, and the kernel winds down.
//
// Measured (D = 128, bf16; 6.5 TB/s is a plain copy's rate): 32 tokens of 32 heads (8 kv heads) over 16000 .. 60000
// cached ones, 1.37 GB: 287-309 us, 4.4-4.8 TB/s; the loads alone take 229 us.  48 tokens over 300 .. 8192, 229 MB:
// 60 us, 3.8 TB/s.  One token of 12 heads over 1536: 8.8 us, of which the join and the launches are 3.
// What bounds it: 290 warp instructions for 16 tokens of a head, 112 of them shifts and masks (128 codes a lane); the
// issue slots are 56% busy, the integer pipe 60%, HBM 65-70%.  Three CTAs an SM at 128 registers: two (with four
// pairs in the ring) take 303 us, four at 96 registers 324 us.  Two slots side by side: 290 us, one after the other 308.
#include <math.h>

#include "attend_q4.cuh"

namespace pbsa {
namespace {

constexpr int AQ_WARPS = 4;                       // computing warps
constexpr int AQ_THREADS = (AQ_WARPS + 1) * 32;   // + the producer
constexpr int AQ_STAGES = 3;                      // of two slots each
// Blocks (a tile's own cost included) that are worth a CTA: with 2, 4 and 8 one token of 12 heads over 1536 takes 9.7,
// 9.2 and 11.0 us, over 8000 14.8, 14.9 and 13.9 us.
constexpr int AQ_MIN_STEPS = 4;

template <int D, int NT>
struct AqSmem {
  static constexpr int ROWS = 8 * NT;
  static constexpr int OSTRIDE = D + 4;
  static constexpr int RING = AQ_STAGES * 2 * Q4<D>::BYTES;
  static constexpr int EX_O = RING;                                      // float[4][ROWS][OSTRIDE]
  static constexpr int EX_ML = EX_O + AQ_WARPS * ROWS * OSTRIDE * 4;     // float2[4][ROWS]
  static constexpr int BARS = EX_ML + AQ_WARPS * ROWS * 8;               // full, empty
  static constexpr int META = BARS + 2 * AQ_STAGES * 8;                  // int[stages]: slots present (two bits)
  static constexpr int TOTAL = META + AQ_STAGES * 4 + 16;
};

__device__ __forceinline__ void mma_codes(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t (&w)[N], const uint8_t* p) {
  if (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  }
}

// NT column groups of 8 query rows; SPLIT terms of q and p (1: bf16, 3: fp32)
template <int D, int NT, int SPLIT>
__global__ void __launch_bounds__(AQ_THREADS, NT == 1 && SPLIT == 1 ? 3 : 2) attend_q4_kernel(const AttendQ4Params p) {
  using Q = Q4<D>;
  using SM = AqSmem<D, NT>;
  constexpr int ROWS = SM::ROWS, W = Q::WORDS;
  extern __shared__ __align__(128) uint8_t sm[];
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + SM::BARS);
  uint64_t* empty = full + AQ_STAGES;
  volatile int* meta = reinterpret_cast<volatile int*>(sm + SM::META);
  volatile int* abort_flag = meta + AQ_STAGES;
  __shared__ Q4Start start_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < AQ_STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], AQ_WARPS);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Q4Share share = q4_share<AQ_THREADS, false>(p, ROWS, Q4_FEW_COST, AQ_MIN_STEPS, &start_s);   // has block barriers
  Q4Walk walk(p, share, start_s, ROWS, Q4_FEW_COST);

  if (warp == AQ_WARPS) {
    // ------------------------------------------------------------- producer
    int issued = 0;   // lane 0's count
    bool stop = false;
    while (!stop && walk.next()) {
      const int* row = p.table + (size_t)walk.r * p.table_ld;
      for (int b0 = walk.b0; b0 < walk.b1 && !stop; b0 += 32) {
        const int mine = b0 + lane < walk.b1 ? __ldg(row + b0 + lane) : -1;
        const int n = min(32, walk.b1 - b0);
        for (int i = 0; i < n && !stop; i += 2) {
          const int slot0 = __shfl_sync(0xffffffffu, mine, i), slot1 = __shfl_sync(0xffffffffu, mine, (i + 1) & 31);
          if (lane == 0 && !*abort_flag) {
            const int s = issued % AQ_STAGES;
            if (!mbar_wait_parked(&empty[s], ((issued / AQ_STAGES) & 1) ^ 1, kWaitLimitNs)) {
              record_error(p.ws, PBSA_ERR_TIMEOUT, issued, K_Q4_ATTEND);
              *abort_flag = 1;
            } else {
              const bool has1 = i + 1 < n;
              const bool ok0 = slot0 >= 0 && slot0 < p.pool_slots, ok1 = has1 && slot1 >= 0 && slot1 < p.pool_slots;
              if (!ok0) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot0, K_Q4_ATTEND);
              if (has1 && !ok1) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot1, K_Q4_ATTEND);
              meta[s] = (ok0 ? 1 : 0) | (ok1 ? 2 : 0);
              uint8_t* dst = sm + s * 2 * Q::BYTES;
              const uint8_t* src = p.pool + (size_t)walk.h * p.pool_slots * Q::BYTES;
              const uint32_t bytes = (ok0 ? Q::BYTES : 0) + (ok1 ? Q::BYTES : 0);
              if (bytes > 0) mbar_arrive_expect_tx(&full[s], bytes);
              else mbar_arrive(&full[s]);
              if (ok0) bulk_load(dst, src + (size_t)slot0 * Q::BYTES, Q::BYTES, &full[s]);
              if (ok1) bulk_load(dst + Q::BYTES, src + (size_t)slot1 * Q::BYTES, Q::BYTES, &full[s]);
              ++issued;
            }
          }
          stop = __any_sync(0xffffffffu, *abort_flag != 0);   // the same for every lane
        }
      }
    }
    // the CTA must not end with copies in flight, whether or not its other warps wait for them
    if (lane == 0)
      for (int i = max(0, issued - AQ_STAGES); i < issued; ++i)
        mbar_wait(&full[i % AQ_STAGES], (i / AQ_STAGES) & 1, kWaitLimitNs);
    return;
  }

  // --------------------------------------------------------------- computing warps
  const int g = lane >> 2, j = lane & 3;
  const float c = p.scale_log2;
  int taken = 0;
  while (walk.next()) {
    const int row0 = walk.mt * ROWS;                   // first row of the tile: row = token * group + head
    const int rows = min(ROWS, walk.rows - row0);
    // B fragments of q (column = row g of the group of 8), and the sums of its rows
    uint32_t qf[SPLIT][NT][2 * W][2];
    float qs[NT][2];
    int lim[NT][2];                                    // keys that column 2j (+1) sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rr = row0 + nt * 8 + g;
      const bool live = nt * 8 + g < rows;
      const int tok = live ? rr / p.group : 0, hd = live ? rr - tok * p.group : 0;
      const long long at = (long long)(walk.q0 + tok) * p.q_ld + (long long)(walk.h * p.group + hd) * D + j * (D / 4);
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        float x[8];
        if (SPLIT == 1) {
          uint4 v = make_uint4(0u, 0u, 0u, 0u);
          if (live) v = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + at + 8 * w));
          qf[0][nt][2 * w][0] = v.x; qf[0][nt][2 * w][1] = v.y;
          qf[0][nt][2 * w + 1][0] = v.z; qf[0][nt][2 * w + 1][1] = v.w;
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += lo_bf16(u[i]) + hi_bf16(u[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (live) v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at + 8 * w + 4 * i));
            x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += x[i];
#pragma unroll
          for (int sp = 0; sp < SPLIT; ++sp)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              qf[sp][nt][2 * w + (i >> 1)][i & 1] = pack_bf16(x[2 * i], x[2 * i + 1]);
              x[2 * i] = bf16_rest(x[2 * i]);
              x[2 * i + 1] = bf16_rest(x[2 * i + 1]);
            }
        }
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = 2 * j + i;
        qs[nt][i] = __shfl_sync(0xffffffffu, sum, col * 4);
        const int cr = nt * 8 + col;
        lim[nt][i] = cr < rows ? (p.causal ? max(walk.kv_len - walk.q_len + (row0 + cr) / p.group + 1, 0) : walk.kv_len)
                               : walk.kv_len;
      }
    }
    const int lim_min = p.causal ? max(walk.kv_len - walk.q_len + row0 / p.group + 1, 0) : walk.kv_len;

    // A column's reference is `sub` once a key has been seen (`over`, 2^8 above it, is -inf until then).
    float o[NT][D / 16][4], sub[NT][2], over[NT][2], l[NT][2], pm[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) { over[nt][i] = -INFINITY; sub[nt][i] = l[nt][i] = pm[nt][i] = 0.f; }
#pragma unroll
      for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][mt][i] = 0.f;
    }

    for (int b = walk.b0; b < walk.b1; b += 2, ++taken) {
      const int s = taken % AQ_STAGES;
      // (after an abort the loop runs on without waiting: the barriers at the tile's end have all warps)
      if (!mbar_try_wait(&full[s], (taken / AQ_STAGES) & 1) && !*abort_flag &&
          !mbar_wait_parked(&full[s], (taken / AQ_STAGES) & 1, kWaitLimitNs)) {
        record_error(p.ws, PBSA_ERR_TIMEOUT, taken, K_Q4_ATTEND);
        *abort_flag = 1;
      }
      __syncwarp();
      const int here = meta[s];
      const uint8_t* blk = sm + s * 2 * Q::BYTES;
      int t0 = b * BT + warp * 16;                     // first of this warp's 16 tokens
      // both slots' instructions interleaved (one slot's chains do not fill the issue slots); a slot that is not
      // there is masked
#pragma unroll
      for (int u = 0; u < 2; ++u, blk += Q::BYTES, t0 += BT) {
        const bool there = (here >> u) & 1;
        uint32_t ka[W], kb[W];
        lds_words<W>(ka, blk + (warp * 16 + g) * Q::KROW + j * (D / 8));
        lds_words<W>(kb, blk + (warp * 16 + g + 8) * Q::KROW + j * (D / 8));
        const uint32_t* ksm = reinterpret_cast<const uint32_t*>(blk + Q::OFF_KS) + warp * 16 + g;
        const uint32_t* vsm = reinterpret_cast<const uint32_t*>(blk + Q::OFF_VS) + warp * 16 + g;
        const uint32_t ksa = ksm[0], ksb = ksm[8], vsa = vsm[0], vsb = vsm[8];
        uint32_t va[W], vb[W];
        lds_words<W>(va, blk + Q::OFF_V + warp * Q::UNIT + lane * Q::LANE);
        lds_words<W>(vb, blk + Q::OFF_V + warp * Q::UNIT + Q::UNIT / 2 + lane * Q::LANE);

        // scores: x[nt][0..1] of token g, [2..3] of token g + 8
        float x[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          // the codes carry 128 (bf16): starting at -128 sum(q) cancels it.  fp32 takes 136 from the codes.
          x[nt][0] = x[nt][2] = SPLIT == 1 ? -128.f * qs[nt][0] : 0.f;
          x[nt][1] = x[nt][3] = SPLIT == 1 ? -128.f * qs[nt][1] : 0.f;
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t a[2][4] = {{nibble_pair<0>(ka[w]), nibble_pair<0>(kb[w]), nibble_pair<1>(ka[w]), nibble_pair<1>(kb[w])},
                              {nibble_pair<2>(ka[w]), nibble_pair<2>(kb[w]), nibble_pair<3>(ka[w]), nibble_pair<3>(kb[w])}};
#pragma unroll
          for (int hp = 0; hp < 2; ++hp) {
            if (SPLIT != 1)
#pragma unroll
              for (int i = 0; i < 4; ++i) a[hp][i] = centred(a[hp][i]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int sp = SPLIT - 1; sp >= 0; --sp)
                mma_codes(x[nt], a[hp], qf[sp][nt][2 * w + hp][0], qf[sp][nt][2 * w + hp][1]);
          }
        }
        {
          const float sa = lo_bf16(ksa), sb = lo_bf16(ksb);
          const float ma = SPLIT == 1 ? hi_bf16(ksa) : fmaf(8.f, sa, hi_bf16(ksa));
          const float mb = SPLIT == 1 ? hi_bf16(ksb) : fmaf(8.f, sb, hi_bf16(ksb));
          const float sac = sa * c, sbc = sb * c, mac = ma * c, mbc = mb * c;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            x[nt][0] = fmaf(sac, x[nt][0], mac * qs[nt][0]);
            x[nt][1] = fmaf(sac, x[nt][1], mac * qs[nt][1]);
            x[nt][2] = fmaf(sbc, x[nt][2], mbc * qs[nt][0]);
            x[nt][3] = fmaf(sbc, x[nt][3], mbc * qs[nt][1]);
          }
        }
        float sva = lo_bf16(vsa), svb = lo_bf16(vsb);
        float mva = fmaf(8.f, sva, hi_bf16(vsa)), mvb = fmaf(8.f, svb, hi_bf16(vsb));
        const bool masked = !there || t0 + 16 > lim_min;          // some column does not see all 16 tokens
        if (masked) {
          // what lies behind the cached tokens was never written: its scales may be anything
          if (!there || t0 + g >= walk.kv_len) sva = mva = 0.f;
          if (!there || t0 + g + 8 >= walk.kv_len) svb = mvb = 0.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (!there || t0 + g + (i >> 1) * 8 >= lim[nt][i & 1]) x[nt][i] = -INFINITY;
        }
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) grow |= fmaxf(x[nt][i], x[nt][i + 2]) > over[nt][i];
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float mx = fmaxf(x[nt][i], x[nt][i + 2]);
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              if (mx > over[nt][i]) {
                // (nothing but zeros was summed before the first key)
                const float al = over[nt][i] == -INFINITY ? 1.f : ex2_approx(sub[nt][i] - mx);
                sub[nt][i] = mx;
                over[nt][i] = mx + 8.f;
                l[nt][i] *= al;
                pm[nt][i] *= al;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) { o[nt][mt][i] *= al; o[nt][mt][i + 2] *= al; }
              }
            }
        }
        uint32_t pb[SPLIT][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] = ex2_approx(x[nt][i] - sub[nt][i & 1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            l[nt][i] += e[i] + e[i + 2];
            pm[nt][i] = fmaf(e[i], mva, fmaf(e[i + 2], mvb, pm[nt][i]));
          }
          float y[4] = {e[0] * sva, e[1] * sva, e[2] * svb, e[3] * svb};
#pragma unroll
          for (int sp = 0; sp < SPLIT; ++sp) {
            pb[sp][nt][0] = transpose8(pack_bf16(y[0], y[1]));
            pb[sp][nt][1] = transpose8(pack_bf16(y[2], y[3]));
            if (sp + 1 < SPLIT)
#pragma unroll
              for (int i = 0; i < 4; ++i) y[i] = bf16_rest(y[i]);
          }
        }
        // value channels as rows: thread's channels are D/8 g .. in nibble order
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t a0[4] = {centred(nibble_pair<0>(va[w])), centred(nibble_pair<1>(va[w])),
                                  centred(nibble_pair<0>(vb[w])), centred(nibble_pair<1>(vb[w]))};
          const uint32_t a1[4] = {centred(nibble_pair<2>(va[w])), centred(nibble_pair<3>(va[w])),
                                  centred(nibble_pair<2>(vb[w])), centred(nibble_pair<3>(vb[w]))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int sp = SPLIT - 1; sp >= 0; --sp) {
              mma_codes(o[nt][2 * w], a0, pb[sp][nt][0], pb[sp][nt][1]);
              mma_codes(o[nt][2 * w + 1], a1, pb[sp][nt][0], pb[sp][nt][1]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ------------------------------------------------------------- the four warps' shares, joined
    float* ex_o = reinterpret_cast<float*>(sm + SM::EX_O);
    float2* ex_ml = reinterpret_cast<float2*>(sm + SM::EX_ML);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int s2 = 4; s2 < 32; s2 <<= 1) {
          l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], s2);
          pm[nt][i] += __shfl_xor_sync(0xffffffffu, pm[nt][i], s2);
        }
        const int col = nt * 8 + 2 * j + i;
        if (g == 0) ex_ml[warp * ROWS + col] = make_float2(over[nt][i] == -INFINITY ? -INFINITY : sub[nt][i], l[nt][i]);
        float* dst = ex_o + (size_t)(warp * ROWS + col) * SM::OSTRIDE + g * (D / 8);
#pragma unroll
        for (int mt = 0; mt < D / 16; mt += 2) {
          // rows g and g + 8 of value tile mt are channels 2 mt and 2 mt + 1 of this thread's D/8
          *reinterpret_cast<float4*>(dst + 2 * mt) =
              make_float4(o[nt][mt][i] + pm[nt][i], o[nt][mt][i + 2] + pm[nt][i], o[nt][mt + 1][i] + pm[nt][i],
                          o[nt][mt + 1][i + 2] + pm[nt][i]);
        }
      }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (!*abort_flag) {
      constexpr int CH = D / 4;                        // float4 per row
      for (int e = tid; e < rows * CH; e += AQ_WARPS * 32) {
        const int r = e / CH, ch = e - r * CH;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < AQ_WARPS; ++w) M = fmaxf(M, ex_ml[w * ROWS + r].x);
        float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < AQ_WARPS; ++w) {
          const float2 ml = ex_ml[w * ROWS + r];
          const float f = q4_weight(ml.x, M);
          const float4 v = *reinterpret_cast<const float4*>(ex_o + (size_t)(w * ROWS + r) * SM::OSTRIDE + 4 * ch);
          L = fmaf(f, ml.y, L);
          acc[0] = fmaf(f, v.x, acc[0]);
          acc[1] = fmaf(f, v.y, acc[1]);
          acc[2] = fmaf(f, v.z, acc[2]);
          acc[3] = fmaf(f, v.w, acc[3]);
        }
        if (walk.piece < 0) {
          q4_write_row<D>(p, walk.q0, row0 + r, walk.h, 4 * ch, acc, M, L, ch == 0);
        } else {
          *q4_few_place<D>(p.part_o, p.part_rows, walk.piece, r, ch) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          if (ch == 0) p.part_ml[(size_t)walk.piece * p.part_rows + r] = make_float2(M, L);
        }
      }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");     // the exchange is used again
  }
  if (tid == 0) p.desc[blockIdx.x] = walk.desc;
}

template <int D, int NT, int SPLIT>
cudaError_t launch_t(AttendQ4Params* p, bool many, int* grid, cudaStream_t st) {
  auto kern = attend_q4_kernel<D, NT, SPLIT>;
  constexpr int smem = AqSmem<D, NT>::TOTAL;
  cudaError_t e = set_smem_once((const void*)kern, smem);
  if (e != cudaSuccess) return e;
  p->part_rows = AqSmem<D, NT>::ROWS;
  const int per_sm = NT == 1 && SPLIT == 1 ? 3 : 2;
  int sms = 0, dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  *grid = sms * per_sm < Q4_MAX_CTAS ? sms * per_sm : Q4_MAX_CTAS;
  p->few_ctas = many ? *grid : 0;
  kern<<<*grid, AQ_THREADS, smem, st>>>(*p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(AttendQ4Params p, int dtype, int max_rows, cudaStream_t st) {
  Q4JoinParams j = {};
  // some may go to the tensor-core kernel, which the lengths decide (q4_share)
  const bool many = dtype == PBSA_BF16 && max_rows > Q4_TC_ROWS;
  p.max_rows = max_rows;
  cudaError_t e = dtype == PBSA_F32 ? launch_t<D, 1, 3>(&p, false, &j.few, st)
                  : max_rows <= 8   ? launch_t<D, 1, 1>(&p, false, &j.few, st)
                                    : launch_t<D, 2, 1>(&p, many, &j.few, st);
  if (e != cudaSuccess) return e;
  j.p = p;
  if (many) {
    // its pieces lie behind the others: the two kernels may run at the same time
    j.tc_desc = p.desc += Q4_MAX_CTAS;
    j.tc_ml = p.part_ml += Q4_FEW_ROWS;
    j.tc_o = p.part_o += (size_t)Q4_FEW_ROWS * D;
    if ((e = launch_attend_q4_tc(p, D, &j.tc, &j.tc_rows, st)) != cudaSuccess) return e;
  }
  cudaLaunchAttribute late;
  const cudaLaunchConfig_t cfg = q4_dependent(j.few + 4 * j.tc, 256, 0, st, &late);
  return cudaLaunchKernelEx(&cfg, attend_q4_join_kernel<D>, j);
}

}  // namespace

size_t attend_q4_ws_bytes(int d) {
  // descriptors, then the sums and the rows of two pieces a CTA
  return (size_t)WS_HEADER_BYTES + (Q4_MAX_CTAS + Q4_TC_MAX_CTAS) * sizeof(Q4Desc) + (size_t)Q4_PART_ROWS * (8 + 4 * (size_t)d);
}

cudaError_t launch_attend_q4(const AttendQ4Params& in, int d, int dtype, int max_rows, cudaStream_t st) {
  AttendQ4Params p = in;
  uint8_t* w = static_cast<uint8_t*>(p.ws) + WS_HEADER_BYTES;
  p.desc = reinterpret_cast<Q4Desc*>(w);
  w += (Q4_MAX_CTAS + Q4_TC_MAX_CTAS) * sizeof(Q4Desc);
  p.part_ml = reinterpret_cast<float2*>(w);
  w += (size_t)Q4_PART_ROWS * sizeof(float2);
  p.part_o = reinterpret_cast<float*>(w);
  return d == 128 ? launch_d<128>(p, dtype, max_rows, st) : launch_d<64>(p, dtype, max_rows, st);
}

}  // namespace pbsa

// Attention of the requests' queries over the 4-bit cache: the form for many query rows (bf16), on the
// 5th-generation tensor cores.
//
// The mathematics is attend_q4.cu's.  128 rows (row = token * group + head of the group, so the heads that
// share a kv head share its keys) fill one M = 128 tile, and every cached byte is used for all rows of a
// tile: the products, the exponentials and the unpacking of the codes bound it.
//  * Work: the line of attend_q4.cuh, with tiles of 256 rows in two halves, so that a key unpacked once serves
//    both; one CTA per SM, pieces one after another (one warp walks them and tells the others).  With the causal rule
//    a tile is charged what it sees, so long prompts are spread evenly.  The kernel runs as a programmatic dependent
//    beside the few-rows kernel's last CTAs, from which it reads nothing.
//  * Each step covers two blocks (128 keys).  One thread each brings K's and V's bytes with bulk copies;
//    two warpgroups, alternate steps, unpack them into shared-memory operand tiles (128-byte swizzle): K as
//    the codes themselves (plus 128, exact in bf16), V as bf16 values s*c + m, rounded once (pbsa_expand_q4 rounds to fp32
//    first, so a value next to the middle of two bf16 numbers may differ by a step).  The scores carry no rounding of K
//    (to bf16 it would put 2^-8 |q . k| / sqrt(d) of noise into each):
//      q . k = s (q . (c + 128) + (m / s - 128) sum(q)).
//    The bracket is one product: (m / s - 128) and sum(q) as three bf16 terms each make a further slice of 16
//    columns of K and Q.  The scale, times the softmax scale, is applied to the scores in fp32, together with the
//    subtraction of the reference: one multiply-add a pair.  (Read as bf16, half the shared-memory reads for three more
//    instructions a pair, chunk and prompts took 2% and 4% longer.)
//  * The halves take turns on the tensor pipe: while one's scores are exponentiated (a warpgroup each, a row
//    a thread), the other's P V and next Q K^T run.  TMEM: S and O of each half (512 columns at D = 128), P as
//    bf16 over S; S(i+1) is issued behind PV(i) by the half's own thread.
//  * The softmax makes one pass over a step's scores: scale, exponential, sum and maximum together, against the
//    reference that the steps before left; P waits in registers, so the pass can be repeated from S where
//    scores exceed the reference by 2^64.  Above 2^8 the reference moves for the next step (O is rescaled then).
//  * All barriers are used once per step with a step count that runs on over the pieces (a piece without
//    blocks takes part in none; a half without rows in none of its own.  A thread that
//    waits on a barrier waits on each of its completions, as a parity tells only neighbours apart).  The ring of key
//    scales has four places: step n's are written once QK(n-2) is done, which follows the softmax of step n-3.
//  * Keys that a row does not see get x = -inf by a select after the scale is applied, and V of tokens
//    that are not cached is zero, so whatever bytes lie there reach no row.
// Waits are bounded; on expiry the error is recorded and every role runs through its pieces without
// waiting, drains its copies and MMAs, frees TMEM and returns.
//
// Measured (D = 128): 4608 tokens of 12 heads over 13824, without the causal rule: 647-681 us, 575-605 TFLOP/s (0.34-0.36 of
// the measured 1685); three prompts of 700 .. 2048 tokens of 32 heads (8 kv heads) over 1000 .. 14000: 937-952 us, 565-570
// TFLOP/s.  The same 4608 tokens over whole blocks that pbsa_expand_q4 has written out take pbsa_attend 305 us, 321-327
// with the expansion (K rounded to bf16 there): a key is unpacked once a call and not once for each of 18 row tiles.
// A step of 256 rows and 128 keys lasts about 5900 cycles; its MMAs take 2800 of the tensor pipe's, its exponentials
// 2048 of either unit's.  What bounds it is the chain of a half: a pass over 128 scores a thread (about
// 2900 cycles, the unpacking and the other half in the same issue slots), then 2300 until P V and the next Q K^T have
// given the next S.  TMEM holds S and O of two halves and no third.  Earlier forms, when the chunk took 707 us and the
// prompts 1168: two threads a row 819 and 1219 (registers), the maximum found before the exponentials 799 and 1205;
// 256-row tiles then gave 701 and 1083.  A start and end of a tile cost about 12000 cycles.  A first reference of zero
// instead of a first pass for the maximum: 668 and 966 us for 654 and 944; K unpacked before Q: 653 and 941.
#include <math.h>

#include "attend_q4.cuh"

namespace pbsa {
namespace {

constexpr int TQ_THREADS = 640;      // warpgroups: control, unpack x 2, softmax x 2
constexpr int TQ_ROWS = 256;         // two halves of 128
// Blocks that are worth a CTA: with 4, 8, 16 and 32 64 tokens of 8 heads over 2 and 30000 tokens take 58, 54, 61 and 84 us, 512
// tokens of 12 heads over 2500 53, 53, 63 and 91, two requests of 256 tokens of 8 heads over 8000 64, 64, 63 and 86.
constexpr int TQ_MIN_STEPS = 8;
// Blocks that a tile's start and end and its second passes over masked steps cost: charged 0, 8, 12, 16 and 24, the three
// prompts take 1063, 1003, 984, 984 and 1009 us, the chunk of 4608 tokens 672, 661, 664, 669 and 677.
constexpr int TQ_TILE_COST = 12;
constexpr int STAGES = 2, SCS = 4;   // operand stages of K and of V, key scales
constexpr uint32_t REG_CTRL = 48, REG_UNPACK = 80, REG_SOFT = 136;   // launched with 96: 48 + 2*80 + 2*136 = 5*96
static_assert(REG_CTRL + 2 * REG_UNPACK + 2 * REG_SOFT <= 5 * 96, "register split exceeds the launch");

enum { T_QFULL = 0, T_CFULL = 1,                                    // codes: of K for either warpgroup, of V
       T_CEMPTY = T_CFULL + 4,                                      // of K, of V
       T_KFULL = T_CEMPTY + 2, T_KEMPTY = T_KFULL + STAGES, T_VFULL = T_KEMPTY + STAGES, T_VEMPTY = T_VFULL + STAGES,
       T_SCFULL = T_VEMPTY + STAGES, T_SFULL = T_SCFULL + SCS, T_PFULL = T_SFULL + 2, T_MMADONE = T_PFULL + 2,   // of a half
       T_TURN = T_MMADONE + 2, T_WFULL = T_TURN + 2, T_WEMPTY = T_WFULL + 2, T_BARS = T_WEMPTY + 2 };
constexpr int WARPS_TOLD = 19;       // warps that read the pieces: all but the one that walks them

// A piece of the CTA's share, as the walking warp passes it on.
struct TqPiece {
  int more, r, b0, b1, mt, h, q0, q_len, kv_len, rows, piece, pad;
};

template <int D>
struct TqSmem {
  static constexpr uint32_t PANELS = D / 64;
  static constexpr uint32_t TILE = PANELS * 16384;                  // 128 rows of 64 columns a panel
  static constexpr uint32_t STEP = 2 * Q4<D>::HALF;                 // two blocks' K codes, or V codes
  static constexpr uint32_t Q = 0;                                  // two halves
  static constexpr uint32_t K = 2 * TILE;
  static constexpr uint32_t V = K + STAGES * TILE;
  static constexpr uint32_t QX = V + STAGES * TILE;                 // 8 more columns of Q's halves: [128 rows][8] bf16
  static constexpr uint32_t KX = QX + 2 * 2048;                     // ... of each K stage
  static constexpr uint32_t ZERO = KX + STAGES * 2048;              // ... and 8 of zeros behind either
  static constexpr uint32_t CODES = ZERO + 2048;                    // a step's K codes, and its V codes
  static constexpr uint32_t SC = CODES + 2 * STEP;                  // float [SCS][128]: scales of the step's keys
  static constexpr uint32_t ONES = SC + SCS * 512;                  // float [128]: of scores that have theirs
  static constexpr uint32_t BARS = ONES + 512;
  static constexpr uint32_t WALK = BARS + T_BARS * 8;               // TqPiece [2]
  static constexpr uint32_t META = WALK + 2 * sizeof(TqPiece);      // int [2][2], int [SCS], TMEM address, abort flag
  static constexpr uint32_t TOTAL = META + 4 * (4 + SCS + 2);
  static constexpr uint32_t BYTES = TOTAL + 1024;
};
static_assert(TqSmem<128>::BYTES <= 232448, "shared memory");

// Pairs of fp32 in 64-bit registers (packed f32x2 arithmetic), kept packed so that no moves pair them up.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(uint32_t lo, uint32_t hi) {
  f32x2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ f32x2 pair(float lo, float hi) { return pair(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ void parts(f32x2 d, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ f32x2 fma2(f32x2 x, f32x2 y, f32x2 z) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
  return d;
}
__device__ __forceinline__ f32x2 add2(f32x2 x, f32x2 y) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
  return d;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// Shared-memory matrix descriptor of 16 columns without swizzle: two blocks of 8 columns, 16 bytes a row, the second
// `next` bytes behind the first.
__device__ __forceinline__ uint64_t plain_desc(uint32_t smem_addr, uint32_t next) {
  return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | (uint64_t)(next >> 4) << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}
// 16 columns of 32 lanes (see tmem_ld32)
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// The wait for tmem_ld16's values, tied to those values alone: arithmetic of other columns may move across it.
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

template <int D>
__global__ void __launch_bounds__(TQ_THREADS, 1) attend_q4_tc_kernel(const AttendQ4Params p) {
  using Q = Q4<D>;
  using SM = TqSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::BARS);
  volatile int* meta = reinterpret_cast<volatile int*>(sm + SM::META);          // [2][2]: the block is there (K, V)
  volatile int* sc_ok = meta + 4;                                         // [SCS]: the same, two bits
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + SM::META) + 4 + SCS;
  volatile int* abort_flag = meta + 4 + SCS + 1;
  __shared__ Q4Start start_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < T_BARS; ++i) {
      const bool full = i == T_CEMPTY || i == T_CEMPTY + 1 || (i >= T_KFULL && i < T_KEMPTY) || (i >= T_VFULL && i < T_VEMPTY) ||
                        (i >= T_SCFULL && i < T_SFULL) || (i >= T_PFULL && i < T_MMADONE) || i == T_TURN || i == T_TURN + 1;
      const bool both = (i >= T_KEMPTY && i < T_VFULL) || (i >= T_VEMPTY && i < T_SCFULL);
      mbar_init(&bars[i], full ? 128 : both ? 2 : i == T_QFULL ? 256 : i >= T_WEMPTY ? WARPS_TOLD : 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (tid < 128) reinterpret_cast<float*>(sm + SM::ONES)[tid] = 1.f;
  if (tid < 512) reinterpret_cast<uint32_t*>(sm + SM::ZERO)[tid] = 0u;
  fence_proxy_async_smem();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const Q4Share share = q4_share<TQ_THREADS, true>(p, TQ_ROWS, TQ_TILE_COST, TQ_MIN_STEPS, &start_s);   // has block barriers
  if (share.x0 >= share.x1) {   // (often all CTAs: see there)
    if (tid == 0) p.desc[blockIdx.x].pieces = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  auto wait = [&](int bar, uint32_t parity) {
    if (*abort_flag) return;
    if (!mbar_wait_parked(&bars[bar], parity, kWaitLimitNs)) {
      record_error(p.ws, PBSA_ERR_TIMEOUT, bar, K_Q4_ATTEND);
      *abort_flag = 1;
    }
  };

  // The k-th piece, for a whole warp (not cut short by an abort: every role goes through every piece).
  auto told = [&](int k) {
    if (!mbar_wait_parked(&bars[T_WFULL + (k & 1)], (k >> 1) & 1, 2 * kWaitLimitNs)) *abort_flag = 1;
    const TqPiece w = reinterpret_cast<const TqPiece*>(sm + SM::WALK)[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars[T_WEMPTY + (k & 1)]);
    return w;
  };

  if (warp < 4) {
    setmaxnreg_dec<REG_CTRL>();
    if (warp == 2) {
      // ------------------------------------------------------------- walks the share
      if (lane == 0) {
        Q4Walk walk(p, share, start_s, TQ_ROWS, TQ_TILE_COST);
        bool more = true;
        for (int k = 0; more; ++k) {
          more = walk.next();
          if (!mbar_wait_parked(&bars[T_WEMPTY + (k & 1)], ((k >> 1) & 1) ^ 1, 2 * kWaitLimitNs)) *abort_flag = 1;
          reinterpret_cast<TqPiece*>(sm + SM::WALK)[k & 1] = {more ? 1 : 0, walk.r, walk.b0, walk.b1, walk.mt, walk.h,
                                                             walk.q0, walk.q_len, walk.kv_len, walk.rows, walk.piece, 0};
          mbar_arrive(&bars[T_WFULL + (k & 1)]);
        }
        p.desc[blockIdx.x] = walk.desc;
      }
      __syncwarp();
    }
    if (warp == 0) {
      // ------------------------------------------------------------- slots' bytes
      int n = 0;   // step (lane 0 brings K codes, lane 1 V codes, each at its own pace)
      for (int k = 0;; ++k) {
        const TqPiece walk = told(k);
        if (!walk.more) break;
        if (lane < 2) {
          const int* row = p.table + (size_t)walk.r * p.table_ld;
          const uint8_t* src = p.pool + (size_t)walk.h * p.pool_slots * Q::BYTES + lane * Q::HALF;
          int next0 = walk.b0 < walk.b1 ? __ldg(row + walk.b0) : -1;
          int next1 = walk.b0 + 1 < walk.b1 ? __ldg(row + walk.b0 + 1) : -1;
          for (int b = walk.b0; b < walk.b1 && !*abort_flag; b += 2) {
            const int slot0 = next0, slot1 = next1;
            const bool has1 = b + 1 < walk.b1;
            if (b + 2 < walk.b1) next0 = __ldg(row + b + 2);
            if (b + 3 < walk.b1) next1 = __ldg(row + b + 3);
            const int cs = lane;
            wait(T_CEMPTY + cs, (n & 1) ^ 1);
            if (*abort_flag) break;
            const bool ok0 = slot0 >= 0 && slot0 < p.pool_slots, ok1 = has1 && slot1 >= 0 && slot1 < p.pool_slots;
            if (!ok0) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot0, K_Q4_ATTEND);
            if (has1 && !ok1) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot1, K_Q4_ATTEND);
            meta[2 * cs] = ok0;
            meta[2 * cs + 1] = ok1;
            uint8_t* dst = sm + SM::CODES + cs * SM::STEP;
            const uint32_t bytes = (ok0 ? Q::HALF : 0) + (ok1 ? Q::HALF : 0);
            uint64_t* full = &bars[T_CFULL + 2 * cs + (n & 1)];   // a barrier a warpgroup: neither sees every step
            if (bytes > 0) mbar_arrive_expect_tx(full, bytes);
            else mbar_arrive(full);
            if (ok0) bulk_load(dst, src + (size_t)slot0 * Q::BYTES, Q::HALF, full);
            if (ok1) bulk_load(dst + Q::HALF, src + (size_t)slot1 * Q::BYTES, Q::HALF, full);
            ++n;
          }
        }
        __syncwarp();
      }
      // the CTA must not end with copies in flight
      if (lane < 2 && n > 0) mbar_wait(&bars[T_CFULL + 2 * lane + ((n - 1) & 1)], ((n - 1) >> 1) & 1, kWaitLimitNs);
      __syncwarp();
    }
    if (warp == 1 || warp == 3) {
      // ------------------------------------------------------------- MMA issuers, one for each half
      const uint32_t w = warp >> 1;
      {
        const uint32_t tS = tmem + w * 128, tO = tmem + 256 + w * 128;
        const uint64_t dq = sw128_desc(smem_u32(sm + SM::Q + w * SM::TILE), 16, 1024);
        const uint64_t dk = sw128_desc(smem_u32(sm + SM::K), 16, 1024);
        const uint64_t dv = sw128_desc(smem_u32(sm + SM::V), 16384, 1024);
        const uint64_t dqx = plain_desc(smem_u32(sm + SM::QX + w * 2048), SM::ZERO - SM::QX - w * 2048);
        constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128, 0, 0), IDESC_PV = idesc_bf16_f32(128, D, 0, 1);
        auto issue_qk = [&](int n) {
          const int sk = n % STAGES;
          wait(T_KFULL + sk, (n / STAGES) & 1);
          if (*abort_flag) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
            mma_bf16_ss(tS, dq + off, dk + ((sk * SM::TILE) >> 4) + off, IDESC_QK, kk > 0 ? 1u : 0u);
          }
          mma_bf16_ss(tS, dqx, plain_desc(smem_u32(sm + SM::KX + sk * 2048), SM::ZERO - SM::KX - sk * 2048), IDESC_QK, 1u);
          mma_commit(&bars[T_SFULL + w]);
          mma_commit(&bars[T_KEMPTY + sk]);
        };
        int n0 = 0, piece = 0, used = 0, done = 0;   // used, done: steps and pieces that this half has taken part in
        for (int k = 0;; ++k) {
          const TqPiece walk = told(k);
          if (!walk.more) break;
          if (walk.b0 == walk.b1) continue;
          const int n1 = n0 + ((walk.b1 - walk.b0 + 1) >> 1);
          const bool takes_part = w == 0 || walk.rows > walk.mt * TQ_ROWS + 128;
          if (lane == 0) {
            wait(T_QFULL, piece & 1);
            if (takes_part) {
              issue_qk(n0);
              for (int n = n0; n < n1 && !*abort_flag; ++n) {
                const int sv = n % STAGES;
                wait(T_PFULL + w, (used + n - n0) & 1);
                wait(T_VFULL + sv, (n / STAGES) & 1);
                if (*abort_flag) break;
                tc_fence_after();
                // P(n) lies over S(n): S(n+1) is issued behind its use, in order
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                  mma_bf16_ts(tO, tS + kk * 8, dv + ((sv * SM::TILE + kk * 2048) >> 4), IDESC_PV, (n > n0 || kk > 0) ? 1u : 0u);
                mma_commit(&bars[T_VEMPTY + sv]);
                if (n + 1 < n1) issue_qk(n + 1);
              }
            } else {
              for (int n = n0; n < n1 && !*abort_flag; ++n) {   // the stages go round without this half
                wait(T_KFULL + n % STAGES, (n / STAGES) & 1);
                mbar_arrive(&bars[T_KEMPTY + n % STAGES]);
                wait(T_VFULL + n % STAGES, (n / STAGES) & 1);
                mbar_arrive(&bars[T_VEMPTY + n % STAGES]);
              }
            }
            if (takes_part) {   // all MMAs of this half: its O is complete, its Q is free
              mma_commit(&bars[T_MMADONE + w]);
              mbar_wait(&bars[T_MMADONE + w], done & 1, kWaitLimitNs);
            }
          }
          __syncwarp();
          if (takes_part) {
            used += n1 - n0;
            ++done;
          }
          n0 = n1;
          ++piece;
        }
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    setmaxnreg_dec<REG_UNPACK>();
    // --------------------------------------------------------------- unpack: steps of the warpgroup's parity
    const int ug = (warp - 4) >> 2, t = tid & 127, uw = warp & 3;
    int n = 0, done0 = 0, done1 = 0;   // pieces that the halves have taken part in
    for (int k = 0;; ++k) {
      const TqPiece walk = told(k);
      if (!walk.more) break;
      if (walk.b0 == walk.b1) continue;
      // Q: a row a thread, and its sum
      if (done0 > 0) wait(T_MMADONE, (done0 - 1) & 1);
      if (done1 > 0) wait(T_MMADONE + 1, (done1 - 1) & 1);
      ++done0;
      if (walk.rows > walk.mt * TQ_ROWS + 128) ++done1;
      {
        const int rr = walk.mt * TQ_ROWS + ug * 128 + t;
        const bool live = rr < walk.rows;
        const int tok = live ? rr / p.group : 0, hd = live ? rr - tok * p.group : 0;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) +
                                                          (long long)(walk.q0 + tok) * p.q_ld +
                                                          (long long)(walk.h * p.group + hd) * D);
        uint8_t* dst = sm + SM::Q + ug * SM::TILE + t * 128;
        float sum = 0.f;
#pragma unroll 4
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = live ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) sum += lo_bf16(u[i]) + hi_bf16(u[i]);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + (((c & 7) ^ (t & 7)) << 4)) = v;
        }
        // the row's sum as three bf16 terms, beside which a key has three of its offset: columns
        // (1, 2, 3, 1, 2, 1) of the one against (1, 1, 1, 2, 2, 3) of the other
        const float s2 = bf16_rest(sum), s3 = bf16_rest(s2);
        *reinterpret_cast<uint4*>(sm + SM::QX + ug * 2048 + t * 16) =
            make_uint4(pack_bf16(sum, s2), pack_bf16(s3, sum), pack_bf16(s2, sum), 0u);
        fence_proxy_async_smem();
        mbar_arrive(&bars[T_QFULL]);
      }
      const int n1 = n + ((walk.b1 - walk.b0 + 1) >> 1), start = n, first = n + ((n ^ ug) & 1);
      auto unpack_k = [&](int n) {
        const int sk = n % STAGES;
        wait(T_CFULL + ug, (n >> 1) & 1);
        const uint8_t* codes = sm + SM::CODES;
        // K: 16 (D = 64: 8) code bytes a lane; 8 lanes write 4 rows of two neighbouring column groups, 8
        // different 16-byte columns after the swizzle.  All of a thread's codes are read before the first is used.
        {
          constexpr int W = Q::WORDS;                   // words of a lane's bytes; 4 lanes a row
          const int row8 = ((lane >> 4) & 1) * 4 + ((lane >> 1) & 3), j = ((lane >> 3) & 1) * 2 + (lane & 1);
          const int row0 = uw * 32 + row8;              // key of the step; + 8 a turn
          const uint8_t* src = codes + (uw >> 1) * Q::HALF + (row0 & 63) * Q::KROW + j * Q::LANE;
          uint32_t w[4][W];
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            if (W == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(src + it * 8 * Q::KROW);
              w[it][0] = v.x; w[it][1] = v.y; w[it][W - 2] = v.z; w[it][W - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(src + it * 8 * Q::KROW);
              w[it][0] = v.x; w[it][1] = v.y;
            }
          }
          uint8_t* dst = sm + SM::K + sk * SM::TILE + ((j * W) >> 3) * 16384 + row0 * 128;
          const uint32_t ksm = *reinterpret_cast<const uint32_t*>(codes + (t >> 6) * Q::HALF + Q::OFF_KS + (t & 63) * 4);
          const int there = (meta[0] ? 1 : 0) | (meta[1] ? 2 : 0);
          mbar_arrive(&bars[T_CEMPTY]);
          wait(T_KEMPTY + sk, ((n / STAGES) & 1) ^ 1);   // QK(n-2) is done, and before it the softmax of step n-3
          {   // key t: its scale, and what the sum of the row is multiplied by (see the top of the file)
            const float m = hi_bf16(ksm);
            float s = lo_bf16(ksm);
            // A scale of 0 (all channels are m, all codes 0): the product is (128 + r) sum(q) = m / s sum(q) in any s.  One far
            // below the minimum keeps what the two large terms leave of their roundings, 2^-20 of 128 s |q|, below the
            // score's own; with s = |m| (1 for zeros) it was up to 2^-13 of m |q|.
            if (s == 0.f) s = fmaxf(fabsf(m) * 0x1p-12f, 0x1p-126f);
            const float r = __fdiv_rn(m, s) - 128.f;
            const float r2 = bf16_rest(r), r3 = bf16_rest(r2);
            const uint32_t r11 = pack_bf16(r, r);
            *reinterpret_cast<uint4*>(sm + SM::KX + sk * 2048 + t * 16) =
                make_uint4(r11, pack_bf16(r, r2), pack_bf16(r2, r3), 0u);
            reinterpret_cast<float*>(sm + SM::SC)[(n % SCS) * 128 + t] = s * p.scale_log2;
            if (t == 0) sc_ok[n % SCS] = there;
            mbar_arrive(&bars[T_SCFULL + n % SCS]);
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const int at = (((j * W + i) & 7) ^ row8) << 4;   // 16-byte column, swizzled
#pragma unroll
            for (int it = 0; it < 4; ++it)
              *reinterpret_cast<uint4*>(dst + it * 1024 + at) = make_uint4(
                  nibble_pair<0>(w[it][i]), nibble_pair<1>(w[it][i]), nibble_pair<2>(w[it][i]), nibble_pair<3>(w[it][i]));
          }
          fence_proxy_async_smem();
          mbar_arrive(&bars[T_KFULL + sk]);
        }
      };
      if (first < n1) unpack_k(first);
      for (n = first; n < n1; n += 2) {
        if (n + 2 < n1) unpack_k(n + 2);   // V(n) may have to wait for PV(n-2); the next S does not
        const int b = walk.b0 + 2 * (n - start), sv = n % STAGES;
        wait(T_CFULL + 2 + ug, (n >> 1) & 1);
        const uint8_t* codes = sm + SM::CODES + SM::STEP;
        const bool ok0 = meta[2] != 0, ok1 = meta[3] != 0;
        // V: 8 channels of two tokens a lane and turn, a block's turns together
        {
          constexpr int HALVES = D / 64;                // 8-channel halves of a lane's bytes in the layout
          constexpr int PER = 8 * 4 * HALVES;           // threads of 8 tokens
          constexpr int GROUPS = 128 / PER, TURNS = 8 / GROUPS;
          const int k = t % HALVES, j = (t / HALVES) & 3, g = (t / (HALVES * 4)) & 7, u8 = t / PER;
          const int col = g * HALVES + k, row0 = u8 * 8 + 2 * j;
          const int at0 = ((col & 7) ^ (2 * j)) << 4, at1 = 128 + (((col & 7) ^ (2 * j + 1)) << 4);
          uint8_t* dst = sm + SM::V + sv * SM::TILE + (col >> 3) * 16384 + row0 * 128;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint8_t* blk = codes + half * Q::HALF;
            const uint8_t* src = blk + (u8 * 32 + g * 4 + j) * Q::LANE + 8 * k;
            uint2 w[TURNS], sc[TURNS];
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
              w[i] = *reinterpret_cast<const uint2*>(src + i * GROUPS * 32 * Q::LANE);
              sc[i] = *reinterpret_cast<const uint2*>(blk + Q::CODE + (row0 + i * GROUPS * 8) * 4);
            }
            // tokens of this block that are cached (none of a block that is not there)
            const int left = (half ? ok1 : ok0) ? walk.kv_len - (b + half) * BT : 0;
            if (left < BT) {
#pragma unroll
              for (int i = 0; i < TURNS; ++i) {
                if (row0 + i * GROUPS * 8 >= left) sc[i].x = 0u;
                if (row0 + i * GROUPS * 8 + 1 >= left) sc[i].y = 0u;
              }
            }
            if (half == 1) mbar_arrive(&bars[T_CEMPTY + 1]);   // all codes have been read
            if (half == 0) wait(T_VEMPTY + sv, ((n / STAGES) & 1) ^ 1);
#pragma unroll
            for (int i = 0; i < TURNS; ++i) {
              const uint32_t s0 = __byte_perm(sc[i].x, 0, 0x1010), m0 = __byte_perm(sc[i].x, 0, 0x3232);
              const uint32_t s1 = __byte_perm(sc[i].y, 0, 0x1010), m1 = __byte_perm(sc[i].y, 0, 0x3232);
              const uint32_t y[8] = {nibble_pair<0>(w[i].x), nibble_pair<1>(w[i].x), nibble_pair<2>(w[i].x),
                                     nibble_pair<3>(w[i].x), nibble_pair<0>(w[i].y), nibble_pair<1>(w[i].y),
                                     nibble_pair<2>(w[i].y), nibble_pair<3>(w[i].y)};
              uint32_t a[4], c[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t lo = sub_bf16x2(y[2 * q], 0x43004300u), hi = sub_bf16x2(y[2 * q + 1], 0x43004300u);
                a[q] = fma_bf16x2(__byte_perm(lo, hi, 0x5410), s0, m0);
                c[q] = fma_bf16x2(__byte_perm(lo, hi, 0x7632), s1, m1);
              }
              uint8_t* to = dst + half * 8192 + i * GROUPS * 1024;
              *reinterpret_cast<uint4*>(to + at0) = make_uint4(a[0], a[1], a[2], a[3]);
              *reinterpret_cast<uint4*>(to + at1) = make_uint4(c[0], c[1], c[2], c[3]);
            }
          }
          fence_proxy_async_smem();
          mbar_arrive(&bars[T_VFULL + sv]);
        }
      }
      n = n1;
    }
  } else {
    setmaxnreg_inc<REG_SOFT>();
    // --------------------------------------------------------------- softmax, a warpgroup for each half
    const int half = (warp - 12) >> 2;
    const int wq = warp & 3;                 // TMEM lane quadrant this warp may access
    const int row = wq * 32 + lane;          // of the half
    const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
    const uint32_t tS = tmem + lane_off + half * 128, tO = tmem + lane_off + 256 + half * 128;
    int n0 = 0, used = 0, done = 0, turn = 0;   // turn: steps that both halves have taken part in
    for (int k = 0;; ++k) {
      const TqPiece walk = told(k);
      if (!walk.more) break;
      const int n1 = n0 + ((walk.b1 - walk.b0 + 1) >> 1);
      const int rr = walk.mt * TQ_ROWS + half * 128 + row;
      const bool live = rr < walk.rows, both = walk.rows > walk.mt * TQ_ROWS + 128, takes_part = half == 0 || both;
      if (walk.b0 == walk.b1) {   // nothing to see: no other role takes part
        if (live) {
          const float zero[4] = {0.f, 0.f, 0.f, 0.f};
          for (int ch = 0; ch < D; ch += 4) {
            if (walk.piece < 0)
              q4_write_row<D>(p, walk.q0, rr, walk.h, ch, zero, -INFINITY, 0.f, ch == 0);
            else
              *q4_tc_place<D>(p.part_o, p.part_rows, walk.piece, half * 128 + row, ch / 4) = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          if (walk.piece >= 0) p.part_ml[(size_t)walk.piece * p.part_rows + half * 128 + row] = make_float2(-INFINITY, 0.f);
        }
        continue;
      }
      // l and O are sums against the reference M; R is the next step's
      float M = -INFINITY, R = -INFINITY, l = 0.f;
      const int lim = live && p.causal ? max(walk.kv_len - walk.q_len + rr / p.group + 1, 0) : walk.kv_len;
      for (int n = n0; takes_part && n < n1; ++n, ++used) {
        wait(T_SFULL + half, used & 1);
        // (complete by now; waited for only after S, as this half may have skipped pieces and so completions)
        wait(T_SCFULL + n % SCS, (n / SCS) & 1);
        const float4* s4 = reinterpret_cast<const float4*>(sm + SM::SC) + (n % SCS) * 32;   // of 4 keys: s * scale * log2 e
        const int ok = sc_ok[n % SCS];
        if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
        tc_fence_after();
        const int see = lim - (walk.b0 + 2 * (n - n0)) * BT;    // of the step's keys
        float top = -INFINITY, psum;
        uint32_t pk[64];
        // Plain: one pass over S.  Careful, where keys are masked, where no key has been seen yet, where R is so
        // large that its rounding in the fused product would count, and where a plain pass has met scores above
        // R + 64 (P could pass its range): x is first written over S and its maximum found, R moves up to it if
        // need be, and the maximum less itself is zero however large it is.
        bool careful = __any_sync(0xffffffffu, see < 128 || R == -INFINITY || fabsf(R) > 4096.f) || ok != 3;
        bool plain = true, passed = false;
        // The halves take turns, so that one's pass runs beside the other's products; the turn is passed on after six
        // of eight chunks (after four, five, six and seven the chunk of 4608 tokens takes 681, 675, 668 and 696 us, without
        // turns 727).
        if (both && (half == 1 || turn > 0)) wait(T_TURN + (half ^ 1), (half == 1 ? turn : turn - 1) & 1);
#pragma unroll 1
        while (true) {
          if (careful && plain) {
            plain = false;
            top = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t x[32];
              tmem_ld32(tS + q * 32, x);
              tmem_wait_ld();
              const int to = (ok >> (q >> 1)) & 1 ? see - q * 32 : 0;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 sc = s4[q * 8 + e / 4];
                const float sw[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float a = __uint_as_float(x[e + i]) * sw[i];
                  x[e + i] = __float_as_uint(to <= e + i ? -INFINITY : a);
                }
                top = fmax3(fmax3(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1])), __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
              }
              tmem_st32(tS + q * 32, x);
            }
            tmem_wait_st();
            s4 = reinterpret_cast<const float4*>(sm + SM::ONES);
            if (R == -INFINITY || top > R + 64.f) R = top;
          }
          const float neg = R == -INFINITY ? 0.f : -R;
          const f32x2 neg2 = pair(neg, neg);
          float mx0 = -INFINITY, mx1 = -INFINITY;
          f32x2 sum0 = 0ull, sum1 = 0ull;
          uint32_t x[2][16];
          tmem_ld16(tS, x[0]);
          float4 sc[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[0][i] = s4[i];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            if (q == 6 && both && !passed) {
              passed = true;
              mbar_arrive(&bars[T_TURN + half]);
              ++turn;
            }
            tmem_wait16(x[q & 1]);
            if (q < 7) {
              tmem_ld16(tS + (q + 1) * 16, x[(q + 1) & 1]);   // in flight behind this chunk
#pragma unroll
              for (int i = 0; i < 4; ++i) sc[(q + 1) & 1][i] = s4[q * 4 + 4 + i];
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
              const float4 s = sc[q & 1][e / 4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float y0, y1;
                parts(fma2(pair(x[q & 1][e + 2 * i], x[q & 1][e + 2 * i + 1]), i ? pair(s.z, s.w) : pair(s.x, s.y), neg2), y0, y1);
                if (i & 1) mx1 = fmax3(mx1, y0, y1);
                else mx0 = fmax3(mx0, y0, y1);
                y0 = ex2_approx(y0);
                y1 = ex2_approx(y1);
                if (i & 1) sum1 = add2(sum1, pair(y0, y1));
                else sum0 = add2(sum0, pair(y0, y1));
                pk[q * 8 + e / 2 + i] = pack_bf16(y0, y1);
              }
            }
          }
          {
            float a, b;
            parts(add2(sum0, sum1), a, b);
            psum = a + b;
          }
          if (!plain) break;
          const float mx = fmaxf(mx0, mx1);
          top = mx - neg;
          if (!__any_sync(0xffffffffu, mx > 64.f)) break;
          careful = true;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st16(tS + q * 16, pk + q * 16);
        // l and O go to this step's reference (S(n) follows PV(n-1), so O is at rest)
        const float alpha = M == R || M == -INFINITY ? 1.f : ex2_approx(M - R);
        l = fmaf(l, alpha, psum);
        M = R;
        if (n > n0 && __any_sync(0xffffffffu, alpha != 1.f)) {     // tcgen05.ld/st are warp-collective
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t ov[32];
            tmem_ld32(tO + q * 32, ov);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(tO + q * 32, ov);
          }
        }
        if (top > R + 8.f) R = top;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&bars[T_PFULL + half]);
      }
      // ------------------------------------------------------------- the piece's end
      if (takes_part) {
        wait(T_MMADONE + half, done & 1);
        tc_fence_after();
        ++done;
        const int tok = rr / p.group, head = walk.h * p.group + rr - tok * p.group;
        const float inv = l == 0.f ? 0.f : 1.0f / l;   // a row without keys is zero
        __nv_bfloat16* to = static_cast<__nv_bfloat16*>(p.o) + (long long)(walk.q0 + tok) * p.o_ld + (long long)head * D;
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t ov[32];
          tmem_ld32(tO + q * 32, ov);
          tmem_wait_ld();
          if (live && !*abort_flag) {
            if (walk.piece < 0) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  w[i] = pack_bf16(__uint_as_float(ov[e + 2 * i]) * inv, __uint_as_float(ov[e + 2 * i + 1]) * inv);
                *reinterpret_cast<uint4*>(to + q * 32 + e) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 4)
                *q4_tc_place<D>(p.part_o, p.part_rows, walk.piece, half * 128 + row, q * 8 + e / 4) =
                    make_float4(__uint_as_float(ov[e]), __uint_as_float(ov[e + 1]), __uint_as_float(ov[e + 2]),
                                __uint_as_float(ov[e + 3]));
            }
          }
        }
        if (walk.piece < 0 && live && !*abort_flag && p.lse != nullptr) p.lse[(size_t)head * p.T + walk.q0 + tok] = q4_lse(M, l);
        if (walk.piece >= 0 && live && !*abort_flag)
          p.part_ml[(size_t)walk.piece * p.part_rows + half * 128 + row] = make_float2(M, l);
      }
      tc_fence_before();
      n0 = n1;
    }
  }

  // ----------------------------------------------------------------- teardown
  // the kernel before may be running still: the join, which follows this one alone, needs both complete
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
cudaError_t launch_t(AttendQ4Params p, int* grid, int* part_rows, cudaStream_t st) {
  auto kern = attend_q4_tc_kernel<D>;
  cudaError_t e = set_smem_once((const void*)kern, (int)TqSmem<D>::BYTES);
  if (e != cudaSuccess) return e;
  // setmaxnreg draws on the registers of the launch: fewer than the split asks for would be waited for without end
  cudaFuncAttributes attr;
  if ((e = cudaFuncGetAttributes(&attr, kern)) != cudaSuccess) return e;
  if (attr.numRegs * 5 < (int)(REG_CTRL + 2 * REG_UNPACK + 2 * REG_SOFT)) return cudaErrorNotSupported;
  p.part_rows = *part_rows = TQ_ROWS;
  int sms = 0, dev = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  *grid = sms < Q4_TC_MAX_CTAS ? sms : Q4_TC_MAX_CTAS;
  cudaLaunchAttribute late;
  const cudaLaunchConfig_t cfg = q4_dependent(*grid, TQ_THREADS, (int)TqSmem<D>::BYTES, st, &late);
  return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_attend_q4_tc(AttendQ4Params p, int d, int* grid, int* part_rows, cudaStream_t st) {
  return d == 128 ? launch_t<128>(p, grid, part_rows, st) : launch_t<64>(p, grid, part_rows, st);
}

}  // namespace pbsa

// How the attention over the 4-bit cache splits its work: the blocks of every tile (request, row tile,
// kv head) form one line in that order, and each CTA of the grid takes an equal share of it.  Each CTA sums the
// lengths for itself, so no host knowledge of them is needed and a captured call follows them (2.3 us at the start of
// a kernel, most of it loads and instruction fetches).  A tile is charged a few blocks beside its own for its start and end
// (Q, the join of the warps, the writes): without, CTAs with many short tiles end last.  For 48 single tokens over 300 .. 8192
// a charge of 0, 2, 3 and 6 blocks gives 67, 63, 60 and 60 us, for mixed fp32 requests of up to 90 tokens 35, 28, 27 and 28.
#pragma once
#include <math.h>

#include "internal.h"
#include "q4.cuh"

namespace pbsa {

constexpr int Q4_MAX_CTAS = 480;      // of a grid of the few-rows kernel (16 rows a piece)
constexpr int Q4_TC_MAX_CTAS = 160;   // of a grid of the tensor-core kernel (256 rows a piece)
constexpr int Q4_FEW_ROWS = 2 * Q4_MAX_CTAS * 16, Q4_PART_ROWS = Q4_FEW_ROWS + 2 * Q4_TC_MAX_CTAS * 256;   // of all pieces
constexpr int Q4_TC_ROWS = 80;        // requests with more rows go to the tensor-core kernel,
constexpr int Q4_TC_STEPS = 32;       // if they are more than this many blocks for each CTA of the few-rows kernel,
constexpr int Q4_FEW_TILE = 16;       // which would take them in tiles of 16 rows,
constexpr int Q4_FEW_COST = 3;        // charged 3 blocks each beside their own (both choices: see q4_share)

// A tile that starts in this CTA and ends in a later one (pieces = 0: none).
struct __align__(8) Q4Desc {
  int pieces, rows, row0, q0, h, pad;
};

struct AttendQ4Params {
  const void* q;
  long long q_ld;            // elements from one token to the next
  const int *q_start, *q_len, *kv_len;
  int R, T, max_q;
  const uint8_t* pool;
  int pool_slots;
  const int* table;
  int table_ld;
  int kv_heads, group;       // query heads = kv_heads * group; query head h * group + i reads kv head h
  int causal;
  float scale_log2;
  void* o;
  long long o_ld;
  float* lse;
  int f32;
  int max_rows;              // no request has more
  int few_ctas;              // of the few-rows kernel, where the tensor-core kernel runs beside it (else 0)
  int part_rows;             // rows of a piece in the workspace
  Q4Desc* desc;
  float2* part_ml;           // (reference maximum in log2 units, sum) of a piece's row
  float* part_o;
  void* ws;
};

// a / b of non-negative numbers; 64-bit divisions are an order slower and rarely needed
__host__ __device__ __forceinline__ long long quotient(long long a, long long b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

// The work of one request: row tiles of each kv head, and what a tile is charged in blocks.  Without the
// causal rule, and for a single tile, that is what it reads.  With it, tile k (from 1) of `tile_rows`
// rows sees past + ceil(tile_rows k / group) tokens, so it reads at most
//   charge(k) = blocks(past) + ceil(tile_rows k / (64 group))
// blocks; the charge has a sum in closed form and is at most a block or two above.
struct Q4Request {
  int q0, q_len, kv_len, tiles, blocks;
  int base;          // blocks(past), or -1: every tile is charged `blocks`
  int num, den;      // tile_rows, 64 * group

  __host__ __device__ long long charged_to(int n) const {   // the first n tiles
    if (base < 0) return (long long)n * blocks;
    if ((uint32_t)den % (uint32_t)num == 0) {      // sum of ceil(k / per): whole groups of `per` tiles, and the rest
      const int per = (uint32_t)den / (uint32_t)num, whole = (uint32_t)n / (uint32_t)per, rest = n - whole * per;
      return (long long)n * base + ((long long)whole * (whole + 1) / 2 * per + (long long)rest * (whole + 1));
    }
    // Otherwise tile_rows = 64 t, and ceil(t k / group) is the number of whole j >= 0 with k > j group / t: up to k = r that
    // makes sum over j of max(0, r - floor(j group / t)).  `group` tiles on, the charge is t more.
    const int t = num / BT, group = den / BT, whole = (uint32_t)n / (uint32_t)group, rest = n - whole * group;
    long long period = 0, last = (long long)t * whole * rest;
    for (int j = 0; j < t; ++j) {
      const int from = (uint32_t)(j * group) / (uint32_t)t;
      period += group - from;
      last += rest > from ? rest - from : 0;
    }
    return (long long)n * base + (long long)whole * (whole - 1) / 2 * t * group + whole * period + last;
  }
  __host__ __device__ int charge(int mt) const {
    return base < 0 ? blocks : base + (int)quotient((long long)num * (mt + 1) + den - 1, den);
  }
  __device__ long long head_steps() const { return charged_to(tiles); }
};

// A request whose numbers are out of range is left out (and recorded once, by the CTA that asks).
// Requests of at most `above` or more than `to` rows have no tiles here.
__device__ __forceinline__ Q4Request q4_request(const AttendQ4Params& p, int r, int tile_rows, int tile_cost, int above, int to,
                                                bool record) {
  Q4Request x;
  x.q0 = p.q_start[r];
  x.q_len = p.q_len[r];
  x.kv_len = p.kv_len[r];
  x.tiles = x.blocks = 0;
  x.base = -1;
  x.num = tile_rows;
  x.den = BT * p.group;
  if (x.q_len == 0) return x;
  if (x.q_len < 0 || x.q_len > p.max_q || x.q0 < 0 || x.q_len > p.T - x.q0 || x.kv_len < 0 ||
      x.kv_len > (long long)p.table_ld * BT) {
    if (record) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, r, K_Q4_ATTEND);
    return x;
  }
  const int rows = x.q_len * p.group;
  if (rows <= above || rows > to) return x;
  x.tiles = (rows + tile_rows - 1) / tile_rows;
  x.blocks = tile_cost + max(1, (x.kv_len + BT - 1) / BT);   // a request without keys has its rows written too
  if (p.causal && x.tiles > 1) x.base = tile_cost + (max(x.kv_len - x.q_len, 0) + BT - 1) / BT;
  return x;
}

// Where a CTA's share starts: the request, kv head, row tile, and the blocks of the tile that lie before.
struct Q4Start {
  Q4Request req;
  int r, h, mt, at;
};
struct Q4Share {
  long long total, x0, x1;
  int ctas;
  int above, to;     // the rows of this kernel's requests
};

// This CTA's share [x0, x1) of the line, and its start in shared memory.  Every thread calls it.
// The tensor-core kernel has 2.7 times the rate, but its tiles of 256 rows want many keys each before they fill the GPU, and
// a tile's start and end last 10 us: it takes the requests of more than Q4_TC_ROWS rows where they are enough work.  One
// prompt, few-rows kernel against tensor-core kernel: 300 tokens of 12 heads 20 and 39 us, 512 tokens 27 and 47, 1000
// tokens 51 and 52 (28 blocks for each CTA), 512 over 1536 49 and 49 (40), 1000 of 32 heads over 4000 393 and 192 (507).
// At 16 requests over 3000: 48 rows 39 and 68 us, 72 rows 57 and 71; at 64 over 6000: 48 rows 207 and 346, 96 rows 395 and 355.
template <int THREADS, bool TC>
__device__ __forceinline__ Q4Share q4_share(const AttendQ4Params& p, int tile_rows, int tile_cost, int min_steps, Q4Start* start) {
  __shared__ long long sums[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + THREADS - 1) / THREADS;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  Q4Share s;
  s.above = TC ? Q4_TC_ROWS : 0;
  s.to = p.max_rows;
  if (p.few_ctas > 0) {
    long long heavy = 0;
    for (int r = r0; r < r1; ++r)
      heavy += p.kv_heads * q4_request(p, r, Q4_FEW_TILE, Q4_FEW_COST, Q4_TC_ROWS, p.max_rows, false).head_steps();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) heavy += __shfl_xor_sync(0xffffffffu, heavy, o);
    if (lane == 0) sums[warp] = heavy;
    __syncthreads();
    heavy = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) heavy += sums[w];
    __syncthreads();
    const bool tc = heavy > (long long)Q4_TC_STEPS * p.few_ctas;   // (both kernels find the same)
    if (TC && !tc) s.to = 0;
    if (!TC && tc) s.to = Q4_TC_ROWS;
  }
  long long mine = 0;
  Q4Request req;
  for (int r = r0; r < r1; ++r) {
    req = q4_request(p, r, tile_rows, tile_cost, s.above, s.to, blockIdx.x == 0);
    mine += p.kv_heads * req.head_steps();
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  s.total = 0;
  long long before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = s.total;
    s.total += sums[w];
  }
  const long long want = quotient(s.total + min_steps - 1, min_steps);
  s.ctas = (int)(want < gridDim.x ? want : gridDim.x);
  s.x0 = s.x1 = 0;
  if ((int)blockIdx.x < s.ctas) {
    // floor(total i / ctas) of this CTA and the next
    const long long whole = quotient(s.total, s.ctas);
    const uint32_t rest = (uint32_t)(s.total - whole * s.ctas);
    s.x0 = whole * blockIdx.x + rest * blockIdx.x / (uint32_t)s.ctas;
    s.x1 = whole * (blockIdx.x + 1) + rest * (blockIdx.x + 1) / (uint32_t)s.ctas;
    long long at = before + upto - mine;
    if (s.x0 >= at && s.x0 < at + mine) {   // one thread
      int r = r0;
      for (;; ++r) {
        if (per > 1) req = q4_request(p, r, tile_rows, tile_cost, s.above, s.to, false);
        const long long n = p.kv_heads * req.head_steps();
        if (s.x0 < at + n) break;
        at += n;
      }
      const long long head = req.head_steps();
      start->h = (int)quotient(s.x0 - at, head);
      const long long off = s.x0 - at - start->h * head;
      int lo = 0, hi = req.tiles - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (req.charged_to(mid) <= off) lo = mid;
        else hi = mid - 1;
      }
      start->req = req;
      start->r = r;
      start->mt = lo;
      start->at = (int)(off - req.charged_to(lo));
    }
  }
  __syncthreads();
  return s;
}

// The pieces of a share, in order.  Every warp of the CTA walks them by itself.
struct Q4Walk {
  const AttendQ4Params& p;
  long long x, x1, total;
  int ctas, tile_rows, tile_cost, above, to;
  Q4Request req;
  int r;
  int at;         // blocks of the current tile that lie before the next piece
  // the current piece: blocks [b0, b1) of row tile mt of head h of request r
  int h, mt, b0, b1, q0, q_len, kv_len, rows;
  int piece;      // its place in the workspace; -1: the whole tile
  Q4Desc desc;    // the tile that goes on in a later CTA

  __device__ Q4Walk(const AttendQ4Params& prm, const Q4Share& s, const Q4Start& start, int tr, int cost)
      : p(prm), x(s.x0), x1(s.x1), total(s.total), ctas(s.ctas), tile_rows(tr), tile_cost(cost), above(s.above), to(s.to) {
    desc.pieces = 0;
    if (x >= x1) return;
    req = start.req;
    r = start.r;
    h = start.h;
    mt = start.mt;
    at = start.at;
    charge = req.charge(mt);
  }

  __device__ bool next() {
    if (x >= x1) return false;
    if (at == charge) {
      at = 0;
      if (++mt == req.tiles) {
        mt = 0;
        if (++h == p.kv_heads) {
          h = 0;
          do req = q4_request(p, ++r, tile_rows, tile_cost, above, to, false);
          while (req.tiles == 0);   // there is one: x < x1
        }
      }
      charge = req.charge(mt);
    }
    q0 = req.q0;
    q_len = req.q_len;
    kv_len = req.kv_len;
    rows = q_len * p.group;
    const int n = (int)min((long long)(charge - at), x1 - x);
    // blocks that the tile's last row sees; what is charged above them costs its share nothing
    const int last = min((mt + 1) * tile_rows, rows) - 1;
    const int seen = p.causal ? max(min(kv_len - q_len + last / p.group + 1, kv_len), 0) : kv_len;
    const int end = (seen + BT - 1) / BT;
    b0 = at;
    b1 = max(at, min(at + n, end));
    if (n == charge) {
      piece = -1;
    } else if (at > 0) {
      piece = 2 * blockIdx.x;
    } else {
      piece = 2 * blockIdx.x + 1;
      // the CTA that holds the tile's last step: the largest i with total * i / ctas <= that step
      const long long end_step = x + charge;
      const int c1 = (int)quotient(end_step * ctas + total - 1, total) - 1;
      desc.pieces = c1 - (int)blockIdx.x + 1;
      desc.row0 = mt * tile_rows;
      desc.rows = min(tile_rows, rows - desc.row0);
      desc.q0 = q0;
      desc.h = h;
    }
    x += n;
    at += n;
    return true;
  }

 private:
  int charge;     // of the current tile
};

// 2^(m - M) of a piece's sums; the sums of a piece that saw no key are zeros (or NaN, which stay)
__device__ __forceinline__ float q4_weight(float m, float M) { return m == -INFINITY ? 1.f : ex2_approx(m - M); }

__device__ __forceinline__ float q4_lse(float M, float L) {
  return L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

// Four channels of an output row, and its lse.
template <int D>
__device__ __forceinline__ void q4_write_row(const AttendQ4Params& p, int q0, int row, int h, int ch, const float (&acc)[4],
                                             float M, float L, bool with_lse) {
  const int tok = row / p.group, head = h * p.group + row - tok * p.group;
  const float inv = L == 0.f ? 0.f : 1.0f / L;   // a row without keys is zero
  const long long at = (long long)(q0 + tok) * p.o_ld + (long long)head * D + ch;
  if (p.f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + at) =
        make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + at) =
        make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
  }
  if (with_lse && p.lse != nullptr)
    p.lse[(size_t)head * p.T + q0 + tok] = q4_lse(M, L);
}

__device__ __forceinline__ Q4Desc q4_desc(const Q4Desc* p) {
  const int2* w = reinterpret_cast<const int2*>(p);
  const int2 a = __ldcg(w), b = __ldcg(w + 1), c = __ldcg(w + 2);
  return {a.x, a.y, b.x, b.y, c.x, c.y};
}

// Where channels 4 ch .. of row r of a piece lie in the workspace.  The few-rows kernel writes rows, a row's
// channels by neighbouring threads; the tensor-core kernel has a thread for each row, so there the rows of four
// channels are neighbours.
template <int D>
__device__ __forceinline__ float4* q4_few_place(float* part_o, int part_rows, int piece, int r, int ch) {
  return reinterpret_cast<float4*>(part_o) + ((size_t)piece * part_rows + r) * (D / 4) + ch;
}
template <int D>
__device__ __forceinline__ float4* q4_tc_place(float* part_o, int part_rows, int piece, int r, int ch) {
  return reinterpret_cast<float4*>(part_o) + ((size_t)piece * (D / 4) + ch) * part_rows + r;
}

// Channels 4 ch .. of a row of the tile that starts in CTA `cta` and ends in a later one: its pieces joined, in order.
template <int D, bool TC>
__device__ __forceinline__ void q4_join_row(const AttendQ4Params& p, const Q4Desc& d, int cta, const float2* part_ml,
                                            float* part_o, int part_rows, int r, int ch) {
  auto at = [&](int k) { return k == 0 ? 2 * cta + 1 : 2 * (cta + k); };
  // 8 pieces at a time, their loads in flight together (a place past the end repeats the last piece, unused)
  float M = -INFINITY, L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int k0 = 0; k0 < d.pieces; k0 += 8) {
    float2 ml[8];
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int piece = at(min(k0 + i, d.pieces - 1));
      ml[i] = __ldcg(part_ml + (size_t)piece * part_rows + r);   // (from L2: this grid may have started before they were written)
      v[i] = __ldcg(TC ? q4_tc_place<D>(part_o, part_rows, piece, r, ch) : q4_few_place<D>(part_o, part_rows, piece, r, ch));
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, ml[i].x);
    const float f0 = M == top ? 1.f : q4_weight(M, top);
    M = top;
    L *= f0;
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] *= f0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (k0 + i < d.pieces) {
        const float f = q4_weight(ml[i].x, M);
        L = fmaf(f, ml[i].y, L);
        acc[0] = fmaf(f, v[i].x, acc[0]);
        acc[1] = fmaf(f, v[i].y, acc[1]);
        acc[2] = fmaf(f, v[i].z, acc[2]);
        acc[3] = fmaf(f, v[i].w, acc[3]);
      }
    }
  }
  q4_write_row<D>(p, d.q0, d.row0 + r, d.h, 4 * ch, acc, M, L, ch == 0);
}

// Joins the pieces of both kernels.  The first `few` CTAs take a tile of the few-rows kernel each.  The others list the
// tensor-core kernel's tiles (each for itself) and share their rows, 8 at a time: there may be one tile of a hundred
// pieces or a hundred tiles of two.  (With 8 CTAs for each tile, 64 tokens of 8 heads over 2 and 30000 tokens take 85 us,
// like this 54, two requests of 256 tokens over 8000 71 and 64; such a list of the few-rows kernel's tiles would cost
// single tokens 0.8 us.)
struct Q4JoinParams {
  AttendQ4Params p;          // descriptors and pieces are the few-rows kernel's
  const Q4Desc* tc_desc;     // ... and these the tensor-core kernel's
  const float2* tc_ml;
  float* tc_o;
  int tc_rows, few, tc;      // CTAs of either
};

template <int D>
__global__ void __launch_bounds__(256) attend_q4_join_kernel(const Q4JoinParams jp) {
  __shared__ int counts[8], list[Q4_TC_MAX_CTAS];
  constexpr int CH = D / 4, RPP = 256 / CH, PARTS = 256 / RPP;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if ((int)blockIdx.x < jp.few) {
    const Q4Desc d = q4_desc(jp.p.desc + blockIdx.x);
    if (d.pieces == 0) return;
    for (int r = tid / CH; r < d.rows; r += RPP)
      q4_join_row<D, false>(jp.p, d, blockIdx.x, jp.p.part_ml, jp.p.part_o, jp.p.part_rows, r, tid % CH);
    return;
  }
  // the same list in every CTA: in the tiles' order
  static_assert(Q4_TC_MAX_CTAS <= 256, "a thread a descriptor");
  const bool mine = tid < jp.tc && __ldcg(&jp.tc_desc[tid].pieces) > 0;
  const unsigned votes = __ballot_sync(0xffffffffu, mine);
  if ((tid & 31) == 0) counts[tid >> 5] = __popc(votes);
  __syncthreads();
  int before = 0, count = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < (tid >> 5)) before += counts[w];
    count += counts[w];
  }
  if (mine) list[before + __popc(votes & ((1u << (tid & 31)) - 1u))] = tid;
  __syncthreads();
  for (int item = blockIdx.x - jp.few; item < count * PARTS; item += gridDim.x - jp.few) {
    const int cta = list[item / PARTS], r = item % PARTS * RPP + tid % RPP;
    const Q4Desc d = q4_desc(jp.tc_desc + cta);
    if (r < d.rows) q4_join_row<D, true>(jp.p, d, cta, jp.tc_ml, jp.tc_o, jp.tc_rows, r, tid / RPP);
  }
}

inline cudaLaunchConfig_t q4_dependent(int grid, int threads, int smem, cudaStream_t st, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// The tensor-core kernel alone, as a programmatic dependent of the few-rows kernel that was launched before it: it reads
// nothing of that one's, but ends after it.  `grid` and `part_rows` for the join are returned.
cudaError_t launch_attend_q4_tc(AttendQ4Params p, int d, int* grid, int* part_rows, cudaStream_t st);

}  // namespace pbsa

// How the attention over the 4-bit cache splits its work: the blocks of every tile (request, row tile,
// kv head) form one line in that order, and each CTA of the grid takes an equal share of it.
#pragma once
#include <math.h>

#include "internal.h"
#include "q4.cuh"

namespace pbsa {

constexpr int Q4_MAX_CTAS = 640;   // of a grid (the workspace holds two pieces for each)
constexpr int Q4_MIN_STEPS = 2;    // blocks that are worth a CTA of their own

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
  int part_rows;             // rows of a piece in the workspace
  Q4Desc* desc;
  float2* part_ml;           // (reference maximum in log2 units, sum) of a piece's row
  float* part_o;
  void* ws;
};

// The work of one request: `tiles` row tiles a head of `blocks` blocks each.
struct Q4Request {
  int q0, q_len, kv_len, tiles, blocks;
  __device__ long long steps(int heads) const { return (long long)heads * tiles * blocks; }
};

// A request whose numbers are out of range is left out (and recorded once, by the CTA that asks).
__device__ __forceinline__ Q4Request q4_request(const AttendQ4Params& p, int r, int tile_rows, bool record) {
  Q4Request x;
  x.q0 = p.q_start[r];
  x.q_len = p.q_len[r];
  x.kv_len = p.kv_len[r];
  x.tiles = x.blocks = 0;
  if (x.q_len == 0) return x;
  if (x.q_len < 0 || x.q_len > p.max_q || x.q0 < 0 || x.q_len > p.T - x.q0 || x.kv_len < 0 ||
      x.kv_len > (long long)p.table_ld * BT) {
    if (record) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, r, K_Q4_ATTEND);
    return x;
  }
  x.tiles = (int)(((long long)x.q_len * p.group + tile_rows - 1) / tile_rows);
  x.blocks = max(1, (x.kv_len + BT - 1) / BT);   // a request without keys has its rows written too
  return x;
}

struct Q4Start {
  int r;
  long long off;     // place of the share's first step inside request r
};
struct Q4Share {
  long long total, x0, x1;
  int ctas, r;
  long long off;
};

// This CTA's share [x0, x1) of the line, and the request it starts in.  Every thread calls it.
template <int THREADS>
__device__ __forceinline__ Q4Share q4_share(const AttendQ4Params& p, int tile_rows, Q4Start* start) {
  __shared__ long long sums[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + THREADS - 1) / THREADS;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += q4_request(p, r, tile_rows, blockIdx.x == 0).steps(p.kv_heads);
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  Q4Share s;
  s.total = 0;
  long long before = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) before = s.total;
    s.total += sums[w];
  }
  const long long want = (s.total + Q4_MIN_STEPS - 1) / Q4_MIN_STEPS;
  s.ctas = (int)(want < gridDim.x ? want : gridDim.x);
  s.x0 = s.x1 = 0;
  if ((int)blockIdx.x < s.ctas) {
    s.x0 = s.total * blockIdx.x / s.ctas;
    s.x1 = s.total * (blockIdx.x + 1) / s.ctas;
    long long at = before + upto - mine;
    if (s.x0 >= at && s.x0 < at + mine) {
      for (int r = r0; r < r1; ++r) {
        const long long n = q4_request(p, r, tile_rows, false).steps(p.kv_heads);
        if (s.x0 < at + n) {
          start->r = r;
          start->off = s.x0 - at;
          break;
        }
        at += n;
      }
    }
  }
  __syncthreads();
  s.r = start->r;
  s.off = start->off;
  return s;
}

// The pieces of a share, in order.  Every warp of the CTA walks them by itself.
struct Q4Walk {
  const AttendQ4Params& p;
  long long x, x1, total, off;
  int ctas, tile_rows;
  Q4Request req;
  int r;
  // the current piece: blocks [b0, b1) of row tile mt of head h of request r
  int h, mt, b0, b1, q0, q_len, kv_len, rows;
  int piece;      // its place in the workspace; -1: the whole tile
  Q4Desc desc;    // the tile that goes on in a later CTA

  __device__ Q4Walk(const AttendQ4Params& prm, const Q4Share& s, int tr)
      : p(prm), x(s.x0), x1(s.x1), total(s.total), off(s.off), ctas(s.ctas), tile_rows(tr), r(s.r) {
    desc.pieces = 0;
    if (x < x1) req = q4_request(p, r, tile_rows, false);
  }

  __device__ bool next() {
    if (x >= x1) return false;
    while (off >= req.steps(p.kv_heads)) {
      off = 0;
      req = q4_request(p, ++r, tile_rows, false);
    }
    const int tile = (int)(off / req.blocks), at = (int)(off - (long long)tile * req.blocks);
    h = tile / req.tiles;
    mt = tile - h * req.tiles;
    q0 = req.q0;
    q_len = req.q_len;
    kv_len = req.kv_len;
    rows = (int)min((long long)q_len * p.group, (long long)0x7fffffff);
    const int n = (int)min((long long)(req.blocks - at), x1 - x);
    // blocks that the tile's last row sees; the blocks behind them cost their share nothing
    const int last = (int)min((long long)(mt + 1) * tile_rows, (long long)rows) - 1;
    const int seen = p.causal ? max(min(kv_len - q_len + last / p.group + 1, kv_len), 0) : kv_len;
    const int end = (seen + BT - 1) / BT;
    b0 = at;
    b1 = max(at, min(at + n, end));
    if (n == req.blocks) {
      piece = -1;
    } else if (at > 0) {
      piece = 2 * blockIdx.x;
    } else {
      piece = 2 * blockIdx.x + 1;
      // the CTA that holds the tile's last step: the largest i with total * i / ctas <= that step
      const long long end_step = x + req.blocks;
      const int c1 = (int)((end_step * ctas + total - 1) / total) - 1;
      desc.pieces = c1 - (int)blockIdx.x + 1;
      desc.row0 = mt * tile_rows;
      desc.rows = min(tile_rows, rows - desc.row0);
      desc.q0 = q0;
      desc.h = h;
    }
    x += n;
    off += n;
    return true;
  }
};

// 2^(m - M) of a piece's sums; the sums of a piece that saw no key are zeros (or NaN, which stay)
__device__ __forceinline__ float q4_weight(float m, float M) { return m == -INFINITY ? 1.f : ex2_approx(m - M); }

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
    p.lse[(size_t)head * p.T + q0 + tok] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace pbsa

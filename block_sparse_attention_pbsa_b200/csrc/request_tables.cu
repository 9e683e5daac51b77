// Block tables and slot maps of a serving step, built on the GPU from the requests' lengths.
//
// With n_r = max(step_r, 0) new tokens of request r, blocks(x) = ceil(x / 64):
//   start_r  = n_0 + .. + n_{r-1}                          (its rows of the step's token tensors)
//   need_r   = blocks(len_r + n_r) - blocks(len_r)          (blocks to take from the free stack)
//   request r is served iff its rows and its table row have room and need_r = 0 or
//   need_0 + .. + need_r <= free + blocks given back by the requests that ended (step_r < 0).
// The blocks given back lie, in request order, on top of the free ones; the i-th block taken is
// the i-th from the top.  Everything is a function of the inputs, so every CTA computes the two
// prefix sums of all requests for itself (a few hundred cycles) and then does its share of the
// maps: no CTA waits for another's results.
//
// Where the state (lengths, the free count) is kept in place, outputs are the same memory as inputs: one
// cluster then holds all CTAs, and those outputs are written after a cluster barrier that every CTA
// reaches with the inputs in its shared memory.  With outputs apart, as many CTAs as the rows fill start
// without one.  Table rows and the free stack need no barrier: a call reads table entries below
// blocks(len_r) and stack entries below the free count, and writes only entries at or above them.
//
// Bound by latency (the sums, a binary search per token, one dependent table read), not bytes: 64 requests of a
// token 4.7 us, 1024 requests with 49152 rows 8.2 us apart (16.4 us as the one cluster of 8 CTAs, which the state in
// place needs); 0.45 MB, 0.07 us at a copy's rate.
#include "common.cuh"
#include "internal.h"

namespace pbsa {
namespace {

constexpr int RT_THREADS = 1024;
constexpr int RT_CLUSTER = 8;
constexpr int RT_MAX_CTAS = 148;

struct TablesParams {
  const int* step_len;
  const int* seq_len;
  int R;
  int* table;
  int ld;
  int* free_slot;
  const int* free_cnt;
  int pool_slots;
  int T;
  int *q_start, *q_len, *kv_len, *free_cnt_out, *slot_map, *position;
  void* ws;
  int in_place;   // kv_len or free_cnt_out may share memory with an input
};

// Inclusive block sums of two values per thread (all threads call it).
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long (*warp_sums)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, a, o), y = __shfl_up_sync(0xffffffffu, b, o);
    if (lane >= o) { a += x; b += y; }
  }
  if (lane == 31) { warp_sums[warp][0] = a; warp_sums[warp][1] = b; }
  __syncthreads();
  if (warp == 0) {
    long long x = warp_sums[lane][0], y = warp_sums[lane][1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) { x += u; y += v; }
    }
    warp_sums[lane][0] = x;
    warp_sums[lane][1] = y;
  }
  __syncthreads();
  if (warp > 0) { a += warp_sums[warp - 1][0]; b += warp_sums[warp - 1][1]; }
}

// First index in [0, n) whose (non-decreasing) value is above x; n if none.
__device__ __forceinline__ int first_above(const int* v, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int blocks_of(long long n) { return (int)((n + BT - 1) / BT); }

__global__ void __launch_bounds__(RT_THREADS) request_tables_kernel(const TablesParams p) {
  extern __shared__ int rt_sm[];
  int* s_end = rt_sm;               // last row of the request + 1, at most T
  int* s_upto = s_end + p.R;        // blocks asked for by the requests up to this one
  int* s_gone = s_upto + p.R;       // blocks given back by the requests up to this one
  int* s_seq = s_gone + p.R;        // length before the step
  int* s_new = s_seq + p.R;         // tokens served (-1: ended, 0: none or refused)
  __shared__ long long warp_sums[32][2];
  __shared__ long long s_total[2];
  __shared__ int s_taken;           // blocks taken by the requests served
  const int tid = threadIdx.x;
  const int per = (p.R + RT_THREADS - 1) / RT_THREADS;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  const int nctas = gridDim.x, rank = blockIdx.x;   // in place, the grid is one cluster

  int cnt = *p.free_cnt;
  if (cnt < 0 || cnt > p.pool_slots) {
    if (tid == 0) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, cnt, K_REQ_TABLES);
    cnt = min(max(cnt, 0), p.pool_slots);
  }
  // rows and blocks given back
  long long rows = 0, gone = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = p.step_len[r];
    int q = p.seq_len[r];
    if (q < 0 || q > (long long)p.ld * BT) {
      record_error(p.ws, PBSA_ERR_DEVICE_INDEX, q, K_REQ_TABLES);
      q = -1;
    }
    s_seq[r] = q;
    s_new[r] = n;
    rows += max(n, 0);
    if (n < 0 && q > 0) gone += blocks_of(q);
  }
  long long rows_upto = rows, gone_upto = gone;
  block_scan2(rows_upto, gone_upto, warp_sums);
  if (tid == 0) s_taken = 0;
  if (tid == RT_THREADS - 1) { s_total[0] = rows_upto; s_total[1] = gone_upto; }
  __syncthreads();
  const long long all_rows = s_total[0], all_gone = s_total[1];
  const long long avail = cnt + all_gone, cap = min(avail, (long long)0x7fffffff);
  // blocks asked for
  long long end = rows_upto - rows, back = gone_upto - gone, need = 0, unused = 0;
  for (int r = r0; r < r1; ++r) {
    const int n = s_new[r], q = s_seq[r];
    end += max(n, 0);
    if (n < 0 && q > 0) back += blocks_of(q);
    s_end[r] = (int)min(end, (long long)p.T);
    s_gone[r] = (int)min(back, (long long)0x7fffffff);
    int want = 0;
    const bool fits = n >= 0 && q >= 0 && end <= p.T && (long long)q + n <= (long long)p.ld * BT;
    if (fits) want = blocks_of((long long)q + n) - blocks_of(q);
    else if (n > 0) s_new[r] = 0;
    s_upto[r] = want;
    need += want;
  }
  long long need_upto = need;
  __syncthreads();   // warp_sums is used again
  block_scan2(need_upto, unused, warp_sums);
  need_upto -= need;
  for (int r = r0; r < r1; ++r) {
    const int want = s_upto[r];
    need_upto += want;
    if (want > 0) {
      if (need_upto <= cap) atomicMax(&s_taken, (int)need_upto);
      else s_new[r] = 0;   // refused, and so is every later request that needs a block
    }
    s_upto[r] = (int)min(need_upto, cap);
  }
  __syncthreads();
  // the inputs that an output may share memory with have been read by this CTA
  if (p.in_place) asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");

  const int taken = s_taken;
  const long long left_all = avail - taken;
  const int left = (int)min(left_all, (long long)p.pool_slots);
  if (left_all > p.pool_slots && tid == 0) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, (int)min(left_all, (long long)0x7fffffff), K_REQ_TABLES);

  auto given_back = [&](int i) {   // the i-th block given back
    const int r = first_above(s_gone, p.R, i);
    if (r >= p.R) return -1;
    return p.table[(size_t)r * p.ld + (i - (r > 0 ? s_gone[r - 1] : 0))];
  };
  auto popped = [&](int i) {       // the i-th block taken
    const long long v = avail - 1 - i;
    return v < cnt ? p.free_slot[v] : given_back((int)(v - cnt));
  };
  const int t0 = rank * RT_THREADS + tid, stride = nctas * RT_THREADS;
  // blocks given back that stay free (those that are taken again are looked at with their rows)
  for (int v = cnt + t0; v < left; v += stride) {
    const int slot = given_back(v - cnt);
    if (slot < 0 || slot >= p.pool_slots) record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot, K_REQ_TABLES);
    p.free_slot[v] = slot;
  }
  // new table entries
  for (int i = t0; i < taken; i += stride) {
    const int r = first_above(s_upto, p.R, i);
    const int b = blocks_of(s_seq[r]) + i - (r > 0 ? s_upto[r - 1] : 0);
    p.table[(size_t)r * p.ld + b] = popped(i);
  }
  // every row's place in the cache
  for (int t = t0; t < p.T; t += stride) {
    const int r = first_above(s_end, p.R, t);
    int at = -1, pos = -1;
    if (r < p.R && s_new[r] > 0) {
      const int before = blocks_of(s_seq[r]);
      pos = s_seq[r] + t - (r > 0 ? s_end[r - 1] : 0);
      const int b = pos / BT;
      const int slot = b < before ? p.table[(size_t)r * p.ld + b] : popped((r > 0 ? s_upto[r - 1] : 0) + b - before);
      if (slot >= 0 && slot < p.pool_slots) at = slot * BT + pos % BT;
      else record_error(p.ws, PBSA_ERR_DEVICE_INDEX, slot, K_REQ_TABLES);
    }
    p.slot_map[t] = at;
    if (p.position != nullptr) p.position[t] = pos;
  }
  if (rank == 0) {
    for (int r = tid; r < p.R; r += RT_THREADS) {
      const int n = s_new[r];
      p.q_start[r] = r > 0 ? s_end[r - 1] : 0;
      p.q_len[r] = max(n, 0);
      p.kv_len[r] = n < 0 ? 0 : max(s_seq[r], 0) + n;
    }
    if (tid == 0) {
      p.q_start[p.R] = (int)min(all_rows, (long long)p.T);
      *p.free_cnt_out = left;
    }
  }
}

}  // namespace

cudaError_t launch_request_tables(const int* step_len, const int* seq_len, int R, int* table, int ld, int* free_slot,
                                  const int* free_cnt, int pool_slots, int T, int* q_start, int* q_len, int* kv_len,
                                  int* free_cnt_out, int* slot_map, int* position, void* ws, cudaStream_t st) {
  // (compared as ranges: the outputs may also overlap an input in part)
  auto overlap = [](const int* a, int na, const int* b, int nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + sizeof(int) * (size_t)nb && y < x + sizeof(int) * (size_t)na;
  };
  const int in_place = overlap(kv_len, R, seq_len, R) || overlap(free_cnt_out, 1, free_cnt, 1) ||
                       overlap(kv_len, R, step_len, R) || overlap(q_len, R, step_len, R) || overlap(q_len, R, seq_len, R);
  const TablesParams p = {step_len, seq_len, R,      table, ld,           free_slot, free_cnt, pool_slots,
                          T,        q_start, q_len, kv_len, free_cnt_out, slot_map,  position, ws, in_place};
  const int smem = 5 * R * (int)sizeof(int);
  cudaError_t e = set_smem_once((const void*)request_tables_kernel, 5 * 8192 * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int fill = (T + RT_THREADS - 1) / RT_THREADS;
  const int ctas = fill <= 1 ? 1 : in_place ? RT_CLUSTER : (fill < RT_MAX_CTAS ? fill : RT_MAX_CTAS);
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(RT_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = in_place ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, request_tables_kernel, p);
}

}  // namespace pbsa

// layout.cuh -- the row layout of a dispatch, shared by the kernels that move
// rows by it (the quantising dispatches and the plain permute).
//
//   layout_prologue / slot_row   after a route plan: every CTA turns the chunk
//                                table into segment starts, then a slot's rank
//                                into its row
//   small_layout                 without one (T*K <= kSmallSlots): every CTA
//                                ranks all slots itself in shared memory
#pragma once

#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace moeperm {

// Layout prologue of a dispatch CTA (see the file comment). Leaves in shared
// memory: the exclusive per-expert prefix over chunks (tbl), the expert row
// base (st: compact start, masked 0) and, for compact, psum (ps).
__device__ __forceinline__ void layout_prologue(const ScatterArgs& p, int32_t* tbl, int32_t* st, int32_t* ps,
                                int32_t* s_wsum) {
  const int tid = threadIdx.x, bd = blockDim.x;
  const int L = p.L, NC = p.nchunks;
  // the whole table in flight at once: 16-byte asynchronous copies (the
  // table starts 16-byte aligned in the workspace), the odd tail by loads
  const int n = NC * L, n4 = n / 4;
  for (int i = tid; i < n4; i += bd) cp_async16(tbl + 4 * i, p.table + 4 * i);
  for (int i = 4 * n4 + tid; i < n; i += bd) tbl[i] = __ldcg(p.table + i);
  cp_async_wait_all();
  __syncthreads();
  for (int e = tid; e < L; e += bd) {
    int run = 0, c = 0;
    for (; c + 8 <= NC; c += 8) {  // 8 loads in flight, then 8 stores
      int h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = tbl[(c + j) * L + e];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        tbl[(c + j) * L + e] = run;
        run += h[j];
      }
    }
    for (; c < NC; ++c) {
      const int h = tbl[c * L + e];
      tbl[c * L + e] = run;
      run += h;
    }
    ps[e] = run;  // count, for now
  }
  __syncthreads();
  if (p.mode == kModeCompact) {
    // segment starts: exclusive scan of align(count) over experts
    const int total = aligned_starts(ps, st, L, p.block_e, INT_MAX, s_wsum);
    for (int e = tid; e < L; e += bd) ps[e] += st[e];  // count -> psum
    if (blockIdx.x == 0 && tid == 0) *p.total = total;
    __syncthreads();
    if (blockIdx.x == 0) {
      for (int e = tid; e < L; e += bd) {
        p.counts[e] = ps[e] - st[e];
        p.starts[e] = st[e];
        p.psum[e] = ps[e];
      }
    }
  } else {
    // masked: masked_m = min(count, cap) and the overflow flag; st is free
    // here (slab rows need no start) and takes the expanded-layout starts of
    // the slab's real rows when psum is asked for (PR #29525 _build_layout)
    bool overflow = false;
    for (int e = tid; e < L; e += bd) {
      const int cnt = ps[e];
      if (blockIdx.x == 0) p.masked_m[e] = min(cnt, p.cap);
      if (cnt > p.cap) overflow = true;
    }
    if (overflow && blockIdx.x == 0) set_status(p.status, kStOverflow);
    if (p.psum != nullptr && blockIdx.x == 0) {  // uniform over the CTA
      aligned_starts(ps, st, L, p.block_e, p.cap, s_wsum);
      for (int e = tid; e < L; e += bd) p.psum[e] = st[e] + min(ps[e], p.cap);
    }
    __syncthreads();
  }
}

// Row of slot a (expert e, chunk-local rank lr) from the prologue's tables;
// -1 if dropped. A rank that does not fit the layout (only possible if the
// workspace was altered between the launches) flags BAD_LAYOUT and drops the
// slot, so no write ever leaves the buffers.
__device__ __forceinline__ int slot_row(const ScatterArgs& p, const int32_t* tbl, const int32_t* st,
                                        int64_t a, int e, int lr) {
  if (e < 0 || e >= p.L) return -1;
  const int base = tbl[(int)(a / p.chunk) * p.L + e];
  if (p.mode == kModeCompact) {
    const int row = st[e] + base + lr;
    if (lr < 0 || row < 0 || (int64_t)row >= p.bound) {
      set_status(p.status, kStBadLayout);
      return -1;
    }
    return row;
  }
  const int j = base + lr;
  if (lr < 0 || j < 0) {
    set_status(p.status, kStBadLayout);
    return -1;
  }
  return j < p.cap ? e * p.cap + j : -1;
}

// Warps of a CTA that ranks all slots itself.
constexpr int kSmallWarps = 8;

// Shared memory of small_layout, in ints: [kSmallWarps][L] per-warp counters,
// [L] expert row bases, [L] counts (compact: then psum), [T*K] row of every
// slot, [T*K] expert of every slot.
__device__ __forceinline__ int32_t* small_rows(const ScatterArgs& p, int32_t* sm) {
  return sm + (kSmallWarps + 2) * p.L;
}
__host__ __device__ inline size_t small_layout_bytes(const ScatterArgs& a) {
  return ((size_t)(kSmallWarps + 2) * a.L + 2 * (size_t)a.T * a.K) * sizeof(int32_t);
}

// Rows of all slots of a small problem, ranked by this CTA alone (kSmallWarps
// x 32 threads, S slots per lane), into small_rows(). CTA 0 writes counts /
// starts / psum / total (or masked_m and the overflow flag), the CTAs share
// the m_indices fill and write src2dst and row weights of their own tokens
// (blockIdx.x, + gridDim.x, ...). s_wsum: at least 33 ints.
template <int S>
__device__ __forceinline__ void small_layout(const ScatterArgs& p, int32_t* sm, int32_t* s_wsum,
                                             int n_live) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int L = p.L, K = p.K;
  const int64_t A = (int64_t)p.T * K, A_live = (int64_t)n_live * K;
  int32_t* hw = sm;
  int32_t* st = hw + kSmallWarps * L;
  int32_t* ps = st + L;
  int32_t* rows_all = ps + L;
  int32_t* exps_all = rows_all + A;

  // stable ranks of all slots
  for (int i = tid; i < kSmallWarps * L; i += (kSmallWarps * 32)) hw[i] = 0;
  const int base = warp * 32 * S;
  int32_t r[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int64_t a = base + i * 32 + lane;
    const int e = (a < A_live) ? __ldg(p.ids + a) : -1;
    r[i] = (e >= 0 && e < L) ? e : -1;
  }
  __syncthreads();
  int32_t* myhw = hw + warp * L;
  const unsigned lt_mask = (1u << lane) - 1u;
  const int nbits = (L > 1) ? 32 - __clz(L - 1) : 0;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int e = r[i];
    unsigned m = __ballot_sync(0xffffffffu, e >= 0);
    for (int b = 0; b < nbits; ++b) {
      const unsigned bit = (unsigned)(e >> b) & 1u;
      const unsigned bal = __ballot_sync(0xffffffffu, bit);
      m &= bit ? bal : ~bal;
    }
    const unsigned peers = (e >= 0) ? m : 0u;
    const int lower = __popc(peers & lt_mask);
    int rank = 0;
    if (e >= 0) rank = myhw[e] + lower;
    __syncwarp();
    if (e >= 0 && lower == 0) myhw[e] += __popc(peers);
    __syncwarp();
    r[i] = (e >= 0) ? ((rank << 11) | (e + 1)) : 0;
  }
  __syncthreads();

  // warp bases and counts per expert; segment starts
  for (int e = tid; e < L; e += (kSmallWarps * 32)) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < kSmallWarps; ++w) {
      const int c = hw[w * L + e];
      hw[w * L + e] = run;
      run += c;
    }
    ps[e] = run;
  }
  __syncthreads();
  if (p.mode == kModeCompact) {
    const int total = aligned_starts(ps, st, L, p.block_e, INT_MAX, s_wsum);
    for (int e = tid; e < L; e += (kSmallWarps * 32)) ps[e] += st[e];  // count -> psum
    if (blockIdx.x == 0 && tid == 0) *p.total = total;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int e = tid; e < L; e += (kSmallWarps * 32)) {
        p.counts[e] = ps[e] - st[e];
        p.starts[e] = st[e];
        p.psum[e] = ps[e];
      }
    if (p.m_indices != nullptr)
      for (int64_t rr = (int64_t)blockIdx.x * (kSmallWarps * 32) + tid; rr < p.bound;
           rr += (int64_t)gridDim.x * (kSmallWarps * 32)) {
        int lo2 = 0, hi2 = L - 1;  // largest e with start[e] <= rr (start[0] = 0)
        while (lo2 < hi2) {
          const int mid = (lo2 + hi2 + 1) >> 1;
          if (st[mid] <= rr) lo2 = mid; else hi2 = mid - 1;
        }
        p.m_indices[rr] = (rr < ps[lo2]) ? lo2 : -1;
      }
  } else {
    // masked: slab rows need no start, so st takes the expanded-layout starts
    // of the slab's real rows when psum is asked for (PR #29525 _build_layout)
    bool overflow = false;
    for (int e = tid; e < L; e += (kSmallWarps * 32)) {
      if (blockIdx.x == 0) p.masked_m[e] = min(ps[e], p.cap);
      if (ps[e] > p.cap) overflow = true;
    }
    if (overflow && blockIdx.x == 0) set_status(p.status, kStOverflow);
    if (p.psum != nullptr && blockIdx.x == 0) {  // uniform over the CTA
      aligned_starts(ps, st, L, p.block_e, p.cap, s_wsum);
      for (int e = tid; e < L; e += (kSmallWarps * 32)) p.psum[e] = st[e] + min(ps[e], p.cap);
    }
    __syncthreads();
  }

  // rows of all slots (each lane resolves its own slots)
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int64_t a = base + i * 32 + lane;
    if (a >= A) continue;
    const int pk = r[i];
    int row = -1;
    if (pk) {
      const int e = (pk & 0x7FF) - 1;
      const int j = hw[warp * L + e] + (pk >> 11);  // rank among all slots of e
      if (p.mode == kModeCompact) row = st[e] + j;
      else if (j < p.cap) row = e * p.cap + j;
    }
    rows_all[a] = row;
    exps_all[a] = pk ? (pk & 0x7FF) - 1 : -1;
  }
  __syncthreads();

  // src2dst and row weights of this CTA's tokens (each slot written once)
  for (int t = blockIdx.x; t < p.T; t += gridDim.x)
    for (int k = tid; k < K; k += (kSmallWarps * 32)) {
      const int64_t a = (int64_t)t * K + k;
      const int row = rows_all[a];
      p.src2dst[a] = row;
      if (row >= 0 && p.row_weights != nullptr) p.row_weights[row] = __ldg(p.w + a);
    }
}

}  // namespace moeperm

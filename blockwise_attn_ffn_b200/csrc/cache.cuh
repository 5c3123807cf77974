// Paged key-value cache: appending new tokens and evicting slots.
//
// Layout: K and V caches [pages, h_kv, page_size, d_k] (16-bit); a page table
// [B, max_pages] of page numbers.  Slot s of sequence b lies in page
// table[b][s / page_size], row s % page_size, for every head.
//
// Both operators only move rows, so HBM bandwidth bounds them: 16-byte
// accesses, every row read and written once, several independent loads in
// flight per thread.  Page numbers are checked on the device: an entry
// outside the pool moves nothing and sets the error word.
#pragma once

#include "common.cuh"

namespace bpt {

constexpr uint32_t kErrIndex = 7u;  // page number, length or slot outside the cache
enum : uint32_t { kSiteAppend = 16, kSiteDecode = 17, kSiteEvict = 18 };

struct CacheView {
  uint4* k;  // rows of d_k / 8 16-byte chunks
  uint4* v;
  const int* table;   // [B][max_pages]
  const int* lens;    // [B]
  uint32_t pages, hkv, ps, max_pages;
  uint32_t cap;       // max_pages * ps slots per sequence
  uint32_t* err;
};

// Row of slot s of sequence b, head t, in units of cache rows; -1 where the
// table names no page of the pool.  (The host bounds pages * hkv * ps below
// 2^31; the byte offsets built from it are 64-bit.)
__device__ __forceinline__ int cache_row(const CacheView& c, uint32_t b, uint32_t t, uint32_t s) {
  const uint32_t pg = s / c.ps;
  const uint32_t page =
      static_cast<uint32_t>(__ldg(c.table + static_cast<long long>(b) * c.max_pages + pg));
  if (page >= c.pages) return -1;
  return static_cast<int>((page * c.hkv + t) * c.ps + (s - pg * c.ps));
}

// A sequence's length, held to the table's capacity (an error outside it).
__device__ __forceinline__ uint32_t cache_len(const CacheView& c, uint32_t b, bool& bad) {
  const int n = __ldg(c.lens + b);
  if (n < 0) {
    bad = true;
    return 0;
  }
  if (static_cast<uint32_t>(n) > c.cap) {
    bad = true;
    return c.cap;
  }
  return static_cast<uint32_t>(n);
}

// ------------------------------------------------------------------ append --
struct AppendParams {
  CacheView c;
  const uint4* k;  // [B][T][h_kv][d_k], strides in 16-byte chunks
  const uint4* v;
  long long k_b, k_t, k_h, v_b, v_t, v_h;
  const int* counts;  // nullable [B]: new tokens of each sequence (<= T)
  int* new_lens;      // [B]
  float* acc;         // nullable [B][h_kv][cap]: set to 0 for new slots
  int* pos;           // nullable [B][h_kv][cap]: set to seen + t
  const int* seen;    // nullable [B]: tokens seen so far (NULL: the slot)
  uint32_t T, row16;  // 16-byte chunks of one row (d_k / 8)
};

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;

// Grid (ceil(T * h_kv * row16 / 1024), B).  A thread takes four 16-byte
// chunks of K and the same of V, 256 chunks apart, so consecutive threads
// read consecutive chunks and eight loads are in flight.
__global__ void __launch_bounds__(kAppendThreads) cache_append_kernel(const AppendParams p) {
  const uint32_t b = blockIdx.y;
  bool bad = false;
  const uint32_t len = cache_len(p.c, b, bad);
  uint32_t cnt = p.T;
  if (p.counts != nullptr) {
    const int n = __ldg(p.counts + b);
    if (n < 0 || static_cast<uint32_t>(n) > p.T) bad = true;
    cnt = n < 0 ? 0u : min(static_cast<uint32_t>(n), p.T);
  }
  if (cnt > p.c.cap - len) {  // no room: the rest is dropped
    bad = true;
    cnt = p.c.cap - len;
  }
  const uint32_t per_tok = p.c.hkv * p.row16;
  const uint32_t total = cnt * per_tok;  // bounded below 2^31 by the host
  uint4 kk[kAppendUnroll], vv[kAppendUnroll];
  long long dst[kAppendUnroll];
  const uint32_t i0 = blockIdx.x * (kAppendThreads * kAppendUnroll) + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kAppendUnroll; ++u) {
    const uint32_t i = i0 + u * kAppendThreads;
    dst[u] = -1;
    if (i >= total) continue;
    const uint32_t t = i / per_tok, r = i - t * per_tok;
    const uint32_t hd = r / p.row16, ch = r - hd * p.row16;
    const uint32_t s = len + t;
    const int row = cache_row(p.c, b, hd, s);
    if (ch == 0) {
      const long long a = (static_cast<long long>(b) * p.c.hkv + hd) * p.c.cap + s;
      if (p.acc != nullptr) p.acc[a] = 0.f;
      if (p.pos != nullptr)
        p.pos[a] = p.seen != nullptr ? __ldg(p.seen + b) + static_cast<int>(t)
                                     : static_cast<int>(s);
    }
    if (row < 0) {
      bad = true;
      continue;
    }
    kk[u] = __ldg(p.k + b * p.k_b + t * p.k_t + hd * p.k_h + ch);
    vv[u] = __ldg(p.v + b * p.v_b + t * p.v_t + hd * p.v_h + ch);
    dst[u] = static_cast<long long>(row) * p.row16 + ch;
  }
#pragma unroll
  for (int u = 0; u < kAppendUnroll; ++u) {
    if (dst[u] < 0) continue;
    p.c.k[dst[u]] = kk[u];
    p.c.v[dst[u]] = vv[u];
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) p.new_lens[b] = static_cast<int>(len + cnt);
  if (bad) record_error(p.c.err, kErrIndex, kSiteAppend);
}

// ------------------------------------------------------------------- evict --
// Per (sequence, head) with more than `budget` slots: keep the protected
// slots (pos < sinks or pos >= seen - recent), then the largest accumulated
// weights, equal ones by the lowest slot, `budget` in all.  Kept slots behind
// the budget (movers, ascending) fill the evicted ones before it (holes,
// ascending): sources and destinations are disjoint, so the moves run in any
// order, in place, and a second call with the same inputs changes nothing.
struct EvictParams {
  CacheView c;
  const float* acc;  // [B][h_kv][cap]
  const int* pos;    // [B][h_kv][cap]
  const int* seen;   // [B]
  float* acc_out;
  int* pos_out;
  int* new_lens;     // [B]
  uint32_t budget, recent, sinks, row16;
  int* lists;        // [B][h_kv][cap]: holes from 0, movers from cap / 2
  int* count;        // [B][h_kv]
};

// Order of the weights as unsigned keys: protected slots first, NaN last,
// both zeros equal.
__device__ __forceinline__ uint32_t evict_key(float w, int pos, int sinks, int since) {
  if (pos < sinks || pos >= since) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = w == 0.f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Positions of at least this are recent.
__device__ __forceinline__ int evict_since(const EvictParams& p, uint32_t b) {
  const long long since = static_cast<long long>(__ldg(p.seen + b)) - p.recent;
  return since < -2147483647LL ? -2147483647 : static_cast<int>(since);
}

constexpr int kEvictThreads = 1024;

// Sum over the block of each thread's predicate before it (exclusive) and in
// all; `warp_tot` [32] is scratch.
__device__ __forceinline__ uint32_t block_rank(bool pred, uint32_t* warp_tot, uint32_t& total) {
  const uint32_t m = __ballot_sync(0xffffffffu, pred);
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) warp_tot[warp] = __popc(m);
  __syncthreads();
  uint32_t v = warp_tot[lane];  // every warp scans the 32 warp totals
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= static_cast<uint32_t>(o)) inc += x;
  }
  total = __shfl_sync(0xffffffffu, inc, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, inc - v, warp);
  __syncthreads();
  return before + __popc(m & ((1u << lane) - 1u));
}

// Grid (h_kv, B): the threshold by a radix select of four 8-bit digits (the
// keys are re-read from L2 for each), then one ordered pass that writes the
// hole and mover lists and the weights and positions of the slots that stay.
__global__ void __launch_bounds__(kEvictThreads) cache_evict_select_kernel(const EvictParams p) {
  const uint32_t hd = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  bool bad = false;
  const uint32_t n = cache_len(p.c, b, bad);
  if (bad && tid == 0) record_error(p.c.err, kErrIndex, kSiteEvict);
  const long long bh = static_cast<long long>(b) * p.c.hkv + hd;
  const float* acc = p.acc + bh * p.c.cap;
  const int* pos = p.pos + bh * p.c.cap;
  float* acc_out = p.acc_out + bh * p.c.cap;
  int* pos_out = p.pos_out + bh * p.c.cap;
  if (n <= p.budget) {
    for (uint32_t s = tid; s < n; s += kEvictThreads) {
      acc_out[s] = acc[s];
      pos_out[s] = pos[s];
    }
    if (tid == 0) p.count[bh] = 0;
    return;
  }
  const int sinks = static_cast<int>(p.sinks);
  const int since = evict_since(p, b);
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick_sh[2];
  __shared__ uint32_t wt[32];
  uint32_t prefix = 0, need = p.budget;  // slots to take among the keys with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (uint32_t s = tid; s < n; s += kEvictThreads) {
      const uint32_t key = evict_key(acc[s], pos[s], sinks, since);
      if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid < 32) {
      // lane l holds digits 255 - 8l .. 248 - 8l: counts from the largest down
      uint32_t sum = 0;
      for (int d = 0; d < 8; ++d) sum += hist[255 - 8 * tid - d];
      uint32_t inc = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= static_cast<uint32_t>(o)) inc += x;
      }
      const uint32_t before = inc - sum;
      if (before < need && inc >= need) {
        uint32_t left = need - before;
        for (int d = 0; d < 8; ++d) {
          const uint32_t h = hist[255 - 8 * tid - d];
          if (left <= h) {
            pick_sh[0] = 255 - 8 * tid - d;
            pick_sh[1] = left;
            break;
          }
          left -= h;
        }
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | pick_sh[0];
    need = pick_sh[1];
    __syncthreads();
  }
  // kept: key above the threshold, or equal and among the first `need` such slots
  int* holes = p.lists + bh * p.c.cap;
  int* movers = holes + p.c.cap / 2;
  uint32_t ties = 0, n_holes = 0, n_movers = 0;
  for (uint32_t s0 = 0; s0 < n; s0 += kEvictThreads) {
    const uint32_t s = s0 + tid;
    const float w = s < n ? acc[s] : 0.f;
    const int ps = s < n ? pos[s] : 0;
    const uint32_t key = s < n ? evict_key(w, ps, sinks, since) : 0u;
    uint32_t tot;
    const bool tie = s < n && key == prefix;
    const uint32_t tr = ties + block_rank(tie, wt, tot);
    ties += tot;
    const bool kept = s < n && (key > prefix || (tie && tr < need));
    if (kept && s < p.budget) {
      acc_out[s] = w;
      pos_out[s] = ps;
    }
    const bool hole = s < p.budget && !kept;  // s < n holds: n > budget
    const uint32_t hr = n_holes + block_rank(hole, wt, tot);
    n_holes += tot;
    if (hole) holes[hr] = static_cast<int>(s);
    const bool mover = s >= p.budget && kept;
    const uint32_t mr = n_movers + block_rank(mover, wt, tot);
    n_movers += tot;
    if (mover) movers[mr] = static_cast<int>(s);
  }
  if (tid == 0) p.count[bh] = static_cast<int>(min(n_holes, n_movers));
}

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 64;  // moves per block and step

// Grid (steps, h_kv, B): move i copies a row of K and of V, its weight and
// its position.  row16 threads take one row (16 bytes each).
__global__ void __launch_bounds__(kMoveThreads) cache_evict_move_kernel(const EvictParams p) {
  const uint32_t hd = blockIdx.y, b = blockIdx.z;
  const long long bh = static_cast<long long>(b) * p.c.hkv + hd;
  const uint32_t cnt = static_cast<uint32_t>(p.count[bh]);
  const int* holes = p.lists + bh * p.c.cap;
  const int* movers = holes + p.c.cap / 2;
  const uint32_t ch = threadIdx.x % p.row16, sub = threadIdx.x / p.row16;
  const uint32_t per = kMoveThreads / p.row16;  // rows at once
  bool bad = false;
  // (written here, behind every reader of lens, so that both may be one array)
  if (blockIdx.x == 0 && hd == 0 && threadIdx.x == 0)
    p.new_lens[b] = static_cast<int>(min(cache_len(p.c, b, bad), p.budget));
  for (uint32_t i0 = blockIdx.x * kMoveRows; i0 < cnt; i0 += gridDim.x * kMoveRows) {
#pragma unroll 4
    for (uint32_t j = sub; j < kMoveRows; j += per) {
      const uint32_t i = i0 + j;
      if (i >= cnt) break;
      const uint32_t from = static_cast<uint32_t>(movers[i]), to = static_cast<uint32_t>(holes[i]);
      const int rf = cache_row(p.c, b, hd, from), rt = cache_row(p.c, b, hd, to);
      if (ch == 0) {
        p.acc_out[bh * p.c.cap + to] = p.acc[bh * p.c.cap + from];
        p.pos_out[bh * p.c.cap + to] = p.pos[bh * p.c.cap + from];
      }
      if (rf < 0 || rt < 0) {
        bad = true;
        continue;
      }
      const long long f = static_cast<long long>(rf) * p.row16 + ch;
      const long long t = static_cast<long long>(rt) * p.row16 + ch;
      const uint4 k = p.c.k[f], v = p.c.v[f];
      p.c.k[t] = k;
      p.c.v[t] = v;
    }
  }
  if (bad) record_error(p.c.err, kErrIndex, kSiteEvict);
}

}  // namespace bpt

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
  uint32_t ps_mul, ps_shift;  // s / ps = (s * ps_mul) >> (32 + ps_shift), s < 2^31 (ps > 1)
  uint32_t cap;       // max_pages * ps slots per sequence
  uint32_t* err;
};

// Row of slot s of sequence b, head t, in units of cache rows; -1 where the
// table names no page of the pool.  (The host bounds pages * hkv * ps below
// 2^31; the byte offsets built from it are 64-bit.)
__device__ __forceinline__ int cache_row(const CacheView& c, uint32_t b, uint32_t t, uint32_t s) {
  const uint32_t pg = c.ps == 1 ? s : __umulhi(s, c.ps_mul) >> c.ps_shift;
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

constexpr int kMoveThreads = 256;

// Moves first * rows + ..., in steps of `step` groups of rows, of the pair's
// `count` ones: each thread copies 16 bytes of a row of K and of V, one of a
// row's threads its weight and position.  The next move's list and table
// entries are looked up while this one's rows are on their way (three loads
// that depend on one another stood before each row otherwise).
__device__ __forceinline__ void evict_moves(const EvictParams& p, uint32_t hd, uint32_t b,
                                            uint32_t count, uint32_t first, uint32_t step,
                                            uint32_t threads) {
  const long long bh = static_cast<long long>(b) * p.c.hkv + hd;
  const int* holes = p.lists + bh * p.c.cap;
  const int* movers = holes + p.c.cap / 2;
  const uint32_t ch = threadIdx.x % p.row16, per = threads / p.row16;  // rows at once
  bool bad = false;
  uint32_t i = first * per + threadIdx.x / p.row16;
  uint32_t from = 0, to = 0;
  int rf = -1, rt = -1;
  auto look_up = [&]() {
    if (i >= count) return;
    from = static_cast<uint32_t>(movers[i]);
    to = static_cast<uint32_t>(holes[i]);
    rf = cache_row(p.c, b, hd, from);
    rt = cache_row(p.c, b, hd, to);
  };
  look_up();
  while (i < count) {
    const bool ok = rf >= 0 && rt >= 0;
    const long long f = static_cast<long long>(ok ? rf : 0) * p.row16 + ch;
    const long long t = static_cast<long long>(ok ? rt : 0) * p.row16 + ch;
    const uint32_t old_from = from, old_to = to;
    uint4 k, v;
    if (ok) {
      k = p.c.k[f];
      v = p.c.v[f];
    }
    i += step * per;
    look_up();
    if (ch == 0) {
      p.acc_out[bh * p.c.cap + old_to] = p.acc[bh * p.c.cap + old_from];
      p.pos_out[bh * p.c.cap + old_to] = p.pos[bh * p.c.cap + old_from];
    }
    if (ok) {
      p.c.k[t] = k;
      p.c.v[t] = v;
    }
    bad |= !ok;
  }
  if (bad) record_error(p.c.err, kErrIndex, kSiteEvict);
}

constexpr int kEvictThreads = 512;  // two blocks per SM
constexpr int kEvictBins = 2048;       // digits of 11, 11 and 10 bits
constexpr int kEvictKeys = 16384;      // keys a block keeps in shared memory
constexpr int kEvictSmem = (kEvictBins + kEvictKeys + kEvictKeys / 32) * 4;
constexpr uint32_t kEvictMaxCluster = 8;

// Exclusive sum over the block's threads and the block's total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_tot, uint32_t& total) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= static_cast<uint32_t>(o)) inc += x;
  }
  __syncthreads();  // warp_tot is free
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  // every warp scans the warp totals
  const uint32_t w = lane < kEvictThreads / 32 ? warp_tot[lane] : 0u;
  uint32_t winc = w;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, winc, o);
    if (lane >= static_cast<uint32_t>(o)) winc += x;
  }
  total = __shfl_sync(0xffffffffu, winc, 31);
  return __shfl_sync(0xffffffffu, winc - w, warp) + inc - v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_u32(p), rank)));
  return v;
}

__device__ __forceinline__ uint4 ld_cluster_v4(const void* p, uint32_t rank) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(map_to_rank(smem_u32(p), rank)));
  return v;
}

// Grid (C h_kv, B), clusters of C blocks (C = 1, 2, 4, 8 by the capacity): the
// blocks of a cluster share a pair's slots, one contiguous piece each.  The
// threshold comes from a radix select over three digits, histograms summed
// over the cluster through distributed shared memory; then ranks of ties,
// holes and movers are exclusive sums over threads (a contiguous run of slots
// each), blocks and cluster, so that every list is in slot order.  Weights and
// positions are read once for the keys (kept in shared memory if the piece
// fits, re-read from L2 otherwise) and once for the slots that stay.
// Measured, 64 pairs of 65536 slots (four blocks each): 51 us, 61 % of the
// issue slots; one block per pair with four 8-bit digits, re-read each time,
// took 182 us, keys without the padding words 111 us (bank conflicts).
// MOVE: a cluster of one block moves its pair's rows itself (and writes
// new_lens, which then is not the lens array that other blocks still read).
template <bool MOVE>
__global__ void __launch_bounds__(kEvictThreads, 2)
    cache_evict_select_kernel(const EvictParams p, const uint32_t C) {
  extern __shared__ __align__(16) uint32_t ev_smem[];
  uint32_t* hist = ev_smem;
  uint32_t* keys = ev_smem + kEvictBins;
  __shared__ uint32_t wt[32];
  __shared__ uint32_t pick_sh[2];
  __shared__ uint32_t tot_sh[4];  // this block's ties, holes, movers
  const uint32_t tid = threadIdx.x, rank = C == 1 ? 0 : cluster_ctarank();
  const uint32_t hd = blockIdx.x / C, b = blockIdx.y;
  auto sync_all = [&]() {
    if (C == 1)
      __syncthreads();
    else
      cluster_sync();
  };
  bool bad = false;
  const uint32_t n = cache_len(p.c, b, bad);
  if (bad && tid == 0) record_error(p.c.err, kErrIndex, kSiteEvict);
  const long long bh = static_cast<long long>(b) * p.c.hkv + hd;
  const float* acc = p.acc + bh * p.c.cap;
  const int* pos = p.pos + bh * p.c.cap;
  float* acc_out = p.acc_out + bh * p.c.cap;
  int* pos_out = p.pos_out + bh * p.c.cap;
  if (MOVE && hd == 0 && tid == 0) p.new_lens[b] = static_cast<int>(min(n, p.budget));
  if (n <= p.budget) {  // the whole cluster
    for (uint32_t s = rank * kEvictThreads + tid; s < n; s += C * kEvictThreads) {
      acc_out[s] = acc[s];
      pos_out[s] = pos[s];
    }
    if (tid == 0 && rank == 0) p.count[bh] = 0;
    return;
  }
  const int sinks = static_cast<int>(p.sinks), since = evict_since(p, b);
  const uint32_t piece = (n + C - 1) / C;
  const uint32_t s0 = min(n, rank * piece), m = min(n, s0 + piece) - s0;  // slots s0 .. s0 + m - 1
  const bool fits = piece <= kEvictKeys;
  auto fresh_key = [&](uint32_t i) { return evict_key(acc[s0 + i], pos[s0 + i], sinks, since); };
  // (a word of padding every 32: threads that walk runs of slots meet no bank twice)
  auto at_key = [](uint32_t i) { return i + (i >> 5); };
  auto key_at = [&](uint32_t i) { return fits ? keys[at_key(i)] : fresh_key(i); };
  uint32_t prefix = 0, need = p.budget;  // slots to take among the keys with this prefix
#pragma unroll 1
  for (int d = 0; d < 3; ++d) {
    const int shift = d == 0 ? 21 : d == 1 ? 10 : 0, bits = d == 2 ? 10 : 11;
    const uint32_t bins = 1u << bits;
    for (uint32_t i = tid; i < kEvictBins; i += kEvictThreads) hist[i] = 0;
    __syncthreads();
    auto add = [&](uint32_t key) {
      if (d == 0 || (key >> (shift + bits)) == prefix)
        atomicAdd(&hist[(key >> shift) & (bins - 1)], 1u);
    };
    if (d == 0) {
      // eight independent pairs of loads at a time; protected slots share one
      // bin, so a warp counts them with one add
#pragma unroll 1
      for (uint32_t i0 = 0; i0 < m; i0 += 8 * kEvictThreads) {
        float w[8];
        int q[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t i = i0 + u * kEvictThreads + tid;
          w[u] = i < m ? acc[s0 + i] : 0.f;
          q[u] = i < m ? pos[s0 + i] : 0;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t i = i0 + u * kEvictThreads + tid;
          const uint32_t key = evict_key(w[u], q[u], sinks, since);
          const uint32_t safe = __ballot_sync(0xffffffffu, i < m && key == 0xFFFFFFFFu);
          if (i < m) {
            if (fits) keys[at_key(i)] = key;
            if (key != 0xFFFFFFFFu) add(key);
          }
          if (safe != 0 && (tid & 31) == 0) atomicAdd(&hist[bins - 1], __popc(safe));
        }
      }
    } else {
      for (uint32_t i = tid; i < m; i += kEvictThreads) add(key_at(i));
    }
    sync_all();
    // bins from the largest down, four per thread
    constexpr uint32_t kPer = kEvictBins / kEvictThreads;
    uint32_t h[kPer] = {}, sum = 0;
    if (kPer * tid < bins) {
      const uint32_t* at = hist + (bins - kPer * (tid + 1));
      if (C == 1) {
#pragma unroll
        for (uint32_t u = 0; u < kPer; ++u) h[u] = at[kPer - 1 - u];
      } else {
#pragma unroll 4
        for (uint32_t r = 0; r < C; ++r) {
          const uint4 v = ld_cluster_v4(at, r);
          h[0] += v.w;
          h[1] += v.z;
          h[2] += v.y;
          h[3] += v.x;
        }
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < kPer; ++u) sum += h[u];
    uint32_t all;
    uint32_t before = block_scan(sum, wt, all);
    if (before < need && before + sum >= need) {
#pragma unroll
      for (uint32_t u = 0; u < kPer; ++u) {
        if (before < need && before + h[u] >= need) {
          pick_sh[0] = bins - 1 - kPer * tid - u;
          pick_sh[1] = need - before;
        }
        before += h[u];
      }
    }
    sync_all();  // the histograms have been read by every block
    prefix = (prefix << bits) | pick_sh[0];
    need = pick_sh[1];
    __syncthreads();
  }
  // ranks: a contiguous run of slots per thread
  const uint32_t per = (m + kEvictThreads - 1) / kEvictThreads;
  const uint32_t i0 = min(m, tid * per), i1 = min(m, i0 + per);
  // totals of the lower blocks, entry e of tot_sh
  auto lower = [&](int e) {
    uint32_t v = 0;
    for (uint32_t r = 0; r < rank; ++r) v += ld_cluster_u32(tot_sh + e, r);
    return v;
  };
  uint32_t ties = 0, total;
  for (uint32_t i = i0; i < i1; ++i) ties += key_at(i) == prefix;
  uint32_t tie_rank = block_scan(ties, wt, total);
  if (tid == 0) tot_sh[0] = total;
  sync_all();
  tie_rank += lower(0);
  uint32_t holes_n = 0, movers_n = 0, tr = tie_rank;
  for (uint32_t i = i0; i < i1; ++i) {
    const uint32_t key = key_at(i);
    const bool kept = key > prefix || (key == prefix && tr < need);
    tr += key == prefix;
    holes_n += !kept && s0 + i < p.budget;
    movers_n += kept && s0 + i >= p.budget;
  }
  uint32_t th, tm;
  uint32_t hr = block_scan(holes_n, wt, th), mr = block_scan(movers_n, wt, tm);
  if (tid == 0) {
    tot_sh[1] = th;
    tot_sh[2] = tm;
  }
  sync_all();
  hr += lower(1);
  mr += lower(2);
  if (rank == C - 1 && tid == 0) p.count[bh] = static_cast<int>(lower(2) + tm);
  int* holes = p.lists + bh * p.c.cap;
  int* movers = holes + p.c.cap / 2;
  // What becomes of each slot: kNone, or its rank in its list.  If the keys are
  // in shared memory the ranks replace them there, and the copies and lists are
  // written by consecutive threads.
  constexpr uint32_t kNone = 0xFFFFFFFFu;
  auto put = [&](uint32_t s, uint32_t v) {
    if (s < p.budget) {
      if (v == kNone) {
        acc_out[s] = acc[s];
        pos_out[s] = pos[s];
      } else {
        holes[v] = static_cast<int>(s);
      }
    } else if (v != kNone) {
      movers[v] = static_cast<int>(s);
    }
  };
  tr = tie_rank;
  for (uint32_t i = i0; i < i1; ++i) {
    const uint32_t key = key_at(i), s = s0 + i;
    const bool kept = key > prefix || (key == prefix && tr < need);
    tr += key == prefix;
    uint32_t v = kNone;
    if (s < p.budget) {
      if (!kept) v = hr++;
    } else if (kept) {
      v = mr++;
    }
    if (fits)
      keys[at_key(i)] = v;
    else
      put(s, v);
  }
  if (fits) {
    __syncthreads();
    // four slots at a time, loads first
#pragma unroll 1
    for (uint32_t j = 0; j < m; j += 4 * kEvictThreads) {
      uint32_t v[4];
      float w[4];
      int q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t i = j + u * kEvictThreads + tid;
        v[u] = i < m ? keys[at_key(i)] : kNone;
        if (i < m && v[u] == kNone && s0 + i < p.budget) {
          w[u] = acc[s0 + i];
          q[u] = pos[s0 + i];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t i = j + u * kEvictThreads + tid, s = s0 + i;
        if (i >= m) continue;
        if (s >= p.budget) {
          if (v[u] != kNone) movers[v[u]] = static_cast<int>(s);
        } else if (v[u] != kNone) {
          holes[v[u]] = static_cast<int>(s);
        } else {
          acc_out[s] = w[u];
          pos_out[s] = q[u];
        }
      }
    }
  }
  if (C > 1) cluster_sync();  // no block leaves while another reads its words
  if constexpr (MOVE) {
    __syncthreads();
    evict_moves(p, hd, b, tm, 0u, 1u, kEvictThreads);
  }
}

// Grid (steps, h_kv, B).  Rows of 256 bytes from and to scattered places:
// 805 MB in 159 us (5.1 TB/s) for 64 pairs of 12288 moves.
__global__ void __launch_bounds__(kMoveThreads) cache_evict_move_kernel(const EvictParams p) {
  const uint32_t hd = blockIdx.y, b = blockIdx.z;
  bool bad = false;
  // (written here, behind every reader of lens, so that both may be one array)
  if (blockIdx.x == 0 && hd == 0 && threadIdx.x == 0)
    p.new_lens[b] = static_cast<int>(min(cache_len(p.c, b, bad), p.budget));
  const uint32_t count = static_cast<uint32_t>(p.count[static_cast<long long>(b) * p.c.hkv + hd]);
  evict_moves(p, hd, b, count, blockIdx.x, gridDim.x, kMoveThreads);
}

}  // namespace bpt

// Gradients of attention with a sliding window and sinks on the tcgen05
// tensor cores (the forward and its visibility rule: attn_window_tc.cuh).
//
// With s = q.k / sqrt(d_k), P = exp(s - m) / l from the forward's (m, l) and
// D = rowsum(dO * O), per head:
//   dP = dO V^T,  dS = P * (dP - D),
//   dV = P^T dO,  dK = dS^T Q / sqrt(d_k),  dQ = dS K / sqrt(d_k);
// dK and dV sum over the query heads that share a kv head.
//
// Four launches, all sums in a fixed order (no atomics on results):
//   window_terms_kernel   per row a' = -(m + ln l) log2 e and -D (reads o, dO
//                         once); for fp16 also the largest norms of rows of dO
//                         and V (reads V once).
//   window_dkv_tc_kernel  one CTA per 128 keys of a kv head (or a part of
//                         their queries): K, V stay, the (query head, query
//                         tile) pairs that see them stream through.
//   window_dq_tc_kernel   one CTA per 128 queries of a head: Q, dO stay, the
//                         key tiles that they see stream through.
//   window_join_kernel    adds the parts of blocks that were cut.
// 7 products of 2 d_k flops per pair for the 5 of the formulas: S and dP are
// computed twice, which keeps dQ out of memory and results independent of
// timing.  Measured at 16384 tokens, 16 heads of 128 on 4, window 2048, fp16: 0.84
// ms in bursts; one after the other and alone, dK/dV take 505 us (3000 clocks per
// 128 x 128 step for 2048 of products: P, dV and the next scores, which go where P
// lies, follow one another), dQ 379, terms 35, the join 7.
//
// The launches overlap (programmatic launches).  dK/dV blocks do all but the
// row terms while the last terms are written.  dQ needs the terms, not dK/dV:
// it may start once every dK/dV block has, and its short blocks fill the SMs
// that the last, long dK/dV blocks leave idle.  Its last block waits for the
// dK/dV grid before it ends, so that whatever follows finds both done.  One
// launch after the other took 896 us instead of 859, and 139 instead of 116 for
// eight ragged sequences of up to 2048 tokens, 12 heads of 64, window 256 (both
// with the rows stored as the lanes hold them; 841 and 100 since).
//
// Query tiles of a key block END at the last valid query that sees it, key
// tiles of a query block at its last visible key: nothing past a sequence's
// length is multiplied, so padding may hold anything.
//
// Key blocks that hold sinks are seen by every later query.  The (head, tile)
// items of a block are cut into parts of at most `part_len`, which is half of
// what an SM does in all, so that no CTA outlasts the rest; parts write fp32
// accumulators and the join adds them in order.
//
// Rounding: P and dS are rounded to the operands' type for the products.
// fp16 has 5 exponent bits, so there both are scaled by powers of two (exact).
// P by 2^8: weights down to 2^-22 stay out of the subnormals.  dS by what its
// range allows: |dP - D| <= 2 R with R = max |dO_i| max |v_j| (2-norms) over the
// rows of a (sequence, kv head), and the scale, between 2^13 / R and 2^14 / R,
// leaves |dS| below 2^15 for any finite values, and out of the subnormals down
// to 2^-27 R (an absolute error of 2^-38 R below that).  Sequences and kv heads
// have scales of their own: none loses bits to a neighbour.
#pragma once

#include <type_traits>

#include "attn_bwd_tc.cuh"
#include "attn_window_tc.cuh"

namespace bpt {

// Tiles that stream through a block have kWinTile<D> rows: 128 queries or keys
// at d_k = 128, where the accumulators leave room for one block per SM; 64 at
// d_k = 64, so that two blocks share an SM (256 of its 512 tensor memory
// columns each): with short windows a block has a few tiles only, and its own
// chain of products and elementwise phases leaves most of the SM idle.
template <int D>
constexpr int kWinTile = D == 128 ? 128 : 64;
// Warps: TMA, UMMA, TMEM owner, row terms (dK/dV only); then one elementwise
// warp per 32 rows and 32 columns of a tile: 16 at d_k = 128, four per
// scheduler (8 warps of 64 columns took twice what the tensor cores need: two
// warps per scheduler do not cover their own latencies).
template <int D>
constexpr int kWinElemWarps = 4 * kWinTile<D> / 32;
template <int D>
constexpr int kWinBwdThreads = 128 + 32 * kWinElemWarps<D>;
template <int D>
constexpr int kWinBwdBlocks = D == 128 ? 1 : 2;  // per SM
// Of every kWinBwdPolyEvery columns, kWinBwdPolyPairs pairs take their exp2
// from a cubic on the FMA pipe.
// Measured on 16384 tokens, 16 heads of 128 on 4, window 2048: one pair 917 us,
// two 911, three 925, four 937 for the whole backward.
constexpr int kWinBwdPolyEvery = 16, kWinBwdPolyPairs = 2;

struct WindowBwdParams {
  int nq, nkv, h, hkv, g, nqb, nblk;
  int window, sinks;
  const int* lens;        // nullable [B]
  const float2* terms;    // [B][h][nq]: (a', -D); (-inf, 0) past the length
  const uint2* range;     // fp16: [B][hkv] largest squared norms of dO's and V's rows; null: bf16
  void* dq;
  long long dq_b, dq_n, dq_h;
  void* dk;
  long long dk_b, dk_n, dk_h;
  void* dv;
  long long dv_b, dv_n, dv_h;
  float scale;            // 1 / sqrt(d_k)
  int part_len;           // items per part
  int split_parts;        // parts of cut blocks per (sequence, kv head)
  float* part;            // [B * hkv][split_parts][2][128][d_k]: dV, dK
  uint32_t* err;
};

// Launches that follow one another in a stream may overlap (programmatic
// launches): a grid starts once every block of the one before it has signalled
// (or ended), and waits where it needs that grid's results, which are complete
// and visible behind the wait.  No wait without such a launch: returns at once.
__device__ __forceinline__ void grid_signal() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Query tiles that see the 128 keys from kb, of queries before row `limit`.
struct WindowQueries {
  int start, end;  // rows; tiles end at `end`
  __host__ __device__ int tiles(int qt) const { return end > start ? (end - start + qt - 1) / qt : 0; }
};
__host__ __device__ inline WindowQueries window_queries(int nq, int nkv, int window, int sinks,
                                                        int kb, int limit) {
  const int off = nkv - nq;
  WindowQueries q;
  q.start = kb > off ? kb - off : 0;
  q.end = nq;
  if (kb >= sinks && kb + 127 + window - off < nq) q.end = kb + 127 + window - off;
  if (limit < q.end) q.end = limit;
  return q;
}
__host__ __device__ inline int window_parts(int nq, int nkv, int window, int sinks, int g, int kb,
                                            int qt, int part_len) {
  const int n = g * window_queries(nq, nkv, window, sinks, kb, nq).tiles(qt);
  return n <= part_len ? 1 : (n + part_len - 1) / part_len;
}

template <typename T>
struct WinScale {
  static constexpr float kP = std::is_same<T, __half>::value ? 8.f : 0.f;  // log2 of P's scale
};
// dS's scale: the power of two s with 2^13 <= s R < 2^14, R^2 the product of the
// two squared norms; 1 where that is no use (R = 0, or not finite).
__device__ __forceinline__ float grad_scale(const uint2* range, long long pair) {
  if (range == nullptr) return 1.f;
  const uint2 v = __ldcg(range + pair);
  const uint32_t e = __float_as_uint(__uint_as_float(v.x) * __uint_as_float(v.y)) >> 23;
  if (e == 0 || e >= 255) return 1.f;
  // R^2 in [2^(e - 127), 2^(e - 126)), R in [2^h, 2^(h + 1)) with h = floor((e - 127) / 2)
  const int h = (static_cast<int>(e) - 127) >> 1;
  return __uint_as_float(static_cast<uint32_t>(127 + 13 - h) << 23);
}

// ------------------------------------------------------------------- terms --
struct WindowTermsParams {
  const void* o;
  long long o_b, o_n, o_h;
  const void* d_o;
  long long d_b, d_n, d_h;
  const void* v;
  long long v_b, v_n, v_h;
  const float2* stats;  // [B][h][nq]
  float2* terms;
  uint32_t* range;      // nullable [B][hkv][2], zeros: see WindowBwdParams
  const int* lens;
  int nq, nkv, h, g;    // g = h / hkv
  uint32_t row_blocks;  // blocks of rows; those behind them have rows of V
  uint32_t* err;
};

constexpr int kTermRows = 4;  // rows per group of lanes, their loads in flight together
template <int D>
constexpr int kTermBlockRows = 256 / (D / 8) * kTermRows;

// Grid (blocks of one kv head's rows, hkv, B): D / 8 lanes per row (16 bytes of
// o and dO each), rows in (i, head of the group) order, a block's rows one group
// apart so that consecutive groups read on.
template <typename T, int D>
__global__ void __launch_bounds__(256) window_terms_kernel(const WindowTermsParams p) {
  grid_signal();
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes;
  constexpr bool kRange = std::is_same<T, __half>::value;
  const int kvh = blockIdx.y, b = blockIdx.z;
  int len = p.lens != nullptr ? __ldg(p.lens + b) : p.nkv;
  if (len < 0 || len > p.nkv) {
    if (threadIdx.x == 0) record_error(p.err, kErrIndex, kSiteWindowLens);
    len = len < 0 ? 0 : p.nkv;
  }
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  float mx = 0.f;  // the largest squared norm of this block's rows (of dO, or of V)
  uint4 a[kTermRows], c[kTermRows];
  bool valid[kTermRows];
  const bool values = kRange && blockIdx.x >= p.row_blocks;
  if (!values) {
    // the block's first row: one 64-bit division for all
    const long long r0 = static_cast<long long>(blockIdx.x) * kTermBlockRows<D>;
    const int i0 = static_cast<int>(r0 / p.g), t0 = static_cast<int>(r0 - static_cast<long long>(i0) * p.g);
    float2 ml[kTermRows];
    long long at[kTermRows];  // index into stats and terms; -1: no row
#pragma unroll
    for (int u = 0; u < kTermRows; ++u) {
      const uint32_t x = t0 + group + u * kGroups;
      const int i = i0 + static_cast<int>(x / static_cast<uint32_t>(p.g));
      const int t = kvh * p.g + static_cast<int>(x % static_cast<uint32_t>(p.g));
      at[u] = i < p.nq ? (static_cast<long long>(b) * p.h + t) * p.nq + i : -1;
      valid[u] = i < p.nq && p.nkv - p.nq + i < len;
      if (valid[u]) {
        a[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.o) + b * p.o_b +
                                                    i * p.o_n + t * p.o_h) + lane);
        c[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.d_o) + b * p.d_b +
                                                    i * p.d_n + t * p.d_h) + lane);
        if (lane == 0) ml[u] = __ldg(p.stats + at[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < kTermRows; ++u) {
      float sum = 0.f, norm = 0.f;
      if (valid[u]) {
        const uint32_t aw[4] = {a[u].x, a[u].y, a[u].z, a[u].w};
        const uint32_t cw[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = unpack16<T>(aw[k]), y = unpack16<T>(cw[k]);
          sum = fmaf(x.x, y.x, fmaf(x.y, y.y, sum));
          if constexpr (kRange) norm = fmaf(y.x, y.x, fmaf(y.y, y.y, norm));
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if constexpr (kRange) norm += __shfl_xor_sync(0xffffffffu, norm, o);
      }
      mx = fmaxf(mx, norm);
      if (at[u] >= 0 && lane == 0) {
        p.terms[at[u]] = valid[u] && ml[u].y > 0.f
                             ? make_float2(-(ml[u].x + logf(ml[u].y)) * kLog2e + WinScale<T>::kP, -sum)
                             : make_float2(-INFINITY, 0.f);
      }
    }
  } else {
    const long long j0 = static_cast<long long>(blockIdx.x - p.row_blocks) * kTermBlockRows<D>;
#pragma unroll
    for (int u = 0; u < kTermRows; ++u) {
      const long long j = j0 + group + u * kGroups;
      valid[u] = j < len;
      if (valid[u])
        c[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.v) + b * p.v_b +
                                                    j * p.v_n + kvh * p.v_h) + lane);
    }
#pragma unroll
    for (int u = 0; u < kTermRows; ++u) {
      float norm = 0.f;
      if (valid[u]) {
        const uint32_t cw[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 y = unpack16<T>(cw[k]);
          norm = fmaf(y.x, y.x, fmaf(y.y, y.y, norm));
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) norm += __shfl_xor_sync(0xffffffffu, norm, o);
      mx = fmaxf(mx, norm);
    }
  }
  if constexpr (kRange) {
    __shared__ uint32_t mx_sh[8];
    const uint32_t w = __reduce_max_sync(0xffffffffu, __float_as_uint(mx));
    if ((threadIdx.x & 31) == 0) mx_sh[threadIdx.x >> 5] = w;
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t m = 0;
      for (int k = 0; k < 8; ++k) m = max(m, mx_sh[k]);
      // (a maximum: the same in any order)
      if (m != 0)
        atomicMax(p.range + (static_cast<long long>(b) * gridDim.y + kvh) * 2 + (values ? 1 : 0), m);
    }
  }
}

// --------------------------------------------------------- elementwise parts --
// P of 32 columns from the scores, 2^(S c + a): kept in fp32 for dS (rounding
// it twice there would show), rounded once for the product with dO.
template <typename T, bool FULL, typename F>
__device__ __forceinline__ void win_p32(uint32_t (&sr)[32], uint32_t (&pk)[16], float c, F&& term,
                                        uint32_t vis) {
  const float2 c2 = make_float2(c, c);
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    const float2 x =
        __ffma2_rn(make_float2(__uint_as_float(sr[k]), __uint_as_float(sr[k + 1])), c2, term(k));
    float2 e;
    if ((k & (kWinBwdPolyEvery - 1)) >= kWinBwdPolyEvery - kWinBwdPolyPairs * 2)
      e = exp2_poly2(x);
    else
      e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
    if constexpr (!FULL) {
      if (!((vis >> k) & 1u)) e.x = 0.f;
      if (!((vis >> (k + 1)) & 1u)) e.y = 0.f;
    }
    sr[k] = __float_as_uint(e.x);
    sr[k + 1] = __float_as_uint(e.y);
    pk[k >> 1] = pack16<T>(e.x, e.y);
  }
}
// dS = P (dP sig + nd) of 32 columns.  (No mask: P is 0 where a key is not
// seen, and everything that is multiplied is finite but for the rows of keys
// past the length, which are stored as zeros.)
template <typename T, typename F>
__device__ __forceinline__ void win_ds32(const uint32_t (&dr)[32], const uint32_t (&pr)[32],
                                         uint32_t (&ds)[16], float sig, F&& nd) {
  const float2 s2 = make_float2(sig, sig);
#pragma unroll
  for (int k = 0; k < 32; k += 2) {
    const float2 v = __fmul2_rn(
        make_float2(__uint_as_float(pr[k]), __uint_as_float(pr[k + 1])),
        __ffma2_rn(make_float2(__uint_as_float(dr[k]), __uint_as_float(dr[k + 1])), s2, nd(k)));
    ds[k >> 1] = pack16<T>(v.x, v.y);
  }
}

template <int D>
struct WindowBwdCfg {
  static constexpr int QT = kWinTile<D>;
  static constexpr int TILE = 128 * D * 2;   // what stays: 128 rows
  static constexpr int STREAM = QT * D * 2;  // what streams through
  static constexpr int CHUNK = 128 * 128;    // 64 columns of 128 rows (d_k = 128 has two)
  // dK/dV: K, V, rings of Q (held from S_t to dK_t: three, so that the next
  // load never waits for a product in flight), dO (dP_t to dV_t) and row terms.
  // The barriers and shared words live behind them: with d_k = 128 the block
  // has no room for padding, so it has no static shared memory and its dynamic
  // part starts on the 1024-byte boundary that the swizzle needs.
  static constexpr int Q_SLOTS = D == 128 ? 3 : 4, DO_SLOTS = D == 128 ? 2 : 3, TERM_SLOTS = 2;
  static constexpr int KV_OFF_Q = 2 * TILE;
  static constexpr int KV_OFF_DO = KV_OFF_Q + Q_SLOTS * STREAM;
  static constexpr int KV_OFF_TERMS = KV_OFF_DO + DO_SLOTS * STREAM;
  static constexpr int KV_OFF_BAR = KV_OFF_TERMS + TERM_SLOTS * 2 * QT * 4;
  static constexpr int KV_SMEM = KV_OFF_BAR + 512;
  // dQ: Q, dO, rings of K (held until dQ_j) and V (until dP_j)
  static constexpr int QK_SLOTS = 3, QV_SLOTS = 2;
  static constexpr int Q_OFF_K = 2 * TILE;
  static constexpr int Q_OFF_V = Q_OFF_K + QK_SLOTS * STREAM;
  static constexpr int Q_OFF_BAR = Q_OFF_V + QV_SLOTS * STREAM;
  static constexpr int Q_SMEM = Q_OFF_BAR + 256 + 1024;
  static constexpr uint32_t COLS = D == 128 ? 512 : 256;  // tensor memory of a block
  static constexpr uint32_t TM_S = 0, TM_DP = QT, TM_DV = 2 * QT, TM_DK = 2 * QT + D;
  // dQ: one score buffer (free once its tile is in registers), two of dP / dS
  static constexpr uint32_t TQ_S = 0, TQ_DP = QT, TQ_A = 3 * QT;
  static_assert(TM_DK + D <= COLS && TQ_A + D <= COLS, "tensor memory");
  static_assert(kWinBwdBlocks<D> * (KV_SMEM + 1024) <= 233472 &&
                    kWinBwdBlocks<D> * (Q_SMEM + 1024) <= 233472, "shared memory");
};

// A 128-row product with A from tensor memory, 64 columns of A: the packed
// pairs of columns 32 c .. lie in words 32 c .. 32 c + 15.
template <int D>
__device__ __forceinline__ void win_issue_ts_half(uint32_t d, uint32_t a, uint32_t b_lo,
                                                  uint32_t idesc, int half, bool first) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int k = 4 * half + q;
    umma_ts(d, a + 32 * (k >> 1) + 8 * (k & 1), b_lo + ((k * 2048) >> 4), sdesc_hi(1024), idesc,
            (!first || k > 0) ? 1u : 0u);
  }
}

// Eight consecutive values of a row as 16 bytes.
template <typename T>
__device__ __forceinline__ uint4 win_pack8(const uint32_t* v, float f) {
  return make_uint4(pack16<T>(__uint_as_float(v[0]) * f, __uint_as_float(v[1]) * f),
                    pack16<T>(__uint_as_float(v[2]) * f, __uint_as_float(v[3]) * f),
                    pack16<T>(__uint_as_float(v[4]) * f, __uint_as_float(v[5]) * f),
                    pack16<T>(__uint_as_float(v[6]) * f, __uint_as_float(v[7]) * f));
}

// ------------------------------------------------------------------ dK, dV --
// Grid (parts of one (sequence, kv head), B * hkv).
template <typename T, int D>
__global__ void __launch_bounds__(kWinBwdThreads<D>, kWinBwdBlocks<D>)
    window_dkv_tc_kernel(const __grid_constant__ CUtensorMap mapQ,
                         const __grid_constant__ CUtensorMap mapK,
                         const __grid_constant__ CUtensorMap mapV,
                         const __grid_constant__ CUtensorMap mapDO, const WindowBwdParams p) {
  using C = WindowBwdCfg<D>;
  extern __shared__ __align__(128) uint8_t win_smem[];
  uint8_t* smem = win_smem;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::KV_OFF_BAR);
  const uint32_t kv_full = smem_u32(bars + 0);
  const uint32_t q_full0 = smem_u32(bars + 1);
  const uint32_t q_empty0 = smem_u32(bars + 5);
  const uint32_t do_full0 = smem_u32(bars + 9);
  const uint32_t do_empty0 = smem_u32(bars + 12);
  const uint32_t s_full = smem_u32(bars + 15);
  const uint32_t dp_full = smem_u32(bars + 16);
  const uint32_t p_half0 = smem_u32(bars + 17);   // [2]
  const uint32_t ds_half0 = smem_u32(bars + 19);  // [2]
  const uint32_t acc_done = smem_u32(bars + 21);
  const uint32_t drain = smem_u32(bars + 22);
  const uint32_t terms_full0 = smem_u32(bars + 23);   // [2]
  const uint32_t terms_empty0 = smem_u32(bars + 25);  // [2]
  // shared words: TMEM base, abort flag, plan (key block, part, first slot of
  // its parts or -1 if the block is not cut)
  int* words = reinterpret_cast<int*>(bars + 28);
  uint32_t* tmem_base_p = reinterpret_cast<uint32_t*>(words);
  int* abort_p = words + 1;
  int* plan_sh = words + 2;
  if ((smem_u32(smem) & 1023u) != 0) {  // (every thread: the swizzle would not match)
    record_error(p.err, kErrTimeout, kSiteAttnProducer);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bk = blockIdx.y;
  const int bidx = bk / p.hkv, kvh = bk - bidx * p.hkv;
  const int off = p.nkv - p.nq;
  int len = p.lens != nullptr ? __ldg(p.lens + bidx) : p.nkv;
  len = min(max(len, 0), p.nkv);

  if (warp == 3) {
    // the key block and part of this CTA: 32 blocks' parts at a time
    int at = 0, slot = 0;
    for (int b0 = 0; b0 < p.nblk; b0 += 32) {
      const int blk = b0 + lane;
      const int n = blk < p.nblk ? window_parts(p.nq, p.nkv, p.window, p.sinks, p.g, blk * 128,
                                                C::QT, p.part_len)
                                 : 0;
      int inc = n, sinc = n > 1 ? n : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, inc, o), c = __shfl_up_sync(0xffffffffu, sinc, o);
        if (lane >= o) {
          inc += a;
          sinc += c;
        }
      }
      const int first = at + inc - n, x = static_cast<int>(blockIdx.x);
      if (x >= first && x < first + n) {
        plan_sh[0] = blk;
        plan_sh[1] = x - first;
        plan_sh[2] = n > 1 ? slot + sinc - n : -1;
      }
      at += __shfl_sync(0xffffffffu, inc, 31);
      slot += __shfl_sync(0xffffffffu, sinc, 31);
      if (x < at) break;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < C::Q_SLOTS; ++s) {
      mbar_init(q_full0 + 8 * s, 1);
      mbar_init(q_empty0 + 8 * s, 1);
    }
    for (int s = 0; s < C::DO_SLOTS; ++s) {
      mbar_init(do_full0 + 8 * s, 1);
      mbar_init(do_empty0 + 8 * s, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    for (int c = 0; c < C::QT / 64; ++c) {
      mbar_init(p_half0 + 8 * c, 8);
      mbar_init(ds_half0 + 8 * c, 8);
    }
    for (int c = 0; c < C::TERM_SLOTS; ++c) {
      mbar_init(terms_full0 + 8 * c, 1);
      mbar_init(terms_empty0 + 8 * c, kWinElemWarps<D>);
    }
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    *abort_p = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_base_p), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_base_p;
  volatile int* abort_flag = abort_p;
  const int jb = plan_sh[0], part = plan_sh[1], slot0 = plan_sh[2];
  const int kb = jb * 128;
  const WindowQueries wq = window_queries(p.nq, p.nkv, p.window, p.sinks, kb, len - off);
  const int tiles = wq.tiles(C::QT);
  const int it0 = slot0 < 0 ? 0 : part * p.part_len;
  const int it1 = slot0 < 0 ? p.g * tiles : min(p.g * tiles, it0 + p.part_len);
  const int n_it = max(0, it1 - it0);
  // (head of the group, query tile) of item it0; tile t starts at row t0 + QT t
  const int hl0 = tiles > 0 ? it0 / tiles : 0, tl0 = it0 - hl0 * tiles;
  const int t0 = wq.end - C::QT * tiles;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    if (n_it > 0) {
      int q_armed[C::Q_SLOTS], do_armed[C::DO_SLOTS];
      for (int s = 0; s < C::Q_SLOTS; ++s) q_armed[s] = -1;
      for (int s = 0; s < C::DO_SLOTS; ++s) do_armed[s] = -1;
      if (leader) {
        mbar_arrive_expect_tx(kv_full, 2 * C::TILE);
        tma_load_5d(smem_u32(smem), &mapK, kv_full, 0, kb, 0, kvh, bidx);
        tma_load_5d(smem_u32(smem + C::TILE), &mapV, kv_full, 0, kb, 0, kvh, bidx);
      }
      int hl = hl0, tl = tl0;
      for (int t = 0; t < n_it; ++t) {
        const int qs = t % C::Q_SLOTS, ds = t % C::DO_SLOTS;
        const uint32_t qph = static_cast<uint32_t>((t / C::Q_SLOTS) & 1);
        const uint32_t dph = static_cast<uint32_t>((t / C::DO_SLOTS) & 1);
        // (the rings are full: what empties them waits for the terms, however
        // long that takes, so the bounded waits start behind it)
        if (t == C::DO_SLOTS) grid_wait();
        if (!mbar_wait_warp(q_empty0 + 8 * qs, qph ^ 1u, abort_flag, p.err, kSiteAttnProducer))
          break;
        q_armed[qs] = static_cast<int>(qph);
        if (leader) {
          mbar_arrive_expect_tx(q_full0 + 8 * qs, C::STREAM);
          tma_load_5d(smem_u32(smem + C::KV_OFF_Q + qs * C::STREAM), &mapQ, q_full0 + 8 * qs, 0,
                      t0 + C::QT * tl, 0, kvh * p.g + hl, bidx);
        }
        __syncwarp();
        if (!mbar_wait_warp(do_empty0 + 8 * ds, dph ^ 1u, abort_flag, p.err, kSiteAttnProducer))
          break;
        do_armed[ds] = static_cast<int>(dph);
        if (leader) {
          mbar_arrive_expect_tx(do_full0 + 8 * ds, C::STREAM);
          tma_load_5d(smem_u32(smem + C::KV_OFF_DO + ds * C::STREAM), &mapDO, do_full0 + 8 * ds, 0,
                      t0 + C::QT * tl, 0, kvh * p.g + hl, bidx);
        }
        __syncwarp();
        if (++tl == tiles) {
          tl = 0;
          ++hl;
        }
      }
      mbar_wait_drain(kv_full, 0, p.err);
      for (int s = 0; s < C::Q_SLOTS; ++s)
        if (q_armed[s] >= 0)
          mbar_wait_drain(q_full0 + 8 * s, static_cast<uint32_t>(q_armed[s]), p.err);
      for (int s = 0; s < C::DO_SLOTS; ++s)
        if (do_armed[s] >= 0)
          mbar_wait_drain(do_full0 + 8 * s, static_cast<uint32_t>(do_armed[s]), p.err);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- UMMA issue
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc16<T>(128, C::QT, false, false);
    constexpr uint32_t idesc_o = idesc16<T>(128, D, false, true);
    const uint32_t k_lo = sdesc_lo(smem_u32(smem), 16);
    const uint32_t v_lo = sdesc_lo(smem_u32(smem + C::TILE), 16);
    auto commit = [&](uint32_t bar) {
      if (leader) umma_commit(bar);
      __syncwarp();
    };
    auto q_slot = [&](int t) { return smem_u32(smem + C::KV_OFF_Q + (t % C::Q_SLOTS) * C::STREAM); };
    auto do_slot = [&](int t) {
      return smem_u32(smem + C::KV_OFF_DO + (t % C::DO_SLOTS) * C::STREAM);
    };
    auto issue_s = [&](int t) -> bool {
      if (!mbar_wait_warp(q_full0 + 8 * (t % C::Q_SLOTS),
                          static_cast<uint32_t>((t / C::Q_SLOTS) & 1), abort_flag, p.err,
                          kSiteAttnMma))
        return false;
      tc_fence_after();
      if (leader) bwd_issue_ss<D>(tmem + C::TM_S, k_lo, sdesc_lo(q_slot(t), 16), idesc_s);
      __syncwarp();
      commit(s_full);
      return true;
    };
    auto issue_dp = [&](int t) -> bool {
      if (!mbar_wait_warp(do_full0 + 8 * (t % C::DO_SLOTS),
                          static_cast<uint32_t>((t / C::DO_SLOTS) & 1), abort_flag, p.err,
                          kSiteAttnMma))
        return false;
      tc_fence_after();
      if (leader) bwd_issue_ss<D>(tmem + C::TM_DP, v_lo, sdesc_lo(do_slot(t), 16), idesc_s);
      __syncwarp();
      commit(dp_full);
      return true;
    };
    auto issue_grad = [&](int t, uint32_t bar0, uint32_t acc, uint32_t a_tm, uint32_t b_lo) {
      for (int hh = 0; hh < C::QT / 64; ++hh) {
        if (!mbar_wait_warp(bar0 + 8 * hh, static_cast<uint32_t>(t & 1), abort_flag, p.err,
                            kSiteAttnMma))
          return false;
        tc_fence_after();
        if (leader) win_issue_ts_half<D>(acc, a_tm, b_lo, idesc_o, hh, t == 0);
        __syncwarp();
      }
      return true;
    };
    bool ok = n_it > 0 && mbar_wait_warp(kv_full, 0, abort_flag, p.err, kSiteAttnMma) &&
              issue_s(0) && issue_dp(0);
    grid_wait();  // (as above: P comes behind the terms)
    for (int t = 0; t < n_it && ok; ++t) {
      // dV += P^T dO_t; then S^T_t has been read in full: the next scores go there
      if (!(ok = issue_grad(t, p_half0, tmem + C::TM_DV, tmem + C::TM_S,
                            sdesc_lo(do_slot(t), C::CHUNK))))
        break;
      commit(do_empty0 + 8 * (t % C::DO_SLOTS));
      if (t + 1 < n_it && !(ok = issue_s(t + 1))) break;
      // dK += dS^T Q_t; then dP^T_t has been read
      if (!(ok = issue_grad(t, ds_half0, tmem + C::TM_DK, tmem + C::TM_DP,
                            sdesc_lo(q_slot(t), C::CHUNK))))
        break;
      commit(q_empty0 + 8 * (t % C::Q_SLOTS));
      if (t + 1 < n_it) ok = issue_dp(t + 1);
    }
    commit(acc_done);
    commit(drain);
    mbar_wait_drain(drain, 0, p.err);
  } else if (warp == 3) {
    // ----------------------------------------------------------- row terms
    grid_wait();
    grid_signal();  // (behind the wait: the dQ blocks read the terms too)
    const float sig = grad_scale(p.range, bk) * exp2f(-WinScale<T>::kP);
    const float2* rows = p.terms + (static_cast<long long>(bidx) * p.h + kvh * p.g + hl0) * p.nq;
    int tl = tl0;
    for (int t = 0; t < n_it; ++t) {
      const int ts = t % C::TERM_SLOTS;
      float2 v[C::QT / 32];
#pragma unroll
      for (int q = 0; q < C::QT / 32; ++q) {
        const int i = t0 + C::QT * tl + lane + 32 * q;
        v[q] = i >= 0 ? __ldcg(rows + i) : make_float2(-INFINITY, 0.f);
      }
      if (!mbar_wait_warp(terms_empty0 + 8 * ts,
                          static_cast<uint32_t>((t / C::TERM_SLOTS) & 1) ^ 1u, abort_flag, p.err,
                          kSiteAttnProducer))
        break;
      float* st = reinterpret_cast<float*>(smem + C::KV_OFF_TERMS) + ts * 2 * C::QT;
#pragma unroll
      for (int q = 0; q < C::QT / 32; ++q) {
        st[lane + 32 * q] = v[q].x;
        st[C::QT + lane + 32 * q] = v[q].y * sig;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(terms_full0 + 8 * ts);
      if (++tl == tiles) {
        tl = 0;
        rows += p.nq;
      }
    }
  } else if (warp >= 4) {
    // --------------------------------------------------------- elementwise
    grid_wait();  // dS's range
    const int e = warp & 3, cc = (warp - 4) >> 2;  // columns 32 cc ..
    const int kr = e * 32 + lane, key = kb + kr;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(e * 32) << 16);
    const float c = p.scale * kLog2e;
    const float scale = grad_scale(p.range, bk);
    const float sig = scale * exp2f(-WinScale<T>::kP);
    int tl = tl0;
    bool ok = n_it > 0;
    for (int t = 0; t < n_it && ok; ++t) {
      const int ts = t % C::TERM_SLOTS;
      const float* st = reinterpret_cast<const float*>(smem + C::KV_OFF_TERMS) + ts * 2 * C::QT;
      const int pq = off + t0 + C::QT * tl;  // position of the tile's first query
      if (++tl == tiles) tl = 0;
      const uint32_t ph = static_cast<uint32_t>(t & 1);
      if (!mbar_wait_warp(terms_full0 + 8 * ts, static_cast<uint32_t>((t / C::TERM_SLOTS) & 1),
                          abort_flag, p.err, kSiteAttnSoftmax) ||
          !mbar_wait_warp(s_full, ph, abort_flag, p.err, kSiteAttnSoftmax)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // every key of the block is seen by every query of the tile
      const bool full = pq >= kb + 127 && (pq + C::QT - 1 < kb + p.window || kb + 128 <= p.sinks);
      const int q_lo = key - pq, q_hi = key < p.sinks ? C::QT : key + p.window - pq;
      const uint32_t vis = full ? 0xFFFFFFFFu : bits_range(q_lo, q_hi, cc);
      uint32_t pr[32], pk[16];
      tmem_ld_32x32b_x32(t_lane + C::TM_S + cc * 32, pr);
      tmem_ld_wait();
      auto term = [&](int k) { return *reinterpret_cast<const float2*>(st + cc * 32 + k); };
      if (full)
        win_p32<T, true>(pr, pk, c, term, vis);
      else
        win_p32<T, false>(pr, pk, c, term, vis);
      tmem_st16(t_lane + C::TM_S + cc * 32, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_half0 + 8 * (cc >> 1));
      if (!mbar_wait_warp(dp_full, ph, abort_flag, p.err, kSiteAttnSoftmax)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t dr[32];
      tmem_ld_32x32b_x32(t_lane + C::TM_DP + cc * 32, dr);
      tmem_ld_wait();
      auto nd = [&](int k) { return *reinterpret_cast<const float2*>(st + C::QT + cc * 32 + k); };
      win_ds32<T>(dr, pr, pk, sig, nd);
      tmem_st16(t_lane + C::TM_DP + cc * 32, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(ds_half0 + 8 * (cc >> 1));
        mbar_arrive(terms_empty0 + 8 * ts);
      }
    }
    const bool done = ok && mbar_wait_warp(acc_done, 0, abort_flag, p.err, kSiteAttnSoftmax);
    tc_fence_after();
    // even column groups store dV, odd ones dK, 64 columns each
    const int half = cc & 1, c0 = 64 * (cc >> 1);
    const float f = half == 0 ? exp2f(-WinScale<T>::kP) : p.scale / scale;
    const uint32_t acc = t_lane + (half == 0 ? C::TM_DV : C::TM_DK);
    if (slot0 >= 0) {
      if (done) {  // (a part without items writes nothing and is not read)
        // four columns of all 128 rows lie together: a warp writes 512 bytes at once
        float* dst = p.part + ((static_cast<long long>(bk) * p.split_parts + slot0 + part) * 2 + half) *
                                  (128 * D) + kr * 4;
#pragma unroll 1
        for (int x = c0; x < c0 + 64; x += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(acc + x, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 32; k += 4)
            *reinterpret_cast<float4*>(dst + (x + k) * 128) =
                make_float4(__uint_as_float(v[k]) * f, __uint_as_float(v[k + 1]) * f,
                            __uint_as_float(v[k + 2]) * f, __uint_as_float(v[k + 3]) * f);
        }
      }
    } else {
      // (staged where the queries were: every product is done)
      static_assert(kWinElemWarps<D> * 4096 <= C::Q_SLOTS * C::STREAM, "staging");
      uint8_t* st = smem + C::KV_OFF_Q + (warp - 4) * 4096;
#pragma unroll 1
      for (int x = 0; x < 8 && done; x += 4) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(acc + c0 + x * 8, v);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          *reinterpret_cast<uint4*>(st + stage_at<8>(lane, x + k)) = win_pack8<T>(v + 8 * k, f);
      }
      __syncwarp();
      T* dst = half == 0 ? static_cast<T*>(p.dv) + bidx * p.dv_b + kvh * p.dv_h
                         : static_cast<T*>(p.dk) + bidx * p.dk_b + kvh * p.dk_h;
      const long long dn = half == 0 ? p.dv_n : p.dk_n;
#pragma unroll 4
      for (int x = lane >> 3; x < 32; x += 4) {
        const int row = kb + e * 32 + x;
        if (row < p.nkv)  // (keys from the length on: no query sees them)
          *reinterpret_cast<uint4*>(dst + row * dn + c0 + (lane & 7) * 8) =
              done && row < len ? *reinterpret_cast<const uint4*>(st + stage_at<8>(x, lane & 7))
                                : make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, C::COLS);
}

// Grid (cut blocks, B * hkv, 8): 32 rows of dV or dK of one block each, the
// parts added in order.
template <typename T, int D>
__global__ void __launch_bounds__(256) window_join_kernel(const WindowBwdParams p) {
  grid_wait();
  const int bk = blockIdx.y, bidx = bk / p.hkv, kvh = bk - bidx * p.hkv;
  const int which = blockIdx.z & 1, quarter = blockIdx.z >> 1;
  int len = p.lens != nullptr ? __ldg(p.lens + bidx) : p.nkv;
  len = min(max(len, 0), p.nkv);
  // the blockIdx.x-th cut block and its first slot
  int blk = 0, slot = 0, seen = 0;
  for (;; ++blk) {
    const int n = window_parts(p.nq, p.nkv, p.window, p.sinks, p.g, blk * 128, kWinTile<D>, p.part_len);
    if (n <= 1) continue;
    if (seen == static_cast<int>(blockIdx.x)) break;
    ++seen;
    slot += n;
  }
  const int items = p.g * window_queries(p.nq, p.nkv, p.window, p.sinks, blk * 128,
                                         len - (p.nkv - p.nq)).tiles(kWinTile<D>);
  const int parts = (items + p.part_len - 1) / p.part_len;  // those that have items
  const float* src = p.part + (static_cast<long long>(bk) * p.split_parts + slot) * (2 * 128 * D) +
                     which * (128 * D);
  for (int x = threadIdx.x; x < 32 * D / 8; x += 256) {
    const int kr = quarter * 32 + x % 32, col = x / 32 * 8, key = blk * 128 + kr;
    if (key >= p.nkv) continue;
    float a[8] = {};
    if (key < len)
      for (int q = 0; q < parts; ++q) {
        const float4* s = reinterpret_cast<const float4*>(src + static_cast<long long>(q) * (2 * 128 * D) +
                                                          col * 128) + kr;
        const float4 u = s[0], v = s[128];
        a[0] += u.x; a[1] += u.y; a[2] += u.z; a[3] += u.w;
        a[4] += v.x; a[5] += v.y; a[6] += v.z; a[7] += v.w;
      }
    T* dst = which == 0 ? static_cast<T*>(p.dv) + bidx * p.dv_b + key * p.dv_n + kvh * p.dv_h
                        : static_cast<T*>(p.dk) + bidx * p.dk_b + key * p.dk_n + kvh * p.dk_h;
    *reinterpret_cast<uint4*>(dst + col) =
        make_uint4(pack16<T>(a[0], a[1]), pack16<T>(a[2], a[3]), pack16<T>(a[4], a[5]),
                   pack16<T>(a[6], a[7]));
  }
}

// ---------------------------------------------------------------------- dQ --
// Grid (query blocks, heads, B); the blocks with most keys first.
template <typename T, int D>
__global__ void __launch_bounds__(kWinBwdThreads<D>, kWinBwdBlocks<D>)
    window_dq_tc_kernel(const __grid_constant__ CUtensorMap mapQ,
                        const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ CUtensorMap mapV,
                        const __grid_constant__ CUtensorMap mapDO, const WindowBwdParams p) {
  using C = WindowBwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::Q_OFF_BAR);
  const uint32_t q_full = smem_u32(bars + 0);
  const uint32_t k_full0 = smem_u32(bars + 1);   // [3]
  const uint32_t k_empty0 = smem_u32(bars + 4);  // [3]
  const uint32_t v_full0 = smem_u32(bars + 7);   // [2]
  const uint32_t v_empty0 = smem_u32(bars + 9);  // [2]
  const uint32_t s_full = smem_u32(bars + 11);
  const uint32_t s_free = smem_u32(bars + 12);    // S_j is in every warp's registers
  const uint32_t dp_full0 = smem_u32(bars + 13);  // [2], by j % 2
  const uint32_t ds_half0 = smem_u32(bars + 15);  // [2][2]: by j % 2, columns 0..63 / 64..127
  const uint32_t acc_done = smem_u32(bars + 19);
  const uint32_t drain = smem_u32(bars + 20);
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int qb = p.nqb - 1 - static_cast<int>(blockIdx.x), head = blockIdx.y, bidx = blockIdx.z;
  const int kvh = head / p.g, off = p.nkv - p.nq;
  int len = p.lens != nullptr ? __ldg(p.lens + bidx) : p.nkv;
  len = min(max(len, 0), p.nkv);
  const int p0 = off + qb * 128;
  const int hi = min(off + min(p.nq, qb * 128 + 128), len);
  const bool any = hi > p0;
  const WindowKeys<C::QT> kt = window_keys<C::QT>(max(0, p0 - p.window + 1), hi, p.sinks, any);
  const int n_kv = kt.n_s + kt.n_w;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::QK_SLOTS; ++s) {
      mbar_init(k_full0 + 8 * s, 1);
      mbar_init(k_empty0 + 8 * s, 1);
    }
    for (int s = 0; s < C::QV_SLOTS; ++s) {
      mbar_init(v_full0 + 8 * s, 1);
      mbar_init(v_empty0 + 8 * s, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_free, kWinElemWarps<D>);
    for (int b = 0; b < 2; ++b) mbar_init(dp_full0 + 8 * b, 1);
    for (int b = 0; b < 4; ++b) mbar_init(ds_half0 + 8 * b, 8);  // 8 warps per 64 columns
    mbar_init(acc_done, 1);
    mbar_init(drain, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&tmem_base_sh), C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort_flag = &abort_sh;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool leader = elect_one();
    if (n_kv > 0) {
      int k_armed[C::QK_SLOTS], v_armed[C::QV_SLOTS];
      for (int s = 0; s < C::QK_SLOTS; ++s) k_armed[s] = -1;
      for (int s = 0; s < C::QV_SLOTS; ++s) v_armed[s] = -1;
      if (leader) {
        mbar_arrive_expect_tx(q_full, 2 * C::TILE);
        tma_load_5d(smem_u32(smem), &mapQ, q_full, 0, qb * 128, 0, head, bidx);
        tma_load_5d(smem_u32(smem + C::TILE), &mapDO, q_full, 0, qb * 128, 0, head, bidx);
      }
      for (int j = 0; j < n_kv; ++j) {
        const int ks = j % C::QK_SLOTS, vs = j % C::QV_SLOTS;
        const uint32_t kph = static_cast<uint32_t>((j / C::QK_SLOTS) & 1);
        const uint32_t vph = static_cast<uint32_t>((j / C::QV_SLOTS) & 1);
        const int key = kt.key(j);
        if (!mbar_wait_warp(k_empty0 + 8 * ks, kph ^ 1u, abort_flag, p.err, kSiteAttnProducer))
          break;
        k_armed[ks] = static_cast<int>(kph);
        if (leader) {
          mbar_arrive_expect_tx(k_full0 + 8 * ks, C::STREAM);
          tma_load_5d(smem_u32(smem + C::Q_OFF_K + ks * C::STREAM), &mapK, k_full0 + 8 * ks, 0, key, 0,
                      kvh, bidx);
        }
        __syncwarp();
        if (!mbar_wait_warp(v_empty0 + 8 * vs, vph ^ 1u, abort_flag, p.err, kSiteAttnProducer))
          break;
        v_armed[vs] = static_cast<int>(vph);
        if (leader) {
          mbar_arrive_expect_tx(v_full0 + 8 * vs, C::STREAM);
          tma_load_5d(smem_u32(smem + C::Q_OFF_V + vs * C::STREAM), &mapV, v_full0 + 8 * vs, 0, key, 0,
                      kvh, bidx);
        }
        __syncwarp();
      }
      mbar_wait_drain(q_full, 0, p.err);
      for (int s = 0; s < C::QK_SLOTS; ++s)
        if (k_armed[s] >= 0)
          mbar_wait_drain(k_full0 + 8 * s, static_cast<uint32_t>(k_armed[s]), p.err);
      for (int s = 0; s < C::QV_SLOTS; ++s)
        if (v_armed[s] >= 0)
          mbar_wait_drain(v_full0 + 8 * s, static_cast<uint32_t>(v_armed[s]), p.err);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- UMMA issue
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc16<T>(128, C::QT, false, false);
    constexpr uint32_t idesc_o = idesc16<T>(128, D, false, true);
    const uint32_t q_lo = sdesc_lo(smem_u32(smem), 16);
    const uint32_t do_lo = sdesc_lo(smem_u32(smem + C::TILE), 16);
    auto commit = [&](uint32_t bar) {
      if (leader) umma_commit(bar);
      __syncwarp();
    };
    auto k_slot = [&](int j) { return smem_u32(smem + C::Q_OFF_K + (j % C::QK_SLOTS) * C::STREAM); };
    auto v_slot = [&](int j) { return smem_u32(smem + C::Q_OFF_V + (j % C::QV_SLOTS) * C::STREAM); };
    auto issue_s = [&](int j) -> bool {
      if (!mbar_wait_warp(k_full0 + 8 * (j % C::QK_SLOTS),
                          static_cast<uint32_t>((j / C::QK_SLOTS) & 1), abort_flag, p.err,
                          kSiteAttnMma))
        return false;
      tc_fence_after();
      if (leader) bwd_issue_ss<D>(tmem + C::TQ_S, q_lo, sdesc_lo(k_slot(j), 16), idesc_s);
      __syncwarp();
      commit(s_full);
      return true;
    };
    auto issue_dp = [&](int j) -> bool {
      if (!mbar_wait_warp(v_full0 + 8 * (j % C::QV_SLOTS),
                          static_cast<uint32_t>((j / C::QV_SLOTS) & 1), abort_flag, p.err,
                          kSiteAttnMma))
        return false;
      tc_fence_after();
      if (leader)
        bwd_issue_ss<D>(tmem + C::TQ_DP + C::QT * static_cast<uint32_t>(j & 1), do_lo,
                        sdesc_lo(v_slot(j), 16), idesc_s);
      __syncwarp();
      commit(dp_full0 + 8 * (j & 1));
      commit(v_empty0 + 8 * (j % C::QV_SLOTS));
      return true;
    };
    bool ok = n_kv > 0 && mbar_wait_warp(q_full, 0, abort_flag, p.err, kSiteAttnMma) &&
              issue_s(0) && issue_dp(0);
    for (int j = 0; j < n_kv && ok; ++j) {
      if (j + 1 < n_kv) {
        // S_j+1 over S_j once that is in registers; dP_j+1 over dS_j-1, which
        // dQ_j-1 (issued before) has read
        ok = mbar_wait_warp(s_free, static_cast<uint32_t>(j & 1), abort_flag, p.err,
                            kSiteAttnMma);
        if (ok) tc_fence_after();
        ok = ok && issue_s(j + 1) && issue_dp(j + 1);
        if (!ok) break;
      }
      for (int hh = 0; hh < C::QT / 64; ++hh) {
        if (!mbar_wait_warp(ds_half0 + 16 * (j & 1) + 8 * hh, static_cast<uint32_t>((j >> 1) & 1),
                            abort_flag, p.err, kSiteAttnMma)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (leader)
          win_issue_ts_half<D>(tmem + C::TQ_A,
                               tmem + C::TQ_DP + C::QT * static_cast<uint32_t>(j & 1),
                               sdesc_lo(k_slot(j), C::CHUNK), idesc_o, hh, j == 0);
        __syncwarp();
      }
      if (!ok) break;
      commit(k_empty0 + 8 * (j % C::QK_SLOTS));
    }
    commit(acc_done);
    commit(drain);
    mbar_wait_drain(drain, 0, p.err);
  } else if (warp >= 4) {
    // --------------------------------------------------------- elementwise
    const int e = warp & 3, cc = (warp - 4) >> 2;  // columns 32 cc ..
    const int qr = e * 32 + lane, i = qb * 128 + qr, pos = p0 + qr;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(e * 32) << 16);
    const float c = p.scale * kLog2e;
    const float scale = grad_scale(p.range, static_cast<long long>(bidx) * p.hkv + kvh);
    const float sig = scale * exp2f(-WinScale<T>::kP);
    float2 tr = make_float2(-INFINITY, 0.f);
    if (i < p.nq) tr = __ldcg(p.terms + (static_cast<long long>(bidx) * p.h + head) * p.nq + i);
    const float2 a2 = make_float2(tr.x, tr.x), nd2 = make_float2(tr.y * sig, tr.y * sig);
    auto term = [&](int) { return a2; };
    auto nd = [&](int) { return nd2; };
    bool ok = n_kv > 0;
    for (int j = 0; j < n_kv && ok; ++j) {
      if (!mbar_wait_warp(s_full, static_cast<uint32_t>(j & 1), abort_flag, p.err,
                          kSiteAttnSoftmax)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t pr[32], pk[16];
      tmem_ld_32x32b_x32(t_lane + C::TQ_S + cc * 32, pr);
      const int kb = kt.key(j);
      const bool sink = j < kt.n_s;
      const bool full = !sink && kb + C::QT - 1 <= p0 && kb >= kt.lo && kb >= p0 + 128 - p.window;
      const uint32_t vis = full ? 0xFFFFFFFFu
                           : sink ? bits_range(0, kt.ns - kb, cc)
                                  : window_bits(pos, kb, kt.lo, p.window, p.sinks, cc);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free);
      if (full)
        win_p32<T, true>(pr, pk, c, term, vis);
      else
        win_p32<T, false>(pr, pk, c, term, vis);
      if (!mbar_wait_warp(dp_full0 + 8 * (j & 1), static_cast<uint32_t>((j >> 1) & 1), abort_flag,
                          p.err, kSiteAttnSoftmax)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tP = t_lane + C::TQ_DP + C::QT * static_cast<uint32_t>(j & 1) + cc * 32;
      uint32_t dr[32];
      tmem_ld_32x32b_x32(tP, dr);
      tmem_ld_wait();
      win_ds32<T>(dr, pr, pk, sig, nd);
      tmem_st16(tP, pk);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_half0 + 16 * (j & 1) + 8 * (cc >> 1));
    }
    const bool done = ok && mbar_wait_warp(acc_done, 0, abort_flag, p.err, kSiteAttnSoftmax);
    tc_fence_after();
    const float f = p.scale / scale;
    // 32 columns per warp, staged where the keys were: every product is done
    static_assert(D / 32 == C::QT / 32, "a column group per warp");
    static_assert(kWinElemWarps<D> * 2048 <= C::QK_SLOTS * C::STREAM, "staging");
    uint8_t* st = smem + C::Q_OFF_K + (warp - 4) * 2048;
    if (done) {
      uint32_t v[32];
      tmem_ld_32x32b_x32(t_lane + C::TQ_A + cc * 32, v);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        *reinterpret_cast<uint4*>(st + stage_at<4>(lane, k)) = win_pack8<T>(v + 8 * k, f);
    }
    __syncwarp();
    T* dst = static_cast<T*>(p.dq) + bidx * p.dq_b + head * p.dq_h + cc * 32;
#pragma unroll
    for (int x = lane >> 2; x < 32; x += 8) {
      const int row = qb * 128 + e * 32 + x;
      if (row < p.nq)
        *reinterpret_cast<uint4*>(dst + row * p.dq_n + (lane & 3) * 8) =
            done && off + row < len ? *reinterpret_cast<const uint4*>(st + stage_at<4>(x, lane & 3))
                                    : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, C::COLS);
  // the grid ends behind the dK/dV grid, for what follows in the stream
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1 && blockIdx.z == gridDim.z - 1)
    grid_wait();
}

}  // namespace bpt

// Attention with a sliding window and sinks on the tcgen05 tensor cores,
// forward.
//
// Query i stands at position p = nkv - nq + i and sees key j if
// j <= p < len and (p - j < window or j < sinks); heads h / h_kv share a
// key/value head.  Per row the online softmax keeps a reference maximum m, the
// sum l and the accumulator o:
//   S = Q K^T, P = exp2((S - m) log2(e)/sqrt(d_k)), l = alpha l + rowsum(P),
//   O = alpha O + P V; at the end o = O / l.
//
// Only key tiles that a row of the CTA sees are loaded: work is
// O(nq (window + sinks)), and the tensor cores bound it (4 d_k flops per
// visible pair against 2 bytes of K and V per key and 256 rows).
//
// A CTA owns one kv head and two 128-row query tiles A and B that are
// neighbours in the order (query block, head of the group): with shared heads
// both tiles have the same keys, without they are consecutive blocks.  Each
// K/V tile is loaded once for both.  Its keys are two lists of 128-key tiles:
// sink tiles (keys 0 .. min(sinks, lo) - 1 from key 0) and window tiles, which
// END at the last key any row sees, so that keys past a sequence's length are
// not touched, and start where they must (TMA rows need no alignment; keys
// before 0 read as zeros and are masked).  A tile that one of A and B does not
// see is skipped for it.
//
// The schedule is that of the dense kernel: warp 0 loads (TMA), warp 1 issues
// PV_A(j), S_A(j+1), PV_B(j), S_B(j+1) ..., four warps per tile run the
// softmax; P stays in tensor memory over S.  The reference moves only when a
// row's maximum grows by more than 2^8 (exp2 units; 2^6 in fp16).  P is rounded
// to the operands' type for the product with V, half a step per weight; scores,
// statistics and O are fp32; l sums the unrounded weights.  fp16 has its smallest
// step at 2^-24, and many small weights may count beside one large: there P and
// l are held 2^9 times as large, so that a weight is off by 2^-34 of the
// reference at most.
//
// Measured at 65536 tokens, 16 heads of 128, window 4096, 4 sinks: 1.95 ms in
// bursts (1093 TFLOP/s of visible pairs), 2.29 ms under the power cap.  With two
// threads per row (maxima exchanged through shared memory) it took 2.18 to 2.35
// ms: the exponentials of a tile keep the scheduler's unit busy as long, and the
// exchange comes on top.
//
// A score that is NaN or +inf makes its row NaN.  The cubic exponential would
// lose it (its clamp turns NaN into a weight of 2^-125), so the row maximum
// keeps NaN and a maximum that is not below +inf spoils the row's sum.
// A masked key has weight 0, but 0 x V_j is NaN if V_j holds NaN or infinity.
// The columns of a row that are not finite are therefore done again over the
// keys that it sees (window_row_again): exact, and free for finite values.
#pragma once

#include <type_traits>

#include "attn_pair_tc.cuh"
#include "cache.cuh"
#include "common.cuh"

namespace bpt {

enum : uint32_t { kSiteWindowLens = 19 };

struct WindowParams {
  int nq, nkv, h, hkv, g;   // g = h / hkv
  int units, npairs;        // per (sequence, kv head): query blocks x g; CTAs
  int window, sinks;
  const int* lens;          // nullable [B]
  const void* q;            // strided rows, elements (loads of rows done again)
  const void* k;
  const void* v;
  long long q_b, q_n, q_h, k_b, k_n, k_h, v_b, v_n, v_h;
  void* o;
  long long o_b, o_n, o_h;
  float scale_log2;         // log2(e) / sqrt(d_k)
  float2* stats;            // nullable [B][h][nq]: (m, l), (-inf, 0) for rows past the length
  uint32_t* err;
};

template <int D>
struct WindowCfg {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int CHUNK = 128 * 128;
  static constexpr int NSLOT = D == 128 ? 5 : 10;
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_BAR = OFF_RING + NSLOT * TILE;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t TMEM_COLS = 512;
  static constexpr uint32_t TM_S_B = 128, TM_O_A = 256, TM_O_B = 256 + D;
  static constexpr int THREADS = 384;
  // P hand-overs per 128-key tile to the issuing warp (measured on the dense
  // kernel: 64 keys at a time at d_k = 128, 32 at d_k = 64)
  static constexpr int HAND = D == 128 ? 2 : 4;
};

// Instruction descriptor of kind::f16 for this type (A, B: 0 fp16, 1 bf16).
template <typename T>
__host__ __device__ constexpr uint32_t idesc16(int M, int N, bool a_mn, bool b_mn) {
  const uint32_t f = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return idesc_f16_f32(M, N, a_mn, b_mn) | (f << 7) | (f << 10);
}

template <typename T>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value)
    return pack_f16x2(lo, hi);
  else
    return pack_bf16x2(lo, hi);
}
template <typename T>
__device__ __forceinline__ float2 unpack16(uint32_t v) {
  if constexpr (std::is_same<T, __half>::value)
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// Bits 0 .. n-1 of a word.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}
// Bits a .. b-1 of the word that holds bits 32 w ...
__device__ __forceinline__ uint32_t bits_range(int a, int b, int w) {
  return bits_below(b - 32 * w) & ~bits_below(a - 32 * w);
}

__device__ __forceinline__ int window_len(const WindowParams& p, int b) {
  if (p.lens == nullptr) return p.nkv;
  const int n = __ldg(p.lens + b);
  if (n < 0 || n > p.nkv) {
    if (threadIdx.x == 0) record_error(p.err, kErrIndex, kSiteWindowLens);
    return n < 0 ? 0 : p.nkv;
  }
  return n;
}

// Keys of a query tile: rows at positions p0 .. p0 + 127, the last valid one
// before `end`.
struct WindowTile {
  int p0, lo, hi;  // visible window keys lo .. hi - 1; hi <= p0: no valid row
  __device__ __forceinline__ bool any() const { return hi > p0; }
};
__device__ __forceinline__ WindowTile window_tile(const WindowParams& p, int qb, int len) {
  WindowTile t;
  const int off = p.nkv - p.nq;
  t.p0 = off + qb * 128;
  t.hi = min(off + min(p.nq, qb * 128 + 128), len);
  t.lo = max(0, t.p0 - p.window + 1);
  return t;
}

// The key tiles (KT keys) over which queries whose windows start at `lo` at the
// earliest and whose last visible key is hi - 1 run: sink tiles from key 0,
// then window tiles that end at hi.  Where the two would overlap, window tiles
// from key 0 serve both (so a sink tile never reaches past hi).
template <int KT = 128>  // keys per tile
struct WindowKeys {
  int lo, ns, n_s, n_w, w0;  // window keys from lo, sinks before it, tiles, first window tile's key
  __device__ __forceinline__ int key(int j) const { return j < n_s ? KT * j : w0 + KT * (j - n_s); }
};
template <int KT = 128>
__device__ __forceinline__ WindowKeys<KT> window_keys(int lo, int hi, int sinks, bool any) {
  WindowKeys<KT> k;
  k.lo = lo;
  k.ns = min(sinks, lo);
  k.n_s = any ? (k.ns + KT - 1) / KT : 0;
  if (lo < KT * k.n_s) k.lo = k.ns = k.n_s = 0;
  k.n_w = any ? (hi - k.lo + KT - 1) / KT : 0;
  k.w0 = hi - KT * k.n_w;
  return k;
}

// Rows leave through shared memory: a warp whose lanes hold a row each would
// touch 32 lines with every store (2000 clocks for a block's 128 x 128 rows of
// dK and dV), rows of NC 16-byte chunks over NC lanes touch 32 / NC.  Measured:
// gradients of eight ragged sequences of up to 2048 tokens, 12 heads of 64,
// window 256, 116 -> 100 us; forward of 200 tokens 11.6 -> 10.9.
// Byte offset of chunk c of a row in a warp's 32 rows; eight lanes meet no bank
// twice.
template <int NC>
__device__ __forceinline__ uint32_t stage_at(int row, int c) {
  return static_cast<uint32_t>(row * NC + (c ^ (NC >= 8 ? row & 7 : (row >> 1) & 3))) * 16u;
}

// The visible bits of keys kb + 32 w .. of a window tile for the row at p:
// keys lo .. p that are within the window or sinks.
__device__ __forceinline__ uint32_t window_bits(int p, int kb, int lo, int window, int sinks,
                                                int w) {
  const int top = p - kb + 1, low = lo - kb;
  return bits_range(max(p - window + 1 - kb, low), top, w) |
         bits_range(low, min(sinks - kb, top), w);
}

// P is exp2((S - m) c + kShift) with a reference m that moves when the row's
// maximum grows by more than 2^kGrow: at most 2^15 in fp16 (65504 is its
// largest value).  A smaller kGrow leaves room for a larger kShift, but O is
// scaled more often.  Measured in fp16 at 65536 tokens, 16 heads of 128, window
// 4096, 4 sinks, growth / shift 4 / 11, 5 / 10, 6 / 9, 7 / 8, 8 / 7: 2519, 2452,
// 2341, 2318, 2324 us under the power cap; 8 / 0: 2354.
template <typename T>
struct WindowScale {
  static constexpr float kShift = std::is_same<T, __half>::value ? 9.f : 0.f;
  static constexpr float kGrow = std::is_same<T, __half>::value ? 6.f : 8.f;
};

// kShift - m c: what is added to S c.  A row that has seen no key yet keeps 0
// (exp2(-inf) = 0); rounded down in fp16, so that P stays within its range for
// large scores.
template <typename T>
__device__ __forceinline__ float window_ref(float m, float c) {
  float ref = -m * c;
  if constexpr (WindowScale<T>::kShift != 0.f) ref = __fmaf_rd(-m, c, WindowScale<T>::kShift);
  return m == -INFINITY ? 0.f : ref;
}

// The largest of three values, NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float m;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// The columns of one row that are not finite, done again by a warp over the
// row's visible keys, with the row's own reference (ref = kShift - m c) and l,
// which masked keys do not touch: no dependence from key to key.  A value that is
// not finite counts whatever its weight (a positive one, if too small for fp32);
// a weight of 0 is a score of -inf.  32 keys at a time: D / 8 lanes take the
// product with one key, each lane the weight of one, then each lane D / 32 columns
// of V.  Stops once every such column is NaN; an l that is not a positive number
// leaves nothing to compute.  Measured at 16384 tokens, 8 heads of 64, window 4096,
// one infinity that every row of one head has in a tile: 7.3 ms (0.26 without it;
// 71 with the keys one after the other); one NaN in a sink: 0.28.
template <typename T, int D>
__device__ __noinline__ void window_row_again(const WindowParams& p, int b, int head, int i,
                                              float ref, float l) {
  constexpr int kL = D / 8, kK = 32 / kL;  // lanes of a key, keys at once
  constexpr int kC = D / 32;               // columns of a lane
  const int lane = threadIdx.x & 31;
  const int pos = p.nkv - p.nq + i, kvh = head / p.g;
  const T* k = static_cast<const T*>(p.k) + b * p.k_b + kvh * p.k_h + lane % kL * 8;
  const T* v = static_cast<const T*>(p.v) + b * p.v_b + kvh * p.v_h + lane * kC;
  T* dst = static_cast<T*>(p.o) + b * p.o_b + i * p.o_n + head * p.o_h + lane * kC;
  float o[kC];
  bool again[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    again[c] = !(fabsf(static_cast<float>(dst[c])) < INFINITY);
    o[c] = 0.f;
  }
  if (!(l > 0.f && l < INFINITY)) {
#pragma unroll
    for (int c = 0; c < kC; ++c) dst[c] = static_cast<T>(__uint_as_float(0x7FC00000u));
    return;
  }
  const float inv_l = 1.f / l;
  float q[8];
  {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + b * p.q_b +
                                                    i * p.q_n + head * p.q_h + lane % kL * 8);
    const uint32_t wq[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float2 x = unpack16<T>(wq[c]);
      q[2 * c] = x.x;
      q[2 * c + 1] = x.y;
    }
  }
  const int lo = max(0, pos - p.window + 1), ns = min(p.sinks, lo), n = ns + pos + 1 - lo;
  auto key_of = [&](int u) { return u < ns ? u : lo + (u - ns); };
  using Cols = typename std::conditional<kC == 2, uint32_t, uint2>::type;
  // (rows past the end are read as the last key's, and not used)
  auto load_v = [&](Cols(&to)[16], int u0) {
#pragma unroll
    for (int x = 0; x < 16; ++x)
      to[x] = __ldg(reinterpret_cast<const Cols*>(v + key_of(min(u0 + x, n - 1)) * p.v_n));
  };
#pragma unroll 1
  for (int u0 = 0; u0 < n; u0 += 32) {
    uint4 kr[kL];
#pragma unroll
    for (int x = 0; x < kL; ++x)
      kr[x] = __ldg(reinterpret_cast<const uint4*>(
          k + key_of(min(u0 + kK * x + lane / kL, n - 1)) * p.k_n));
    Cols vr[16];
    load_v(vr, u0);
    float s = -INFINITY;  // of key u0 + kK (lane % kL) + lane / kL
#pragma unroll
    for (int x = 0; x < kL; ++x) {
      const uint32_t wk[4] = {kr[x].x, kr[x].y, kr[x].z, kr[x].w};
      float d = 0.f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 y = unpack16<T>(wk[c]);
        d = fmaf(q[2 * c], y.x, fmaf(q[2 * c + 1], y.y, d));
      }
#pragma unroll
      for (int h = kL / 2; h > 0; h >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, h);
      if (x == lane % kL) s = d;
    }
    const float w =
        s == -INFINITY ? 0.f : fmaxf(ex2_approx(fmaf(s, p.scale_log2, ref)) * inv_l, 0x1p-126f);
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      if (h > 0) load_v(vr, u0 + h);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int at = h + x;
        const float wx = __shfl_sync(0xFFFFFFFFu, w, at % kK * kL + at / kK);
        if (u0 + at >= n) continue;
        const uint32_t* cols = reinterpret_cast<const uint32_t*>(&vr[x]);
#pragma unroll
        for (int c = 0; c < kC; c += 2) {
          const float2 y = unpack16<T>(cols[c / 2]);
          o[c] = fmaf(wx, y.x, o[c]);
          o[c + 1] = fmaf(wx, y.y, o[c + 1]);
        }
      }
    }
    bool settled = true;
#pragma unroll
    for (int c = 0; c < kC; ++c) settled &= !again[c] || o[c] != o[c];
    if (__all_sync(0xFFFFFFFFu, settled)) break;
  }
#pragma unroll
  for (int c = 0; c < kC; ++c)
    if (again[c]) dst[c] = static_cast<T>(o[c]);
}

// 16-column groups (of eight per row) whose exp2 runs as a cubic on the FMA
// pipe, so that it shares the work of the exponential unit (unmasked tiles).
// Measured at 65536 tokens, 16 heads of 128, window 4096: none 1961 us, one
// group 1942, two 1970, three 2021, four 2155.
constexpr uint32_t kWindowPolyGroups = 0x80u;

template <typename T, int D>
__global__ void __launch_bounds__(384, 1)
    attn_window_tc_kernel(const __grid_constant__ CUtensorMap mapQ,
                          const __grid_constant__ CUtensorMap mapK,
                          const __grid_constant__ CUtensorMap mapV, const WindowParams p) {
  using C = WindowCfg<D>;
  constexpr int kPerHand = 4 / C::HAND;  // 32-key chunks per hand-over
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  const uint32_t q_full = smem_u32(bars + 0);
  const uint32_t ring_full0 = smem_u32(bars + 1);
  const uint32_t ring_empty0 = smem_u32(bars + 1 + C::NSLOT);
  const uint32_t s_full0 = smem_u32(bars + 1 + 2 * C::NSLOT);   // [A, B]
  const uint32_t p_chunk0 = smem_u32(bars + 3 + 2 * C::NSLOT);  // [A: 0..3, B: 0..3]
  const uint32_t o_done0 = smem_u32(bars + 11 + 2 * C::NSLOT);  // [A, B]
  const uint32_t drain = smem_u32(bars + 13 + 2 * C::NSLOT);
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // within a (sequence, kv head): the last query blocks (most keys) first
  const int bk = blockIdx.x / p.npairs;
  const int pair = p.npairs - 1 - (static_cast<int>(blockIdx.x) - bk * p.npairs);
  const int bidx = bk / p.hkv, kvh = bk - bidx * p.hkv;
  const int len = window_len(p, bidx);
  const int uA = 2 * pair, uB = 2 * pair + 1;
  const bool has_b = uB < p.units;
  const int qbA = uA / p.g, qbB = has_b ? uB / p.g : qbA;
  const int headA = kvh * p.g + (uA - qbA * p.g);
  const int headB = has_b ? kvh * p.g + (uB - qbB * p.g) : headA;
  const WindowTile tA = window_tile(p, qbA, len), tB = window_tile(p, qbB, len);
  const bool anyA = tA.any(), anyB = has_b && tB.any();
  // (block A is never after block B: if A has no valid row, B has none)
  const WindowKeys<> kt = window_keys<>(tA.lo, anyB ? tB.hi : tA.hi, p.sinks, anyA);
  const int lo = kt.lo, ns = kt.ns, n_s = kt.n_s, w0 = kt.w0, n_kv = kt.n_s + kt.n_w;
  // tiles seen by a query tile: the sink tiles and first .. last (sinks past
  // lo lie in the window tiles, so there a tile starts at lo too)
  auto first_of = [&](const WindowTile& t) {
    return n_s + ((p.sinks > lo ? lo : t.lo) - w0) / 128;
  };
  auto last_of = [&](const WindowTile& t) { return n_s + (t.hi - 1 - w0) / 128; };
  const int fA = first_of(tA), lA = last_of(tA);
  const int fB = first_of(tB), lB = last_of(tB);
  auto seen = [&](int x, int j) {
    if (x == 0) return anyA && (j < n_s || (j >= fA && j <= lA));
    return anyB && (j < n_s || (j >= fB && j <= lB));
  };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(ring_full0 + 8 * s, 1);
      mbar_init(ring_empty0 + 8 * s, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full0 + 8 * x, 1);
      for (int c = 0; c < 4; ++c) mbar_init(p_chunk0 + 8 * (4 * x + c), 4);
      mbar_init(o_done0 + 8 * x, 1);
    }
    mbar_init(drain, 1);
    abort_sh = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&tmem_base_sh), C::TMEM_COLS);
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
    int armed[C::NSLOT];
    for (int s = 0; s < C::NSLOT; ++s) armed[s] = -1;
    if (n_kv > 0) {
      if (leader) {
        mbar_arrive_expect_tx(q_full, C::TILE * (anyB ? 2 : 1));
        tma_load_5d(smem_u32(smem), &mapQ, q_full, 0, qbA * 128, 0, headA, bidx);
        if (anyB) tma_load_5d(smem_u32(smem + C::TILE), &mapQ, q_full, 0, qbB * 128, 0, headB, bidx);
      }
      int slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int j = 0; j < n_kv && ok; ++j) {
        const int kb = kt.key(j);
        for (int w = 0; w < 2; ++w) {
          if (!mbar_wait_warp(ring_empty0 + 8 * slot, phase ^ 1u, abort_flag, p.err,
                              kSiteAttnProducer)) {
            ok = false;
            break;
          }
          armed[slot] = static_cast<int>(phase);
          if (leader) {
            mbar_arrive_expect_tx(ring_full0 + 8 * slot, C::TILE);
            tma_load_5d(smem_u32(smem + C::OFF_RING + slot * C::TILE), w == 0 ? &mapK : &mapV,
                        ring_full0 + 8 * slot, 0, kb, 0, kvh, bidx);
          }
          if (++slot == C::NSLOT) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      mbar_wait_drain(q_full, 0, p.err);
      for (int s = 0; s < C::NSLOT; ++s)
        if (armed[s] >= 0)
          mbar_wait_drain(ring_full0 + 8 * s, static_cast<uint32_t>(armed[s]), p.err);
    }
  } else if (warp == 1) {
    // ----------------------------------------------------------- UMMA issue
    const bool leader = elect_one();
    constexpr uint32_t idesc_s = idesc16<T>(128, 128, false, false);
    constexpr uint32_t idesc_o = idesc16<T>(128, D, false, true);
    constexpr uint32_t hi_w = sdesc_hi(1024);
    const uint32_t qa_lo = sdesc_lo(smem_u32(smem), 16);
    const uint32_t qb_lo = sdesc_lo(smem_u32(smem + C::TILE), 16);
    const uint32_t ring = smem_u32(smem + C::OFF_RING);
    auto slot_of = [&](int t) { return t % C::NSLOT; };
    auto phase_of = [&](int t) { return static_cast<uint32_t>((t / C::NSLOT) & 1); };
    auto commit = [&](uint32_t bar) {
      if (leader) umma_commit(bar);
      __syncwarp();
    };
    auto issue_s = [&](int x, uint32_t k_lo) {
      const uint32_t q_lo = x == 0 ? qa_lo : qb_lo, d_tmem = tmem + (x == 0 ? 0u : C::TM_S_B);
      if (leader) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * C::CHUNK + (k & 3) * 32) >> 4;
          umma_ss(d_tmem, q_lo + off, hi_w, k_lo + off, hi_w, idesc_s, k > 0 ? 1u : 0u);
        }
      }
      __syncwarp();
      commit(s_full0 + 8 * x);
    };
    uint32_t pph[2] = {0, 0};
    bool o_started[2] = {false, false};
    bool ok = n_kv > 0 && mbar_wait_warp(q_full, 0, abort_flag, p.err, kSiteAttnMma) &&
              mbar_wait_warp(ring_full0, 0, abort_flag, p.err, kSiteAttnMma);
    if (ok) {
      tc_fence_after();
      for (int x = 0; x < 2; ++x)
        if (seen(x, 0)) issue_s(x, sdesc_lo(ring, 16));
      commit(ring_empty0);
    }
    for (int j = 0; j < n_kv && ok; ++j) {
      const int tv = 2 * j + 1, tk = 2 * j + 2;  // ring positions of V_j and K_j+1
      if (!mbar_wait_warp(ring_full0 + 8 * slot_of(tv), phase_of(tv), abort_flag, p.err,
                          kSiteAttnMma))
        break;
      bool k_ready = false;
      const uint32_t v_lo = sdesc_lo(ring + slot_of(tv) * C::TILE, C::CHUNK);
      const uint32_t k_lo = sdesc_lo(ring + slot_of(tk) * C::TILE, 16);
      for (int x = 0; x < 2 && ok; ++x) {
        const bool now = seen(x, j), next = j + 1 < n_kv && seen(x, j + 1);
        if (now) {
          const uint32_t tS = tmem + (x == 0 ? 0u : C::TM_S_B);
          const uint32_t tO = tmem + (x == 0 ? C::TM_O_A : C::TM_O_B);
          for (int hh = 0; hh < C::HAND; ++hh) {
            if (!mbar_wait_warp(p_chunk0 + 8 * (4 * x + hh), pph[x], abort_flag, p.err,
                                kSiteAttnMma)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int q = 0; q < 2 * kPerHand; ++q) {
                const int k = 2 * hh * kPerHand + q;  // 16-key step
                umma_ts(tO, tS + 8 * k, v_lo + ((k * 2048) >> 4), hi_w, idesc_o,
                        (o_started[x] || k > 0) ? 1u : 0u);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          pph[x] ^= 1u;
          o_started[x] = true;
          if (j == (x == 0 ? lA : lB)) commit(o_done0 + 8 * x);
        }
        if (next) {
          if (!k_ready) {
            if (!mbar_wait_warp(ring_full0 + 8 * slot_of(tk), phase_of(tk), abort_flag, p.err,
                                kSiteAttnMma)) {
              ok = false;
              break;
            }
            k_ready = true;
          }
          issue_s(x, k_lo);
        }
      }
      if (!ok) break;
      commit(ring_empty0 + 8 * slot_of(tv));
      if (k_ready) commit(ring_empty0 + 8 * slot_of(tk));
    }
    commit(drain);
    mbar_wait_drain(drain, 0, p.err);
  } else if (warp >= 4) {
    // -------------------------------------------------------------- softmax
    const int x = (warp - 4) >> 2;  // 0: tile A, 1: tile B
    const int e = warp & 3;         // TMEM lane quarter
    const int r = e * 32 + lane;    // query row within the tile
    const bool any = x == 0 ? anyA : anyB;
    const int p0 = x == 0 ? tA.p0 : tB.p0;
    const int first = x == 0 ? fA : fB, last = x == 0 ? lA : lB;
    const int head = x == 0 ? headA : headB;
    const int i = (x == 0 ? qbA : qbB) * 128 + r;
    const int pos = p0 + r;
    const bool in_q = i < p.nq && (x == 0 || has_b);
    const bool valid = in_q && pos < len;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(e * 32) << 16);
    const uint32_t tS = t_lane + (x == 0 ? 0u : C::TM_S_B);
    const uint32_t tO = t_lane + (x == 0 ? C::TM_O_A : C::TM_O_B);
    const uint32_t s_full = s_full0 + 8 * x;
    const uint32_t p_chunk = p_chunk0 + 8 * (4 * x);
    const float c = p.scale_log2;
    float m_run = -INFINITY;   // reference maximum
    float m_true = -INFINITY;  // the row's exact maximum
    float l = 0.f;
    bool o_live = false;
    bool ok = any;
    uint32_t ph = 0;
    for (int j = n_s > 0 ? 0 : first; j <= last && ok; j = j + 1 == n_s ? first : j + 1) {
      if (!mbar_wait_warp(s_full, ph, abort_flag, p.err, kSiteAttnSoftmax)) {
        ok = false;
        break;
      }
      ph ^= 1u;
      tc_fence_after();
      uint32_t sr[128];
#pragma unroll
      for (int cc = 0; cc < 4; ++cc)
        tmem_ld_32x32b_x32(tS + cc * 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[cc * 32]));
      tmem_ld_wait();
      const int kb = kt.key(j);
      // a window tile that every row of the block sees whole
      const bool full = j >= n_s && kb + 127 <= p0 && kb >= lo && kb >= p0 + 128 - p.window;
      if (!full) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t vis = j < n_s ? bits_range(0, ns - kb, w)
                                       : window_bits(pos, kb, lo, p.window, p.sinks, w);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((vis >> k) & 1u)) sr[32 * w + k] = __float_as_uint(-INFINITY);
        }
      }
      float mxp[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) mxp[k] = -INFINITY;
#pragma unroll
      for (int k = 0; k < 128; k += 16)
#pragma unroll
        for (int q = 0; q < 8; ++q)
          mxp[q] = max3_nan(mxp[q], __uint_as_float(sr[k + q]), __uint_as_float(sr[k + 8 + q]));
      mxp[0] = max3_nan(mxp[0], mxp[1], mxp[2]);
      mxp[3] = max3_nan(mxp[3], mxp[4], mxp[5]);
      const float mx = max3_nan(mxp[0], mxp[3], max3_nan(mxp[6], mxp[7], mxp[7]));
      m_true = max3_nan(m_true, mx, mx);
      const float spoil = mx < INFINITY ? 0.f : __uint_as_float(0x7FC00000u);
      float m_new = m_run;
      bool need = false;
      if (mx > m_run) {
        need = (m_run == -INFINITY) || ((mx - m_run) * c > WindowScale<T>::kGrow);
        if (need) m_new = mx;
      }
      const bool warp_need = __any_sync(0xffffffffu, need) && o_live;
      const float alpha =
          need ? (m_run == -INFINITY ? 0.f : ex2_approx((m_run - m_new) * c)) : 1.f;
      if (warp_need) {
#pragma unroll 1
        for (int cc = 0; cc < D / 8; ++cc) {
          uint32_t v[8];
          tmem_ld_32x32b_x8(tO + cc * 8, v);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
          tmem_st_32x32b_x8(tO + cc * 8, v);
        }
      }
      const float ref = window_ref<T>(m_new, c);
      const float2 cc2 = make_float2(c, c), mref2 = make_float2(ref, ref);
      float2 sum2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                        make_float2(0.f, 0.f)};
      auto exp_row = [&](auto poly) {
        constexpr uint32_t kMask = decltype(poly)::value;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const int col = cc * 32 + k;
            const float2 a = __ffma2_rn(
                make_float2(__uint_as_float(sr[col]), __uint_as_float(sr[col + 1])), cc2, mref2);
            float2 e2;
            if ((kMask >> (col >> 4)) & 1u)
              e2 = exp2_poly2(a);
            else
              e2 = make_float2(ex2_approx(a.x), ex2_approx(a.y));
            sum2[(k >> 1) & 3] = __fadd2_rn(sum2[(k >> 1) & 3], e2);
            pk[k >> 1] = pack16<T>(e2.x, e2.y);
          }
          tmem_st_32x32b_x16(tS + cc * 16, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && (cc + 1) % kPerHand == 0) mbar_arrive(p_chunk + 8 * (cc / kPerHand));
        }
      };
      if (full)
        exp_row(std::integral_constant<uint32_t, kWindowPolyGroups>{});
      else
        exp_row(std::integral_constant<uint32_t, 0u>{});
      sum2[0] = __fadd2_rn(__fadd2_rn(sum2[0], sum2[1]), __fadd2_rn(sum2[2], sum2[3]));
      l = alpha * l + (sum2[0].x + sum2[0].y) + spoil;
      m_run = m_new;
      o_live = true;
    }
    if (ok) ok = mbar_wait_warp(o_done0 + 8 * x, 0, abort_flag, p.err, kSiteAttnSoftmax);
    if (ok || !any) {
      tc_fence_after();
      const float inv_l = valid ? 1.0f / l : 0.f;
      const float last_ref = window_ref<T>(m_run, c);
      if (p.stats != nullptr && in_q) {
        // in the units of s = q.k / sqrt(d_k): m the exact maximum, l relative to it
        const float m_s = m_true * c * 0.69314718055994531f;
        const float l_s = l * ex2_approx((m_run - m_true) * c - WindowScale<T>::kShift);
        p.stats[(static_cast<long long>(bidx) * p.h + head) * p.nq + i] =
            valid ? make_float2(m_s, l_s) : make_float2(-INFINITY, 0.f);
      }
      constexpr int NC = D / 8;
      uint8_t* st = smem + x * C::TILE + e * (32 * D * 2);  // the tile's Q rows: not needed any more
      float odd = 0.f;  // becomes NaN if an output is not finite
#pragma unroll 1
      for (int cc = 0; cc < D / 32 && any; ++cc) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tO + cc * 32, v);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float a = __uint_as_float(v[q * 8 + 2 * k]) * inv_l;
            const float b = __uint_as_float(v[q * 8 + 2 * k + 1]) * inv_l;
            odd = fmaf(a, 0.f, fmaf(b, 0.f, odd));
            w[k] = valid ? pack16<T>(a, b) : 0u;
          }
          *reinterpret_cast<uint4*>(st + stage_at<NC>(lane, 4 * cc + q)) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
      T* dst = static_cast<T*>(p.o) + bidx * p.o_b + head * p.o_h;
      const int rows = x == 0 || has_b ? p.nq - (i - lane) : 0;  // of this warp's 32
#pragma unroll 4
      for (int q = lane / NC; q < 32; q += 32 / NC)
        if (q < rows)
          *reinterpret_cast<uint4*>(dst + (i - lane + q) * p.o_n + lane % NC * 8) =
              any ? *reinterpret_cast<const uint4*>(st + stage_at<NC>(q, lane % NC))
                  : make_uint4(0u, 0u, 0u, 0u);
      uint32_t again = __ballot_sync(0xffffffffu, valid && odd != 0.f);
      if (again) {
        __syncwarp();
        for (; again; again &= again - 1) {
          const int rr = __ffs(again) - 1;
          window_row_again<T, D>(p, bidx, head, i - lane + rr,
                                 __shfl_sync(0xffffffffu, last_ref, rr),
                                 __shfl_sync(0xffffffffu, l, rr));
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace bpt

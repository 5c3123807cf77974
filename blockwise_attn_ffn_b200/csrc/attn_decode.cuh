// Attention of one new token per sequence over the paged key-value cache.
//
// Sequence b, head t (kv head t / (h / h_kv)), s_j = q . k_j / sqrt(d_k) over
// the visible slots j < len (all of them, or with a window the last `window`
// and the first `sinks`):  o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m).
//
// Bound: every visible row of K and V is read once from HBM; at 2-4 flops per
// byte and query head nothing else comes near.  So the kernel is built around
// a steady stream of loads:
//  - The work is the flat list of 64-slot tiles of all (sequence, kv head)
//    pairs, cut into equal runs, one per CTA (fewer runs if there are fewer tiles), whatever the lengths: a long
//    sequence is split over many CTAs, short ones share one.  The lengths are
//    read on the device, so no plan has to be made for a batch.
//  - The query heads that share a kv head are the 16 rows of one warp MMA
//    (m16n8k16), so each K/V row is read once for all of them.  (The legacy
//    MMA is enough here: padded to 16 rows it needs ~110 TFLOP/s at full HBM
//    rate, and a tcgen05 tile would pad to 128.)
//  - Each of the four warps takes 16 slots of a tile with its own ring of
//    cp.async stages and its own softmax state: no block barrier until a
//    (sequence, head) run ends.
// A run that covers all tiles of its pair writes the output; otherwise its
// unnormalised fp32 accumulator and (m, l) go to the workspace, and the join
// kernel combines them in run order (no atomics: results do not depend on
// timing).  P is rounded to the cache's type for the PV product (relative
// error half a step, averaged over the keys); scores, statistics and sums are
// fp32.
#pragma once

#include <type_traits>

#include "cache.cuh"
#include "common.cuh"

namespace bpt {

constexpr int kDecodeWarps = 4;
constexpr int kDecodeThreads = kDecodeWarps * 32;
constexpr int kDecodeTile = 16 * kDecodeWarps;  // slots per tile
constexpr int kDecodeRows = 16;                 // query heads per MMA
constexpr int kDecodeCtasPerSm = 2;
constexpr int kDecodeMaxSms = 160;               // the workspace holds partials for so many

struct DecodeParams {
  CacheView c;
  const void* q;
  long long q_b, q_h;  // strides, elements
  void* out;
  long long o_b, o_h;
  uint32_t B, h, g, chunks;  // g = h / h_kv; chunks of 16 heads per kv head
  uint32_t window, sinks;    // window 0: every slot
  float scale_log2;
  float* part_o;   // [2 * ctas][16][D]
  float2* part_ml; // [2 * ctas][16]
  float2* seg_ml;  // [B * h_kv * chunks][16]: (m, l) of pairs done by one CTA
  uint32_t ctas;   // grid of the split kernel
  float* scores;   // nullable [B][h][cap]: s log2(e) of visible slots
  const float* acc;  // nullable [B][h_kv][cap]
  float* acc_out;
};

// The visible slots of a sequence as a dense list: index u -> slot.
struct DecodeSeq {
  uint32_t len, n, ns, lo;  // n visible: the first ns, then lo .. len - 1
  __device__ __forceinline__ uint32_t slot(uint32_t u) const { return u < ns ? u : lo + (u - ns); }
  __device__ __forceinline__ uint32_t tiles() const { return (n + kDecodeTile - 1) / kDecodeTile; }
};

__device__ __forceinline__ DecodeSeq decode_seq(const DecodeParams& p, uint32_t b, bool& bad) {
  DecodeSeq s;
  s.len = cache_len(p.c, b, bad);
  s.lo = p.window != 0 && s.len > p.window ? s.len - p.window : 0;
  s.ns = min(p.sinks, s.lo);
  s.n = s.ns + (s.len - s.lo);
  return s;
}

// Run c covers tiles [W c / G, W (c + 1) / G).
__device__ __forceinline__ uint32_t run_start(uint32_t W, uint32_t G, uint32_t c) {
  return static_cast<uint32_t>(static_cast<unsigned long long>(W) * c / G);
}
// The run that covers tile x < W.
__device__ __forceinline__ uint32_t run_of(uint32_t W, uint32_t G, uint32_t x) {
  uint32_t c = static_cast<uint32_t>((static_cast<unsigned long long>(x) * G) / W);
  while (c + 1 < G && run_start(W, G, c + 1) <= x) ++c;
  return c;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int bytes = valid ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// D (+)= A B, 16 x 8 x 16, fp32 accumulate.
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value)
    return pack_f16x2(lo, hi);
  else
    return pack_bf16x2(lo, hi);
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (std::is_same<T, __half>::value)
    return __float2half_rn(v);
  else
    return __float2bfloat16_rn(v);
}

template <int D>
struct DecodeCfg {
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int SUB = 16 * D * 2;       // 16 rows of K or of V
  static constexpr int STAGE = 2 * SUB;
  static constexpr int RED_LD = D + 8;         // floats; 8 rows on different banks
  static constexpr int OFF_RED = kDecodeWarps * STAGES * STAGE;
  static constexpr int OFF_ML = OFF_RED + 16 * RED_LD * 4;
  static constexpr int SMEM = OFF_ML + kDecodeWarps * 16 * 8;
};

// Sum over the block of one value per thread.
__device__ __forceinline__ uint32_t block_sum_u32(uint32_t v, uint32_t* scratch) {
  v = __reduce_add_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t t = 0;
  for (uint32_t w = 0; w < (blockDim.x >> 5); ++w) t += scratch[w];
  __syncthreads();
  return t;
}

// All tiles of the batch; `per` = pairs per sequence (h_kv * chunks).
__device__ __forceinline__ uint32_t decode_total(const DecodeParams& p, uint32_t per,
                                                 uint32_t* scratch) {
  uint32_t v = 0;
  bool bad = false;
  for (uint32_t b = threadIdx.x; b < p.B; b += blockDim.x) v += decode_seq(p, b, bad).tiles() * per;
  return block_sum_u32(v, scratch);
}
// Tiles of the sequences before b.
__device__ __forceinline__ uint32_t decode_before(const DecodeParams& p, uint32_t b, uint32_t per,
                                                  uint32_t* scratch) {
  uint32_t v = 0;
  bool bad = false;
  for (uint32_t i = threadIdx.x; i < b; i += blockDim.x) v += decode_seq(p, i, bad).tiles() * per;
  return block_sum_u32(v, scratch);
}

template <typename T, int D>
__global__ void __launch_bounds__(kDecodeThreads, kDecodeCtasPerSm)
    attn_decode_split_kernel(const DecodeParams p) {
  using C = DecodeCfg<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t scratch[kDecodeWarps];
  __shared__ uint32_t find_sh[2];
  __shared__ uint32_t vmask[kDecodeWarps][C::STAGES];
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t per = p.c.hkv * p.chunks;
  const uint32_t W = decode_total(p, per, scratch);
  const uint32_t G = min(p.ctas, W);  // no run is empty
  if (blockIdx.x >= G) return;        // the whole block
  const uint32_t w0 = run_start(W, G, blockIdx.x), w1 = run_start(W, G, blockIdx.x + 1);
  // the sequence of tile w0: blocks of sequences, scanned until it is found
  uint32_t base = 0;
  for (uint32_t b0 = 0; b0 < p.B; b0 += kDecodeThreads) {
    bool bad = false;
    const uint32_t b = b0 + tid;
    const uint32_t mine = b < p.B ? decode_seq(p, b, bad).tiles() * per : 0;
    if (bad) record_error(p.c.err, kErrIndex, kSiteDecode);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= static_cast<uint32_t>(o)) inc += x;
    }
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    uint32_t off = base, tot = 0;
    for (uint32_t w = 0; w < kDecodeWarps; ++w) {
      if (w < warp) off += scratch[w];
      tot += scratch[w];
    }
    if (off + inc - mine <= w0 && w0 < off + inc) {
      find_sh[0] = b;
      find_sh[1] = off + inc - mine;
    }
    __syncthreads();
    base += tot;
    if (base > w0) break;
  }

  // A position in the tile list: sequence, pair in it, tile in the pair.
  struct Cursor {
    uint32_t b, pair, t, tiles;
    DecodeSeq s;
  };
  bool bad = false;
  Cursor cc;
  cc.b = find_sh[0];
  cc.s = decode_seq(p, cc.b, bad);
  cc.tiles = cc.s.tiles();
  cc.pair = (w0 - find_sh[1]) / cc.tiles;
  cc.t = (w0 - find_sh[1]) - cc.pair * cc.tiles;
  auto advance = [&](Cursor& c) {
    if (++c.t < c.tiles) return;
    c.t = 0;
    if (++c.pair < per) return;
    c.pair = 0;
    do {
      ++c.b;
      if (c.b >= p.B) {
        c.tiles = 0;
        return;
      }
      c.s = decode_seq(p, c.b, bad);
      c.tiles = c.s.tiles();
    } while (c.tiles == 0);
  };

  const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
  // the cache row of this lane's slot (lane % 16) of the tile at c; -1: none
  auto fetch_row = [&](const Cursor& c) -> int {
    const uint32_t u = c.t * kDecodeTile + warp * 16 + (lane & 15);
    if (c.tiles == 0 || u >= c.s.n) return -1;
    const int row = cache_row(p.c, c.b, c.pair / p.chunks, c.s.slot(u));
    bad |= row < 0;
    return row;
  };
  constexpr int kChunks = D / 8;             // 16-byte chunks of a row
  constexpr int kRowsPerOp = 32 / kChunks;   // rows one warp-wide copy covers
  auto issue = [&](uint32_t stage, int row) {
    const uint32_t ch = lane % kChunks, sub = lane / kChunks;
    const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
    for (int i = 0; i < 16 / kRowsPerOp; ++i) {
      const uint32_t r = i * kRowsPerOp + sub;
      const int rr = __shfl_sync(0xffffffffu, row, r);
      const long long off = rr < 0 ? 0 : static_cast<long long>(rr) * kChunks + ch;
      const uint32_t d = dst + r * (D * 2) + ((ch ^ (r & 7)) << 4);
      cp_async16(d, p.c.k + off, rr >= 0);
      cp_async16(d + C::SUB, p.c.v + off, rr >= 0);
    }
    const uint32_t m = __ballot_sync(0xffffffffu, row >= 0);
    if (lane == 0) vmask[warp][stage] = m & 0xFFFFu;
  };

  // fill the ring: the load cursor runs STAGES - 1 tiles ahead, its rows are
  // looked up one tile earlier still
  const uint32_t total = w1 - w0;
  Cursor lc = cc;
  uint32_t loaded = 0;
  int row_next = fetch_row(lc);
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if (loaded < total) {
      issue(s, row_next);
      advance(lc);
      ++loaded;
      row_next = loaded < total ? fetch_row(lc) : -1;
    }
    cp_async_commit();
  }

  uint32_t qf[D / 16][4];
  float o[D / 8][4];
  float m0, m1, l0, l1;
  const uint32_t r0 = lane >> 2, c0 = (lane & 3) * 2;
  bool fresh = true;        // the next tile starts a pair (or the run)
  uint32_t seg_t0 = cc.t;   // first tile of the current pair in this run
  bool first_seg = true;
  uint32_t stage = 0;
  for (uint32_t it = 0; it < total; ++it) {
    const uint32_t kvh = cc.pair / p.chunks, ck = cc.pair - kvh * p.chunks;
    const uint32_t head0 = kvh * p.g + ck * kDecodeRows;
    const uint32_t heads = min(static_cast<uint32_t>(kDecodeRows), p.g - ck * kDecodeRows);
    if (fresh) {
      fresh = false;
      seg_t0 = cc.t;
      const T* q = static_cast<const T*>(p.q) + cc.b * p.q_b + head0 * p.q_h;
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t row = r0 + (x & 1) * 8;
          qf[k][x] = row < heads ? __ldg(reinterpret_cast<const uint32_t*>(
                                       q + row * p.q_h + k * 16 + c0 + (x >> 1) * 8))
                                 : 0u;
        }
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
      m0 = m1 = -INFINITY;
      l0 = l1 = 0.f;
    }
    cp_async_wait<C::STAGES - 2>();
    __syncwarp();
    {
      uint32_t ls = stage + C::STAGES - 1;
      if (ls >= C::STAGES) ls -= C::STAGES;
      if (loaded < total) {
        issue(ls, row_next);
        advance(lc);
        ++loaded;
        row_next = loaded < total ? fetch_row(lc) : -1;
      }
      cp_async_commit();
    }
    const uint32_t kb = ring + stage * C::STAGE, vb = kb + C::SUB;
    const uint32_t valid = vmask[warp][stage];
    // S = Q K^T: 16 heads x 16 slots
    float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    {
      const uint32_t key = ((lane >> 4) << 3) + (lane & 7), kc = (lane >> 3) & 1;
      const uint32_t a = kb + key * (D * 2);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t r[4];
        ldsm_x4(r, a + (((2 * k + kc) ^ (key & 7)) << 4));
        mma_16816<T>(s[0], qf[k], r[0], r[1]);
        mma_16816<T>(s[1], qf[k], r[2], r[3]);
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        s[n][x] = ((valid >> (n * 8 + c0 + (x & 1))) & 1u) ? s[n][x] * p.scale_log2 : -INFINITY;
    if (p.scores != nullptr) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t row = r0 + (x >> 1) * 8;
          const uint32_t u = cc.t * kDecodeTile + warp * 16 + n * 8 + c0 + (x & 1);
          if (row < heads && u < cc.s.n)
            p.scores[(static_cast<long long>(cc.b) * p.h + head0 + row) * p.c.cap + cc.s.slot(u)] =
                s[n][x];
        }
    }
    float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
    float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 1));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 1));
    x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, 2));
    x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, 2));
    const float n0 = fmaxf(m0, x0), n1 = fmaxf(m1, x1);
    if (__any_sync(0xffffffffu, n0 > m0 || n1 > m1)) {
      const float a0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - n0);
      const float a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - n1);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= a0;
        o[n][1] *= a0;
        o[n][2] *= a1;
        o[n][3] *= a1;
      }
      l0 *= a0;
      l1 *= a1;
      m0 = n0;
      m1 = n1;
    }
    // a row that has seen nothing keeps reference 0: exp2(-inf) = 0
    const float f0 = m0 == -INFINITY ? 0.f : m0, f1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      s[n][0] = ex2_approx(s[n][0] - f0);
      s[n][1] = ex2_approx(s[n][1] - f0);
      s[n][2] = ex2_approx(s[n][2] - f1);
      s[n][3] = ex2_approx(s[n][3] - f1);
      l0 += s[n][0] + s[n][1];
      l1 += s[n][2] + s[n][3];
    }
    const uint32_t pf[4] = {pack2<T>(s[0][0], s[0][1]), pack2<T>(s[0][2], s[0][3]),
                            pack2<T>(s[1][0], s[1][1]), pack2<T>(s[1][2], s[1][3])};
    {
      const uint32_t key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
      const uint32_t a = vb + key * (D * 2);
#pragma unroll
      for (int n = 0; n < D / 16; ++n) {
        uint32_t r[4];
        ldsm_x4_t(r, a + (((2 * n + half) ^ (key & 7)) << 4));
        mma_16816<T>(o[2 * n], pf, r[0], r[1]);
        mma_16816<T>(o[2 * n + 1], pf, r[2], r[3]);
      }
    }
    if (++stage == C::STAGES) stage = 0;

    const bool pair_end = cc.t + 1 == cc.tiles;
    if (pair_end || it + 1 == total) {
      // join the four warps: reference maximum, then the accumulators
      l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
      l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
      l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
      float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
      float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
      if ((lane & 3) == 0) {
        ml[warp * 16 + r0] = make_float2(m0, l0);
        ml[warp * 16 + r0 + 8] = make_float2(m1, l1);
      }
      __syncthreads();
      float M[2], L[2], f[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t row = r0 + x * 8;
        M[x] = -INFINITY;
        for (int w = 0; w < kDecodeWarps; ++w) M[x] = fmaxf(M[x], ml[w * 16 + row].x);
        L[x] = 0.f;
        for (int w = 0; w < kDecodeWarps; ++w) {
          const float2 v = ml[w * 16 + row];
          L[x] += v.x == -INFINITY ? 0.f : v.y * ex2_approx(v.x - M[x]);
        }
        const float mine = x == 0 ? m0 : m1;
        f[x] = mine == -INFINITY ? 0.f : ex2_approx(mine - M[x]);
      }
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][0] *= f[0];
        o[n][1] *= f[0];
        o[n][2] *= f[1];
        o[n][3] *= f[1];
      }
      auto rows_do = [&](auto f) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t row = r0 + x * 8;
          if (row >= heads) continue;
          float* d = red + row * C::RED_LD + c0;
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
            f(reinterpret_cast<float2*>(d + n * 8), o[n][2 * x], o[n][2 * x + 1]);
        }
      };
      // warp 0 adds the others' accumulators in warp order, one buffer
#pragma unroll 1
      for (uint32_t w = 1; w < kDecodeWarps; ++w) {
        if (warp == w)
          rows_do([](float2* d, float& a, float& b) { *d = make_float2(a, b); });
        __syncthreads();
        if (warp == 0)
          rows_do([](float2* d, float& a, float& b) {
            const float2 v = *d;
            a += v.x;
            b += v.y;
          });
        __syncthreads();
      }
      if (warp == 0) {
        const bool whole = seg_t0 == 0 && pair_end;
        const uint32_t ps = blockIdx.x * 2 + (first_seg ? 0 : 1);
        const long long seg = static_cast<long long>(cc.b) * per + cc.pair;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t row = r0 + x * 8;
          if (row >= heads) continue;
          if ((lane & 3) == 0)
            (whole ? p.seg_ml + seg * 16 : p.part_ml + ps * 16LL)[row] = make_float2(M[x], L[x]);
          if (whole) {
            const float inv = L[x] > 0.f ? 1.f / L[x] : 0.f;
            T* dst = static_cast<T*>(p.out) + cc.b * p.o_b + (head0 + row) * p.o_h + c0;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<uint32_t*>(dst + n * 8) =
                  pack2<T>(o[n][2 * x] * inv, o[n][2 * x + 1] * inv);
          } else {
            float* dst = p.part_o + (ps * 16LL + row) * D + c0;
#pragma unroll
            for (int n = 0; n < D / 8; ++n)
              *reinterpret_cast<float2*>(dst + n * 8) = make_float2(o[n][2 * x], o[n][2 * x + 1]);
          }
        }
      }
      __syncthreads();  // ml is free again
      fresh = true;
      first_seg = false;
    }
    advance(cc);
  }
  cp_async_wait<0>();
  if (bad) record_error(p.c.err, kErrIndex, kSiteDecode);
}

constexpr int kJoinThreads = 256;
constexpr int kJoinSlots = 2048;  // slots of accumulated weight per block

// Where pair `seg` of sequence b lies: its tiles [s0, s1) and the runs lo..hi
// that hold it.  Partial of run c: its first pair unless the run began before.
struct DecodeSpan {
  uint32_t s0, s1, lo, hi, W, G;
  __device__ __forceinline__ uint32_t part(uint32_t c) const {
    return 2 * c + (run_start(W, G, c) < s0 ? 1 : 0);
  }
};
__device__ __forceinline__ DecodeSpan decode_span(const DecodeParams& p, uint32_t b, uint32_t pair,
                                                  uint32_t per, uint32_t tiles, uint32_t W,
                                                  uint32_t before) {
  DecodeSpan d;
  d.W = W;
  d.G = min(p.ctas, W);
  d.s0 = before + pair * tiles;
  d.s1 = d.s0 + tiles;
  d.lo = run_of(W, d.G, d.s0);
  d.hi = run_of(W, d.G, d.s1 - 1);
  return d;
}

// Grid (B * h_kv, 1 + slot blocks).  y = 0: joins the partial results of the
// pair's heads, one warp per head, and writes zeros for an empty sequence.
// y > 0: acc_out = acc + the weight each slot received, from the saved scores
// and the joined (m, l).
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attn_decode_join_kernel(const DecodeParams p) {
  __shared__ uint32_t scratch[kJoinThreads / 32];
  __shared__ float2 ml_sh[256];
  const uint32_t per = p.c.hkv * p.chunks;
  const uint32_t b = blockIdx.x / p.c.hkv, kvh = blockIdx.x - b * p.c.hkv;
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  bool bad = false;
  const DecodeSeq sq = decode_seq(p, b, bad);
  if (bad && tid == 0) record_error(p.c.err, kErrIndex, kSiteDecode);
  const uint32_t tiles = sq.tiles();
  if (blockIdx.y > 0 && (blockIdx.y - 1) * kJoinSlots >= sq.len) return;
  const uint32_t W = decode_total(p, per, scratch);
  const uint32_t before = decode_before(p, b, per, scratch);
  if (blockIdx.y == 0) {
    for (uint32_t r = warp; r < p.g; r += kJoinThreads / 32) {
      const uint32_t ck = r / kDecodeRows, row = r - ck * kDecodeRows;
      T* dst = static_cast<T*>(p.out) + b * p.o_b + (kvh * p.g + r) * p.o_h;
      if (tiles == 0) {
        for (uint32_t c = lane; c < D; c += 32) dst[c] = from_float<T>(0.f);
        continue;
      }
      const DecodeSpan sp = decode_span(p, b, kvh * p.chunks + ck, per, tiles, W, before);
      if (sp.lo == sp.hi) continue;  // written by its run
      float M = -INFINITY;
      for (uint32_t c = sp.lo; c <= sp.hi; ++c)
        M = fmaxf(M, p.part_ml[sp.part(c) * 16LL + row].x);
      float L = 0.f;
      float a[D / 32] = {};
      for (uint32_t c = sp.lo; c <= sp.hi; ++c) {
        const long long pr = sp.part(c) * 16LL + row;
        const float2 v = p.part_ml[pr];
        const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - M);
        L += v.y * f;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) a[k] += f * p.part_o[pr * D + k * 32 + lane];
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) dst[k * 32 + lane] = from_float<T>(a[k] * inv);
    }
    return;
  }
  // accumulated weights: (m, 1 / l) of the pair's heads first
  for (uint32_t r = tid; r < p.g; r += kJoinThreads) {
    if (tiles == 0) break;
    const uint32_t ck = r / kDecodeRows, row = r - ck * kDecodeRows;
    const uint32_t pair = kvh * p.chunks + ck;
    const DecodeSpan sp = decode_span(p, b, pair, per, tiles, W, before);
    float2 v;
    if (sp.lo == sp.hi) {
      v = p.seg_ml[(static_cast<long long>(b) * per + pair) * 16 + row];
    } else {
      v = make_float2(-INFINITY, 0.f);
      for (uint32_t c = sp.lo; c <= sp.hi; ++c)
        v.x = fmaxf(v.x, p.part_ml[sp.part(c) * 16LL + row].x);
      for (uint32_t c = sp.lo; c <= sp.hi; ++c) {
        const float2 y = p.part_ml[sp.part(c) * 16LL + row];
        v.y += y.x == -INFINITY ? 0.f : y.y * ex2_approx(y.x - v.x);
      }
    }
    ml_sh[r] = make_float2(v.x == -INFINITY ? 0.f : v.x, v.y > 0.f ? 1.f / v.y : 0.f);
  }
  __syncthreads();
  const long long a0 = (static_cast<long long>(b) * p.c.hkv + kvh) * p.c.cap;
  const float* sc = p.scores + (static_cast<long long>(b) * p.h + kvh * p.g) * p.c.cap;
  const uint32_t s_end = min(sq.len, blockIdx.y * kJoinSlots);
  for (uint32_t s = (blockIdx.y - 1) * kJoinSlots + tid; s < s_end; s += kJoinThreads) {
    float w = 0.f;
    if (s >= sq.lo || s < sq.ns)
      for (uint32_t r = 0; r < p.g; ++r)
        w += ex2_approx(sc[static_cast<long long>(r) * p.c.cap + s] - ml_sh[r].x) * ml_sh[r].y;
    p.acc_out[a0 + s] = p.acc[a0 + s] + w;
  }
}

}  // namespace bpt

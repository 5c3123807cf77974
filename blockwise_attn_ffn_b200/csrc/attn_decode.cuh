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
//    pairs, cut into equal runs, one per CTA (fewer if there are fewer tiles),
//    whatever the lengths: a long sequence is split over many CTAs, short ones
//    share one.  The lengths are
//    read on the device, so no plan has to be made for a batch.
//  - The query heads that share a kv head are the 8 columns of one warp MMA
//    (m16n8k16; two of them for more than 8 heads) whose 16 rows are slots:
//    S^T = K Q^T and O^T = V^T P^T, so each K/V row is read once for all heads
//    and little is padded.  (With the heads as the 16 rows, a batch with 4
//    heads per kv head spent 600 instructions per 16 slots and reached 5.0
//    TB/s.  The legacy MMA is enough here: a tcgen05 tile would pad the heads
//    to 128.)
//  - Each of the four warps takes 16 slots of a tile with its own ring of
//    cp.async stages and its own softmax state: no block barrier until a
//    (sequence, head) run ends.  The reference maximum moves only when it
//    grows by more than 2^8 (2^4 in fp16).
// A run that covers all tiles of its pair writes the output; otherwise its
// unnormalised fp32 accumulator and (m, l) go to the workspace, and the run
// that comes last (a counter per run that starts
// such a pair, left at zero again) joins the parts in
// run order: one launch, and results do not depend on timing.  A second kernel
// adds the weights up where they are wanted.  P is rounded to the cache's type
// for the PV product, half a step per weight; scores, statistics and sums are
// fp32.  fp16 has its smallest step at 2^-24, and many small weights may count
// beside one large: there P and l are held 2^11 times as large and the reference
// moves sooner, so that a weight is off by 2^-36 of the reference at most.
#pragma once

#include <type_traits>

#include "cache.cuh"
#include "common.cuh"

namespace bpt {

constexpr int kDecodeWarps = 4;
constexpr int kDecodeThreads = kDecodeWarps * 32;
constexpr int kDecodeTile = 16 * kDecodeWarps;  // slots per tile
// Blocks per SM and bytes of a block's ring.  Measured, 64 ragged sequences of
// up to 8192 slots, 8 kv heads of 128 with 4 query heads each: three blocks
// with two stages per warp 236 us (6.2 TB/s), two with three stages 243, one
// with six 321.  16 heads at once need 250 registers: two blocks.
template <int D, int NT>
struct DecodeShape {
  static constexpr int CTAS = NT == 2 ? 2 : D == 128 ? 3 : 4;
  static constexpr int RING = NT == 2 ? 98304 : D == 128 ? 65536 : 32768;
};
constexpr int kDecodeMaxCtas = 4;
constexpr int kDecodeMaxSms = 160;               // the workspace holds partials for so many

struct DecodeParams {
  CacheView c;
  const void* q;
  long long q_b, q_h;  // strides, elements
  void* out;
  long long o_b, o_h;
  uint32_t B, h, g, chunks;  // g = h / h_kv; chunks of `rows` heads per kv head
  uint32_t rows;             // 8 or 16
  uint32_t window, sinks;    // window 0: every slot
  float scale_log2;
  float* part_o;   // [2 * ctas][16][D]
  float2* part_ml; // [2 * ctas][16]: m, and l as P is scaled
  float2* seg_ml;  // [B * h_kv * chunks][16]: joined (m, l), where weights are wanted
  uint32_t* count; // [ctas]: parts that are done of the pair that run c starts and does not end
  uint32_t ctas;   // grid of the split kernel
  float* scores;   // nullable [B][h][scores_ld]: s log2(e) of the visible slots, dense
  long long scores_ld;
  const float* acc;  // nullable [B][h_kv][cap]
  float* acc_out;
};

// P is exp2(s - m + kShift) with a reference m that moves when the maximum grows
// by more than 2^kGrow: at most 2^15 in fp16 (65504 is its largest value).
template <typename T>
struct DecodeScale {
  static constexpr float kShift = std::is_same<T, __half>::value ? 11.f : 0.f;
  static constexpr float kGrow = std::is_same<T, __half>::value ? 4.f : 8.f;
  static constexpr float kUnit = std::is_same<T, __half>::value ? 0x1p-11f : 1.f;  // 2^-kShift
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
// Runs of W tiles: none is empty.  (Longer runs for short caches measured slower: a
// run pays 2 to 3 us for every pair that it ends, a part of a pair little more.)
__device__ __forceinline__ uint32_t decode_runs(const DecodeParams& p, uint32_t W) {
  return min(p.ctas, W);
}
// The run that covers tile x < W.
__device__ __forceinline__ uint32_t run_of(uint32_t W, uint32_t G, uint32_t x) {
  uint32_t c = static_cast<uint32_t>((static_cast<unsigned long long>(x) * G) / W);
  while (c + 1 < G && run_start(W, G, c + 1) <= x) ++c;
  return c;
}

// K and V rows are read once per call: in L2 they make room for one another
// first, not for the scores, the parts to join or what else the program keeps
// there.  Measured after writes that fill L2: 64 ragged sequences up to 8192
// slots, 32 heads of 128 on 8, with weights 291 -> 274 us; 131072 slots of one
// sequence 123 -> 111.  Without weights (249, 251), and call after call (266, 267;
// 335, 332), the difference is within noise.
__device__ __forceinline__ uint64_t evict_first_policy() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid,
                                           uint64_t policy) {
  const int bytes = valid ? 16 : 0;  // 0: the 16 bytes are zero-filled, nothing is read
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
               "l"(src), "r"(bytes), "l"(policy)
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
// Transposes an 8 x 8 matrix of 16-bit elements held as one register per lane.
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int NT>
struct DecodeCfg {
  static constexpr int ROWS = 8 * NT;          // query heads at once
  static constexpr int SUB = 16 * D * 2;       // 16 rows of K or of V
  static constexpr int STAGE = 2 * SUB;
  static constexpr int STAGES = DecodeShape<D, NT>::RING / (kDecodeWarps * STAGE);
  static constexpr int RED_LD = D + 4;         // floats; four head pairs and 8 rows meet 32 banks
  static constexpr int BUFS = NT == 1 ? 2 : 1;  // join buffers (16 heads: two blocks fill the SM)
  static constexpr int OFF_RED = kDecodeWarps * STAGES * STAGE;
  static constexpr int OFF_ML = OFF_RED + BUFS * ROWS * RED_LD * 4;
  static constexpr int SMEM = OFF_ML + kDecodeWarps * ROWS * 8;
  // (with 1 KB of the SM's and up to 1 KB of static shared memory per block)
  static_assert(DecodeShape<D, NT>::CTAS * (SMEM + 2048) <= 233472, "blocks per SM");
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
// Joins the parts of a pair that runs lo .. hi hold, by the whole block: the
// part of run c is its first one, but `second` says whether lo's is its second
// (the run began in an earlier pair).  Parts come from other SMs: read past L1.
template <typename T, int D>
__device__ __noinline__ void decode_join(const DecodeParams& p, uint32_t lo, uint32_t hi,
                                         uint32_t second, uint32_t heads, long long seg, T* out) {
  constexpr uint32_t kLanes = D / 4;  // threads of a row, four columns each
  const uint32_t col = threadIdx.x % kLanes * 4;
  for (uint32_t row = threadIdx.x / kLanes; row < heads; row += kDecodeThreads / kLanes) {
    auto at = [&](uint32_t c) { return (2LL * c + (c == lo ? second : 0u)) * 16 + row; };
    float M = -INFINITY;
#pragma unroll 4
    for (uint32_t c = lo; c <= hi; ++c) M = fmaxf(M, __ldcg(p.part_ml + at(c)).x);
    float L = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (uint32_t c = lo; c <= hi; ++c) {
      const float2 v = __ldcg(p.part_ml + at(c));
      const float4 x = __ldcg(reinterpret_cast<const float4*>(p.part_o + at(c) * D + col));
      const float f = v.x == -INFINITY ? 0.f : ex2_approx(v.x - M);
      L += v.y * f;
      a.x += f * x.x;
      a.y += f * x.y;
      a.z += f * x.z;
      a.w += f * x.w;
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;
    if (p.scores != nullptr && col == 0)
      p.seg_ml[seg * 16 + row] = make_float2(M, L * DecodeScale<T>::kUnit);
    *reinterpret_cast<uint2*>(out + row * p.o_h + col) =
        make_uint2(pack2<T>(a.x * inv, a.y * inv), pack2<T>(a.z * inv, a.w * inv));
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kDecodeThreads, (DecodeShape<D, NT>::CTAS))
    attn_decode_split_kernel(const DecodeParams p) {
  using C = DecodeCfg<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t scratch[kDecodeWarps];
  __shared__ uint32_t find_sh[2], join_sh[4];
  __shared__ uint32_t vmask[kDecodeWarps][C::STAGES];
  const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t per = p.c.hkv * p.chunks;
  // All tiles of the batch, W, cut into G runs (none empty), and the sequence of
  // this run's first tile, w0: with up to 128 sequences in one pass over the
  // lengths, else one for W and one that stops at w0.
  uint32_t W = 0, G = 0, w0 = 0, w1 = 0, base = 0;
  const bool one_pass = p.B <= kDecodeThreads;
  if (!one_pass) {
    W = decode_total(p, per, scratch);
    G = decode_runs(p, W);
    w0 = run_start(W, G, blockIdx.x);
  }
  for (uint32_t b0 = 0; b0 < p.B; b0 += kDecodeThreads) {
    bool bad = false;
    const uint32_t b = b0 + tid;
    const uint32_t mine = b < p.B ? decode_seq(p, b, bad).tiles() * per : 0;
    if (bad && blockIdx.x == 0) record_error(p.c.err, kErrIndex, kSiteDecode);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= static_cast<uint32_t>(o)) inc += x;
    }
    if (lane == 31) scratch[warp] = inc;
    // sequences without visible slots: zeros, by block b % grid
    if (b < p.B && mine == 0 && b % gridDim.x == blockIdx.x)
      for (uint32_t x = 0; x < p.h * (D / 8); ++x)
        *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + b * p.o_b + (x / (D / 8)) * p.o_h +
                                  x % (D / 8) * 8) = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    uint32_t off = base, tot = 0;
    for (uint32_t w = 0; w < kDecodeWarps; ++w) {
      if (w < warp) off += scratch[w];
      tot += scratch[w];
    }
    if (one_pass) {
      W = tot;
      G = decode_runs(p, W);
      w0 = run_start(W, G, blockIdx.x);
    }
    if (blockIdx.x < G && off + inc - mine <= w0 && w0 < off + inc) {
      find_sh[0] = b;
      find_sh[1] = off + inc - mine;
    }
    __syncthreads();
    base += tot;
  }
  if (blockIdx.x >= G) return;  // the whole block
  w1 = run_start(W, G, blockIdx.x + 1);

  // A position in the tile list: sequence, pair in it, tile in the pair.
  struct Cursor {
    uint32_t b, pair, t, tiles;
    uint32_t base;  // first tile of the sequence in the list
    DecodeSeq s;
  };
  bool bad = false;
  Cursor cc;
  cc.b = find_sh[0];
  cc.base = find_sh[1];
  cc.s = decode_seq(p, cc.b, bad);
  cc.tiles = cc.s.tiles();
  cc.pair = (w0 - find_sh[1]) / cc.tiles;
  cc.t = (w0 - find_sh[1]) - cc.pair * cc.tiles;
  auto advance = [&](Cursor& c) {
    if (++c.t < c.tiles) return;
    c.t = 0;
    if (++c.pair < per) return;
    c.pair = 0;
    c.base += per * c.tiles;
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
    const int row = cache_row(p.c, c.b, p.chunks == 1 ? c.pair : c.pair / p.chunks, c.s.slot(u));
    bad |= row < 0;
    return row;
  };
  constexpr int kChunks = D / 8;             // 16-byte chunks of a row
  constexpr int kRowsPerOp = 32 / kChunks;   // rows one warp-wide copy covers
  const uint64_t policy = evict_first_policy();
  auto issue = [&](uint32_t stage, int row) {
    const uint32_t ch = lane % kChunks, sub = lane / kChunks;
    const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
    for (int i = 0; i < 16 / kRowsPerOp; ++i) {
      const uint32_t r = i * kRowsPerOp + sub;
      const int rr = __shfl_sync(0xffffffffu, row, r);
      const long long off = rr < 0 ? 0 : static_cast<long long>(rr) * kChunks + ch;
      const uint32_t d = dst + r * (D * 2) + ((ch ^ (r & 7)) << 4);
      cp_async16(d, p.c.k + off, rr >= 0, policy);
      cp_async16(d + C::SUB, p.c.v + off, rr >= 0, policy);
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

  uint32_t qb[NT][D / 16][2];   // Q^T: columns are heads
  float o[D / 16][NT][4];       // O^T: rows 16 i + r0 (+ 8), heads 8 nt + c0 (+ 1)
  float m[NT][2], l[NT][2];     // per head; l over this lane's slots
  const uint32_t r0 = lane >> 2, c0 = (lane & 3) * 2;
  bool fresh = true;        // the next tile starts a pair (or the run)
  uint32_t seg_t0 = cc.t;   // first tile of the current pair in this run
  bool first_seg = true;
  uint32_t stage = 0, head0 = 0, heads = 0;
  float* score = nullptr;   // this lane's first head's row
  for (uint32_t it = 0; it < total; ++it) {
    if (fresh) {
      fresh = false;
      seg_t0 = cc.t;
      const uint32_t kvh = cc.pair / p.chunks, ck = cc.pair - kvh * p.chunks;
      head0 = kvh * p.g + ck * C::ROWS;
      heads = min(static_cast<uint32_t>(C::ROWS), p.g - ck * C::ROWS);
      const T* q = static_cast<const T*>(p.q) + cc.b * p.q_b + head0 * p.q_h;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            qb[nt][k][x] = 8 * nt + r0 < heads
                               ? __ldg(reinterpret_cast<const uint32_t*>(
                                     q + (8 * nt + r0) * p.q_h + k * 16 + c0 + 8 * x))
                               : 0u;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) o[i][nt][x] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
      }
      if (p.scores != nullptr)
        score = p.scores + (static_cast<long long>(cc.b) * p.h + head0 + c0) * p.scores_ld;
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
    // S^T = K Q^T: 16 slots x heads, even and odd steps apart (shorter chains)
    float s[NT][4] = {}, s2[NT][4] = {};
    {
      const uint32_t key = (((lane >> 3) & 1) << 3) + (lane & 7), kc = lane >> 4;
      const uint32_t a = kb + key * (D * 2);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t r[4];
        ldsm_x4(r, a + (((2 * k + kc) ^ (key & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma_16816<T>((k & 1) ? s2[nt] : s[nt], r, qb[nt][k][0], qb[nt][k][1]);
      }
    }
    const bool part_tile = valid != 0xFFFFu;
    bool grow = false;
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int x = 0; x < 4; ++x) s[nt][x] = (s[nt][x] + s2[nt][x]) * p.scale_log2;
      if (part_tile) {
        if (!((valid >> r0) & 1u)) s[nt][0] = s[nt][1] = -INFINITY;
        if (!((valid >> (r0 + 8)) & 1u)) s[nt][2] = s[nt][3] = -INFINITY;
      }
      if (p.scores != nullptr) {
        const uint32_t u = cc.t * kDecodeTile + warp * 16 + r0;
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (8 * nt + c0 + (x & 1) < heads && u + 8 * (x >> 1) < cc.s.n)
            score[(8 * nt + (x & 1)) * p.scores_ld + u + 8 * (x >> 1)] = s[nt][x];
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float v = fmaxf(s[nt][j], s[nt][2 + j]);
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        mx[nt][j] = v;
        // (from -inf any score grows, and -inf itself, NaN here, does not)
        grow |= v - m[nt][j] > DecodeScale<T>::kGrow;
      }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float n = fmaxf(m[nt][j], mx[nt][j]);
          const float a = m[nt][j] == -INFINITY ? 0.f : ex2_approx(m[nt][j] - n);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[i][nt][j] *= a;
            o[i][nt][2 + j] *= a;
          }
          l[nt][j] *= a;
          m[nt][j] = n;
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // a head that has seen nothing keeps reference 0: exp2(-inf) = 0; rounded
      // up, so that P stays within its range for scores of any size
      const float f0 = m[nt][0] == -INFINITY ? 0.f : __fadd_ru(m[nt][0], -DecodeScale<T>::kShift);
      const float f1 = m[nt][1] == -INFINITY ? 0.f : __fadd_ru(m[nt][1], -DecodeScale<T>::kShift);
      s[nt][0] = ex2_approx(s[nt][0] - f0);
      s[nt][1] = ex2_approx(s[nt][1] - f1);
      s[nt][2] = ex2_approx(s[nt][2] - f0);
      s[nt][3] = ex2_approx(s[nt][3] - f1);
      l[nt][0] += s[nt][0] + s[nt][2];
      l[nt][1] += s[nt][1] + s[nt][3];
      pb[nt][0] = movm_t(pack2<T>(s[nt][0], s[nt][1]));
      pb[nt][1] = movm_t(pack2<T>(s[nt][2], s[nt][3]));
    }
    {
      const uint32_t key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
      const uint32_t a = vb + key * (D * 2);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t r[4];
        ldsm_x4_t(r, a + (((2 * i + half) ^ (key & 7)) << 4));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_16816<T>(o[i][nt], r, pb[nt][0], pb[nt][1]);
      }
    }
    if (++stage == C::STAGES) stage = 0;

    const bool pair_end = cc.t + 1 == cc.tiles;
    if (pair_end || it + 1 == total) {
      // join the four warps: reference maximum, then the accumulators in order
      float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
      float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = l[nt][j];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (r0 == 0) ml[warp * C::ROWS + 8 * nt + c0 + j] = make_float2(m[nt][j], v);
        }
      __syncthreads();
      float f[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float M = -INFINITY;
          for (int w = 0; w < kDecodeWarps; ++w)
            M = fmaxf(M, ml[w * C::ROWS + 8 * nt + c0 + j].x);
          f[nt][j] = m[nt][j] == -INFINITY ? 0.f : ex2_approx(m[nt][j] - M);
        }
      // the first BUFS warps store, the others add to their buffer in turn
#pragma unroll 1
      for (uint32_t round = 0; round < kDecodeWarps / C::BUFS; ++round) {
        if (warp / C::BUFS == round) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t row = 8 * nt + c0 + (x & 1);
                if (row >= heads) continue;
                float* d = red + (warp % C::BUFS * C::ROWS + row) * C::RED_LD + 16 * i + r0 + 8 * (x >> 1);
                const float v = o[i][nt][x] * f[nt][x & 1];
                *d = round == 0 ? v : *d + v;
              }
        }
        __syncthreads();
      }
      const bool whole = seg_t0 == 0 && pair_end;
      const long long seg = static_cast<long long>(cc.b) * per + cc.pair;
      const uint32_t ps = blockIdx.x * 2 + (first_seg ? 0 : 1);
      constexpr uint32_t kLanes = D / 4;  // threads of a row, four columns each
      const uint32_t col = tid % kLanes * 4;
      for (uint32_t row = tid / kLanes; row < heads; row += kDecodeThreads / kLanes) {
        float4 v = *reinterpret_cast<const float4*>(red + row * C::RED_LD + col);
        if constexpr (C::BUFS == 2) {
          const float4 y =
              *reinterpret_cast<const float4*>(red + (C::ROWS + row) * C::RED_LD + col);
          v = make_float4(v.x + y.x, v.y + y.y, v.z + y.z, v.w + y.w);
        }
        float M = -INFINITY, L = 0.f;
        for (int w = 0; w < kDecodeWarps; ++w) M = fmaxf(M, ml[w * C::ROWS + row].x);
        for (int w = 0; w < kDecodeWarps; ++w) {
          const float2 x = ml[w * C::ROWS + row];
          L += x.x == -INFINITY ? 0.f : x.y * ex2_approx(x.x - M);
        }
        if (!whole) {
          if (col == 0) p.part_ml[ps * 16LL + row] = make_float2(M, L);
          *reinterpret_cast<float4*>(p.part_o + (ps * 16LL + row) * D + col) = v;
          continue;
        }
        if (p.scores != nullptr && col == 0)
          p.seg_ml[seg * 16 + row] = make_float2(M, L * DecodeScale<T>::kUnit);
        const float inv = L > 0.f ? 1.f / L : 0.f;
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + cc.b * p.o_b + (head0 + row) * p.o_h +
                                  col) =
            make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
      }
      if (!whole) {
        __threadfence();  // this part is visible to everyone before it is counted
        __syncthreads();
        if (tid == 0) {
          const uint32_t s0 = cc.base + cc.pair * cc.tiles;
          const uint32_t lo = run_of(W, G, s0), hi = run_of(W, G, s0 + cc.tiles - 1);
          const bool last = atomicAdd(p.count + lo, 1u) == hi - lo;
          if (last) p.count[lo] = 0;
          join_sh[0] = last ? 1u : 0u;
          join_sh[1] = lo;
          join_sh[2] = hi;
          join_sh[3] = run_start(W, G, lo) < s0 ? 1u : 0u;  // lo's second part
        }
      }
      if (!whole) {
        __syncthreads();
        if (join_sh[0]) {
          __threadfence();
          decode_join<T, D>(p, join_sh[1], join_sh[2], join_sh[3], heads, seg,
                            static_cast<T*>(p.out) + cc.b * p.o_b + head0 * p.o_h);
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

constexpr int kWeightThreads = 256;
// Slots per block, four per thread.  Eight per thread: the same for 64 sequences
// (266 us with the attention), 92 us instead of 86 for 16.
constexpr int kWeightSlots = 4 * kWeightThreads;

// Grid (slot blocks, h_kv, B): acc_out = acc + the weight each slot received,
// from the saved scores and the joined (m, l).
__global__ void __launch_bounds__(kWeightThreads) attn_decode_weights_kernel(const DecodeParams p) {
  __shared__ float2 ml_sh[256];
  const uint32_t b = blockIdx.z, kvh = blockIdx.y, tid = threadIdx.x;
  bool bad = false;
  const DecodeSeq sq = decode_seq(p, b, bad);
  if (blockIdx.x * kWeightSlots >= sq.len) return;
  // (m, 1 / l) of the pair's heads
  for (uint32_t r = tid; r < p.g; r += kWeightThreads) {
    const uint32_t ck = r / p.rows, row = r - ck * p.rows;
    const long long seg = (static_cast<long long>(b) * p.c.hkv + kvh) * p.chunks + ck;
    const float2 v = p.seg_ml[seg * 16 + row];
    // (l = 0: no slot was visible; l = NaN makes every weight NaN)
    ml_sh[r] = make_float2(v.x == -INFINITY ? 0.f : v.x, v.y == 0.f ? 0.f : 1.f / v.y);
  }
  __syncthreads();
  const long long a0 = (static_cast<long long>(b) * p.c.hkv + kvh) * p.c.cap;
  const float* sc = p.scores + (static_cast<long long>(b) * p.h + kvh * p.g) * p.scores_ld;
  const uint32_t first = blockIdx.x * kWeightSlots + tid;
  // (the loads of a thread's slots are independent)
  float w[4] = {}, old[4];
  const float* at[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t s = first + x * kWeightThreads;
    const bool seen = s < sq.len && (s >= sq.lo || s < sq.ns);
    at[x] = seen ? sc + (s < sq.ns ? s : sq.ns + (s - sq.lo)) : nullptr;
    old[x] = s < sq.len ? p.acc[a0 + s] : 0.f;
  }
  for (uint32_t r = 0; r < p.g; ++r) {
    const float2 ml = ml_sh[r];
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (at[x] != nullptr) w[x] += ex2_approx(at[x][r * p.scores_ld] - ml.x) * ml.y;
  }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const uint32_t s = first + x * kWeightThreads;
    if (s < sq.len) p.acc_out[a0 + s] = old[x] + w[x];
  }
}

}  // namespace bpt

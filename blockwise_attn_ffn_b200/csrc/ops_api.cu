// Host side of the attention operators that stand beside the layer calls: the
// paged key-value cache (append, one-token attention, eviction) and attention
// with a sliding window (forward, backward).  Argument checks, workspace
// layouts and launches; nothing is allocated and nothing synchronises.
//
// Workspaces: the first kOpsHeader bytes hold the error word and counters,
// zeroed by the caller once (every call leaves the counters at zero,
// bpt_read_device_error clears the error word), so a call launches nothing but
// its own kernels.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <mutex>

#include "bpt.h"
#include "ops_internal.h"

// The shared device helpers define functions in namespace bpt; in this unit
// the namespace gets its own name, so that both units link into one library.
#define bpt bpt_ops
#include "attn_decode.cuh"
#include "attn_window_bwd_tc.cuh"
#include "attn_window_tc.cuh"
#include "cache.cuh"
#include "common.cuh"

namespace {

using bpt_host::kOpsHeader;
constexpr size_t kCountOffset = 256;  // decode: counters of split pairs, one per block
static_assert(bpt::kErrIndex == BPT_ERR_INDEX, "status code");

size_t align_to(size_t v, size_t a) { return (v + a - 1) / a * a; }
bool unaligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

struct Range {
  uintptr_t a, b;
  Range(const void* p, size_t n)
      : a(reinterpret_cast<uintptr_t>(p)), b(reinterpret_cast<uintptr_t>(p) + (p ? n : 0)) {}
  bool meets(const Range& o) const { return a < o.b && o.a < b; }
};
bool any_meets(const Range& r, std::initializer_list<Range> others) {
  for (const Range& o : others)
    if (r.meets(o)) return true;
  return false;
}

// Extent in bytes of a strided 16-bit array (strides in elements, >= 0).
size_t extent(std::initializer_list<std::pair<int64_t, int64_t>> dims, int64_t last) {
  int64_t e = last;
  for (const auto& d : dims) e += (d.first - 1) * d.second;
  return size_t(e) * 2;
}

// Streaming multiprocessors of the current device (an sm_100 GPU).
struct OpsDevice {
  bool init = false, ok = false;
  int sms = 0;
};
std::mutex g_ops_mu;
OpsDevice g_ops_dev[64];

template <typename K>
bool smem_fails(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
         cudaSuccess;
}

bpt_status ops_device(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return BPT_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_ops_mu);
  OpsDevice& d = g_ops_dev[dev];
  if (!d.init) {
    int major = 0, minor = 0, n = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return BPT_ERR_CUDA;
    d.ok = major == 10 && minor == 0;
    d.sms = n;
    using bf = __nv_bfloat16;
    if (d.ok &&
        (smem_fails(bpt::cache_evict_select_kernel<false>, bpt::kEvictSmem) ||
         smem_fails(bpt::cache_evict_select_kernel<true>, bpt::kEvictSmem) ||
         smem_fails(bpt::attn_decode_split_kernel<bf, 64, 1>, bpt::DecodeCfg<64, 1>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<bf, 64, 2>, bpt::DecodeCfg<64, 2>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<bf, 128, 1>, bpt::DecodeCfg<128, 1>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<bf, 128, 2>, bpt::DecodeCfg<128, 2>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<__half, 64, 1>, bpt::DecodeCfg<64, 1>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<__half, 64, 2>, bpt::DecodeCfg<64, 2>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<__half, 128, 1>, bpt::DecodeCfg<128, 1>::SMEM) ||
         smem_fails(bpt::attn_decode_split_kernel<__half, 128, 2>, bpt::DecodeCfg<128, 2>::SMEM) ||
         smem_fails(bpt::attn_window_tc_kernel<bf, 64>, bpt::WindowCfg<64>::SMEM) ||
         smem_fails(bpt::attn_window_tc_kernel<bf, 128>, bpt::WindowCfg<128>::SMEM) ||
         smem_fails(bpt::attn_window_tc_kernel<__half, 64>, bpt::WindowCfg<64>::SMEM) ||
         smem_fails(bpt::attn_window_tc_kernel<__half, 128>, bpt::WindowCfg<128>::SMEM) ||
         smem_fails(bpt::window_dkv_tc_kernel<bf, 64>, bpt::WindowBwdCfg<64>::KV_SMEM) ||
         smem_fails(bpt::window_dkv_tc_kernel<bf, 128>, bpt::WindowBwdCfg<128>::KV_SMEM) ||
         smem_fails(bpt::window_dkv_tc_kernel<__half, 64>, bpt::WindowBwdCfg<64>::KV_SMEM) ||
         smem_fails(bpt::window_dkv_tc_kernel<__half, 128>, bpt::WindowBwdCfg<128>::KV_SMEM) ||
         smem_fails(bpt::window_dq_tc_kernel<bf, 64>, bpt::WindowBwdCfg<64>::Q_SMEM) ||
         smem_fails(bpt::window_dq_tc_kernel<bf, 128>, bpt::WindowBwdCfg<128>::Q_SMEM) ||
         smem_fails(bpt::window_dq_tc_kernel<__half, 64>, bpt::WindowBwdCfg<64>::Q_SMEM) ||
         smem_fails(bpt::window_dq_tc_kernel<__half, 128>, bpt::WindowBwdCfg<128>::Q_SMEM)))
      return BPT_ERR_CUDA;
    d.init = true;
  }
  if (!d.ok) return BPT_ERR_UNSUPPORTED;
  *sms = d.sms;
  return BPT_OK;
}

// ------------------------------------------------------------------- cache --
bpt_status check_cache(const bpt_cache* c) {
  if (c == nullptr) return BPT_ERR_INVALID_ARG;
  if (c->reserved != 0) return BPT_ERR_INVALID_ARG;
  if (c->dtype != BPT_BF16 && c->dtype != BPT_F16) return BPT_ERR_INVALID_ARG;
  if (c->batch < 0 || c->pages <= 0 || c->kv_heads <= 0 || c->page_size <= 0 || c->max_pages <= 0)
    return BPT_ERR_INVALID_ARG;
  if (c->d_k != 64 && c->d_k != 128) return BPT_ERR_UNSUPPORTED;
  if (c->batch > 65535 || c->kv_heads > 65535) return BPT_ERR_UNSUPPORTED;
  const int64_t lim = int64_t(1) << 31;
  // rows and slots are 32-bit; byte offsets 64-bit
  if (c->pages >= lim || c->page_size >= lim || c->max_pages >= lim) return BPT_ERR_UNSUPPORTED;
  if (c->max_pages * c->page_size >= lim || c->pages * c->page_size >= lim ||
      c->pages * c->page_size * c->kv_heads >= lim)
    return BPT_ERR_UNSUPPORTED;
  return BPT_OK;
}
size_t cache_bytes(const bpt_cache* c) {
  return size_t(c->pages) * size_t(c->kv_heads * c->page_size) * size_t(c->d_k) * 2;
}
bpt_status check_cache_pointers(const bpt_cache* c) {
  for (const void* p : {c->k, c->v})
    if (p == nullptr || unaligned(p, 16)) return BPT_ERR_INVALID_ARG;
  for (const int32_t* p : {c->page_table, c->lens})
    if (p == nullptr || unaligned(p, 4)) return BPT_ERR_INVALID_ARG;
  const size_t n = cache_bytes(c);
  if (Range(c->k, n).meets(Range(c->v, n))) return BPT_ERR_INVALID_ARG;
  return BPT_OK;
}
size_t slots_bytes(const bpt_cache* c) {  // [batch][kv_heads][max_pages * page_size] words
  return size_t(c->batch) * size_t(c->kv_heads) * size_t(c->max_pages * c->page_size) * 4;
}
bpt::CacheView view_of(const bpt_cache* c, uint32_t* err) {
  bpt::CacheView v{};
  v.k = static_cast<uint4*>(c->k);
  v.v = static_cast<uint4*>(c->v);
  v.table = c->page_table;
  v.lens = c->lens;
  v.pages = uint32_t(c->pages);
  v.hkv = uint32_t(c->kv_heads);
  v.ps = uint32_t(c->page_size);
  v.max_pages = uint32_t(c->max_pages);
  v.cap = uint32_t(c->max_pages * c->page_size);
  // ps_mul = ceil(2^(31 + l) / ps) with 2^(l-1) < ps <= 2^l: the product's
  // error stays below 2^-l for 31-bit slots, so the quotient is exact
  if (v.ps > 1) {
    int l = 0;
    while ((uint64_t(1) << l) < v.ps) ++l;
    v.ps_mul = uint32_t(((uint64_t(1) << (31 + l)) + v.ps - 1) / v.ps);
    v.ps_shift = uint32_t(l - 1);
  }
  v.err = err;
  return v;
}
uint32_t clamp_u31(int64_t v) { return uint32_t(std::min<int64_t>(v, 0x7FFFFFFF)); }

// Workspace of the cache's own operators: header, eviction lists and counts.
struct CacheLayout {
  size_t off_lists, off_count, total;
};
CacheLayout cache_layout(const bpt_cache* c) {
  CacheLayout l{};
  l.off_lists = kOpsHeader;
  l.off_count = align_to(l.off_lists + slots_bytes(c), 256);
  l.total = align_to(l.off_count + size_t(c->batch * c->kv_heads) * 4, 256);
  return l;
}

struct DecodeLayout {
  size_t off_o, off_ml, off_seg, off_scores, total;
  int64_t chunks, rows;
};
// Row length of the saved scores (dense over the visible slots), even.
int64_t scores_ld(const bpt_cache* c) { return (c->max_pages * c->page_size + 1) / 2 * 2; }
bpt_status decode_layout(const bpt_cache* c, int64_t heads, int with_acc, DecodeLayout* l) {
  if (heads <= 0 || heads % c->kv_heads != 0) return BPT_ERR_INVALID_ARG;
  const int64_t g = heads / c->kv_heads;
  if (g > 256) return BPT_ERR_UNSUPPORTED;
  // query heads that go through one pass over the keys: 8 or 16
  l->rows = g <= 8 ? 8 : 16;
  l->chunks = (g + l->rows - 1) / l->rows;
  const int64_t tiles = (c->max_pages * c->page_size + bpt::kDecodeTile - 1) / bpt::kDecodeTile;
  const int64_t pairs = c->batch * c->kv_heads * l->chunks;
  if (pairs >= (int64_t(1) << 31) || (pairs > 0 && tiles >= (int64_t(1) << 31) / pairs) ||
      c->batch * c->kv_heads >= (int64_t(1) << 31))
    return BPT_ERR_UNSUPPORTED;
  const size_t parts = size_t(2 * bpt::kDecodeMaxCtas * bpt::kDecodeMaxSms) * 16;
  static_assert(kCountOffset + bpt::kDecodeMaxCtas * bpt::kDecodeMaxSms * 4 <= kOpsHeader,
                "counters");
  l->off_o = kOpsHeader;
  l->off_ml = align_to(l->off_o + parts * size_t(c->d_k) * 4, 256);
  l->off_seg = align_to(l->off_ml + parts * 8, 256);
  l->off_scores = align_to(l->off_seg + size_t(pairs) * 16 * 8, 256);
  l->total = l->off_scores;
  if (with_acc)
    l->total = align_to(l->off_scores + size_t(c->batch * heads) *
                                            size_t(scores_ld(c)) * 4, 256);
  return BPT_OK;
}

template <typename T, int D>
cudaError_t launch_decode(const bpt::DecodeParams& p, unsigned slot_blocks, cudaStream_t s) {
  if (p.rows == 8)
    bpt::attn_decode_split_kernel<T, D, 1>
        <<<p.ctas, bpt::kDecodeThreads, bpt::DecodeCfg<D, 1>::SMEM, s>>>(p);
  else
    bpt::attn_decode_split_kernel<T, D, 2>
        <<<p.ctas, bpt::kDecodeThreads, bpt::DecodeCfg<D, 2>::SMEM, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (slot_blocks == 0) return cudaSuccess;
  bpt::attn_decode_weights_kernel<<<dim3(slot_blocks, p.c.hkv, p.B), bpt::kWeightThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ window --
PFN_cuTensorMapEncodeTiled_v12000 g_ops_encode = nullptr;

bpt_status ops_encoder() {
  std::lock_guard<std::mutex> lk(g_ops_mu);
  if (g_ops_encode) return BPT_OK;
  void* fn = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) !=
          cudaSuccess ||
      q != cudaDriverEntryPointSuccess || fn == nullptr)
    return BPT_ERR_CUDA;
  g_ops_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  return BPT_OK;
}

// Strided rows [batch, n, heads, d_k] viewed as [batch][heads][d_k/64][n][64]:
// a box is `rows` rows of one head, 64-column chunks one after another in shared
// memory (128-byte swizzle).  Rows outside 0 .. n-1 read as zeros.
bool map_rows(CUtensorMap* m, const bpt_rows& r, int64_t batch, int64_t n, int64_t heads,
              int64_t dk, int rows = 128) {
  const int64_t any = 128;  // the stride of a dimension of one entry is not used
  cuuint64_t dims[5] = {64, cuuint64_t(n), cuuint64_t(dk / 64), cuuint64_t(heads),
                        cuuint64_t(batch)};
  cuuint64_t st[4] = {cuuint64_t(n > 1 ? r.stride_n * 2 : any), 128,
                      cuuint64_t(heads > 1 ? r.stride_h * 2 : any),
                      cuuint64_t(batch > 1 ? r.stride_b * 2 : any)};
  cuuint32_t box[5] = {64, cuuint32_t(rows), cuuint32_t(dk / 64), 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return g_ops_encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, r.data, dims, st, box, es,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bpt_status check_window(const bpt_window* w) {
  if (w == nullptr) return BPT_ERR_INVALID_ARG;
  if (w->dtype != BPT_BF16 && w->dtype != BPT_F16) return BPT_ERR_INVALID_ARG;
  if (w->reserved != 0 || w->batch < 0 || w->n_q < 0 || w->n_kv < 0 || w->heads <= 0 ||
      w->kv_heads <= 0 || w->heads % w->kv_heads != 0 || w->n_q > w->n_kv || w->window <= 0 ||
      w->sinks < 0)
    return BPT_ERR_INVALID_ARG;
  if (w->d_k != 64 && w->d_k != 128) return BPT_ERR_UNSUPPORTED;
  const int64_t lim = int64_t(1) << 30;  // (key + window stays below 2^31)
  if (w->n_kv > lim / 2 || w->heads > lim || w->batch > lim) return BPT_ERR_UNSUPPORTED;
  // CTAs of a launch (a 31-bit grid), one per two query tiles at most
  const int64_t tiles = (w->n_kv + 127) / 128, hb = w->heads * std::max<int64_t>(1, w->batch);
  if (hb >= lim || tiles >= (int64_t(1) << 31) / hb) return BPT_ERR_UNSUPPORTED;
  return BPT_OK;
}

// A strided 16-bit tensor the kernels may read: 16-byte rows, positive
// strides (a broadcast dimension has to be materialised).
bool rows_ok(const bpt_rows& r, int64_t batch, int64_t n, int64_t heads) {
  if (r.data == nullptr || unaligned(r.data, 16)) return false;
  const std::pair<int64_t, int64_t> dims[3] = {
      {batch, r.stride_b}, {n, r.stride_n}, {heads, r.stride_h}};
  for (const auto& d : dims)
    if (d.first > 1 && (d.second <= 0 || d.second % 8 != 0 || d.second >= (int64_t(1) << 38)))
      return false;
  return true;
}
Range rows_range(const bpt_rows& r, int64_t batch, int64_t n, int64_t heads, int64_t dk) {
  return Range(r.data, extent({{batch, r.stride_b}, {n, r.stride_n}, {heads, r.stride_h}}, dk));
}
// Written rows must not meet one another: ordered by stride, each dimension
// steps past the extent of the smaller ones.
bool rows_apart(const bpt_rows& r, int64_t batch, int64_t n, int64_t heads, int64_t dk) {
  std::pair<int64_t, int64_t> d[3] = {{r.stride_b, batch}, {r.stride_n, n}, {r.stride_h, heads}};
  std::sort(d, d + 3);
  int64_t ext = dk;
  for (const auto& x : d)
    if (x.second > 1) {
      if (x.first < ext) return false;
      ext += x.first * (x.second - 1);
    }
  return true;
}

// Whether rows of a and b meet.  Rows at elements x and y share one if
// |delta + sum of the indexes times their strides| < d_k, indexes of a counting
// down and of b up; dimensions that both have with one stride count as one, from
// 1 - n_a to n_b - 1.  From the largest stride down, only the indexes that the
// smaller ones can make up for are followed: a handful for tensors whose own rows
// are apart.  More than kMeetSteps count as a meeting.
constexpr int kMeetSteps = 4096;
struct MeetDim {
  int64_t stride, lo, hi;
};
bool meet_from(const MeetDim* d, int n, int64_t at, int64_t dk, int* steps) {
  if (++*steps > kMeetSteps) return true;
  if (n == 0) return at > -dk && at < dk;
  int64_t lo = at, hi = at;  // what the smaller dimensions can reach
  for (int i = 1; i < n; ++i) {
    lo += d[i].lo * d[i].stride;
    hi += d[i].hi * d[i].stride;
  }
  // x stride + [lo, hi] meets (-dk, dk)
  auto floor_div = [](int64_t a, int64_t b) { return a >= 0 ? a / b : -((-a + b - 1) / b); };
  const int64_t first = std::max(d[0].lo, -floor_div(dk - 1 + hi, d[0].stride));
  const int64_t last = std::min(d[0].hi, floor_div(dk - 1 - lo, d[0].stride));
  for (int64_t x = first; x <= last; ++x)
    if (meet_from(d + 1, n - 1, at + x * d[0].stride, dk, steps)) return true;
  return false;
}
bool rows_meet(const bpt_rows& a, const int64_t (&na)[3], const bpt_rows& b, const int64_t (&nb)[3],
               int64_t dk) {
  const int64_t sa[3] = {a.stride_b, a.stride_n, a.stride_h};
  const int64_t sb[3] = {b.stride_b, b.stride_n, b.stride_h};
  if (!Range(a.data, extent({{na[0], sa[0]}, {na[1], sa[1]}, {na[2], sa[2]}}, dk))
           .meets(Range(b.data, extent({{nb[0], sb[0]}, {nb[1], sb[1]}, {nb[2], sb[2]}}, dk))))
    return false;
  MeetDim d[6];
  int n = 0;
  for (int i = 0; i < 3; ++i)
    if (na[i] > 1) d[n++] = {sa[i], 1 - na[i], 0};
  for (int i = 0; i < 3; ++i) {
    if (nb[i] <= 1) continue;
    int k = 0;
    while (k < n && !(d[k].stride == sb[i] && d[k].hi == 0)) ++k;
    if (k < n)
      d[k].hi = nb[i] - 1;
    else
      d[n++] = {sb[i], 0, nb[i] - 1};
  }
  std::sort(d, d + n, [](const MeetDim& x, const MeetDim& y) { return x.stride > y.stride; });
  const auto pa = reinterpret_cast<uintptr_t>(a.data), pb = reinterpret_cast<uintptr_t>(b.data);
  const int64_t delta = pb >= pa ? int64_t((pb - pa) / 2) : -int64_t((pa - pb) / 2);
  int steps = 0;
  return meet_from(d, n, delta, dk, &steps);
}

template <typename T, int D>
cudaError_t launch_window(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                          const bpt::WindowParams& p, int64_t batch, cudaStream_t s) {
  using C = bpt::WindowCfg<D>;
  bpt::attn_window_tc_kernel<T, D>
      <<<unsigned(batch * p.hkv * p.npairs), C::THREADS, C::SMEM, s>>>(q, k, v, p);
  return cudaGetLastError();
}

// Parts of the dK/dV work and workspace of the backward.
struct WindowBwdPlan {
  int part_len;
  int64_t parts, cut_parts, cut_blocks;  // per (sequence, kv head)
  size_t off_terms, off_range, range_bytes, off_part, total;
};
constexpr int kPlanSms = 148;  // the GPU the work is cut for

WindowBwdPlan window_bwd_plan(const bpt_window* w) {
  WindowBwdPlan p{};
  const int nq = int(w->n_q), nkv = int(w->n_kv), g = int(w->heads / w->kv_heads);
  const int win = int(std::min<int64_t>(w->window, nkv)), snk = int(std::min<int64_t>(w->sinks, nkv));
  const int nblk = (nkv + 127) / 128;
  const int qt = w->d_k == 128 ? bpt::kWinTile<128> : bpt::kWinTile<64>;
  const int blocks = w->d_k == 128 ? bpt::kWinBwdBlocks<128> : bpt::kWinBwdBlocks<64>;
  int64_t items = 0;
  for (int b = 0; b < nblk; ++b)
    items += int64_t(g) * bpt::window_queries(nq, nkv, win, snk, b * 128, nq).tiles(qt);
  items *= w->batch * w->kv_heads;
  // half of one resident block's share, at least 8 items (a part costs 128 KB of traffic
  // and a join, about what an item costs)
  p.part_len = int(std::min<int64_t>(0x7FFFFFFF, std::max<int64_t>(
      8, (items + 2 * blocks * kPlanSms - 1) / (2 * blocks * kPlanSms))));
  for (int b = 0; b < nblk; ++b) {
    const int n = bpt::window_parts(nq, nkv, win, snk, g, b * 128, qt, p.part_len);
    p.parts += n;
    if (n > 1) {
      p.cut_parts += n;
      p.cut_blocks += 1;
    }
  }
  p.off_terms = kOpsHeader;
  p.off_range = align_to(p.off_terms + size_t(w->batch * w->heads) * size_t(w->n_q) * 8, 256);
  p.range_bytes = w->dtype == BPT_F16 ? size_t(w->batch * w->kv_heads) * 8 : 0;
  p.off_part = align_to(p.off_range + p.range_bytes, 256);
  p.total = align_to(p.off_part + size_t(w->batch * w->kv_heads) * size_t(p.cut_parts) *
                                      size_t(2 * 128 * 4) * size_t(w->d_k), 256);
  return p;
}

bpt_status check_window_bwd(const bpt_window* w) {
  const bpt_status st = check_window(w);
  if (st != BPT_OK) return st;
  if (w->batch > 65535 || w->heads > 65535 || w->batch * w->kv_heads > 65535 ||
      w->n_q >= (int64_t(1) << 34) / std::max<int64_t>(1, w->batch * w->heads))
    return BPT_ERR_UNSUPPORTED;
  return BPT_OK;
}

// A launch that may start before the one in front of it has ended (the kernel
// waits where it has to).
template <typename K, typename... A>
cudaError_t launch_early(K kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int D>
cudaError_t launch_window_bwd(const CUtensorMap* stay, const CUtensorMap* stream,
                              bpt::WindowTermsParams tp, const bpt::WindowBwdParams& p,
                              const WindowBwdPlan& plan, int64_t batch, cudaStream_t s) {
  using C = bpt::WindowBwdCfg<D>;
  constexpr int64_t per = bpt::kTermBlockRows<D>;
  tp.row_blocks = uint32_t((int64_t(p.nq) * p.g + per - 1) / per);
  const int64_t value_blocks = tp.range != nullptr ? (int64_t(p.nkv) + per - 1) / per : 0;
  bpt::window_terms_kernel<T, D>
      <<<dim3(tp.row_blocks + unsigned(value_blocks), unsigned(p.hkv), unsigned(batch)), 256, 0, s>>>(
          tp);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // dK/dV start on their products while the last terms are written; dQ's blocks,
  // which need the terms alone, fill the SMs that the last dK/dV blocks leave
  e = launch_early(bpt::window_dkv_tc_kernel<T, D>,
                   dim3(unsigned(plan.parts), unsigned(batch * p.hkv)), bpt::kWinBwdThreads<D>,
                   C::KV_SMEM, s, stream[0], stay[1], stay[2], stream[3], p);
  if (e != cudaSuccess) return e;
  e = launch_early(bpt::window_dq_tc_kernel<T, D>,
                   dim3(unsigned(p.nqb), unsigned(p.h), unsigned(batch)), bpt::kWinBwdThreads<D>,
                   C::Q_SMEM, s, stay[0], stream[1], stream[2], stay[3], p);
  if (e != cudaSuccess || plan.cut_blocks == 0) return e;
  return launch_early(bpt::window_join_kernel<T, D>,
                      dim3(unsigned(plan.cut_blocks), unsigned(batch * p.hkv), 8), 256, 0, s, p);
}

}  // namespace

namespace bpt_host {

bpt_status cache_append(const bpt_cache* cache, const void* k_new, const void* v_new,
                        int64_t tokens, const int64_t* strides, const int32_t* counts,
                        int32_t* new_lens, float* acc, int32_t* pos, const int32_t* seen,
                        void* workspace, size_t workspace_bytes, bpt_stream_t stream,
                        uint32_t* err, bool check_only) {
  if (err == nullptr) err = static_cast<uint32_t*>(workspace);
  bpt_status st = check_cache(cache);
  if (st != BPT_OK) return st;
  if (tokens < 0) return BPT_ERR_INVALID_ARG;
  if (cache->batch == 0) return BPT_OK;
  st = check_cache_pointers(cache);
  if (st != BPT_OK) return st;
  const int64_t B = cache->batch, h = cache->kv_heads, dk = cache->d_k;
  if (new_lens == nullptr || unaligned(new_lens, 4) || workspace == nullptr ||
      unaligned(workspace, 256) || unaligned(counts, 4) || unaligned(acc, 4) ||
      unaligned(pos, 4) || unaligned(seen, 4) || strides == nullptr)
    return BPT_ERR_INVALID_ARG;
  if (workspace_bytes < kOpsHeader) return BPT_ERR_WORKSPACE;
  if (tokens > 0) {
    for (const void* p : {k_new, v_new})
      if (p == nullptr || unaligned(p, 16)) return BPT_ERR_INVALID_ARG;
    const int64_t dims[3] = {B, tokens, h};  // (a dimension of one entry has no stride)
    for (int i = 0; i < 6; ++i)
      if (dims[i % 3] > 1 && (strides[i] < 0 || strides[i] % 8 != 0)) return BPT_ERR_INVALID_ARG;
    if (tokens >= (int64_t(1) << 31) / (h * dk / 8)) return BPT_ERR_UNSUPPORTED;
  }
  const Range rk(cache->k, cache_bytes(cache)), rv(cache->v, cache_bytes(cache)),
      rl(cache->lens, size_t(B) * 4), rn(new_lens, size_t(B) * 4),
      rt(cache->page_table, size_t(B * cache->max_pages) * 4), ra(acc, slots_bytes(cache)),
      rp(pos, slots_bytes(cache)), rc(counts, size_t(B) * 4), rs(seen, size_t(B) * 4),
      rw(workspace, kOpsHeader);
  const size_t kb = tokens > 0 ? extent({{B, strides[0]}, {tokens, strides[1]}, {h, strides[2]}}, dk) : 0;
  const size_t vb = tokens > 0 ? extent({{B, strides[3]}, {tokens, strides[4]}, {h, strides[5]}}, dk) : 0;
  const Range ik(k_new, kb), iv(v_new, vb);
  // every array that is written meets no other one
  if (any_meets(rk, {ik, iv, rl, rn, rt, ra, rp, rc, rs, rw}) ||
      any_meets(rv, {ik, iv, rl, rn, rt, ra, rp, rc, rs, rw}) ||
      any_meets(rn, {ik, iv, rl, rt, ra, rp, rc, rs, rw}) ||
      any_meets(ra, {ik, iv, rl, rt, rp, rc, rs, rw}) ||
      any_meets(rp, {ik, iv, rl, rt, rc, rs, rw}) || any_meets(rw, {ik, iv, rl, rt, rc, rs}))
    return BPT_ERR_INVALID_ARG;
  if (check_only) return BPT_OK;
  int sms = 0;
  st = ops_device(&sms);
  if (st != BPT_OK) return st;
  bpt::AppendParams p{};
  p.c = view_of(cache, err);
  p.k = static_cast<const uint4*>(k_new);
  p.v = static_cast<const uint4*>(v_new);
  p.k_b = strides[0] / 8;
  p.k_t = strides[1] / 8;
  p.k_h = strides[2] / 8;
  p.v_b = strides[3] / 8;
  p.v_t = strides[4] / 8;
  p.v_h = strides[5] / 8;
  p.counts = counts;
  p.new_lens = new_lens;
  p.acc = acc;
  p.pos = pos;
  p.seen = seen;
  p.T = uint32_t(tokens);
  p.row16 = uint32_t(dk / 8);
  const int64_t per_block = bpt::kAppendThreads * bpt::kAppendUnroll;
  const int64_t blocks = std::max<int64_t>(1, (tokens * h * (dk / 8) + per_block - 1) / per_block);
  bpt::cache_append_kernel<<<dim3(unsigned(blocks), unsigned(B)), bpt::kAppendThreads, 0,
                             reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ERR_CUDA;
}

bpt_status attn_decode(const bpt_cache* cache, const void* q, int64_t heads,
                       int64_t q_stride_b, int64_t q_stride_h, int64_t window, int64_t sinks,
                       const float* acc, float* acc_out, void* out, int64_t out_stride_b,
                       int64_t out_stride_h, void* workspace, size_t workspace_bytes,
                       bpt_stream_t stream, uint32_t* err, bool check_only) {
  if (err == nullptr) err = static_cast<uint32_t*>(workspace);
  bpt_status st = check_cache(cache);
  if (st != BPT_OK) return st;
  if (window < 0 || sinks < 0 || (acc == nullptr) != (acc_out == nullptr))
    return BPT_ERR_INVALID_ARG;
  DecodeLayout l;
  st = decode_layout(cache, heads, acc != nullptr, &l);
  if (st != BPT_OK) return st;
  if (cache->batch == 0) return BPT_OK;
  st = check_cache_pointers(cache);
  if (st != BPT_OK) return st;
  const int64_t B = cache->batch, dk = cache->d_k;
  for (const void* p : {q, static_cast<const void*>(out)})
    if (p == nullptr || unaligned(p, 16)) return BPT_ERR_INVALID_ARG;
  auto bad_stride = [](int64_t n, int64_t x) { return n > 1 && (x < 0 || x % 8 != 0); };
  if (bad_stride(B, q_stride_b) || bad_stride(heads, q_stride_h) || bad_stride(B, out_stride_b) ||
      bad_stride(heads, out_stride_h))
    return BPT_ERR_INVALID_ARG;
  // output rows must not meet one another
  if ((heads > 1 && out_stride_h < dk) || (B > 1 && out_stride_b < dk) ||
      (B > 1 && heads > 1 && out_stride_b < (heads - 1) * out_stride_h + dk &&
       out_stride_h < (B - 1) * out_stride_b + dk))
    return BPT_ERR_INVALID_ARG;
  if (workspace == nullptr || unaligned(workspace, 256) || unaligned(acc, 4) ||
      unaligned(acc_out, 4))
    return BPT_ERR_INVALID_ARG;
  if (workspace_bytes < l.total) return BPT_ERR_WORKSPACE;
  const Range rk(cache->k, cache_bytes(cache)), rv(cache->v, cache_bytes(cache)),
      rl(cache->lens, size_t(B) * 4), rt(cache->page_table, size_t(B * cache->max_pages) * 4),
      ra(acc, acc ? slots_bytes(cache) : 0), rao(acc_out, acc ? slots_bytes(cache) : 0),
      rq(q, extent({{B, q_stride_b}, {heads, q_stride_h}}, dk)),
      ro(out, extent({{B, out_stride_b}, {heads, out_stride_h}}, dk)), rw(workspace, l.total);
  // acc may be updated in place; nothing else that is written meets another array
  if ((acc_out != acc && rao.meets(ra)) || any_meets(rao, {rk, rv, rl, rt, rq, ro, rw}) ||
      any_meets(ro, {rk, rv, rl, rt, rq, ra, rw}) || any_meets(rw, {rk, rv, rl, rt, rq, ra}))
    return BPT_ERR_INVALID_ARG;
  if (check_only) return BPT_OK;
  int sms = 0;
  st = ops_device(&sms);
  if (st != BPT_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  bpt::DecodeParams p{};
  p.c = view_of(cache, err);
  p.q = q;
  p.q_b = q_stride_b;
  p.q_h = q_stride_h;
  p.out = out;
  p.o_b = out_stride_b;
  p.o_h = out_stride_h;
  p.B = uint32_t(B);
  p.h = uint32_t(heads);
  p.g = uint32_t(heads / cache->kv_heads);
  p.chunks = uint32_t(l.chunks);
  p.rows = uint32_t(l.rows);
  p.scores_ld = scores_ld(cache);
  p.window = clamp_u31(window);
  p.sinks = clamp_u31(sinks);
  p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(dk)));
  p.count = reinterpret_cast<uint32_t*>(ws + kCountOffset);
  p.part_o = reinterpret_cast<float*>(ws + l.off_o);
  p.part_ml = reinterpret_cast<float2*>(ws + l.off_ml);
  p.seg_ml = reinterpret_cast<float2*>(ws + l.off_seg);
  const int per_sm = l.rows == 16 ? bpt::DecodeShape<128, 2>::CTAS
                     : dk == 128  ? bpt::DecodeShape<128, 1>::CTAS
                                  : bpt::DecodeShape<64, 1>::CTAS;
  p.ctas = uint32_t(per_sm * std::min(sms, bpt::kDecodeMaxSms));
  p.scores = acc != nullptr ? reinterpret_cast<float*>(ws + l.off_scores) : nullptr;
  p.acc = acc;
  p.acc_out = acc_out;
  const unsigned slot_blocks =
      acc != nullptr ? unsigned((p.c.cap + bpt::kWeightSlots - 1) / bpt::kWeightSlots) : 0u;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->dtype == BPT_BF16)
    e = dk == 128 ? launch_decode<__nv_bfloat16, 128>(p, slot_blocks, s)
                  : launch_decode<__nv_bfloat16, 64>(p, slot_blocks, s);
  else
    e = dk == 128 ? launch_decode<__half, 128>(p, slot_blocks, s)
                  : launch_decode<__half, 64>(p, slot_blocks, s);
  return e == cudaSuccess ? BPT_OK : BPT_ERR_CUDA;
}

bpt_status window_forward(const bpt_window* w, const bpt_rows* q, const bpt_rows* k,
                          const bpt_rows* v, const int32_t* lens, const bpt_rows* out,
                          float* stats, void* workspace, size_t workspace_bytes,
                          bpt_stream_t stream, uint32_t* err) {
  if (err == nullptr) err = static_cast<uint32_t*>(workspace);
  bpt_status st = check_window(w);
  if (st != BPT_OK) return st;
  if (q == nullptr || k == nullptr || v == nullptr || out == nullptr) return BPT_ERR_INVALID_ARG;
  if (w->batch == 0 || w->n_q == 0) return BPT_OK;
  const int64_t B = w->batch, nq = w->n_q, nkv = w->n_kv, h = w->heads, hkv = w->kv_heads,
                dk = w->d_k;
  if (!rows_ok(*q, B, nq, h) || !rows_ok(*k, B, nkv, hkv) || !rows_ok(*v, B, nkv, hkv) ||
      !rows_ok(*out, B, nq, h) || !rows_apart(*out, B, nq, h, dk) || unaligned(lens, 4) ||
      unaligned(stats, 8) || workspace == nullptr || unaligned(workspace, 256))
    return BPT_ERR_INVALID_ARG;
  if (workspace_bytes < kOpsHeader) return BPT_ERR_WORKSPACE;
  const Range rq = rows_range(*q, B, nq, h, dk), rk = rows_range(*k, B, nkv, hkv, dk),
              rv = rows_range(*v, B, nkv, hkv, dk), rl(lens, size_t(B) * 4),
              rs(stats, size_t(B * h) * size_t(nq) * 8), rw(workspace, kOpsHeader);
  const Range ro = rows_range(*out, B, nq, h, dk);
  if (any_meets(ro, {rq, rk, rv, rl, rs, rw}) || any_meets(rs, {rq, rk, rv, rl, rw}) ||
      any_meets(rw, {rq, rk, rv, rl}))
    return BPT_ERR_INVALID_ARG;
  int sms = 0;
  st = ops_device(&sms);
  if (st != BPT_OK) return st;
  st = ops_encoder();
  if (st != BPT_OK) return st;
  CUtensorMap mq, mk, mv;
  if (!map_rows(&mq, *q, B, nq, h, dk) || !map_rows(&mk, *k, B, nkv, hkv, dk) ||
      !map_rows(&mv, *v, B, nkv, hkv, dk))
    return BPT_ERR_CUDA;
  bpt::WindowParams p{};
  p.nq = int(nq);
  p.nkv = int(nkv);
  p.h = int(h);
  p.hkv = int(hkv);
  p.g = int(h / hkv);
  p.units = int((nq + 127) / 128) * p.g;
  p.npairs = (p.units + 1) / 2;
  p.window = int(std::min<int64_t>(w->window, nkv));
  p.sinks = int(std::min<int64_t>(w->sinks, nkv));
  p.lens = lens;
  p.q = q->data;
  p.k = k->data;
  p.v = v->data;
  p.q_b = q->stride_b; p.q_n = q->stride_n; p.q_h = q->stride_h;
  p.k_b = k->stride_b; p.k_n = k->stride_n; p.k_h = k->stride_h;
  p.v_b = v->stride_b; p.v_n = v->stride_n; p.v_h = v->stride_h;
  p.o = out->data;
  p.o_b = out->stride_b; p.o_n = out->stride_n; p.o_h = out->stride_h;
  p.scale_log2 = float(1.4426950408889634 / std::sqrt(double(dk)));
  p.stats = reinterpret_cast<float2*>(stats);
  p.err = err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (w->dtype == BPT_BF16)
    e = dk == 128 ? launch_window<__nv_bfloat16, 128>(mq, mk, mv, p, B, s)
                  : launch_window<__nv_bfloat16, 64>(mq, mk, mv, p, B, s);
  else
    e = dk == 128 ? launch_window<__half, 128>(mq, mk, mv, p, B, s)
                  : launch_window<__half, 64>(mq, mk, mv, p, B, s);
  return e == cudaSuccess ? BPT_OK : BPT_ERR_CUDA;
}

bpt_status window_backward(const bpt_window* w, const bpt_rows* q, const bpt_rows* k,
                           const bpt_rows* v, const bpt_rows* o, const float* stats,
                           const bpt_rows* d_o, const int32_t* lens, const bpt_rows* dq,
                           const bpt_rows* dk, const bpt_rows* dv, void* workspace,
                           size_t workspace_bytes, bpt_stream_t stream, uint32_t* err) {
  if (err == nullptr) err = static_cast<uint32_t*>(workspace);
  bpt_status st = check_window_bwd(w);
  if (st != BPT_OK) return st;
  for (const bpt_rows* r : {q, k, v, o, d_o, dq, dk, dv})
    if (r == nullptr) return BPT_ERR_INVALID_ARG;
  const int64_t B = w->batch, nq = w->n_q, nkv = w->n_kv, h = w->heads, hkv = w->kv_heads,
                c = w->d_k;
  // (with keys but without queries the gradients of the keys are zeros: the
  // call would be of no use and is refused)
  if (B == 0 || nkv == 0) return BPT_OK;
  if (nq == 0) return BPT_ERR_INVALID_ARG;
  if (!rows_ok(*q, B, nq, h) || !rows_ok(*k, B, nkv, hkv) || !rows_ok(*v, B, nkv, hkv) ||
      !rows_ok(*o, B, nq, h) || !rows_ok(*d_o, B, nq, h) || !rows_ok(*dq, B, nq, h) ||
      !rows_ok(*dk, B, nkv, hkv) || !rows_ok(*dv, B, nkv, hkv) ||
      !rows_apart(*dq, B, nq, h, c) || !rows_apart(*dk, B, nkv, hkv, c) ||
      !rows_apart(*dv, B, nkv, hkv, c) || stats == nullptr || unaligned(stats, 8) ||
      unaligned(lens, 4) || workspace == nullptr || unaligned(workspace, 256))
    return BPT_ERR_INVALID_ARG;
  // Gradients may interleave with one another (the parts of one packed
  // gradient), but share no row, and they meet nothing that is read (below).
  const int64_t by_q[3] = {B, nq, h}, by_k[3] = {B, nkv, hkv};
  if (rows_meet(*dq, by_q, *dk, by_k, c) || rows_meet(*dq, by_q, *dv, by_k, c) ||
      rows_meet(*dk, by_k, *dv, by_k, c))
    return BPT_ERR_INVALID_ARG;
  const WindowBwdPlan plan = window_bwd_plan(w);
  if (workspace_bytes < plan.total) return BPT_ERR_WORKSPACE;
  const Range rq = rows_range(*q, B, nq, h, c), rk = rows_range(*k, B, nkv, hkv, c),
              rv = rows_range(*v, B, nkv, hkv, c), ro = rows_range(*o, B, nq, h, c),
              rd = rows_range(*d_o, B, nq, h, c), rl(lens, size_t(B) * 4),
              rs(stats, size_t(B * h) * size_t(nq) * 8), rw(workspace, plan.total);
  for (const Range& r : {rows_range(*dq, B, nq, h, c), rows_range(*dk, B, nkv, hkv, c),
                         rows_range(*dv, B, nkv, hkv, c), rw})
    if (any_meets(r, {rq, rk, rv, ro, rd, rl, rs})) return BPT_ERR_INVALID_ARG;
  if (any_meets(rw, {rows_range(*dq, B, nq, h, c), rows_range(*dk, B, nkv, hkv, c),
                     rows_range(*dv, B, nkv, hkv, c)}))
    return BPT_ERR_INVALID_ARG;
  int sms = 0;
  st = ops_device(&sms);
  if (st != BPT_OK) return st;
  st = ops_encoder();
  if (st != BPT_OK) return st;
  // q, k, v, dO in boxes of 128 rows and of those that stream through a block
  CUtensorMap stay[4], stream_maps[4];
  const int qt = c == 128 ? bpt::kWinTile<128> : bpt::kWinTile<64>;
  const bpt_rows* in[4] = {q, k, v, d_o};
  for (int i = 0; i < 4; ++i) {
    const bool is_q = i == 0 || i == 3;
    const int64_t n = is_q ? nq : nkv, hh = is_q ? h : hkv;
    if (!map_rows(&stay[i], *in[i], B, n, hh, c)) return BPT_ERR_CUDA;
    if (qt == 128)
      stream_maps[i] = stay[i];
    else if (!map_rows(&stream_maps[i], *in[i], B, n, hh, c, qt))
      return BPT_ERR_CUDA;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t* range = nullptr;
  if (w->dtype == BPT_F16) {
    range = reinterpret_cast<uint32_t*>(ws + plan.off_range);
    if (cudaMemsetAsync(range, 0, plan.range_bytes, s) != cudaSuccess) return BPT_ERR_CUDA;
  }
  bpt::WindowTermsParams tp{};
  tp.o = o->data;
  tp.o_b = o->stride_b; tp.o_n = o->stride_n; tp.o_h = o->stride_h;
  tp.d_o = d_o->data;
  tp.d_b = d_o->stride_b; tp.d_n = d_o->stride_n; tp.d_h = d_o->stride_h;
  tp.v = v->data;
  tp.v_b = v->stride_b; tp.v_n = v->stride_n; tp.v_h = v->stride_h;
  tp.stats = reinterpret_cast<const float2*>(stats);
  tp.terms = reinterpret_cast<float2*>(ws + plan.off_terms);
  tp.range = range;
  tp.lens = lens;
  tp.nq = int(nq); tp.nkv = int(nkv); tp.h = int(h); tp.g = int(h / hkv);
  tp.err = err;
  bpt::WindowBwdParams p{};
  p.nq = int(nq); p.nkv = int(nkv); p.h = int(h); p.hkv = int(hkv); p.g = int(h / hkv);
  p.nqb = int((nq + 127) / 128); p.nblk = int((nkv + 127) / 128);
  p.window = int(std::min<int64_t>(w->window, nkv));
  p.sinks = int(std::min<int64_t>(w->sinks, nkv));
  p.lens = lens;
  p.terms = tp.terms;
  p.range = reinterpret_cast<const uint2*>(range);
  p.dq = dq->data;
  p.dq_b = dq->stride_b; p.dq_n = dq->stride_n; p.dq_h = dq->stride_h;
  p.dk = dk->data;
  p.dk_b = dk->stride_b; p.dk_n = dk->stride_n; p.dk_h = dk->stride_h;
  p.dv = dv->data;
  p.dv_b = dv->stride_b; p.dv_n = dv->stride_n; p.dv_h = dv->stride_h;
  p.scale = float(1.0 / std::sqrt(double(c)));
  p.part_len = plan.part_len;
  p.split_parts = int(plan.cut_parts);
  p.part = reinterpret_cast<float*>(ws + plan.off_part);
  p.err = tp.err;
  cudaError_t e;
  using bf = __nv_bfloat16;
  if (w->dtype == BPT_BF16)
    e = c == 128 ? launch_window_bwd<bf, 128>(stay, stream_maps, tp, p, plan, B, s)
                 : launch_window_bwd<bf, 64>(stay, stream_maps, tp, p, plan, B, s);
  else
    e = c == 128 ? launch_window_bwd<__half, 128>(stay, stream_maps, tp, p, plan, B, s)
                 : launch_window_bwd<__half, 64>(stay, stream_maps, tp, p, plan, B, s);
  return e == cudaSuccess ? BPT_OK : BPT_ERR_CUDA;
}

}  // namespace bpt_host

extern "C" {

bpt_status bpt_cache_workspace_size(const bpt_cache* cache, size_t* bytes) {
  if (bytes == nullptr) return BPT_ERR_INVALID_ARG;
  const bpt_status st = check_cache(cache);
  if (st != BPT_OK) return st;
  *bytes = cache_layout(cache).total;
  return BPT_OK;
}

bpt_status bpt_cache_append(const bpt_cache* cache, const void* k_new, const void* v_new,
                            int64_t tokens, const int64_t* strides, const int32_t* counts,
                            int32_t* new_lens, float* acc, int32_t* pos, const int32_t* seen,
                            void* workspace, size_t workspace_bytes, bpt_stream_t stream) {
  return bpt_host::cache_append(cache, k_new, v_new, tokens, strides, counts, new_lens, acc, pos,
                                seen, workspace, workspace_bytes, stream, nullptr);
}

bpt_status bpt_cache_evict(const bpt_cache* cache, int64_t budget, int64_t recent, int64_t sinks,
                           const float* acc, const int32_t* pos, const int32_t* seen,
                           float* acc_out, int32_t* pos_out, int32_t* new_lens, void* workspace,
                           size_t workspace_bytes, bpt_stream_t stream) {
  bpt_status st = check_cache(cache);
  if (st != BPT_OK) return st;
  if (budget <= 0 || recent < 0 || sinks < 0) return BPT_ERR_INVALID_ARG;
  if (cache->batch == 0) return BPT_OK;
  st = check_cache_pointers(cache);
  if (st != BPT_OK) return st;
  const int64_t B = cache->batch;
  for (const void* p : {static_cast<const void*>(acc), static_cast<const void*>(pos),
                        static_cast<const void*>(seen), static_cast<const void*>(acc_out),
                        static_cast<const void*>(pos_out), static_cast<const void*>(new_lens)})
    if (p == nullptr || unaligned(p, 4)) return BPT_ERR_INVALID_ARG;
  if (workspace == nullptr || unaligned(workspace, 256)) return BPT_ERR_INVALID_ARG;
  const CacheLayout l = cache_layout(cache);
  if (workspace_bytes < l.total) return BPT_ERR_WORKSPACE;
  const size_t sb = slots_bytes(cache);
  const Range rk(cache->k, cache_bytes(cache)), rv(cache->v, cache_bytes(cache)),
      rl(cache->lens, size_t(B) * 4), rn(new_lens, size_t(B) * 4),
      rt(cache->page_table, size_t(B * cache->max_pages) * 4), ra(acc, sb), rp(pos, sb),
      rao(acc_out, sb), rpo(pos_out, sb), rs(seen, size_t(B) * 4), rw(workspace, l.total);
  // the state may be updated in place (acc_out == acc, pos_out == pos,
  // new_lens == lens); nothing else that is written meets another array
  if ((acc_out != acc && rao.meets(ra)) || (pos_out != pos && rpo.meets(rp)) ||
      (new_lens != cache->lens && rn.meets(rl)) ||
      any_meets(rao, {rp, rpo, rk, rv, rl, rn, rt, rs, rw}) ||
      any_meets(rpo, {ra, rk, rv, rl, rn, rt, rs, rw}) ||
      any_meets(rk, {ra, rp, rl, rn, rt, rs, rw}) || any_meets(rv, {ra, rp, rl, rn, rt, rs, rw}) ||
      any_meets(rn, {ra, rp, rt, rs, rw}) || any_meets(rw, {ra, rp, rl, rt, rs}))
    return BPT_ERR_INVALID_ARG;
  int sms = 0;
  st = ops_device(&sms);
  if (st != BPT_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  bpt::EvictParams p{};
  p.c = view_of(cache, static_cast<uint32_t*>(workspace));
  p.acc = acc;
  p.pos = pos;
  p.seen = seen;
  p.acc_out = acc_out;
  p.pos_out = pos_out;
  p.new_lens = new_lens;
  p.budget = clamp_u31(budget);
  p.recent = clamp_u31(recent);
  p.sinks = clamp_u31(sinks);
  p.row16 = uint32_t(cache->d_k / 8);
  p.lists = reinterpret_cast<int*>(ws + l.off_lists);
  p.count = reinterpret_cast<int*>(ws + l.off_count);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned hkv = unsigned(cache->kv_heads);
  // Blocks per pair: about 4096 slots each (four per thread), at most a
  // portable cluster.  Up to there one block holds a pair and moves its rows
  // itself: eight caches of 1300 slots, 12 heads, take 16.5 us with a launch of
  // its own for the moves, which is only needed where new_lens is lens.
  unsigned C = 1;
  while (C < bpt::kEvictMaxCluster && p.c.cap > C * 4096u &&
         B * int64_t(hkv) * int64_t(2 * C) <= 2 * sms)
    C *= 2;
  const bool fused = C == 1 && new_lens != cache->lens;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(hkv * C, unsigned(B));
  cfg.blockDim = dim3(bpt::kEvictThreads);
  cfg.dynamicSmemBytes = bpt::kEvictSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  if ((fused ? cudaLaunchKernelEx(&cfg, bpt::cache_evict_select_kernel<true>, p, uint32_t(C))
             : cudaLaunchKernelEx(&cfg, bpt::cache_evict_select_kernel<false>, p, uint32_t(C))) !=
      cudaSuccess) {
    (void)cudaGetLastError();
    return BPT_ERR_CUDA;
  }
  if (fused) return BPT_OK;
  // at most min(budget, capacity / 2) rows of a pair move; enough blocks to
  // fill the device, at least one step each
  const int64_t moves = std::min<int64_t>(p.budget, int64_t(p.c.cap) / 2);
  const int64_t per = bpt::kMoveThreads / int64_t(p.row16);
  const int64_t steps = (moves + per - 1) / per;
  const int64_t fill = std::max<int64_t>(1, int64_t(sms) * 16 / (B * int64_t(hkv)));
  const unsigned gx = unsigned(std::max<int64_t>(1, std::min(steps, fill)));
  bpt::cache_evict_move_kernel<<<dim3(gx, hkv, unsigned(B)), bpt::kMoveThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? BPT_OK : BPT_ERR_CUDA;
}

bpt_status bpt_attn_decode_workspace_size(const bpt_cache* cache, int64_t heads, int with_acc,
                                          size_t* bytes) {
  if (bytes == nullptr) return BPT_ERR_INVALID_ARG;
  bpt_status st = check_cache(cache);
  if (st != BPT_OK) return st;
  DecodeLayout l;
  st = decode_layout(cache, heads, with_acc, &l);
  if (st != BPT_OK) return st;
  *bytes = l.total;
  return BPT_OK;
}

bpt_status bpt_attn_decode(const bpt_cache* cache, const void* q, int64_t heads,
                           int64_t q_stride_b, int64_t q_stride_h, int64_t window, int64_t sinks,
                           const float* acc, float* acc_out, void* out, int64_t out_stride_b,
                           int64_t out_stride_h, void* workspace, size_t workspace_bytes,
                           bpt_stream_t stream) {
  return bpt_host::attn_decode(cache, q, heads, q_stride_b, q_stride_h, window, sinks, acc,
                               acc_out, out, out_stride_b, out_stride_h, workspace,
                               workspace_bytes, stream, nullptr);
}

bpt_status bpt_attn_window_workspace_size(const bpt_window* w, size_t* bytes) {
  if (bytes == nullptr) return BPT_ERR_INVALID_ARG;
  const bpt_status st = check_window(w);
  if (st != BPT_OK) return st;
  *bytes = kOpsHeader;
  return BPT_OK;
}

bpt_status bpt_attn_window_forward(const bpt_window* w, const bpt_rows* q, const bpt_rows* k,
                                   const bpt_rows* v, const int32_t* lens, const bpt_rows* out,
                                   float* stats, void* workspace, size_t workspace_bytes,
                                   bpt_stream_t stream) {
  return bpt_host::window_forward(w, q, k, v, lens, out, stats, workspace, workspace_bytes, stream,
                                  nullptr);
}

bpt_status bpt_attn_window_backward_workspace_size(const bpt_window* w, size_t* bytes) {
  if (bytes == nullptr) return BPT_ERR_INVALID_ARG;
  const bpt_status st = check_window_bwd(w);
  if (st != BPT_OK) return st;
  *bytes = window_bwd_plan(w).total;
  return BPT_OK;
}

bpt_status bpt_attn_window_backward(const bpt_window* w, const bpt_rows* q, const bpt_rows* k,
                                    const bpt_rows* v, const bpt_rows* o, const float* stats,
                                    const bpt_rows* d_o, const int32_t* lens, const bpt_rows* dq,
                                    const bpt_rows* dk, const bpt_rows* dv, void* workspace,
                                    size_t workspace_bytes, bpt_stream_t stream) {
  return bpt_host::window_backward(w, q, k, v, o, stats, d_o, lens, dq, dk, dv, workspace,
                                   workspace_bytes, stream, nullptr);
}

}  // extern "C"

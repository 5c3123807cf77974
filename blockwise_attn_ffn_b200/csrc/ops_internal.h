// The attention operators as the layer calls use them: the public calls of the
// same names with the device error word to write (null: the workspace's own);
// check_only: every check of the arguments, nothing enqueued.
#pragma once

#include "bpt.h"

#define BPT_INTERNAL __attribute__((visibility("hidden")))

namespace bpt_host {

// Head of every workspace of these operators: the error word and the counters
// of the decode attention.  The same for all sizes and operators, so that one
// workspace serves any of them in turn.
constexpr size_t kOpsHeader = 4096;

BPT_INTERNAL bpt_status cache_append(const bpt_cache* cache, const void* k_new, const void* v_new,
                                     int64_t tokens, const int64_t* strides, const int32_t* counts,
                                     int32_t* new_lens, float* acc, int32_t* pos,
                                     const int32_t* seen, void* workspace, size_t workspace_bytes,
                                     bpt_stream_t stream, uint32_t* err, bool check_only = false);
BPT_INTERNAL bpt_status attn_decode(const bpt_cache* cache, const void* q, int64_t heads,
                                    int64_t q_stride_b, int64_t q_stride_h, int64_t window,
                                    int64_t sinks, const float* acc, float* acc_out, void* out,
                                    int64_t out_stride_b, int64_t out_stride_h, void* workspace,
                                    size_t workspace_bytes, bpt_stream_t stream, uint32_t* err,
                                    bool check_only = false);
BPT_INTERNAL bpt_status window_forward(const bpt_window* w, const bpt_rows* q, const bpt_rows* k,
                                       const bpt_rows* v, const int32_t* lens, const bpt_rows* out,
                                       float* stats, void* workspace, size_t workspace_bytes,
                                       bpt_stream_t stream, uint32_t* err);
BPT_INTERNAL bpt_status window_backward(const bpt_window* w, const bpt_rows* q, const bpt_rows* k,
                                        const bpt_rows* v, const bpt_rows* o, const float* stats,
                                        const bpt_rows* d_o, const int32_t* lens,
                                        const bpt_rows* dq, const bpt_rows* dk, const bpt_rows* dv,
                                        void* workspace, size_t workspace_bytes,
                                        bpt_stream_t stream, uint32_t* err);

}  // namespace bpt_host

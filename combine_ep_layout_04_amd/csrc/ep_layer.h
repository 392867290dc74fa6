// ep_layer.h -- launches of the router, the row movement and the 4-bit
// products (ep_router.hip, ep_permute.hip, ep_w4.hip), apart from
// ep_internal.h: what the counters of the dispatch and combine kernels were
// taken on does not change with these.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

// dtype: 0 bf16, 1 fp16, 2 fp32.

struct RouterArgs {
    const void* logits;
    int64_t num_tokens, ld;
    int num_experts, num_topk, softmax;
    const float* bias;
    int num_groups, topk_groups, group_top, renormalize;
    float scale;
    int64_t* topk_idx;
    float* topk_weights;
    float* probs;
};
hipError_t launch_router(int dtype, const RouterArgs& a, hipStream_t stream);

struct RouterBackwardArgs {
    const void* logits;
    int64_t num_tokens, ld;
    int num_experts, num_topk, softmax, renormalize;
    float scale;
    const int64_t* topk_idx;
    const float* grad_weights;
    const float* grad_probs;
    void* grad_logits;
};
hipError_t launch_router_backward(int dtype, const RouterBackwardArgs& a, hipStream_t stream);

// Rows moved between token order and expert order.  gather: out[t] = sum_j
// w * rows[slot]; else out[slot] = w * tokens[t].  With grad_weights also
// <tokens[t], rows[slot]> per pair.
struct MoveArgs {
    bool gather;
    const void* tokens;
    int64_t ld_tokens;
    const void* rows;
    int64_t ld_rows;
    void* out;
    int64_t ld_out;
    int64_t num_tokens, num_rows;
    int hidden, num_topk;
    const int32_t* slot;
    const float* weights;
    float* grad_weights;
};
hipError_t launch_move_rows(int dtype, const MoveArgs& a, hipStream_t stream);
// Workgroups the call may launch (it is refused past INT32_MAX).
int64_t move_rows_max_blocks(int dtype, int64_t num_tokens, int hidden, int num_topk);

hipError_t launch_clear_rows(int dtype, const int32_t* counts, const int32_t* offsets,
                             int num_experts, void* rows, int64_t ld, int64_t num_rows, int hidden,
                             hipStream_t stream);

// The packed 4-bit weights: sections and sizes.
struct W4Shape {
    int halves, half_n, row_blocks, k_tiles, tile_groups;
    int64_t scales_at, zeros_at, bytes;
};
W4Shape w4_shape(int num_experts, int n, int k, int group, bool zeros, bool glu);
hipError_t launch_w4_pack(int dtype, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                          int num_experts, int n, int k, int group, bool glu, void* packed,
                          hipStream_t stream);
struct W4Args {
    const void* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    const void* packed;
    int num_experts, n, k, group;
    bool zeros, glu;
    const int32_t* offsets;
    const int32_t* counts;
    int64_t num_rows;
    void* out;
    int64_t ld_out;
};
int64_t w4_max_blocks(const W4Args& a);
hipError_t launch_w4(int dtype, const W4Args& a, hipStream_t stream);

}  // namespace ep

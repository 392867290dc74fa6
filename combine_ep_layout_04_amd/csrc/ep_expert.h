// ep_expert.h -- launches of the experts' products (ep_expert.hip,
// ep_expert_few.hip, ep_expert_backward.hip, ep_expert_fp8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

// dtype: 0 bf16, 1 fp16.  Rows [num_rows] in segments of the layout; weights
// [num_experts, n, k], packed.
struct ExpertArgs {
    const void* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    const void* w;
    int num_experts, n, k;
    const int32_t* offsets;
    const int32_t* counts;
    int64_t num_rows;
    bool gated;
    void* out;
    int64_t ld_out;
    void* pre;          // gated only, may be NULL
    int64_t ld_pre;
};
hipError_t launch_expert(int dtype, const ExpertArgs& a, hipStream_t stream);
// For few rows an expert (ep_expert_few.hip).
hipError_t launch_expert_few(int dtype, const ExpertArgs& a, hipStream_t stream);
// Workgroups the call may launch (it is refused past INT32_MAX).
int64_t expert_max_blocks(const ExpertArgs& a);

struct ExpertBackwardArgs {
    const void* grad;       // [num_rows, n]
    int64_t ld_grad;
    bool padded;            // grad's rows are padded to 8 columns with zeros
    const void* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    bool x_padded;          // x's rows are
    const void* w;
    int num_experts, n, k;
    const int32_t* offsets;
    const int32_t* counts;
    int64_t num_rows;
    void* grad_rows;        // [num_rows, k] or NULL
    int64_t ld_grad_rows;
    void* grad_w;           // [num_experts, n, k] or NULL
    bool wide_w;            // grad_w in fp32, else in dtype
    // where to lay rows out first, padded to 8 columns with zeros, or NULL;
    // with src x has to be
    void* grad_copy;
    void* x_copy;
};
hipError_t launch_expert_backward(int dtype, const ExpertBackwardArgs& a, hipStream_t stream);

// Gradient of silu(gate) * up: out [num_rows, ld_out] holds both halves (n / 2
// each) side by side, its columns past n cleared.
struct GluBackwardArgs {
    const void* grad;       // [num_rows, n / 2]
    int64_t ld_grad;
    const void* pre;        // [num_rows, n]
    int64_t ld_pre;
    int64_t num_rows;
    int n;
    void* out;
    int64_t ld_out;         // a multiple of 8, at least n
};
hipError_t launch_glu_backward(int dtype, const GluBackwardArgs& a, hipStream_t stream);

// Rows and weights in 8 bits.
struct ExpertFp8Args {
    const void* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    int x_format;           // 0 E4M3, 1 E5M2
    const void* x_scales;
    bool scale_bytes;       // UE8M0 bytes, else fp32
    int64_t scale_row, scale_block;     // strides of x_scales, in elements
    const void* w;
    const float* w_scales;  // [num_experts, ceil(n / 128), ceil(k / 128)]
    int num_experts, n, k;
    const int32_t* offsets;
    const int32_t* counts;
    int64_t num_rows;
    bool gated;
    void* out;
    int64_t ld_out;
};
hipError_t launch_expert_fp8(int dtype, const ExpertFp8Args& a, hipStream_t stream);
int64_t expert_fp8_max_blocks(const ExpertFp8Args& a);

}  // namespace ep

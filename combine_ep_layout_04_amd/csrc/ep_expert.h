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
    // with src and grad_w x has to be
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
// Whether a launch can hold the call's workgroups and threads (else it is refused).
bool expert_fp8_fits(const ExpertFp8Args& a);

// Whether the kernels for few rows take a call, or the tiles.  The former read
// the weights once per 16 or 32 rows, in one workgroup per 32 to 64 of their
// rows; the latter hold 256 of them, so they need as many tiles to fill the
// chip.  us, few against tiles: 64 experts 2048 -> 2x1408 (704 tiles), 8 rows
// an expert 132 to 136, 16 rows 158 to 138, 32 rows 180 to 142, 8-bit 68 to 76,
// 91 to 77, 139 to 80; 16 experts 2048 -> 4096 (256 tiles) 12 rows 59 to 51;
// 8 experts (128 tiles) 24 rows 38 to 45, 32 rows 41 to 46; 1 expert (16 tiles)
// 64 rows 10.7 to 24.5, 128 rows 17.6 to 25.0; 2 experts (32 tiles) 64 rows
// 22.0 to 24.7, 128 rows 35.8 to 25.8.  The last border, 64 rows, is that of 32
// tiles; 16 tiles and fewer lose by it from 65 to 128 rows.  It would move with
// the walk of ep_product.h, which gives so few tiles to a few XCDs only.
inline bool few_rows(int64_t num_rows, int num_experts, int n)
{
    const int64_t hold = num_rows < num_experts ? num_rows : num_experts;  // experts that can have a row
    const int64_t tiles = hold * n / 256;
    return num_rows / hold <= (tiles > 128 ? 8 : tiles > 32 ? 32 : 64);
}

}  // namespace ep

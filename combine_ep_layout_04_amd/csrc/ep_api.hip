// ep_api.hip -- the C ABI declared in include/ep.h: argument checks on the
// host, then stream-ordered launches.  Nothing here allocates, frees or
// synchronises; every failure is a returned status code (the pages' host
// library maps CUDA errors to an internal-error code and returns invalid-
// argument / invalid-usage codes; it never has to exit for bad input here).

#include <stdarg.h>
#include <stdio.h>

#include "ep.h"
#include "ep_expert.h"
#include "ep_internal.h"
#include "ep_layer.h"

static_assert(EP_LAYOUT_NOALLOC_SCRATCH_BYTES == ep::kLayoutScratchBytes,
              "the header states the layout scratch size");
static_assert(EP_MAX_EXPERTS == ep::kLayoutScratchExperts, "the scratch covers every expert count");

namespace {

thread_local char g_last_error[256] = "";

ep_status_t fail(ep_status_t status, const char* fmt, ...)
{
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof g_last_error, fmt, ap);
    va_end(ap);
    return status;
}

ep_status_t from_hip(hipError_t err, const char* what)
{
    if (err == hipSuccess) return EP_SUCCESS;
    return fail(EP_RUNTIME_ERROR, "%s: %s", what, hipGetErrorString(err));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

ep_status_t check_tokens(int64_t num_tokens, int num_topk)
{
    if (num_tokens < 0) return fail(EP_INVALID_ARGUMENT, "num_tokens < 0");
    if (num_topk < 1 || num_topk > EP_MAX_TOPK)
        return fail(EP_INVALID_ARGUMENT, "num_topk %d outside [1, %d]", num_topk, EP_MAX_TOPK);
    if (num_tokens * (int64_t)num_topk >= ((int64_t)1 << 31))
        return fail(EP_UNSUPPORTED, "num_tokens * num_topk must be < 2^31");
    return EP_SUCCESS;
}

ep_status_t check_hidden(int hidden, int multiple)
{
    if (hidden < 1 || hidden > EP_MAX_HIDDEN || hidden % multiple != 0)
        return fail(EP_INVALID_ARGUMENT, "hidden %d must be a positive multiple of %d, at most %d",
                    hidden, multiple, EP_MAX_HIDDEN);
    return EP_SUCCESS;
}

}  // namespace

extern "C" {

int ep_version(void) { return (1 << 16) | 0; }

const char* ep_status_string(int status)
{
    switch (status) {
    case EP_SUCCESS: return "EP_SUCCESS";
    case EP_INVALID_ARGUMENT: return "EP_INVALID_ARGUMENT";
    case EP_UNSUPPORTED: return "EP_UNSUPPORTED";
    case EP_RUNTIME_ERROR: return "EP_RUNTIME_ERROR";
    default: return "EP_UNKNOWN_STATUS";
    }
}

const char* ep_last_error(void) { return g_last_error; }

size_t ep_layout_workspace_size(int64_t num_tokens, int num_topk, int num_experts)
{
    if (num_tokens < 0 || num_topk < 1 || num_topk > EP_MAX_TOPK || num_experts < 1 ||
        num_experts > EP_MAX_EXPERTS || num_tokens * (int64_t)num_topk >= ((int64_t)1 << 31))
        return 0;
    return ep::layout_workspace_bytes(num_tokens * (int64_t)num_topk, num_experts);
}

int64_t ep_layout_max_rows(int64_t num_tokens, int num_topk, int num_experts, int alignment,
                           int64_t expert_capacity)
{
    if (num_tokens < 0 || num_topk < 1 || num_topk > EP_MAX_TOPK || num_experts < 1 ||
        num_experts > EP_MAX_EXPERTS || alignment < 1 || alignment > EP_MAX_ALIGNMENT ||
        expert_capacity < 0 || (expert_capacity > 0 && expert_capacity % alignment != 0) ||
        num_tokens * (int64_t)num_topk >= ((int64_t)1 << 31))
        return -1;
    const int64_t pairs = num_tokens * (int64_t)num_topk;
    if (expert_capacity > 0) return (int64_t)num_experts * expert_capacity;
    // every expert with at least one pair may add up to alignment-1 rows
    const int64_t touched = pairs < num_experts ? pairs : num_experts;
    return pairs + touched * (alignment - 1);
}

ep_status_t ep_layout_ex(const int64_t* topk_idx, int64_t num_tokens, int num_topk, int num_experts,
                         int alignment, int64_t expert_capacity, int32_t* counts, int32_t* offsets,
                         int32_t* slot, int32_t* src, int32_t* num_invalid, int32_t* num_dropped,
                         void* workspace, size_t workspace_bytes, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts,
                    EP_MAX_EXPERTS);
    if (alignment < 1 || alignment > EP_MAX_ALIGNMENT)
        return fail(EP_INVALID_ARGUMENT, "alignment %d outside [1, %d]", alignment,
                    EP_MAX_ALIGNMENT);
    if (expert_capacity < 0 || (expert_capacity > 0 && expert_capacity % alignment != 0))
        return fail(EP_INVALID_ARGUMENT,
                    "expert_capacity %lld must be 0 or a positive multiple of alignment %d",
                    (long long)expert_capacity, alignment);
    const int64_t rows = ep_layout_max_rows(num_tokens, num_topk, num_experts, alignment,
                                            expert_capacity);
    if (rows < 0 || rows >= ((int64_t)1 << 31))
        return fail(EP_UNSUPPORTED, "the layout could need %lld rows; rows must stay below 2^31",
                    (long long)rows);
    if (!counts || !offsets) return fail(EP_INVALID_ARGUMENT, "counts and offsets are required");
    if (num_tokens > 0 && (!topk_idx || !slot))
        return fail(EP_INVALID_ARGUMENT, "topk_idx and slot are required");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(EP_INVALID_ARGUMENT, "workspace must be non-NULL and 256-byte aligned");
    const size_t need = ep_layout_workspace_size(num_tokens, num_topk, num_experts);
    if (workspace_bytes < need)
        return fail(EP_INVALID_ARGUMENT, "workspace %zu bytes < %zu required", workspace_bytes, need);
    if ((reinterpret_cast<uintptr_t>(topk_idx) & 7u))
        return fail(EP_INVALID_ARGUMENT, "topk_idx must be 8-byte aligned");
    return from_hip(ep::launch_layout(topk_idx, num_tokens, num_topk, num_experts, alignment,
                                      (int)expert_capacity, counts, offsets, slot, src,
                                      num_invalid, num_dropped, workspace,
                                      static_cast<hipStream_t>(stream)),
                    "ep_layout launch");
}

ep_status_t ep_layout(const int64_t* topk_idx, int64_t num_tokens, int num_topk, int num_experts,
                      int32_t* counts, int32_t* offsets, int32_t* slot, int32_t* src,
                      int32_t* num_invalid, void* workspace, size_t workspace_bytes, void* stream)
{
    return ep_layout_ex(topk_idx, num_tokens, num_topk, num_experts, 1, 0, counts, offsets, slot,
                        src, num_invalid, nullptr, workspace, workspace_bytes, stream);
}

ep_status_t ep_layout_noalloc(const int64_t* topk_idx, int64_t num_tokens, int num_topk,
                              int num_experts, int32_t* counts, int32_t* offsets, int32_t* slot,
                              int32_t* src, int32_t* num_invalid, void* stream)
{
    g_last_error[0] = '\0';
    const size_t need = ep_layout_workspace_size(num_tokens, num_topk, num_experts);
    if (need == 0)   // an invalid shape: ep_layout_ex names the argument, before any HIP call
        return ep_layout_ex(topk_idx, num_tokens, num_topk, num_experts, 1, 0, counts, offsets,
                            slot, src, num_invalid, nullptr, nullptr, 0, stream);
    const size_t have = ep::layout_scratch_bytes();
    if (need > have)
        return fail(EP_UNSUPPORTED,
                    "ep_layout_noalloc: this shape needs %zu bytes of scratch, more than the %zu "
                    "bytes the library holds per device",
                    need, have);
    void* scratch = nullptr;
    const ep_status_t st = from_hip(ep::layout_scratch(&scratch), "ep_layout_noalloc scratch address");
    if (st) return st;
    return ep_layout_ex(topk_idx, num_tokens, num_topk, num_experts, 1, 0, counts, offsets, slot,
                        src, num_invalid, nullptr, scratch, have, stream);
}

// scale_ld: 0, or a positive multiple of the 16-byte column alignment
static ep_status_t check_scale_ld(int64_t scale_ld, int elem_bytes)
{
    const int64_t align = 16 / elem_bytes;
    if (scale_ld < 0 || (scale_ld > 0 && scale_ld % align != 0))
        return fail(EP_INVALID_ARGUMENT,
                    "scale_ld %lld must be 0 (row-major) or a positive multiple of %lld",
                    (long long)scale_ld, (long long)align);
    return EP_SUCCESS;
}

ep_status_t ep_dispatch_ex(const void* x, int64_t num_tokens, int hidden, int num_topk,
                           const int32_t* slot, const float* topk_weights, int out_dtype,
                           int scale_format, void* recv_x, void* recv_scales, float* recv_weights,
                           int64_t scale_ld, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    if (out_dtype != EP_OUT_BF16 && out_dtype != EP_OUT_FP8_E4M3 && out_dtype != EP_OUT_FP8_E5M2)
        return fail(EP_INVALID_ARGUMENT, "unknown out_dtype %d", out_dtype);
    if (scale_format != EP_SCALE_FP32 && scale_format != EP_SCALE_FP32_POW2 &&
        scale_format != EP_SCALE_UE8M0)
        return fail(EP_INVALID_ARGUMENT, "unknown scale_format %d", scale_format);
    const bool fp8 = out_dtype != EP_OUT_BF16;
    if (!fp8 && scale_format != EP_SCALE_FP32)
        return fail(EP_INVALID_ARGUMENT, "bf16 output takes no scale format");
    st = check_hidden(hidden, fp8 ? 128 : 8);
    if (st) return st;
    if (!fp8 && scale_ld != 0) return fail(EP_INVALID_ARGUMENT, "bf16 output takes no scale_ld");
    st = check_scale_ld(scale_ld, scale_format == EP_SCALE_UE8M0 ? 1 : 4);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x || !slot || !recv_x) return fail(EP_INVALID_ARGUMENT, "x, slot and recv_x are required");
    if (!aligned16(x) || !aligned16(recv_x))
        return fail(EP_INVALID_ARGUMENT, "x and recv_x must be 16-byte aligned");
    if (recv_weights && !topk_weights)
        return fail(EP_INVALID_ARGUMENT, "recv_weights needs topk_weights");
    if (fp8) {
        if (!recv_scales) return fail(EP_INVALID_ARGUMENT, "fp8 dispatch needs recv_scales");
        if (scale_format != EP_SCALE_UE8M0 && (reinterpret_cast<uintptr_t>(recv_scales) & 3u))
            return fail(EP_INVALID_ARGUMENT, "fp32 recv_scales must be 4-byte aligned");
        return from_hip(ep::launch_dispatch_fp8(x, num_tokens, hidden, num_topk, slot, topk_weights,
                                                out_dtype == EP_OUT_FP8_E5M2 ? 1 : 0, scale_format,
                                                recv_x, recv_scales, recv_weights, scale_ld,
                                                static_cast<hipStream_t>(stream)),
                        "ep_dispatch (fp8) launch");
    }
    if (recv_scales) return fail(EP_INVALID_ARGUMENT, "recv_scales must be NULL for bf16 output");
    return from_hip(ep::launch_dispatch_bf16(x, num_tokens, hidden, num_topk, slot, topk_weights,
                                             recv_x, recv_weights, static_cast<hipStream_t>(stream)),
                    "ep_dispatch (bf16) launch");
}

size_t ep_dispatch_colmajor_workspace_size(int64_t num_tokens, int hidden, int scale_format)
{
    if (num_tokens < 0 || hidden < 128 || hidden > EP_MAX_HIDDEN || hidden % 128 != 0 ||
        (scale_format != EP_SCALE_FP32 && scale_format != EP_SCALE_FP32_POW2 &&
         scale_format != EP_SCALE_UE8M0))
        return 0;
    return ep::colmajor_workspace_bytes(num_tokens, hidden, scale_format);
}

ep_status_t ep_dispatch_colmajor_scales(const void* x, int64_t num_tokens, int hidden, int num_topk,
                                        const int32_t* slot, const int32_t* src,
                                        const float* topk_weights, int out_dtype, int scale_format,
                                        void* recv_x, void* recv_scales, float* recv_weights,
                                        int64_t scale_ld, int64_t num_rows, void* workspace,
                                        size_t workspace_bytes, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    if (out_dtype != EP_OUT_FP8_E4M3 && out_dtype != EP_OUT_FP8_E5M2)
        return fail(EP_INVALID_ARGUMENT, "out_dtype %d: column-major scales come with an 8-bit cast",
                    out_dtype);
    if (scale_format != EP_SCALE_FP32 && scale_format != EP_SCALE_FP32_POW2 &&
        scale_format != EP_SCALE_UE8M0)
        return fail(EP_INVALID_ARGUMENT, "unknown scale_format %d", scale_format);
    st = check_hidden(hidden, 128);
    if (st) return st;
    if (scale_ld <= 0) return fail(EP_INVALID_ARGUMENT, "scale_ld must be positive (column-major)");
    st = check_scale_ld(scale_ld, scale_format == EP_SCALE_UE8M0 ? 1 : 4);
    if (st) return st;
    if (num_rows < 0 || num_rows > INT32_MAX)
        return fail(EP_INVALID_ARGUMENT, "num_rows %lld outside [0, 2^31-1] (slot entries are int32)",
                    (long long)num_rows);
    if (scale_ld < num_rows)
        return fail(EP_INVALID_ARGUMENT, "scale_ld %lld is below num_rows %lld", (long long)scale_ld,
                    (long long)num_rows);
    const size_t need = ep_dispatch_colmajor_workspace_size(num_tokens, hidden, scale_format);
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(EP_INVALID_ARGUMENT, "workspace must be non-NULL and 256-byte aligned");
    if (workspace_bytes < need)
        return fail(EP_INVALID_ARGUMENT, "workspace %zu bytes < %zu required", workspace_bytes, need);
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x || !slot || !src || !recv_x || !recv_scales)
        return fail(EP_INVALID_ARGUMENT, "x, slot, src, recv_x and recv_scales are required");
    if (!aligned16(x) || !aligned16(recv_x))
        return fail(EP_INVALID_ARGUMENT, "x and recv_x must be 16-byte aligned");
    if (scale_format != EP_SCALE_UE8M0 && (reinterpret_cast<uintptr_t>(recv_scales) & 3u))
        return fail(EP_INVALID_ARGUMENT, "fp32 recv_scales must be 4-byte aligned");
    if (recv_weights && !topk_weights)
        return fail(EP_INVALID_ARGUMENT, "recv_weights needs topk_weights");
    return from_hip(ep::launch_dispatch_fp8_colmajor(
                        x, num_tokens, hidden, num_topk, slot, src, topk_weights,
                        out_dtype == EP_OUT_FP8_E5M2 ? 1 : 0, scale_format, recv_x, recv_scales,
                        recv_weights, scale_ld, num_rows, workspace,
                        static_cast<hipStream_t>(stream)),
                    "ep_dispatch_colmajor_scales launch");
}

ep_status_t ep_dispatch(const void* x, int64_t num_tokens, int hidden, int num_topk,
                        const int32_t* slot, const float* topk_weights, int out_dtype, void* recv_x,
                        float* recv_scales, float* recv_weights, void* stream)
{
    return ep_dispatch_ex(x, num_tokens, hidden, num_topk, slot, topk_weights, out_dtype,
                          EP_SCALE_FP32, recv_x, recv_scales, recv_weights, 0, stream);
}

ep_status_t ep_dispatch_prequantized(const void* x_q, const float* x_scales, int64_t num_tokens,
                                     int hidden, int num_topk, const int32_t* slot,
                                     const float* topk_weights, void* recv_q, float* recv_scales,
                                     float* recv_weights, int64_t scale_ld, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 128);
    if (st) return st;
    st = check_scale_ld(scale_ld, 4);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x_q || !x_scales || !slot || !recv_q || !recv_scales)
        return fail(EP_INVALID_ARGUMENT, "x_q, x_scales, slot, recv_q and recv_scales are required");
    if (!aligned16(x_q) || !aligned16(recv_q))
        return fail(EP_INVALID_ARGUMENT, "x_q and recv_q must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(x_scales) & 3u) || (reinterpret_cast<uintptr_t>(recv_scales) & 3u))
        return fail(EP_INVALID_ARGUMENT, "scales must be 4-byte aligned");
    if (recv_weights && !topk_weights)
        return fail(EP_INVALID_ARGUMENT, "recv_weights needs topk_weights");
    return from_hip(ep::launch_dispatch_prequant(x_q, x_scales, num_tokens, hidden, num_topk, slot,
                                                 topk_weights, recv_q, recv_scales, recv_weights,
                                                 scale_ld, static_cast<hipStream_t>(stream)),
                    "ep_dispatch_prequantized launch");
}

ep_status_t ep_dispatch_prequantized_colmajor(const void* x_q, const float* x_scales,
                                              int64_t num_tokens, int hidden, int num_topk,
                                              const int32_t* slot, const int32_t* src,
                                              const float* topk_weights, void* recv_q,
                                              float* recv_scales, float* recv_weights,
                                              int64_t scale_ld, int64_t num_rows, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 128);
    if (st) return st;
    if (scale_ld <= 0) return fail(EP_INVALID_ARGUMENT, "scale_ld must be positive (column-major)");
    st = check_scale_ld(scale_ld, 4);
    if (st) return st;
    if (num_rows < 0 || num_rows > INT32_MAX)
        return fail(EP_INVALID_ARGUMENT, "num_rows %lld outside [0, 2^31-1] (slot entries are int32)",
                    (long long)num_rows);
    if (scale_ld < num_rows)
        return fail(EP_INVALID_ARGUMENT, "scale_ld %lld is below num_rows %lld", (long long)scale_ld,
                    (long long)num_rows);
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x_q || !x_scales || !slot || !src || !recv_q || !recv_scales)
        return fail(EP_INVALID_ARGUMENT,
                    "x_q, x_scales, slot, src, recv_q and recv_scales are required");
    if (!aligned16(x_q) || !aligned16(recv_q))
        return fail(EP_INVALID_ARGUMENT, "x_q and recv_q must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(x_scales) & 3u) || (reinterpret_cast<uintptr_t>(recv_scales) & 3u))
        return fail(EP_INVALID_ARGUMENT, "scales must be 4-byte aligned");
    if (recv_weights && !topk_weights)
        return fail(EP_INVALID_ARGUMENT, "recv_weights needs topk_weights");
    return from_hip(ep::launch_dispatch_prequant_colmajor(
                        x_q, x_scales, num_tokens, hidden, num_topk, slot, src, topk_weights, recv_q,
                        recv_scales, recv_weights, scale_ld, num_rows,
                        static_cast<hipStream_t>(stream)),
                    "ep_dispatch_prequantized_colmajor launch");
}

ep_status_t ep_combine(const void* y, const int32_t* slot, const float* topk_weights,
                       int64_t num_tokens, int hidden, int num_topk, void* out, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 8);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (!y || !slot || !out) return fail(EP_INVALID_ARGUMENT, "y, slot and out are required");
    if (!aligned16(y) || !aligned16(out))
        return fail(EP_INVALID_ARGUMENT, "y and out must be 16-byte aligned");
    return from_hip(ep::launch_combine(y, slot, topk_weights, num_tokens, hidden, num_topk, out,
                                       nullptr, nullptr, static_cast<hipStream_t>(stream)),
                    "ep_combine launch");
}

ep_status_t ep_combine_backward(const void* grad_out, const void* y, const int32_t* slot,
                                const float* topk_weights, int64_t num_tokens, int hidden,
                                int num_topk, void* grad_y, float* grad_topk_weights, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 8);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (!grad_out || !slot || !grad_y)
        return fail(EP_INVALID_ARGUMENT, "grad_out, slot and grad_y are required");
    if (grad_topk_weights && !y)
        return fail(EP_INVALID_ARGUMENT, "grad_topk_weights needs the expert outputs y");
    if (!aligned16(grad_out) || !aligned16(grad_y) || (y && !aligned16(y)))
        return fail(EP_INVALID_ARGUMENT, "grad_out, y and grad_y must be 16-byte aligned");
    return from_hip(ep::launch_combine_backward(grad_out, y, slot, topk_weights, num_tokens, hidden,
                                                num_topk, grad_y, grad_topk_weights,
                                                static_cast<hipStream_t>(stream)),
                    "ep_combine_backward launch");
}

ep_status_t ep_dispatch_backward(const void* grad_recv, const float* grad_recv_weights,
                                 const int32_t* slot, int64_t num_tokens, int hidden, int num_topk,
                                 void* grad_x, float* grad_topk_weights, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 8);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (!grad_recv || !slot || !grad_x)
        return fail(EP_INVALID_ARGUMENT, "grad_recv, slot and grad_x are required");
    if ((grad_topk_weights == nullptr) != (grad_recv_weights == nullptr))
        return fail(EP_INVALID_ARGUMENT,
                    "grad_recv_weights and grad_topk_weights are given together or not at all");
    if (!aligned16(grad_recv) || !aligned16(grad_x))
        return fail(EP_INVALID_ARGUMENT, "grad_recv and grad_x must be 16-byte aligned");
    return from_hip(ep::launch_combine(grad_recv, slot, nullptr, num_tokens, hidden, num_topk,
                                       grad_x, grad_recv_weights, grad_topk_weights,
                                       static_cast<hipStream_t>(stream)),
                    "ep_dispatch_backward launch");
}


// ---- per-(token, rank) path

static ep_status_t check_ranks(int num_experts, int num_ranks)
{
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts,
                    EP_MAX_EXPERTS);
    if (num_ranks < 1 || num_ranks > EP_MAX_RANKS)
        return fail(EP_INVALID_ARGUMENT, "num_ranks %d outside [1, %d]", num_ranks, EP_MAX_RANKS);
    if (num_experts % num_ranks != 0)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d is not a multiple of num_ranks %d",
                    num_experts, num_ranks);
    return EP_SUCCESS;
}

ep_status_t ep_routing_map(const int64_t* topk_idx, int64_t num_tokens, int num_topk,
                           int num_experts, uint8_t* routing_map, int32_t* num_invalid,
                           void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts,
                    EP_MAX_EXPERTS);
    if (num_tokens > 0 && (!topk_idx || !routing_map))
        return fail(EP_INVALID_ARGUMENT, "topk_idx and routing_map are required");
    if ((reinterpret_cast<uintptr_t>(topk_idx) & 7u))
        return fail(EP_INVALID_ARGUMENT, "topk_idx must be 8-byte aligned");
    if ((reinterpret_cast<uintptr_t>(num_invalid) & 3u))
        return fail(EP_INVALID_ARGUMENT, "num_invalid must be 4-byte aligned");
    return from_hip(ep::launch_routing_map(topk_idx, num_tokens, num_topk, num_experts,
                                           routing_map, num_invalid,
                                           static_cast<hipStream_t>(stream)),
                    "ep_routing_map launch");
}

size_t ep_rank_layout_workspace_size(int64_t tokens_per_rank, int num_experts, int num_ranks)
{
    if (tokens_per_rank < 0 || num_ranks < 1 || num_ranks > EP_MAX_RANKS || num_experts < 1 ||
        num_experts > EP_MAX_EXPERTS || num_experts % num_ranks != 0)
        return 0;
    const size_t bytes = ep::rank_layout_workspace_bytes(tokens_per_rank, num_experts, num_ranks);
    return (bytes + 255) & ~(size_t)255;
}

ep_status_t ep_rank_layout(const uint8_t* global_routing_map, int64_t tokens_per_rank,
                           int num_experts, int num_ranks, int rank, int k_out,
                           int32_t* sparse_to_dense_map, uint8_t* local_expert_routing_map,
                           int32_t* recv_src, int64_t* recv_topk_idx, int32_t* expert_counts,
                           int32_t* num_recv, int32_t* num_overflow, void* workspace,
                           size_t workspace_bytes, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_ranks(num_experts, num_ranks);
    if (st) return st;
    if (tokens_per_rank < 0) return fail(EP_INVALID_ARGUMENT, "tokens_per_rank < 0");
    if (rank < 0 || rank >= num_ranks)
        return fail(EP_INVALID_ARGUMENT, "rank %d outside [0, %d)", rank, num_ranks);
    if (k_out < 1 || k_out > EP_MAX_TOPK)
        return fail(EP_INVALID_ARGUMENT, "k_out %d outside [1, %d]", k_out, EP_MAX_TOPK);
    if (tokens_per_rank * (int64_t)num_ranks >= ((int64_t)1 << 31))
        return fail(EP_UNSUPPORTED, "num_ranks * tokens_per_rank must be < 2^31");
    if (!expert_counts || !num_recv)
        return fail(EP_INVALID_ARGUMENT, "expert_counts and num_recv are required");
    if (tokens_per_rank > 0 && (!global_routing_map || !sparse_to_dense_map ||
                                !local_expert_routing_map || !recv_src || !recv_topk_idx))
        return fail(EP_INVALID_ARGUMENT,
                    "global_routing_map, sparse_to_dense_map, local_expert_routing_map, recv_src "
                    "and recv_topk_idx are required");
    if ((reinterpret_cast<uintptr_t>(local_expert_routing_map) & 3u) ||
        (reinterpret_cast<uintptr_t>(sparse_to_dense_map) & 3u) ||
        (reinterpret_cast<uintptr_t>(recv_src) & 3u) ||
        (reinterpret_cast<uintptr_t>(expert_counts) & 3u))
        return fail(EP_INVALID_ARGUMENT, "int32 outputs and the local map must be 4-byte aligned");
    if ((reinterpret_cast<uintptr_t>(recv_topk_idx) & 7u))
        return fail(EP_INVALID_ARGUMENT, "recv_topk_idx must be 8-byte aligned");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return fail(EP_INVALID_ARGUMENT, "workspace must be non-NULL and 256-byte aligned");
    const size_t need = ep_rank_layout_workspace_size(tokens_per_rank, num_experts, num_ranks);
    if (workspace_bytes < need)
        return fail(EP_INVALID_ARGUMENT, "workspace %zu bytes < %zu required", workspace_bytes, need);
    return from_hip(ep::launch_rank_layout(global_routing_map, tokens_per_rank, num_experts,
                                           num_ranks, rank, k_out, sparse_to_dense_map,
                                           local_expert_routing_map, recv_src, recv_topk_idx,
                                           expert_counts, num_recv, num_overflow, workspace,
                                           static_cast<hipStream_t>(stream)),
                    "ep_rank_layout launch");
}

ep_status_t ep_dispatch_ranked(const void* x, const int64_t* topk_idx, const float* topk_weights,
                               int64_t num_tokens, int hidden, int num_topk, int num_experts,
                               int num_ranks, const int32_t* sparse_to_dense_map,
                               void* const* dest_x, float* const* dest_weights, int64_t dest_rows,
                               void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 8);
    if (st) return st;
    st = check_ranks(num_experts, num_ranks);
    if (st) return st;
    if (dest_rows < 0) return fail(EP_INVALID_ARGUMENT, "dest_rows < 0");
    if (!dest_x) return fail(EP_INVALID_ARGUMENT, "dest_x (a host array of pointers) is required");
    ep::RankPtrs px = {}, pw = {};
    for (int d = 0; d < num_ranks; ++d) {
        if (!dest_x[d] || !aligned16(dest_x[d]))
            return fail(EP_INVALID_ARGUMENT, "dest_x[%d] must be non-NULL and 16-byte aligned", d);
        px.p[d] = dest_x[d];
        if (dest_weights) {
            if ((reinterpret_cast<uintptr_t>(dest_weights[d]) & 3u))
                return fail(EP_INVALID_ARGUMENT, "dest_weights[%d] must be 4-byte aligned", d);
            pw.p[d] = dest_weights[d];
        }
    }
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x || !sparse_to_dense_map)
        return fail(EP_INVALID_ARGUMENT, "x and sparse_to_dense_map are required");
    if (!aligned16(x)) return fail(EP_INVALID_ARGUMENT, "x must be 16-byte aligned");
    if (dest_weights && (!topk_idx || (reinterpret_cast<uintptr_t>(topk_idx) & 7u)))
        return fail(EP_INVALID_ARGUMENT, "dest_weights needs an 8-byte aligned topk_idx");
    const ep::RankPtrs none = {};
    return from_hip(ep::launch_dispatch_ranked(x, topk_idx, topk_weights, num_tokens, hidden * 2,
                                               num_topk, num_experts, num_ranks,
                                               sparse_to_dense_map, px, pw, dest_weights != nullptr,
                                               nullptr, none, 0, dest_rows,
                                               static_cast<hipStream_t>(stream)),
                    "ep_dispatch_ranked launch");
}

ep_status_t ep_dispatch_ranked_prequantized(const void* x_q, const float* x_scales,
                                            const int64_t* topk_idx, const float* topk_weights,
                                            int64_t num_tokens, int hidden, int num_topk,
                                            int num_experts, int num_ranks,
                                            const int32_t* sparse_to_dense_map, void* const* dest_q,
                                            float* const* dest_scales, float* const* dest_weights,
                                            int64_t dest_rows, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 128);
    if (st) return st;
    st = check_ranks(num_experts, num_ranks);
    if (st) return st;
    if (dest_rows < 0) return fail(EP_INVALID_ARGUMENT, "dest_rows < 0");
    if (!dest_q || !dest_scales)
        return fail(EP_INVALID_ARGUMENT, "dest_q and dest_scales (host arrays of pointers) are required");
    ep::RankPtrs pq = {}, ps = {}, pw = {};
    for (int d = 0; d < num_ranks; ++d) {
        if (!dest_q[d] || !aligned16(dest_q[d]))
            return fail(EP_INVALID_ARGUMENT, "dest_q[%d] must be non-NULL and 16-byte aligned", d);
        if (!dest_scales[d] || (reinterpret_cast<uintptr_t>(dest_scales[d]) & 3u))
            return fail(EP_INVALID_ARGUMENT, "dest_scales[%d] must be non-NULL and 4-byte aligned", d);
        pq.p[d] = dest_q[d];
        ps.p[d] = dest_scales[d];
        if (dest_weights) {
            if ((reinterpret_cast<uintptr_t>(dest_weights[d]) & 3u))
                return fail(EP_INVALID_ARGUMENT, "dest_weights[%d] must be 4-byte aligned", d);
            pw.p[d] = dest_weights[d];
        }
    }
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x_q || !x_scales || !sparse_to_dense_map)
        return fail(EP_INVALID_ARGUMENT, "x_q, x_scales and sparse_to_dense_map are required");
    if (!aligned16(x_q)) return fail(EP_INVALID_ARGUMENT, "x_q must be 16-byte aligned");
    if ((reinterpret_cast<uintptr_t>(x_scales) & 3u))
        return fail(EP_INVALID_ARGUMENT, "x_scales must be 4-byte aligned");
    if (dest_weights && (!topk_idx || (reinterpret_cast<uintptr_t>(topk_idx) & 7u)))
        return fail(EP_INVALID_ARGUMENT, "dest_weights needs an 8-byte aligned topk_idx");
    return from_hip(ep::launch_dispatch_ranked(x_q, topk_idx, topk_weights, num_tokens, hidden,
                                               num_topk, num_experts, num_ranks,
                                               sparse_to_dense_map, pq, pw, dest_weights != nullptr,
                                               x_scales, ps, hidden / 128, dest_rows,
                                               static_cast<hipStream_t>(stream)),
                    "ep_dispatch_ranked_prequantized launch");
}

ep_status_t ep_dispatch_ranked_fp8(const void* x, const int64_t* topk_idx, const float* topk_weights,
                                   int64_t num_tokens, int hidden, int num_topk, int num_experts,
                                   int num_ranks, const int32_t* sparse_to_dense_map,
                                   int out_dtype, int scale_format, void* const* dest_q,
                                   void* const* dest_scales, float* const* dest_weights,
                                   int64_t dest_rows, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    if (out_dtype != EP_OUT_FP8_E4M3 && out_dtype != EP_OUT_FP8_E5M2)
        return fail(EP_INVALID_ARGUMENT, "out_dtype %d is not an 8-bit format", out_dtype);
    if (scale_format != EP_SCALE_FP32 && scale_format != EP_SCALE_FP32_POW2 &&
        scale_format != EP_SCALE_UE8M0)
        return fail(EP_INVALID_ARGUMENT, "unknown scale_format %d", scale_format);
    st = check_hidden(hidden, 128);
    if (st) return st;
    st = check_ranks(num_experts, num_ranks);
    if (st) return st;
    if (dest_rows < 0) return fail(EP_INVALID_ARGUMENT, "dest_rows < 0");
    if (ep::ranked_fp8_blocks(num_tokens, hidden, num_ranks) > INT32_MAX)
        return fail(EP_UNSUPPORTED, "num_tokens too large for hidden %d and %d ranks", hidden,
                    num_ranks);
    if (!dest_q || !dest_scales)
        return fail(EP_INVALID_ARGUMENT, "dest_q and dest_scales (host arrays of pointers) are required");
    const bool bytes = scale_format == EP_SCALE_UE8M0;
    ep::RankPtrs pq = {}, ps = {}, pw = {};
    for (int d = 0; d < num_ranks; ++d) {
        if (!dest_q[d] || !aligned16(dest_q[d]))
            return fail(EP_INVALID_ARGUMENT, "dest_q[%d] must be non-NULL and 16-byte aligned", d);
        if (!dest_scales[d] || (!bytes && (reinterpret_cast<uintptr_t>(dest_scales[d]) & 3u)))
            return fail(EP_INVALID_ARGUMENT, "dest_scales[%d] must be non-NULL%s", d,
                        bytes ? "" : " and 4-byte aligned");
        pq.p[d] = dest_q[d];
        ps.p[d] = dest_scales[d];
        if (dest_weights) {
            if ((reinterpret_cast<uintptr_t>(dest_weights[d]) & 3u))
                return fail(EP_INVALID_ARGUMENT, "dest_weights[%d] must be 4-byte aligned", d);
            pw.p[d] = dest_weights[d];
        }
    }
    if (num_tokens == 0) return EP_SUCCESS;
    if (!x || !sparse_to_dense_map)
        return fail(EP_INVALID_ARGUMENT, "x and sparse_to_dense_map are required");
    if (!aligned16(x)) return fail(EP_INVALID_ARGUMENT, "x must be 16-byte aligned");
    if (dest_weights && (!topk_idx || (reinterpret_cast<uintptr_t>(topk_idx) & 7u)))
        return fail(EP_INVALID_ARGUMENT, "dest_weights needs an 8-byte aligned topk_idx");
    return from_hip(ep::launch_dispatch_ranked_fp8(x, topk_idx, topk_weights, num_tokens, hidden,
                                                   num_topk, num_experts, num_ranks,
                                                   sparse_to_dense_map,
                                                   out_dtype == EP_OUT_FP8_E5M2 ? 1 : 0,
                                                   scale_format, pq, ps, pw,
                                                   dest_weights != nullptr, dest_rows,
                                                   static_cast<hipStream_t>(stream)),
                    "ep_dispatch_ranked_fp8 launch");
}

// Checks shared by the two fused-permute entry points; fills the pointer
// tables (src_s only when scales is true).
static ep_status_t fused_permute_args(const void* const* src_x, const float* const* src_s,
                                      bool scales, const int64_t* const* src_topk_idx,
                                      const float* const* src_topk_weights,
                                      int64_t tokens_per_rank, int hidden, int hidden_multiple,
                                      int num_topk, int num_experts, int num_ranks, int rank,
                                      int64_t rows, float* recv_weights, ep::RankPtrs& px,
                                      ep::RankPtrs& ps, ep::RankPtrs& pi, ep::RankPtrs& pw)
{
    if (tokens_per_rank < 0) return fail(EP_INVALID_ARGUMENT, "tokens_per_rank < 0");
    ep_status_t st = check_ranks(num_experts, num_ranks);
    if (st) return st;
    st = check_tokens(tokens_per_rank * num_ranks, num_topk);
    if (st) return st;
    st = check_hidden(hidden, hidden_multiple);
    if (st) return st;
    if (rank < 0 || rank >= num_ranks)
        return fail(EP_INVALID_ARGUMENT, "rank %d outside [0, %d)", rank, num_ranks);
    if (rows < 0) return fail(EP_INVALID_ARGUMENT, "rows < 0");
    if (tokens_per_rank == 0) return EP_SUCCESS;   // nothing is read or written
    if (!src_x) return fail(EP_INVALID_ARGUMENT, "src_x (a host array of pointers) is required");
    if (scales && !src_s)
        return fail(EP_INVALID_ARGUMENT, "src_scales (a host array of pointers) is required");
    if (recv_weights && !src_topk_idx)
        return fail(EP_INVALID_ARGUMENT, "recv_weights needs src_topk_idx");
    for (int d = 0; d < num_ranks; ++d) {
        if (!src_x[d] || !aligned16(src_x[d]))
            return fail(EP_INVALID_ARGUMENT, "src_x[%d] must be non-NULL and 16-byte aligned", d);
        px.p[d] = const_cast<void*>(src_x[d]);
        if (scales) {
            if (!src_s[d] || (reinterpret_cast<uintptr_t>(src_s[d]) & 3u))
                return fail(EP_INVALID_ARGUMENT,
                            "src_scales[%d] must be non-NULL and 4-byte aligned", d);
            ps.p[d] = const_cast<float*>(src_s[d]);
        }
        if (recv_weights) {
            if (!src_topk_idx[d] || (reinterpret_cast<uintptr_t>(src_topk_idx[d]) & 7u))
                return fail(EP_INVALID_ARGUMENT,
                            "src_topk_idx[%d] must be non-NULL and 8-byte aligned", d);
            pi.p[d] = const_cast<int64_t*>(src_topk_idx[d]);
            if (src_topk_weights) {
                if ((reinterpret_cast<uintptr_t>(src_topk_weights[d]) & 3u))
                    return fail(EP_INVALID_ARGUMENT, "src_topk_weights[%d] must be 4-byte aligned",
                                d);
                pw.p[d] = const_cast<float*>(src_topk_weights[d]);
            }
        }
    }
    return EP_SUCCESS;
}

static ep_status_t fused_permute_outputs(const int32_t* recv_src, const int32_t* slot,
                                         const void* recv_x, const int64_t* recv_topk_idx,
                                         const float* recv_weights, const int32_t* num_recv)
{
    if (!recv_src || !slot || !recv_x || (recv_weights && !recv_topk_idx))
        return fail(EP_INVALID_ARGUMENT,
                    "recv_src, slot, recv_x (and recv_topk_idx with recv_weights) are required");
    if (!aligned16(recv_x)) return fail(EP_INVALID_ARGUMENT, "recv_x must be 16-byte aligned");
    if (num_recv && (reinterpret_cast<uintptr_t>(num_recv) & 3u))
        return fail(EP_INVALID_ARGUMENT, "num_recv must be 4-byte aligned");
    return EP_SUCCESS;
}

ep_status_t ep_dispatch_fused_permute(const void* const* src_x, const int64_t* const* src_topk_idx,
                                      const float* const* src_topk_weights, int64_t tokens_per_rank,
                                      int hidden, int num_topk, int num_experts, int num_ranks,
                                      int rank, const int32_t* recv_src,
                                      const int64_t* recv_topk_idx, const int32_t* num_recv,
                                      const int32_t* slot, int64_t rows, void* recv_x,
                                      float* recv_weights, void* stream)
{
    g_last_error[0] = '\0';
    ep::RankPtrs px = {}, ps = {}, pi = {}, pw = {};
    ep_status_t st = fused_permute_args(src_x, nullptr, false, src_topk_idx, src_topk_weights,
                                        tokens_per_rank, hidden, 8, num_topk, num_experts,
                                        num_ranks, rank, rows, recv_weights, px, ps, pi, pw);
    if (st) return st;
    if (tokens_per_rank == 0) return EP_SUCCESS;
    st = fused_permute_outputs(recv_src, slot, recv_x, recv_topk_idx, recv_weights, num_recv);
    if (st) return st;
    return from_hip(ep::launch_dispatch_fused_permute(px, pi, pw, tokens_per_rank, hidden, num_topk,
                                                      num_experts, num_ranks, rank, recv_src,
                                                      recv_topk_idx, num_recv, slot, rows, recv_x,
                                                      recv_weights, static_cast<hipStream_t>(stream)),
                    "ep_dispatch_fused_permute launch");
}

ep_status_t ep_dispatch_fused_permute_prequantized(
    const void* const* src_q, const float* const* src_scales, const int64_t* const* src_topk_idx,
    const float* const* src_topk_weights, int64_t tokens_per_rank, int hidden, int num_topk,
    int num_experts, int num_ranks, int rank, const int32_t* recv_src,
    const int64_t* recv_topk_idx, const int32_t* num_recv, const int32_t* slot, int64_t rows,
    void* recv_q, float* recv_scales, float* recv_weights, void* stream)
{
    g_last_error[0] = '\0';
    ep::RankPtrs px = {}, ps = {}, pi = {}, pw = {};
    ep_status_t st = fused_permute_args(src_q, src_scales, true, src_topk_idx, src_topk_weights,
                                        tokens_per_rank, hidden, 128, num_topk, num_experts,
                                        num_ranks, rank, rows, recv_weights, px, ps, pi, pw);
    if (st) return st;
    if (tokens_per_rank == 0) return EP_SUCCESS;
    st = fused_permute_outputs(recv_src, slot, recv_q, recv_topk_idx, recv_weights, num_recv);
    if (st) return st;
    if (!recv_scales || (reinterpret_cast<uintptr_t>(recv_scales) & 3u))
        return fail(EP_INVALID_ARGUMENT, "recv_scales must be non-NULL and 4-byte aligned");
    return from_hip(ep::launch_dispatch_fused_permute_prequant(
                        px, ps, pi, pw, tokens_per_rank, hidden, num_topk, num_experts, num_ranks,
                        rank, recv_src, recv_topk_idx, num_recv, slot, rows, recv_q, recv_scales,
                        recv_weights, static_cast<hipStream_t>(stream)),
                    "ep_dispatch_fused_permute_prequantized launch");
}

ep_status_t ep_combine_ranked(const void* const* src_y, int64_t src_rows,
                              const int32_t* sparse_to_dense_map, int64_t num_tokens, int hidden,
                              int num_ranks, void* out, void* stream)
{
    g_last_error[0] = '\0';
    if (num_tokens < 0) return fail(EP_INVALID_ARGUMENT, "num_tokens < 0");
    if (num_ranks < 1 || num_ranks > EP_MAX_RANKS)
        return fail(EP_INVALID_ARGUMENT, "num_ranks %d outside [1, %d]", num_ranks, EP_MAX_RANKS);
    if (num_tokens * (int64_t)num_ranks >= ((int64_t)1 << 31))
        return fail(EP_UNSUPPORTED, "num_tokens * num_ranks must be < 2^31");
    ep_status_t st = check_hidden(hidden, 8);
    if (st) return st;
    if (src_rows < 0) return fail(EP_INVALID_ARGUMENT, "src_rows < 0");
    if (!src_y) return fail(EP_INVALID_ARGUMENT, "src_y (a host array of pointers) is required");
    ep::RankPtrs ps = {};
    for (int d = 0; d < num_ranks; ++d) {
        if (!src_y[d] || !aligned16(src_y[d]))
            return fail(EP_INVALID_ARGUMENT, "src_y[%d] must be non-NULL and 16-byte aligned", d);
        ps.p[d] = const_cast<void*>(src_y[d]);
    }
    if (num_tokens == 0) return EP_SUCCESS;
    if (!sparse_to_dense_map || !out)
        return fail(EP_INVALID_ARGUMENT, "sparse_to_dense_map and out are required");
    if (!aligned16(out)) return fail(EP_INVALID_ARGUMENT, "out must be 16-byte aligned");
    return from_hip(ep::launch_combine_ranked(ps, src_rows, sparse_to_dense_map, num_tokens, hidden,
                                              num_ranks, out, static_cast<hipStream_t>(stream)),
                    "ep_combine_ranked launch");
}

ep_status_t ep_dispatch_ranked_backward(const void* const* grad_recv_x,
                                        const float* const* grad_recv_weights, int64_t src_rows,
                                        const int64_t* topk_idx, const int32_t* sparse_to_dense_map,
                                        int64_t num_tokens, int hidden, int num_topk,
                                        int num_experts, int num_ranks, void* grad_x,
                                        float* grad_topk_weights, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_ranks(num_experts, num_ranks);
    if (st) return st;
    if (num_tokens * (int64_t)num_ranks >= ((int64_t)1 << 31))
        return fail(EP_UNSUPPORTED, "num_tokens * num_ranks must be < 2^31");
    if (src_rows < 0) return fail(EP_INVALID_ARGUMENT, "src_rows < 0");
    if (!grad_recv_x && !grad_recv_weights)
        return fail(EP_INVALID_ARGUMENT, "nothing to do: grad_recv_x and grad_recv_weights are NULL");
    if ((grad_recv_x != nullptr) != (grad_x != nullptr))
        return fail(EP_INVALID_ARGUMENT, "grad_recv_x and grad_x go together");
    if ((grad_recv_weights != nullptr) != (grad_topk_weights != nullptr))
        return fail(EP_INVALID_ARGUMENT, "grad_recv_weights and grad_topk_weights go together");
    ep::RankPtrs px = {}, pw = {};
    if (grad_recv_x) {
        st = check_hidden(hidden, 8);
        if (st) return st;
        for (int d = 0; d < num_ranks; ++d) {
            if (!grad_recv_x[d] || !aligned16(grad_recv_x[d]))
                return fail(EP_INVALID_ARGUMENT, "grad_recv_x[%d] must be non-NULL and 16-byte aligned",
                            d);
            px.p[d] = const_cast<void*>(grad_recv_x[d]);
        }
        if (num_tokens > 0 && !aligned16(grad_x))
            return fail(EP_INVALID_ARGUMENT, "grad_x must be 16-byte aligned");
    }
    if (grad_recv_weights) {
        for (int d = 0; d < num_ranks; ++d) {
            if ((reinterpret_cast<uintptr_t>(grad_recv_weights[d]) & 3u))
                return fail(EP_INVALID_ARGUMENT, "grad_recv_weights[%d] must be 4-byte aligned", d);
            pw.p[d] = const_cast<float*>(grad_recv_weights[d]);
        }
        if (num_tokens > 0 && (!topk_idx || (reinterpret_cast<uintptr_t>(topk_idx) & 7u)))
            return fail(EP_INVALID_ARGUMENT, "grad_recv_weights needs an 8-byte aligned topk_idx");
        if (num_tokens > 0 && (reinterpret_cast<uintptr_t>(grad_topk_weights) & 3u))
            return fail(EP_INVALID_ARGUMENT, "grad_topk_weights must be 4-byte aligned");
    }
    if (num_tokens == 0) return EP_SUCCESS;
    if (!sparse_to_dense_map) return fail(EP_INVALID_ARGUMENT, "sparse_to_dense_map is required");
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (grad_recv_x) {
        st = from_hip(ep::launch_combine_ranked(px, src_rows, sparse_to_dense_map, num_tokens,
                                                hidden, num_ranks, grad_x, s),
                      "ep_dispatch_ranked_backward launch (tokens)");
        if (st) return st;
    }
    if (grad_recv_weights)
        return from_hip(ep::launch_ranked_weight_grad(pw, src_rows, topk_idx, sparse_to_dense_map,
                                                      num_tokens, num_topk, num_experts, num_ranks,
                                                      grad_topk_weights, s),
                        "ep_dispatch_ranked_backward launch (weights)");
    return EP_SUCCESS;
}

// ---- router, row movement, 4-bit products

static size_t dtype_bytes(int dtype) { return dtype == EP_FP32 ? 4 : 2; }
static bool off_by(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

static ep_status_t check_dtype(int dtype, bool fp32)
{
    if (dtype == EP_BF16 || dtype == EP_FP16 || (fp32 && dtype == EP_FP32)) return EP_SUCCESS;
    return fail(EP_INVALID_ARGUMENT, "dtype %d must be EP_BF16%s", dtype,
                fp32 ? ", EP_FP16 or EP_FP32" : " or EP_FP16");
}

static ep_status_t check_router(int dtype, int64_t num_tokens, int num_experts, int64_t ld_logits,
                                int num_topk, int score)
{
    ep_status_t st = check_dtype(dtype, true);
    if (st) return st;
    st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts, EP_MAX_EXPERTS);
    if (ld_logits < num_experts)
        return fail(EP_INVALID_ARGUMENT, "ld_logits %lld < num_experts %d", (long long)ld_logits,
                    num_experts);
    if (score != EP_SCORE_SOFTMAX && score != EP_SCORE_SIGMOID)
        return fail(EP_INVALID_ARGUMENT, "unknown score %d", score);
    return EP_SUCCESS;
}

ep_status_t ep_router(const void* logits, int dtype, int64_t num_tokens, int num_experts,
                      int64_t ld_logits, int num_topk, int score, const float* bias,
                      int num_groups, int topk_groups, int group_top, int renormalize, float scale,
                      int64_t* topk_idx, float* topk_weights, float* probs, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_router(dtype, num_tokens, num_experts, ld_logits, num_topk, score);
    if (st) return st;
    if (num_groups < 1 || num_groups > EP_MAX_GROUPS || num_experts % num_groups != 0)
        return fail(EP_INVALID_ARGUMENT, "num_groups %d must divide num_experts %d and be at most %d",
                    num_groups, num_experts, EP_MAX_GROUPS);
    if (topk_groups < 1 || topk_groups > num_groups)
        return fail(EP_INVALID_ARGUMENT, "topk_groups %d outside [1, %d]", topk_groups, num_groups);
    if (group_top < 1 || group_top > 2)
        return fail(EP_INVALID_ARGUMENT, "group_top %d must be 1 or 2", group_top);
    if (num_topk > num_experts / num_groups * topk_groups)
        return fail(EP_INVALID_ARGUMENT, "num_topk %d exceeds the %d experts of %d groups", num_topk,
                    num_experts / num_groups * topk_groups, topk_groups);
    if (num_tokens == 0) return EP_SUCCESS;
    if (!logits || !topk_idx || !topk_weights)
        return fail(EP_INVALID_ARGUMENT, "logits, topk_idx and topk_weights are required");
    if (off_by(logits, dtype_bytes(dtype)) || off_by(bias, 4) || off_by(topk_idx, 8) ||
        off_by(topk_weights, 4) || off_by(probs, 16))
        return fail(EP_INVALID_ARGUMENT, "logits, bias, topk_idx and topk_weights must be aligned to "
                                         "their elements, probs to 16 bytes");
    const ep::RouterArgs a = {logits, num_tokens, ld_logits, num_experts, num_topk,
                              score == EP_SCORE_SOFTMAX, bias, num_groups, topk_groups, group_top,
                              renormalize != 0, scale, topk_idx, topk_weights, probs};
    return from_hip(ep::launch_router(dtype, a, static_cast<hipStream_t>(stream)), "ep_router launch");
}

ep_status_t ep_router_backward(const void* logits, int dtype, int64_t num_tokens, int num_experts,
                               int64_t ld_logits, int num_topk, int score, int renormalize,
                               float scale, const int64_t* topk_idx, const float* grad_weights,
                               const float* grad_probs, void* grad_logits, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_router(dtype, num_tokens, num_experts, ld_logits, num_topk, score);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (!logits || !topk_idx || !grad_weights || !grad_logits)
        return fail(EP_INVALID_ARGUMENT,
                    "logits, topk_idx, grad_weights and grad_logits are required");
    if (off_by(logits, dtype_bytes(dtype)) || off_by(topk_idx, 8) || off_by(grad_weights, 4) ||
        off_by(grad_probs, 4) || off_by(grad_logits, dtype_bytes(dtype)))
        return fail(EP_INVALID_ARGUMENT, "every argument must be aligned to its element");
    const ep::RouterBackwardArgs a = {logits, num_tokens, ld_logits, num_experts, num_topk,
                                      score == EP_SCORE_SOFTMAX, renormalize != 0, scale, topk_idx,
                                      grad_weights, grad_probs, grad_logits};
    return from_hip(ep::launch_router_backward(dtype, a, static_cast<hipStream_t>(stream)),
                    "ep_router_backward launch");
}

static ep_status_t check_rows(int dtype, int64_t num_tokens, int hidden, int num_topk,
                              int64_t num_rows)
{
    ep_status_t st = check_dtype(dtype, true);
    if (st) return st;
    st = check_tokens(num_tokens, num_topk);
    if (st) return st;
    st = check_hidden(hidden, 1);
    if (st) return st;
    if (num_rows < 0 || num_rows >= ((int64_t)1 << 31))
        return fail(EP_INVALID_ARGUMENT, "num_rows %lld outside [0, 2^31)", (long long)num_rows);
    if (ep::move_rows_max_blocks(dtype, num_tokens, hidden, num_topk) > INT32_MAX)
        return fail(EP_UNSUPPORTED, "num_tokens * hidden needs more than 2^31 workgroups");
    return EP_SUCCESS;
}

static ep_status_t check_matrix(const void* p, int64_t ld, int hidden, int dtype, const char* name)
{
    if (!p) return fail(EP_INVALID_ARGUMENT, "%s is required", name);
    if (off_by(p, dtype_bytes(dtype)))
        return fail(EP_INVALID_ARGUMENT, "%s must be aligned to its element", name);
    if (ld < hidden)
        return fail(EP_INVALID_ARGUMENT, "the row stride %lld of %s is below hidden %d", (long long)ld,
                    name, hidden);
    return EP_SUCCESS;
}

static ep_status_t check_pairs(const int32_t* slot, const float* w, const float* grad_w)
{
    if (!slot) return fail(EP_INVALID_ARGUMENT, "slot is required");
    if (off_by(slot, 4) || off_by(w, 4) || off_by(grad_w, 4))
        return fail(EP_INVALID_ARGUMENT, "slot, topk_weights and grad_weights must be 4-byte aligned");
    return EP_SUCCESS;
}

static ep_status_t check_clear(const int32_t* counts, const int32_t* offsets, int num_experts)
{
    if ((counts != nullptr) != (offsets != nullptr))
        return fail(EP_INVALID_ARGUMENT, "counts and offsets go together");
    if (counts == nullptr) return EP_SUCCESS;
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts, EP_MAX_EXPERTS);
    if (off_by(counts, 4) || off_by(offsets, 4))
        return fail(EP_INVALID_ARGUMENT, "counts and offsets must be 4-byte aligned");
    return EP_SUCCESS;
}

ep_status_t ep_permute(const void* x, int dtype, int64_t num_tokens, int hidden, int64_t ld_x,
                       int num_topk, const int32_t* slot, const float* topk_weights, void* rows,
                       int64_t ld_rows, int64_t num_rows, const int32_t* counts,
                       const int32_t* offsets, int num_experts, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_rows(dtype, num_tokens, hidden, num_topk, num_rows);
    if (st) return st;
    st = check_clear(counts, offsets, num_experts);
    if (st) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (num_rows > 0) {
        st = check_matrix(rows, ld_rows, hidden, dtype, "rows");
        if (st) return st;
    }
    if (num_tokens > 0) {
        st = check_matrix(x, ld_x, hidden, dtype, "x");
        if (st) return st;
        st = check_pairs(slot, topk_weights, nullptr);
        if (st) return st;
    }
    if (num_rows == 0) return EP_SUCCESS;
    if (counts) {
        st = from_hip(ep::launch_clear_rows(dtype, counts, offsets, num_experts, rows, ld_rows,
                                            num_rows, hidden, s),
                      "ep_permute launch (clear)");
        if (st) return st;
    }
    const ep::MoveArgs a = {false, x, ld_x, nullptr, 0, rows, ld_rows, num_tokens, num_rows, hidden,
                            num_topk, slot, topk_weights, nullptr};
    return from_hip(ep::launch_move_rows(dtype, a, s), "ep_permute launch");
}

ep_status_t ep_permute_backward(const void* grad_rows, int dtype, int64_t num_tokens, int hidden,
                                int64_t ld_grad_rows, int64_t num_rows, int num_topk,
                                const int32_t* slot, const float* topk_weights, const void* x,
                                int64_t ld_x, void* grad_x, int64_t ld_grad_x, float* grad_weights,
                                void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_rows(dtype, num_tokens, hidden, num_topk, num_rows);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (num_rows > 0) {
        st = check_matrix(grad_rows, ld_grad_rows, hidden, dtype, "grad_rows");
        if (st) return st;
    }
    st = check_matrix(grad_x, ld_grad_x, hidden, dtype, "grad_x");
    if (st) return st;
    st = check_pairs(slot, topk_weights, grad_weights);
    if (st) return st;
    if (grad_weights) {
        st = check_matrix(x, ld_x, hidden, dtype, "x (with grad_weights)");
        if (st) return st;
    }
    const ep::MoveArgs a = {true, grad_weights ? x : nullptr, grad_weights ? ld_x : 0,
                            num_rows > 0 ? grad_rows : nullptr, num_rows > 0 ? ld_grad_rows : 0,
                            grad_x, ld_grad_x, num_tokens, num_rows, hidden, num_topk, slot,
                            topk_weights, grad_weights};
    return from_hip(ep::launch_move_rows(dtype, a, static_cast<hipStream_t>(stream)),
                    "ep_permute_backward launch");
}

ep_status_t ep_unpermute(const void* rows, int dtype, int64_t num_tokens, int hidden,
                         int64_t ld_rows, int64_t num_rows, int num_topk, const int32_t* slot,
                         const float* topk_weights, void* out, int64_t ld_out, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_rows(dtype, num_tokens, hidden, num_topk, num_rows);
    if (st) return st;
    if (num_tokens == 0) return EP_SUCCESS;
    if (num_rows > 0) {
        st = check_matrix(rows, ld_rows, hidden, dtype, "rows");
        if (st) return st;
    }
    st = check_matrix(out, ld_out, hidden, dtype, "out");
    if (st) return st;
    st = check_pairs(slot, topk_weights, nullptr);
    if (st) return st;
    const ep::MoveArgs a = {true, nullptr, 0, num_rows > 0 ? rows : nullptr,
                            num_rows > 0 ? ld_rows : 0, out, ld_out, num_tokens, num_rows, hidden,
                            num_topk, slot, topk_weights, nullptr};
    return from_hip(ep::launch_move_rows(dtype, a, static_cast<hipStream_t>(stream)),
                    "ep_unpermute launch");
}

ep_status_t ep_unpermute_backward(const void* grad_out, int dtype, int64_t num_tokens, int hidden,
                                  int64_t ld_grad_out, int num_topk, const int32_t* slot,
                                  const float* topk_weights, const void* rows, int64_t ld_rows,
                                  void* grad_rows, int64_t ld_grad_rows, int64_t num_rows,
                                  float* grad_weights, const int32_t* counts,
                                  const int32_t* offsets, int num_experts, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_rows(dtype, num_tokens, hidden, num_topk, num_rows);
    if (st) return st;
    st = check_clear(counts, offsets, num_experts);
    if (st) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (num_rows > 0) {
        st = check_matrix(grad_rows, ld_grad_rows, hidden, dtype, "grad_rows");
        if (st) return st;
        if (grad_weights) {
            st = check_matrix(rows, ld_rows, hidden, dtype, "rows (with grad_weights)");
            if (st) return st;
        }
    }
    if (num_tokens > 0) {
        st = check_matrix(grad_out, ld_grad_out, hidden, dtype, "grad_out");
        if (st) return st;
        st = check_pairs(slot, topk_weights, grad_weights);
        if (st) return st;
    }
    if (counts && num_rows > 0) {
        st = from_hip(ep::launch_clear_rows(dtype, counts, offsets, num_experts, grad_rows,
                                            ld_grad_rows, num_rows, hidden, s),
                      "ep_unpermute_backward launch (clear)");
        if (st) return st;
    }
    const bool dots = grad_weights != nullptr && num_rows > 0;
    const ep::MoveArgs a = {false, grad_out, ld_grad_out, dots ? rows : nullptr, dots ? ld_rows : 0,
                            num_rows > 0 ? grad_rows : nullptr, num_rows > 0 ? ld_grad_rows : 0,
                            num_tokens, num_rows, hidden, num_topk, slot, topk_weights, grad_weights};
    return from_hip(ep::launch_move_rows(dtype, a, s), "ep_unpermute_backward launch");
}

static ep_status_t check_w4(int num_experts, int out_features, int in_features, int group_size,
                            int gated)
{
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts, EP_MAX_EXPERTS);
    if (out_features < 1 || out_features > EP_MAX_W4_ROWS || (gated && out_features % 2 != 0))
        return fail(EP_INVALID_ARGUMENT, "out_features %d outside [1, %d], or odd and gated",
                    out_features, EP_MAX_W4_ROWS);
    if (in_features < 32 || in_features > EP_MAX_HIDDEN || in_features % 32 != 0)
        return fail(EP_INVALID_ARGUMENT, "in_features %d must be a positive multiple of 32, at most %d",
                    in_features, EP_MAX_HIDDEN);
    if (group_size != 32 && group_size != 64 && (group_size < 128 || group_size % 128 != 0))
        return fail(EP_INVALID_ARGUMENT, "group_size %d must be 32, 64 or a multiple of 128",
                    group_size);
    return EP_SUCCESS;
}

size_t ep_w4_packed_size(int num_experts, int out_features, int in_features, int group_size,
                         int has_zeros, int gated)
{
    if (check_w4(num_experts, out_features, in_features, group_size, gated)) {
        g_last_error[0] = '\0';
        return 0;
    }
    return (size_t)ep::w4_shape(num_experts, out_features, in_features, group_size, has_zeros != 0,
                                gated != 0).bytes;
}

ep_status_t ep_w4_pack(const void* codes, const void* scales, const void* zeros, int dtype,
                       int num_experts, int out_features, int in_features, int group_size,
                       int gated, void* packed, size_t packed_bytes, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_dtype(dtype, false);
    if (st) return st;
    st = check_w4(num_experts, out_features, in_features, group_size, gated);
    if (st) return st;
    if (!codes || !scales || !packed)
        return fail(EP_INVALID_ARGUMENT, "codes, scales and packed are required");
    if (off_by(scales, 2) || off_by(packed, 256))
        return fail(EP_INVALID_ARGUMENT, "scales must be 2-byte, packed 256-byte aligned");
    const size_t need = ep_w4_packed_size(num_experts, out_features, in_features, group_size,
                                          zeros != nullptr, gated);
    if (packed_bytes < need)
        return fail(EP_INVALID_ARGUMENT, "packed holds %zu bytes, needs %zu", packed_bytes, need);
    if (need / 16 / 256 > (size_t)INT32_MAX)
        return fail(EP_UNSUPPORTED, "the weights need more than 2^31 workgroups");
    return from_hip(ep::launch_w4_pack(dtype, static_cast<const uint8_t*>(codes), scales,
                                       static_cast<const uint8_t*>(zeros), num_experts, out_features,
                                       in_features, group_size, gated != 0, packed,
                                       static_cast<hipStream_t>(stream)),
                    "ep_w4_pack launch");
}

ep_status_t ep_expert_matmul_w4(const void* x, int dtype, int64_t ld_x, int64_t num_x_rows,
                                const int32_t* src, const void* packed, size_t packed_bytes,
                                int num_experts, int out_features, int in_features, int group_size,
                                int has_zeros, int gated, const int32_t* offsets,
                                const int32_t* counts, int64_t num_rows, void* out, int64_t ld_out,
                                void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_dtype(dtype, false);
    if (st) return st;
    st = check_w4(num_experts, out_features, in_features, group_size, gated);
    if (st) return st;
    if (num_rows < 0 || num_rows >= ((int64_t)1 << 31))
        return fail(EP_INVALID_ARGUMENT, "num_rows %lld outside [0, 2^31)", (long long)num_rows);
    if (!offsets && (num_experts != 1 || counts))
        return fail(EP_INVALID_ARGUMENT, "offsets is required with more than one expert or counts");
    if (num_rows == 0) return EP_SUCCESS;
    st = check_matrix(x, ld_x, in_features, dtype, "x");
    if (st) return st;
    st = check_matrix(out, ld_out, gated ? out_features / 2 : out_features, dtype, "out");
    if (st) return st;
    if (num_x_rows < 1 || (!src && num_x_rows < num_rows))
        return fail(EP_INVALID_ARGUMENT, "x has %lld rows for %lld rows of the product",
                    (long long)num_x_rows, (long long)num_rows);
    if (!packed || off_by(packed, 256))
        return fail(EP_INVALID_ARGUMENT, "packed must be non-NULL and 256-byte aligned");
    if (off_by(src, 4) || off_by(offsets, 4) || off_by(counts, 4))
        return fail(EP_INVALID_ARGUMENT, "src, offsets and counts must be 4-byte aligned");
    const size_t need = ep_w4_packed_size(num_experts, out_features, in_features, group_size,
                                          has_zeros, gated);
    if (packed_bytes < need)
        return fail(EP_INVALID_ARGUMENT, "packed holds %zu bytes, needs %zu", packed_bytes, need);
    const ep::W4Args a = {x, ld_x, num_x_rows, src, packed, num_experts, out_features, in_features,
                          group_size, has_zeros != 0, gated != 0, offsets, counts, num_rows, out,
                          ld_out};
    if (ep::w4_max_blocks(a) > INT32_MAX)
        return fail(EP_UNSUPPORTED, "the product needs more than 2^31 workgroups");
    return from_hip(ep::launch_w4(dtype, a, static_cast<hipStream_t>(stream)),
                    "ep_expert_matmul_w4 launch");
}

// What the experts' products share: the shape and the rows.
static ep_status_t check_expert(int num_experts, int out_features, int in_features, bool gated,
                                const int32_t* offsets, const int32_t* counts, int64_t num_rows)
{
    if (num_experts < 1 || num_experts > EP_MAX_EXPERTS)
        return fail(EP_INVALID_ARGUMENT, "num_experts %d outside [1, %d]", num_experts, EP_MAX_EXPERTS);
    if (out_features < 1 || out_features > EP_MAX_OUT_FEATURES || (gated && out_features % 2 != 0))
        return fail(EP_INVALID_ARGUMENT, "out_features %d outside [1, %d], or odd and gated",
                    out_features, EP_MAX_OUT_FEATURES);
    if (in_features < 1 || in_features > EP_MAX_HIDDEN)
        return fail(EP_INVALID_ARGUMENT, "in_features %d outside [1, %d]", in_features, EP_MAX_HIDDEN);
    if (num_rows < 0 || num_rows >= ((int64_t)1 << 31))
        return fail(EP_INVALID_ARGUMENT, "num_rows %lld outside [0, 2^31)", (long long)num_rows);
    if (!offsets && (num_experts != 1 || counts))
        return fail(EP_INVALID_ARGUMENT, "offsets is required with more than one expert or counts");
    if (off_by(offsets, 4) || off_by(counts, 4))
        return fail(EP_INVALID_ARGUMENT, "offsets and counts must be 4-byte aligned");
    return EP_SUCCESS;
}

static ep_status_t check_rows_of(const void* x, int64_t ld_x, int64_t num_x_rows, const int32_t* src,
                                 int in_features, int dtype, int64_t num_rows)
{
    const ep_status_t st = check_matrix(x, ld_x, in_features, dtype, "x");
    if (st) return st;
    if (num_x_rows < 1 || (!src && num_x_rows < num_rows))
        return fail(EP_INVALID_ARGUMENT, "x has %lld rows for %lld rows of the product",
                    (long long)num_x_rows, (long long)num_rows);
    if (off_by(src, 4)) return fail(EP_INVALID_ARGUMENT, "src must be 4-byte aligned");
    return EP_SUCCESS;
}

static ep_status_t expert_forward(const void* x, int dtype, int64_t ld_x, int64_t num_x_rows,
                                  const int32_t* src, const void* weights, int num_experts,
                                  int out_features, int in_features, bool gated,
                                  const int32_t* offsets, const int32_t* counts, int64_t num_rows,
                                  void* out, int64_t ld_out, void* pre, int64_t ld_pre, void* stream,
                                  const char* what)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_dtype(dtype, false);
    if (st) return st;
    st = check_expert(num_experts, out_features, in_features, gated, offsets, counts, num_rows);
    if (st) return st;
    if (num_rows == 0) return EP_SUCCESS;
    st = check_rows_of(x, ld_x, num_x_rows, src, in_features, dtype, num_rows);
    if (st) return st;
    st = check_matrix(weights, in_features, in_features, dtype, "weights");
    if (st) return st;
    st = check_matrix(out, ld_out, gated ? out_features / 2 : out_features, dtype, "out");
    if (st) return st;
    if (pre) {
        st = check_matrix(pre, ld_pre, out_features, dtype, "pre");
        if (st) return st;
    }
    const ep::ExpertArgs a = {x, ld_x, num_x_rows, src, weights, num_experts, out_features, in_features,
                              offsets, counts, num_rows, gated, out, ld_out, pre, ld_pre};
    if (ep::expert_max_blocks(a) > INT32_MAX)
        return fail(EP_UNSUPPORTED, "the product needs more than 2^31 workgroups");
    return from_hip(ep::launch_expert(dtype, a, static_cast<hipStream_t>(stream)), what);
}

ep_status_t ep_expert_matmul(const void* x, int dtype, int64_t ld_x, int64_t num_x_rows,
                             const int32_t* src, const void* weights, int num_experts,
                             int out_features, int in_features, const int32_t* offsets,
                             const int32_t* counts, int64_t num_rows, void* out, int64_t ld_out,
                             void* stream)
{
    return expert_forward(x, dtype, ld_x, num_x_rows, src, weights, num_experts, out_features,
                          in_features, false, offsets, counts, num_rows, out, ld_out, nullptr, 0,
                          stream, "ep_expert_matmul launch");
}

ep_status_t ep_expert_glu(const void* x, int dtype, int64_t ld_x, int64_t num_x_rows,
                          const int32_t* src, const void* weights, int num_experts,
                          int out_features, int in_features, const int32_t* offsets,
                          const int32_t* counts, int64_t num_rows, void* out, int64_t ld_out,
                          void* pre, int64_t ld_pre, void* stream)
{
    return expert_forward(x, dtype, ld_x, num_x_rows, src, weights, num_experts, out_features,
                          in_features, true, offsets, counts, num_rows, out, ld_out, pre, ld_pre,
                          stream, "ep_expert_glu launch");
}

// Row stride of rows in the backward's workspace: whole 16-byte vectors.
static int64_t expert_workspace_ld(int features) { return ((int64_t)features + 7) / 8 * 8; }

// The workspace holds the gradient of the product's outputs where it is made
// (gated) or laid out, and behind it the rows of x where these are laid out.
static bool lays_out_grad(int out_features, bool gated) { return gated || out_features % 8 != 0; }
static bool lays_out_x(int in_features, bool gathered) { return gathered || in_features % 8 != 0; }

size_t ep_expert_backward_workspace_size(int64_t num_rows, int out_features, int in_features, int gated,
                                         int gathered)
{
    if (num_rows < 0 || num_rows >= ((int64_t)1 << 31) || out_features < 1 ||
        out_features > EP_MAX_OUT_FEATURES || (gated && out_features % 2 != 0) || in_features < 1 ||
        in_features > EP_MAX_HIDDEN)
        return 0;
    const size_t grad = lays_out_grad(out_features, gated != 0) ? (size_t)expert_workspace_ld(out_features) : 0;
    const size_t x = lays_out_x(in_features, gathered != 0) ? (size_t)expert_workspace_ld(in_features) : 0;
    return (size_t)num_rows * (grad + x) * 2;
}

static ep_status_t expert_backward(const void* grad_out, int dtype, int64_t ld_grad_out,
                                   const void* pre, int64_t ld_pre, const void* x, int64_t ld_x,
                                   int64_t num_x_rows, const int32_t* src, const void* weights,
                                   int num_experts, int out_features, int in_features, bool gated,
                                   const int32_t* offsets, const int32_t* counts, int64_t num_rows,
                                   void* grad_rows, int64_t ld_grad_rows, void* grad_weights,
                                   int grad_weights_dtype, void* workspace, size_t workspace_bytes,
                                   void* stream, const char* what)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_dtype(dtype, false);
    if (st) return st;
    st = check_expert(num_experts, out_features, in_features, gated, offsets, counts, num_rows);
    if (st) return st;
    if (!grad_rows && !grad_weights)
        return fail(EP_INVALID_ARGUMENT, "one of grad_rows and grad_weights is required");
    if (grad_weights) {
        if (grad_weights_dtype != dtype && grad_weights_dtype != EP_FP32)
            return fail(EP_INVALID_ARGUMENT, "grad_weights_dtype %d must be dtype %d or EP_FP32",
                        grad_weights_dtype, dtype);
        if (off_by(grad_weights, dtype_bytes(grad_weights_dtype)))
            return fail(EP_INVALID_ARGUMENT, "grad_weights must be aligned to its element");
    }
    if (num_rows == 0 && !grad_weights) return EP_SUCCESS;
    if (num_rows > 0) {
        st = check_matrix(grad_out, ld_grad_out, gated ? out_features / 2 : out_features, dtype, "grad_out");
        if (st) return st;
        if (grad_weights) {
            st = check_rows_of(x, ld_x, num_x_rows, src, in_features, dtype, num_rows);
            if (st) return st;
        }
        if (grad_rows) {
            st = check_matrix(weights, in_features, in_features, dtype, "weights");
            if (st) return st;
            st = check_matrix(grad_rows, ld_grad_rows, in_features, dtype, "grad_rows");
            if (st) return st;
        }
        if (gated) {
            st = check_matrix(pre, ld_pre, out_features, dtype, "pre");
            if (st) return st;
        }
        // without grad_weights x is not read, so not laid out either
        const size_t need = ep_expert_backward_workspace_size(num_rows, out_features, grad_weights ? in_features : 8,
                                                              gated, grad_weights && src);
        if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need))
            return fail(EP_INVALID_ARGUMENT,
                        "workspace must be 16-byte aligned and hold %zu bytes, holds %zu", need,
                        workspace ? workspace_bytes : (size_t)0);
    }
    ep::ExpertBackwardArgs a = {grad_out, ld_grad_out, false, x, ld_x, num_x_rows, src, false, weights,
                                num_experts, out_features, in_features, offsets, counts, num_rows,
                                grad_rows, ld_grad_rows, grad_weights, grad_weights_dtype == EP_FP32,
                                nullptr, nullptr};
    char* const work = static_cast<char*>(workspace);
    const bool grad_there = lays_out_grad(out_features, gated);
    if (num_rows > 0 && grad_there && !gated) a.grad_copy = work;
    if (num_rows > 0 && grad_weights && lays_out_x(in_features, src != nullptr))
        a.x_copy = work + (grad_there ? num_rows * expert_workspace_ld(out_features) * 2 : 0);
    // counted as the other calls' rows are: 16-byte vectors, 256 a workgroup
    if (num_rows * (expert_workspace_ld(out_features > in_features ? out_features : in_features) / 8) / 256 >=
        INT32_MAX)
        return fail(EP_UNSUPPORTED, "the gradients need more than 2^31 workgroups");
    if (gated) {
        a.grad = workspace;
        a.ld_grad = expert_workspace_ld(out_features);
        a.padded = true;
        const ep::GluBackwardArgs g = {grad_out, ld_grad_out, pre, ld_pre, num_rows, out_features,
                                       workspace, a.ld_grad};
        st = from_hip(ep::launch_glu_backward(dtype, g, static_cast<hipStream_t>(stream)), what);
        if (st) return st;
    }
    return from_hip(ep::launch_expert_backward(dtype, a, static_cast<hipStream_t>(stream)), what);
}

ep_status_t ep_expert_matmul_backward(const void* grad_out, int dtype, int64_t ld_grad_out,
                                      const void* x, int64_t ld_x, int64_t num_x_rows,
                                      const int32_t* src, const void* weights, int num_experts,
                                      int out_features, int in_features, const int32_t* offsets,
                                      const int32_t* counts, int64_t num_rows, void* grad_rows,
                                      int64_t ld_grad_rows, void* grad_weights,
                                      int grad_weights_dtype, void* workspace, size_t workspace_bytes,
                                      void* stream)
{
    return expert_backward(grad_out, dtype, ld_grad_out, nullptr, 0, x, ld_x, num_x_rows, src, weights,
                           num_experts, out_features, in_features, false, offsets, counts, num_rows,
                           grad_rows, ld_grad_rows, grad_weights, grad_weights_dtype, workspace,
                           workspace_bytes, stream, "ep_expert_matmul_backward launch");
}

ep_status_t ep_expert_glu_backward(const void* grad_out, int dtype, int64_t ld_grad_out,
                                   const void* pre, int64_t ld_pre, const void* x, int64_t ld_x,
                                   int64_t num_x_rows, const int32_t* src, const void* weights,
                                   int num_experts, int out_features, int in_features,
                                   const int32_t* offsets, const int32_t* counts, int64_t num_rows,
                                   void* grad_rows, int64_t ld_grad_rows, void* grad_weights,
                                   int grad_weights_dtype, void* workspace, size_t workspace_bytes,
                                   void* stream)
{
    return expert_backward(grad_out, dtype, ld_grad_out, pre, ld_pre, x, ld_x, num_x_rows, src, weights,
                           num_experts, out_features, in_features, true, offsets, counts, num_rows,
                           grad_rows, ld_grad_rows, grad_weights, grad_weights_dtype, workspace,
                           workspace_bytes, stream, "ep_expert_glu_backward launch");
}

ep_status_t ep_expert_matmul_fp8(const void* x, int x_format, int64_t ld_x, int64_t num_x_rows,
                                 const void* x_scales, int scale_format, int64_t scale_row_stride,
                                 int64_t scale_block_stride, const int32_t* src,
                                 const void* weights, const float* weight_scales, int num_experts,
                                 int out_features, int in_features, int gated,
                                 const int32_t* offsets, const int32_t* counts, int64_t num_rows,
                                 void* out, int out_dtype, int64_t ld_out, void* stream)
{
    g_last_error[0] = '\0';
    ep_status_t st = check_dtype(out_dtype, false);
    if (st) return st;
    if (x_format != EP_OUT_FP8_E4M3 && x_format != EP_OUT_FP8_E5M2)
        return fail(EP_INVALID_ARGUMENT, "x_format %d must be EP_OUT_FP8_E4M3 or EP_OUT_FP8_E5M2", x_format);
    if (scale_format != EP_SCALE_FP32 && scale_format != EP_SCALE_FP32_POW2 && scale_format != EP_SCALE_UE8M0)
        return fail(EP_INVALID_ARGUMENT, "unknown scale_format %d", scale_format);
    st = check_expert(num_experts, out_features, in_features, gated != 0, offsets, counts, num_rows);
    if (st) return st;
    if (in_features % 16 != 0)
        return fail(EP_INVALID_ARGUMENT, "in_features %d must be a multiple of 16", in_features);
    if (num_rows == 0) return EP_SUCCESS;
    if (!x || !aligned16(x) || ld_x < in_features || ld_x % 16 != 0)
        return fail(EP_INVALID_ARGUMENT, "x must be 16-byte aligned, its row stride %lld a multiple of 16 "
                                         "and at least in_features %d", (long long)ld_x, in_features);
    if (num_x_rows < 1 || (!src && num_x_rows < num_rows))
        return fail(EP_INVALID_ARGUMENT, "x has %lld rows for %lld rows of the product",
                    (long long)num_x_rows, (long long)num_rows);
    if (!weights || !aligned16(weights))
        return fail(EP_INVALID_ARGUMENT, "weights must be non-NULL and 16-byte aligned");
    if (!x_scales || !weight_scales || off_by(weight_scales, 4) || off_by(src, 4) ||
        (scale_format != EP_SCALE_UE8M0 && off_by(x_scales, 4)))
        return fail(EP_INVALID_ARGUMENT, "x_scales and weight_scales are required, and they and src must be "
                                         "aligned to their elements");
    if (scale_row_stride < 0 || scale_block_stride < 0)
        return fail(EP_INVALID_ARGUMENT, "the scales' strides must not be negative");
    st = check_matrix(out, ld_out, gated ? out_features / 2 : out_features, out_dtype, "out");
    if (st) return st;
    const ep::ExpertFp8Args a = {x, ld_x, num_x_rows, src, x_format == EP_OUT_FP8_E5M2 ? 1 : 0, x_scales,
                                 scale_format == EP_SCALE_UE8M0, scale_row_stride, scale_block_stride,
                                 weights, weight_scales, num_experts, out_features, in_features,
                                 offsets, counts, num_rows, gated != 0, out, ld_out};
    if (!ep::expert_fp8_fits(a))
        return fail(EP_UNSUPPORTED, "the product needs more workgroups or threads than a launch can have");
    return from_hip(ep::launch_expert_fp8(out_dtype, a, static_cast<hipStream_t>(stream)),
                    "ep_expert_matmul_fp8 launch");
}

}  // extern "C"

// ep_permute.hip -- token rows sorted by expert and back, in bf16, fp16 or
// fp32, of any width and row stride, with weights on either way, and the
// gradients.
//
//   permute             rows[slot[t,j]] = w[t,j] * x[t]
//   its backward        grad_x[t] = sum_j w[t,j] * g[slot[t,j]]
//                       grad_w[t,j] = <x[t], g[slot[t,j]]>
//   unpermute           out[t] = sum_j w[t,j] * y[slot[t,j]]
//   its backward        grad_y[slot[t,j]] = w[t,j] * g[t]
//                       grad_w[t,j] = <g[t], y[slot[t,j]]>
//
// So there are two movements, scatter and gather, each with or without the
// dot products; unit weights without w.  A slot of -1 (or one past the rows
// given) is no row: it is neither read nor written, adds nothing, and its
// weight gradient is 0.
//
// Products and sums are in fp32, the sum in increasing j by fused
// multiply-adds from +0; a result is rounded once to the rows' type (a
// weighted row: the fp32 product, then the type, at most half a step plus
// 2^-24 of the value).  grad_w is an fp32 dot product in a fixed order.
//
// All of it is bound by memory, so every row is read once and written once,
// 16 bytes a lane.  Measured on MI355X, 8192 tokens of 4096 bf16, k 8: permute
// 111 us (5.4 TB/s), unpermute 103 (5.9), permute backward with weight
// gradients 110 (6.1), unpermute backward 217 (5.3).  The movements without dot products take one 2 KiB (or
// 1 KiB) tile of one token's row per workgroup, which keeps many short
// independent streams in flight; with dot products a workgroup owns the
// token, so that the sum over the row's width is joined inside it, in a
// fixed order and without atomics.
//
// FAST: every row starts on 16 bytes and is a whole number of vectors, and
// accesses go through buffer resources (past the row's end, and in a masked
// row, a load gives zeros, without a branch).  Otherwise vectors are loaded
// and stored at whatever element the row starts on, and the last vector is
// moved back to end with the row.

#include "ep_device.h"
#include "ep_internal.h"
#include "ep_layer.h"
#include "ep_types.h"

namespace ep {
namespace {

template <typename T>
using UVec = typename Unaligned16<T>::type;

// Where vector v of a row of H elements starts: the last one is moved back to
// end with the row (its first elements are another vector's too, with the
// same values).  Rows shorter than a vector have one, taken by elements.
template <typename T, bool FAST>
__device__ __forceinline__ int vec_start(int H, int v)
{
    const int e = v * kVec<T>;
    return FAST || e + kVec<T> <= H ? e : H - kVec<T>;
}

// Vector v of a row of H elements; `here` false reads nothing.
template <typename T, bool FAST, int cpol>
__device__ __forceinline__ uint4 load_vec(const T* row, bool here, int H, int v)
{
    constexpr int EV = kVec<T>;
    if constexpr (FAST) {
        return load_row16<cpol>(buffer_rsrc(row, here ? H * (int)sizeof(T) : 0), v * 16);
    } else {
        uint4 d = make_uint4(0u, 0u, 0u, 0u);
        if (!here || v * EV >= H) return d;
        if (H >= EV) {
            const UVec<T>* p = reinterpret_cast<const UVec<T>*>(row + vec_start<T, FAST>(H, v));
            d = __builtin_bit_cast(uint4, (u32x4)(cpol == kCpolNT ? __builtin_nontemporal_load(p) : *p));
        } else {
            T raw[EV] = {};
#pragma unroll
            for (int c = 0; c < EV; ++c)
                if (c < H) raw[c] = row[c];
            __builtin_memcpy(&d, raw, 16);
        }
        return d;
    }
}

template <typename T, bool FAST>
__device__ __forceinline__ void store_vec(T* row, int H, int v, const uint4& d)
{
    constexpr int EV = kVec<T>;
    if (v * EV >= H) return;
    if constexpr (FAST) {
        store_row16(buffer_rsrc(row, H * (int)sizeof(T)), v * 16, d);
    } else if (H >= EV) {
        // not streaming: the lines that two vectors share are put together
        // in the L2
        *reinterpret_cast<UVec<T>*>(row + vec_start<T, FAST>(H, v)) =
            (UVec<T>)__builtin_bit_cast(u32x4, d);
    } else {
        T raw[EV];
        __builtin_memcpy(raw, &d, 16);
#pragma unroll
        for (int c = 0; c < EV; ++c)
            if (c < H) row[c] = raw[c];
    }
}

// The bits of vector v that no vector before it holds (a dot product counts
// an element once).
template <typename T, bool FAST>
__device__ __forceinline__ uint4 own_bits(int H, int v)
{
    uint32_t m[4] = {~0u, ~0u, ~0u, ~0u};
    if constexpr (!FAST) {
        const int skip = H >= kVec<T> ? (v * kVec<T> - vec_start<T, FAST>(H, v)) * (int)sizeof(T) * 8 : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = skip - 32 * i;
            m[i] = s <= 0 ? ~0u : s >= 32 ? 0u : ~0u << s;
        }
    }
    return make_uint4(m[0], m[1], m[2], m[3]);
}
__device__ __forceinline__ uint4 operator&(const uint4& a, const uint4& b)
{
    return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w);
}

template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4& d, float w)
{
    float f[kVec<T>];
    unpack<T>(d, f);
#pragma unroll
    for (int c = 0; c < kVec<T>; ++c) f[c] *= w;
    return pack<T>(f);
}

template <typename T>
__device__ __forceinline__ void add_scaled(float (&acc)[kVec<T>], const uint4& d, float w)
{
    float f[kVec<T>];
    unpack<T>(d, f);
#pragma unroll
    for (int c = 0; c < kVec<T>; ++c) acc[c] = __builtin_fmaf(w, f[c], acc[c]);
}

template <typename T>
__device__ __forceinline__ float dot_vec(const uint4& a, const uint4& b, float acc)
{
    float f[kVec<T>], g[kVec<T>];
    unpack<T>(a, f);
    unpack<T>(b, g);
#pragma unroll
    for (int c = 0; c < kVec<T>; ++c) acc = __builtin_fmaf(f[c], g[c], acc);
    return acc;
}

// Rows and weights of choices j0 .. j0 + N - 1 of token t, -1 for no row.
// t and j0 are the same in the whole workgroup, so these are scalar loads
// into scalar registers: whichever lanes are active where they are used.
template <int N>
struct Choices {
    int32_t row[N];
    float w[N];
    __device__ __forceinline__ Choices(const int32_t* __restrict__ slot,
                                       const float* __restrict__ weights, int64_t t, int j0, int k,
                                       int64_t rows)
    {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int32_t r = j0 + q < k ? slot[t * k + j0 + q] : -1;
            row[q] = r < rows ? r : -1;
            w[q] = weights == nullptr ? 1.0f : row[q] >= 0 ? weights[t * k + j0 + q] : 0.0f;
        }
    }
};

// ---- scatter: one tile of one token's row to up to kScatterSlots slots.

constexpr int kScatterSlots = 4;

template <typename T, bool FAST, int NT>
__global__ __launch_bounds__(NT)
void scatter_kernel(const T* __restrict__ x, int64_t ldx, int H, int k, int tpr, int64_t num_tiles,
                    int groups, const int32_t* __restrict__ slot, const float* __restrict__ w,
                    T* __restrict__ rows, int64_t ldr, int64_t num_rows)
{
    int64_t tile;
    int gi;
    if (!xcd_tile(blockIdx.x, groups, num_tiles, tile, gi)) return;
    const int64_t t = tile / tpr;
    const Choices<kScatterSlots> c(slot, w, t, gi * kScatterSlots, k, num_rows);
    auto one = [&](int v) {
        const uint4 d = load_vec<T, FAST, 0>(x + t * ldx, true, H, v);
#pragma unroll
        for (int q = 0; q < kScatterSlots; ++q) {
            const int32_t r = c.row[q];
            if (r >= 0) store_vec<T, FAST>(rows + r * ldr, H, v, w != nullptr ? scaled<T>(d, c.w[q]) : d);
        }
    };
    if constexpr (FAST) {
        one((int)(tile - t * tpr) * NT + (int)threadIdx.x);
    } else {
        const int nvec = (H + kVec<T> - 1) / kVec<T>;
        for (int v = (int)threadIdx.x; v < nvec; v += NT) one(v);
    }
}

// ---- gather: one tile of one token's row from its k slots.

template <typename T, bool FAST, int NT, int KB>
__global__ __launch_bounds__(NT)
void gather_kernel(const T* __restrict__ y, int64_t ldy, int H, int k, int tpr,
                   const int32_t* __restrict__ slot, const float* __restrict__ w, T* __restrict__ out,
                   int64_t ldo, int64_t num_rows)
{
    const int64_t t = blockIdx.x / tpr;
    const int v = (int)(blockIdx.x - t * tpr) * NT + (int)threadIdx.x;
    float acc[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += KB) {
        const Choices<KB> c(slot, w, t, j0, k, num_rows);
        uint4 d[KB];
#pragma unroll
        for (int q = 0; q < KB; ++q) {
            const int32_t r = c.row[q];
            d[q] = load_vec<T, FAST, kCpolNT>(y + (r >= 0 ? r * ldy : 0), r >= 0, H, v);
        }
        // no row: zeros times its weight, 0 or 1
#pragma unroll
        for (int q = 0; q < KB; ++q) add_scaled<T>(acc, d[q], c.w[q]);
    }
    store_vec<T, FAST>(out + t * ldo, H, v, pack<T>(acc));
}

// ---- with dot products: a workgroup per token; up to KB choices together.
// a is the token's row, b the rows by expert.
//   SUM      out[t] = sum w b[slot]       (k <= KB: one pass over the choices)
//   SCATTER  out[slot] = w * a[t]
//   neither  the dot products alone

enum DotMode { kDotOnly, kDotSum, kDotScatter };

template <typename T, bool FAST, int NT, int KB, int MODE>
__global__ __launch_bounds__(NT)
void dot_kernel(const T* __restrict__ a, int64_t lda, const T* __restrict__ b, int64_t ldb, int H,
                int k, const int32_t* __restrict__ slot, const float* __restrict__ w,
                T* __restrict__ out, int64_t ldo, int64_t num_rows, float* __restrict__ grad_w)
{
    __shared__ float part[NT / 64][KB];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x;
    const int nvec = (H + kVec<T> - 1) / kVec<T>;
    for (int j0 = 0; j0 < k; j0 += KB) {
        const Choices<KB> c(slot, w, t, j0, k, num_rows);
        float dots[KB];
#pragma unroll
        for (int q = 0; q < KB; ++q) dots[q] = 0.0f;
        for (int v = tid; v < nvec; v += NT) {
            const uint4 av = load_vec<T, FAST, 0>(a + t * lda, true, H, v);
            uint4 bv[KB];
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const int32_t r = c.row[q];
                bv[q] = load_vec<T, FAST, kCpolNT>(b + (r >= 0 ? r * ldb : 0), r >= 0, H, v);
            }
            float acc[kVec<T>];
#pragma unroll
            for (int i = 0; i < kVec<T>; ++i) acc[i] = 0.0f;
            const uint4 own = own_bits<T, FAST>(H, v);
            const uint4 ao = av & own;
#pragma unroll
            for (int q = 0; q < KB; ++q) {
                const int32_t r = c.row[q];
                if (r >= 0) dots[q] = dot_vec<T>(ao, bv[q] & own, dots[q]);
                if constexpr (MODE == kDotSum) add_scaled<T>(acc, bv[q], c.w[q]);
                if constexpr (MODE == kDotScatter)
                    if (r >= 0) store_vec<T, FAST>(out + r * ldo, H, v, scaled<T>(av, c.w[q]));
            }
            if constexpr (MODE == kDotSum) store_vec<T, FAST>(out + t * ldo, H, v, pack<T>(acc));
        }
#pragma unroll
        for (int q = 0; q < KB; ++q) {
#pragma unroll
            for (int s = 32; s >= 1; s >>= 1) dots[q] += __shfl_xor(dots[q], s, 64);
            if ((tid & 63) == 0) part[tid >> 6][q] = dots[q];
        }
        __syncthreads();
        if (tid < KB && j0 + tid < k) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NT / 64; ++i) s += part[i][tid];
            const int32_t r = slot[t * k + j0 + tid];
            grad_w[t * k + j0 + tid] = r >= 0 && r < num_rows ? s : 0.0f;
        }
        __syncthreads();
    }
}

// ---- rows that no choice names, cleared: the tail of each expert's segment
// past its count, and what lies past the last segment.  A workgroup looks
// kClearRows rows up (by bisection of the offsets, a row a lane) and clears
// those it finds, 16 bytes a lane.  Few rows a workgroup: where a whole
// stretch is empty, that stretch is spread over many of them (5% of 65536
// rows of 7168 bf16: 13 us on top of the permute, 44 with 64 rows a workgroup
// stored by elements; no row empty: 3.5 us).

constexpr int kClearRows = 16;

template <typename T, bool FAST>
__global__ __launch_bounds__(256)
void clear_kernel(const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets, int E,
                  T* __restrict__ rows, int64_t ldr, int64_t num_rows, int H)
{
    const int64_t r0 = (int64_t)blockIdx.x * kClearRows;
    const int lane = (int)threadIdx.x & 63;
    const int64_t r = r0 + lane;
    bool empty = false;
    if (lane < kClearRows && r < num_rows) {
        int lo = 0, hi = E;             // offsets[lo] <= r < offsets[hi], or r past them all
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (offsets[mid] <= r) lo = mid;
            else hi = mid;
        }
        empty = r >= (int64_t)offsets[lo] + counts[lo] || r < offsets[0];
    }
    uint64_t todo = __ballot(empty);
    const int nvec = (H + kVec<T> - 1) / kVec<T>;
    while (todo != 0) {
        const int b = __ffsll((unsigned long long)todo) - 1;
        todo &= todo - 1;
        for (int v = (int)threadIdx.x; v < nvec; v += 256)
            store_vec<T, FAST>(rows + (r0 + b) * ldr, H, v, make_uint4(0u, 0u, 0u, 0u));
    }
}

// 128-lane tiles, or 64-lane ones where the last 128-lane tile would be at
// most half full or the row fits 64 lanes (narrow_tiles states the figures).
bool use64(int nvec) { return nvec <= 64 || narrow_tiles(nvec); }

template <typename T, bool FAST>
hipError_t scatter_of(const MoveArgs& a, hipStream_t stream)
{
    const int nvec = (a.hidden + kVec<T> - 1) / kVec<T>;
    // A long row that is not whole vectors goes to one workgroup: its parts
    // share lines, which only meet in one XCD's L2 (bf16, 8192 tokens: 4097
    // wide, k 8: 157 us against 176 in tiles; 2047 wide, k 4: 39 against 43;
    // 1001 wide, k 2, 126 vectors: 14 us in a workgroup of 256, 10 in one of
    // 128).
    const int nt = !FAST ? (nvec <= 64 ? 64 : nvec <= 128 ? 128 : 256) : use64(nvec) ? 64 : 128;
    const int tpr = FAST ? (nvec + nt - 1) / nt : 1;
    const int groups = (a.num_topk + kScatterSlots - 1) / kScatterSlots;
    const int64_t tiles = a.num_tokens * tpr;
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8 * groups));
    auto go = [&](auto n) {
        constexpr int NT = decltype(n)::value;
        hipLaunchKernelGGL((scatter_kernel<T, FAST, NT>), grid, dim3(NT), 0, stream,
                           static_cast<const T*>(a.tokens), a.ld_tokens, a.hidden, a.num_topk, tpr,
                           tiles, groups, a.slot, a.weights, static_cast<T*>(a.out), a.ld_out,
                           a.num_rows);
        return hipGetLastError();
    };
    if (nt == 64) return go(std::integral_constant<int, 64>());
    if constexpr (!FAST)
        if (nt == 256) return go(std::integral_constant<int, 256>());
    return go(std::integral_constant<int, 128>());
}

template <typename T, bool FAST>
hipError_t gather_of(const MoveArgs& a, hipStream_t stream)
{
    const int nvec = (a.hidden + kVec<T> - 1) / kVec<T>;
    const int nt = use64(nvec) ? 64 : 128;
    const int tpr = (nvec + nt - 1) / nt;
    const dim3 grid((unsigned)(a.num_tokens * tpr));
    auto go = [&](auto n, auto kb) {
        constexpr int NT = decltype(n)::value, KB = decltype(kb)::value;
        hipLaunchKernelGGL((gather_kernel<T, FAST, NT, KB>), grid, dim3(NT), 0, stream,
                           static_cast<const T*>(a.rows), a.ld_rows, a.hidden, a.num_topk, tpr,
                           a.slot, a.weights, static_cast<T*>(a.out), a.ld_out, a.num_rows);
        return hipGetLastError();
    };
    auto with = [&](auto n) {
        if (a.num_topk <= 2) return go(n, std::integral_constant<int, 2>());
        if (a.num_topk <= 4) return go(n, std::integral_constant<int, 4>());
        return go(n, std::integral_constant<int, 8>());
    };
    return nt == 64 ? with(std::integral_constant<int, 64>()) : with(std::integral_constant<int, 128>());
}

template <typename T, bool FAST, int MODE>
hipError_t dot_of(const MoveArgs& a, hipStream_t stream)
{
    const int nvec = (a.hidden + kVec<T> - 1) / kVec<T>;
    const dim3 grid((unsigned)a.num_tokens);
    auto go = [&](auto n, auto kb) {
        constexpr int NT = decltype(n)::value, KB = decltype(kb)::value;
        hipLaunchKernelGGL((dot_kernel<T, FAST, NT, KB, MODE>), grid, dim3(NT), 0, stream,
                           static_cast<const T*>(a.tokens), a.ld_tokens,
                           static_cast<const T*>(a.rows), a.ld_rows, a.hidden, a.num_topk, a.slot,
                           a.weights, static_cast<T*>(a.out), a.ld_out, a.num_rows, a.grad_weights);
        return hipGetLastError();
    };
    auto with = [&](auto n) {
        if (a.num_topk <= 2) return go(n, std::integral_constant<int, 2>());
        if (a.num_topk <= 4) return go(n, std::integral_constant<int, 4>());
        return go(n, std::integral_constant<int, 8>());
    };
    return nvec <= 64 ? with(std::integral_constant<int, 64>()) : with(std::integral_constant<int, 256>());
}

template <typename T, bool FAST>
hipError_t move_of(const MoveArgs& a, hipStream_t stream)
{
    if (a.gather) {
        // the fused pass holds a vector of all choices at once; more than 8
        // take the sum and the dot products in two passes, which read the
        // rows twice (8192 x 4096 bf16, caches emptied: k 8 121 us, 103
        // without dot products; k 9 226, 118; k 16 372, 196; k 64 1374, 714)
        if (a.grad_weights != nullptr && a.num_topk <= 8) return dot_of<T, FAST, kDotSum>(a, stream);
        hipError_t err = gather_of<T, FAST>(a, stream);
        if (err != hipSuccess || a.grad_weights == nullptr) return err;
        return dot_of<T, FAST, kDotOnly>(a, stream);
    }
    if (a.grad_weights != nullptr) return dot_of<T, FAST, kDotScatter>(a, stream);
    return scatter_of<T, FAST>(a, stream);
}

template <typename T>
hipError_t move_typed(const MoveArgs& a, hipStream_t stream)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(a.tokens) | reinterpret_cast<uintptr_t>(a.rows) |
                         reinterpret_cast<uintptr_t>(a.out) |
                         (uintptr_t)((a.ld_tokens | a.ld_rows | a.ld_out | a.hidden) * (int64_t)sizeof(T));
    return at % 16 == 0 ? move_of<T, true>(a, stream) : move_of<T, false>(a, stream);
}

template <typename T>
hipError_t clear_typed(const int32_t* counts, const int32_t* offsets, int num_experts, void* rows,
                       int64_t ld, int64_t num_rows, int hidden, hipStream_t stream)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(rows) | (uintptr_t)((ld | hidden) * (int64_t)sizeof(T));
    const dim3 grid((unsigned)((num_rows + kClearRows - 1) / kClearRows));
    if (at % 16 == 0)
        hipLaunchKernelGGL((clear_kernel<T, true>), grid, dim3(256), 0, stream, counts, offsets,
                           num_experts, static_cast<T*>(rows), ld, num_rows, hidden);
    else
        hipLaunchKernelGGL((clear_kernel<T, false>), grid, dim3(256), 0, stream, counts, offsets,
                           num_experts, static_cast<T*>(rows), ld, num_rows, hidden);
    return hipGetLastError();
}

}  // namespace

int64_t move_rows_max_blocks(int dtype, int64_t num_tokens, int hidden, int num_topk)
{
    const int ev = dtype == 2 ? 4 : 8;
    const int nvec = (hidden + ev - 1) / ev;
    const int groups = (num_topk + kScatterSlots - 1) / kScatterSlots;
    return (num_tokens * ((nvec + 63) / 64) + 7) / 8 * 8 * groups;
}

hipError_t launch_move_rows(int dtype, const MoveArgs& a, hipStream_t stream)
{
    if (a.num_tokens == 0) return hipSuccess;
    if (dtype == 0) return move_typed<Bf16>(a, stream);
    if (dtype == 1) return move_typed<Fp16>(a, stream);
    return move_typed<float>(a, stream);
}

hipError_t launch_clear_rows(int dtype, const int32_t* counts, const int32_t* offsets,
                             int num_experts, void* rows, int64_t ld, int64_t num_rows, int hidden,
                             hipStream_t stream)
{
    if (num_rows == 0) return hipSuccess;
    if (dtype == 0) return clear_typed<Bf16>(counts, offsets, num_experts, rows, ld, num_rows, hidden, stream);
    if (dtype == 1) return clear_typed<Fp16>(counts, offsets, num_experts, rows, ld, num_rows, hidden, stream);
    return clear_typed<float>(counts, offsets, num_experts, rows, ld, num_rows, hidden, stream);
}

}  // namespace ep

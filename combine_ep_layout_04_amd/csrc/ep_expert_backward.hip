// ep_expert_backward.hip -- the gradients of the experts' products, in 16
// bits: with d[r] the gradient of out[r] = W[e] x[r],
//
//   grad_rows[r, k] = sum_n d[r, n] W[e, n, k]
//   grad_w[e, n, k] = sum_r d[r, n] x[r, k]     over the rows r of expert e
//
// and, for the gated product, d from the gradient of silu(gate) * up:
//
//   d_gate = g up s (1 + gate (1 - s)),  d_up = g gate s,  s = 1 / (1 + exp(-gate)).
//
// In the first the weights, in the second both operands lie across the
// reduction; they are transposed on the way from LDS to the registers
// (ColOperand), so nothing is transposed in memory.  Sums are fp32 in a fixed
// order, no atomics.
//
// 32768 rows of 32 experts, 7168 -> 4096 gated, bf16: 3770 us, 1.02 PFLOP/s:
// the activation's gradient 105 to 120, the rows' 1650 (matrix cores busy 78% of
// the cycles), the weights' 2130 (53%: both operands by transposing reads of 8
// bytes, and 13% for the stores, 1.9 GB of which one covers 16 bytes of a line).
#include "ep_expert.h"
#include "ep_product.h"

namespace ep {
namespace {

template <typename T>
struct RowsGrad {
    const T* grad;
    int64_t ld_grad;
    const T* w;
    int n, k;
    Segments seg;
    T* out;
    int64_t ld_out;
    TileWalk walk;
    bool turned;        // tiles begin at different steps of the reduction
};

// A tile of BP columns (k) by BQ rows; the reduction goes along n.
template <typename T, bool DIRECT, int BP, int BQ, int WP, int WQ, int RING>
__global__ __launch_bounds__(WP * WQ * 64)
void rows_grad_kernel(RowsGrad<T> a)
{
    constexpr int kThreads = WP * WQ * 64;
    constexpr int PB = BP / WP / 32, QB = BQ / WQ / 32;
    using Off = std::conditional_t<DIRECT, uint32_t, uint64_t>;
    using P = ColOperand<BP, kThreads, Off>;
    using Q = RowOperand<BQ, kThreads, Off>;
    using R = Ring<P, Q, RING>;
    __shared__ __attribute__((aligned(128))) char lds[DIRECT ? R::kLds : 2 * (P::kBytes + Q::kBytes)];

    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int p0 = wave / WQ * (PB * 32), q0 = wave % WQ * (QB * 32);

    struct Tile {
        RowBlock rb;
        int64_t k0;
    };
    int i = 0;
    auto find = [&](Tile& t) {
        int col;
        if (!next_tile(a.walk, a.seg, BQ, i, t.rb, col)) return false;
        t.k0 = (int64_t)col * BP;
        return true;
    };
    auto prepare = [&](Work<P, Q>& w, const Tile& t) {
        const int steps = (a.n + 63) / 64;
        w.p.init(reinterpret_cast<const char*>(a.w + (int64_t)t.rb.expert * a.n * a.k), (int64_t)a.k * 2, a.n, t.k0,
                 a.k);
        // DIRECT: a chunk that ends past n reads what lies behind the row,
        // where the caller keeps zeros
        w.q.init(reinterpret_cast<const char*>(a.grad + t.rb.first * a.ld_grad),
                 DIRECT ? (a.n * 2 + 15) / 16 * 16 : a.n * 2,
                 [&](int i) { return (Off)(i < t.rb.rows ? i : 0) * (Off)(a.ld_grad * 2); });
        w.steps = steps > R::kFewestSteps ? steps : R::kFewestSteps;
        w.whole = a.n / 64;
        w.turn = 0;
        if (a.turned && w.steps == steps) {
            w.turn = (int)((unsigned)(t.k0 / 32 * 5 + t.rb.expert * 3) % (unsigned)steps);
            if (w.whole < steps) w.whole = 0;
        }
    };
    auto store = [&](const f32x16_t (&acc)[PB][QB], const Tile& t) {
        const int lane = opaque(threadIdx.x) & 63;
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int r = q0 + j * 32 + (lane & 31);
            const bool live = r < t.rb.rows;
            const int64_t row = t.rb.first + (live ? r : 0);
#pragma unroll
            for (int i = 0; i < PB; ++i)
                store_block(acc[i][j], a.out + row * a.ld_out, t.k0 + p0 + i * 32, a.k, live);
        }
    };
    tiles<T, DIRECT, P, Q, PB, QB, RING, kThreads, Tile>(lds, p0, q0, find, prepare, store, (a.n + 63) / 64);
}

template <typename T>
struct WeightGrad {
    const T* grad;
    int64_t ld_grad;
    const T* x;
    int64_t ld_x;
    int n, k;
    Segments seg;
    void* out;
    int k_tiles, n_tiles;
    int64_t tiles;
};

// A tile of BP columns (k) by BQ outputs (n) of one expert; the reduction
// goes over its rows.  Experts without rows get zeros.
template <typename T, typename O, bool DIRECT, int BP, int BQ, int WP, int WQ, int RING>
__global__ __launch_bounds__(WP * WQ * 64)
void weight_grad_kernel(WeightGrad<T> a)
{
    constexpr int kThreads = WP * WQ * 64;
    constexpr int PB = BP / WP / 32, QB = BQ / WQ / 32;
    using Off = std::conditional_t<DIRECT, uint32_t, uint64_t>;
    using P = ColOperand<BP, kThreads, Off>;
    using Q = ColOperand<BQ, kThreads, Off>;
    using R = Ring<P, Q, RING>;
    __shared__ __attribute__((aligned(128))) char lds[DIRECT ? R::kLds : 2 * (P::kBytes + Q::kBytes)];

    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int p0 = wave / WQ * (PB * 32), q0 = wave % WQ * (QB * 32);

    struct Tile {
        RowBlock rb;
        int64_t k0, n0;
    };
    int i = 0;
    O* const out = static_cast<O*>(a.out);
    auto store = [&](const f32x16_t (&acc)[PB][QB], const Tile& t) {
        const int lane = opaque(threadIdx.x) & 63;
        O* to = out + (int64_t)t.rb.expert * a.n * a.k;
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int64_t n = t.n0 + q0 + j * 32 + (lane & 31);
            const bool live = n < a.n;
#pragma unroll
            for (int i = 0; i < PB; ++i)
                store_block(acc[i][j], to + (live ? n : 0) * a.k, t.k0 + p0 + i * 32, a.k, live);
        }
    };
    auto find = [&](Tile& t) {
        const int64_t at = tile_of(i++);
        if (at >= a.tiles) return false;
        const int64_t per = (int64_t)a.k_tiles * a.n_tiles;
        const int expert = (int)(at / per);
        const unsigned of = (unsigned)(at % per);
        t.n0 = (int64_t)(of / (unsigned)a.k_tiles) * BQ;
        t.k0 = (int64_t)(of % (unsigned)a.k_tiles) * BP;
        t.rb = RowBlock{expert, 0, a.seg.num_rows};
        if (a.seg.offsets != nullptr) {
            t.rb.first = uniform(a.seg.offsets[expert]);
            t.rb.rows = uniform(a.seg.counts != nullptr ? a.seg.counts[expert]
                                                        : a.seg.offsets[expert + 1] - t.rb.first);
            bound_rows(t.rb, a.seg.num_rows);
        }
        if (t.rb.rows <= 0) t.rb.rows = t.rb.first = 0;     // no rows: steps of zeros
        return true;
    };
    auto prepare = [&](Work<P, Q>& w, const Tile& t) {
        const int steps = blocks_of(t.rb.rows, 64);
        w.p.init(reinterpret_cast<const char*>(a.x + t.rb.first * a.ld_x), a.ld_x * 2, t.rb.rows, t.k0, a.k);
        w.q.init(reinterpret_cast<const char*>(a.grad + t.rb.first * a.ld_grad), a.ld_grad * 2, t.rb.rows, t.n0, a.n);
        w.steps = DIRECT && steps < R::kFewestSteps ? R::kFewestSteps : steps;
        w.whole = t.rb.rows / 64;
        w.turn = 0;
    };
    tiles<T, DIRECT, P, Q, PB, QB, RING, kThreads, Tile>(lds, p0, q0, find, prepare, store, 0);
}

// The same for experts of few rows, where the time is that of writing the
// gradients: one place in LDS for a step's operands, and as many workgroups on
// a CU as keep its memory pipeline busy instead of loads ahead.  Results leave
// through LDS, so that a store covers whole lines: rows of 128 columns, chunk c
// of row n at place c ^ (n % 16).
// us for both gradients of 64 experts, weights' in this form and through the
// ring: 128 rows an expert 507 to 610, 256 rows (1408 -> 2048) 354 to 390, 512
// rows 716 to 700.
template <typename T, typename O>
__global__ __launch_bounds__(256, 4)
void weight_grad_short_kernel(WeightGrad<T> a)
{
    constexpr int kThreads = 256, PB = 2, QB = 2;
    using P = ColOperand<128, kThreads>;
    using Q = ColOperand<128, kThreads>;
    __shared__ __attribute__((aligned(128))) char lds[P::kBytes + Q::kBytes];

    const int64_t at = tile_of(0), per = (int64_t)a.k_tiles * a.n_tiles;
    if (at >= a.tiles) return;
    const int expert = (int)(at / per);
    const unsigned of = (unsigned)(at % per);
    const int64_t n0 = (int64_t)(of / (unsigned)a.k_tiles) * 128, k0 = (int64_t)(of % (unsigned)a.k_tiles) * 128;
    RowBlock rb = {expert, 0, a.seg.num_rows};
    if (a.seg.offsets != nullptr) {
        rb.first = uniform(a.seg.offsets[expert]);
        rb.rows = uniform(a.seg.counts != nullptr ? a.seg.counts[expert] : a.seg.offsets[expert + 1] - rb.first);
        bound_rows(rb, a.seg.num_rows);
    }
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int p0 = wave / 2 * 64, q0 = wave % 2 * 64, lane = threadIdx.x & 63;
    f32x16_t acc[PB][QB];
    clear(acc);
    if (rb.rows > 0) {
        P p;
        Q q;
        p.init(reinterpret_cast<const char*>(a.x + rb.first * a.ld_x), a.ld_x * 2, rb.rows, k0, a.k);
        q.init(reinterpret_cast<const char*>(a.grad + rb.first * a.ld_grad), a.ld_grad * 2, rb.rows, n0, a.n);
        const uint32_t to = lds_address(lds) + wave * 1024;
        const int steps = blocks_of(rb.rows, 64);
        for (int s = 0; s < steps; ++s) {
            if (s > 0) wait_barrier();
            load_operand<0>(p, to, s);
            load_operand<0>(q, to + P::kBytes, s);
            wait_barrier();
            const int parts = (rb.rows - s * 64 + 15) / 16;
#pragma unroll
            for (int part = 0; part < 4; ++part) {
                if (part >= parts) break;
                uint4 pv[PB], qv[QB];
#pragma unroll
                for (int j = 0; j < QB; ++j) qv[j] = Q::part(lds + P::kBytes, q0, j, part);
#pragma unroll
                for (int i = 0; i < PB; ++i) pv[i] = P::part(lds, p0, i, part);
#pragma unroll
                for (int i = 0; i < PB; ++i)
#pragma unroll
                    for (int j = 0; j < QB; ++j)
                        acc[i][j] = mma32(pv[i], qv[j], acc[i][j], static_cast<const T*>(nullptr));
            }
        }
        wait_barrier();
    }
    O* out = static_cast<O*>(a.out) + (int64_t)expert * a.n * a.k;
    if constexpr (std::is_same_v<O, float>) {
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int64_t n = n0 + q0 + j * 32 + (lane & 31);
            const bool live = n < a.n;
#pragma unroll
            for (int i = 0; i < PB; ++i)
                store_block(acc[i][j], out + (live ? n : 0) * a.k, k0 + p0 + i * 32, a.k, live);
        }
    } else {
#pragma unroll
        for (int j = 0; j < QB; ++j)
#pragma unroll
            for (int i = 0; i < PB; ++i) {
                const int n = q0 + j * 32 + (lane & 31);
                put_block<T>(acc[i][j], [&](int c) {
                    return lds + n * 256 + ((((p0 + i * 32 + c) / 8) ^ (n & 15)) << 4);
                });
            }
        wait_barrier();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int n = i * 16 + (threadIdx.x >> 4), c = threadIdx.x & 15;
            const uint4 v = *reinterpret_cast<const uint4*>(lds + n * 256 + ((c ^ (n & 15)) << 4));
            if (n0 + n < a.n) store_chunk(v, out + (n0 + n) * a.k, k0 + c * 8, a.k);
        }
    }
}

// Workgroups of 256 for a unit per thread, in all fewer than the 2^32 threads
// that a launch can have; the threads take turns past that.
unsigned flat_grid(int64_t units)
{
    constexpr int64_t kMost = 1 << 23;
    return (unsigned)((units + 255) / 256 < kMost ? (units + 255) / 256 : kMost);
}

// Both halves' gradients, a row's units of 8 outputs per thread.  Memory
// bound: reads 3, writes 2 values an output; 32768 rows of 2048 outputs 120 us,
// 5.6 TB/s.  d is rounded to 16 bits, the type the matrix cores take: half a
// step relative to each term of the sums that follow, so that gradients of
// bf16 are off by 0.0024 (root of the mean square, relative) where one rounding
// of the result alone is 0.0017.  d in two parts of 16 bits would double the
// matrix work of both products, which is their time.
template <typename T>
__global__ __launch_bounds__(256)
void glu_backward_kernel(const T* __restrict__ grad, int64_t ld_grad, const T* __restrict__ pre, int64_t ld_pre,
                         int64_t num_rows, int half, T* __restrict__ out, int64_t ld_out, int units)
{
    auto unit = [&](int64_t row, int c) {
        const T* g = grad + row * ld_grad + c;
        const T* p = pre + row * ld_pre + c;
        T* o = out + row * ld_out + c;
        const int left = half - c;
        auto both = [](float g, float gate, float up, float& d_gate, float& d_up) {
            const float s = sigmoid_of(gate), gs = g * s;
            d_gate = gs * up * (1.0f + gate * (1.0f - s));
            d_up = gs * gate;
        };
        if (left >= 8) {
            float gv[8], gate[8], up[8], dg[8], du[8];
            unpack<T>(fetch16<T>(reinterpret_cast<const char*>(g), 8), gv);
            unpack<T>(fetch16<T>(reinterpret_cast<const char*>(p), 8), gate);
            unpack<T>(fetch16<T>(reinterpret_cast<const char*>(p + half), 8), up);
#pragma unroll
            for (int i = 0; i < 8; ++i) both(gv[i], gate[i], up[i], dg[i], du[i]);
            const uint4 a = pack<T>(dg), b = pack<T>(du);
            __builtin_memcpy(o, &a, 16);
            __builtin_memcpy(o + half, &b, 16);
        } else {
            for (int i = 0; i < 8 && i < left; ++i) {
                float dg, du;
                both(to_float(g[i]), to_float(p[i]), to_float(p[half + i]), dg, du);
                o[i] = from_float<T>(dg);
                o[half + i] = from_float<T>(du);
            }
        }
        if (c == 0)     // the row's padding
            for (int64_t i = 2 * (int64_t)half; i < ld_out; ++i) out[row * ld_out + i] = T{0};
    };
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < num_rows * units; at += stride)
        unit(at / units, (int)(at % units) * 8);
}

template <typename T, bool DIRECT, int BP, int BQ, int WP, int WQ, int RING>
hipError_t launch_rows(const ExpertBackwardArgs& a, hipStream_t stream)
{
    RowsGrad<T> p = {static_cast<const T*>(a.grad), a.ld_grad, static_cast<const T*>(a.w), a.n, a.k,
                     {a.offsets, a.counts, a.num_experts, (int)a.num_rows},
                     static_cast<T*>(a.grad_rows), a.ld_grad_rows, {}, BQ <= 128};
    p.walk.group = 8;
    p.walk.col_tiles = (a.k + BP - 1) / BP;
    p.walk.tiles = tile_count(max_row_blocks(a.num_rows, a.num_experts, BQ), p.walk.group, p.walk.col_tiles);
    hipLaunchKernelGGL((rows_grad_kernel<T, DIRECT, BP, BQ, WP, WQ, RING>),
                       dim3(tile_grid(p.walk.tiles, DIRECT ? 1 : 2)), dim3(WP * WQ * 64), 0, stream, p);
    return hipGetLastError();
}

template <typename T, typename O, bool DIRECT, int BP, int BQ, int WP, int WQ, int RING>
hipError_t launch_weights(const ExpertBackwardArgs& a, hipStream_t stream)
{
    WeightGrad<T> p = {static_cast<const T*>(a.grad), a.ld_grad, static_cast<const T*>(a.x), a.ld_x,
                       a.n, a.k, {a.offsets, a.counts, a.num_experts, (int)a.num_rows},
                       a.grad_w, (a.k + BP - 1) / BP, (a.n + BQ - 1) / BQ, 0};
    p.tiles = (int64_t)a.num_experts * p.k_tiles * p.n_tiles;
    hipLaunchKernelGGL((weight_grad_kernel<T, O, DIRECT, BP, BQ, WP, WQ, RING>),
                       dim3(tile_grid(p.tiles, DIRECT ? 1 : 2)), dim3(WP * WQ * 64), 0, stream, p);
    return hipGetLastError();
}

template <typename T, typename O>
hipError_t launch_weights_short(const ExpertBackwardArgs& a, hipStream_t stream)
{
    WeightGrad<T> p = {static_cast<const T*>(a.grad), a.ld_grad, static_cast<const T*>(a.x), a.ld_x,
                       a.n, a.k, {a.offsets, a.counts, a.num_experts, (int)a.num_rows},
                       a.grad_w, (a.k + 127) / 128, (a.n + 127) / 128, 0};
    p.tiles = (int64_t)a.num_experts * p.k_tiles * p.n_tiles;
    hipLaunchKernelGGL((weight_grad_short_kernel<T, O>), dim3((unsigned)((p.tiles + 255) / 256 * 256)), dim3(256), 0,
                       stream, p);
    return hipGetLastError();
}

// Elements of 16 bits that 32-bit offsets reach.
bool in_reach(int64_t elements) { return elements <= (int64_t)1 << 31; }
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// Rows laid out for the kernels above: gathered, and padded with zeros to
// whole 16-byte chunks.  A chunk per thread.
template <typename T>
__global__ __launch_bounds__(256)
void lay_out_kernel(const T* __restrict__ x, int64_t ld_x, int64_t x_rows, const int32_t* __restrict__ src,
                    int64_t num_rows, int cols, int chunks, uint4* __restrict__ out)
{
    const int64_t stride = (int64_t)gridDim.x * 256;
    for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < num_rows * chunks; at += stride) {
        int64_t row = at / chunks;
        const int c = (int)(at % chunks) * 8;
        if (src != nullptr) {
            row = src[row];
            if (row < 0 || row >= x_rows) row = 0;
        }
        out[at] = fetch16<T>(reinterpret_cast<const char*>(x + row * ld_x + c), cols - c);
    }
}

template <typename T>
hipError_t lay_out(const void* x, int64_t ld_x, int64_t x_rows, const int32_t* src, int64_t num_rows, int cols,
                   void* out, hipStream_t stream)
{
    const int chunks = (cols + 7) / 8;
    hipLaunchKernelGGL(lay_out_kernel<T>, dim3(flat_grid(num_rows * chunks)), dim3(256), 0, stream,
                       static_cast<const T*>(x), ld_x, x_rows, src, num_rows, cols, chunks, static_cast<uint4*>(out));
    return hipGetLastError();
}

template <typename T, typename O>
hipError_t weights_sized(const ExpertBackwardArgs& a, hipStream_t stream)
{
    const bool direct = (a.k % 8 == 0 || a.x_padded) && a.ld_x % 8 == 0 && (a.n % 8 == 0 || a.padded) &&
                        a.ld_grad % 8 == 0 && in_reach(64 * a.ld_x) && in_reach(64 * a.ld_grad) && !off16(a.x) &&
                        !off16(a.grad);
    if (!direct) return launch_weights<T, O, false, 128, 128, 2, 2, 4>(a, stream);
    // few rows an expert: the time of writing, else that of multiplying; a
    // workgroup per tile, as long as a launch can have their threads (2^32)
    const int64_t tiles = (int64_t)a.num_experts * ((a.n + 127) / 128) * ((a.k + 127) / 128);
    if (a.num_rows / a.num_experts < 400 && tiles < (1 << 24) - 256) return launch_weights_short<T, O>(a, stream);
    return launch_weights<T, O, true, 256, 256, 2, 2, 5>(a, stream);
}

template <typename T>
hipError_t backward(ExpertBackwardArgs a, hipStream_t stream)
{
    if (a.grad_copy != nullptr) {
        const hipError_t err = lay_out<T>(a.grad, a.ld_grad, a.num_rows, nullptr, a.num_rows, a.n, a.grad_copy, stream);
        if (err != hipSuccess) return err;
        a.grad = a.grad_copy;
        a.ld_grad = (a.n + 7) / 8 * 8;
        a.padded = true;
    }
    if (a.x_copy != nullptr) {
        const hipError_t err = lay_out<T>(a.x, a.ld_x, a.x_rows, a.src, a.num_rows, a.k, a.x_copy, stream);
        if (err != hipSuccess) return err;
        a.x = a.x_copy;
        a.ld_x = (a.k + 7) / 8 * 8;
        a.x_padded = true;
    }
    if (a.grad_rows != nullptr && a.num_rows > 0) {
        const bool direct = a.k % 8 == 0 && (a.n % 8 == 0 || a.padded) && a.ld_grad % 8 == 0 &&
                            in_reach(256 * a.ld_grad) && !off16(a.w) && !off16(a.grad);
        // us, 256 x 256 to 256 x 128, 64 experts 2048 -> 2048: 128 rows an expert
        // 186 to 142, 192 rows 136 to 162, 256 rows 189 to 196, 400 rows 246 to
        // 285, 1000 rows 508 to 587
        const int64_t hold = a.num_rows < a.num_experts ? a.num_rows : a.num_experts;
        const hipError_t err = !direct ? launch_rows<T, false, 128, 128, 2, 2, 4>(a, stream)
                               : a.num_rows / hold >= 192 ? launch_rows<T, true, 256, 256, 2, 2, 5>(a, stream)
                                                          : launch_rows<T, true, 256, 128, 2, 2, 5>(a, stream);
        if (err != hipSuccess) return err;
    }
    if (a.grad_w == nullptr) return hipSuccess;
    return a.wide_w ? weights_sized<T, float>(a, stream) : weights_sized<T, T>(a, stream);
}

}  // namespace

hipError_t launch_expert_backward(int dtype, const ExpertBackwardArgs& a, hipStream_t stream)
{
    return dtype == 0 ? backward<Bf16>(a, stream) : backward<Fp16>(a, stream);
}

hipError_t launch_glu_backward(int dtype, const GluBackwardArgs& a, hipStream_t stream)
{
    if (a.num_rows == 0) return hipSuccess;
    const int half = a.n / 2, units = (half + 7) / 8;
    const unsigned blocks = flat_grid(a.num_rows * units);
    if (dtype == 0)
        hipLaunchKernelGGL((glu_backward_kernel<Bf16>), dim3(blocks), dim3(256), 0, stream,
                           static_cast<const Bf16*>(a.grad), a.ld_grad, static_cast<const Bf16*>(a.pre), a.ld_pre,
                           a.num_rows, half, static_cast<Bf16*>(a.out), a.ld_out, units);
    else
        hipLaunchKernelGGL((glu_backward_kernel<Fp16>), dim3(blocks), dim3(256), 0, stream,
                           static_cast<const Fp16*>(a.grad), a.ld_grad, static_cast<const Fp16*>(a.pre), a.ld_pre,
                           a.num_rows, half, static_cast<Fp16*>(a.out), a.ld_out, units);
    return hipGetLastError();
}

}  // namespace ep

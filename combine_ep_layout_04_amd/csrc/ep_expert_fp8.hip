// ep_expert_fp8.hip -- the experts' products of rows and weights held in
// 8-bit floating point, scaled per 128 inputs:
//
//   out[r, n] = sum_b xs[r, b] ws[e, n / 128, b] sum_{k in b} cx[r, k] cw[e, n, k]
//
// with codes cx (E4M3 or E5M2), cw (E4M3), b the blocks of 128 inputs.  A
// block's sum is multiplied by both scales (their fp32 product) and added in
// fp32.  The gated form as in ep_expert.hip.
//
// Tiles (many rows an expert) take the matrix cores' 8-bit instructions, which
// are twice as fast as the 16-bit ones.  These line up each 8 products by the
// largest's exponent and drop what lies 2^-13 of it below (seen with pairs
// that cancel and a third product of falling size; products of one 8 do not
// meet those of the next before the fp32 sum): a product is off by up to
// 2^-13 of the largest of its 8, about 2^-13 of the result for K random terms
// and under a result's own rounding in bf16 (2^-9) and fp16 (2^-12).  With
// few rows the time is that of the weights' bytes, so there the codes are
// widened to bf16, exactly, and nothing is dropped.
//
// 32768 rows of 32 experts, gated 7168 -> 4096: 1175 us, 1.64 PFLOP/s; the
// matrix cores are busy 47% of the cycles, the vector units, which scale each
// block's sum (16 multiply-adds for 2 matrix instructions), 42%.  512 rows of 256 experts,
// 2048 -> 7168: 516 us, 6.2 TB/s of weights read.  One token through 8 experts,
// gated 7168 -> 4096: 44 us, 5.3 TB/s.
//
// The weights are the matrix instruction's first operand, so the 16 values a
// lane holds of a 32 x 32 block belong to one row of x: one factor for all 16.
#include "ep_expert.h"
#include "ep_product.h"

#pragma clang diagnostic ignored "-Winline-asm"     // m0 in clobber lists

namespace ep {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct Codes {
    uint4 lo, hi;
};
__device__ __forceinline__ i32x8_t bits(const Codes& c)
{
    return i32x8_t{(int)c.lo.x, (int)c.lo.y, (int)c.lo.z, (int)c.lo.w,
                   (int)c.hi.x, (int)c.hi.y, (int)c.hi.z, (int)c.hi.w};
}
// FORMAT of the second operand: 0 E4M3, 1 E5M2.
template <int FORMAT>
__device__ __forceinline__ f32x16_t mma32x8(const Codes& a, const Codes& b, f32x16_t c)
{
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(bits(a), bits(b), c, 0, FORMAT, 0, 0, 0, 0);
}
// Eight codes as bf16 (every one is a bf16 value).
template <int FORMAT>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, std::integral_constant<bool, false>)
{
    if constexpr (FORMAT == 0)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, false));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, 1.0f, false));
}
template <int FORMAT>
__device__ __forceinline__ uint32_t widen2(uint32_t codes, std::integral_constant<bool, true>)
{
    if constexpr (FORMAT == 0)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, 1.0f, true));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(codes, 1.0f, true));
}
template <int FORMAT>
__device__ __forceinline__ bf16x8_t widen(uint32_t lo, uint32_t hi)
{
    constexpr std::integral_constant<bool, false> low{};
    constexpr std::integral_constant<bool, true> high{};
    return __builtin_bit_cast(bf16x8_t, make_uint4(widen2<FORMAT>(lo, low), widen2<FORMAT>(lo, high),
                                                   widen2<FORMAT>(hi, low), widen2<FORMAT>(hi, high)));
}
// 128 codes of 16 rows by 128 of 16 columns; xw: the columns' widened.
__device__ __forceinline__ f32x4_t mma_block(const Codes& w, const bf16x8_t (&xw)[4])
{
    f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<0>(w.lo.x, w.lo.y), xw[0], d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<0>(w.lo.z, w.lo.w), xw[1], d, 0, 0, 0);
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<0>(w.hi.x, w.hi.y), xw[2], d, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen<0>(w.hi.z, w.hi.w), xw[3], d, 0, 0, 0);
}

struct Scaled {
    const char* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    const void* x_scales;
    bool scale_bytes;
    int64_t scale_row, scale_block;
    const char* w;
    const float* w_scales;
    int n, k, n_blocks, k_blocks;
    Segments seg;
    void* out;
    int64_t ld_out;
    int col_tiles, group;
    int64_t tiles;
    unsigned first_block;   // of this launch, few rows
};

// A scale as it lies in memory, and its value: 2^(byte - 127).
__device__ __forceinline__ uint32_t raw_scale(const Scaled& a, int64_t at)
{
    return a.scale_bytes ? static_cast<const uint8_t*>(a.x_scales)[at]
                         : __float_as_uint(static_cast<const float*>(a.x_scales)[at]);
}
__device__ __forceinline__ float scale_value(const Scaled& a, uint32_t raw)
{
    if (!a.scale_bytes) return __uint_as_float(raw);
    return __uint_as_float(raw == 0 ? 0x00400000u : raw << 23);
}

// Operand of a 32-row instruction over 64 codes: part s (of 2) of the step.
// Which 32 of the 64 a lane holds is the same for both operands.
__device__ __forceinline__ Codes codes_part(const char* lds, int row0, int b, int s)
{
    const int l = threadIdx.x & 63, r = l & 31, h = l >> 5, turn = (r >> 1) & 7;
    const char* p = lds + (row0 + r) * 128 + b * 4096;
    return Codes{*reinterpret_cast<const uint4*>(p + (((4 * s + h) ^ turn) << 4)),
                 *reinterpret_cast<const uint4*>(p + (((4 * s + 2 + h) ^ turn) << 4))};
}

// Any sizes: tiles of 128 x 128, two stages.  The second of the gated product's
// halves need not start with a block of 128 outputs: a tile's rows of it lie in
// two blocks.
template <typename T, int FORMAT, bool GLU>
__global__ __launch_bounds__(256)
void fp8_kernel(Scaled a)
{
    constexpr int BP = 128, BQ = 128, WQ = 2, PB = 2, QB = 2;
    using P = RowOperand<BP, 256, uint64_t>;
    using Q = RowOperand<BQ, 256, uint64_t>;
    constexpr int kStage = P::kBytes + Q::kBytes;
    __shared__ __attribute__((aligned(128))) char lds[2 * kStage];

    int i = 0, tile;
    RowBlock rb;
    if (!next_tile(TileWalk{a.tiles, a.col_tiles, a.group}, a.seg, BQ, i, rb, tile)) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int p0 = wave / WQ * (PB * 32), q0 = wave % WQ * (QB * 32);
    const int half = a.n / 2;
    const int n0 = tile * (GLU ? BP / 2 : BP);

    P p;
    Q q;
    // offsets from the tile's first row (of the gate half)
    p.init(a.w + ((int64_t)rb.expert * a.n + n0) * a.k, a.k, [&](int i) {
        int n;
        if constexpr (GLU) {
            n = i / 64 * 32 + (i & 31);
            n = (n0 + n < half ? n : half - 1 - n0) + (i & 32 ? half : 0);
        } else {
            n = n0 + i < a.n ? i : a.n - 1 - n0;
        }
        return (uint64_t)n * (uint64_t)a.k;
    });
    // a row of the tile, from the first (of all of x with src)
    auto x_row = [&](int i) {
        int r = i < rb.rows ? i : 0;
        if (a.src != nullptr) {
            r = a.src[rb.first + r];
            if (r < 0 || r >= a.x_rows) r = 0;
        }
        return r;
    };
    const int64_t x0 = a.src != nullptr ? 0 : rb.first;
    q.init(a.x + x0 * a.ld_x, a.k, [&](int i) { return (uint64_t)x_row(i) * (uint64_t)a.ld_x; });

    // scales: of this lane's rows, and of the tile's weights (the gate's and
    // the up's two)
    int64_t xs_at[QB];
#pragma unroll
    for (int j = 0; j < QB; ++j) xs_at[j] = (x0 + x_row(q0 + j * 32 + (lane & 31))) * a.scale_row;
    constexpr int kW = GLU ? 3 : 1;
    const float* ws_row[kW];
    const float* ws = a.w_scales + (int64_t)rb.expert * a.n_blocks * a.k_blocks;
    int up_bound = 0;       // outputs of the up half from here on take the next block
    if constexpr (GLU) {
        ws_row[0] = ws + (int64_t)(n0 / 128) * a.k_blocks;
        const int b = (half + n0) / 128;
        ws_row[1] = ws + (int64_t)b * a.k_blocks;
        ws_row[2] = ws + (int64_t)(b + 1 < a.n_blocks ? b + 1 : b) * a.k_blocks;
        up_bound = (b + 1) * 128 - half;
    } else {
        const int b = (n0 + p0) / 128;
        ws_row[0] = ws + (int64_t)(b < a.n_blocks ? b : a.n_blocks - 1) * a.k_blocks;
    }
    uint32_t xs_next[QB];
    float ws_next[kW];
    auto load_scales = [&](int s) {
#pragma unroll
        for (int j = 0; j < QB; ++j) xs_next[j] = raw_scale(a, xs_at[j] + s * a.scale_block);
#pragma unroll
        for (int i = 0; i < kW; ++i) ws_next[i] = ws_row[i][s];
    };

    f32x16_t acc[PB][QB];
#pragma unroll
    for (int i = 0; i < PB; ++i)
#pragma unroll
        for (int j = 0; j < QB; ++j) acc[i][j] = f32x16_t{};

    const int steps = a.k_blocks;
    const uint32_t at = lds_address(lds) + wave * 1024;
    auto load_all = [&](uint32_t to, int s) {
        load_operand<0>(p, to, s);
        load_operand<0>(q, to + P::kBytes, s);
    };
    load_all(at, 0);
    load_scales(0);
    for (int s = 0; s < steps; ++s) {
        wait_barrier();
        // the scales have arrived with the loads waited for; so that the
        // compiler knows before loads it does not count
        float xs[QB], wsv[kW];
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            asm volatile("" : "+v"(xs_next[j]));
            xs[j] = scale_value(a, xs_next[j]);
        }
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            asm volatile("" : "+v"(ws_next[i]));
            wsv[i] = ws_next[i];
        }
        const int now = (s & 1) * kStage, next = kStage - now;
        if (s + 1 < steps) {
            load_all(at + next, s + 1);
            load_scales(s + 1);
        }
        const char* pl = lds + now;
        const char* ql = lds + now + P::kBytes;
        Codes qc[QB][2];
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            qc[j][0] = codes_part(ql, q0, j, 0);
            qc[j][1] = codes_part(ql, q0, j, 1);
        }
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const Codes c0 = codes_part(pl, p0, i, 0), c1 = codes_part(pl, p0, i, 1);
#pragma unroll
            for (int j = 0; j < QB; ++j) {
                f32x16_t d = mma32x8<FORMAT>(c0, qc[j][0], f32x16_t{});
                d = mma32x8<FORMAT>(c1, qc[j][1], d);
                if constexpr (GLU) {
                    if (i & 1) {
                        const float f = xs[j] * wsv[1], g = xs[j] * wsv[2];
                        const int n = n0 + (p0 + (i - 1) * 32) / 2 + 4 * (lane >> 5);
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            acc[i][j][e] = __builtin_fmaf(d[e], n + e / 4 * 8 + e % 4 < up_bound ? f : g, acc[i][j][e]);
                        continue;
                    }
                }
                const float f = xs[j] * wsv[0];
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] = __builtin_fmaf(d[e], f, acc[i][j][e]);
            }
        }
    }

    T* out = static_cast<T*>(a.out);
#pragma unroll
    for (int j = 0; j < QB; ++j) {
        const int r = q0 + j * 32 + (lane & 31);
        const bool live = r < rb.rows;
        T* row = out + (rb.first + (live ? r : 0)) * a.ld_out;
        if constexpr (GLU) {
#pragma unroll
            for (int i = 0; i < PB; i += 2) {
                f32x16_t f;
#pragma unroll
                for (int e = 0; e < 16; ++e) f[e] = silu_of(acc[i][j][e]) * acc[i + 1][j][e];
                store_block(f, row, n0 + (p0 + i * 32) / 2, half, live);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PB; ++i) store_block(acc[i][j], row, n0 + p0 + i * 32, a.n, live);
        }
    }
}

// A tile's work with its scales: where this lane's rows' scales and the
// weights' lie (ws[1]: of the up half), and how many blocks there are.
struct ScaledWork : Work<RowOperand<256, 512>, RowOperand<128, 512>> {
    const char* xs;
    const float* ws[2];
    int blocks;
};

// Tiles of 256 outputs by 128 rows, eight wavefronts of 64 by 64 (PB x QB
// blocks), through the ring of ep_product.h: a step is a block of 128 codes.
//
// A pair of matrix instructions makes a block's sum over the step, from 0; it
// is scaled and added while the next pair runs (a lane's 16 values belong to
// one row, so one factor does).  The operands of the next row block are read
// meanwhile; those of the rows change, as their last pair has read them, with
// the step.  Scales of rows are loaded like operands, 64 a wavefront, into a
// place of its own for each of 4 steps; those of weights are scalar loads.
template <int FORMAT, bool GLU, bool BYTES>
struct ScaledSteps : Ring<RowOperand<256, 512>, RowOperand<128, 512>, 5> {
    using P = RowOperand<256, 512>;
    using Q = RowOperand<128, 512>;
    using R = Ring<P, Q, 5>;
    using W = ScaledWork;
    typedef const __attribute__((address_space(4))) float* scalar_ptr;
    static constexpr int PB = 2, QB = 2, kPairs = PB * QB, kHalves = GLU ? 2 : 1;
    static constexpr int kScalesAt = R::kLds, kAllLds = R::kLds + 8 * 4 * 256;
    // the first half of the loads that follow a step go out with its last row
    // block
    static constexpr int kFirst = R::kLoads / 2;

    int p0, q0;
    int64_t block_stride;   // bytes between a row's scales
    Codes p[2][2], q[QB][2];
    f32x16_t d[2];
    uint32_t xs[QB];        // of the next step
    float ws[kHalves];
    float f[QB][kHalves], last;

    __device__ __forceinline__ ScaledSteps(char* shared, int p_row, int q_row, const Scaled& a)
        : R(shared), p0(p_row), q0(q_row), block_stride(a.scale_block * (BYTES ? 1 : 4)), last(0.0f)
    {
    }

    // The scales of step s to their place: lane l those of the wavefront's row l.
    __device__ __forceinline__ void load_scales(const W& w, const W& nw, int s)
    {
        const bool mine = s < w.steps;
        const int step = mine ? s : s - w.steps, blocks = mine ? w.blocks : nw.blocks;
        const char* from = (mine ? w.xs : nw.xs) + (step < blocks ? step : 0) * block_stride;
        const uint32_t to = lds_address(lds) + kScalesAt + (at_wave() * 4 + (place(s, w) & 3)) * 256;
        if constexpr (BYTES)
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off" ::"s"(uniform((int)to)),
                         "v"(from)
                         : "m0");
        else
            asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(uniform((int)to)),
                         "v"(from)
                         : "m0");
    }
    __device__ __forceinline__ static int at_wave() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }
    // steps are counted through all tiles
    int done = 0;
    __device__ __forceinline__ int place(int s, const W&) const { return done + s; }

    __device__ __forceinline__ void read_scales(const W& w, const W& nw, int s)
    {
        const char* from = lds + kScalesAt + (at_wave() * 4 + (place(s, w) & 3)) * 256 + (threadIdx.x & 31) * 4;
#pragma unroll
        for (int j = 0; j < QB; ++j) xs[j] = *reinterpret_cast<const uint32_t*>(from + j * 128);
        const bool mine = s < w.steps;
        const int step = mine ? s : s - w.steps;
        const W& of = mine ? w : nw;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) ws[h] = ((scalar_ptr)of.ws[h])[step < of.blocks ? step : 0];
        live = step < of.blocks;
    }
    bool live;
    __device__ __forceinline__ void factors()
    {
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const float x = !BYTES ? __uint_as_float(xs[j])
                                   : __uint_as_float(xs[j] == 0 ? 0x00400000u : xs[j] << 23);
#pragma unroll
            for (int h = 0; h < kHalves; ++h) f[j][h] = live ? x * ws[h] : 0.0f;
        }
    }
    __device__ __forceinline__ void read_p(int set, int p_at, int i)
    {
        p[set][0] = codes_part(lds + p_at, p0, i, 0);
        p[set][1] = codes_part(lds + p_at, p0, i, 1);
    }
    __device__ __forceinline__ void read_q(int q_at, int j)
    {
        q[j][0] = codes_part(lds + q_at, q0, j, 0);
        q[j][1] = codes_part(lds + q_at, q0, j, 1);
    }

    // The pair for block (N / QB, N % QB) of a step, and what takes its turn.
    template <int KIND, int N>
    __device__ __forceinline__ void pair(f32x16_t (&acc)[PB][QB], W& w, W& nw, int s, int p_old, int q_old, int p_next,
                                         int q_next)
    {
        constexpr int i = N / QB, j = N % QB, kWas = (N + kPairs - 1) % kPairs;
        constexpr bool kLastBlock = i == PB - 1;
        const int p_at = p_now, q_at = q_now;
        if constexpr (kLastBlock && j == 0) wait_barrier<R::kLeft>();
        d[N & 1] = mma32x8<FORMAT>(p[i & 1][0], q[j][0], f32x16_t{});
        if constexpr (j == 0 && !kLastBlock) read_p((i + 1) & 1, p_at, i + 1);
        if constexpr (j == 0 && kLastBlock) {
            read_scales(w, nw, s + 1);
            read_p(0, p_next, 0);
        }
        d[N & 1] = mma32x8<FORMAT>(p[i & 1][1], q[j][1], d[N & 1]);
        if constexpr (kLastBlock) {
            if constexpr (j == 0) load_scales(w, nw, s + kQ);
            this->template load_some<kFirst * j / QB, kFirst * (j + 1) / QB, KIND>(w, nw, s, p_at, q_at);
        } else {
            constexpr int kRest = R::kLoads - kFirst, kSlots = kPairs - QB;
            this->template load_some<kFirst + kRest * N / kSlots, kFirst + kRest * (N + 1) / kSlots, KIND>(
                w, nw, s - 1, p_old, q_old);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e)
            acc[kWas / QB][kWas % QB][e] = __builtin_fmaf(d[(N + 1) & 1][e], last, acc[kWas / QB][kWas % QB][e]);
        asm volatile("" : "+v"(acc[kWas / QB][kWas % QB]));     // here, not when all pairs are done
        last = f[j][GLU ? i & 1 : 0];
        if constexpr (kLastBlock) read_q(q_next, j);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (N + 1 < kPairs) pair<KIND, N + 1>(acc, w, nw, s, p_old, q_old, p_next, q_next);
    }

    template <int KIND>
    __device__ __forceinline__ void step(f32x16_t (&acc)[PB][QB], W& w, W& nw, int s)
    {
        factors();
        pair<KIND, 0>(acc, w, nw, s, R::p_before(p_now), R::q_before(q_now), R::p_after(p_now), R::q_after(q_now));
        advance();
    }

    __device__ __forceinline__ void begin(W& w)
    {
        start<0>(w);
        load_scales(w, w, 0);
        load_scales(w, w, 1);
        load_some<0, kFirst, 2>(w, w, -1, p_before(p_now), q_before(q_now));
        wait_barrier();
        read_scales(w, w, 0);
        read_q(q_now, 0);
        read_q(q_now, 1);
        read_p(0, p_now, 0);
        d[0] = d[1] = f32x16_t{};
    }

    template <typename Prepare>
    __device__ __forceinline__ void tile(f32x16_t (&acc)[PB][QB], W& w, W& nw, Prepare prepare)
    {
        int s = 0;
        last = 0.0f;        // nothing to add before the first pair
        for (; s + kAhead < w.whole; ++s) step<1>(acc, w, w, s);
        prepare(nw);
        for (; s < w.steps; ++s) step<2>(acc, w, nw, s);
        done += w.steps;
        // the last pair's sum
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[PB - 1][QB - 1][e] = __builtin_fmaf(d[1][e], last, acc[PB - 1][QB - 1][e]);
        d[1] = f32x16_t{};
    }
};

template <typename T, int FORMAT, bool GLU, bool BYTES>
__global__ __launch_bounds__(512)
void fp8_tiles_kernel(Scaled a)
{
    using S = ScaledSteps<FORMAT, GLU, BYTES>;
    using W = ScaledWork;
    constexpr int BP = 256, BQ = 128, PB = S::PB, QB = S::QB;
    __shared__ __attribute__((aligned(128))) char lds[S::kAllLds];
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int p0 = wave / 2 * 64, q0 = wave % 2 * 64;
    const int half = a.n / 2;

    struct Tile {
        RowBlock rb;
        int n0;
    };
    int i = 0;
    const TileWalk walk = {a.tiles, a.col_tiles, a.group};
    auto find = [&](Tile& t) {
        int col;
        if (!next_tile(walk, a.seg, BQ, i, t.rb, col)) return false;
        t.n0 = col * (GLU ? BP / 2 : BP);
        return true;
    };
    auto prepare = [&](W& w, const Tile& t) {
        w.p.init(a.w + ((int64_t)t.rb.expert * a.n + t.n0) * a.k, a.k, [&](int r) {
            int n;
            if constexpr (GLU) {
                n = r / 64 * 32 + (r & 31);
                n = (t.n0 + n < half ? n : half - 1 - t.n0) + (r & 32 ? half : 0);
            } else {
                n = t.n0 + r < a.n ? r : a.n - 1 - t.n0;
            }
            return (uint32_t)n * (uint32_t)a.k;
        });
        auto x_row = [&](int i) {
            int r = i < t.rb.rows ? i : 0;
            if (a.src != nullptr) {
                r = a.src[t.rb.first + r];
                if (r < 0 || r >= a.x_rows) r = 0;
            }
            return r;
        };
        const int64_t x0 = a.src != nullptr ? 0 : t.rb.first;
        w.q.init(a.x + x0 * a.ld_x, a.k, [&](int i) { return (uint32_t)x_row(i) * (uint32_t)a.ld_x; });
        w.xs = static_cast<const char*>(a.x_scales) +
               (x0 + x_row(q0 + (opaque(threadIdx.x) & 63))) * a.scale_row * (BYTES ? 1 : 4);
        const float* ws = a.w_scales + (int64_t)t.rb.expert * a.n_blocks * a.k_blocks;
        const int b = GLU ? t.n0 / 128 : (t.n0 + p0) / 128;
        w.ws[0] = ws + (int64_t)(b < a.n_blocks ? b : a.n_blocks - 1) * a.k_blocks;
        w.ws[1] = GLU ? ws + (int64_t)((half + t.n0) / 128) * a.k_blocks : w.ws[0];
        w.blocks = a.k_blocks;
        w.steps = a.k_blocks > S::kFewestSteps ? a.k_blocks : S::kFewestSteps;
        w.whole = a.k / 128;
        w.turn = 0;
    };
    T* out = static_cast<T*>(a.out);
    auto store = [&](const f32x16_t (&acc)[PB][QB], const Tile& t) {
        const int lane = opaque(threadIdx.x) & 63;
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int r = q0 + j * 32 + (lane & 31);
            const bool live = r < t.rb.rows;
            T* row = out + (t.rb.first + (live ? r : 0)) * a.ld_out;
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < PB; i += 2) {
                    f32x16_t f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = silu_of(acc[i][j][e]) * acc[i + 1][j][e];
                    store_block(f, row, t.n0 + (p0 + i * 32) / 2, half, live);
                }
            } else {
#pragma unroll
                for (int i = 0; i < PB; ++i) store_block(acc[i][j], row, t.n0 + p0 + i * 32, a.n, live);
            }
        }
    };

    Tile t, nt;
    if (!find(t)) return;
    W w, nw;
    f32x16_t acc[PB][QB];
    S ring(lds, p0, q0, a);
    prepare(w, t);
    ring.begin(w);
    bool more = true;
    clear(acc);
    for (;;) {
        ring.tile(acc, w, nw, [&](W& next) {
            nt = t;
            Tile found;
            more = find(found);
            if (more) nt = found;
            prepare(next, nt);
        });
        store(acc, t);
        if (!more) break;
        clear(acc);
        w = nw;
        t = nt;
    }
    wait_barrier();
}

// Few rows an expert: as ep_expert_few.hip, a step of 128 codes at a time.
// SPLIT: gated halves that are not whole blocks of 16 outputs, so that a block
// of 16 may lie in two scales.
template <typename T, int FORMAT, bool GLU, bool SPLIT, int RT, int CT, int WAVES>
__global__ __launch_bounds__(WAVES * 64)
void fp8_few_kernel(Scaled a)
{
    extern __shared__ f32x4_t part[];       // [wave][RT][CT][64]
    constexpr int kHalves = GLU ? 2 : 1, kBlocks = RT / kHalves;
    const unsigned block = a.first_block + blockIdx.x, units = a.col_tiles;
    const int unit = (int)(block % units);
    const RowBlock it = find_rows(a.seg, CT * 16, (int)(block / units));
    if (it.rows <= 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int col = lane & 15, quad = lane >> 4;
    const int half_n = a.n / kHalves;

    const char* wr[RT];
    constexpr int kS = SPLIT ? 4 : 1;
    const float* ws[RT][kS];    // scales of the (four) outputs a lane holds of a row block
    const float* ws0 = a.w_scales + (int64_t)it.expert * a.n_blocks * a.k_blocks;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int up = GLU && (r & 1) ? half_n : 0;
        const int n = (unit * kBlocks + r / kHalves) * 16;
        const int mine = n + col < half_n ? n + col : half_n - 1;
        wr[r] = a.w + ((int64_t)it.expert * a.n + mine + up) * a.k + quad * 16;
#pragma unroll
        for (int i = 0; i < kS; ++i) {
            const int o = n + (SPLIT ? quad * 4 + i : 0);
            ws[r][i] = ws0 + (int64_t)(((o < half_n ? o : half_n - 1) + up) / 128) * a.k_blocks;
        }
    }
    struct Step {
        Codes w[RT], x[CT];
        float s[RT][kS];
        uint32_t xs[CT];
    };
    const char* xr[CT];
    int64_t xs_at[CT];
    // 128 codes of a row from k on: two chunks of 16 in this lane.  Chunks past
    // a.k are read from the row's start, and taken as 0.
    auto load_codes = [&](const char* row, int k) {
        const bool lo = k + quad * 16 < a.k, hi = k + 64 + quad * 16 < a.k;
        return Codes{*reinterpret_cast<const uint4*>(row + (lo ? k : -quad * 16)),
                     *reinterpret_cast<const uint4*>(row + (hi ? k + 64 : -quad * 16))};
    };
    auto drop = [&](Codes& c, int k) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        if (k + quad * 16 >= a.k) c.lo = none;
        if (k + 64 + quad * 16 >= a.k) c.hi = none;
    };
    auto load_weights = [&](Step& t, int kt) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            t.w[r] = load_codes(wr[r], kt * 128);
#pragma unroll
            for (int i = 0; i < kS; ++i) t.s[r][i] = ws[r][i][kt];
        }
    };
    auto load_x = [&](Step& t, int kt) {
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            t.x[c] = load_codes(xr[c], kt * 128);
            t.xs[c] = raw_scale(a, xs_at[c] + kt * a.scale_block);
        }
    };

    f32x4_t acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // The weights' first loads go out before the rows of x are known.  Rows
    // past the item's repeat its first row; their results are dropped.
    Step t;
    int kt = wave;
    load_weights(t, kt);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int in = c * 16 + col;
        int64_t r = it.first + (in < it.rows ? in : 0);
        if (a.src != nullptr) {
            r = a.src[r];
            if (r < 0 || r >= a.x_rows) r = 0;
        }
        xr[c] = a.x + r * a.ld_x + quad * 16;
        xs_at[c] = r * a.scale_row;
    }
    load_x(t, kt);
    while (true) {
        const int next = kt + waves;
        Step n;
        if (next < a.k_blocks) {
            load_weights(n, next);
            load_x(n, next);
        }
        if (kt * 128 + 128 > a.k) {
#pragma unroll
            for (int r = 0; r < RT; ++r) drop(t.w[r], kt * 128);
#pragma unroll
            for (int c = 0; c < CT; ++c) drop(t.x[c], kt * 128);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            const bf16x8_t xw[4] = {widen<FORMAT>(t.x[c].lo.x, t.x[c].lo.y), widen<FORMAT>(t.x[c].lo.z, t.x[c].lo.w),
                                    widen<FORMAT>(t.x[c].hi.x, t.x[c].hi.y), widen<FORMAT>(t.x[c].hi.z, t.x[c].hi.w)};
            const float xs = scale_value(a, t.xs[c]);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const f32x4_t d = mma_block(t.w[r], xw);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[r][c][i] = __builtin_fmaf(d[i], xs * t.s[r][SPLIT ? i : 0], acc[r][c][i]);
            }
        }
        if (next >= a.k_blocks) break;
        kt = next;
        t = n;
    }

#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) part[((wave * RT + r) * CT + c) * 64 + lane] = acc[r][c];
    __syncthreads();
    for (int o = threadIdx.x; o < kBlocks * CT * 64; o += blockDim.x) {
        const int ol = o & 63;
        const int c = (o >> 6) % CT;
        const int b = (o >> 6) / CT;
        f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
        for (int w = 0; w < waves; ++w) {
            v += part[((w * RT + b * kHalves) * CT + c) * 64 + ol];
            if constexpr (GLU) u += part[((w * RT + b * 2 + 1) * CT + c) * 64 + ol];
        }
        const int n = (unit * kBlocks + b) * 16 + (ol >> 4) * 4;
        const int in = c * 16 + (ol & 15);
        if (in >= it.rows) continue;
        if constexpr (GLU) v = f32x4_t{silu_of(v.x) * u.x, silu_of(v.y) * u.y, silu_of(v.z) * u.z, silu_of(v.w) * u.w};
        T* row = static_cast<T*>(a.out) + (int64_t)(it.first + in) * a.ld_out;
        const uint2 q = pack4<T>(v.x, v.y, v.z, v.w);
        if (n + 4 <= half_n) {
            __builtin_memcpy(row + n, &q, 8);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < half_n) row[n + i] = T{(uint16_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1)))};
        }
    }
}

Scaled scaled(const ExpertFp8Args& a)
{
    return Scaled{static_cast<const char*>(a.x), a.ld_x, a.x_rows, a.src, a.x_scales, a.scale_bytes,
                  a.scale_row, a.scale_block, static_cast<const char*>(a.w), a.w_scales, a.n, a.k,
                  (a.n + 127) / 128, (a.k + 127) / 128,
                  {a.offsets, a.counts, a.num_experts, (int)a.num_rows}, a.out, a.ld_out, 0, 8, 0, 0};
}

// Rows that 32-bit offsets do not reach, or two scales a tile: fp8_kernel.
bool general(const ExpertFp8Args& a)
{
    const int64_t reach = (a.src != nullptr ? a.x_rows : 256) * a.ld_x;
    const int64_t gate = a.gated ? (a.n / 2 + 256) * (int64_t)a.k : 0;
    return (a.gated && a.n / 2 % 128 != 0) || reach >= (int64_t)1 << 32 || gate >= (int64_t)1 << 32;
}
int general_cols(const ExpertFp8Args& a) { return a.gated ? (a.n / 2 + 63) / 64 : (a.n + 127) / 128; }
// Workgroups of fp8_kernel, each of 256 threads.
int64_t general_blocks(const ExpertFp8Args& a)
{
    return (tile_count(max_row_blocks(a.num_rows, a.num_experts, 128), 8, general_cols(a)) + 255) / 256 * 256;
}

template <typename T, int FORMAT, bool GLU>
hipError_t launch(const ExpertFp8Args& a, hipStream_t stream)
{
    Scaled p = scaled(a);
    p.col_tiles = general_cols(a);
    p.tiles = tile_count(max_row_blocks(a.num_rows, a.num_experts, 128), p.group, p.col_tiles);
    hipLaunchKernelGGL((fp8_kernel<T, FORMAT, GLU>), dim3((unsigned)general_blocks(a)), dim3(256), 0, stream, p);
    return hipGetLastError();
}

template <typename T, int FORMAT, bool GLU, bool SPLIT, int RT, int CT, int WAVES>
hipError_t launch_few(const ExpertFp8Args& a, hipStream_t stream)
{
    Scaled p = scaled(a);
    constexpr int kBlocks = GLU ? RT / 2 : RT;
    p.col_tiles = (((GLU ? a.n / 2 : a.n) + 15) / 16 + kBlocks - 1) / kBlocks;
    const int waves = WAVES < p.k_blocks ? WAVES : p.k_blocks;
    const int64_t items = max_row_blocks(a.num_rows, a.num_experts, 16 * CT);
    const int64_t blocks = items * p.col_tiles;
    for (int64_t first = 0; first < blocks; first += kMostBlocks) {
        p.first_block = (unsigned)first;
        const int64_t count = blocks - first < kMostBlocks ? blocks - first : kMostBlocks;
        hipLaunchKernelGGL((fp8_few_kernel<T, FORMAT, GLU, SPLIT, RT, CT, WAVES>), dim3((unsigned)count),
                           dim3(waves * 64), (size_t)waves * RT * CT * 1024, stream, p);
    }
    return hipGetLastError();
}

template <typename T, int FORMAT, bool GLU, bool SPLIT>
hipError_t few_sized(const ExpertFp8Args& a, hipStream_t stream)
{
    const int64_t hold = a.num_rows < a.num_experts ? a.num_rows : a.num_experts;
    if (a.num_rows / hold > 16) return launch_few<T, FORMAT, GLU, SPLIT, 2, 2, 4>(a, stream);
    const int64_t blocks = max_row_blocks(a.num_rows, a.num_experts, 16) * ((a.n + 15) / 16);
    // us for 64 outputs and 4 wavefronts, 32 and 2, 32 and 8: 512 rows of 256
    // experts 7168 -> 4096 (65536 blocks of 16 x 16 outputs) 526, 531, 763; 4 rows
    // of 64 experts, 2048 -> 2816 (2816 blocks) 18.7 (4 x 1 x 2), 17.9, 19.4 (2 x 1
    // x 4); one row, 4096 -> 4096 (256 blocks) 15.0, -, 9.7
    if (blocks >= 8192) return launch_few<T, FORMAT, GLU, SPLIT, 4, 1, 4>(a, stream);
    if (blocks >= 1024) return launch_few<T, FORMAT, GLU, SPLIT, 2, 1, 2>(a, stream);
    return launch_few<T, FORMAT, GLU, SPLIT, 2, 1, 8>(a, stream);
}

template <typename T, int FORMAT, bool GLU>
hipError_t sized(const ExpertFp8Args& a, hipStream_t stream)
{
    if (few_rows(a.num_rows, a.num_experts, a.n)) {
        if (GLU && a.n / 2 % 16 != 0) return few_sized<T, FORMAT, GLU, GLU>(a, stream);
        return few_sized<T, FORMAT, GLU, false>(a, stream);
    }
    if (general(a)) return launch<T, FORMAT, GLU>(a, stream);
    Scaled p = scaled(a);
    p.col_tiles = GLU ? (a.n / 2 + 127) / 128 : (a.n + 255) / 256;
    p.tiles = tile_count(max_row_blocks(a.num_rows, a.num_experts, 128), p.group, p.col_tiles);
    const dim3 grid(tile_grid(p.tiles, 1));
    if (a.scale_bytes)
        hipLaunchKernelGGL((fp8_tiles_kernel<T, FORMAT, GLU, true>), grid, dim3(512), 0, stream, p);
    else
        hipLaunchKernelGGL((fp8_tiles_kernel<T, FORMAT, GLU, false>), grid, dim3(512), 0, stream, p);
    return hipGetLastError();
}

template <typename T>
hipError_t typed(const ExpertFp8Args& a, hipStream_t stream)
{
    if (a.x_format == 0) return a.gated ? sized<T, 0, true>(a, stream) : sized<T, 0, false>(a, stream);
    return a.gated ? sized<T, 1, true>(a, stream) : sized<T, 1, false>(a, stream);
}

}  // namespace

hipError_t launch_expert_fp8(int dtype, const ExpertFp8Args& a, hipStream_t stream)
{
    if (a.num_rows == 0) return hipSuccess;
    return dtype == 0 ? typed<Bf16>(a, stream) : typed<Fp16>(a, stream);
}

bool expert_fp8_fits(const ExpertFp8Args& a)
{
    if (max_row_blocks(a.num_rows, a.num_experts, 16) * ((a.n + 31) / 32 + 1) > INT32_MAX) return false;
    return a.num_rows == 0 || few_rows(a.num_rows, a.num_experts, a.n) || !general(a) ||
           general_blocks(a) * 256 <= UINT32_MAX;
}

}  // namespace ep

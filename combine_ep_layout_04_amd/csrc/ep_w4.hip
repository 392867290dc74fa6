// ep_w4.hip -- the experts' products with 4-bit weights: for each row r of
// expert e, out[r, n] = sum_k scale[e, n, k / G] * (code[e, n, k] -
// zero[e, n, k / G]) * x[r, k], for few rows per expert, optionally with the
// gated activation out = silu(gate) * up over the two halves of n.
//
// Measured on MI355X: 64 tokens through 8 of 256 experts, 2048 -> 7168, 286 us
// (5.9 TB/s of weights, scales and rows); one token, 7168 -> 2 x 2048 gated,
// 25 us (4.8 TB/s).
//
// What bounds it: with few rows per expert every weight is used for a few
// products only, so the time is that of streaming the chosen experts'
// weights.  At half a byte per weight the vector unit has about 2.4
// operations per weight while a weight arrives, too few to unpack, scale and
// multiply-add each one; so the matrix cores take the products (a 16-row
// tile costs the same for 1 and for 16 tokens) and the unpacking is kept
// below one operation per weight:
//
//   * a code n enters the matrix core as the 16-bit float 16 + n, made by
//     setting four mantissa bits under a constant exponent: one rotate and
//     one and-or for two weights;
//   * the 16 and the zero point leave again per group, by
//     sum (16 + n) x - (16 + z) sum x, with sum x from the same matrix
//     instruction on a row of ones.  Codes, 16 + n and ones are exact in 16
//     bits and all sums are fp32: what the subtraction leaves is off by fp32
//     roundings of sum (32 + n + z) |x|, at most 62 scale sum |x| for the
//     result, however near to each other codes and zero points are;
//   * in bf16 both rows are taken 2^-12 times, and the result 2^12 times at
//     the end: 128 terms of at most 31 / 4096 x then stay below the largest
//     float for every finite x, where 31 x passed it from 1e37 on.  Nothing is
//     lost at the other end: the matrix instruction keeps subnormal numbers,
//     and a 2^-149 is 2^-137 in the result, under bf16's smallest step;
//   * the scale is applied once per group, to the fp32 sum.
//
// Layout of the packed weights (made once by ep_w4_pack): tiles of 16 rows
// by 128 k, 1 KiB each, in the order a wavefront reads them: lane l holds 16
// bytes, whose word i has the 8 codes k = 32 i + 8 (l / 16) .. + 7 of row
// l % 16 -- the matrix instruction's operand once unpacked, and one group of
// 32 a word index, so that groups of 32 and 64 also end between
// instructions.  Tiles of one row block follow one another along k, so a
// workgroup streams consecutive memory.  With the gated activation the row
// blocks of the two halves alternate.  Scales and zero points are held per
// tile, as the 4 rows of a lane's results for each group inside the tile (a
// group of more than 128 repeats its scale: 32 bytes a tile).  Rows are
// padded to 16 (scale 0), k to 128 (the kernels take x as 0 there).
//
// Split: a workgroup makes RT row blocks (16 RT outputs) for up to 16 CT
// rows of one expert, its wavefronts take turns at the k tiles and are
// joined through LDS in a fixed order: the few outputs of a single token
// still fill the chip, x is read once per workgroup, and results do not
// depend on timing.

#include "ep_device.h"
#include "ep_internal.h"
#include "ep_layer.h"
#include "ep_types.h"

namespace ep {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8_t __attribute__((ext_vector_type(8)));

// 16 + n as a 16-bit float: the code's place in the mantissa, the exponent
// of 16, and the float 1.0 (twice each: two weights a word), all in units of
// 1 / kUnit.
template <typename T>
struct Code;
template <>
struct Code<Bf16> {
    static constexpr int kShift = 3;
    static constexpr uint32_t kMask = 0x00780078u, kBase = 0x3B803B80u, kOnes = 0x39803980u;
    static constexpr float kUnit = 4096.0f;
};
template <>
struct Code<Fp16> {
    static constexpr int kShift = 6;
    static constexpr uint32_t kMask = 0x03C003C0u, kBase = 0x4C004C00u, kOnes = 0x3C003C00u;
    static constexpr float kUnit = 1.0f;
};

__device__ __forceinline__ f32x4_t mma(const uint4& a, const uint4& b, f32x4_t c, const Bf16*)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma(const uint4& a, const uint4& b, f32x4_t c, const Fp16*)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(fp16x8_t, a),
                                                  __builtin_bit_cast(fp16x8_t, b), c, 0, 0, 0);
}

// The two constants of the unpacking, in a scalar and a vector register: as
// literals they would take an and and an or each, since the one instruction
// that does both has no room for a literal.
template <typename T>
struct Unpacker {
    uint32_t mask, base;
    __device__ __forceinline__ Unpacker()
    {
        asm("s_mov_b32 %0, %1" : "=s"(mask) : "i"(Code<T>::kMask));
        asm("v_mov_b32 %0, %1" : "=v"(base) : "i"(Code<T>::kBase));
    }
    // Eight codes of a packed word as eight 16-bit floats 16 + n.
    __device__ __forceinline__ uint4 operator()(uint32_t w) const
    {
        return make_uint4((w & mask) | base, (__builtin_amdgcn_alignbit(w, w, 4) & mask) | base,
                          (__builtin_amdgcn_alignbit(w, w, 8) & mask) | base,
                          (__builtin_amdgcn_alignbit(w, w, 12) & mask) | base);
    }
};

// v / (1 + exp(-v)) by the hardware's exponential and reciprocal (one unit in
// the last place each; rounding the exponent's argument adds |v| * 2^-24).
// Below about -87, where 1 / (1 + exp(-v)) has no normal float, 0 for a value
// under 1e-35.
__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896f * v));
}

template <typename T>
__device__ __forceinline__ f32x4_t four(const uint2& s)
{
    f32x4_t f;
    f.x = to_float(T{(uint16_t)(s.x & 0xFFFFu)});
    f.y = to_float(T{(uint16_t)(s.x >> 16)});
    f.z = to_float(T{(uint16_t)(s.y & 0xFFFFu)});
    f.w = to_float(T{(uint16_t)(s.y >> 16)});
    return f;
}

// Inclusive sum over a wavefront's lanes, by lane moves in registers.
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);      // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);     // lane 15 to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);     // lane 31 to the upper half
    return v;
}

// The item-th (expert, block of TM rows) pair in expert order, found by a
// whole wavefront, 256 experts at a time: a lane counts the blocks of four
// experts (their loads go out together: what follows waits for them once).
struct Item {
    int expert, first, rows;
};
__device__ __forceinline__ Item find_item(const int32_t* offsets, const int32_t* counts, int E,
                                          int num_rows, int TM, int item)
{
    const int lane = threadIdx.x & 63;
    Item it = {0, 0, 0};
    if (offsets == nullptr) {         // one expert, all rows
        it.first = item * TM;
        it.rows = num_rows - it.first < TM ? num_rows - it.first : TM;
        return it;
    }
    int done = 0;
    for (int base = 0; base < E; base += 256) {
        const int e0 = base + lane * 4;
        int start[5], n[4], blocks[4];
#pragma unroll
        for (int i = 0; i < 5; ++i) start[i] = offsets[e0 + i < E ? e0 + i : E];
        if (counts != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = e0 + i < E ? counts[e0 + i] : 0;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = start[i + 1] - start[i];
        }
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            blocks[i] = (n[i] + TM - 1) / TM;
            mine += blocks[i];
        }
        const int upto = done + wave_scan(mine);
        const uint64_t past = __ballot(upto > item);
        if (past != 0) {
            int before = upto - mine;
            int expert = 0, first = 0, rows = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (item >= before && item < before + blocks[i]) {
                    const int skip = (item - before) * TM;
                    expert = e0 + i;
                    first = start[i] + skip;
                    rows = n[i] - skip < TM ? n[i] - skip : TM;
                }
                before += blocks[i];
            }
            const int at = __ffsll((unsigned long long)past) - 1;
            it.expert = __builtin_amdgcn_readlane(expert, at);
            it.first = __builtin_amdgcn_readlane(first, at);
            it.rows = __builtin_amdgcn_readlane(rows, at);
            break;
        }
        done = __builtin_amdgcn_readlane(upto, 63);
    }
    // never past the rows the caller gave, whatever the offsets say
    if (it.first < 0 || it.first >= num_rows) it.rows = 0;
    else if (it.rows > num_rows - it.first) it.rows = num_rows - it.first;
    return it;
}

// What one k tile needs, in registers: weights, x, scales, zero points.
template <int GS, int RT, int CT>
struct Stage {
    uint4 a[RT];
    uint4 x[CT][4];
    uint2 s[RT][GS];
    uint32_t z[RT][GS];
};

// GS: groups that end inside a 128-wide k tile (1 for groups of 128 and
// more); RT row blocks and CT blocks of 16 rows per workgroup of at most
// WAVES wavefronts.
template <typename T, int GS, bool ZEROS, bool GLU, int RT, int CT, int WAVES>
__global__ __launch_bounds__(WAVES * 64)
void w4_kernel(const T* __restrict__ x, int64_t ldx, int64_t x_rows, const int32_t* __restrict__ src,
               const uint4* __restrict__ weights, const uint2* __restrict__ scales,
               const uint32_t* __restrict__ zeros, const int32_t* __restrict__ offsets,
               const int32_t* __restrict__ counts, int E, int num_rows, int K, int half_n,
               int row_blocks, int k_tiles, int units,
               T* __restrict__ out, int64_t ldo)
{
    extern __shared__ f32x4_t part[];       // [wave][2][CT][64]
    const int unit = blockIdx.x % units;
    const Item it = find_item(offsets, counts, E, num_rows, CT * 16, (int)(blockIdx.x / units));
    if (it.rows <= 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int col = lane & 15;              // row of x within a block of 16, row of a weight tile
    const int quad = lane >> 4;

    const int64_t block0 = (int64_t)it.expert * row_blocks + (int64_t)unit * RT;
    int last = row_blocks - unit * RT - 1;  // the last unit may hold fewer row blocks
    if (last > RT - 1) last = RT - 1;
    const uint4* wp[RT];
    const uint2* sp[RT];
    const uint32_t* zp[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        const int64_t b = block0 + (r < last ? r : last);
        wp[r] = weights + b * k_tiles * 64;
        sp[r] = scales + b * k_tiles * GS * 4;
        zp[r] = zeros + b * k_tiles * GS * 4;
    }

    using St = Stage<GS, RT, CT>;
    const T* xr[CT];
    auto load_weights = [&](St& st, int kt) {
#pragma unroll
        for (int r = 0; r < RT; ++r) st.a[r] = wp[r][kt * 64 + lane];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                st.s[r][g] = sp[r][(kt * 4 + quad) * GS + g];
                if constexpr (ZEROS) st.z[r][g] = zp[r][(kt * 4 + quad) * GS + g];
            }
    };
    auto load_x = [&](St& st, int kt) {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = kt * 128 + i * 32;    // k past K: read at 0, taken as 0 below
                st.x[c][i] = __builtin_bit_cast(uint4, (u32x4)*reinterpret_cast<
                                 const typename Unaligned16<T>::type*>(xr[c] + (k < K ? k : 0)));
            }
    };

    const Unpacker<T> decode;
    f32x4_t acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    const uint4 ones = make_uint4(Code<T>::kOnes, Code<T>::kOnes, Code<T>::kOnes, Code<T>::kOnes);

    auto compute = [&](St& st, int kt) {
        if (kt * 128 + 128 > K) {                   // the last tile, K not a multiple of 128
#pragma unroll
            for (int i = 1; i < 4; ++i)
                if (kt * 128 + i * 32 >= K) {
#pragma unroll
                    for (int c = 0; c < CT; ++c) st.x[c][i] = make_uint4(0u, 0u, 0u, 0u);
                }
        }
#pragma unroll
        for (int g = 0; g < GS; ++g) {
            f32x4_t sum[CT];
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                sum[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4 / GS; ++i)
                    sum[c] = mma(ones, st.x[c][g * (4 / GS) + i], sum[c], static_cast<const T*>(nullptr));
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const f32x4_t s = four<T>(st.s[r][g]);
                f32x4_t off;
                if constexpr (ZEROS) {
                    const uint32_t z = st.z[r][g];
                    off.x = 16.0f + (float)(z & 255u);
                    off.y = 16.0f + (float)((z >> 8) & 255u);
                    off.z = 16.0f + (float)((z >> 16) & 255u);
                    off.w = 16.0f + (float)(z >> 24);
                } else {
                    off = f32x4_t{24.0f, 24.0f, 24.0f, 24.0f};
                }
                const uint32_t words[4] = {st.a[r].x, st.a[r].y, st.a[r].z, st.a[r].w};
                f32x4_t d[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) d[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4 / GS; ++i) {
                    const uint4 a = decode(words[g * (4 / GS) + i]);
#pragma unroll
                    for (int c = 0; c < CT; ++c)
                        d[c] = mma(a, st.x[c][g * (4 / GS) + i], d[c], static_cast<const T*>(nullptr));
                }
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const float sx = sum[c].x;
                    acc[r][c].x = __builtin_fmaf(s.x, __builtin_fmaf(-off.x, sx, d[c].x), acc[r][c].x);
                    acc[r][c].y = __builtin_fmaf(s.y, __builtin_fmaf(-off.y, sx, d[c].y), acc[r][c].y);
                    acc[r][c].z = __builtin_fmaf(s.z, __builtin_fmaf(-off.z, sx, d[c].z), acc[r][c].z);
                    acc[r][c].w = __builtin_fmaf(s.w, __builtin_fmaf(-off.w, sx, d[c].w), acc[r][c].w);
                }
            }
        }
    };

    // The weights' first loads go out before the rows of x are known.
    // Rows past the item's repeat its first row; their results are dropped.
    St st;
    int kt = wave;
    if (kt < k_tiles) load_weights(st, kt);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int in = c * 16 + col;
        int64_t r = it.first + (in < it.rows ? in : 0);
        if (src != nullptr) {
            r = src[r];
            if (r < 0 || r >= x_rows) r = 0;
        }
        xr[c] = x + r * ldx + quad * 8;
    }
    if (kt < k_tiles) load_x(st, kt);
    while (kt < k_tiles) {
        compute(st, kt);
        kt += waves;
        if (kt < k_tiles) {
            load_weights(st, kt);
            load_x(st, kt);
        }
    }

    // join the wavefronts, two row blocks at a time, and store
    constexpr int kJoin = RT < 2 ? 1 : 2;
#pragma unroll
    for (int r0 = 0; r0 < RT; r0 += kJoin) {
        if (r0 > 0) __syncthreads();
#pragma unroll
        for (int j = 0; j < kJoin; ++j)
#pragma unroll
            for (int c = 0; c < CT; ++c) part[((wave * kJoin + j) * CT + c) * 64 + lane] = acc[r0 + j][c];
        __syncthreads();
        constexpr int kOut = GLU ? 1 : kJoin;      // output blocks of this step
        for (int o = threadIdx.x; o < kOut * CT * 64; o += blockDim.x) {
            const int ol = o & 63;
            const int c = (o >> 6) % CT;
            const int j = (o >> 6) / CT;
            f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
            for (int w = 0; w < waves; ++w) {
                v += part[((w * kJoin + j) * CT + c) * 64 + ol];
                if constexpr (GLU) u += part[((w * kJoin + 1) * CT + c) * 64 + ol];
            }
            constexpr float kUnit = Code<T>::kUnit;
            float f[4] = {v.x * kUnit, v.y * kUnit, v.z * kUnit, v.w * kUnit};
            if constexpr (GLU) {
                const float up[4] = {u.x * kUnit, u.y * kUnit, u.z * kUnit, u.w * kUnit};
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = silu(f[i]) * up[i];
            }
            const int blk = GLU ? (unit * RT + r0) / 2 : unit * RT + r0 + j;
            const int n = blk * 16 + (ol >> 4) * 4;
            const int in = c * 16 + (ol & 15);
            if (in < it.rows && r0 + j <= last && n < half_n) {
                T* p = out + (int64_t)(it.first + in) * ldo + n;
                T q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = from_float<T>(f[i]);
                if (n + 4 <= half_n) {
                    __builtin_memcpy(p, q, 8);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (n + i < half_n) p[i] = q[i];
                }
            }
        }
    }
}

// ---- packing: the tiles of codes, then one thread per scale

__device__ __forceinline__ int row_of_block(int b, int i, int halves, int half_n)
{
    // row blocks of the halves alternate; -1 for a padded row
    const int n = b / halves * 16 + i;
    return n < half_n ? (b % halves) * half_n + n : -1;
}

// A wavefront a tile: lane l reads the 32 codes of chunk l % 4 of row l / 4
// (64 bytes a row), the words change places through LDS, and the tile goes
// out as it lies in memory.
__global__ __launch_bounds__(256)
void w4_pack_codes_kernel(const uint8_t* __restrict__ codes, int N, int K, int halves, int half_n,
                          int row_blocks, int k_tiles, int shift, int64_t tiles,
                          uint4* __restrict__ out)
{
    typedef uint32_t bytes16 __attribute__((ext_vector_type(4), aligned(1)));
    __shared__ uint32_t turn[4][256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t tile = (int64_t)blockIdx.x * 4 + wave;
    if (tile < tiles) {
        const int kt = (int)(tile % k_tiles);
        const int64_t eb = tile / k_tiles;
        const int row = lane >> 2, chunk = lane & 3;
        const int n = row_of_block((int)(eb % row_blocks), row, halves, half_n);
        const int k = kt * 128 + chunk * 32;
        u32x4 c = {0, 0, 0, 0};
        if (n >= 0 && k < K)
            c = (u32x4)*reinterpret_cast<const bytes16*>(
                codes + ((eb / row_blocks * N + n) * (int64_t)K + k) / 2);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            // even codes to the low half, odd ones to the high half, then
            // turned so that the first pair lies in the mantissas
            uint32_t w = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w |= ((c[q] >> (8 * j)) & 15u) << (4 * j);
                w |= ((c[q] >> (8 * j + 4)) & 15u) << (16 + 4 * j);
            }
            turn[wave][(row + 16 * q) * 4 + chunk] = (w << shift) | (w >> (32 - shift));
        }
    }
    __syncthreads();
    if (tile < tiles) {
        const uint32_t* t = &turn[wave][lane * 4];
        out[tile * 64 + lane] = make_uint4(t[0], t[1], t[2], t[3]);
    }
}

__global__ __launch_bounds__(256)
void w4_pack_scales_kernel(const uint16_t* __restrict__ scales, const uint8_t* __restrict__ zeros,
                           int N, int K, int group, int in_groups, int gs, int halves, int half_n,
                           int row_blocks, int k_tiles, int64_t total, uint16_t* __restrict__ out_s,
                           uint8_t* __restrict__ out_z)
{
    // [expert][row block][k tile][4 quads][gs groups][4 rows]
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (at >= total) return;
    const int i = (int)(at & 3);
    int64_t rest = at >> 2;
    const int g = (int)(rest % gs);
    rest /= gs;
    const int quad = (int)(rest & 3);
    rest >>= 2;
    const int kt = (int)(rest % k_tiles);
    const int64_t eb = rest / k_tiles;
    const int n = row_of_block((int)(eb % row_blocks), quad * 4 + i, halves, half_n);
    const int k = kt * 128 + g * (128 / gs);
    const bool in = n >= 0 && k < K;
    const int64_t from = in ? (eb / row_blocks * N + n) * (int64_t)in_groups + k / group : 0;
    out_s[at] = in ? scales[from] : (uint16_t)0;
    if (out_z != nullptr) out_z[at] = in ? zeros[from] : (uint8_t)0;
}

}  // namespace

W4Shape w4_shape(int num_experts, int n, int k, int group, bool zeros, bool glu)
{
    W4Shape s;
    s.halves = glu ? 2 : 1;
    s.half_n = n / s.halves;
    s.row_blocks = (s.half_n + 15) / 16 * s.halves;
    s.k_tiles = (k + 127) / 128;
    s.tile_groups = group >= 128 ? 1 : 128 / group;
    const int64_t tiles = (int64_t)num_experts * s.row_blocks * s.k_tiles;
    s.scales_at = tiles * 1024;
    s.zeros_at = (s.scales_at + tiles * s.tile_groups * 32 + 255) / 256 * 256;
    s.bytes = zeros ? (s.zeros_at + tiles * s.tile_groups * 16 + 255) / 256 * 256 : s.zeros_at;
    return s;
}

hipError_t launch_w4_pack(int dtype, const uint8_t* codes, const void* scales, const uint8_t* zeros,
                          int num_experts, int n, int k, int group, bool glu, void* packed,
                          hipStream_t stream)
{
    const W4Shape s = w4_shape(num_experts, n, k, group, zeros != nullptr, glu);
    char* base = static_cast<char*>(packed);
    const int64_t tiles = s.scales_at / 1024;
    hipLaunchKernelGGL(w4_pack_codes_kernel, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, stream,
                       codes, n, k, s.halves, s.half_n, s.row_blocks, s.k_tiles,
                       dtype == 0 ? Code<Bf16>::kShift : Code<Fp16>::kShift, tiles,
                       reinterpret_cast<uint4*>(base));
    hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int64_t total = (int64_t)num_experts * s.row_blocks * s.k_tiles * s.tile_groups * 16;
    hipLaunchKernelGGL(w4_pack_scales_kernel, dim3((unsigned)((total + 255) / 256)), dim3(256), 0, stream,
                       static_cast<const uint16_t*>(scales), zeros, n, k, group, (k + group - 1) / group,
                       s.tile_groups, s.halves, s.half_n, s.row_blocks, s.k_tiles, total,
                       reinterpret_cast<uint16_t*>(base + s.scales_at),
                       zeros != nullptr ? reinterpret_cast<uint8_t*>(base + s.zeros_at) : nullptr);
    return hipGetLastError();
}

namespace {

template <typename T, int GS, bool ZEROS, bool GLU, int RT, int CT, int WAVES>
hipError_t w4_launch(const W4Args& a, const W4Shape& s, int64_t items, int waves, hipStream_t stream)
{
    const int units = (s.row_blocks + RT - 1) / RT;
    const char* base = static_cast<const char*>(a.packed);
    const size_t lds = (size_t)waves * (RT < 2 ? 1 : 2) * CT * 1024;
    hipLaunchKernelGGL((w4_kernel<T, GS, ZEROS, GLU, RT, CT, WAVES>), dim3((unsigned)(items * units)),
                       dim3(waves * 64), lds, stream, static_cast<const T*>(a.x), a.ld_x, a.x_rows,
                       a.src, reinterpret_cast<const uint4*>(base),
                       reinterpret_cast<const uint2*>(base + s.scales_at),
                       reinterpret_cast<const uint32_t*>(base + s.zeros_at), a.offsets, a.counts,
                       a.num_experts, (int)a.num_rows, a.k, s.half_n, s.row_blocks, s.k_tiles,
                       units, static_cast<T*>(a.out), a.ld_out);
    return hipGetLastError();
}

// The split, by the rows an expert holds on average and by the 16-row output
// blocks the grid has to make (row blocks of the weights times items).  More
// row blocks a workgroup read x less often and join less; more wavefronts
// and smaller workgroups give a small grid enough loads in flight.  Measured
// on MI355X in a graph, us, RT x CT x wavefronts, bf16, the weights in copies
// that hold 0.8 GB or more together, so not in the caches; groups of 128, in
// brackets with zero points.  The rule's choice stands first.
//   at most 16 rows an expert:
//      256 blocks (1 row, 8192 -> 4096)          2x1x16 10 [11]   2x1x4 16 [16]   4x1x4 20 [20]
//      448        (1 row, 8192 -> 7168)          2x1x16 11 [12]   2x1x4 16 [17]
//      576        (1 row, 8192 -> 9216)          2x1x4 18 [18]   2x1x16 19 [20]   2x1x8 17 [17]
//     1496        (2 x 8 of 64, 2048 -> 1408)    2x1x4 10 [11]   4x1x4 11 [11]
//     2176        (2 x 8 of 64, 2048 -> 2048)    4x1x4 12 [12]   2x1x4 13 [13]
//    30.7 k       (64 x 8 of 64, 2048 -> 5120)   4x1x4 76 [80]   8x1x2 79 [83]
//    35328        (64 x 8 of 64, 2048 -> 5888)   8x1x2 83 [92]   4x1x4 86 [90]
//   129024        (64 x 8 of 256, 2048 -> 7168)  8x1x2 296 [336]   4x1x4 329 [347]   4x1x1 299 [313]
//   more than 16:
//      768        (64 rows, 4096 -> 4096)        2x2x8 13 [13]   4x2x4 15 [16]
//     1344        (64 rows, 4096 -> 7168)        2x2x8 21 [21]   4x2x4 16 [16]
//     1728        (64 rows, 4096 -> 9216)        4x2x4 24 [25]   2x2x8 29 [30]   8x2x4 22 [22]
//     3584        (64 x 2 of 4, 2048 -> 7168)    4x2x4 22 [22]   8x2x4 21 [28]
//     4352        (512 rows, 4096 -> 4096)       8x2x4 33 [42]   4x2x4 42 [44]   8x2x2 46 [37]
//     5760        (512 x 2 of 8, 2048 -> 2304)   8x2x4 34 [42]   8x2x2 31 [42]   4x2x4 33 [34]
//     7040        (512 x 2 of 8, 2048 -> 2816)   8x2x2 34 [43]   8x2x4 38 [53]   4x2x4 39 [40]
//    14080        (512 x 2 of 8, 2048 -> 5632)   8x2x2 61 [79]   8x2x1 55 [71]
//    16896        (512 x 8 of 64, 2048 -> 1408)  8x2x1 61 [75]   8x2x2 67 [83]   4x2x4 78 [79]
//    33792        (512 x 8 of 64, 2048 -> 2816)  8x2x1 119 [144]   8x2x2 120 [144]
// So the borders are good to a few per cent but for grids just below 1536,
// between 4096 and 6144 and between 10000 and 16384, where a neighbour is up
// to a quarter faster; with zero points, which take the 8 x 2 tile from two
// wavefronts a SIMD to one, 4 x 2 would be up to a quarter faster between
// 4608 and 14080 blocks.
//
// Groups of 32 and 64 hold 2 to 4 times the scales of a row block: eight row
// blocks do not fit the registers.  Groups of 64, of 32 and of 32 with zero
// points:
//     3808 blocks (2 x 8 of 64, 2048 -> 3584)    2x1x4 19, 22, 25   4x1x4 19, 23, 28
//     4352        (2 x 8 of 64, 2048 -> 4096)    4x1x4 21, 24, 29   2x1x4 21, 24, 29
//    24576        (64 x 8 of 64, 2048 -> 4096)   4x1x4 68, 87, 100   2x1x4 77, 89, 107
//    30.7 k       (64 x 8 of 64, 2048 -> 5120)   4x1x4 84, 111, 127   4x1x2 81, 100, 124
//    35328        (64 x 8 of 64, 2048 -> 5888)   4x1x2 91, 112, 143   4x1x4 96, 126, 148
//   129024        (64 x 8 of 256, 2048 -> 7168)  4x1x2 336, 423, 525   4x1x4 374, 486, 578   4x1x1 319, 401, 523
//   more than 16 rows an expert:
//     1344        (64 rows, 4096 -> 7168)        2x2x8 23, 25, 26   4x2x4 16, 19, 22
//     1728        (64 rows, 4096 -> 9216)        4x2x4 25, 34, 40   2x2x8 33, 35, 37
//     3584        (64 x 2 of 4, 2048 -> 7168)    4x2x4 25, 34, 37   4x2x1 25, 31, 36
//     4608        (64 x 2 of 4, 2048 -> 9216)    4x2x1 26, 32, 37   4x2x4 27, 40, 48
//    33792        (512 x 8 of 64, 2048 -> 2816)  4x2x1 154, 205, 241   2x2x2 213, 230, 247
//
// num_rows stands for the rows there are: in a padded layout it is their bound
// only, and the split is that of a larger grid, most of whose workgroups find
// no row and leave (8 of 256 experts, packed, aligned to 128 rows, 16 rows an
// expert: 64 tokens 2048 -> 7168 300, 374, 305; 1 token 7168 -> 4096 28, 46,
// 47; 512 tokens of 8 of 64, 2048 -> 2816, 96 rows an expert: 120, 121, 122).
template <typename T, int GS, bool ZEROS, bool GLU>
hipError_t w4_sized(const W4Args& a, const W4Shape& s, hipStream_t stream)
{
    // items: at most one per expert holding rows, and one more for every
    // full block of rows
    const int64_t hold = a.num_rows < a.num_experts ? a.num_rows : a.num_experts;
    const bool few = a.num_rows / hold <= 16;
    const int64_t items = hold + a.num_rows / (few ? 16 : 32);
    const int64_t blocks = items * s.row_blocks;
    auto cap = [&](int waves) { return waves < s.k_tiles ? waves : s.k_tiles; };
    if (few) {
        if (blocks >= 32768) {
            if constexpr (GS == 1) return w4_launch<T, GS, ZEROS, GLU, 8, 1, 4>(a, s, items, cap(2), stream);
            else return w4_launch<T, GS, ZEROS, GLU, 4, 1, 4>(a, s, items, cap(2), stream);
        }
        if (blocks >= (GS == 1 ? 1536 : 4096))
            return w4_launch<T, GS, ZEROS, GLU, 4, 1, 4>(a, s, items, cap(4), stream);
        if (blocks >= 512) return w4_launch<T, GS, ZEROS, GLU, 2, 1, 4>(a, s, items, cap(4), stream);
        constexpr int kMost = GS == 1 ? 16 : 8;
        return w4_launch<T, GS, ZEROS, GLU, 2, 1, kMost>(a, s, items, cap(kMost), stream);
    }
    if (blocks >= 4096) {
        if constexpr (GS == 1)
            return w4_launch<T, GS, ZEROS, GLU, 8, 2, 4>(
                a, s, items, cap(blocks >= 16384 ? 1 : blocks >= 6144 ? 2 : 4), stream);
        else
            return w4_launch<T, GS, ZEROS, GLU, 4, 2, 4>(a, s, items, 1, stream);
    }
    if (blocks >= 1536) return w4_launch<T, GS, ZEROS, GLU, 4, 2, 4>(a, s, items, cap(4), stream);
    return w4_launch<T, GS, ZEROS, GLU, 2, 2, 8>(a, s, items, cap(8), stream);
}

template <typename T, int GS>
hipError_t w4_typed(const W4Args& a, const W4Shape& s, hipStream_t stream)
{
    if (a.zeros) return a.glu ? w4_sized<T, GS, true, true>(a, s, stream) : w4_sized<T, GS, true, false>(a, s, stream);
    return a.glu ? w4_sized<T, GS, false, true>(a, s, stream) : w4_sized<T, GS, false, false>(a, s, stream);
}

template <typename T>
hipError_t w4_grouped(const W4Args& a, const W4Shape& s, hipStream_t stream)
{
    if (a.group == 32) return w4_typed<T, 4>(a, s, stream);
    if (a.group == 64) return w4_typed<T, 2>(a, s, stream);
    return w4_typed<T, 1>(a, s, stream);
}

}  // namespace

// Workgroups of the smallest tiles: what the grid has to hold at most.
int64_t w4_max_blocks(const W4Args& a)
{
    const W4Shape s = w4_shape(a.num_experts, a.n, a.k, a.group, a.zeros, a.glu);
    const int64_t hold = a.num_rows < a.num_experts ? a.num_rows : a.num_experts;
    return (hold + a.num_rows / 16) * ((s.row_blocks + 1) / 2);
}

hipError_t launch_w4(int dtype, const W4Args& a, hipStream_t stream)
{
    if (a.num_rows == 0) return hipSuccess;
    const W4Shape s = w4_shape(a.num_experts, a.n, a.k, a.group, a.zeros, a.glu);
    return dtype == 0 ? w4_grouped<Bf16>(a, s, stream) : w4_grouped<Fp16>(a, s, stream);
}

}  // namespace ep

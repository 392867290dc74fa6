// ep_expert_few.hip -- the experts' products in 16 bits for few rows an
// expert (decoding): every weight is used for a few rows only, so the time is
// that of streaming the chosen experts' weights.
//
// A workgroup makes 16 RT outputs for up to 16 CT rows of one expert.  Its
// wavefronts take turns at tiles of 128 inputs, each reading the weights
// straight into the matrix instruction's operand (a lane 16 bytes of its
// row), and are joined through LDS in a fixed order: the few outputs of a
// single token still fill the chip, and results do not depend on timing.
//
// 512 rows of 64 experts, 2048 -> 7168, 1.88 GB of weights: 319 us, 5.9 TB/s
// (a large copy moves 6.6).  One token through 4 experts, gated 2048 -> 2x1408,
// 46 MB: 12 us, of which a launch and the first loads' way are the most.
#include "ep_expert.h"
#include "ep_product.h"

namespace ep {
namespace {

__device__ __forceinline__ f32x4_t mma16(const uint4& a, const uint4& b, f32x4_t c, const Bf16*)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma16(const uint4& a, const uint4& b, f32x4_t c, const Fp16*)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(fp16x8_t, a),
                                                  __builtin_bit_cast(fp16x8_t, b), c, 0, 0, 0);
}

template <typename T>
struct Few {
    const T* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    const T* w;
    int n, k, half_n;       // half_n: outputs (n, or n / 2 if gated)
    Segments seg;
    T* out;
    int64_t ld_out;
    T* pre;
    int64_t ld_pre;
    int units, k_tiles;
    unsigned first_block;   // of this launch
};

// With the gated activation the RT row blocks are RT / 2 of the gate half,
// each followed by the one of the up half that belongs to it.
template <typename T, bool GLU, int RT, int CT, int WAVES>
__global__ __launch_bounds__(WAVES * 64)
void few_kernel(Few<T> a)
{
    extern __shared__ f32x4_t part[];       // [wave][RT][CT][64]
    constexpr int kHalves = GLU ? 2 : 1, kBlocks = RT / kHalves;
    const unsigned block = a.first_block + blockIdx.x, units = a.units;
    const int unit = (int)(block % units);
    const RowBlock it = find_rows(a.seg, CT * 16, (int)(block / units));
    if (it.rows <= 0) return;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int col = lane & 15, quad = lane >> 4;

    const T* wr[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
        int n = (unit * kBlocks + r / kHalves) * 16 + col;
        if (n >= a.half_n) n = a.half_n - 1;
        if (GLU && (r & 1)) n += a.half_n;
        wr[r] = a.w + ((int64_t)it.expert * a.n + n) * a.k + quad * 8;
    }
    const T* xr[CT];
    auto load = [&](uint4 (&w)[RT][4], uint4 (&x)[CT][4], int kt) {
        const int k = kt * 128;
        if (k + 128 <= a.k) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[r][i] = fetch16<T>(reinterpret_cast<const char*>(wr[r] + k + i * 32), 8);
#pragma unroll
            for (int c = 0; c < CT; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[c][i] = fetch16<T>(reinterpret_cast<const char*>(xr[c] + k + i * 32), 8);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int left = a.k - k - i * 32 - quad * 8;
#pragma unroll
                for (int r = 0; r < RT; ++r)
                    w[r][i] = fetch16<T>(reinterpret_cast<const char*>(wr[r] + k + i * 32), left);
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    x[c][i] = fetch16<T>(reinterpret_cast<const char*>(xr[c] + k + i * 32), left);
            }
        }
    };

    f32x4_t acc[RT][CT];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[r][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    // Rows past the item's repeat its first row; their results are dropped.
#pragma unroll
    for (int c = 0; c < CT; ++c) {
        const int in = c * 16 + col;
        int64_t r = it.first + (in < it.rows ? in : 0);
        if (a.src != nullptr) {
            r = a.src[r];
            if (r < 0 || r >= a.x_rows) r = 0;
        }
        xr[c] = a.x + r * a.ld_x + quad * 8;
    }
    for (int kt = wave; kt < a.k_tiles; kt += waves) {
        uint4 w[RT][4], x[CT][4];
        load(w, x, kt);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
                for (int c = 0; c < CT; ++c)
                    acc[r][c] = mma16(w[r][i], x[c][i], acc[r][c], static_cast<const T*>(nullptr));
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
        auto store = [&](const f32x4_t& f, T* row) {
            const uint2 q = pack4<T>(f.x, f.y, f.z, f.w);
            if (n + 4 <= a.half_n) {
                __builtin_memcpy(row + n, &q, 8);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (n + i < a.half_n) row[n + i] = T{(uint16_t)((i < 2 ? q.x : q.y) >> (16 * (i & 1)))};
            }
        };
        const int64_t row = it.first + in;
        if constexpr (GLU) {
            const f32x4_t f = {silu_of(v.x) * u.x, silu_of(v.y) * u.y, silu_of(v.z) * u.z, silu_of(v.w) * u.w};
            store(f, a.out + row * a.ld_out);
            if (a.pre != nullptr) {
                store(v, a.pre + row * a.ld_pre);
                store(u, a.pre + row * a.ld_pre + a.half_n);
            }
        } else {
            store(v, a.out + row * a.ld_out);
        }
    }
}

template <typename T, bool GLU, int RT, int CT, int WAVES>
hipError_t launch(const ExpertArgs& a, int64_t items, hipStream_t stream)
{
    const int half_n = GLU ? a.n / 2 : a.n;
    constexpr int kBlocks = GLU ? RT / 2 : RT;
    const int units = ((half_n + 15) / 16 + kBlocks - 1) / kBlocks;
    const int k_tiles = (a.k + 127) / 128;
    const int waves = WAVES < k_tiles ? WAVES : k_tiles;
    Few<T> f = {static_cast<const T*>(a.x), a.ld_x, a.x_rows, a.src, static_cast<const T*>(a.w), a.n, a.k,
                      half_n, {a.offsets, a.counts, a.num_experts, (int)a.num_rows},
                      static_cast<T*>(a.out), a.ld_out, static_cast<T*>(a.pre), a.ld_pre, units, k_tiles, 0};
    const int64_t blocks = items * units;
    for (int64_t first = 0; first < blocks; first += kMostBlocks) {
        f.first_block = (unsigned)first;
        const int64_t count = blocks - first < kMostBlocks ? blocks - first : kMostBlocks;
        hipLaunchKernelGGL((few_kernel<T, GLU, RT, CT, WAVES>), dim3((unsigned)count), dim3(waves * 64),
                           (size_t)waves * RT * CT * 1024, stream, f);
    }
    return hipGetLastError();
}

template <typename T, bool GLU>
hipError_t sized(const ExpertArgs& a, hipStream_t stream)
{
    const int64_t hold = a.num_rows < a.num_experts ? a.num_rows : a.num_experts;
    const int64_t items = max_row_blocks(a.num_rows, a.num_experts, 16);
    if (a.num_rows / hold <= 16) {
        // 32 outputs a workgroup and 8 wavefronts while there are no more than one
        // such workgroup a CU (512 blocks of 16 x 16 outputs), else 64 and 4.  us,
        // the former to the latter: one row, K 4096, 256 blocks 12.5 to 19.4, 384
        // blocks 14.5 to 19.8, 512 blocks 17.9 to 20.9, 576 blocks 25.3 to 22.3, 640
        // blocks 26.0 to 22.7, 896 blocks 28.9 to 27.2; 8 rows of 8 experts, gated, K
        // 2048, 512 blocks 10.3 to 12.6, 640 blocks 14.4 to 13.1; 4 rows of 4
        // experts, K 7168, 512 blocks 24.5 to 37.2, 640 blocks 38.0 to 36.9; 64
        // experts 2048 -> 2x1408, 1 row an expert 88.1 to 88.9, 8 rows 142 to 132
        if (items * ((a.n + 15) / 16) > 512) return launch<T, GLU, 4, 1, 4>(a, items, stream);
        return launch<T, GLU, 2, 1, 8>(a, items, stream);
    }
    // 24 rows of one expert, 4096 -> 4096: 16.8 us, with 64 outputs 24.2
    return launch<T, GLU, 2, 2, 4>(a, max_row_blocks(a.num_rows, a.num_experts, 32), stream);
}

}  // namespace

hipError_t launch_expert_few(int dtype, const ExpertArgs& a, hipStream_t stream)
{
    if (dtype == 0) return a.gated ? sized<Bf16, true>(a, stream) : sized<Bf16, false>(a, stream);
    return a.gated ? sized<Fp16, true>(a, stream) : sized<Fp16, false>(a, stream);
}

}  // namespace ep

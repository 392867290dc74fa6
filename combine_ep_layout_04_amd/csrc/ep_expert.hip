// ep_expert.hip -- the experts' products in 16 bits: out[r] = W[e] x[r] for
// the rows r of each expert e, or silu(gate) * up of the two halves of W[e]
// x[r], computed in one kernel.
//
// A workgroup makes a tile of BP outputs by BQ rows of one expert.  The
// weights are the matrix instruction's first operand, the rows its second:
// a lane ends with runs of outputs of one row.  For the gated product a tile
// takes 32 rows of the gate half, the 32 rows of the up half that belong to
// them, and so on: both land in the same lane, and the activation and the
// product happen in registers, in fp32, before the one rounding.
#include "ep_expert.h"
#include "ep_product.h"

namespace ep {
namespace {

template <typename T>
struct Product {
    const T* x;
    int64_t ld_x, x_rows;
    const int32_t* src;
    const T* w;
    int n, k;
    Segments seg;
    T* out;
    int64_t ld_out;
    T* pre;
    int64_t ld_pre;
    TileWalk walk;
    // Tiles begin at different steps of the reduction.  Few rows stream the
    // weights, and rows of them that are a power of two apart meet the same
    // channels of memory while all tiles are at the same step: 512 tokens, top 8
    // of 64 experts, gated 2048 -> 2x1408, 146 us, else 172.
    bool turned;
};

// WP x WQ wavefronts, a ring of RING operand tiles.  DIRECT: rows and weights
// in whole 16-byte chunks and in reach of 32-bit offsets, loaded into LDS
// directly; else by way of registers.
template <typename T, bool GLU, bool DIRECT, int BP, int BQ, int WP, int WQ, int RING>
__global__ __launch_bounds__(WP * WQ * 64)
void expert_kernel(Product<T> a)
{
    constexpr int kThreads = WP * WQ * 64;
    constexpr int PB = BP / WP / 32, QB = BQ / WQ / 32;
    using Off = std::conditional_t<DIRECT, uint32_t, uint64_t>;
    using P = RowOperand<BP, kThreads, Off>;
    using Q = RowOperand<BQ, kThreads, Off>;
    using R = Ring<P, Q, RING>;
    __shared__ __attribute__((aligned(128))) char lds[DIRECT ? R::kLds : 2 * (P::kBytes + Q::kBytes)];

    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const int p0 = wave / WQ * (PB * 32), q0 = wave % WQ * (QB * 32);
    const int half = a.n / 2;

    struct Tile {
        RowBlock rb;
        int n0;
    };
    int i = 0;
    auto find = [&](Tile& t) {
        int col;
        if (!next_tile(a.walk, a.seg, BQ, i, t.rb, col)) return false;
        t.n0 = col * (GLU ? BP / 2 : BP);
        return true;
    };
    auto prepare = [&](Work<P, Q>& w, const Tile& t) {
        const int bytes = a.k * 2, steps = (bytes + 127) / 128;
        // offsets from the tile's first row (of the gate half)
        const T* from = a.w + ((int64_t)t.rb.expert * a.n + t.n0) * a.k;
        w.p.init(reinterpret_cast<const char*>(from), bytes, [&](int r) {
            int n;
            if constexpr (GLU) {
                n = r / 64 * 32 + (r & 31);
                n = (t.n0 + n < half ? n : half - 1 - t.n0) + (r & 32 ? half : 0);
            } else {
                n = t.n0 + r < a.n ? r : a.n - 1 - t.n0;
            }
            return (Off)n * (Off)bytes;
        });
        const T* x = a.src != nullptr ? a.x : a.x + t.rb.first * a.ld_x;
        w.q.init(reinterpret_cast<const char*>(x), bytes, [&](int i) {
            int r = i < t.rb.rows ? i : 0;
            if (a.src != nullptr) {
                r = a.src[t.rb.first + r];
                if (r < 0 || r >= a.x_rows) r = 0;
            }
            return (Off)r * (Off)(a.ld_x * 2);
        });
        w.steps = steps > R::kFewestSteps ? steps : R::kFewestSteps;
        w.whole = bytes / 128;
        w.turn = 0;
        if (a.turned && w.steps == steps) {
            w.turn = (int)((unsigned)(t.n0 / 32 * 5 + t.rb.expert * 3) % (unsigned)steps);
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
            if constexpr (GLU) {
#pragma unroll
                for (int i = 0; i < PB; i += 2) {
                    const int64_t c = t.n0 + (p0 + i * 32) / 2;
                    f32x16_t f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[e] = silu_of(acc[i][j][e]) * acc[i + 1][j][e];
                    store_block(f, a.out + row * a.ld_out, c, half, live);
                    if (a.pre != nullptr) {
                        store_block(acc[i][j], a.pre + row * a.ld_pre, c, half, live);
                        store_block(acc[i + 1][j], a.pre + row * a.ld_pre + half, c, half, live);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < PB; ++i)
                    store_block(acc[i][j], a.out + row * a.ld_out, t.n0 + p0 + i * 32, a.n, live);
            }
        }
    };

    tiles<T, DIRECT, P, Q, PB, QB, RING, kThreads, Tile>(lds, p0, q0, find, prepare, store, (a.k + 63) / 64);
}

template <typename T, bool GLU, bool DIRECT, int BP, int BQ, int WP, int WQ, int RING>
hipError_t launch(const ExpertArgs& a, hipStream_t stream)
{
    Product<T> p = {static_cast<const T*>(a.x), a.ld_x, a.x_rows, a.src, static_cast<const T*>(a.w), a.n, a.k,
                    {a.offsets, a.counts, a.num_experts, (int)a.num_rows},
                    static_cast<T*>(a.out), a.ld_out, static_cast<T*>(a.pre), a.ld_pre, {}, BQ <= 128};
    constexpr int kCols = GLU ? BP / 2 : BP;
    const int n = GLU ? a.n / 2 : a.n;
    p.walk.group = 8;
    p.walk.col_tiles = (n + kCols - 1) / kCols;
    p.walk.tiles = tile_count(max_row_blocks(a.num_rows, a.num_experts, BQ), p.walk.group, p.walk.col_tiles);
    hipLaunchKernelGGL((expert_kernel<T, GLU, DIRECT, BP, BQ, WP, WQ, RING>),
                       dim3(tile_grid(p.walk.tiles, DIRECT ? 1 : 2)), dim3(WP * WQ * 64), 0, stream, p);
    return hipGetLastError();
}

// Elements of 16 bits that 32-bit offsets reach.
bool in_reach(int64_t elements) { return elements <= (int64_t)1 << 31; }

template <typename T, bool GLU>
hipError_t sized(const ExpertArgs& a, hipStream_t stream)
{
    const int64_t reach = (a.src != nullptr ? a.x_rows : 256) * a.ld_x, gate = GLU ? (a.n / 2 + 256) * (int64_t)a.k : 0;
    const bool direct = a.k % 8 == 0 && a.ld_x % 8 == 0 && in_reach(reach) && in_reach(gate) &&
                        ((reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.w)) & 15) == 0;
    // by way of registers (2 workgroups a CU): 4084 rows of 60 experts, 1999 ->
    // 1411, 133 us, 173 TFLOP/s: 720 tiles in 512 places, the last round part full
    if (!direct) return launch<T, GLU, false, 128, 128, 2, 2, 4>(a, stream);
    const int64_t hold = a.num_rows < a.num_experts ? a.num_rows : a.num_experts;
    // Tiles of 256 rows have half the LDS reads a product, tiles of 128 fill the
    // chip and the experts' ends better.  us, 256 to 128, 64 experts gated 2048
    // -> 2x1408: 192 rows an expert 215 to 227, 320 rows 331 to 316, 400 rows
    // 338 to 369, 512 rows 407 to 437, 1000 rows 662 to 764; below that 128
    // against 128 x 128 by registers: 64 rows 147 to 151, 160 rows 221 to 287
    if (a.num_rows / hold >= 192) return launch<T, GLU, true, 256, 256, 2, 2, 5>(a, stream);
    return launch<T, GLU, true, 256, 128, 2, 2, 5>(a, stream);
}

}  // namespace

hipError_t launch_expert(int dtype, const ExpertArgs& a, hipStream_t stream)
{
    if (a.num_rows == 0) return hipSuccess;
    if (few_rows(a.num_rows, a.num_experts, a.n)) return launch_expert_few(dtype, a, stream);
    if (dtype == 0) return a.gated ? sized<Bf16, true>(a, stream) : sized<Bf16, false>(a, stream);
    return a.gated ? sized<Fp16, true>(a, stream) : sized<Fp16, false>(a, stream);
}

int64_t expert_max_blocks(const ExpertArgs& a)
{
    // of ep_expert_few.hip's smallest tiles; the tiles above have as many
    // workgroups as the chip holds
    return max_row_blocks(a.num_rows, a.num_experts, 16) * ((a.n + 31) / 32 + 1);
}

}  // namespace ep

// ep_product.h -- what the experts' products share: operand tiles on their
// way from memory through LDS into the matrix cores, and the walk over the
// ragged rows of the experts.
//
// The matrix instruction's first operand gives the rows of its result, the
// second the columns.  Here the second is always the one whose index picks
// the output row in memory (a token; for the weights' gradient an output
// channel), so that a lane holds one output row and runs of neighbouring
// columns, and stores them 16 bytes at a time.
//
// A tile takes 128 bytes of the reduction a step (64 elements of 16 bits, 128
// of 8).  It is kept in LDS as it comes, one 16-byte chunk per lane of the
// loads that write LDS directly, with the chunks of a row turned so that the
// reads of the matrix operands meet every bank once:
//
//   * an operand that lies along the reduction in memory (RowOperand): rows of
//     8 chunks; chunk c of row r at place c ^ ((r / 2) % 8).  A lane reads 16
//     bytes of its row.
//   * an operand that lies across it (ColOperand): a row of the tile is one
//     step of the reduction, in 64-byte groups; group g of row r at place
//     g ^ (r % 4).  Lanes read it with the transposing LDS load (16 lanes, 4
//     rows of 16 elements: lane i gets column i).
#pragma once

#include "ep_device.h"
#include "ep_types.h"

namespace ep {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 fp16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x16_t mma32(const uint4& a, const uint4& b, f32x16_t c, const Bf16*)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                   __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mma32(const uint4& a, const uint4& b, f32x16_t c, const Fp16*)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(fp16x8_t, a),
                                                  __builtin_bit_cast(fp16x8_t, b), c, 0, 0, 0);
}

// v / (1 + exp(-v)) by the hardware's exponential and reciprocal (one unit in
// the last place each; rounding the exponent's argument adds |v| * 2^-24).
// Below about -87, where 1 / (1 + exp(-v)) has no normal float, 0 for a value
// under 1e-35.
__device__ __forceinline__ float sigmoid_of(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896f * v));
}
__device__ __forceinline__ float silu_of(float v) { return v * sigmoid_of(v); }

// ---- rows of the experts

// Inclusive sum over a wavefront's lanes, by lane moves in registers.
__device__ __forceinline__ int lanes_upto(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);      // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);     // lane 15 to the next row
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);     // lane 31 to the upper half
    return v;
}

// The rows of a call: segments of the layout.
struct Segments {
    const int32_t* offsets;     // NULL: one expert, all rows
    const int32_t* counts;      // NULL: to the next offset
    int num_experts, num_rows;
};

// A block of rows of one expert.
struct RowBlock {
    int expert, first, rows;
};

// Never past the rows the caller gave, whatever the offsets say.
__device__ __forceinline__ void bound_rows(RowBlock& b, int num_rows)
{
    if (b.first < 0 || b.first >= num_rows) b.rows = 0;
    else if (b.rows > num_rows - b.first) b.rows = num_rows - b.first;
}

// The item-th block of at most TM rows, in expert order, found by a whole
// wavefront, 256 experts at a time; rows 0 past the last.
__device__ __forceinline__ RowBlock find_rows(const Segments& s, int TM, int item)
{
    const int lane = threadIdx.x & 63;
    RowBlock b = {0, 0, 0};
    if (s.offsets == nullptr) {
        const int64_t first = (int64_t)item * TM;
        if (first >= s.num_rows) return b;
        b.first = (int)first;
        b.rows = s.num_rows - b.first < TM ? s.num_rows - b.first : TM;
        return b;
    }
    const int E = s.num_experts;
    int done = 0;
    for (int base = 0; base < E; base += 256) {
        const int e0 = base + lane * 4;
        int start[5], n[4], blocks[4];
#pragma unroll
        for (int i = 0; i < 5; ++i) start[i] = s.offsets[e0 + i < E ? e0 + i : E];
        if (s.counts != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = e0 + i < E ? s.counts[e0 + i] : 0;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) n[i] = start[i + 1] - start[i];
        }
        int mine = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            blocks[i] = n[i] > 0 ? (n[i] + TM - 1) / TM : 0;
            mine += blocks[i];
        }
        const int upto = done + lanes_upto(mine);
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
            b.expert = __builtin_amdgcn_readlane(expert, at);
            b.first = __builtin_amdgcn_readlane(first, at);
            b.rows = __builtin_amdgcn_readlane(rows, at);
            break;
        }
        done = __builtin_amdgcn_readlane(upto, 63);
    }
    bound_rows(b, s.num_rows);
    return b;
}

// Blocks of TM rows there can be at most: one for every full block of rows
// and a part of one for every expert that holds rows.
inline int64_t max_row_blocks(int64_t num_rows, int num_experts, int TM)
{
    return num_rows / TM + (num_rows < num_experts ? num_rows : num_experts);
}

// Workgroup b runs on XCD b % 8.  Each XCD takes runs of kRun tiles, which
// its 32 CUs work on together: `group` row blocks by kRun / group column
// tiles, so both operands are read into that XCD's L2 a few times only.
constexpr int kRun = 32;
inline int64_t tile_grid(int64_t items, int group, int col_tiles)
{
    const int64_t all = (items + group - 1) / group * group * col_tiles;
    return (all + 8 * kRun - 1) / (8 * kRun) * (8 * kRun);
}
__device__ __forceinline__ unsigned run_place()
{
    const unsigned j = blockIdx.x >> 3, xcd = blockIdx.x & 7;
    return (j / kRun * 8 + xcd) * kRun + j % kRun;
}
__device__ __forceinline__ void place_of(int group, int col_tiles, int& item, int& col)
{
    const unsigned at = run_place();
    const unsigned per = (unsigned)group * (unsigned)col_tiles;
    const unsigned rest = at % per;
    item = (int)(at / per * group + rest % group);
    col = (int)(rest / group);
}

// ---- operand tiles

// What lanes read in place of chunks past the end.
__device__ const uint4 kZeroChunk[1] = {{0u, 0u, 0u, 0u}};

// 16 bytes a lane from global memory to LDS: lane l's go to lds + 16 l.  The
// compiler does not count these loads: wait_barrier() waits for them.
__device__ __forceinline__ void load_lds(uint32_t lds, const char* from)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(from)
                 : "memory", "m0");
}

// This wavefront's loads into LDS have arrived and its LDS accesses are done,
// then so are those of the whole workgroup.
__device__ __forceinline__ void wait_barrier()
{
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint32_t lds_address(const char* p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// `valid` elements of 16 bits from p, the rest 0.
template <typename T>
__device__ __forceinline__ uint4 fetch16(const char* p, int valid)
{
    if (valid >= 8)
        return __builtin_bit_cast(uint4, (u32x4)*reinterpret_cast<const typename Unaligned16<T>::type*>(p));
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < valid) w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// An operand that lies along the reduction: ROWS rows by 128 bytes.
template <int ROWS, int THREADS>
struct RowOperand {
    static constexpr int kLoads = ROWS * 8 / THREADS;
    static constexpr int kBytes = ROWS * 128;
    const char* at[kLoads];
    int chunk;

    // row_at(i): the start of row i of the tile.
    template <typename F>
    __device__ __forceinline__ void init(F row_at)
    {
        const int t = threadIdx.x;
        chunk = (t & 7) ^ ((t >> 4) & 7);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) at[i] = row_at(t / 8 + i * (THREADS / 8)) + chunk * 16;
    }
    // Step `step` into LDS; of the reduction `bytes` are there (a whole
    // number of chunks).
    __device__ __forceinline__ void load(uint32_t lds, int step, int bytes) const
    {
        const bool out = step * 128 + 128 > bytes && step * 128 + chunk * 16 >= bytes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_lds(lds + i * THREADS * 16,
                     out ? reinterpret_cast<const char*>(kZeroChunk) : at[i] + (int64_t)step * 128);
    }
    // The same by way of registers, for rows that do not start on 16 bytes
    // or do not end with a chunk.
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int step, int bytes) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = fetch16<T>(at[i] + (int64_t)step * 128, (bytes - step * 128 - chunk * 16) / 2);
    }
    __device__ __forceinline__ static void put(char* lds, const uint4 (&v)[kLoads])
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<uint4*>(lds + (i * THREADS + threadIdx.x) * 16) = v[i];
    }
    // Operand of a 32-row matrix instruction: 8 elements of 16 bits, part s
    // (of 4) of the step, rows 32 b .. of this wavefront's.
    __device__ __forceinline__ static uint4 part(const char* lds, int row0, int b, int s)
    {
        const int l = threadIdx.x & 63, r = l & 31;
        return *reinterpret_cast<const uint4*>(lds + (row0 + r) * 128 + b * 4096 +
                                               (((2 * s + (l >> 5)) ^ ((r >> 1) & 7)) << 4));
    }
};

// An operand of 16-bit elements that lies across the reduction: 64 rows (its
// steps) by COLS columns.
template <int COLS, int THREADS>
struct ColOperand {
    static constexpr int kChunks = COLS / 8;
    static constexpr int kLoads = 64 * kChunks / THREADS;
    static constexpr int kBytes = 64 * COLS * 2;
    static constexpr int kRowStep = THREADS / kChunks;      // a multiple of 4: the turn is the same for all
    static_assert(kRowStep % 4 == 0, "rows of a thread share their turn");
    int row;            // of the tile, this thread's first
    int64_t column;     // byte offset of its chunk in a row
    int valid;          // elements of it that are there

    // Columns first .. of `cols`.
    __device__ __forceinline__ void init(int64_t first, int64_t cols)
    {
        const int t = threadIdx.x, p = t % kChunks;
        row = t / kChunks;
        const int64_t c = first + ((((p >> 2) ^ (row & 3)) << 2) | (p & 3)) * 8;
        valid = c + 8 <= cols ? 8 : c < cols ? (int)(cols - c) : 0;
        column = valid > 0 ? c * 2 : 0;
    }
    // row_at(i): the start of this thread's i-th row of this step (row +
    // i kRowStep); `left` rows are there.
    template <typename F>
    __device__ __forceinline__ void load(uint32_t lds, int left, F row_at) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const char* p = row_at(i) + column;
            load_lds(lds + i * THREADS * 16,
                     row + i * kRowStep < left ? p : reinterpret_cast<const char*>(kZeroChunk));
        }
    }
    template <typename T, typename F>
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int left, F row_at) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = fetch16<T>(row_at(i) + column, row + i * kRowStep < left ? valid : 0);
    }
    __device__ __forceinline__ static void put(char* lds, const uint4 (&v)[kLoads])
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<uint4*>(lds + (i * THREADS + threadIdx.x) * 16) = v[i];
    }
    // Operand of a 32-column matrix instruction: part s of the step, columns
    // col0 + 32 b ...
    __device__ __forceinline__ static uint4 part(const char* lds, int col0, int b, int s)
    {
        typedef __attribute__((address_space(3))) s16x4_t* lds_ptr;
        const int l = threadIdx.x & 63, i = l & 15;
        const int group = col0 / 32 + b;
        const char* p = lds + (16 * s + 8 * (l >> 5) + (i >> 2)) * (COLS * 2) +
                        ((group ^ (i >> 2)) << 6) + ((l >> 4) & 1) * 32 + (i & 3) * 8;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)p);
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(p + 4 * COLS * 2));
        const uint2 a = __builtin_bit_cast(uint2, lo), c = __builtin_bit_cast(uint2, hi);
        return make_uint4(a.x, a.y, c.x, c.y);
    }
};

// One step: PB x QB blocks of 32 x 32 from the operands' tiles.
template <typename T, typename P, typename Q, int PB, int QB>
__device__ __forceinline__ void multiply(const char* p_lds, const char* q_lds, int p0, int q0,
                                         f32x16_t (&acc)[PB][QB])
{
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint4 p[PB], q[QB];
#pragma unroll
        for (int j = 0; j < QB; ++j) q[j] = Q::part(q_lds, q0, j, s);
#pragma unroll
        for (int i = 0; i < PB; ++i) p[i] = P::part(p_lds, p0, i, s);
#pragma unroll
        for (int i = 0; i < PB; ++i)
#pragma unroll
            for (int j = 0; j < QB; ++j) acc[i][j] = mma32(p[i], q[j], acc[i][j], static_cast<const T*>(nullptr));
    }
}

// ---- results

// Two packed pairs of 16-bit results.
template <typename T>
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d)
{
    const T q[4] = {from_float<T>(a), from_float<T>(b), from_float<T>(c), from_float<T>(d)};
    return make_uint2(q[0].bits | (uint32_t)q[1].bits << 16, q[2].bits | (uint32_t)q[3].bits << 16);
}

// A 32 x 32 block: this lane's output row `row` (at its column 0), columns
// col .. of `cols`.  A lane holds runs of 4 columns, 4 (l / 32) + 8 i; lanes
// l and l + 32 hold the two halves of the same row and trade them, so that
// each stores runs of 8.
template <typename T>
__device__ __forceinline__ void store_block(const f32x16_t& v, T* row, int64_t col, int64_t cols, bool live)
{
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint2 a = pack4<T>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        const uint2 b = pack4<T>(v[4 * i + 4], v[4 * i + 5], v[4 * i + 6], v[4 * i + 7]);
        const auto x = __builtin_amdgcn_permlane32_swap(a.x, b.x, false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(a.y, b.y, false, false);
        const uint4 q = make_uint4(x[0], y[0], x[1], y[1]);
        const int64_t c = col + 8 * i + 8 * h;
        if (live) {
            if (c + 8 <= cols) {
                __builtin_memcpy(row + c, &q, 16);
            } else {
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c + k < cols) row[c + k] = T{(uint16_t)(w[k / 2] >> (16 * (k & 1)))};
            }
        }
    }
}
__device__ __forceinline__ void store_block(const f32x16_t& v, float* row, int64_t col, int64_t cols, bool live)
{
    const int h = (threadIdx.x >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = col + 8 * i + 4 * h;
        if (live) {
            const f32x4_t q = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            if (c + 4 <= cols) {
                __builtin_memcpy(row + c, &q, 16);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (c + k < cols) row[c + k] = q[k];
            }
        }
    }
}

}  // namespace ep

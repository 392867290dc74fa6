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
//     8 chunks, chunk c of row r at place c ^ ((r / 2) % 8).  A lane reads 16
//     bytes of its row.
//   * an operand that lies across it (ColOperand): a row of the tile is one
//     step of the reduction, in 64-byte groups; group g of row r at place
//     g ^ (r % 4).  Lanes read it with the transposing LDS load (16 lanes, 4
//     rows of 16 elements: lane i gets column i).
//
// No access of either kind meets a bank twice (counted: 0 conflicts).
//
// Many rows are bound by the matrix cores: 256 x 256 results by 4 wavefronts
// of 128 x 128, which is what the registers hold, take 16 bytes from LDS per
// 1024 products.  32768 rows of 32 experts, 7168 -> 4096 gated: 1670 us, 1.15
// PFLOP/s, and 1.30 with the rows that fill the last tiles of the experts up;
// the clock falls to about 1.65 GHz under this load, and the matrix cores are
// busy 82% of the cycles.  Slower at this size: 8 wavefronts and two
// stages 1990 us, steps of 64 bytes 1877 (twice the requests to L2), all loads
// of a step in one go 1987, tiles of 128 x 128 2372.  Within 2%: 2, 4, 8 or 16
// row blocks taken together, a workgroup per tile in place of ones that stay.
// Few rows are bound by the weights' bytes; see the rules at the launches.
#pragma once

#include <type_traits>

#include "ep_count.h"
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
// wavefront, 256 experts at a time.  Past the last one rows is 0, expert -1
// and first the number of blocks.
__device__ __forceinline__ RowBlock find_rows(const Segments& s, int TM, int item)
{
    const int lane = threadIdx.x & 63;
    RowBlock b = {-1, 0, 0};
    if (s.offsets == nullptr) {
        const int64_t first = (int64_t)item * TM;
        b.first = blocks_of(s.num_rows, TM);
        if (first >= s.num_rows) return b;
        b.expert = 0;
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
            blocks[i] = blocks_of(n[i], TM);
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
    if (b.expert < 0) b.first = done;
    else bound_rows(b, s.num_rows);
    return b;
}

// Workgroups of at most 512 threads that one launch is given: a launch takes
// fewer than 2^32 threads.  A call of more is several launches.  (One launch of
// two dimensions: 45.0 us where this takes 44.1, one token, 8 bits.)
constexpr int64_t kMostBlocks = 1 << 22;

// Workgroup b runs on XCD b % 8.  Each XCD takes runs of kRun tiles, which
// its 32 CUs work on together: `group` row blocks by kRun / group column
// tiles, so both operands are read into that XCD's L2 a few times only.  A
// workgroup takes its place in every run of its XCD in turn; two or more to a
// CU take neighbouring runs.  A run is 32 tiles however few there are, and row
// blocks are rounded up to whole groups: fewer than 256 tiles leave XCDs idle (8
// experts of 60 rows and 2048 outputs, 64 tiles, are on two of the eight), so
// calls of middle size run at a half to a quarter of what the chip could.
constexpr int kRun = 32, kXcds = 8;

inline int64_t tile_count(int64_t items, int group, int col_tiles)
{
    return (items + group - 1) / group * group * col_tiles;
}
// Workgroups for so many tiles, `per_cu` to a CU.
inline unsigned tile_grid(int64_t tiles, int per_cu)
{
    const int64_t runs = (tiles + kRun - 1) / kRun, most = kXcds * per_cu;
    return (unsigned)(((runs < most ? (runs + kXcds - 1) / kXcds * kXcds : most)) * kRun);
}
// The i-th tile of this workgroup.
__device__ __forceinline__ int64_t tile_of(int i)
{
    const unsigned xcd = blockIdx.x % kXcds, j = blockIdx.x / kXcds;
    const unsigned runs = gridDim.x / (kXcds * kRun);       // of an XCD at a time
    return (((int64_t)i * runs + j / kRun) * kXcds + xcd) * kRun + j % kRun;
}

// Row blocks and column tiles: the walk over the tiles of a call.
struct TileWalk {
    int64_t tiles;
    int col_tiles, group;
};
// This workgroup's next tile with rows from its i-th on; false past the last.
__device__ __forceinline__ bool next_tile(const TileWalk& t, const Segments& seg, int TM, int& i, RowBlock& rb,
                                          int& col)
{
    for (;; ++i) {
        const int64_t at = tile_of(i), per = (int64_t)t.group * t.col_tiles;
        if (at >= t.tiles) return false;
        const int64_t of = at / per * t.group;
        const unsigned rest = (unsigned)(at % per);
        rb = find_rows(seg, TM, (int)(of + rest % t.group));
        if (rb.rows > 0) {
            col = (int)(rest / t.group);
            ++i;
            return true;
        }
        if (rb.expert < 0 && of >= rb.first) return false;      // the whole group lies past the last block
    }
}

// ---- operand tiles

// v, whose origin the compiler does not see: what follows from it is computed
// where it is used, and not kept in registers through the steps of a tile.
__device__ __forceinline__ int opaque(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

// What lanes read in place of chunks past the end.
__device__ const uint4 kZeroChunk[1] = {{0u, 0u, 0u, 0u}};

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uniform(const char* p)
{
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    return reinterpret_cast<const char*>((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

// 16 bytes a lane from global memory to LDS, from base + off: lane l's go to
// lds + AT + 16 l.  The compiler does not count these loads: wait_barrier()
// waits for them.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"     // m0 in the clobber list
template <int AT>
__device__ __forceinline__ void load_lds(uint32_t lds, const char* base, uint32_t off)
{
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3"
                 :
                 : "s"(lds), "n"(AT), "v"(off), "s"(uniform(base))
                 : "m0", "scc");
}
// The same where some lanes have nothing to read: zeros for these.
template <int AT>
__device__ __forceinline__ void load_lds_or_zero(uint32_t lds, const char* base, uint64_t off, bool live)
{
    const char* from = live ? base + off : reinterpret_cast<const char*>(kZeroChunk);
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off"
                 :
                 : "s"(lds), "n"(AT), "v"(from)
                 : "m0", "scc");
}

#pragma clang diagnostic pop

// This wavefront's loads into LDS have arrived but for the last LEFT, and its
// LDS accesses are done; then so are those of the whole workgroup.
template <int LEFT = 0>
__device__ __forceinline__ void wait_barrier()
{
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(LEFT) : "memory");
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
// OFF holds the rows' offsets; with 32 bits a load takes no address arithmetic.
template <int ROWS, int THREADS, typename OFF = uint32_t>
struct RowOperand {
    static constexpr int kLoads = ROWS * 8 / THREADS;
    static constexpr int kBytes = ROWS * 128;
    static constexpr int kRowStep = THREADS / 8;    // a multiple of 16: the turn is the same for all
    static_assert(kRowStep % 16 == 0, "rows of a thread share their turn");
    const char* base;
    OFF off[kLoads];
    int chunk, bytes;

    // What the places of row r's chunks are turned by.
    __device__ __forceinline__ static int turn(int r) { return (r >> 1) & 7; }

    // Rows of `length` bytes; row i of the tile starts off_of(i) bytes behind
    // `from` (the same in every lane).
    template <typename F>
    __device__ __forceinline__ void init(const char* from, int length, F off_of)
    {
        const int t = opaque(threadIdx.x);
        base = uniform(from);
        bytes = length;
        chunk = (t & 7) ^ turn(t / 8);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = off_of(t / 8 + i * kRowStep) + chunk * 16;
    }
    // This thread's I-th chunk of step s into LDS (32-bit offsets).
    template <int I>
    __device__ __forceinline__ void load(uint32_t lds, int s) const
    {
        load_lds<I * THREADS * 16>(lds, base + (int64_t)s * 128, off[I]);
    }
    // The same for a step that may be the last, of a reduction that is a whole
    // number of chunks.
    template <int I>
    __device__ __forceinline__ void load_end(uint32_t lds, int s) const
    {
        load_lds_or_zero<I * THREADS * 16>(lds, base + (int64_t)s * 128, off[I], s * 128 + chunk * 16 < bytes);
    }
    // By way of registers, for rows that do not start on 16 bytes or do not
    // end with a chunk.
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int s) const
    {
        if (s * 128 + 128 <= bytes) {       // no branch between the loads
#pragma unroll
            for (int i = 0; i < kLoads; ++i) v[i] = fetch16<T>(base + (int64_t)s * 128 + off[i], 8);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                v[i] = fetch16<T>(base + (int64_t)s * 128 + off[i], (bytes - s * 128 - chunk * 16) / 2);
        }
    }
    // Chunk c of the row of this lane in block b of the wavefront's rows.
    __device__ __forceinline__ static uint4 chunk_of(const char* lds, int row0, int b, int c)
    {
        const int r = threadIdx.x & 31;
        return *reinterpret_cast<const uint4*>(lds + (row0 + r) * 128 + b * 4096 + ((c ^ turn(r)) << 4));
    }
    // Operand of a 32-row matrix instruction: 8 elements of 16 bits, part s
    // of the step.
    __device__ __forceinline__ static uint4 part(const char* lds, int row0, int b, int s)
    {
        return chunk_of(lds, row0, b, 2 * s + ((threadIdx.x >> 5) & 1));
    }
};

// An operand of 16-bit elements that lies across the reduction: 64 rows (its
// steps) by COLS columns.
template <int COLS, int THREADS, typename OFF = uint32_t>
struct ColOperand {
    static constexpr int kChunks = COLS / 8;
    static constexpr int kLoads = 64 * kChunks / THREADS;
    static constexpr int kBytes = 64 * COLS * 2;
    static constexpr int kRowStep = THREADS / kChunks;  // a multiple of 4: the turn is the same for all
    static_assert(kRowStep % 4 == 0, "rows of a thread share their turn");
    const char* base;
    OFF off[kLoads];
    int64_t ld;                 // bytes
    int row, rows;              // of the tile this thread's first; of the reduction
    int valid;                  // elements of its chunk that are there
    bool inside;                // all columns are

    // `count` rows, `stride` bytes apart, from `from` on; columns first .. of
    // `cols`.
    __device__ __forceinline__ void init(const char* from, int64_t stride, int count, int64_t first, int64_t cols)
    {
        const int t = opaque(threadIdx.x), p = t % kChunks;
        row = t / kChunks;
        base = uniform(from);
        ld = stride;
        rows = count;
        const int64_t c = first + ((((p >> 2) ^ (row & 3)) << 2) | (p & 3)) * 8;
        valid = c + 8 <= cols ? 8 : c < cols ? (int)(cols - c) : 0;
        inside = first + COLS <= cols;
        const OFF column = valid > 0 ? (OFF)c * 2 : 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = (OFF)((row + i * kRowStep) * ld) + column;
    }
    // This thread's I-th chunk of step s into LDS.
    template <int I>
    __device__ __forceinline__ void load(uint32_t lds, int s) const
    {
        load_lds<I * THREADS * 16>(lds, base + s * 64 * ld, off[I]);
    }
    // The same for a step that may be the last.
    template <int I>
    __device__ __forceinline__ void load_end(uint32_t lds, int s) const
    {
        load_lds_or_zero<I * THREADS * 16>(lds, base + s * 64 * ld, off[I], s * 64 + row + I * kRowStep < rows);
    }
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int s) const
    {
        const char* from = base + (int64_t)s * 64 * ld;
        if (inside && whole_step(s, rows)) {        // no branch between the loads
#pragma unroll
            for (int i = 0; i < kLoads; ++i) v[i] = fetch16<T>(from + off[i], 8);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                v[i] = fetch16<T>(from + off[i], s * 64 + row + i * kRowStep < rows ? valid : 0);
        }
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

// All of a thread's chunks of a step that may be the last into LDS.
template <int I, typename O>
__device__ __forceinline__ void load_operand(O& o, uint32_t to, int s)
{
    if constexpr (I < O::kLoads) {
        o.template load_end<I>(to, s);
        load_operand<I + 1>(o, to, s);
    }
}

// A thread's chunks from registers to its operand's place in LDS.
template <int THREADS, int LOADS>
__device__ __forceinline__ void put_chunks(char* lds, const uint4 (&v)[LOADS])
{
#pragma unroll
    for (int i = 0; i < LOADS; ++i) *reinterpret_cast<uint4*>(lds + (i * THREADS + threadIdx.x) * 16) = v[i];
}

// ---- the steps

// A tile's operands and its length: steps of the reduction (at least
// kFewestSteps: what is not there is zeros), and how many of them are known to
// be whole.  The steps are taken from `turn` on, round.
template <typename P, typename Q>
struct Work {
    P p;
    Q q;
    int steps, whole, turn;

    __device__ __forceinline__ int step(int s) const { return s + turn < steps ? s + turn : s + turn - steps; }
};

// The ring of operand tiles in LDS that a workgroup's tiles go through one
// after another, 128 bytes of the reduction a step.
//
// P has (RING + 1) / 2 places, Q RING / 2 (256 x 256 with 3 and 2: all of
// LDS), and P is loaded a step further ahead where it has one more.  The ring
// does not stop between tiles: the last steps of one send the loads of the
// first steps of the next, which arrive while results are stored.
template <typename P, typename Q, int RING>
struct Ring {
    using W = Work<P, Q>;
    static constexpr int kP = (RING + 1) / 2, kQ = RING / 2;    // places
    static constexpr int kQAt = kP * P::kBytes;                 // where Q's begin
    static constexpr int kLds = kQAt + kQ * Q::kBytes;
    static constexpr int kLoads = P::kLoads + Q::kLoads;
    // loads that may be under way when a step changes: those behind the next
    // step's
    static constexpr int kLeft = (kQ - 2) * kLoads + (kP - kQ) * P::kLoads;
    static constexpr int kAhead = kP;           // steps to the last load that follows a step
    static constexpr int kFewestSteps = kAhead; // so that loads never reach past the next tile
    static_assert(kQ >= 2, "two steps at least");

    char* lds;
    uint32_t at;
    int p_now, q_now;       // the step's places, from lds

    __device__ __forceinline__ Ring(char* shared) : lds(shared), p_now(0), q_now(kQAt)
    {
        at = lds_address(lds) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) * 1024;
    }
    __device__ __forceinline__ static int p_after(int v) { return v + P::kBytes < kQAt ? v + P::kBytes : 0; }
    __device__ __forceinline__ static int q_after(int v) { return v + Q::kBytes < kLds ? v + Q::kBytes : kQAt; }
    __device__ __forceinline__ static int p_before(int v) { return v > 0 ? v - P::kBytes : kQAt - P::kBytes; }
    __device__ __forceinline__ static int q_before(int v) { return v > kQAt ? v - Q::kBytes : kLds - Q::kBytes; }
    __device__ __forceinline__ void advance()
    {
        p_now = p_after(p_now);
        q_now = q_after(q_now);
    }

    template <int I, typename O>
    __device__ __forceinline__ static void load_near(O& mine, O& next, const W& w, const W& nw, uint32_t to, int s)
    {
        if (s < w.steps) mine.template load_end<I>(to, w.step(s));
        else next.template load_end<I>(to, nw.step(s - w.steps));
    }
    // The I-th of the loads that follow step s with its places p_at and q_at:
    // Q's, then P's.  KIND 1: of whole steps of this tile; 2: of steps that may
    // be the last, or the next tile's.
    template <int I, int KIND>
    __device__ __forceinline__ void load_one(W& w, W& nw, int s, int p_at, int q_at)
    {
        if constexpr (I < Q::kLoads) {
            if constexpr (KIND == 1) w.q.template load<I>(at + q_at, w.step(s + kQ));
            else load_near<I>(w.q, nw.q, w, nw, at + q_at, s + kQ);
        } else {
            if constexpr (KIND == 1) w.p.template load<I - Q::kLoads>(at + p_at, w.step(s + kP));
            else load_near<I - Q::kLoads>(w.p, nw.p, w, nw, at + p_at, s + kP);
        }
    }
    template <int I, int UPTO, int KIND>
    __device__ __forceinline__ void load_some(W& w, W& nw, int s, int p_at, int q_at)
    {
        if constexpr (I < UPTO) {
            load_one<I, KIND>(w, nw, s, p_at, q_at);
            load_some<I + 1, UPTO, KIND>(w, nw, s, p_at, q_at);
        }
    }
    // The first tile's first loads: what the steps before it would have sent,
    // of the last of them the first SENT only.
    template <int SENT>
    __device__ __forceinline__ void begin(W& w)
    {
        start<0>(w);
        load_some<0, SENT, 2>(w, w, -1, p_before(p_now), q_before(q_now));
        wait_barrier<kLeft + SENT>();
    }
    template <int S>
    __device__ __forceinline__ void start(W& w)
    {
        if constexpr (S + 1 < kP) {
            load_operand<0>(w.p, at + S * P::kBytes, w.step(S));
            if constexpr (S + 1 < kQ) load_operand<0>(w.q, at + kQAt + S * Q::kBytes, w.step(S));
            start<S + 1>(w);
        }
    }
};

// PB x QB blocks of 32 x 32 per wavefront of 16-bit operands from the ring.
//
// Two sets of operands in registers: those of a part (16 elements of the
// reduction, 32 bytes) are read while the part before it is multiplied.  The
// step changes before its last part, whose operands are in registers by then:
// its multiplications cover the first reads of the next step.  From there to
// the next such place the loads into the two places that became free go out,
// dealt out evenly: sent in one go they fill the queue of the memory pipeline,
// and the wavefront stands still before its matrix instructions.  Reads and
// loads take their turns after matrix instructions, by hand.
template <typename T, typename P, typename Q, int PB, int QB, int RING>
struct Steps : Ring<P, Q, RING> {
    using R = Ring<P, Q, RING>;
    using W = Work<P, Q>;
    using R::kLoads;
    static constexpr int kMuls = PB * QB, kReads = PB + QB;

    int p0, q0;
    uint4 p[2][PB], q[2][QB];

    __device__ __forceinline__ Steps(char* shared, int p_row, int q_row) : R(shared), p0(p_row), q0(q_row) {}

    template <int I, int UPTO>
    __device__ __forceinline__ void read_some(int set, int p_at, int q_at, int part)
    {
        if constexpr (I < UPTO) {
            if constexpr (I < QB) q[set][I] = Q::part(this->lds + q_at, q0, I, part);
            else p[set][I - QB] = P::part(this->lds + p_at, p0, I - QB, part);
            read_some<I + 1, UPTO>(set, p_at, q_at, part);
        }
    }

    // Matrix instruction M of a part and what takes its turn after it: reads of
    // part `next` of the step at p_to and q_to into the other set, and the
    // SHARE-th quarter of the loads that follow step s at p_at and q_at.
    template <int SET, int KIND, int SHARE, int M = 0>
    __device__ __forceinline__ void part(f32x16_t (&acc)[PB][QB], W& w, W& nw, int p_to, int q_to, int next, int s,
                                         int p_at, int q_at)
    {
        if constexpr (M < kMuls) {
            constexpr int i = M / QB, j = M % QB;
            acc[i][j] = mma32(p[SET][i], q[SET][j], acc[i][j], static_cast<const T*>(nullptr));
            // all reads within the first three quarters
            constexpr int kFrom = kReads * M * 4 / (kMuls * 3), kTo = kReads * (M + 1) * 4 / (kMuls * 3);
            read_some<(kFrom < kReads ? kFrom : kReads), (kTo < kReads ? kTo : kReads)>(SET ^ 1, p_to, q_to, next);
            constexpr int kOf = kLoads * SHARE / 4, kCount = kLoads * (SHARE + 1) / 4 - kOf;
            this->template load_some<kOf + kCount * M / kMuls, kOf + kCount * (M + 1) / kMuls, KIND>(w, nw, s, p_at,
                                                                                                     q_at);
            __builtin_amdgcn_sched_barrier(0);
            part<SET, KIND, SHARE, M + 1>(acc, w, nw, p_to, q_to, next, s, p_at, q_at);
        }
    }

    template <int KIND>
    __device__ __forceinline__ void step(f32x16_t (&acc)[PB][QB], W& w, W& nw, int s)
    {
        const int p_at = this->p_now, q_at = this->q_now;
        const int p_old = R::p_before(p_at), q_old = R::q_before(q_at);
        const int p_next = R::p_after(p_at), q_next = R::q_after(q_at);
        part<0, KIND, 1>(acc, w, nw, p_at, q_at, 1, s - 1, p_old, q_old);
        part<1, KIND, 2>(acc, w, nw, p_at, q_at, 2, s - 1, p_old, q_old);
        part<0, KIND, 3>(acc, w, nw, p_at, q_at, 3, s - 1, p_old, q_old);
        wait_barrier<R::kLeft>();
        part<1, KIND, 0>(acc, w, nw, p_next, q_next, 0, s, p_at, q_at);
        this->advance();
    }

    __device__ __forceinline__ void begin(W& w)
    {
        R::template begin<kLoads / 4>(w);
        read_some<0, kReads>(0, this->p_now, this->q_now, 0);
    }

    // A whole tile, and the first loads of the next, which prepare(nw) finds
    // when they come near (so that it takes no registers before).
    template <typename Prepare>
    __device__ __forceinline__ void tile(f32x16_t (&acc)[PB][QB], W& w, W& nw, Prepare prepare)
    {
        int s = 0;
        for (; s + R::kAhead < w.whole; ++s) step<1>(acc, w, w, s);
        prepare(nw);
        for (; s < w.steps; ++s) step<2>(acc, w, nw, s);
    }
};

// Keeps sums in the accumulation registers here: between tiles too, so that
// results are fetched from there one block at a time.
template <int PB, int QB>
__device__ __forceinline__ void hold(f32x16_t (&acc)[PB][QB])
{
#pragma unroll
    for (int i = 0; i < PB; ++i)
#pragma unroll
        for (int j = 0; j < QB; ++j) asm volatile("" : "+a"(acc[i][j]));
}
template <int PB, int QB>
__device__ __forceinline__ void clear(f32x16_t (&acc)[PB][QB])
{
#pragma unroll
    for (int i = 0; i < PB; ++i)
#pragma unroll
        for (int j = 0; j < QB; ++j) acc[i][j] = f32x16_t{};
}

// The same by way of registers, for operands off 16 bytes: two stages.
template <typename T, typename P, typename Q, int PB, int QB, int THREADS>
__device__ __forceinline__ void steps_by_registers(P& first, Q& second, char* lds, int steps, int p0, int q0,
                                                   f32x16_t (&acc)[PB][QB])
{
    constexpr int kStage = P::kBytes + Q::kBytes;
    uint4 pv[P::kLoads], qv[Q::kLoads];
    auto fetch = [&](int s) {
        first.template fetch<T>(pv, s);
        second.template fetch<T>(qv, s);
    };
    auto put = [&](int s) {
        put_chunks<THREADS>(lds + (s & 1) * kStage, pv);
        put_chunks<THREADS>(lds + (s & 1) * kStage + P::kBytes, qv);
    };
    fetch(0);
    put(0);
    for (int s = 0; s < steps; ++s) {
        __syncthreads();
        const char* now = lds + (s & 1) * kStage;
        if (s + 1 < steps) fetch(s + 1);
#pragma unroll
        for (int part = 0; part < 4; ++part) {
            uint4 p[PB], q[QB];
#pragma unroll
            for (int j = 0; j < QB; ++j) q[j] = Q::part(now + P::kBytes, q0, j, part);
#pragma unroll
            for (int i = 0; i < PB; ++i) p[i] = P::part(now, p0, i, part);
#pragma unroll
            for (int i = 0; i < PB; ++i)
#pragma unroll
                for (int j = 0; j < QB; ++j)
                    acc[i][j] = mma32(p[i], q[j], acc[i][j], static_cast<const T*>(nullptr));
        }
        if (s + 1 < steps) put(s + 1);
    }
}

// The tiles of a workgroup.  find(t): the next one; prepare(work, t): its
// operands; store(acc, t).  By way of registers `steps` is their length, or 0:
// the work's.
template <typename T, bool DIRECT, typename P, typename Q, int PB, int QB, int RING, int THREADS, typename Tile,
          typename Find, typename Prepare, typename Store>
__device__ __forceinline__ void tiles(char* lds, int p0, int q0, Find find, Prepare prepare, Store store, int steps)
{
    Tile t;
    if (!find(t)) return;
    f32x16_t acc[PB][QB];
    if constexpr (DIRECT) {
        Tile nt;
        Work<P, Q> w, nw;
        Steps<T, P, Q, PB, QB, RING> ring(lds, p0, q0);
        prepare(w, t);
        ring.begin(w);
        bool more = true;
        clear(acc);
        for (;;) {
            // behind the last tile its own first steps are loaded again, and
            // waited for, so that every tile runs the same code
            ring.tile(acc, w, nw, [&](Work<P, Q>& next) {
                nt = t;
                Tile found;
                more = find(found);
                if (more) nt = found;
                prepare(next, nt);
            });
            hold(acc);
            store(acc, t);
            if (!more) break;
            clear(acc);
            hold(acc);
            w = nw;
            t = nt;
        }
        wait_barrier();
    } else {
        do {
            Work<P, Q> w;
            prepare(w, t);
            clear(acc);
            steps_by_registers<T, P, Q, PB, QB, THREADS>(w.p, w.q, lds, steps > 0 ? steps : w.steps, p0, q0, acc);
            store(acc, t);
            __syncthreads();
        } while (find(t));
    }
}

// ---- results

// Two packed pairs of 16-bit results.
template <typename T>
__device__ __forceinline__ uint2 pack4(float a, float b, float c, float d)
{
    typedef std::conditional_t<std::is_same_v<T, Bf16>, bf16x2_t, fp16x2_t> pair;
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), pair)),
                      __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{c, d}), pair)));
}

// A 32 x 32 block: this lane's output row `row` (at its column 0), columns
// col .. of `cols`.  A lane holds runs of 4 columns, 4 (l / 32) + 8 i; lanes
// l and l + 32 hold the two halves of the same row and trade them, so that
// each stores runs of 8.
template <typename T, typename F>
__device__ __forceinline__ void put_block(const f32x16_t& v, F chunk_at)
{
    // chunk_at(c): where the 8 columns from c on go
    const int h = (opaque(threadIdx.x) >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint2 a = pack4<T>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        const uint2 b = pack4<T>(v[4 * i + 4], v[4 * i + 5], v[4 * i + 6], v[4 * i + 7]);
        const auto x = __builtin_amdgcn_permlane32_swap(a.x, b.x, false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(a.y, b.y, false, false);
        *reinterpret_cast<uint4*>(chunk_at(8 * i + 8 * h)) = make_uint4(x[0], y[0], x[1], y[1]);
    }
}
// 8 columns from c on, of `cols`, of a row.
template <typename T>
__device__ __forceinline__ void store_chunk(const uint4& q, T* row, int64_t c, int64_t cols)
{
    if (c + 8 <= cols) {
        __builtin_memcpy(row + c, &q, 16);
    } else if (c < cols) {
        uint64_t lo = q.x | (uint64_t)q.y << 32, hi = q.z | (uint64_t)q.w << 32;
#pragma clang loop unroll(disable)
        for (int64_t k = c; k < cols; ++k) {
            row[k] = T{(uint16_t)lo};
            lo = lo >> 16 | hi << 48;
            hi >>= 16;
        }
    }
}
template <typename T>
__device__ __forceinline__ void store_block(const f32x16_t& v, T* row, int64_t col, int64_t cols, bool live)
{
    const int h = (opaque(threadIdx.x) >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint2 a = pack4<T>(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        const uint2 b = pack4<T>(v[4 * i + 4], v[4 * i + 5], v[4 * i + 6], v[4 * i + 7]);
        const auto x = __builtin_amdgcn_permlane32_swap(a.x, b.x, false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(a.y, b.y, false, false);
        if (live) store_chunk(make_uint4(x[0], y[0], x[1], y[1]), row, col + 8 * i + 8 * h, cols);
    }
    __builtin_amdgcn_sched_barrier(0);      // one block's values at a time
}
__device__ __forceinline__ void store_block(const f32x16_t& v, float* row, int64_t col, int64_t cols, bool live)
{
    const int h = (opaque(threadIdx.x) >> 5) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t c = col + 8 * i + 4 * h;
        if (live && c + 4 <= cols) {
            const f32x4_t q = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
            __builtin_memcpy(row + c, &q, 16);
        } else if (live) {
#pragma unroll
            for (int k = 0; k < 3; ++k)
                if (c + k < cols) row[c + k] = v[4 * i + k];
        }
    }
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace ep

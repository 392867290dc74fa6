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
#pragma once

#include <type_traits>

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

// 16 bytes a lane from global memory to LDS, from base + off: lane l's go to
// lds + AT + 16 l.  The compiler does not count these loads: wait_barrier()
// waits for them.
template <int AT>
__device__ __forceinline__ void load_lds(uint32_t lds, const char* base, uint32_t off)
{
    asm volatile("s_add_u32 m0, %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3"
                 :
                 : "s"(lds), "n"(AT), "v"(off), "s"(base)
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
        const int t = threadIdx.x;
        base = from;
        bytes = length;
        chunk = (t & 7) ^ turn(t / 8);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = off_of(t / 8 + i * kRowStep) + chunk * 16;
    }
    // This thread's I-th chunk of step s into LDS.
    template <int I>
    __device__ __forceinline__ void load(uint32_t lds, int s) const
    {
        if constexpr (sizeof(OFF) == 4) load_lds<I * THREADS * 16>(lds, base + (int64_t)s * 128, off[I]);
        else load_lds_or_zero<I * THREADS * 16>(lds, base + (int64_t)s * 128, off[I], true);
    }
    // The same for a step that may be the last, of a reduction that is a whole
    // number of chunks.
    template <int I>
    __device__ __forceinline__ void load_end(uint32_t lds, int s) const
    {
        load_lds_or_zero<I * THREADS * 16>(lds, base + (int64_t)s * 128, off[I], s * 128 + chunk * 16 < bytes);
    }
    __device__ __forceinline__ void found() const {}
    // By way of registers, for rows that do not start on 16 bytes or do not
    // end with a chunk.
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int s) const
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            v[i] = fetch16<T>(base + (int64_t)s * 128 + off[i], (bytes - s * 128 - chunk * 16) / 2);
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
// steps) by COLS columns.  With GATHER the rows are picked by an index each.
template <int COLS, int THREADS, bool GATHER = false, typename OFF = uint32_t>
struct ColOperand {
    static constexpr int kChunks = COLS / 8;
    static constexpr int kLoads = 64 * kChunks / THREADS;
    static constexpr int kBytes = 64 * COLS * 2;
    static constexpr int kRowStep = THREADS / kChunks;  // a multiple of 4: the turn is the same for all
    static constexpr int kSide = 64 / kChunks;          // rows a wavefront loads at a time
    static_assert(kRowStep % 4 == 0, "rows of a thread share their turn");
    typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;
    const char* base;
    OFF off[kLoads];
    int64_t ld;                 // bytes
    int row, rows;              // of the tile this thread's first; of the reduction
    int valid;                  // elements of its chunk that are there
    int wave_row;
    scalar_ptr index;           // GATHER: of the reduction's rows, below `bound`
    int64_t bound;
    int next[GATHER ? kLoads : 1][kSide];   // of the coming step's rows

    // `count` rows, `stride` bytes apart, from `from` on (GATHER: picked by
    // `pick`, below `limit`); columns first .. of `cols`.
    __device__ __forceinline__ void init(const char* from, int64_t stride, int count, int64_t first, int64_t cols,
                                         const int32_t* pick = nullptr, int64_t limit = 0)
    {
        const int t = threadIdx.x, p = t % kChunks;
        row = t / kChunks;
        wave_row = __builtin_amdgcn_readfirstlane(row);
        base = from;
        ld = stride;
        rows = count;
        index = (scalar_ptr)pick;
        bound = limit;
        const int64_t c = first + ((((p >> 2) ^ (row & 3)) << 2) | (p & 3)) * 8;
        valid = c + 8 <= cols ? 8 : c < cols ? (int)(cols - c) : 0;
        const OFF column = valid > 0 ? (OFF)c * 2 : 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) off[i] = (GATHER ? 0 : (OFF)((row + i * kRowStep) * ld)) + column;
        if constexpr (GATHER) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) find(0, i);
        }
    }
    // GATHER: the indices are read ahead, by scalar loads, whose waiting does
    // not touch the loads into LDS.
    __device__ __forceinline__ void find(int s, int i)
    {
#pragma unroll
        for (int j = 0; j < kSide; ++j) {
            const int in = s * 64 + wave_row + i * kRowStep + j;
            next[i][j] = index[in < rows ? in : 0];
        }
    }
    // Makes the compiler wait for them here.
    __device__ __forceinline__ void found()
    {
        if constexpr (GATHER) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
#pragma unroll
                for (int j = 0; j < kSide; ++j) asm volatile("" : "+s"(next[i][j]));
        }
    }
    // The offset of this thread's i-th row of the coming step, from `base`;
    // reads the index after it.
    __device__ __forceinline__ uint32_t gathered(int s, int i)
    {
        uint32_t o = 0;
#pragma unroll
        for (int j = 0; j < kSide; ++j) {
            const int r = next[i][j];
            const uint32_t at = r < 0 || r >= bound ? 0u : (uint32_t)r * (uint32_t)ld;
            o = j == 0 || (int)(threadIdx.x & 63) / kChunks == j ? at : o;
        }
        find(s + 1, i);
        return o;
    }
    template <int I>
    __device__ __forceinline__ void load(uint32_t lds, int s)
    {
        if constexpr (GATHER) load_lds<I * THREADS * 16>(lds, base, gathered(s, I) + off[I]);
        else load_lds<I * THREADS * 16>(lds, base + s * 64 * ld, off[I]);
    }
    template <int I>
    __device__ __forceinline__ void load_end(uint32_t lds, int s)
    {
        const bool live = s * 64 + row + I * kRowStep < rows;
        if constexpr (GATHER) load_lds_or_zero<I * THREADS * 16>(lds, base, gathered(s, I) + off[I], live);
        else load_lds_or_zero<I * THREADS * 16>(lds, base + s * 64 * ld, off[I], live);
    }
    template <typename T>
    __device__ __forceinline__ void fetch(uint4 (&v)[kLoads], int s)
    {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int in = s * 64 + row + i * kRowStep;
            const char* from = base + (int64_t)s * 64 * ld + off[i];
            if constexpr (GATHER) {
                const int r = index[in < rows ? in : 0];
                from = base + (r < 0 || r >= bound ? 0 : r * ld) + off[i];
            }
            v[i] = fetch16<T>(from, in < rows ? valid : 0);
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

// A thread's chunks from registers to its operand's place in LDS.
template <int THREADS, int LOADS>
__device__ __forceinline__ void put_chunks(char* lds, const uint4 (&v)[LOADS])
{
#pragma unroll
    for (int i = 0; i < LOADS; ++i) *reinterpret_cast<uint4*>(lds + (i * THREADS + threadIdx.x) * 16) = v[i];
}

// ---- the steps

// A tile's steps: PB x QB blocks of 32 x 32 per wavefront over the reduction,
// 128 bytes of it a step, from LDS.
//
// The two operands' tiles of a step take turns in a ring of RING places
// (P of step 0, Q of 0, P of 1, ...; with 5 places of 32 KiB all of LDS): an
// odd ring keeps more than a step in flight where LDS does not hold three.
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
struct Steps {
    static constexpr int kPlace = P::kBytes > Q::kBytes ? P::kBytes : Q::kBytes;
    static constexpr int kMuls = PB * QB, kReads = PB + QB;
    static constexpr int kLds = kPlace * RING;
    static constexpr int kLoads = P::kLoads + Q::kLoads;
    static constexpr bool kOdd = RING % 2 == 1;
    // loads that may be under way when a step changes: those of the tiles
    // behind the next step's
    static constexpr int kLeft = (RING - 4) / 2 * kLoads + (kOdd ? P::kLoads : 0);
    static_assert(RING >= 4, "two steps at least");

    P& first;
    Q& second;
    char* lds;
    uint32_t at;
    int p0, q0, steps;
    uint4 p[2][PB], q[2][QB];

    __device__ __forceinline__ Steps(P& a, Q& b, char* shared, int p_row, int q_row, int num_steps)
        : first(a), second(b), lds(shared), p0(p_row), q0(q_row), steps(num_steps)
    {
        at = lds_address(lds) + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) * 1024;
    }

    __device__ __forceinline__ static int place(int v) { return v >= RING * kPlace ? v - RING * kPlace : v; }

    // The I-th load of those that go out from step s's last part on, into the
    // places of step s: `now` (P) and behind it (Q).
    template <int I, bool END>
    __device__ __forceinline__ void load_one(int s, int now)
    {
        if constexpr (kOdd) {
            // Q's next tile falls on P's place and comes first
            if constexpr (I < Q::kLoads) {
                const int to = s + RING / 2;
                if constexpr (END) {
                    if (to < steps) second.template load_end<I>(at + now, to);
                } else {
                    second.template load<I>(at + now, to);
                }
            } else {
                const int to = s + RING / 2 + 1;
                if constexpr (END) {
                    if (to < steps) first.template load_end<I - Q::kLoads>(at + place(now + kPlace), to);
                } else {
                    first.template load<I - Q::kLoads>(at + place(now + kPlace), to);
                }
            }
        } else {
            const int to = s + RING / 2;
            if constexpr (I < P::kLoads) {
                if constexpr (END) {
                    if (to < steps) first.template load_end<I>(at + now, to);
                } else {
                    first.template load<I>(at + now, to);
                }
            } else {
                if constexpr (END) {
                    if (to < steps) second.template load_end<I - P::kLoads>(at + place(now + kPlace), to);
                } else {
                    second.template load<I - P::kLoads>(at + place(now + kPlace), to);
                }
            }
        }
    }
    template <int I, int UPTO, bool END>
    __device__ __forceinline__ void load_some(int s, int now)
    {
        if constexpr (I < UPTO) {
            load_one<I, END>(s, now);
            load_some<I + 1, UPTO, END>(s, now);
        }
    }

    template <int R>
    __device__ __forceinline__ void read_one(int set, int now, int part)
    {
        if constexpr (R < QB) q[set][R] = Q::part(lds + place(now + kPlace), q0, R, part);
        else p[set][R - QB] = P::part(lds + now, p0, R - QB, part);
    }
    template <int R, int UPTO>
    __device__ __forceinline__ void read_some(int set, int now, int part)
    {
        if constexpr (R < UPTO) {
            read_one<R>(set, now, part);
            read_some<R + 1, UPTO>(set, now, part);
        }
    }

    // Matrix instruction M of a part and what takes its turn after it: reads of
    // part `next` of the step at `then` into the other set, and the SHARE-th
    // quarter of the loads that follow step s at `now`.  LOADS: 0 none, 1 of
    // full steps, 2 of steps that may be the last or behind it.
    template <int SET, bool READ, int LOADS, int SHARE, int M = 0>
    __device__ __forceinline__ void part(f32x16_t (&acc)[PB][QB], int then, int next, int s, int now)
    {
        if constexpr (M < kMuls) {
            constexpr int i = M / QB, j = M % QB;
            acc[i][j] = mma32(p[SET][i], q[SET][j], acc[i][j], static_cast<const T*>(nullptr));
            if constexpr (READ) {
                // all reads within the first three quarters
                constexpr int kFrom = kReads * M * 4 / (kMuls * 3), kTo = kReads * (M + 1) * 4 / (kMuls * 3);
                read_some<(kFrom < kReads ? kFrom : kReads), (kTo < kReads ? kTo : kReads)>(SET ^ 1, then, next);
            }
            if constexpr (LOADS != 0) {
                constexpr int kOf = kLoads * SHARE / 4, kCount = kLoads * (SHARE + 1) / 4 - kOf;
                load_some<kOf + kCount * M / kMuls, kOf + kCount * (M + 1) / kMuls, LOADS == 2>(s, now);
            }
            __builtin_amdgcn_sched_barrier(0);
            part<SET, READ, LOADS, SHARE, M + 1>(acc, then, next, s, now);
        }
    }

    // Step s, whose P lies at `now`.  REST, MORE: the loads that go out in its
    // first three parts and its last (as LOADS of part()); LEFT: loads that may
    // be under way when it changes; NEXT: another step follows.
    template <int REST, int MORE, int LEFT, bool NEXT>
    __device__ __forceinline__ void step(f32x16_t (&acc)[PB][QB], int s, int now)
    {
        const int before = now - 2 * kPlace < 0 ? now + (RING - 2) * kPlace : now - 2 * kPlace;
        const int then = place(now + 2 * kPlace);
        part<0, true, REST, 1>(acc, now, 1, s - 1, before);
        part<1, true, REST, 2>(acc, now, 2, s - 1, before);
        part<0, true, REST, 3>(acc, now, 3, s - 1, before);
        if constexpr (NEXT) wait_barrier<LEFT>();
        if constexpr (MORE != 0) {
            first.found();
            second.found();
        }
        part<1, NEXT, MORE, 0>(acc, then, 0, s, now);
    }

    // full: steps that are whole (all, or all but the last).
    __device__ __forceinline__ void run(f32x16_t (&acc)[PB][QB], int full)
    {
        constexpr int kLast = (RING - 1) / 2;       // the last tile in the ring belongs to this step from now
        constexpr int kAhead = (RING + 1) / 2;      // the last load that follows a step to this one
        start<0>();
        if (steps > kLast) wait_barrier<(RING - 2) / 2 * kLoads + (kOdd ? P::kLoads : 0)>();
        else wait_barrier();
        read_some<0, kReads>(0, 0, 0);
        int s = 0, now = 0;
        auto turn = [&] {
            ++s;
            now = place(now + 2 * kPlace);
        };
        if (steps > kLast) {
            step<0, 2, kLeft, true>(acc, s, now);
            turn();
            for (; s + kAhead < full; turn()) step<1, 1, kLeft, true>(acc, s, now);
            for (; s + kLast < steps; turn()) step<2, 2, kLeft, true>(acc, s, now);
        }
        for (; s + 1 < steps; turn()) step<2, 2, 0, true>(acc, s, now);
        step<0, 0, 0, false>(acc, s, now);
    }
    template <int U>
    __device__ __forceinline__ void start()
    {
        if constexpr (U < RING) {
            if (U / 2 < steps) {
                if constexpr (U % 2 == 0) all<0, P>(first, U * kPlace, U / 2);
                else all<0, Q>(second, U * kPlace, U / 2);
            }
            start<U + 1>();
        }
    }
    template <int I, typename O>
    __device__ __forceinline__ void all(O& o, int to, int s)
    {
        if constexpr (I < O::kLoads) {
            o.template load_end<I>(at + to, s);
            all<I + 1, O>(o, to, s);
        }
    }
};

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

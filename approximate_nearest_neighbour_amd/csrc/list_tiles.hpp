// Tiles of products of 16-bit and 32-bit rows: the kernel that the products per
// list, their gradient and the adapters share.
//
// A workgroup of MW x NW waves forms a tile of TM x TN sums, each wave WM x WN
// blocks of 32 x 32 in registers, from chunks of KS values of the contraction.
// Both operands' chunks go through LDS, the next while one is multiplied.
//
// An operand's rows either run along the contraction ("along": x, and matrices
// [n][d]) or across it ("across": matrices [d][n], and both operands of the
// matrices' gradient, whose contraction runs over rows).  In LDS
//   along:  TM (or TN) lines of KS values; a matrix instruction's operand is one
//           16-byte read of a lane,
//   across: KS lines of TM (TN) values; the transposing reads of gfx950 bring
//           four values along the contraction to a lane, two of them an operand.
// The 16-byte blocks of a line are permuted by an exclusive or with bits of the
// line's number, so that lanes that read together touch every bank equally.
//
// float32 values are split into three bfloat16 parts, x = hi + mid + lo, each the
// nearest to what the parts before leave: |mid| <= 2^-8 |x|, |lo| <= 2^-16 |x|, and
// the three hold all 24 bits.  A product is the sum of six of the nine part products,
// the smallest first; the three dropped, mid lo, lo mid and lo lo, are below 2^-23 of
// it together (2^-25 on average), so that a sum of products is as near as float32's
// own: 512 x 512 results of 2048 random products are off by 7.0e-7 of their norm, the
// library's float32 product by 8.1e-7.  Six bfloat16 instructions take 6 / 16 of the
// time of the float32 one.  What rounds to an infinity in bfloat16 (magnitudes from
// 255.5 2^120 on) becomes a NaN this way; below 2^-110 the third part is one of
// bfloat16's numbers below the normal ones, which are multiples of 2^-133.
#pragma once

#include "list_plan.hpp"
#include "rows.hpp"
#include "rows_internal.hpp"
#include "tile_ops.hpp"

#include <algorithm>
#include <type_traits>

namespace ivfpq {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// What a tile kernel forms.
enum ListForm {
    kRowsAlong,  // rows per list times matrices [n][d]
    kRowsAcross, // rows per list times matrices [d][n]
    kGradient,   // per list, the sum of outer products of two rows
    kHidden,     // rows per list times down matrices, to the adapters' hidden rows
    kAdapter     // rows times one matrix [n][d], and hidden rows times up matrices
};

template <int FORM>
struct FormOf {
    static constexpr bool A_ALONG = FORM != kGradient;
    static constexpr bool B_ALONG = FORM == kRowsAlong || FORM == kHidden || FORM == kAdapter;
    static constexpr bool PER_LIST_ROWS = FORM == kRowsAlong || FORM == kRowsAcross ||
                                          FORM == kHidden;
};

template <typename T>
struct Parts { // planes in LDS and the type of the matrix instructions' operands
    static constexpr int N = 1;
    using E = T;
};
template <>
struct Parts<float> {
    static constexpr int N = 3;
    using E = __bf16;
};

template <typename E>
__device__ __forceinline__ f32x16 mfma16(s16x8 a, s16x8 b, f32x16 c)
{
    typedef E V __attribute__((ext_vector_type(8)));
    if constexpr (std::is_same<E, __bf16>::value)
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V, a),
                                                       __builtin_bit_cast(V, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V, a),
                                                      __builtin_bit_cast(V, b), c, 0, 0, 0);
}

// The part of the rows that tile number `slot` lies in, and its rows: list e (-1 or
// nlist: rows of no list), rows [p0, p1) (none: an empty number).  64 parts a step.
struct PartTile {
    int e;
    int64_t p0, p1;
};

__device__ __forceinline__ PartTile find_part(const int32_t *offsets, int nlist, int64_t rows,
                                              int64_t slot, int tm, bool by_row)
{
    const int lane = lane_id(), from = first_part(offsets);
    int first = 0, count = nlist + 2;
    while (count > 1) {
        const int step = (count + 63) / 64;
        const int i = first + lane * step;
        const bool upto = i < first + count &&
                          part_slot(part_begin(offsets, nlist, rows, i), i - from, tm, by_row) <= slot;
        const uint64_t m = __ballot(upto);
        const int who = m ? 63 - __builtin_clzll(m) : 0;
        const int left = count - who * step;
        first += who * step;
        count = left < step ? left : step;
    }
    first = __builtin_amdgcn_readfirstlane(first);
    const int64_t begin = part_begin(offsets, nlist, rows, first);
    const int64_t end = part_begin(offsets, nlist, rows, first + 1);
    const int64_t p0 = slot_row(slot, begin, end, first - from, tm, by_row);
    return {first - 1, p0, min(p0 + tm, end)};
}

// A tile's operand in LDS: LINES lines of LEN 16-bit values a plane.
template <bool ALONG, int SIZE, int KS>
struct Place {
    static constexpr int LINES = ALONG ? SIZE : KS, LEN = ALONG ? KS : SIZE;
    static constexpr int BLOCKS = LEN / 8;               // 16-byte blocks of a line
    static constexpr int PER256 = BLOCKS >= 16 ? 1 : 16 / BLOCKS; // lines in 256 bytes
    static constexpr int PLANE = LINES * LEN * 2;        // bytes
    // Where block b of a line stands.  Along: lanes read one block of 16 lines in a
    // row, which the exclusive or spreads over the 256 bytes of all banks.  Across:
    // they read 64 bytes of lines 4 i to 4 i + 3, which go to the four quarters.
    __device__ __forceinline__ static int swizzle(int line)
    {
        if constexpr (ALONG)
            return (line / PER256) & (BLOCKS - 1);
        else
            return PER256 == 1 ? (line & 3) << 2 : ((line >> 1) & 1) << 2;
    }
    __device__ __forceinline__ static int at(int line, int block)
    {
        return line * LEN * 2 + ((block ^ swizzle(line)) * 16);
    }
};

// Offsets of a lane's operand reads.  Row r of a block of 32 is `first + r`,
// or dealt (deal_row) where PAIR.
template <bool ALONG, int SIZE, int KS, int COUNT, bool PAIR>
struct Reader {
    using P = Place<ALONG, SIZE, KS>;
    int off[ALONG ? KS / 16 : COUNT];

    __device__ __forceinline__ void init(int first)
    {
        const int lane = lane_id(), half = lane >> 5;
        if constexpr (ALONG) {
            const int row = deal_row<PAIR>(lane & 31);
#pragma unroll
            for (int s = 0; s < KS / 16; ++s)
                off[s] = P::at(first + row, 2 * s + half);
        } else {
            // lanes 16 g + 4 j + q bring line 8 half + j, four values from 16 (g & 1) + 4 q on
            const int j = (lane >> 2) & 3, q = lane & 3;
            const int quad = PAIR ? ((q & 1) << 1) | (q >> 1) : q;
            const int line = half * 8 + j;
#pragma unroll
            for (int i = 0; i < COUNT; ++i) {
                const int value = first + i * 32 + ((lane >> 4) & 1) * 16 + quad * 4;
                off[i] = P::at(line, value / 8) + (value & 4) * 2;
            }
        }
    }
    // the operand of block i and step s
    __device__ __forceinline__ s16x8 read(const uint8_t *plane, int i, int s) const
    {
        if constexpr (ALONG) {
            // blocks of 32 lines keep the permutation: it depends on the line modulo 32
            return *reinterpret_cast<const s16x8 *>(plane + off[s] + i * 32 * P::LEN * 2);
        } else {
            typedef __attribute__((address_space(3))) s16x4 L4;
            const uint8_t *p = plane + off[i] + s * 16 * P::LEN * 2;
            const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L4 *)p);
            const s16x4 hi =
                __builtin_amdgcn_ds_read_tr16_b64_v4i16((L4 *)(p + 4 * P::LEN * 2));
            return s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        }
    }
};

// Eight values of a line in registers.  ODD: 16-bit values whose place may not be a
// multiple of four bytes, where loads of 16 bytes take twice as long: the aligned four
// bytes that hold them are read (which end in the same four bytes as the values do)
// and shifted together when they have arrived (`ready`).  The blocks of few rows take
// it, which wait for their loads (128 rows of 2001 x 2001 with adapters of rank 16: 48 us
// without, 31 so); the tiles through registers do not, as theirs are two chunks ahead (16,384
// rows of 16 lists of 1501 x 1001: 130 us, so 153).
template <typename T, bool ODD = false>
struct Eight {
    static_assert(!ODD || sizeof(T) == 2, "four-byte values are aligned");
    static constexpr int Q = sizeof(T) / 2; // 16-byte pieces
    typedef T V __attribute__((ext_vector_type(8 / Q), aligned(sizeof(T))));
    typedef uint32_t Words __attribute__((ext_vector_type(4 * Q)));
    Words v;
    uint32_t last, shift; // ODD

    __device__ __forceinline__ void read(const T *p)
    {
        if constexpr (ODD) {
            typedef uint32_t W4 __attribute__((ext_vector_type(4), aligned(4)));
            const uint32_t half = (uint32_t)(uintptr_t)p & 2;
            const uint8_t *from = reinterpret_cast<const uint8_t *>(p) - half;
            v = *reinterpret_cast<const W4 *>(from);
            last = *reinterpret_cast<const uint32_t *>(from + 12 + 2 * half);
            shift = 8 * half;
        } else {
#pragma unroll
            for (int h = 0; h < Q; ++h) {
                const u32x4 w = __builtin_bit_cast(u32x4, reinterpret_cast<const V *>(p)[h]);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[h * 4 + i] = w[i];
            }
        }
    }
    // once after read, before anything else
    __device__ __forceinline__ void ready()
    {
        if constexpr (ODD) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = __builtin_amdgcn_alignbit(i < 3 ? v[(i + 1) & 3] : last, v[i], shift);
        }
    }
    __device__ __forceinline__ void keep(bool there) // or all zero
    {
#pragma unroll
        for (int i = 0; i < 4 * Q; ++i)
            v[i] = there ? v[i] : 0u;
    }
    // The eight values from number `at` of an array of `all` on, in two steps, so that
    // loads are under way together and no branch waits for one.  Near the array's end
    // its last eight are read, and moved down when they are stored.  TINY: the array may
    // have fewer than eight.
    template <bool TINY>
    __device__ __forceinline__ void read_near(const T *array, int64_t at, int64_t all)
    {
        if constexpr (!TINY) {
            read(array + min(at, all - 8));
        } else {
            T x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = array[min(at + i, all - 1)];
#pragma unroll
            for (int i = 0; i < 4 * Q; ++i) {
                if constexpr (Q == 1)
                    v[i] = (uint32_t)__builtin_bit_cast(uint16_t, x[2 * i]) |
                           (uint32_t)__builtin_bit_cast(uint16_t, x[2 * i + 1]) << 16;
                else
                    v[i] = __builtin_bit_cast(uint32_t, x[i]);
            }
            last = v[3];
            shift = 0;
        }
    }
    // ... of which the first `count` are kept, the others zero.
    template <bool TINY>
    __device__ __forceinline__ void settle(int64_t at, int64_t all, int count)
    {
        if constexpr (!TINY) {
            const int past = (int)min(at - min(at, all - 8), (int64_t)8);
            if (__any(past > 0)) {
#pragma unroll
                for (int b = 8; b >= 1; b >>= 1) {
                    const bool move = past & b;
                    if constexpr (Q == 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t up = b == 1 ? (v[i] >> 16 | (i < 3 ? v[(i + 1) & 3] << 16 : 0))
                                                : i + b / 2 < 4 ? v[(i + b / 2) & 3] : 0u;
                            v[i] = move ? up : v[i];
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            v[i] = move ? (i + b < 8 ? v[(i + b) & 7] : 0u) : v[i];
                    }
                }
            }
        }
        const int n = min(max(count, 0), 8);
#pragma unroll
        for (int i = 0; i < 4 * Q; ++i) {
            if constexpr (Q == 1)
                v[i] &= n >= 2 * i + 2 ? ~0u : n == 2 * i + 1 ? 0xFFFFu : 0u;
            else
                v[i] = i < n ? v[i] : 0u;
        }
    }
    // float32 values to their three parts, two at a time: a conversion rounds two values, and
    // the rounded ones are the upper halves of float32 numbers
    __device__ __forceinline__ void split(u32x4 (&out)[3]) const
    {
        typedef float F2 __attribute__((ext_vector_type(2)));
        typedef __bf16 B2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            F2 x = {__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])};
#pragma unroll
            for (int p = 0; p < 3; ++p) {
                const uint32_t near =
                    __builtin_bit_cast(uint32_t, __builtin_convertvector(x, B2));
                out[p][i] = near;
                x[0] -= __uint_as_float(near << 16);
                x[1] -= __uint_as_float(near & 0xFFFF0000u);
            }
        }
    }
    // to the planes at `to`, `plane` bytes apart
    __device__ __forceinline__ void store(uint8_t *to, int plane) const
    {
        if constexpr (Q == 1) {
            *reinterpret_cast<Words *>(to) = v;
        } else {
            u32x4 out[3];
            split(out);
#pragma unroll
            for (int p = 0; p < 3; ++p)
                *reinterpret_cast<u32x4 *>(to + p * plane) = out[p];
        }
    }
};

// One product; the launchers fill it in.
struct ListJob {
    const void *a = nullptr, *b = nullptr; // first operand: rows; second: matrices (gradient: rows)
    void *out = nullptr;
    int64_t rows = 0;  // sorted rows (kAdapter: rows)
    int64_t arows = 0; // rows of the operand that `order` points into
    int m = 0;         // kGradient: rows of a matrix
    int n = 0;         // columns of the results
    int kdim = 0;      // contraction (kGradient: the list's rows instead)
    const int32_t *offsets = nullptr, *order = nullptr;
    FastDiv k;
    int nlist = 0;
    uint32_t mt = 0, nt = 0; // tiles along both sides (kGradient: mt of one list)
    bool by_row = false;
    const int32_t *by_size = nullptr; // kGradient: the lists, the longest first (nullptr: as they are)
    int splits = 1; // kGradient: workgroups that share a list's rows, a result each
    int64_t block0 = 0; // the launch's first workgroup
    // adapters: hidden rows (HiddenPlace; rp values each, r and zeros), the list of each row,
    // up matrices [nlist][n][r], scales [nlist] or nullptr
    void *hidden = nullptr;
    int32_t *row_list = nullptr;
    const int32_t *pos = nullptr;
    const void *up = nullptr;
    const float *scales = nullptr;
    int r = 0, rp = 0;
};

// Row of the gathered operand that sorted row p takes; -1 where there is none.
__device__ __forceinline__ int64_t source_row(const ListJob &p, int64_t row)
{
    if (!p.order)
        return row < p.arows ? row : -1;
    const int32_t slot = p.order[row];
    const int64_t q = slot >= 0 ? (int64_t)p.k.div((uint32_t)slot) : -1;
    return q < p.arows ? q : -1;
}

// Hidden rows in the workspace, as the matrix instructions' operands: blocks of 32 rows, in a
// block steps of 16 values, in a step two times 32 pieces of eight values, the rows' first
// and then their second ones.  16-bit types have three bfloat16 parts of each value, which
// hold float32's 24 bits (see above), a step's parts one after the other.
template <typename T>
struct HiddenPlace {
    using E = typename std::conditional<sizeof(T) == 4, float, __bf16>::type;
    static constexpr int PARTS = sizeof(T) == 4 ? 1 : 3;
    // values before row t's piece of eight from value `at` on (first part; 512 values a part)
    __device__ __forceinline__ static int64_t piece(int64_t t, int at, int rp)
    {
        return (t >> 5) * (rp * 32 * PARTS) + (at >> 4) * (512 * PARTS) + (at & 8) * 32 +
               (t & 31) * 8;
    }
    __device__ __forceinline__ static void put(void *hidden, int64_t t, int at, int rp, float h)
    {
        E *to = static_cast<E *>(hidden) + piece(t, at, rp) + (at & 7);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
            const E part = (E)h;
            to[q * 512] = part;
            h -= (float)part;
        }
    }
};
constexpr int kHiddenParts = 3; // as operands

// kHidden: the rows of a tile of no list have none.
__device__ __forceinline__ void no_list_rows(const ListJob &p, const PartTile &tile, bool first,
                                             int tid, int threads)
{
    for (int64_t row = tile.p0 + tid; first && row < tile.p1; row += threads) {
        const int64_t t = source_row(p, row);
        if (t >= 0)
            p.row_list[t] = -1;
    }
}

// Operands of the matrix instructions from eight values: the values, or their parts.
template <typename T, bool ODD>
__device__ __forceinline__ void operands_of(const Eight<T, ODD> &x, s16x8 (&out)[Parts<T>::N])
{
    if constexpr (sizeof(T) == 2) {
        out[0] = __builtin_bit_cast(s16x8, x.v);
    } else {
        u32x4 parts[3];
        x.split(parts);
#pragma unroll
        for (int p = 0; p < 3; ++p)
            out[p] = __builtin_bit_cast(s16x8, parts[p]);
    }
}

// What an up matrix's values become where they meet hidden rows, whose parts are bfloat16:
// bfloat16 ones stay, the 11 bits of binary16 ones are two bfloat16 parts, whose range
// holds theirs, float32 ones are three.
template <typename T>
struct UpParts {
    static constexpr int N = sizeof(T) == 4 ? 3 : std::is_same<T, _Float16>::value ? 2 : 1;
    template <bool ODD>
    __device__ __forceinline__ static void of(const Eight<T, ODD> &x, s16x8 (&out)[N])
    {
        if constexpr (N == 2) {
            typedef _Float16 H8 __attribute__((ext_vector_type(8)));
            typedef float F8 __attribute__((ext_vector_type(8)));
            typedef __bf16 B8 __attribute__((ext_vector_type(8)));
            const F8 v = __builtin_convertvector(__builtin_bit_cast(H8, x.v), F8);
            const B8 high = __builtin_convertvector(v, B8);
            out[0] = __builtin_bit_cast(s16x8, high);
            out[1] = __builtin_bit_cast(
                s16x8, __builtin_convertvector(v - __builtin_convertvector(high, F8), B8));
        } else {
            operands_of(x, out);
        }
    }
};

// A wave's hidden rows (not dealt: a lane has one column of sixteen rows), and the rows'
// lists.  `p0`, `n0`: the wave's first row and column.
template <typename T, int WM, int WN>
__device__ __forceinline__ void store_hidden(const ListJob &p, const PartTile &tile, int64_t p0,
                                             int n0, bool first, int threads,
                                             const f32x16 (&acc)[WM][WN])
{
    const int r = lane_id() & 31, half = lane_id() >> 5;
    const float scale = p.scales ? p.scales[tile.e] : 1.f;
    for (int64_t row = tile.p0 + threadIdx.x; first && row < tile.p1; row += threads) {
        const int64_t t = source_row(p, row);
        if (t >= 0)
            p.row_list[t] = tile.e;
    }
#pragma unroll
    for (int j = 0; j < WN; ++j) {
        const int col = n0 + j * 32 + r;
        if (col >= p.rp)
            continue;
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                const int64_t row = p0 + i * 32 + (q >> 2) * 8 + half * 4 + (q & 3);
                const int64_t t = row < tile.p1 ? source_row(p, row) : -1;
                if (t < 0)
                    continue;
                HiddenPlace<T>::put(p.hidden, t, col, p.rp,
                                    col < p.r ? acc[i][j][q] * scale : 0.f);
            }
    }
}

// The list of an adapter's row, as two loads that may be under way for long.
struct RowList {
    int32_t pos, e;
    __device__ __forceinline__ void load(const ListJob &p, int64_t row, int64_t end)
    {
        pos = row < end ? p.pos[row] : -1;
        e = row < end ? p.row_list[row] : -1;
    }
    // -1: none (a masked row's entry is whatever the workspace held)
    __device__ __forceinline__ int list(const ListJob &p) const
    {
        return (uint32_t)pos < (uint64_t)p.rows && (uint32_t)e < (uint32_t)p.nlist ? e : -1;
    }
};

// Offset of a load that reads nothing: past any range (ranges are below 2^31 bytes).
constexpr uint32_t kNowhere = 0x80000000u;

// A memory range of less than 2^31 bytes from byte `from` on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t range_of(const void *base, int64_t from,
                                                           int64_t bytes)
{
    from = uniform(from);
    const int64_t left = min(max(bytes - from, (int64_t)0), (int64_t)0x7FFFFFFF);
    const uint8_t *p = static_cast<const uint8_t *>(base) + from;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)uniform(left),
                                             0x00027000);
}

// A wave's first sums: each row's hidden row times the up matrix of the row's own list, while
// the first chunks of x and W are under way.  A block of 32 rows takes its lists one after
// the other, all its hidden rows times that list's up matrix, of which the list's
// rows keep the sums.  So nothing of one row, or of one list's matrices, reaches a row of
// another list, neither an infinity or NaN nor a rounding.  Blocks that have the same list
// alone share the up matrix's operands.  Hidden rows go from memory to registers, as
// their place is the operands'; rows of an up matrix would take 64 short pieces a load
// that way, and go through a part of LDS of the wave's own where the copies can read them.
// bfloat16, 8192 rows of 16 requests, 4096 x 4096, rank 64: 256 us, without any list 247
// (binary16, whose up matrices take two parts: 270 for one list of all rows, bfloat16 253).
// Every list among 32 rows costs its products anew: 4096 rows dealt one by one to 8 lists of
// rank 16 146 us, to 64 lists of rank 64 397, about 120 where a list's rows are together.
// `p0`, `n0`: the wave's first row and column; `rows`: of row i 32 + (lane & 31); `slab`:
// SLAB bytes of LDS (0: none).
template <typename T, int SLAB, bool PAIR, bool TINY, int WM, int WN>
__device__ __forceinline__ void adapter_sums(const ListJob &p, int64_t p0, int n0,
                                             const RowList (&rows)[WM], uint8_t *slab,
                                             f32x16 (&acc)[WM][WN])
{
    constexpr bool COPY = SLAB > 0;
    static_assert(!COPY || (sizeof(T) == 2 && SLAB >= WN * 32 * 64), "16-bit rows, 32 values");
    // values of an up matrix's rows brought together, hidden values loaded together
    constexpr int UPS = !COPY ? 16 : SLAB >= WN * 32 * 128 ? 64 : 32, STEPS = COPY ? 2 : 1;
    constexpr int GROUPS = UPS / 16 / STEPS, AHEAD = WM * WN < 8 ? GROUPS : 1; // registers
    using Up = Eight<T>;
    using Place = HiddenPlace<T>;
    const int lane = lane_id(), r = lane & 31, half = lane >> 5;
    const int64_t all_up = (int64_t)p.nlist * p.n * p.r;
    using Lines = ivfpq::Place<true, WN * 32, COPY ? UPS : 64>;
    Reader<true, WN * 32, COPY ? UPS : 64, WN, PAIR> reader;
    if constexpr (COPY)
        reader.init(0);
    Up u[WN]; // not COPY
    auto up_at = [&](int seg, int j, int at) { // columns past the last repeat it; not stored
        return ((int64_t)seg * p.n + min(n0 + j * 32 + deal_row<PAIR>(r), p.n - 1)) * p.r + at;
    };
    // values u0 on of list seg's matrix
    auto load_up = [&](int seg, int u0) {
        if constexpr (COPY) {
            const __amdgpu_buffer_rsrc_t range =
                range_of(p.up, ((int64_t)seg * p.n + n0) * p.r * 2, all_up * 2);
            wait_lds(); // the slab is read
#pragma unroll
            for (int c = 0; c < Lines::PLANE / 1024; ++c) {
                const int line = (c * 64 + lane) / Lines::BLOCKS;
                const int at = u0 + ((lane % Lines::BLOCKS) ^ Lines::swizzle(line)) * 8;
                copy16_to_lds(range, at < p.r ? (uint32_t)(line * p.r + at) * 2 : kNowhere, 0,
                              slab + c * 1024);
            }
        } else {
#pragma unroll
            for (int j = 0; j < WN; ++j)
                u[j].template read_near<TINY>(static_cast<const T *>(p.up),
                                              up_at(seg, j, u0 + half * 8), all_up);
        }
    };
    auto settle_up = [&](int seg, int u0) { // once after load_up
        if constexpr (COPY) {
            wait_vm<0>();
        } else {
#pragma unroll
            for (int j = 0; j < WN; ++j)
                u[j].template settle<TINY>(up_at(seg, j, u0 + half * 8), all_up,
                                           p.r - u0 - half * 8);
        }
    };
    // block i's hidden rows; past the last block, whose results are dropped, that one's
    struct Hiddens {
        Eight<typename Place::E> h[STEPS][Place::PARTS];
    };
    auto load_hidden = [&](Hiddens &to, int i, int k0) {
        const typename Place::E *from = static_cast<const typename Place::E *>(p.hidden) +
                                        Place::piece(min(p0 + i * 32, (p.rows - 1) & ~(int64_t)31),
                                                     0, p.rp) + lane * 8;
#pragma unroll
        for (int k = 0; k < STEPS; ++k)
#pragma unroll
            for (int q = 0; q < Place::PARTS; ++q)
                to.h[k][q].read(from +
                                (min(k0 + k * 16, p.rp - 16) / 16 * Place::PARTS + q) * 512);
    };
    // group g of the values from u0 on
    auto products = [&](const Hiddens &h, int u0, int g, f32x16 (&d)[WN]) {
#pragma unroll
        for (int k = 0; k < STEPS; ++k) {
            const int step = g * STEPS + k;
            if (u0 + step * 16 >= p.rp)
                break;
            s16x8 oh[kHiddenParts];
            if constexpr (Place::PARTS == 1)
                operands_of(h.h[k][0], oh);
            else
#pragma unroll
                for (int q = 0; q < kHiddenParts; ++q)
                    oh[q] = __builtin_bit_cast(s16x8, h.h[k][q].v);
#pragma unroll
            for (int j = 0; j < WN; ++j) {
                s16x8 ou[UpParts<T>::N];
                if constexpr (COPY) {
                    Up x;
                    x.v = __builtin_bit_cast(u32x4, reader.read(slab, j, step));
                    UpParts<T>::of(x, ou);
                } else {
                    UpParts<T>::of(u[j], ou);
                }
                // parts whose numbers add to 2, then 1, then 0
#pragma unroll
                for (int sum = kHiddenParts - 1; sum >= 0; --sum)
#pragma unroll
                    for (int q = 0; q <= sum; ++q)
                        if (sum - q < UpParts<T>::N)
                            d[j] = PAIR ? mfma16<__bf16>(ou[sum - q], oh[q], d[j])
                                        : mfma16<__bf16>(oh[q], ou[sum - q], d[j]);
            }
        }
    };
    // the sums' row of result q
    auto row_of = [&](int q) { return PAIR ? r : (q >> 2) * 8 + half * 4 + (q & 3); };

    int list[WM];
    uint32_t left[WM]; // a block's rows whose list is to come
#pragma unroll
    for (int i = 0; i < WM; ++i) {
        list[i] = rows[i].list(p);
        left[i] = (uint32_t)__ballot(list[i] >= 0);
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q)
                acc[i][j][q] = 0.f;
    }
    if constexpr (WM > 1) {
        const int seg = left[0] ? __builtin_amdgcn_readlane(list[0], __builtin_ctz(left[0])) : -1;
        bool same = seg >= 0;
#pragma unroll
        for (int i = 0; i < WM; ++i)
            same = same && left[i] == (uint32_t)__ballot(list[i] == seg);
        if (same) {
            for (int u0 = 0; u0 < p.rp; u0 += UPS) {
                Hiddens h[2];
                load_up(seg, u0);
                load_hidden(h[0], 0, u0);
                settle_up(seg, u0);
#pragma unroll
                for (int c = 0; c < GROUPS * WM; ++c) {
                    if (c + 1 < GROUPS * WM)
                        load_hidden(h[(c + 1) & 1], (c + 1) % WM, u0 + (c + 1) / WM * STEPS * 16);
                    products(h[c & 1], u0, c / WM, acc[c % WM]);
                }
            }
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j)
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        acc[i][j][q] = left[i] >> row_of(q) & 1 ? acc[i][j][q] : 0.f;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < WM; ++i) {
        while (left[i]) {
            const int seg = __builtin_amdgcn_readlane(list[i], __builtin_ctz(left[i]));
            const uint32_t mine = (uint32_t)__ballot(list[i] == seg);
            left[i] &= ~mine;
            f32x16 d[WN];
#pragma unroll
            for (int j = 0; j < WN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    d[j][q] = 0.f;
            for (int u0 = 0; u0 < p.rp; u0 += UPS) {
                Hiddens h[AHEAD];
                load_up(seg, u0);
#pragma unroll
                for (int g = 0; g < AHEAD; ++g)
                    load_hidden(h[g], i, u0 + g * STEPS * 16);
                settle_up(seg, u0);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    if (g >= AHEAD)
                        load_hidden(h[g % AHEAD], i, u0 + g * STEPS * 16);
                    products(h[g % AHEAD], u0, g, d);
                }
            }
#pragma unroll
            for (int j = 0; j < WN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[i][j][q] = mine >> row_of(q) & 1 ? d[j][q] : acc[i][j][q];
        }
    }
}

// Operands through registers, for float32 (split on the way to LDS) and for 16-bit rows
// that the copies cannot read.  Bound by the matrix instructions, six a product, and the
// split beside them in float32 (the gradient of 65,536 rows, 2048 x 2048: 3.5 ms, 158 TF,
// the library's float32 product 153), by the loads' latency where tiles are few (1554 odd
// rows of 16 lists of 1000 x 1501: 27 us, 16 chunks of two workgroups a CU).
template <typename T, typename TO, int FORM, int KS, int WM, int WN, int MW, int NW, bool TINY>
__global__ __launch_bounds__(64 * MW * NW, 2) void list_tile_kernel(ListJob p)
{
    using F = FormOf<FORM>;
    constexpr int WAVES = MW * NW, THREADS = 64 * WAVES, TM = 32 * WM * MW, TN = 32 * WN * NW;
    constexpr bool PAIR = sizeof(TO) == 2; // the second operand goes first (see deal_row)
    constexpr int NP = Parts<T>::N;
    using E = typename Parts<T>::E;
    using PA = Place<F::A_ALONG, TM, KS>;
    using PB = Place<F::B_ALONG, TN, KS>;
    constexpr int STAGE = NP * (PA::PLANE + PB::PLANE);
    __shared__ __align__(16) uint8_t stage0[STAGE], stage1[STAGE];

    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % MW, wn = wave / MW;
    const int64_t block = p.block0 + blockIdx.x;
    const uint32_t nt = (uint32_t)(block % p.nt);
    const int64_t mt = block / p.nt;
    const int n0 = (int)nt * TN;

    PartTile tile;
    int m0 = 0, split = 0;
    if constexpr (FORM == kGradient) {
        const int nth = (int)(mt / p.mt), list = nth / p.splits;
        split = nth - list * p.splits;
        const int e = p.by_size ? p.by_size[list] : list;
        m0 = (int)(mt - (int64_t)nth * p.mt) * TM;
        tile = {e, part_begin(p.offsets, p.nlist, p.rows, e + 1),
                part_begin(p.offsets, p.nlist, p.rows, e + 2)};
        split_rows(tile.p0, tile.p1, split, p.splits);
    } else if constexpr (FORM == kAdapter) {
        tile = {0, mt * TM, min(mt * TM + TM, p.rows)};
    } else {
        tile = find_part(p.offsets, p.nlist, p.rows, mt, TM, p.by_row);
        if (tile.p0 >= tile.p1)
            return;
    }
    tile.p0 = uniform(tile.p0);
    tile.p1 = uniform(tile.p1);
    const bool listed = FORM == kAdapter || (tile.e >= 0 && tile.e < p.nlist);
    const int64_t kdim = !listed ? 0 : FORM == kGradient ? max(tile.p1 - tile.p0, (int64_t)0)
                                                         : (int64_t)p.kdim;
    if (FORM == kHidden && !listed) {
        no_list_rows(p, tile, nt == 0, tid, THREADS);
        return;
    }

    const int64_t chunks = (kdim + KS - 1) / KS;

    f32x16 acc[WM][WN];
    if constexpr (FORM == kAdapter) {
        RowList lists[WM];
#pragma unroll
        for (int i = 0; i < WM; ++i)
            lists[i].load(p, tile.p0 + (wm * WM + i) * 32 + (lane & 31), tile.p1);
        adapter_sums<T, 0, PAIR, TINY>(p, tile.p0 + wm * WM * 32, n0 + wn * WN * 32, lists, nullptr,
                                       acc);
    } else {
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[i][j][q] = 0.f;
    }

    // pieces of eight values, a thread's own of both operands
    constexpr int QA = PA::LINES * PA::BLOCKS / THREADS, QB = PB::LINES * PB::BLOCKS / THREADS;
    static_assert(QA * THREADS == PA::LINES * PA::BLOCKS && QB * THREADS == PB::LINES * PB::BLOCKS,
                  "whole pieces a thread");
    const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
    int64_t arow[F::A_ALONG ? QA : 1];
    if constexpr (F::A_ALONG) {
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int64_t row = tile.p0 + (j * THREADS + tid) / PA::BLOCKS;
            arow[j] = row >= tile.p1 ? -1 : F::PER_LIST_ROWS ? source_row(p, row) : row;
        }
    }
    // kGradient: the slots of the next chunk's rows, a chunk ahead of the rows themselves
    int32_t slots[FORM == kGradient ? QB : 1];
    auto load_slots = [&](int64_t c) {
        if constexpr (FORM == kGradient) {
#pragma unroll
            for (int j = 0; j < QB; ++j) {
                const int64_t row = tile.p0 + min(c * KS + (j * THREADS + tid) / PB::BLOCKS, kdim - 1);
                slots[j] = p.order ? p.order[row] : (int32_t)row;
            }
        }
    };
    // Whether a chunk has a line's end or a line that is not there (a gather may find no
    // row); the others are read as they stand.
    const bool edge_a = F::A_ALONG ? tile.p1 - tile.p0 < TM || (F::PER_LIST_ROWS && p.order)
                                   : m0 + TM > p.m;
    const bool edge_b = FORM == kGradient || n0 + TN > p.n;

    // A chunk on its way: read at once, settled (ends, missing lines) when it goes to LDS.
    struct Chunk {
        Eight<T> a[QA], b[QB];
        int64_t at[FORM == kGradient ? QB : 1]; // kGradient: where b's pieces come from
        int count[FORM == kGradient ? QB : 1];
    };
    // Where a piece of a chunk begins in its array, and how many of its values there are:
    // the first chunk's place, and the same step for all pieces.
    struct Part {
        int64_t at;
        int count;
    };
    int64_t first_a[QA], first_b[QB];
#pragma unroll
    for (int j = 0; j < QA; ++j) {
        const int piece = j * THREADS + tid, line = piece / PA::BLOCKS;
        const int value = piece % PA::BLOCKS * 8;
        if constexpr (F::A_ALONG)
            first_a[j] = max(arow[j], (int64_t)0) * p.kdim + value;
        else
            first_a[j] = (tile.p0 + line) * p.m + m0 + value;
    }
#pragma unroll
    for (int j = 0; j < QB; ++j) {
        const int piece = j * THREADS + tid, line = piece / PB::BLOCKS;
        const int value = piece % PB::BLOCKS * 8;
        const int64_t list = F::PER_LIST_ROWS ? max(tile.e, 0) : 0;
        if constexpr (F::B_ALONG)
            first_b[j] = (list * p.n + min(n0 + line, p.n - 1)) * p.kdim + value;
        else
            first_b[j] = (list * p.kdim + line) * p.n + n0 + value;
    }
    const int64_t step_a = F::A_ALONG ? KS : (int64_t)KS * p.m;
    const int64_t step_b = F::B_ALONG ? KS : (int64_t)KS * p.n;
    auto part_a = [&](int64_t c, int j) -> Part {
        const int piece = j * THREADS + tid, line = piece / PA::BLOCKS;
        const int left = (int)(kdim - c * KS), value = piece % PA::BLOCKS * 8;
        if constexpr (F::A_ALONG)
            return {first_a[j] + c * step_a, arow[j] >= 0 ? left - value : 0};
        else
            return {first_a[j] + c * step_a, line < left ? p.m - m0 - value : 0};
    };
    auto part_b = [&](int64_t c, int j) -> Part { // all but kGradient
        const int piece = j * THREADS + tid, line = piece / PB::BLOCKS;
        const int left = (int)(kdim - c * KS), value = piece % PB::BLOCKS * 8;
        if constexpr (F::B_ALONG)
            return {first_b[j] + c * step_b, n0 + line < p.n ? left - value : 0};
        else
            return {first_b[j] + c * step_b, line < left ? p.n - n0 - value : 0};
    };
    const int64_t all_a = F::A_ALONG ? p.arows * p.kdim : p.rows * p.m;
    const int64_t all_b = FORM == kGradient ? p.arows * p.n
                                            : (FORM == kAdapter ? 1 : (int64_t)p.nlist) * p.n * p.kdim;
    auto load = [&](Chunk &to, int64_t c) {
#pragma unroll
        for (int j = 0; j < QA; ++j)
            to.a[j].template read_near<TINY>(a, part_a(c, j).at, all_a);
        if constexpr (FORM == kGradient) {
#pragma unroll
            for (int j = 0; j < QB; ++j) {
                const int piece = j * THREADS + tid;
                const uint32_t q = !p.order ? (uint32_t)slots[j]
                                   : slots[j] >= 0 ? p.k.div((uint32_t)slots[j]) : ~0u;
                const bool there =
                    q < (uint64_t)p.arows && c * KS + piece / PB::BLOCKS < kdim;
                to.at[j] = (there ? (int64_t)q : 0) * p.n + n0 + piece % PB::BLOCKS * 8;
                to.count[j] = there ? p.n - n0 - piece % PB::BLOCKS * 8 : 0;
                to.b[j].template read_near<TINY>(b, to.at[j], all_b);
            }
            load_slots(min(c + 1, chunks - 1));
        } else {
#pragma unroll
            for (int j = 0; j < QB; ++j)
                to.b[j].template read_near<TINY>(b, part_b(c, j).at, all_b);
        }
    };
    auto store = [&](Chunk &from, int64_t c, uint8_t *to) {
        const bool none = c >= chunks, last = (c + 1) * KS > kdim;
        if (last || edge_a || TINY) {
#pragma unroll
            for (int j = 0; j < QA; ++j) {
                const Part q = part_a(c, j);
                from.a[j].template settle<TINY>(q.at, all_a, q.count);
            }
        }
        if (last || edge_b || TINY) {
#pragma unroll
            for (int j = 0; j < QB; ++j) {
                Part q;
                if constexpr (FORM == kGradient)
                    q = {from.at[j], none ? 0 : from.count[j]};
                else
                    q = part_b(c, j);
                from.b[j].template settle<TINY>(q.at, all_b, q.count);
            }
        }
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int piece = j * THREADS + tid;
            from.a[j].store(to + PA::at(piece / PA::BLOCKS, piece % PA::BLOCKS), PA::PLANE);
        }
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int piece = j * THREADS + tid;
            from.b[j].store(to + NP * PA::PLANE + PB::at(piece / PB::BLOCKS, piece % PB::BLOCKS),
                            PB::PLANE);
        }
    };
    Reader<F::A_ALONG, TM, KS, WM, false> reada;
    Reader<F::B_ALONG, TN, KS, WN, PAIR> readb;
    reada.init(wm * WM * 32);
    readb.init(wn * WN * 32);

    // Whether chunk c has no value's end among what is read for results that are stored, nor
    // the array's own end: then it needs no settling but for lines that a gather does not
    // find, and its conversion, copies and the products of the chunk before are one
    // stretch without a branch, in which the compiler lays them side by side.
    auto plain = [&](int64_t c) {
        const int64_t k1 = (c + 1) * KS;
        bool fits = !TINY && k1 <= kdim;
        if constexpr (!F::A_ALONG)
            fits = fits && (tile.p0 + k1 - 1) * p.m + m0 + TM <= all_a;
        if constexpr (FORM == kGradient)
            fits = fits && n0 + TN <= p.n;
        else if constexpr (!F::B_ALONG)
            fits = fits && ((int64_t)tile.e * p.kdim + k1 - 1) * p.n + n0 + TN <= all_b;
        return fits;
    };
    auto store_plain = [&](Chunk &from, uint8_t *to) {
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int piece = j * THREADS + tid;
            if constexpr (F::PER_LIST_ROWS)
                from.a[j].keep(arow[j] >= 0);
            from.a[j].store(to + PA::at(piece / PA::BLOCKS, piece % PA::BLOCKS), PA::PLANE);
        }
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int piece = j * THREADS + tid;
            if constexpr (FORM == kGradient)
                from.b[j].keep(from.count[j] > 0);
            from.b[j].store(to + NP * PA::PLANE + PB::at(piece / PB::BLOCKS, piece % PB::BLOCKS),
                            PB::PLANE);
        }
    };
    auto multiply = [&](const uint8_t *now) {
#pragma unroll
        for (int s = 0; s < KS / 16; ++s) {
            s16x8 oa[NP][WM], ob[NP][WN];
#pragma unroll
            for (int q = 0; q < NP; ++q) {
#pragma unroll
                for (int i = 0; i < WM; ++i)
                    oa[q][i] = reada.read(now + q * PA::PLANE, i, s);
#pragma unroll
                for (int j = 0; j < WN; ++j)
                    ob[q][j] = readb.read(now + NP * PA::PLANE + q * PB::PLANE, j, s);
            }
            // parts whose numbers add to 2, then 1, then 0
#pragma unroll
            for (int sum = NP - 1; sum >= 0; --sum)
#pragma unroll
                for (int q = 0; q <= sum; ++q)
#pragma unroll
                    for (int i = 0; i < WM; ++i)
#pragma unroll
                        for (int j = 0; j < WN; ++j)
                            acc[i][j] = PAIR ? mfma16<E>(ob[sum - q][j], oa[q][i], acc[i][j])
                                             : mfma16<E>(oa[q][i], ob[sum - q][j], acc[i][j]);
        }
    };
    // Chunk c lies in LDS, c + 1 and c + 2 are on their way in registers: a load has two
    // chunks' time.  At the end the last chunk is loaded again and stored as zeros, so
    // that the loads under way are known, and waited for one by one, and so that the
    // loop has one end (with two the sums would take their registers twice).
    if (chunks > 0) {
        const int64_t end = chunks - 1;
        Chunk x, y;
        load_slots(0);
        load(x, 0);
        __builtin_amdgcn_sched_barrier(0);
        load(y, min((int64_t)1, end));
        __builtin_amdgcn_sched_barrier(0);
        store(x, 0, stage0);
        load(x, min((int64_t)2, end));
        __builtin_amdgcn_sched_barrier(0);
        lds_barrier();
        // the products of chunk c, and chunk c + 1 to LDS, c + 3 on its way
        auto step = [&](auto fits, Chunk &next, int64_t c, const uint8_t *now, uint8_t *to) {
            if constexpr (fits) {
                store_plain(next, to);
                load(next, min(c + 3, end));
            } else {
                store(next, c + 1, to);
                load(next, min(c + 3, end));
                __builtin_amdgcn_sched_barrier(0);
            }
            multiply(now);
            lds_barrier(); // the next chunk is here, and the last reads of this one are done
        };
        int64_t c = 0;
        for (; plain(c + 2); c += 2) { // so c + 1 is plain too
            step(std::true_type{}, y, c, stage0, stage1);
            step(std::true_type{}, x, c + 1, stage1, stage0);
        }
        for (; c <= end; c += 2) {
            step(std::false_type{}, y, c, stage0, stage1);
            step(std::false_type{}, x, c + 1, stage1, stage0);
        }
    }

    const int r = lane & 31, half = lane >> 5;
    const int64_t matrix = FORM == kGradient ? (int64_t)split * p.nlist + tile.e : 0;
    const int64_t row_base = FORM == kGradient ? matrix * p.m + m0 : tile.p0;
    const int64_t row_end = FORM == kGradient ? (matrix + 1) * p.m : tile.p1;
    if constexpr (FORM == kHidden) {
        static_assert(!PAIR, "hidden rows");
        store_hidden<T>(p, tile, tile.p0 + wm * WM * 32, n0 + wn * WN * 32, nt == 0, THREADS, acc);
        return;
    }
    TO *out = static_cast<TO *>(p.out);
    if constexpr (PAIR) {
#pragma unroll
        for (int i = 0; i < WM; ++i) {
            const int64_t row = row_base + (wm * WM + i) * 32 + r;
            if (row >= row_end)
                continue;
#pragma unroll
            for (int j = 0; j < WN; ++j)
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int n = n0 + (wn * WN + j) * 32 + 16 * q + 8 * half;
                    Piece<TO> o;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        o.v[e] = acc[i][j][q * 8 + e];
                    o.store(out + row * p.n + n, p.n - n);
                }
        }
    } else {
#pragma unroll
        for (int j = 0; j < WN; ++j) {
            const int n = n0 + (wn * WN + j) * 32 + r;
            if (n >= p.n)
                continue;
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int64_t row =
                        row_base + (wm * WM + i) * 32 + (q >> 2) * 8 + half * 4 + (q & 3);
                    if (row < row_end)
                        out[row * p.n + n] = (TO)acc[i][j][q];
                }
        }
    }
}

// ---------------------------------------------------------------------------
// tiles of 16-bit operands copied from memory into LDS without registers
// ---------------------------------------------------------------------------

// Which tile a workgroup forms: groups of `high` by `wide` tiles go to the XCDs in turn
// (every eighth workgroup runs on the same one), m first inside a group, so that the
// tiles that an XCD's 32 CUs form together share operands in its cache, and numbers
// that turn out empty are spread over all.
struct TileGroups {
    uint32_t high, wide, across; // across: groups along n
    int64_t mt;
    uint32_t nt;
    __device__ __forceinline__ bool tile(int64_t block, int64_t &m, uint32_t &n) const
    {
        const uint32_t size = high * wide, x = (uint32_t)block & 7;
        const int64_t i = block >> 3, turn = i / size, group = turn * 8 + x;
        const uint32_t in = (uint32_t)(i - turn * size);
        m = group / across * high + in % high;
        n = (uint32_t)(group % across) * wide + in / high;
        return m < mt && n < nt;
    }
};

// Large tiles are bound by the matrix instructions and what feeds them: 8192 x 8192 x 8192
// in bfloat16 1.03 ms (1.07 PF; the library's product 0.88 ms; without copies 0.76), both
// operands across the contraction 0.86 ms (1.27 PF); 65,536 rows of 128 lists of 2048 x
// 2048 671 us (0.82 PF).  Small ones by memory: 32 rows of 64 such lists 45 us, of which
// 210 MB are read (4.6 TB/s).
template <typename T, typename TO, int FORM, int KS, int STAGES, int WM, int WN, int MW, int NW>
__global__ __launch_bounds__(64 * MW * NW, FORM == kAdapter && STAGES == 2 ? 2 : 1)
void list_copy_kernel(ListJob p, TileGroups groups)
{
    static_assert(sizeof(T) == 2, "float32 operands go through registers");
    using F = FormOf<FORM>;
    constexpr int WAVES = MW * NW, THREADS = 64 * WAVES, TM = 32 * WM * MW, TN = 32 * WN * NW;
    constexpr bool PAIR = sizeof(TO) == 2;
    using PA = Place<F::A_ALONG, TM, KS>;
    using PB = Place<F::B_ALONG, TN, KS>;
    constexpr int STAGE = PA::PLANE + PB::PLANE;
    // objects of their own, so that the compiler knows a copy into one from a read of
    // another
    __shared__ __align__(16) uint8_t stage0[STAGE], stage1[STAGE];
    __shared__ __align__(16) uint8_t stage2[STAGES > 2 ? STAGE : 16], stage3[STAGES > 3 ? STAGE : 16];

    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % MW, wn = wave / MW;
    int64_t mt;
    uint32_t nt;
    if (!groups.tile(p.block0 + blockIdx.x, mt, nt))
        return;
    const int n0 = (int)nt * TN;

    PartTile tile;
    int m0 = 0, split = 0;
    if constexpr (FORM == kGradient) {
        const int nth = (int)(mt / p.mt), list = nth / p.splits;
        split = nth - list * p.splits;
        const int e = p.by_size ? p.by_size[list] : list;
        m0 = (int)(mt - (int64_t)nth * p.mt) * TM;
        tile = {e, part_begin(p.offsets, p.nlist, p.rows, e + 1),
                part_begin(p.offsets, p.nlist, p.rows, e + 2)};
        split_rows(tile.p0, tile.p1, split, p.splits);
    } else if constexpr (FORM == kAdapter) {
        tile = {0, mt * TM, min(mt * TM + TM, p.rows)};
    } else {
        tile = find_part(p.offsets, p.nlist, p.rows, mt, TM, p.by_row);
        if (tile.p0 >= tile.p1)
            return;
    }
    tile.p0 = uniform(tile.p0);
    tile.p1 = uniform(tile.p1);
    tile.e = __builtin_amdgcn_readfirstlane(tile.e);
    const bool listed = FORM == kAdapter || (tile.e >= 0 && tile.e < p.nlist);
    if (FORM == kHidden && !listed) {
        no_list_rows(p, tile, nt == 0, tid, THREADS);
        return;
    }
    const int64_t kdim = !listed ? 0 : FORM == kGradient ? max(tile.p1 - tile.p0, (int64_t)0)
                                                         : (int64_t)p.kdim;
    const int chunks = (int)((kdim + KS - 1) / KS); // a list has fewer than 2^31 rows
    RowList lists[WM]; // under way before the first copies
    if constexpr (FORM == kAdapter) {
#pragma unroll
        for (int i = 0; i < WM; ++i)
            lists[i].load(p, tile.p0 + (wm * WM + i) * 32 + (lane & 31), tile.p1);
    }

    // copies: instruction j of a wave brings 1 KB of consecutive LDS lines, a lane 16 bytes
    constexpr int CA = PA::PLANE / 1024 / WAVES, CB = PB::PLANE / 1024 / WAVES;
    static_assert(CA * 1024 * WAVES == PA::PLANE && CB * 1024 * WAVES == PB::PLANE, "whole copies");
    constexpr int LA = 64 / PA::BLOCKS, LB = 64 / PB::BLOCKS; // lines of a copy
    auto line_a = [&](int j) { return (wave * CA + j) * LA + lane / PA::BLOCKS; };
    auto line_b = [&](int j) { return (wave * CB + j) * LB + lane / PB::BLOCKS; };
    // the block of its line that a lane brings
    auto block_a = [&](int j) { return (lane % PA::BLOCKS) ^ PA::swizzle(line_a(j)); };
    auto block_b = [&](int j) { return (lane % PB::BLOCKS) ^ PB::swizzle(line_b(j)); };
    uint32_t offa[CA], offb[CB]; // bytes from the start of the chunk's range
    const int64_t lda = F::A_ALONG ? p.kdim : p.m, ldb = F::B_ALONG ? p.kdim : p.n;
    const bool gather_a = F::PER_LIST_ROWS && p.order;
#pragma unroll
    for (int j = 0; j < CA; ++j) {
        if constexpr (F::A_ALONG) {
            const int64_t row = tile.p0 + line_a(j);
            int64_t from = -1;
            if (row < tile.p1)
                from = F::PER_LIST_ROWS ? source_row(p, row) : row;
            const int64_t first = gather_a ? 0 : tile.p0;
            offa[j] = from < 0 ? kNowhere : (uint32_t)((from - first) * lda * 2) + block_a(j) * 16;
        } else {
            offa[j] = (uint32_t)(line_a(j) * lda * 2) + block_a(j) * 16;
        }
    }
#pragma unroll
    for (int j = 0; j < CB; ++j)
        offb[j] = (uint32_t)(line_b(j) * ldb * 2) + block_b(j) * 16;
    const int64_t abytes = (FORM == kGradient ? p.rows : p.arows) * lda * 2;
    const int64_t bmats = FORM == kAdapter ? 1 : p.nlist;
    const int64_t bbytes = FORM == kGradient ? p.arows * ldb * 2 : bmats * p.n * (int64_t)p.kdim * 2;
    const __amdgpu_buffer_rsrc_t arange =
        range_of(p.a, F::A_ALONG && !gather_a ? tile.p0 * lda * 2 : 0, abytes);
    const __amdgpu_buffer_rsrc_t brange = range_of(
        p.b, F::B_ALONG ? ((FORM == kAdapter ? 0 : (int64_t)max(tile.e, 0) * p.n) + n0) * ldb * 2 : 0,
        bbytes);
    // A gathered second operand (kGradient): the slots of a lane's lines are loaded two
    // chunks ahead, and become offsets before the chunk's copies are issued; the wait at
    // the end of a chunk is for them too.
    static_assert(FORM != kGradient || STAGES == 2, "slots are waited for by the next chunk");
    const bool gather_b = FORM == kGradient && p.order;
    int32_t slots[FORM == kGradient ? CB : 1];
    auto load_slots = [&](int c) {
        if constexpr (FORM == kGradient) {
            if (gather_b && kdim > 0)
#pragma unroll
                for (int j = 0; j < CB; ++j)
                    slots[j] = p.order[tile.p0 + min((int64_t)c * KS + line_b(j), kdim - 1)];
        }
    };
    auto place_slots = [&](int c) { // offb of chunk c
        if constexpr (FORM == kGradient) {
            if (gather_b)
#pragma unroll
                for (int j = 0; j < CB; ++j) {
                    const uint32_t row = slots[j] >= 0 ? p.k.div((uint32_t)slots[j]) : ~0u;
                    const bool there = (int64_t)c * KS + line_b(j) < kdim && row < (uint64_t)p.arows;
                    offb[j] = there ? row * (uint32_t)(ldb * 2) + block_b(j) * 16 : kNowhere;
                }
        }
    };

    // Copy q of chunk c (A's copies, then B's) into the chunk's LDS place.  Past the last
    // chunk nothing is read, and the place cleared: so the number of copies under way
    // is known.
    auto fetch = [&](int c, uint8_t *to, int q) {
        const bool of_a = q < CA;
        const int j = of_a ? q : q - CA;
        to += of_a ? (wave * CA + j) * 1024 : PA::PLANE + (wave * CB + j) * 1024;
        const int64_t k0 = (int64_t)c * KS;
        const int left = (int)min(kdim - k0, (int64_t)KS); // values in the chunk
        // The range check of a copy subtracts the scalar offset from the range's bytes, so
        // it may not pass them: inside a row, and a range holds at least one.
        const int along = left > 0 ? c * KS * 2 : 0;
        if (of_a) {
            if constexpr (F::A_ALONG)
                copy16_to_lds(arange, block_a(j) * 8 < left ? offa[j] : kNowhere, along, to);
            else
                copy16_to_lds(range_of(p.a, ((tile.p0 + k0) * lda + m0) * 2, abytes),
                              line_a(j) < left ? offa[j] : kNowhere, 0, to);
        } else if constexpr (F::B_ALONG) {
            copy16_to_lds(brange, block_b(j) * 8 < left ? offb[j] : kNowhere, along, to);
        } else if (FORM == kGradient && p.order) {
            copy16_to_lds(range_of(p.b, (int64_t)n0 * 2, bbytes), offb[j], 0, to);
        } else {
            const int64_t row = FORM == kGradient ? tile.p0 + k0
                                                  : (int64_t)max(tile.e, 0) * p.kdim + k0;
            copy16_to_lds(range_of(p.b, (row * ldb + n0) * 2, bbytes),
                          line_b(j) < left ? offb[j] : kNowhere, 0, to);
        }
    };
    auto place = [&](auto i) -> uint8_t * {
        constexpr int I = decltype(i)::value % STAGES;
        if constexpr (I == 0)
            return stage0;
        else if constexpr (I == 1)
            return stage1;
        else if constexpr (I == 2)
            return stage2;
        else
            return stage3;
    };
    constexpr std::integral_constant<int, 0> i0{};
    constexpr std::integral_constant<int, 1> i1{};
    constexpr std::integral_constant<int, 2> i2{};
    constexpr std::integral_constant<int, 3> i3{};

    load_slots(0);
    place_slots(0);
    load_slots(1);
    auto fetch_all = [&](int c, uint8_t *to) {
#pragma unroll
        for (int q = 0; q < CA + CB; ++q)
            fetch(c, to, q);
    };
    fetch_all(0, place(i0));
    if constexpr (STAGES > 2)
        fetch_all(1, place(i1));
    if constexpr (STAGES > 3)
        fetch_all(2, place(i2));

    f32x16 acc[WM][WN];
    if constexpr (FORM == kAdapter) {
        // LDS: the last stage, whose first copies come after the next barrier
        constexpr int SLAB = STAGE / WAVES / 1024 * 1024;
        adapter_sums<T, SLAB, PAIR, false>(p, tile.p0 + wm * WM * 32, n0 + wn * WN * 32, lists,
                                           place(std::integral_constant<int, STAGES - 1>{}) +
                                               wave * SLAB,
                                           acc);
    } else {
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[i][j][q] = 0.f;
    }
    Reader<F::A_ALONG, TM, KS, WM, false> reada;
    Reader<F::B_ALONG, TN, KS, WN, PAIR> readb;
    reada.init(wm * WM * 32);
    readb.init(wn * WN * 32);
    struct Operands {
        s16x8 a[WM], b[WN];
    } o[2];
#pragma unroll
    for (int i = 0; i < WM; ++i)
        o[1].a[i] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < WN; ++j)
        o[1].b[j] = s16x8{0, 0, 0, 0, 0, 0, 0, 0};
    // operand number q of step s: a[0], then b, then the rest of a, as the products take them
    auto read = [&](const uint8_t *from, int s, Operands &to, int q) {
        if (q == 0)
            to.a[0] = reada.read(from, 0, s);
        else if (q <= WN)
            to.b[q - 1] = readb.read(from + PA::PLANE, q - 1, s);
        else
            to.a[q - WN] = reada.read(from, q - WN, s);
    };
    constexpr int STEPS = KS / 16, PRODUCTS = WM * WN, READS = WM + WN, COPIES = CA + CB;
    static_assert(STEPS % 2 == 0, "the last step's operands lie in o[1]");
    constexpr int PARTS = STAGES == 2 ? STEPS / 2 : STEPS; // steps that issue copies
    // how many of `count` things are issued before product m
    auto before = [](int count, int m) { return (count * m + PRODUCTS - 1) / PRODUCTS; };
    // Chunk c in stage i: a step's products, the last chunk's last step first, with the
    // reads of the next step's operands and the copies of the chunk STAGES - 1 ahead
    // (to where the chunk before lay) issued between them: issued together they would
    // keep a wave from its products while the others issue theirs.
    auto chunk = [&](auto i, int c) {
        constexpr int I = decltype(i)::value;
        const uint8_t *now = place(i);
        uint8_t *ahead = place(std::integral_constant<int, I + STAGES - 1>{});
        place_slots(c + 1);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            if (s == PARTS)
                load_slots(c + 2);
            const Operands &x = o[(s + 1) & 1];
            const int c0 = COPIES * min(s, PARTS) / PARTS, c1 = COPIES * min(s + 1, PARTS) / PARTS;
#pragma unroll
            for (int m = 0; m < PRODUCTS; ++m) {
                const int bi = m / WN, bj = m % WN;
                acc[bi][bj] = PAIR ? mfma16<T>(x.b[bj], x.a[bi], acc[bi][bj])
                                   : mfma16<T>(x.a[bi], x.b[bj], acc[bi][bj]);
#pragma unroll
                for (int q = before(READS, m); q < before(READS, m + 1); ++q)
                    read(now, s, o[s & 1], q);
#pragma unroll
                for (int q = c0 + before(c1 - c0, m); q < c0 + before(c1 - c0, m + 1); ++q)
                    fetch(c + STAGES - 1, ahead, q);
                __builtin_amdgcn_sched_barrier(0);
            }
        }
        wait_vm<(STAGES - 2) * (CA + CB)>(); // the next chunk
        lds_barrier(); // every wave's part of it is here, and this one's last reads done
    };
    if (chunks > 0) {
        wait_vm<(STAGES - 2) * (CA + CB)>();
        lds_barrier();
        for (int c = 0; c < chunks; c += STAGES) {
            chunk(i0, c);
            chunk(i1, c + 1);
            if constexpr (STAGES > 2)
                chunk(i2, c + 2);
            if constexpr (STAGES > 3)
                chunk(i3, c + 3);
        }
#pragma unroll
        for (int m = 0; m < PRODUCTS; ++m) {
            const int bi = m / WN, bj = m % WN;
            acc[bi][bj] = PAIR ? mfma16<T>(o[1].b[bj], o[1].a[bi], acc[bi][bj])
                               : mfma16<T>(o[1].a[bi], o[1].b[bj], acc[bi][bj]);
        }
    }
    wait_vm<0>(); // no copy is under way to where results may go, or past the end

    if constexpr (FORM == kHidden) {
        static_assert(!PAIR, "hidden rows");
        store_hidden<T>(p, tile, tile.p0 + wm * WM * 32, n0 + wn * WN * 32, nt == 0, THREADS, acc);
        return;
    }
    const int r = lane & 31, half = lane >> 5;
    const int64_t matrix = FORM == kGradient ? (int64_t)split * p.nlist + tile.e : 0;
    const int64_t row_base = FORM == kGradient ? matrix * p.m + m0 : tile.p0;
    const int64_t row_end = FORM == kGradient ? (matrix + 1) * p.m : tile.p1;
    TO *out = static_cast<TO *>(p.out);
    if constexpr (PAIR) {
        // Through LDS, a wave's own part of a stage, so that a store covers whole rows of
        // its columns.
        typedef TO T8 __attribute__((ext_vector_type(8)));
        typedef TO T8U __attribute__((ext_vector_type(8), aligned(sizeof(TO))));
        constexpr int PART = STAGE / WAVES / 16 * 16;
        constexpr int JS = 32 * WN * 64 <= PART ? WN : WN / 2; // blocks of columns at a time
        constexpr int BR = JS * 4, ROWB = BR * 16;
        constexpr int SLAB = PART / (32 * ROWB) < WM ? PART / (32 * ROWB) : WM;
        static_assert(SLAB >= 1 && WM % SLAB == 0, "rows through LDS");
        lds_barrier();
        uint8_t *mine = stage0 + wave * PART;
#pragma unroll
        for (int b0 = 0; b0 < WM; b0 += SLAB)
#pragma unroll
            for (int j0 = 0; j0 < WN; j0 += JS) {
#pragma unroll
                for (int i = 0; i < SLAB; ++i)
#pragma unroll
                    for (int j = 0; j < JS; ++j)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            T8 v;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                v[e] = (TO)acc[b0 + i][j0 + j][q * 8 + e];
                            const int b = (j * 4 + q * 2 + half) ^ (r & (BR - 1));
                            *reinterpret_cast<T8 *>(mine + (i * 32 + r) * ROWB + b * 16) = v;
                        }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int k = 0; k < SLAB * 32 * BR / 64; ++k) {
                    const int line = (k * 64 + lane) / BR, b = lane % BR;
                    const T8 v = *reinterpret_cast<const T8 *>(mine + line * ROWB +
                                                               (b ^ (line & (BR - 1))) * 16);
                    const int64_t row = row_base + (wm * WM + b0) * 32 + line;
                    const int n = n0 + (wn * WN + j0) * 32 + b * 8;
                    if (row >= row_end || n >= p.n)
                        continue;
                    TO *to = out + row * p.n + n;
                    if (n + 8 <= p.n) {
                        *reinterpret_cast<T8U *>(to) = v;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < p.n)
                                to[e] = v[e];
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
    } else {
#pragma unroll
        for (int j = 0; j < WN; ++j) {
            const int n = n0 + (wn * WN + j) * 32 + r;
            if (n >= p.n)
                continue;
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int64_t row =
                        row_base + (wm * WM + i) * 32 + (q >> 2) * 8 + half * 4 + (q & 3);
                    if (row < row_end)
                        out[row * p.n + n] = (TO)acc[i][j][q];
                }
        }
    }
}

// Whether the copies can read a product's operands: 16-byte blocks of rows that are
// multiples of 16 bytes, ranges of less than 2^31 bytes.
template <int FORM>
bool copies_fit(const ListJob &p)
{
    auto whole = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
    const int64_t lda = FormOf<FORM>::A_ALONG ? p.kdim : p.m;
    const int64_t ldb = FormOf<FORM>::B_ALONG ? p.kdim : p.n;
    const int64_t most = (int64_t)0x7FFFFFFF - (1 << 22);
    const bool gathers = FORM != kAdapter && p.order;
    const int64_t gathered = gathers ? p.arows * (FORM == kGradient ? ldb : lda) * 2 : 0;
    return whole(p.a) && whole(p.b) && lda % 8 == 0 && ldb % 8 == 0 &&
           std::max(lda, ldb) * 2 * 256 < most && gathered < most &&
           (FORM != kAdapter || (whole(p.up) && p.r % 8 == 0));
}

// Tiles of `high` by `wide` results that a product has; half of the lists end inside one.
template <int FORM>
int64_t count_tiles(const ListJob &p, int high, int wide)
{
    const int64_t nt = (p.n + wide - 1) / wide;
    if (FORM == kGradient)
        return p.nlist * ((p.m + high - 1) / high) * nt;
    const int64_t ends = FORM == kAdapter ? 0 : (p.rows < p.nlist ? p.rows : p.nlist) / 2;
    return ((p.rows + high - 1) / high + ends) * nt;
}

template <typename T, typename TO, int FORM, int KS, int STAGES, int WM, int WN, int MW, int NW>
hipError_t launch_copies(ListJob p, hipStream_t stream)
{
    constexpr int TM = 32 * WM * MW, TN = 32 * WN * NW, THREADS = 64 * MW * NW;
    p.nt = (uint32_t)((p.n + TN - 1) / TN);
    int64_t mt;
    if (FORM == kGradient) {
        p.mt = (uint32_t)((p.m + TM - 1) / TM);
        mt = (int64_t)p.mt * p.nlist * p.splits;
    } else if (FORM == kAdapter) {
        mt = (p.rows + TM - 1) / TM;
    } else {
        p.by_row = slots_by_row(p.rows, p.nlist, TM);
        mt = tile_slots(p.rows, p.nlist, TM);
    }
    TileGroups g;
    g.mt = mt;
    g.nt = p.nt;
    // 32 tiles a group, more if there are enough groups (8192 x 8192 x 8192: 4 x 16 tiles
    // a group 1027 us, 2 rows of 32 tiles 1135; 8 or 16 rows of tiles are no better)
    g.high = 4;
    g.wide = 8;
    auto count = [&](int64_t high, int64_t wide) {
        return (mt + high - 1) / high * ((p.nt + wide - 1) / wide);
    };
    while (g.high > 1 && count(g.high, g.wide) < 8)
        g.high /= 2;
    while (g.wide > 1 && count(g.high, g.wide) < 8)
        g.wide /= 2;
    while (FORM != kGradient && g.wide < p.nt && count(g.high, 2 * g.wide) >= 64)
        g.wide *= 2;
    // a list's tiles on all XCDs alike, as lists differ in length
    while (FORM == kGradient && p.nlist > 1 && g.wide > 1 &&
           (int64_t)p.mt * p.splits * p.nt < 8 * g.high * g.wide)
        g.wide /= 2;
    g.across = (p.nt + g.wide - 1) / g.wide;
    const int64_t blocks = (count(g.high, g.wide) + 7) / 8 * 8 * g.high * g.wide;
    const int64_t most = most_blocks(THREADS);
    for (int64_t b = 0; b < blocks; b += most) {
        p.block0 = b;
        hipLaunchKernelGGL((list_copy_kernel<T, TO, FORM, KS, STAGES, WM, WN, MW, NW>),
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(THREADS),
                           0, stream, p, g);
    }
    return hipGetLastError();
}

// Whether an operand has fewer than eight values in all, and so is read value by value.
template <int FORM>
bool any_tiny(const ListJob &p)
{
    const int64_t a = FORM == kGradient ? p.rows * p.m : p.arows * p.kdim;
    const int64_t b = FORM == kGradient ? p.arows * p.n
                                        : (FORM == kAdapter ? 1 : (int64_t)p.nlist) * p.n * p.kdim;
    return a < 8 || b < 8 || (FORM == kAdapter && (int64_t)p.nlist * p.n * p.r < 8);
}

// ONLY_TINY: the caller has another kernel for all but tiny operands.
template <typename T, typename TO, int FORM, int KS, int WM, int WN, int MW, int NW,
          bool ONLY_TINY = false>
hipError_t launch_tiles(ListJob p, hipStream_t stream)
{
    constexpr int TM = 32 * WM * MW, TN = 32 * WN * NW, THREADS = 64 * MW * NW;
    const int cols = FORM == kHidden ? p.rp : p.n;
    p.nt = (uint32_t)((cols + TN - 1) / TN);
    int64_t mt;
    if (FORM == kGradient) {
        p.mt = (uint32_t)((p.m + TM - 1) / TM);
        mt = (int64_t)p.mt * p.nlist * p.splits;
    } else if (FORM == kAdapter) {
        mt = (p.rows + TM - 1) / TM;
    } else {
        p.by_row = slots_by_row(p.rows, p.nlist, TM);
        mt = tile_slots(p.rows, p.nlist, TM);
    }
    const int64_t blocks = mt * p.nt, most = most_blocks(THREADS);
    auto kernel = list_tile_kernel<T, TO, FORM, KS, WM, WN, MW, NW, true>;
    if constexpr (!ONLY_TINY)
        if (!any_tiny<FORM>(p))
            kernel = list_tile_kernel<T, TO, FORM, KS, WM, WN, MW, NW, false>;
    for (int64_t b = 0; b < blocks; b += most) {
        p.block0 = b;
        hipLaunchKernelGGL(kernel,
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(THREADS),
                           0, stream, p);
    }
    return hipGetLastError();
}

} // namespace ivfpq

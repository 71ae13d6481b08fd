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
// nearest to what the parts before leave: |mid| <= 2^-9 |x|, |lo| <= 2^-18 |x|,
// and what three parts leave is below 2^-27 |x|.  A product is the sum of six of
// the nine part products, the smallest first; the three dropped are below 2^-26 of
// it together, less than float32's own half step.  Six bfloat16 instructions take
// 6 / 16 of the time of the float32 one.  An infinity becomes a NaN this way.
#pragma once

#include "list_plan.hpp"
#include "rows.hpp"
#include "rows_internal.hpp"
#include "tile_ops.hpp"

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
    const int lane = lane_id();
    int first = 0, count = nlist + 2;
    while (count > 1) {
        const int step = (count + 63) / 64;
        const int i = first + lane * step;
        const bool upto = i < first + count &&
                          part_slot(part_begin(offsets, nlist, rows, i), i, tm, by_row) <= slot;
        const uint64_t m = __ballot(upto);
        const int who = m ? 63 - __builtin_clzll(m) : 0;
        const int left = count - who * step;
        first += who * step;
        count = left < step ? left : step;
    }
    first = __builtin_amdgcn_readfirstlane(first);
    const int64_t begin = part_begin(offsets, nlist, rows, first);
    const int64_t end = part_begin(offsets, nlist, rows, first + 1);
    const int64_t p0 = slot_row(slot, begin, end, first, tm, by_row);
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

// Eight values of a line in registers, on their way to LDS.
template <typename T>
struct Eight {
    static constexpr int Q = sizeof(T) / 2; // 16-byte pieces
    T v[8];
    // those past `valid` are zero
    __device__ __forceinline__ void load(const T *p, int64_t valid)
    {
        typedef T V __attribute__((ext_vector_type(8 / Q), aligned(sizeof(T))));
        if (valid >= 8) {
#pragma unroll
            for (int h = 0; h < Q; ++h) {
                const V w = reinterpret_cast<const V *>(p)[h];
#pragma unroll
                for (int i = 0; i < 8 / Q; ++i)
                    v[h * (8 / Q) + i] = w[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = i < valid ? p[i] : (T)0.f;
        }
    }
    // to the planes at `to`, `plane` bytes apart
    __device__ __forceinline__ void store(uint8_t *to, int plane) const
    {
        using E = typename Parts<T>::E;
        typedef E V __attribute__((ext_vector_type(8)));
        V out[Parts<T>::N];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (std::is_same<T, float>::value) {
                // the largest finite values stay finite in bfloat16
                const float x = v[i];
                const E hi = (E)__builtin_amdgcn_fmed3f(x, -0x1.FEp127f, 0x1.FEp127f);
                const float r1 = x - (float)hi;
                const E mid = (E)r1;
                out[0][i] = hi;
                out[1][i] = mid;
                out[2][i] = (E)(r1 - (float)mid);
            } else {
                out[0][i] = v[i];
            }
        }
#pragma unroll
        for (int p = 0; p < Parts<T>::N; ++p)
            *reinterpret_cast<V *>(to + p * plane) = out[p];
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
    int64_t block0 = 0;
    // adapters: hidden rows [t][width] (16-bit: high parts, then low parts, rp each),
    // the list of each row, up matrices [nlist][n][r], scales [nlist] or nullptr
    void *hidden = nullptr;
    int32_t *row_list = nullptr;
    const int32_t *pos = nullptr;
    const void *up = nullptr;
    const float *scales = nullptr;
    int r = 0, rp = 0, width = 0;
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

template <typename T, typename TO, int FORM, int KS, int WM, int WN, int MW, int NW>
__global__ __launch_bounds__(64 * MW * NW) void list_tile_kernel(ListJob p)
{
    using F = FormOf<FORM>;
    constexpr int WAVES = MW * NW, THREADS = 64 * WAVES, TM = 32 * WM * MW, TN = 32 * WN * NW;
    constexpr bool PAIR = sizeof(TO) == 2; // the second operand goes first (see deal_row)
    constexpr int NP = Parts<T>::N;
    using E = typename Parts<T>::E;
    using PA = Place<F::A_ALONG, TM, KS>;
    using PB = Place<F::B_ALONG, TN, KS>;
    constexpr int STAGE = NP * (PA::PLANE + PB::PLANE);
    __shared__ __align__(16) uint8_t stage[2][STAGE];
    __shared__ int segs[FORM == kAdapter ? TM + 1 : 1]; // lists of the tile's rows, their number
    __shared__ int tile_list[FORM == kAdapter ? TM : 1];

    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % MW, wn = wave / MW;
    const int64_t block = p.block0 + blockIdx.x;
    const uint32_t nt = (uint32_t)(block % p.nt);
    const int64_t mt = block / p.nt;
    const int n0 = (int)nt * TN;

    PartTile tile;
    int m0 = 0;
    if constexpr (FORM == kGradient) {
        const int e = (int)(mt / p.mt);
        m0 = (int)(mt - (int64_t)e * p.mt) * TM;
        tile = {e, part_begin(p.offsets, p.nlist, p.rows, e + 1),
                part_begin(p.offsets, p.nlist, p.rows, e + 2)};
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
    if (FORM == kHidden && !listed)
        return;

    int64_t chunks = (kdim + KS - 1) / KS;
    const int64_t main_chunks = chunks;
    const int per_seg = FORM == kAdapter ? (p.width + KS - 1) / KS : 1;
    if constexpr (FORM == kAdapter) {
        // the lists of the tile's rows, each once
        for (int i = tid; i < TM; i += THREADS) {
            const int64_t row = tile.p0 + i;
            int e = -1;
            if (row < tile.p1 && (uint32_t)p.pos[row] < (uint64_t)p.rows) {
                e = p.row_list[row];
                e = e < p.nlist ? e : -1;
            }
            tile_list[i] = e;
        }
        __syncthreads();
        if (wave == 0) {
            int last = -1, found = 0;
            for (;;) { // ascending, at most TM times
                uint32_t next = 0xFFFFFFFFu;
#pragma unroll
                for (int i = 0; i < (TM + 63) / 64; ++i) {
                    const int e = i * 64 + lane < TM ? tile_list[i * 64 + lane] : -1;
                    next = e > last ? min(next, (uint32_t)e) : next;
                }
                next = min(next, xor_lane<1>(next));
                next = min(next, xor_lane<2>(next));
                next = min(next, xor_lane<4>(next));
                next = min(next, xor_lane<8>(next));
                next = min(next, xor_lane<16>(next));
                next = min(next, xor_lane<32>(next));
                if (next == 0xFFFFFFFFu)
                    break;
                last = (int)next;
                if (lane == 0)
                    segs[found] = last;
                ++found;
            }
            if (lane == 0)
                segs[TM] = found;
        }
        __syncthreads();
        chunks += (int64_t)segs[TM] * per_seg;
    }

    f32x16 acc[WM][WN];
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q)
                acc[i][j][q] = 0.f;

    // pieces of eight values, a thread's own of both operands
    constexpr int QA = PA::LINES * PA::BLOCKS / THREADS, QB = PB::LINES * PB::BLOCKS / THREADS;
    static_assert(QA * THREADS == PA::LINES * PA::BLOCKS && QB * THREADS == PB::LINES * PB::BLOCKS,
                  "whole pieces a thread");
    const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
    Eight<T> ra[QA], rb[QB];
    int64_t arow[F::A_ALONG ? QA : 1];
    if constexpr (F::A_ALONG) {
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int64_t row = tile.p0 + (j * THREADS + tid) / PA::BLOCKS;
            arow[j] = row >= tile.p1 ? -1 : F::PER_LIST_ROWS ? source_row(p, row) : row;
        }
    }
    auto load = [&](int64_t c) {
        const bool extra = FORM == kAdapter && c >= main_chunks;
        if (extra) {
            const int x = (int)(c - main_chunks), seg = segs[x / per_seg];
            const int k0 = x % per_seg * KS;
            const T *hidden = static_cast<const T *>(p.hidden);
            const T *up = static_cast<const T *>(p.up) + (int64_t)seg * p.n * p.r;
#pragma unroll
            for (int j = 0; j < QA; ++j) {
                const int piece = j * THREADS + tid, row = piece / PA::BLOCKS;
                const int at = k0 + piece % PA::BLOCKS * 8;
                const bool mine = tile_list[row] == seg;
                ra[j].load(hidden + (tile.p0 + (mine ? row : 0)) * p.width + at,
                           mine ? p.width - at : 0);
            }
#pragma unroll
            for (int j = 0; j < QB; ++j) {
                const int piece = j * THREADS + tid, row = n0 + piece / PB::BLOCKS;
                const int at = k0 + piece % PB::BLOCKS * 8;
                const int col = at < p.rp ? at : at - p.rp; // the low parts meet the same values
                const bool inside = row < p.n && at < p.width;
                rb[j].load(up + (int64_t)(inside ? row : 0) * p.r + (inside ? col : 0),
                           inside ? p.r - col : 0);
            }
            return;
        }
        const int64_t k0 = c * KS;
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int piece = j * THREADS + tid, line = piece / PA::BLOCKS;
            const int value = piece % PA::BLOCKS * 8;
            if constexpr (F::A_ALONG) {
                const bool live = arow[j] >= 0;
                ra[j].load(a + (live ? arow[j] : 0) * p.kdim + k0 + value,
                           live ? kdim - k0 - value : 0);
            } else {
                const bool live = k0 + line < kdim;
                ra[j].load(a + (tile.p0 + (live ? k0 + line : 0)) * p.m + m0 + value,
                           live ? p.m - m0 - value : 0);
            }
        }
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int piece = j * THREADS + tid, line = piece / PB::BLOCKS;
            const int value = piece % PB::BLOCKS * 8;
            if constexpr (F::B_ALONG) {
                const int64_t base = F::PER_LIST_ROWS ? (int64_t)tile.e * p.n : 0;
                const bool live = n0 + line < p.n;
                rb[j].load(b + (base + (live ? n0 + line : 0)) * p.kdim + k0 + value,
                           live ? kdim - k0 - value : 0);
            } else {
                int64_t row = k0 + line < kdim ? k0 + line : -1;
                if constexpr (FORM == kGradient)
                    row = row >= 0 ? source_row(p, tile.p0 + row) : -1;
                else
                    row = row >= 0 ? (int64_t)tile.e * p.kdim + row : -1;
                rb[j].load(b + (row >= 0 ? row : 0) * p.n + n0 + value,
                           row >= 0 ? p.n - n0 - value : 0);
            }
        }
    };
    auto store = [&](uint8_t *to) {
#pragma unroll
        for (int j = 0; j < QA; ++j) {
            const int piece = j * THREADS + tid;
            ra[j].store(to + PA::at(piece / PA::BLOCKS, piece % PA::BLOCKS), PA::PLANE);
        }
#pragma unroll
        for (int j = 0; j < QB; ++j) {
            const int piece = j * THREADS + tid;
            rb[j].store(to + NP * PA::PLANE + PB::at(piece / PB::BLOCKS, piece % PB::BLOCKS),
                        PB::PLANE);
        }
    };
    Reader<F::A_ALONG, TM, KS, WM, false> reada;
    Reader<F::B_ALONG, TN, KS, WN, PAIR> readb;
    reada.init(wm * WM * 32);
    readb.init(wn * WN * 32);

    if (chunks > 0) {
        load(0);
        store(stage[0]);
    }
    if (chunks > 1)
        load(1);
    lds_barrier();
    for (int64_t c = 0; c < chunks; ++c) {
        const uint8_t *now = stage[c & 1];
        if (c + 1 < chunks)
            store(stage[(c + 1) & 1]);
        if (c + 2 < chunks)
            load(c + 2);
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
        lds_barrier(); // the next chunk is here, and the last reads of this one are done
    }

    const int r = lane & 31, half = lane >> 5;
    const int64_t row_base = FORM == kGradient ? (int64_t)tile.e * p.m + m0 : tile.p0;
    const int64_t row_end = FORM == kGradient ? (int64_t)(tile.e + 1) * p.m : tile.p1;
    if constexpr (FORM == kHidden) {
        // a lane has one column of sixteen rows (PAIR is false: TO is float)
        static_assert(!PAIR, "hidden rows");
        const float scale = p.scales ? p.scales[tile.e] : 1.f;
        if (nt == 0)
            for (int64_t row = tile.p0 + tid; row < tile.p1; row += THREADS) {
                const int64_t t = source_row(p, row);
                if (t >= 0)
                    p.row_list[t] = tile.e;
            }
#pragma unroll
        for (int j = 0; j < WN; ++j) {
            const int col = n0 + (wn * WN + j) * 32 + r;
            if (col >= p.rp)
                continue;
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int q = 0; q < 16; ++q) {
                    const int64_t row =
                        row_base + (wm * WM + i) * 32 + (q >> 2) * 8 + half * 4 + (q & 3);
                    const int64_t t = row < row_end ? source_row(p, row) : -1;
                    if (t < 0)
                        continue;
                    const float h = acc[i][j][q] * scale; // zero past column r
                    T *to = static_cast<T *>(p.hidden) + t * p.width + col;
                    to[0] = (T)h;
                    if constexpr (NP == 1)
                        to[p.rp] = (T)(h - (float)to[0]);
                }
        }
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

template <typename T, typename TO, int FORM, int KS, int WM, int WN, int MW, int NW>
hipError_t launch_tiles(ListJob p, hipStream_t stream)
{
    constexpr int TM = 32 * WM * MW, TN = 32 * WN * NW, THREADS = 64 * MW * NW;
    const int cols = FORM == kHidden ? p.rp : p.n;
    p.nt = (uint32_t)((cols + TN - 1) / TN);
    int64_t mt;
    if (FORM == kGradient) {
        p.mt = (uint32_t)((p.m + TM - 1) / TM);
        mt = (int64_t)p.mt * p.nlist;
    } else if (FORM == kAdapter) {
        mt = (p.rows + TM - 1) / TM;
    } else {
        p.by_row = slots_by_row(p.rows, p.nlist, TM);
        mt = tile_slots(p.rows, p.nlist, TM);
    }
    const int64_t blocks = mt * p.nt, most = most_blocks(THREADS);
    for (int64_t b = 0; b < blocks; b += most) {
        p.block0 = b;
        hipLaunchKernelGGL((list_tile_kernel<T, TO, FORM, KS, WM, WN, MW, NW>),
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(THREADS),
                           0, stream, p);
    }
    return hipGetLastError();
}

} // namespace ivfpq

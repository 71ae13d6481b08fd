// Rows of a table by number, scaled, and the gradient of the table: per list, the
// sum of the rows sorted to it.
#include "common.hpp"
#include "list_plan.hpp"
#include "rows.hpp"
#include "rows_internal.hpp"

namespace ivfpq {

// Lanes that share a row: enough for one piece each, at most a wave.
static int piece_lanes(int64_t pieces)
{
    int l = 1;
    while (l < pieces && l < 64)
        l *= 2;
    return l;
}

// out[i] = scale table[ids[i]], rounded once; zero where the number is outside the
// table.  A thread has one piece of kLookupRows rows that lie `step` apart: their
// numbers are under way together, then their pieces.  Bound by memory and, for few rows,
// by the launch: 64 rows 6.4 us with the call; 16,384 rows of 2048 in bfloat16 21 us (134
// MB, 6.4 TB/s).
constexpr int kLookupRows = 4;

template <typename T>
__global__ __launch_bounds__(256) void table_lookup_kernel(const T *__restrict__ table, int64_t rows,
                                                           int d, FastDiv pieces,
                                                           const int32_t *__restrict__ ids,
                                                           int64_t n, int64_t step, float scale,
                                                           T *__restrict__ out, int64_t row0)
{
    constexpr int N = Piece<T>::N;
    const uint32_t g = blockIdx.x * 256u + threadIdx.x;
    const int64_t i0 = row0 + pieces.div(g);
    if (i0 >= step)
        return;
    const int c = (int)(g - (uint32_t)(i0 - row0) * pieces.c) * N;
    int64_t id[kLookupRows];
    Piece<T> v[kLookupRows];
#pragma unroll
    for (int i = 0; i < kLookupRows; ++i)
        id[i] = i0 + i * step < n ? ids[i0 + i * step] : -1;
#pragma unroll
    for (int i = 0; i < kLookupRows; ++i) {
        const bool inside = (uint64_t)id[i] < (uint64_t)rows;
        if (inside)
            v[i].load(table + id[i] * d + c, d - c);
        else
            v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < kLookupRows; ++i) {
        const int64_t row = i0 + i * step;
        if (row >= n)
            break;
        // zero whatever the factor is where there is no row
        const float factor = (uint64_t)id[i] < (uint64_t)rows ? scale : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[i].v[e] *= factor;
        v[i].store(out + row * d + c, d - c);
    }
}

template <typename T>
static hipError_t lookup_as(const void *table, int64_t rows, int d, const int32_t *ids, int64_t n,
                            float scale, void *out, hipStream_t stream)
{
    const int64_t pieces = (d + Piece<T>::N - 1) / Piece<T>::N;
    const int64_t step = (n + kLookupRows - 1) / kLookupRows;
    const int64_t most = 0x7FFFFF00ll / pieces; // rows of one launch: 32-bit piece numbers
    for (int64_t r = 0; r < step; r += most) {
        const int64_t now = (step - r < most ? step - r : most) * pieces;
        hipLaunchKernelGGL(table_lookup_kernel<T>, dim3((unsigned)((now + 255) / 256)), dim3(256),
                           0, stream, static_cast<const T *>(table), rows, d,
                           FastDiv((uint32_t)pieces), ids, n, step, scale, static_cast<T *>(out), r);
    }
    return hipGetLastError();
}

hipError_t launch_table_lookup(const void *table, int type, int64_t rows, int d, const int32_t *ids,
                               int64_t n, float scale, void *out, hipStream_t stream)
{
    switch (type) {
    case kF32: return lookup_as<float>(table, rows, d, ids, n, scale, out, stream);
    case kBF16: return lookup_as<__bf16>(table, rows, d, ids, n, scale, out, stream);
    default: return lookup_as<_Float16>(table, rows, d, ids, n, scale, out, stream);
    }
}

// ---------------------------------------------------------------------------
// gradient of the table
// ---------------------------------------------------------------------------

// Eight columns of a row of d: four from c[0] on and four from c[1] on, where the lanes
// that share a row have the first fours side by side, then the second ones, so that
// loads and stores of either type are of whole lines.
struct Columns {
    int c[2];
    __device__ __forceinline__ Columns(int first, int lane, int lanes)
        : c{first + lane * 4, first + (lanes + lane) * 4}
    {
    }
};

// Sums of rows.  Several rows are loaded together, and no load has a branch of its own
// (row 0 or a column inside stands for what is not there, and is dropped), or each
// would be waited for before the next.  16 rows at a time leave half the waves: 16,384
// rows of 4096 to 32,000 lists 61 us with 8, 84 with 16.
constexpr int kSumRows = 8;

template <typename T>
struct RowSum {
    typedef T V __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    float v[2][4];

    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[h][e] = 0.f;
    }
    struct Batch {
        T x[kSumRows][2][4];
        bool live[kSumRows];
    };
    // rows t[i] of grad [nvec][d], -1: none
    __device__ __forceinline__ static void load(Batch &b, const T *grad, int64_t nvec, int d,
                                                Columns at, const int (&t)[kSumRows])
    {
        const T *from[kSumRows];
#pragma unroll
        for (int i = 0; i < kSumRows; ++i) {
            b.live[i] = (uint32_t)t[i] < (uint64_t)nvec;
            from[i] = grad + (int64_t)(b.live[i] ? t[i] : 0) * d;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (at.c[h] + 4 <= d) {
#pragma unroll
                for (int i = 0; i < kSumRows; ++i) {
                    const V w = *reinterpret_cast<const V *>(from[i] + at.c[h]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        b.x[i][h][e] = w[e];
                }
            } else { // the row's end: values past it are not stored
#pragma unroll
                for (int i = 0; i < kSumRows; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        b.x[i][h][e] = from[i][min(at.c[h] + e, d - 1)];
            }
        }
    }
    __device__ __forceinline__ void add(const Batch &b, int i)
    {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[h][e] = b.live[i] ? v[h][e] + (float)b.x[i][h][e] : v[h][e];
    }
    // sorted rows [lo, hi), ascending in float32
    __device__ __forceinline__ void add_rows(const T *grad, int64_t nvec, FastDiv k, int d,
                                             Columns at, const int32_t *order, int64_t lo,
                                             int64_t hi)
    {
        for (int64_t p = lo; p < hi; p += kSumRows) {
            int t[kSumRows];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                t[i] = order[min(p + i, hi - 1)];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                t[i] = p + i < hi && t[i] >= 0 ? (int)k.div((uint32_t)t[i]) : -1;
            Batch b;
            load(b, grad, nvec, d, at, t);
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                add(b, i);
        }
    }
    // times scale to a row of d values
    // NT: past the caches, for rows that nothing reads soon
    template <bool NT = false, typename TO>
    __device__ __forceinline__ void store(TO *row, int d, Columns at, float scale) const
    {
        typedef TO W __attribute__((ext_vector_type(4), aligned(sizeof(TO))));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (at.c[h] + 4 <= d) {
                W w;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = (TO)(v[h][e] * scale);
                if constexpr (NT)
                    __builtin_nontemporal_store(w, reinterpret_cast<W *>(row + at.c[h]));
                else
                    *reinterpret_cast<W *>(row + at.c[h]) = w;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (at.c[h] + e < d)
                        row[at.c[h] + e] = (TO)(v[h][e] * scale);
            }
        }
    }
};

struct TableGrad {
    const void *grad;
    int64_t nvec, n; // rows of grad, slots
    int d;
    const int32_t *offsets, *order;
    FastDiv k;
    int nlist;
    float scale;
    int64_t span;  // slots of a span
    float *part;   // [2 spans][d]: sums of long lists' parts
    void *out;
    int lanes, strips;
    int lists; // table_grad_wave_kernel: lists of a wave
};

// A list with more than `span` slots is long: its slots are summed by spans of the
// sorted order, side by side, and joined afterwards.  A span meets at most two long
// lists, the one of its first slot and the one of its last, as any other would lie
// inside it.  A wave per span, end and 512 columns.
template <typename T>
__global__ __launch_bounds__(256) void table_span_kernel(TableGrad g, int64_t waves, int64_t wave0)
{
    const int lane = lane_id();
    const int64_t id = wave0 + (int64_t)blockIdx.x * 4 +
                       __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (id >= waves)
        return;
    const int strips = (g.d + 511) / 512;
    const int64_t which = id / strips;
    const Columns at((int)(id % strips) * 512, lane, 64);
    const int64_t from = which / 2 * g.span, to = min(from + g.span, g.n);
    const int64_t slot = which & 1 ? to - 1 : from;
    // the list of `slot`: the last that begins at or before it
    auto begin = [&](int64_t e) { return part_begin(g.offsets, g.nlist, g.n, (int)e + 1); };
    int64_t first = 0, count = g.nlist;
    while (count > 1) {
        const int64_t step = (count + 63) / 64, i = first + lane * step;
        const uint64_t m = __ballot(i < first + count && begin(i) <= slot);
        const int who = m ? 63 - __builtin_clzll(m) : 0;
        first += who * step;
        count = min(count - who * step, step);
    }
    const int64_t lo = begin(first), hi = begin(first + 1);
    if (slot < lo || slot >= hi || hi - lo <= g.span || (which & 1 && lo <= from))
        return; // of no list, of a short one, or of the list that the first slot has
    const T *grad = static_cast<const T *>(g.grad);
    const int64_t p0 = max(lo, from), p1 = min(hi, to);
    RowSum<T> s;
    s.clear();
    for (int64_t base = p0; base < p1; base += 64) { // 64 slots a load
        const int n = (int)min(p1 - base, (int64_t)64);
        const int mine = lane < n ? g.order[base + lane] : -1;
        const int row = mine >= 0 ? (int)g.k.div((uint32_t)mine) : -1;
        for (int first = 0; first < n; first += kSumRows) {
            int t[kSumRows];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                t[i] = __builtin_amdgcn_readlane(row, first + i);
            typename RowSum<T>::Batch b;
            RowSum<T>::load(b, grad, g.nvec, g.d, at, t);
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                s.add(b, i);
        }
    }
    s.store(g.part + which * g.d, g.d, at, 1.f);
}

// The joined sums of a long list's spans, ascending, added to s.
template <typename T>
__device__ __forceinline__ void add_spans(RowSum<T> &s, const TableGrad &g, int64_t lo, int64_t hi,
                                          Columns at)
{
    // the first span may be the one whose last slot's list this is
    const int64_t i0 = lo / g.span, i1 = (hi + g.span - 1) / g.span;
    for (int64_t i = i0; i < i1; i += kSumRows) {
        int t[kSumRows];
#pragma unroll
        for (int j = 0; j < kSumRows; ++j)
            t[j] = i + j < i1 ? (int)(2 * (i + j) + (lo > (i + j) * g.span ? 1 : 0)) : -1;
        typename RowSum<float>::Batch b;
        RowSum<float>::load(b, g.part, 2 * i1, g.d, at, t);
#pragma unroll
        for (int j = 0; j < kSumRows; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    s.v[h][e] = b.live[j] ? s.v[h][e] + b.x[j][h][e] : s.v[h][e];
    }
}

// Row l of the table's gradient: zero for an empty list, the sum of a short one's rows,
// the joined sums of a long one.  A group of lanes a row: for rows of at most 256
// values (30,000 of 128 to as many lists: 14 us, a wave a row 20; of 512: 22).
template <typename T, typename TO>
__global__ __launch_bounds__(256) void table_grad_kernel(TableGrad g, int64_t groups, int64_t group0)
{
    const int64_t l = group0 + (int64_t)blockIdx.x * (256 / g.lanes) + threadIdx.x / g.lanes;
    if (l >= groups)
        return;
    const Columns at(0, threadIdx.x & (g.lanes - 1), g.lanes);
    const int64_t lo = part_begin(g.offsets, g.nlist, g.n, (int)l + 1);
    const int64_t hi = part_begin(g.offsets, g.nlist, g.n, (int)l + 2);
    RowSum<T> s;
    s.clear();
    if (hi - lo <= g.span)
        s.add_rows(static_cast<const T *>(g.grad), g.nvec, g.k, g.d, at, g.order, lo, hi);
    else
        add_spans(s, g, lo, hi, at);
    s.store(static_cast<TO *>(g.out) + l * g.d, g.d, at, lo < hi ? g.scale : 0.f);
}

// The same for longer rows: a wave has 512 columns of up to kTableRows lists in a row.
// Their offsets are one load, their slots come 64 a load, and the rows eight at a
// time, whichever lists they belong to, so that short lists wait for memory together;
// most rows of a large table are empty and only stored.  Fewer lists a wave where there
// would be fewer than 4096 waves: 65,536 rows of 2048 to 1000 lists 253 us with 16, 75
// with one; 16,384 of 4096 to 32,000 lists 61 and 152.  At 16 the bound is memory: 16,384
// rows of 4096 in bfloat16 to 32,000 lists 134 MB read and 262 written, 6.5 TB/s.
constexpr int kTableRows = 16;

template <typename T, typename TO, bool NT>
__global__ __launch_bounds__(256) void table_grad_wave_kernel(TableGrad g, int64_t waves,
                                                              int64_t wave0)
{
    const int lane = lane_id();
    const int64_t id = wave0 + (int64_t)blockIdx.x * 4 +
                       __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (id >= waves)
        return;
    const int64_t l0 = id / g.strips * g.lists;
    const Columns cols((int)(id % g.strips) * 512, lane, 64);
    const int count = (int)min((int64_t)g.nlist - l0, (int64_t)g.lists);
    const T *grad = static_cast<const T *>(g.grad);
    // positions fit 32 bits; lane i: where list l0 + i begins
    const int begins = (int)part_begin(g.offsets, g.nlist, g.n, (int)(l0 + min(lane, count)) + 1);
    auto begin_of = [&](int i) { return __builtin_amdgcn_readlane(begins, i); };
    RowSum<T> s;
    s.clear();
    int at = 0; // list that is being summed, its next position and its end
    int p = 0, end = 0;
    auto put = [&](int list, float scale) { // an empty list's with 0, whatever the factor is
        s.template store<NT>(static_cast<TO *>(g.out) + (l0 + list) * g.d, g.d, cols, scale);
        s.clear();
    };
    // On to the first list from `at` on that has positions to sum; empty ones are stored,
    // the positions of long ones passed (those are joined at the end).
    auto advance = [&] {
        for (; at < count; ++at) {
            p = begin_of(at);
            end = begin_of(at + 1);
            if (end > p && end - p <= g.span)
                return;
            if (end <= p)
                put(at, 0.f);
        }
    };
    advance();
    while (at < count) {
        // the slots of the next 64 positions, of which eight at a time are taken
        const int base = p, last = begin_of(count);
        const int mine = position_before(base, lane, last) ? g.order[base + lane] : -1;
        const int row = mine >= 0 ? (int)g.k.div((uint32_t)mine) : -1;
        while (at < count && p - base < 64 && p >= base) {
            // p is before the end of its list (and that past `last` only if the offsets do
            // not ascend), so a turn takes at least one position
            const int first = p - base, n = min(min(64 - first, kSumRows), max(last, end) - p);
            int t[kSumRows];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
                t[i] = i < n ? __builtin_amdgcn_readlane(row, min(first + i, 63)) : -1;
            typename RowSum<T>::Batch b;
            RowSum<T>::load(b, grad, g.nvec, g.d, cols, t);
            const int from = p;
#pragma unroll
            for (int i = 0; i < kSumRows; ++i) {
                if (i < n && p == from + i && at < count) { // not past a long list
                    s.add(b, i);
                    ++p;
                    if (p == end) {
                        put(at++, g.scale);
                        advance();
                    }
                }
            }
        }
    }
    for (at = 0; at < count; ++at) {
        const int lo = begin_of(at), hi = begin_of(at + 1);
        if (hi - lo > g.span) {
            add_spans(s, g, lo, hi, cols);
            put(at, g.scale);
        }
    }
}

// Slots of a span: a quarter of the square root of all, as the spans of a long list are
// summed side by side and their sums one after the other.  65,536 rows of 2048 to ten
// lists of very different lengths: 126 us with 64 slots, 93 with 128, 267 with 1024;
// to 1000 such lists 77, 89 and 522; 262,144 rows of 256 to 20: 217, 127 and 207.
static int64_t span_of(int64_t n)
{
    int64_t s = 64;
    while (s < 4096 && 16 * s * s < n)
        s *= 2;
    return s;
}

size_t table_grad_bytes(int64_t n, int d)
{
    const int64_t span = span_of(n);
    return n <= span ? 0 : (size_t)((n + span - 1) / span) * 2 * (size_t)d * 4;
}

template <typename T, typename TO>
static hipError_t table_grad_as(TableGrad g, hipStream_t stream)
{
    const int64_t most = most_blocks(256);
    if (g.n > g.span) {
        const int64_t waves = (g.n + g.span - 1) / g.span * 2 * ((g.d + 511) / 512);
        const int64_t blocks = (waves + 3) / 4;
        for (int64_t b = 0; b < blocks; b += most)
            hipLaunchKernelGGL(table_span_kernel<T>,
                               dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(256),
                               0, stream, g, waves, b * 4);
    }
    g.lanes = piece_lanes((g.d + 7) / 8);
    g.strips = (g.d + 511) / 512;
    if (g.lanes == 64) {
        g.lists = kTableRows;
        while (g.lists > 1 && (int64_t)g.nlist * g.strips < (int64_t)g.lists * 4096)
            g.lists /= 2;
        const int64_t waves = ((int64_t)g.nlist + g.lists - 1) / g.lists * g.strips;
        const int64_t blocks = (waves + 3) / 4;
        // Gradients of half of the last-level cache (256 MB) and more go past it: 32,000 lists
        // of 4096 in float32 (500 MiB) 107 us, 128 through it; 195 MiB 45 and 47; 125 MiB 31
        // and 26.
        const bool past = (int64_t)g.nlist * g.d * (int64_t)sizeof(TO) >= (int64_t)128 << 20;
        const auto kernel = past ? table_grad_wave_kernel<T, TO, true>
                                 : table_grad_wave_kernel<T, TO, false>;
        for (int64_t b = 0; b < blocks; b += most)
            hipLaunchKernelGGL(kernel,
                               dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(256),
                               0, stream, g, waves, b * 4);
        return hipGetLastError();
    }
    const int64_t per = 256 / g.lanes, blocks = (g.nlist + per - 1) / per;
    for (int64_t b = 0; b < blocks; b += most)
        hipLaunchKernelGGL((table_grad_kernel<T, TO>),
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(256), 0,
                           stream, g, (int64_t)g.nlist, b * per);
    return hipGetLastError();
}

template <typename T>
static hipError_t table_grad_to(const TableGrad &g, int out_type, hipStream_t stream)
{
    return out_type == kF32 ? table_grad_as<T, float>(g, stream) : table_grad_as<T, T>(g, stream);
}

hipError_t launch_table_grad(const void *grad, int type, int64_t nvec, int d,
                             const int32_t *offsets, const int32_t *order, int k, int nlist,
                             float scale, int out_type, void *out, void *ws, hipStream_t stream)
{
    TableGrad g{};
    g.grad = grad;
    g.nvec = nvec;
    g.n = nvec * k;
    g.d = d;
    g.offsets = offsets;
    g.order = order;
    g.k = FastDiv((uint32_t)k);
    g.nlist = nlist;
    g.scale = scale;
    g.span = span_of(g.n);
    g.part = static_cast<float *>(ws);
    g.out = out;
    switch (type) {
    case kF32: return table_grad_as<float, float>(g, stream);
    case kBF16: return table_grad_to<__bf16>(g, out_type, stream);
    default: return table_grad_to<_Float16>(g, out_type, stream);
    }
}

} // namespace ivfpq

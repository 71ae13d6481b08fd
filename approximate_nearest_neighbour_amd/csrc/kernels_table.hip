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
// numbers are under way together, then their pieces.
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
#pragma unroll
        for (int e = 0; e < N; ++e)
            v[i].v[e] *= scale;
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

// The sum of sorted rows [lo, hi), eight values of columns c on a lane, in ascending
// order in float32; kSumRows of them under way together.
constexpr int kSumRows = 8;

template <typename T>
struct RowSum {
    static constexpr int N = Piece<T>::N, Q = 8 / N;
    float v[8];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = 0.f;
    }
    __device__ __forceinline__ void add_rows(const T *grad, int64_t nvec, FastDiv k, int d, int c,
                                             const int32_t *order, int64_t lo, int64_t hi)
    {
        for (int64_t p = lo; p < hi; p += kSumRows) {
            int64_t t[kSumRows];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i) {
                const int32_t u = p + i < hi ? order[p + i] : -1;
                t[i] = u >= 0 ? (int64_t)k.div((uint32_t)u) : -1;
            }
            Piece<T> r[kSumRows][Q];
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    if ((uint64_t)t[i] < (uint64_t)nvec)
                        r[i][q].load(grad + t[i] * d + c + q * N, d - c - q * N);
                    else
                        r[i][q].zero();
                }
#pragma unroll
            for (int i = 0; i < kSumRows; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] += r[i][e / N].v[e % N];
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
    const int c = (int)(id % strips) * 512 + lane * 8;
    const int64_t from = which / 2 * g.span, to = min(from + g.span, g.n);
    const int64_t at = which & 1 ? to - 1 : from;
    // the list of slot `at`: the last that begins at or before it
    auto begin = [&](int64_t e) { return part_begin(g.offsets, g.nlist, g.n, (int)e + 1); };
    int64_t first = 0, count = g.nlist;
    while (count > 1) {
        const int64_t step = (count + 63) / 64, i = first + lane * step;
        const uint64_t m = __ballot(i < first + count && begin(i) <= at);
        const int who = m ? 63 - __builtin_clzll(m) : 0;
        first += who * step;
        count = min(count - who * step, step);
    }
    const int64_t lo = begin(first), hi = begin(first + 1);
    if (at < lo || at >= hi || hi - lo <= g.span || (which & 1 && lo <= from))
        return; // of no list, of a short one, or of the list that the first slot has
    if (c >= g.d)
        return;
    RowSum<T> s;
    s.clear();
    s.add_rows(static_cast<const T *>(g.grad), g.nvec, g.k, g.d, c, g.order, max(lo, from),
               min(hi, to));
    float *part = g.part + which * g.d + c;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c + e < g.d)
            part[e] = s.v[e];
}

// Row l of the table's gradient: zero for an empty list, the sum of a short one's rows,
// the joined sums of a long one, ascending.  A group of lanes a row and strip.
template <typename T, typename TO>
__global__ __launch_bounds__(256) void table_grad_kernel(TableGrad g, int64_t groups, int64_t group0)
{
    const int64_t id = group0 + (int64_t)blockIdx.x * (256 / g.lanes) + threadIdx.x / g.lanes;
    if (id >= groups)
        return;
    const int64_t l = id / g.strips;
    const int c = ((int)(id % g.strips) * g.lanes + (threadIdx.x & (g.lanes - 1))) * 8;
    if (c >= g.d)
        return;
    const int64_t lo = part_begin(g.offsets, g.nlist, g.n, (int)l + 1);
    const int64_t hi = part_begin(g.offsets, g.nlist, g.n, (int)l + 2);
    RowSum<T> s;
    s.clear();
    if (hi - lo <= g.span) {
        s.add_rows(static_cast<const T *>(g.grad), g.nvec, g.k, g.d, c, g.order, lo, hi);
    } else {
        for (int64_t i = lo / g.span; i * g.span < hi; ++i) {
            const float *part = g.part + (2 * i + (lo > i * g.span ? 1 : 0)) * g.d + c;
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s.v[e] += c + e < g.d ? part[e] : 0.f;
        }
    }
    TO *out = static_cast<TO *>(g.out) + l * g.d + c;
    constexpr int N = Piece<TO>::N;
#pragma unroll
    for (int q = 0; q < 8 / N; ++q) {
        Piece<TO> o;
#pragma unroll
        for (int e = 0; e < N; ++e)
            o.v[e] = s.v[q * N + e] * g.scale;
        o.store(out + q * N, g.d - c - q * N);
    }
}

// Slots of a span: near the square root of all, so that a long list has about as
// many spans to join as a span has rows.
static int64_t span_of(int64_t n)
{
    int64_t s = 32;
    while (s < 4096 && s * s < n)
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
    g.strips = (g.d + g.lanes * 8 - 1) / (g.lanes * 8);
    const int64_t groups = (int64_t)g.nlist * g.strips, per = 256 / g.lanes;
    const int64_t blocks = (groups + per - 1) / per;
    for (int64_t b = 0; b < blocks; b += most)
        hipLaunchKernelGGL((table_grad_kernel<T, TO>),
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(256), 0,
                           stream, g, groups, b * per);
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

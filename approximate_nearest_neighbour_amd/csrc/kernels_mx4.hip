// Microscaled 4-bit rows and their products.
//
// A row of d values is ceil(d / 32) blocks of 32 (padded with zeros); a block
// holds 32 four-bit floats (e2m1: sign, two exponent bits, one mantissa bit,
// magnitudes 0 .5 1 1.5 2 3 4 6) and one exponent byte s, and stands for
// e2m1 * 2^(s - 127).  Value k of a row sits in byte k / 2, the even one in
// the low nibble.  The format is that of the OCP Microscaling specification
// (MXFP4), which the matrix cores of gfx950 multiply directly.
#include "common.hpp"
#include "internal.hpp"
#include "rows.hpp"

namespace ivfpq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// rows to 4 bits and back
// ---------------------------------------------------------------------------

// Four lanes share a block, eight values each.  s = exponent of the block's
// largest magnitude minus 2 (the exponent of 4, the largest power of two of
// e2m1), at least 0; the values times 2^(127 - s) are exact, then rounded to
// the nearest e2m1, halves to even, saturating at 6.  A block with an
// infinity or a NaN gets s = 255, which stands for NaN.
template <typename T>
__global__ __launch_bounds__(256) void mx4_quantize_kernel(const T *__restrict__ x, uint32_t total,
                                                           int d, int64_t stride, FastDiv per_row,
                                                           uint8_t *__restrict__ codes,
                                                           uint8_t *__restrict__ scales)
{
    const uint32_t g = blockIdx.x * 256u + threadIdx.x; // eighth of a row's values
    if (g >= total)
        return;
    const uint32_t row = per_row.div(g);
    const int at = (int)(g - row * per_row.c) * 8;
    const T *p = x + (int64_t)row * stride + at;
    constexpr int N = Piece<T>::N;
    Piece<T> in[8 / N];
    uint32_t top = 0;
#pragma unroll
    for (int h = 0; h < 8 / N; ++h) {
        in[h].load(p + h * N, d - at - h * N);
#pragma unroll
        for (int i = 0; i < N; ++i)
            top = max(top, __float_as_uint(in[h].v[i]) & 0x7FFFFFFFu);
    }
    top = max(top, xor_lane<1>(top));
    top = max(top, xor_lane<2>(top));
    const uint32_t e = top >> 23;
    const bool bad = e == 255;
    const uint32_t s = e > 2 ? e - 2 : 0;
    const float f = bad ? 0.f : __uint_as_float((254 - s) << 23); // 2^(127 - s)
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = bad ? 0.f : in[i / N].v[i % N] * f;
    uint32_t q = 0;
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[0], y[1], 1.f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[2], y[3], 1.f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[4], y[5], 1.f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[6], y[7], 1.f, 3);
    reinterpret_cast<uint32_t *>(codes)[g] = q;
    if ((g & 3) == 0)
        scales[g >> 2] = bad ? 255 : (uint8_t)s;
}

template <typename T>
static hipError_t quantize_rows(const void *x, int64_t rows, int d, int64_t stride, uint8_t *codes,
                                uint8_t *scales, hipStream_t stream)
{
    const int kb = (d + 31) / 32;
    const int64_t most = 0x7FFFFF00ll / (kb * 4); // rows of one launch: 32-bit piece numbers
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t now = rows - r < most ? rows - r : most;
        const uint32_t total = (uint32_t)(now * kb * 4);
        hipLaunchKernelGGL(mx4_quantize_kernel<T>, dim3((total + 255) / 256), dim3(256), 0, stream,
                           static_cast<const T *>(x) + r * stride, total, d, stride,
                           FastDiv((uint32_t)kb * 4), codes + r * kb * 16, scales + r * kb);
    }
    return hipGetLastError();
}

hipError_t launch_mx4_quantize(const void *x, int type, int64_t rows, int d, int64_t stride,
                               uint8_t *codes, uint8_t *scales, hipStream_t stream)
{
    switch (type) {
    case kF32: return quantize_rows<float>(x, rows, d, stride, codes, scales, stream);
    case kBF16: return quantize_rows<__bf16>(x, rows, d, stride, codes, scales, stream);
    default: return quantize_rows<_Float16>(x, rows, d, stride, codes, scales, stream);
    }
}

// 2^(s - 127) in float32, exact (a denormal for s = 0); NaN for s = 255.
__device__ __forceinline__ float scale_value(uint32_t s)
{
    return __uint_as_float(s == 255 ? 0x7FC00000u : s == 0 ? 0x00400000u : s << 23);
}

// Eight values a lane: four bytes of codes, one piece of output (float32: two).
template <typename T>
__global__ __launch_bounds__(256) void mx4_dequantize_kernel(const uint8_t *__restrict__ codes,
                                                             const uint8_t *__restrict__ scales,
                                                             uint32_t total, int d, FastDiv per_row,
                                                             T *__restrict__ out)
{
    const uint32_t g = blockIdx.x * 256u + threadIdx.x;
    if (g >= total)
        return;
    const uint32_t row = per_row.div(g);
    const int at = (int)(g - row * per_row.c) * 8;
    const uint32_t q = reinterpret_cast<const uint32_t *>(codes)[g];
    const float f = scale_value(scales[g >> 2]);
    const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 0);
    const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 1);
    const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 2);
    const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.f, 3);
    const float v[8] = {v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
    constexpr int N = Piece<T>::N;
    T *p = out + (int64_t)row * d + at;
#pragma unroll
    for (int h = 0; h < 8 / N; ++h) {
        Piece<T> o;
#pragma unroll
        for (int i = 0; i < N; ++i)
            o.v[i] = v[h * N + i] * f;
        o.store(p + h * N, d - at - h * N);
    }
}

template <typename T>
static hipError_t dequantize_rows(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                  void *out, hipStream_t stream)
{
    const int kb = (d + 31) / 32;
    const int64_t most = 0x7FFFFF00ll / (kb * 4);
    for (int64_t r = 0; r < rows; r += most) {
        const int64_t now = rows - r < most ? rows - r : most;
        const uint32_t total = (uint32_t)(now * kb * 4);
        hipLaunchKernelGGL(mx4_dequantize_kernel<T>, dim3((total + 255) / 256), dim3(256), 0,
                           stream, codes + r * kb * 16, scales + r * kb, total, d,
                           FastDiv((uint32_t)kb * 4), static_cast<T *>(out) + r * d);
    }
    return hipGetLastError();
}

hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                 int type, void *out, hipStream_t stream)
{
    switch (type) {
    case kF32: return dequantize_rows<float>(codes, scales, rows, d, out, stream);
    case kBF16: return dequantize_rows<__bf16>(codes, scales, rows, d, out, stream);
    default: return dequantize_rows<_Float16>(codes, scales, rows, d, out, stream);
    }
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------

// The rows of A that tile number t of a list product covers: output rows
// [p0, p1) of one list e (e = nlist: rows past the last list, which are zero).
struct ListTile {
    int e;
    int64_t p0, p1;
};

// Tiles of TM rows, list after list, the rows past offsets[nlist] last.  Every
// wave finds its tile by itself: 64 lists at a time, a lane each, their tile
// counts summed across the lanes.  Offsets outside [0, rows] are clamped.
template <int TM>
__device__ __forceinline__ ListTile find_tile(const int32_t *offsets, int nlist, int64_t rows,
                                              uint32_t t)
{
    const int lane = lane_id();
    const int64_t last = rows;
    uint32_t base = 0;
    for (int e0 = 0; e0 < nlist; e0 += 64) {
        const int e = e0 + lane;
        int64_t lo = 0, hi = 0;
        if (e < nlist) {
            lo = min(max((int64_t)offsets[e], (int64_t)0), last);
            hi = min(max((int64_t)offsets[e + 1], (int64_t)0), last);
        }
        const uint32_t tiles = hi > lo ? (uint32_t)((hi - lo + TM - 1) / TM) : 0;
        const uint32_t upto = wave_inclusive_sum(tiles);
        const uint64_t past = __ballot(base + upto > t);
        if (past) {
            const int who = __builtin_ctzll(past);
            const uint32_t before = base + (uint32_t)__builtin_amdgcn_readlane((int)(upto - tiles), who);
            const int64_t plo = __builtin_amdgcn_readlane((int)lo, who);
            const int64_t phi = __builtin_amdgcn_readlane((int)hi, who);
            const int64_t p0 = plo + (int64_t)(t - before) * TM;
            return {e0 + who, p0, min(p0 + TM, phi)};
        }
        base += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    }
    const int64_t end = min(max((int64_t)offsets[nlist], (int64_t)0), last);
    const int64_t p0 = end + (int64_t)(t - base) * TM;
    return {nlist, p0, min(p0 + TM, last)};
}

__device__ __forceinline__ i32x8 low_half(i32x4 v)
{
    return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}

// 16 x 16 results and 128 products each: a lane holds one block (32 values)
// of row lane % 16 of either operand, block lane / 16 of the four, and its
// exponent byte.  Result i of a lane: row 4 (lane / 16) + i of the first
// operand, row lane % 16 of the second.
__device__ __forceinline__ f32x4 mfma_mx4(i32x4 a, uint32_t sa, i32x4 b, uint32_t sb, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(low_half(a), low_half(b), c, 4, 4, 0,
                                                            (int)sa, 0, (int)sb);
}

// One workgroup: 16 rows of A by 16 rows of B, its waves splitting the blocks
// of a row between them and joining their sums through LDS.
template <typename T, bool LIST, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void mx4_direct_kernel(Mx4Product p)
{
    __shared__ f32x4 part[WAVES][64];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t nt = ((uint32_t)p.n + 15) / 16;
    const uint32_t mt = blockIdx.x / nt;
    const int n0 = (int)(blockIdx.x - mt * nt) * 16;
    ListTile tile{0, (int64_t)mt * 16, min((int64_t)mt * 16 + 16, p.m)};
    if constexpr (LIST)
        tile = find_tile<16>(p.offsets, p.nlist, p.m, mt);
    if (tile.p0 >= tile.p1)
        return;
    const int r = lane & 15, g = lane >> 4;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (tile.e < p.nlist || !LIST) {
        // rows past the tile's end repeat its last row; their results are not stored
        int64_t arow = min(tile.p0 + r, tile.p1 - 1);
        if constexpr (LIST) {
            if (p.order) {
                const int32_t slot = p.order[arow];
                arow = slot >= 0 ? slot / p.k : -1;
            }
            if (arow >= p.arows || arow < 0)
                arow = 0;
        }
        const int64_t brow = (LIST ? (int64_t)tile.e * p.n : 0) + min(n0 + r, p.n - 1);
        const uint8_t *a = p.a + arow * p.kb * 16, *as = p.as + arow * p.kb;
        const uint8_t *b = p.b + brow * p.kb * 16, *bs = p.bs + brow * p.kb;
        for (int k0 = wave * 4; k0 < p.kb; k0 += 4 * WAVES) {
            const int k = k0 + g;
            i32x4 va = {0, 0, 0, 0}, vb = {0, 0, 0, 0};
            uint32_t sa = 127, sb = 127;
            if (k < p.kb) {
                va = *reinterpret_cast<const i32x4 *>(a + (int64_t)k * 16);
                vb = *reinterpret_cast<const i32x4 *>(b + (int64_t)k * 16);
                sa = as[k];
                sb = bs[k];
            }
            acc = mfma_mx4(vb, sb, va, sa, acc);
        }
    }
    part[wave][lane] = acc;
    __syncthreads();
    if (wave != 0)
        return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
        acc += part[w][lane];
    const int64_t row = tile.p0 + r;
    if (row >= tile.p1)
        return;
    T *out = static_cast<T *>(p.out) + row * p.n + n0 + 4 * g;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + 4 * g + i < p.n)
            out[i] = (T)acc[i];
}

// Large tiles.
//
// A workgroup of four waves forms a (32 WM) x (32 WN) tile, each wave a
// quarter of it: WM x WN sums of 16 x 16 in accumulator registers.  A row's
// blocks come eight at a time (a chunk, 128 bytes of codes), both operands'
// rows copied from memory into LDS without passing through registers; while
// the matrix cores work on one chunk the next one arrives in the other half
// of the LDS.  Inside a chunk the operands of the second half are read from
// LDS while the first half is multiplied, and those of the next chunk's first
// half while the second is.
//
// Code rows lie in LDS 128 bytes apart, their eight 16-byte blocks permuted by
// an exclusive or with three bits of the row, so that eight lanes that read
// the same block of eight rows touch all banks once.  Exponent bytes lie as
// the lanes want them: the bytes of all of a lane's operands side by side, so
// that one read brings them and the instruction's byte selector picks.
//
// Results of a lane are consecutive columns: four for each sum, or eight over
// two sums for 16-bit outputs, whose B rows are dealt to the sums accordingly
// (pair_row); every store is then 16 bytes, 64 side by side.

__device__ const uint32_t kZeroBlock[4] = {0, 0, 0, 0};

__device__ __forceinline__ void copy16_to_lds(const uint8_t *src, uint8_t *lds)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)src,
                                     (__attribute__((address_space(3))) void *)lds, 16, 0, 0);
}

// The product with the exponent bytes' selectors as run-time values that are
// constants after unrolling.
__device__ __forceinline__ f32x4 mfma_mx4_sel(i32x4 a, uint32_t sa, int sel_a, i32x4 b, uint32_t sb,
                                              int sel_b, f32x4 c)
{
#define MX4_CASE(A, B)                                                                             \
    case A * 4 + B:                                                                                \
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(low_half(a), low_half(b), c, 4, 4, \
                                                                A, (int)sa, B, (int)sb);
    switch (sel_a * 4 + sel_b) {
        MX4_CASE(0, 0) MX4_CASE(0, 1) MX4_CASE(0, 2) MX4_CASE(0, 3)
        MX4_CASE(1, 0) MX4_CASE(1, 1) MX4_CASE(1, 2) MX4_CASE(1, 3)
        MX4_CASE(2, 0) MX4_CASE(2, 1) MX4_CASE(2, 2) MX4_CASE(2, 3)
        MX4_CASE(3, 0) MX4_CASE(3, 1) MX4_CASE(3, 2) MX4_CASE(3, 3)
    }
#undef MX4_CASE
    return c;
}

// Row of a wave's 16 W that operand row r of sum f holds, and back.  PAIR:
// rows 32 h + 8 q + 4 o + i for f = 2 h + o, r = 4 q + i.
template <bool PAIR>
__device__ __forceinline__ int pair_row(int f, int r)
{
    return PAIR ? (f >> 1) * 32 + (r >> 2) * 8 + (f & 1) * 4 + (r & 3) : f * 16 + r;
}

template <bool PAIR>
__device__ __forceinline__ void pair_row_back(int n, int &f, int &r)
{
    f = PAIR ? (n >> 5) * 2 + ((n >> 2) & 1) : n >> 4;
    r = PAIR ? ((n >> 3) & 3) * 4 + (n & 3) : n & 15;
}

// The three bits of a row that permute its blocks: different for lanes 0..7
// (and 8..15) of an operand read.
template <bool PAIR>
__device__ __forceinline__ int block_swizzle(int row)
{
    return PAIR ? (row & 3) | ((row >> 1) & 4) : row & 7;
}

// Eight exponent bytes from byte c0 of a row's kb, zero past its end.
__device__ __forceinline__ uint64_t scale_bytes(const uint8_t *row, int c0, int kb)
{
    typedef uint64_t U __attribute__((aligned(1)));
    if (c0 + 8 <= kb)
        return *reinterpret_cast<const U *>(row + c0);
    uint64_t v = 0;
    for (int i = 0; c0 + i < kb; ++i)
        v |= (uint64_t)row[c0 + i] << (8 * i);
    return v;
}

// W exponent byte pairs of a lane, two a register.
template <int W>
struct ScaleRegs {
    uint32_t v[(W + 1) / 2];
    __device__ __forceinline__ void read(const uint16_t *p)
    {
        if constexpr (W == 8) {
            const u32x4 t = *reinterpret_cast<const u32x4 *>(p);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = t[i];
        } else if constexpr (W == 4) {
            const u32x2 t = *reinterpret_cast<const u32x2 *>(p);
            v[0] = t[0];
            v[1] = t[1];
        } else if constexpr (W == 2) {
            v[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            v[0] = *p;
        }
    }
};

// Tile numbers: the workgroups of one XCD (every eighth) take a contiguous
// range of tiles, and that range runs through groups of kGroup tiles along m
// by all tiles along n, so that tiles in flight together share operands in
// the XCD's cache.
constexpr uint32_t kGroup = 8;

__device__ __forceinline__ void tile_of_block(uint32_t mt, uint32_t nt, uint32_t &m, uint32_t &n)
{
    const uint32_t all = gridDim.x, x = blockIdx.x & 7, i = blockIdx.x >> 3;
    const uint32_t per = all >> 3, extra = all & 7;
    const uint32_t id = x * per + min(x, extra) + i;
    const uint32_t group = id / (kGroup * nt);
    const uint32_t first = group * kGroup;
    const uint32_t rows = min(kGroup, mt - first);
    const uint32_t in = id - group * kGroup * nt;
    m = first + in % rows;
    n = in / rows;
}

template <typename T, bool LIST, int WM, int WN>
__global__ __launch_bounds__(256) void mx4_tile_kernel(Mx4Product p, uint32_t mtiles,
                                                       uint32_t ntiles)
{
    constexpr bool PAIR = sizeof(T) == 2;
    constexpr int TM = 32 * WM, TN = 32 * WN;
    __shared__ __align__(16) uint8_t code[2][(TM + TN) * 128];
    __shared__ __align__(16) uint16_t scale[2][(TM + TN) * 4];

    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint32_t mt, nt;
    tile_of_block(mtiles, ntiles, mt, nt);
    const int n0 = (int)nt * TN;
    ListTile tile{0, (int64_t)mt * TM, min((int64_t)mt * TM + TM, p.m)};
    if constexpr (LIST)
        tile = find_tile<TM>(p.offsets, p.nlist, p.m, mt);
    if (tile.p0 >= tile.p1)
        return;
    const int wm = wave & 1, wn = wave >> 1;
    const int r = lane & 15, g = lane >> 4;
    T *out = static_cast<T *>(p.out);

    f32x4 acc[WM][WN];
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
        for (int j = 0; j < WN; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (!LIST || tile.e < p.nlist) {
        // rows past the tile's end repeat its last row; their results are not stored
        auto a_row = [&](int row) -> int64_t {
            int64_t q = min(tile.p0 + row, tile.p1 - 1);
            if constexpr (LIST) {
                if (p.order) {
                    const int32_t slot = p.order[q];
                    q = slot >= 0 ? slot / p.k : -1;
                }
                q = q >= 0 && q < p.arows ? q : 0;
            }
            return q;
        };
        auto b_row = [&](int row) -> int64_t {
            return (LIST ? (int64_t)tile.e * p.n : 0) + min(n0 + row, p.n - 1);
        };
        // copies: instruction j of a wave brings rows 8 (4 j + wave) .. + 7, a lane one block
        const int sub = lane >> 3;
        const int ablk = (lane & 7) ^ sub;
        const int bblk = (lane & 7) ^ block_swizzle<PAIR>(wave * 8 + sub);
        const uint8_t *src[WM + WN];
#pragma unroll
        for (int j = 0; j < WM; ++j)
            src[j] = p.a + (a_row((j * 4 + wave) * 8 + sub) * p.kb + ablk) * 16;
#pragma unroll
        for (int j = 0; j < WN; ++j)
            src[WM + j] = p.b + (b_row((j * 4 + wave) * 8 + sub) * p.kb + bblk) * 16;
        // exponent bytes: a thread per row of either operand
        const uint8_t *asrc = p.as + a_row(min((int)threadIdx.x, TM - 1)) * p.kb;
        const uint8_t *bsrc = p.bs + b_row(min((int)threadIdx.x, TN - 1)) * p.kb;
        int bf, br;
        pair_row_back<PAIR>((int)threadIdx.x % (16 * WN), bf, br);
        const int aput = (int)threadIdx.x / (16 * WM) * 64 * WM + ((int)threadIdx.x & 15) * WM +
                         (int)threadIdx.x % (16 * WM) / 16;
        const int bput = TM * 4 + (int)threadIdx.x / (16 * WN) * 64 * WN + br * WN + bf;

        const int chunks = (p.kb + 7) >> 3;
        uint64_t asc = 0, bsc = 0;
        auto fetch = [&](int c) {
            uint8_t *to = code[c & 1] + wave * 1024;
            const int left = p.kb - c * 8;
            const uint8_t *zero = reinterpret_cast<const uint8_t *>(kZeroBlock);
#pragma unroll
            for (int j = 0; j < WM + WN; ++j) {
                const uint8_t *from = src[j];
                if (left < 8) // blocks past the row's end are zero
                    from = (j < WM ? ablk : bblk) < left ? from : zero;
                copy16_to_lds(from, to + (j < WM ? j * 4096 : TM * 128 + (j - WM) * 4096));
                src[j] += 128;
            }
            asc = scale_bytes(asrc, c * 8, p.kb);
            bsc = scale_bytes(bsrc, c * 8, p.kb);
        };
        auto put_scales = [&](int c) {
            uint16_t *to = scale[c & 1];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (TM == 256 || (int)threadIdx.x < TM)
                    to[aput + q * 16 * WM] =
                        (uint16_t)((asc >> (8 * q) & 255) | (asc >> (24 + 8 * q) & 0xFF00));
                if (TN == 256 || (int)threadIdx.x < TN)
                    to[bput + q * 16 * WN] =
                        (uint16_t)((bsc >> (8 * q) & 255) | (bsc >> (24 + 8 * q) & 0xFF00));
            }
        };
        // operand reads: half h of a chunk is blocks 4 h .. 4 h + 3, one a lane group
        int aoff[2], boff[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            aoff[h] = wm * WM * 2048 + r * 128 + (((4 * h + g) ^ (r & 7)) * 16);
#pragma unroll
            for (int o = 0; o < 2; ++o) {
                const int row = pair_row<PAIR>(o, r);
                boff[h][o] = TM * 128 + wn * WN * 2048 + row * 128 +
                             (((4 * h + g) ^ block_swizzle<PAIR>(row)) * 16);
            }
        }
        struct Operands {
            i32x4 a[WM], b[WN];
        };
        auto read_a = [&](const uint8_t *from, int h, int i) {
            return *reinterpret_cast<const i32x4 *>(from + aoff[h] + i * 2048);
        };
        auto read_b = [&](const uint8_t *from, int h, int j) {
            return *reinterpret_cast<const i32x4 *>(
                from + boff[h][j & 1] + (PAIR ? (j >> 1) * 4096 : (j & ~1) * 2048));
        };
        ScaleRegs<WM> sa;
        ScaleRegs<WN> sb;
        const int sa_at = wm * 64 * WM + (g * 16 + r) * WM;
        const int sb_at = TM * 4 + wn * 64 * WN + (g * 16 + r) * WN;

        fetch(0);
        __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
        put_scales(0);
        lds_barrier();
        if (chunks > 1)
            fetch(1);
        Operands x, y;
#pragma unroll
        for (int i = 0; i < WM; ++i)
            x.a[i] = read_a(code[0], 0, i);
#pragma unroll
        for (int j = 0; j < WN; ++j)
            x.b[j] = read_b(code[0], 0, j);
        sa.read(scale[0] + sa_at);
        sb.read(scale[0] + sb_at);
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
            const uint8_t *now = code[c & 1], *next = code[(c + 1) & 1];
#pragma unroll
            for (int i = 0; i < WM; ++i)
                y.a[i] = read_a(now, 1, i);
#pragma unroll
            for (int j = 0; j < WN; ++j)
                y.b[j] = read_b(now, 1, j);
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j)
                    acc[i][j] = mfma_mx4_sel(x.b[j], sb.v[j / 2], (j & 1) * 2, x.a[i], sa.v[i / 2],
                                             (i & 1) * 2, acc[i][j]);
            if (c + 1 < chunks) {
                __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
                put_scales(c + 1);
            }
            lds_barrier(); // everyone has read this chunk and brought the next one
            if (c + 2 < chunks)
                fetch(c + 2);
            ScaleRegs<WM> ta;
            ScaleRegs<WN> tb;
            ta.read(scale[(c + 1) & 1] + sa_at);
            tb.read(scale[(c + 1) & 1] + sb_at);
#pragma unroll
            for (int i = 0; i < WM; ++i)
                x.a[i] = read_a(next, 0, i);
#pragma unroll
            for (int j = 0; j < WN; ++j)
                x.b[j] = read_b(next, 0, j);
#pragma unroll
            for (int i = 0; i < WM; ++i)
#pragma unroll
                for (int j = 0; j < WN; ++j)
                    acc[i][j] = mfma_mx4_sel(y.b[j], sb.v[j / 2], (j & 1) * 2 + 1, y.a[i],
                                             sa.v[i / 2], (i & 1) * 2 + 1, acc[i][j]);
            sa = ta;
            sb = tb;
        }
    }
    constexpr int N = Piece<T>::N;
#pragma unroll
    for (int i = 0; i < WM; ++i) {
        const int64_t row = tile.p0 + (wm * WM + i) * 16 + r;
        if (row >= tile.p1)
            continue;
#pragma unroll
        for (int j = 0; j < WN; j += N / 4) {
            const int n = n0 + wn * WN * 16 + (PAIR ? j * 16 + g * 8 : j * 16 + g * 4);
            Piece<T> o;
#pragma unroll
            for (int q = 0; q < N; ++q)
                o.v[q] = acc[i][j + q / 4][q % 4];
            o.store(out + row * p.n + n, p.n - n);
        }
    }
}

template <typename T, bool LIST, int WM, int WN>
static hipError_t tiles_as(const Mx4Product &p, hipStream_t stream)
{
    const int64_t nt = (p.n + 32ll * WN - 1) / (32 * WN);
    int64_t mt = (p.m + 32ll * WM - 1) / (32 * WM);
    if (LIST) // every list may end inside a tile, and so may the last rows
        mt = p.m / (32 * WM) + (p.m < (int64_t)p.nlist + 1 ? p.m : (int64_t)p.nlist + 1);
    hipLaunchKernelGGL((mx4_tile_kernel<T, LIST, WM, WN>), dim3((unsigned)(nt * mt)), dim3(256), 0,
                       stream, p, (uint32_t)mt, (uint32_t)nt);
    return hipGetLastError();
}

template <typename T>
static hipError_t product_as(const Mx4Product &p, hipStream_t stream)
{
    if (p.m > 64) {
        if (p.offsets)
            return tiles_as<T, true, 4, 4>(p, stream);
        if (p.m > 1024)
            return tiles_as<T, false, 8, 8>(p, stream);
        return tiles_as<T, false, 4, 4>(p, stream);
    }
    const int64_t nt = ((int64_t)p.n + 15) / 16;
    int64_t mt = (p.m + 15) / 16;
    if (p.offsets) // every list may end inside a tile, and so may the last rows
        mt = p.m / 16 + (p.m < (int64_t)p.nlist + 1 ? p.m : (int64_t)p.nlist + 1);
    if (nt * mt > 0x7FFFFFFFll)
        return hipErrorInvalidValue;
    const dim3 grid((unsigned)(nt * mt));
    if (p.offsets)
        hipLaunchKernelGGL((mx4_direct_kernel<T, true, 4>), grid, dim3(256), 0, stream, p);
    else
        hipLaunchKernelGGL((mx4_direct_kernel<T, false, 4>), grid, dim3(256), 0, stream, p);
    return hipGetLastError();
}

hipError_t launch_mx4_product(const Mx4Product &p, int type, hipStream_t stream)
{
    switch (type) {
    case kF32: return product_as<float>(p, stream);
    case kBF16: return product_as<__bf16>(p, stream);
    default: return product_as<_Float16>(p, stream);
    }
}

} // namespace ivfpq

// Microscaled 4-bit rows and their products.
//
// A row of d values is ceil(d / 32) blocks of 32 (padded with zeros); a block
// holds 32 four-bit floats (e2m1: sign, two exponent bits, one mantissa bit,
// magnitudes 0 .5 1 1.5 2 3 4 6) and one exponent byte s, and stands for
// e2m1 * 2^(s - 127).  Value k of a row sits in byte k / 2, the even one in
// the low nibble.  The format is that of the OCP Microscaling specification
// (MXFP4), which the matrix cores of gfx950 multiply directly.
#include "common.hpp"
#include "mx4_plan.hpp"
#include "rows.hpp"
#include "rows_internal.hpp"

namespace ivfpq {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// rows to 4 bits and back
// ---------------------------------------------------------------------------

// Four lanes share a block, eight values each.  s = exponent of the block's
// largest magnitude minus 2 (the exponent of 4, the largest power of two of
// e2m1), at least 0; the values times 2^(127 - s) are exact, then rounded to
// the nearest e2m1, halves to even, saturating at 6.  A block with an
// infinity or a NaN gets s = 255, which stands for NaN.  Bound by the rows'
// bytes: a lane reads 16 or 32 of them side by side and writes four, a wave 16
// whole blocks.  1,000,000 x 96 in float32 94 us, 4.6 TB/s (a large copy: 4.8).
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

// Eight values a lane: four bytes of codes, one piece of output (float32: two),
// each value rounded once from its exact float32 product.  Bound by the bytes:
// 1,000,000 x 96 to float32 93 us, 4.7 TB/s.
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
// [p0, p1) of one list e (e = nlist: rows of no list, which are zero).
struct ListTile {
    int e;
    int64_t p0, p1;
};

// Tiles of TM rows, list after list, then the rows before offsets[0] and those
// past offsets[nlist].  Every wave finds its tile by itself: 64 lists at a time, a
// lane each, their tile counts summed across the lanes.  Offsets outside [0, rows]
// are clamped.  The walk grows with the lists and so does the number of waves, so
// this is made for some hundred lists: 16,384 rows, 256 x 256, of 128 lists 10 us,
// of 1024 lists 38 us, of 8192 lists 1.4 ms, of 65,536 lists 18 ms.
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
            const uint32_t before =
                base + (uint32_t)__builtin_amdgcn_readlane((int)(upto - tiles), who);
            const int64_t plo = __builtin_amdgcn_readlane((int)lo, who);
            const int64_t phi = __builtin_amdgcn_readlane((int)hi, who);
            const int64_t p0 = plo + (int64_t)(t - before) * TM;
            return {e0 + who, p0, min(p0 + TM, phi)};
        }
        base += (uint32_t)__builtin_amdgcn_readlane((int)upto, 63);
    }
    const int64_t begin = min(max((int64_t)offsets[0], (int64_t)0), last);
    const int64_t end = min(max((int64_t)offsets[nlist], (int64_t)0), last);
    const uint32_t before = (uint32_t)((begin + TM - 1) / TM);
    if (t - base < before) {
        const int64_t p0 = (int64_t)(t - base) * TM;
        return {nlist, p0, min(p0 + TM, begin)};
    }
    const int64_t p0 = end + (int64_t)(t - base - before) * TM;
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

// Few rows of A: bound by the bytes of B, which go from memory straight to
// registers.  A wave forms 16 rows by 16 columns; of a workgroup's eight, KS
// share the blocks of the same columns out between them and join their sums
// through LDS.  Sixteen blocks a turn, a lane group g taking blocks 4 s + g of
// the four steps s (64 bytes side by side a row and step); the next turn's
// operands are under way while this one's are multiplied.  The exponent bytes
// of a turn are one 16-byte load, of which word s, byte g is the lane's.  Sums
// are float32, rounded once to the output's type.  One row by 8192 x 4096: 5.8
// us for 17.8 MB, of which the launch is about half; 4 rows of 8 lists each, 25
// of 64 matrices of 2048 x 2048: 14 us for 56 MB, 4 TB/s (a streaming read: 6.45).
template <typename T, bool LIST, int KS>
__global__ __launch_bounds__(512) void mx4_direct_kernel(Mx4Product p, uint32_t ntiles)
{
    constexpr int GROUPS = 8 / KS;
    __shared__ f32x4 part[KS == 1 ? 1 : 8][64];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t block = blockIdx.x + p.block0, mt = block / ntiles;
    const int n0 = ((int)(block - mt * ntiles) * GROUPS + wave / KS) * 16;
    ListTile tile{0, (int64_t)mt * 16, min((int64_t)mt * 16 + 16, p.m)};
    if constexpr (LIST)
        tile = find_tile<16>(p.offsets, p.nlist, p.m, mt);
    if (tile.p0 >= tile.p1)
        return;
    const int r = lane & 15, g = lane >> 4;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
    if (tile.e < p.nlist || !LIST) {
        const int64_t brow = (LIST ? (int64_t)tile.e * p.n : 0) + min(n0 + r, p.n - 1);
        const uint8_t *b = p.b + brow * p.kb * 16, *bs = p.bs + brow * p.kb;
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
        const uint8_t *a = p.a + arow * p.kb * 16, *as = p.as + arow * p.kb;
        struct Turn {
            i32x4 b[4], a[4];
            u32x4 sb, sa;
        };
        auto load = [&](int k0, Turn &t) {
            typedef uint32_t U __attribute__((ext_vector_type(4), aligned(1)));
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int64_t at = (int64_t)min(k0 + 4 * s + g, p.kb - 1) * 16;
                t.b[s] = *reinterpret_cast<const i32x4 *>(b + at);
                t.a[s] = *reinterpret_cast<const i32x4 *>(a + at);
            }
            if (k0 + 16 <= p.kb) {
                t.sb = *reinterpret_cast<const U *>(bs + k0) >> (8 * g);
                t.sa = *reinterpret_cast<const U *>(as + k0) >> (8 * g);
            } else { // the row's end: bytes of zero past it (two factors of 2^-127)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int k = k0 + 4 * s + g;
                    t.sb[s] = k < p.kb ? bs[k] : 0;
                    t.sa[s] = k < p.kb ? as[k] : 0;
                }
            }
        };
        auto multiply = [&](const Turn &t) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
                acc = mfma_mx4(t.b[s], t.sb[s], t.a[s], t.sa[s], acc);
        };
        int k0 = wave % KS * 16;
        Turn x, y;
        if (k0 < p.kb)
            load(k0, x);
        for (; k0 < p.kb; k0 += 32 * KS) {
            if (k0 + 16 * KS < p.kb)
                load(k0 + 16 * KS, y);
            multiply(x);
            if (k0 + 16 * KS >= p.kb)
                break;
            if (k0 + 32 * KS < p.kb)
                load(k0 + 32 * KS, x);
            multiply(y);
        }
    }
    if constexpr (KS > 1) {
        part[wave][lane] = acc;
        __syncthreads();
        if (wave % KS != 0)
            return;
#pragma unroll
        for (int w = 1; w < KS; ++w)
            acc += part[wave + w][lane];
    }
    typedef T V __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    const int n = n0 + 4 * g;
    const int64_t row = tile.p0 + r;
    if (row >= tile.p1 || n >= p.n)
        return;
    T *out = static_cast<T *>(p.out) + row * p.n + n;
    if (n + 4 <= p.n) {
        V v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (T)acc[i];
        *reinterpret_cast<V *>(out) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < p.n)
                out[i] = (T)acc[i];
    }
}

// Large tiles.
//
// A workgroup of MW x NW waves forms a tile of (32 WM MW) x (32 WN NW) results,
// each wave its share of WM x WN sums of 32 x 32 in accumulator registers.  A
// row's blocks come eight at a time (a chunk: 128 bytes of codes, four matrix
// instructions deep), both operands' rows copied from memory into LDS without
// passing through registers; one chunk is multiplied while the next arrives in
// the other LDS object.  The operands of one step are read from LDS while those
// of the step before are multiplied, across the chunks' ends too.
//
// Code rows lie in LDS 128 bytes apart, their eight 16-byte blocks permuted by
// an exclusive or with three bits of the row, so that sixteen lanes that read
// the same block of sixteen rows touch all banks once.  A row's exponent bytes
// lie as two words, the even blocks' and the odd ones': a lane's four steps are
// the four bytes of one word, picked by the instruction's byte selector.
//
// Results: for float32 a lane holds one column of sixteen rows, and a store
// covers 128 bytes of two rows.  For 16-bit outputs the operands change places:
// a lane holds four times four consecutive columns of one row, B's rows dealt
// to the sums so that pairs of these are eight consecutive columns (deal_row).
// In all but the small tiles they go through LDS, so that a store covers 64 or 128
// bytes of each row.
//
// A workgroup makes a run of tiles along n with the same rows of A: the next
// tile's first chunk arrives while the last one of a tile is multiplied, and a
// tile's stores are under way while the next is begun.
//
// 8192 x 8192 x 8192 to bfloat16: 266 us, 4.1 PF (the matrix instructions
// alone, from registers, 6.45 PF: the clock falls to 1.3-1.6 GHz; here 1.8 GHz
// with the matrix cores busy 53 % of the cycles).  Without the copies of operands
// it would be 208 us, without the stores 249; operands that all come from the
// XCD's cache change nothing.  A chunk takes about 3900 cycles, 2048 of them for
// its products; 64 KB of it are copied into LDS and the waves read 192 KB, 2048
// cycles as well at 128 bytes a cycle (the counter of LDS reads is active in 24 %
// of the cycles).  The 16-bit kernels keep 3 (lists: 6) registers of a tile's
// stores in scratch memory.  128 lists of 512 rows on average, 2048 x 2048: 240
// us, of which the stores are 65 (268 MB), the matrices from memory 20, rows that
// only fill tiles up 28.  128 x 128 tiles for both: 365 and 289 us.
//
// ONE: rows of at most one chunk (d <= 256) and single tiles, bound by the
// stores of the results: small tiles in row order, several workgroups a CU,
// some storing while others load (1000 x 262,144 x 96 in float32: 183 us for
// 1.05 GB of results, a plain fill 154 us; 128 x 128 tiles in the order of the
// large kernel 212 us; runs of tiles 247 us, each waiting for the stores of
// the one before).

// A value that is the same in every lane, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

// A memory range for the copies: reads past it give zeros (the scalar offset
// counts in that check).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t *base, int64_t from,
                                                            int64_t bytes)
{
    from = uniform(from);
    const uint32_t size =
        (uint32_t)uniform(min(max(bytes - from, (int64_t)0), (int64_t)0xFFFFFFFF));
    const uint8_t *p = base + from;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(p), 0, (int)size, 0x00027000);
}

// 16 bytes a lane to consecutive LDS addresses, from byte off (a lane's) + at.
__device__ __forceinline__ void copy16_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, int at,
                                              uint8_t *lds)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        from, (__attribute__((address_space(3))) void *)lds, 16, (int)off, at, 0, 0);
}

// Until at most N of this wave's memory operations are under way (the
// compiler knows the instruction, and so what need not be waited for again).
template <int N>
__device__ __forceinline__ void wait_vm()
{
    __asm__ volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4) << 14);
    __asm__ volatile("" ::: "memory");
}

__device__ __forceinline__ f32x16 mfma_mx4_32(i32x4 a, uint32_t sa, i32x4 b, uint32_t sb, int step,
                                              f32x16 c)
{
#define MX4_CASE(S)                                                                               \
    case S:                                                                                       \
        return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low_half(a), low_half(b), c, 4, 4, \
                                                               S, (int)sa, S, (int)sb);
    switch (step) { // a constant after unrolling
        MX4_CASE(0) MX4_CASE(1) MX4_CASE(2) MX4_CASE(3)
    }
#undef MX4_CASE
    return c;
}

// Row of B's 32 that operand row r of a sum holds.  A lane's results i = 4 a + c
// are operand rows 8 a + 4 half + c; PAIR makes them rows 16 (a / 2) + 8 half +
// 4 (a % 2) + c, else they are those rows themselves.
template <bool PAIR>
__device__ __forceinline__ int deal_row(int r)
{
    return PAIR ? (r >> 4) * 16 + ((r >> 2) & 1) * 8 + ((r >> 3) & 1) * 4 + (r & 3) : r;
}

// Sixteen exponent bytes of a row, two chunks' worth.  The load may be waited
// for later than it is issued, so what depends on its position comes apart.
struct ScaleBytes {
    u32x4 v;
    int early; // bytes that the load began early
    // from byte `at` on, but never past `total` (at least 16): near the end it starts earlier
    __device__ __forceinline__ void load(const uint8_t *scales, int64_t at, int64_t total)
    {
        typedef uint32_t U __attribute__((ext_vector_type(4), aligned(1)));
        const int64_t from = min(at, total - 16);
        early = (int)(at - from);
        v = *reinterpret_cast<const U *>(scales + from);
    }
    // The first eight of them (ODD: the others), those past the first `left`
    // zero: their blocks vanish from the sums (two factors of 2^-127) whatever
    // codes stand there.
    template <int ODD>
    __device__ __forceinline__ uint64_t get(int left) const
    {
        const int skip = early + 8 * ODD;
        const uint64_t lo = (uint64_t)v[1] << 32 | v[0], hi = (uint64_t)v[3] << 32 | v[2];
        const uint64_t w = skip < 8 ? lo : hi;
        uint64_t r = w >> (8 * (skip & 7));
        r |= skip > 0 && skip < 8 ? hi << (64 - 8 * (skip & 7)) : 0;
        const uint64_t keep = left >= 8 ? ~0ull : left > 0 ? (1ull << (8 * left)) - 1 : 0;
        return skip < 16 ? r & keep : 0;
    }
};

// Tile numbers.  Tiles go in groups of `high` along m by all runs along n, so
// that those in flight together on one XCD share operands in its cache.  The
// workgroups of an XCD (every eighth) take a contiguous range of them; for
// lists, whose number of tiles is only bounded, every eighth group, so that the
// tiles that turn out empty, the last ones, are the same share for all.
struct TileOrder {
    uint32_t mt, nruns, high, blocks;
    template <bool LIST>
    __device__ __forceinline__ void of_block(uint32_t block, uint32_t &m, uint32_t &n) const
    {
        const uint32_t x = block & 7, i = block >> 3, size = high * nruns;
        uint32_t id;
        if constexpr (LIST) {
            id = (i / size * 8 + x) * size + i % size;
        } else {
            const uint32_t per = blocks >> 3, extra = blocks & 7;
            id = x * per + min(x, extra) + i;
        }
        const uint32_t first = id / size * high;
        const uint32_t rows = first < mt ? min(high, mt - first) : high;
        const uint32_t in = id % size;
        m = first + in % rows;
        n = in / rows;
    }
};

// KG: groups of MW x NW waves of a workgroup that share the chunks of one tile
// out between them (two chunks in a row each) and join their sums through LDS.
template <typename T, bool LIST, int WM, int WN, int MW, int NW, int KG, bool ONE>
__global__ __launch_bounds__(64 * MW * NW * KG) void mx4_tile_kernel(Mx4Product p, TileOrder order,
                                                                     int most)
{
    constexpr bool PAIR = sizeof(T) == 2;
    constexpr int WAVES = MW * NW, TM = 32 * WM * MW, TN = 32 * WN * NW;
    constexpr int CA = TM / (8 * WAVES), CB = TN / (8 * WAVES); // copies of a wave, of a chunk
    static_assert(TM % (8 * WAVES) == 0 && TN % (8 * WAVES) == 0 && WAVES % 2 == 0, "copies");
    static_assert(TM + TN <= 64 * WAVES, "a thread per row brings the exponent bytes");
    constexpr int PLACE = (TM + TN) * 128; // bytes of a chunk
    // two objects, so that the compiler knows a copy into one from a read of the other
    __shared__ __align__(16) uint8_t both0[KG * PLACE], both1[ONE ? 16 : KG * PLACE];
    __shared__ uint32_t scales[KG][ONE ? 1 : 2][2][TM + TN];

    const int lane = lane_id();
    const int wave_all = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int kg = KG == 1 ? 0 : wave_all / WAVES, wave = KG == 1 ? wave_all : wave_all % WAVES;
    uint8_t *const code0 = both0 + kg * PLACE, *const code1 = both1 + kg * PLACE;
    auto &scale = scales[kg];
    const uint32_t block = blockIdx.x + p.block0;
    uint32_t mt, nr;
    if constexpr (ONE) { // bound by its stores: workgroups side by side write side by side
        mt = block / order.nruns;
        nr = block - mt * order.nruns;
    } else {
        order.of_block<LIST>(block, mt, nr);
    }
    if (mt >= order.mt || nr >= order.nruns)
        return;
    const int n0 = (int)nr * most * TN;
    const int run = run_tiles(p.n, n0, TN, most);
    ListTile tile{0, (int64_t)mt * TM, min((int64_t)mt * TM + TM, p.m)};
    if constexpr (LIST)
        tile = find_tile<TM>(p.offsets, p.nlist, p.m, mt);
    if (tile.p0 >= tile.p1)
        return;
    tile.p0 = uniform(tile.p0);
    const int wm = wave % MW, wn = wave / MW;
    const int r = lane & 31, half = lane >> 5;
    T *out = static_cast<T *>(p.out);

    f32x16 acc[WM][WN];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    acc[i][j][q] = 0.f;
    };
    typedef T T8 __attribute__((ext_vector_type(8)));
    typedef T T8U __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    // the sums to the tile's rows, columns at and on
    auto put = [&](int at) {
        at += wn * WN * 32;
        // not known to be the same from tile to tile, or every address of the
        // sums is computed once and kept in registers through the products
        int64_t row0 = tile.p0;
        __asm__ volatile("" : "+s"(row0));
        if constexpr (!PAIR) {
#pragma unroll
            for (int j = 0; j < WN; ++j) {
                const int n = at + j * 32 + r;
                if (n >= p.n)
                    continue;
#pragma unroll
                for (int i = 0; i < WM; ++i)
#pragma unroll
                    for (int q = 0; q < 16; ++q) {
                        const int64_t row =
                            row0 + (wm * WM + i) * 32 + (q >> 2) * 8 + half * 4 + (q & 3);
                        if (row < tile.p1)
                            out[row * p.n + n] = (T)acc[i][j][q];
                    }
            }
        } else if constexpr (WN == 1 && !ONE) {
#pragma unroll
            for (int i = 0; i < WM; ++i) {
                const int64_t row = row0 + (wm * WM + i) * 32 + r;
                if (row >= tile.p1)
                    continue;
#pragma unroll
                for (int j = 0; j < WN; ++j)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int n = at + j * 32 + 16 * q + 8 * half;
                        Piece<T> o;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            o.v[e] = acc[i][j][q * 8 + e];
                        o.store(out + row * p.n + n, p.n - n);
                    }
            }
        } else {
            // Through LDS (this wave's part of what no copy is on its way to), so
            // that a store is whole rows of the wave's columns: 8192 x 8192 x 8192
            // 281 -> 266 us, 8000 x 8001 x 1024 92 -> 58 us, 1000 x 100,001 x 96 91 ->
            // 54 us.  Small tiles, which are not bound by their stores, store 16 bytes
            // a lane themselves: 128 lists of 16 rows, 1024 x 1024, 18.5 us, through
            // LDS 21.8 us.
            constexpr int BR = WN * 4, ROWB = BR * 16, PART = (TM + TN) * 128 / WAVES;
            constexpr int SLAB = PART / (32 * ROWB) < WM ? PART / (32 * ROWB) : WM;
            static_assert(SLAB >= 1 && WM % SLAB == 0, "rows through LDS");
            uint8_t *mine = (ONE ? code0 : code1) + wave * PART;
#pragma unroll
            for (int i0 = 0; i0 < WM; i0 += SLAB) {
#pragma unroll
                for (int i = 0; i < SLAB; ++i)
#pragma unroll
                    for (int j = 0; j < WN; ++j)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            T8 o;
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o[e] = (T)acc[i0 + i][j][q * 8 + e];
                            const int b = (j * 4 + q * 2 + half) ^ (r & (BR - 1));
                            *reinterpret_cast<T8 *>(mine + (i * 32 + r) * ROWB + b * 16) = o;
                        }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                for (int k = 0; k < SLAB * 32 * BR / 64; ++k) {
                    const int line = (k * 64 + lane) / BR, b = lane % BR;
                    const T8 o = *reinterpret_cast<const T8 *>(mine + line * ROWB +
                                                               (b ^ (line & (BR - 1))) * 16);
                    const int64_t row = row0 + (wm * WM + i0) * 32 + line;
                    const int n = at + b * 8;
                    if (row >= tile.p1 || n >= p.n)
                        continue;
                    T *to = out + row * p.n + n;
                    if (n + 8 <= p.n) {
                        *reinterpret_cast<T8U *>(to) = o;
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < p.n)
                                to[e] = o[e];
                    }
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            }
            lds_barrier(); // before copies to where other waves' rows may still lie
        }
    };
    clear();
    if (LIST && tile.e == p.nlist) {
        for (int t = 0; t < run && kg == 0; ++t)
            put(n0 + t * TN);
        return;
    }

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
    // copies: instruction j of a wave brings rows 8 (WAVES j + wave) .. + 7, a lane one block
    const int sub = lane >> 3;
    const int blk = (lane & 7) ^ (((wave & 1) * 8 + sub) >> 1);
    const int64_t arow0 = LIST && p.order ? 0 : tile.p0; // rows are counted from here
    const int64_t brow0 = (LIST ? (int64_t)tile.e * p.n : 0) + n0;
    const int64_t brows = (LIST ? (int64_t)p.nlist : 1) * p.n;
    uint32_t off[CA + CB]; // byte of the lane's block in its row's first chunk
#pragma unroll
    for (int j = 0; j < CA; ++j)
        off[j] = (uint32_t)(a_row((j * WAVES + wave) * 8 + sub) - arow0) * (uint32_t)p.kb * 16 +
                 blk * 16;
#pragma unroll
    for (int j = 0; j < CB; ++j)
        off[CA + j] = (uint32_t)((j * WAVES + wave) * 8 + sub) * (uint32_t)p.kb * 16 + blk * 16;
    const auto abuf = buffer_of(p.a, arow0 * p.kb * 16, p.arows * p.kb * 16);
    auto b_of = [&](int t) { // B's rows from tile t of the run on
        return buffer_of(p.b, (brow0 + t * TN) * p.kb * 16, brows * p.kb * 16);
    };
    const int chunks = (p.kb + 7) >> 3;
    const int own = own_chunks(chunks, KG);
    auto chunk_of = [&](int c) { return row_chunk(c, kg, KG); };
    // Chunk c into its LDS place.  What lies past a row's end (the next row's
    // blocks, or zeros past the matrix) is multiplied too, with exponent bytes
    // of zero; rows past the last one of B give results that are not stored.
    // `at` is less than a row's bytes, and either buffer starts with a row of its
    // matrix, so the bytes left are always more than `at`.
    auto fetch_a = [&](int c, uint8_t *to) {
        const int at = __builtin_amdgcn_readfirstlane(chunk_byte(c, kg, KG, chunks));
#pragma unroll
        for (int j = 0; j < CA; ++j)
            copy16_to_lds(abuf, off[j], at, to + wave * 1024 + j * WAVES * 1024);
    };
    auto fetch_b = [&](__amdgpu_buffer_rsrc_t from, int c, uint8_t *to) {
        const int at = __builtin_amdgcn_readfirstlane(chunk_byte(c, kg, KG, chunks));
#pragma unroll
        for (int j = 0; j < CB; ++j)
            copy16_to_lds(from, off[CA + j], at, to + wave * 1024 + j * WAVES * 1024);
    };
    // exponent bytes: a thread per row of A, then of B
    const int srow = (int)threadIdx.x - kg * 64 * WAVES;
    const bool of_a = srow < TM;
    const uint8_t *sfrom = of_a ? p.as : p.bs;
    const int64_t sline = of_a ? a_row(srow) : brow0 + srow - TM;
    const int64_t slast = (of_a ? p.arows : brows) - 1;
    ScaleBytes bytes;
    auto load_scales = [&](int t, int c) { // chunks c and c + 1 of tile t
        const int64_t line = min(of_a ? sline : sline + t * TN, slast);
        bytes.load(sfrom, line * p.kb + min(chunk_of(c), chunks - 1) * 8, (slast + 1) * p.kb);
    };
    auto put_scales = [&](int c, auto odd) { // chunk c, the first or the other one loaded
        constexpr int ODD = decltype(odd)::value;
        const uint64_t v = bytes.get<ODD>(p.kb - chunk_of(c) * 8);
        if (TM + TN == 64 * WAVES || srow < TM + TN) {
            const uint32_t lo = (uint32_t)v, hi = (uint32_t)(v >> 32);
            scale[ODD][0][srow] = __builtin_amdgcn_perm(hi, lo, 0x06040200);
            scale[ODD][1][srow] = __builtin_amdgcn_perm(hi, lo, 0x07050301);
        }
    };
    // operand reads: step s takes blocks 2 s and 2 s + 1, one a half wave
    const int brow = deal_row<PAIR>(r);
    int aoff[4], boff[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        aoff[s] = wm * WM * 4096 + r * 128 + (((2 * s + half) ^ ((r >> 1) & 7)) * 16);
        boff[s] = wn * WN * 4096 + brow * 128 + (((2 * s + half) ^ ((brow >> 1) & 7)) * 16);
    }
    const int sa_at = wm * WM * 32 + r, sb_at = TM + wn * WN * 32 + brow;
    struct Operands {
        i32x4 a[WM], b[WN];
    };
    auto read = [&](const uint8_t *froma, const uint8_t *fromb, int s, Operands &o) {
#pragma unroll
        for (int i = 0; i < WM; ++i)
            o.a[i] = *reinterpret_cast<const i32x4 *>(froma + aoff[s] + i * 4096);
#pragma unroll
        for (int j = 0; j < WN; ++j)
            o.b[j] = *reinterpret_cast<const i32x4 *>(fromb + boff[s] + j * 4096);
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    Operands o[2];
    uint32_t sa[WM], sb[WN]; // exponent bytes of the chunk, a lane's four steps
    auto multiply = [&](int s) {
#pragma unroll
        for (int i = 0; i < WM; ++i)
#pragma unroll
            for (int j = 0; j < WN; ++j)
                acc[i][j] = PAIR ? mfma_mx4_32(o[s & 1].b[j], sb[j], o[s & 1].a[i], sa[i], s,
                                               acc[i][j])
                                 : mfma_mx4_32(o[s & 1].a[i], sa[i], o[s & 1].b[j], sb[j], s,
                                               acc[i][j]);
    };
    // The chunk that lies in the places given but for its last step, whose
    // operands are left in registers: they are multiplied while the next
    // chunk's first ones are read (`before`: so were those of the chunk before).
    // `copies` brings the next chunk and `scales` its exponent bytes.
    auto chunk = [&](auto parity, bool before, const uint8_t *froma, const uint8_t *fromb,
                     auto copies, auto scales) {
        constexpr int ODD = decltype(parity)::value;
        uint32_t na[WM], nb[WN];
        read(froma, fromb, 0, o[0]);
#pragma unroll
        for (int i = 0; i < WM; ++i)
            na[i] = scale[ODD][half][sa_at + i * 32];
#pragma unroll
        for (int j = 0; j < WN; ++j)
            nb[j] = scale[ODD][half][sb_at + j * 32];
        __builtin_amdgcn_sched_barrier(0);
        copies();
        __builtin_amdgcn_sched_barrier(0);
        if (before)
            multiply(3);
#pragma unroll
        for (int i = 0; i < WM; ++i)
            sa[i] = na[i];
#pragma unroll
        for (int j = 0; j < WN; ++j)
            sb[j] = nb[j];
        scales();
#pragma unroll
        for (int s = 0; s < 3; ++s) {
            read(froma, fromb, s + 1, o[(s + 1) & 1]);
            multiply(s);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vm<0>();  // the next chunk (and what was stored before this one)
        lds_barrier(); // every wave's part of it is here, and this one's last reads done
    };
    // the groups' sums into the first one's, in the groups' order; no copy is under
    // way and every operand read
    auto join = [&] {
        static_assert(KG == 1 || (WM == 1 && WN == 1 && WAVES * 8 * 256 <= PLACE), "sums in LDS");
        float *f0 = reinterpret_cast<float *>(both0), *f1 = reinterpret_cast<float *>(both1);
        const int at = wave * 512 + lane;
        if (kg > 0)
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                f0[kg * (PLACE / 4) + at + q * 64] = acc[0][0][q];
                f1[kg * (PLACE / 4) + at + q * 64] = acc[0][0][8 + q];
            }
        lds_barrier();
        if (kg == 0)
#pragma unroll
            for (int g = 1; g < KG; ++g)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    acc[0][0][q] += f0[g * (PLACE / 4) + at + q * 64];
                    acc[0][0][8 + q] += f1[g * (PLACE / 4) + at + q * 64];
                }
    };
    auto bnow = b_of(0);
    load_scales(0, 0);
    fetch_a(0, code0);
    fetch_b(bnow, 0, code0 + TM * 128);
    put_scales(0, even);
    wait_vm<0>();
    lds_barrier();
    if constexpr (ONE) {
        chunk(even, false, code0, code0 + TM * 128, [] {}, [] {});
        multiply(3);
        put(n0);
    } else {
#pragma unroll 1
        for (int t = 0; t < run; ++t) { // more than one only if a row's chunks are even in number
            const auto bnext = b_of(t + 1);
#pragma unroll 1
            for (int c = 0; c < own; c += 2) {
                const bool last = c + 2 >= own;
                const int after = last ? 0 : c + 2;
                chunk(
                    even, c > 0, code0, code0 + TM * 128,
                    [&] {
                        if (KG == 1 && !second_chunk(c, own))
                            return;
                        fetch_a(c + 1, code1);
                        fetch_b(bnow, c + 1, code1 + TM * 128);
                    },
                    [&] {
                        put_scales(c + 1, odd);
                        load_scales(last ? t + 1 : t, after);
                    });
                if (KG > 1 || second_chunk(c, own))
                    chunk(
                        odd, true, code1, code1 + TM * 128,
                        [&] {
                            if (!chunk_after(c, own, t, run))
                                return;
                            fetch_a(after, code0);
                            fetch_b(last ? bnext : bnow, after, code0 + TM * 128);
                        },
                        [&] { put_scales(after, even); });
            }
            bnow = bnext;
            multiply(3);
            if constexpr (KG > 1) {
                join();
                if (kg > 0)
                    return;
            }
            put(n0 + t * TN);
            clear();
        }
    }
}

// Tiles of a run: of 1, 2, 4 and 8 the one that ends first when `slots`
// workgroups are under way together, a tile taking its chunks and one more, a
// run about three chunks besides (first copies, last stores).  The callers' slots
// are those of the large and the middle tiles, one and two workgroups a CU; of the
// small ones two or three fit a CU, but they are counted as one.  Tiles of lists
// are of different cost and end at different times: half a run at the end, not
// a whole last round (128 lists of 512 rows, 2048 x 2048: runs of 1, 2, 4 and 8
// 251, 235, 249 and 312 us).
template <bool LIST>
static int run_length(int64_t mt, int64_t nt, int chunks, int64_t slots)
{
    int best = 1;
    int64_t least = INT64_MAX;
    for (int run = 1; run <= 8 && (run == 1 || chunks % 2 == 0); run *= 2) {
        const int64_t runs = mt * ((nt + run - 1) / run);
        const int64_t halves = LIST ? 2 * runs + slots : (runs + slots - 1) / slots * 2 * slots;
        const int64_t cost = halves * ((int64_t)run * (chunks + 1) + 3);
        if (cost < least) {
            least = cost;
            best = run;
        }
    }
    return best;
}

template <typename Kernel, typename... Args>
static hipError_t launch_blocks(Kernel kernel, int64_t blocks, int threads, hipStream_t stream,
                                Mx4Product p, Args... args)
{
    const int64_t most = most_blocks(threads);
    for (int64_t b = 0; b < blocks; b += most) {
        p.block0 = (uint32_t)b;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks - b < most ? blocks - b : most)),
                           dim3(threads), 0, stream, p, args...);
    }
    return hipGetLastError();
}

template <typename T, bool LIST, int WM, int WN, int MW, int NW, int KG = 1, bool ONE = false>
static hipError_t tiles_as(const Mx4Product &p, hipStream_t stream)
{
    constexpr int64_t TM = 32 * WM * MW, TN = 32 * WN * NW;
    const int64_t nt = (p.n + TN - 1) / TN;
    int64_t mt = (p.m + TM - 1) / TM, likely = mt;
    if (LIST) { // half of the lists that may end inside a tile
        mt = most_list_tiles(p.m, p.nlist, TM);
        likely = p.m / TM + (mt - p.m / TM) / 2 + 1;
    }
    const int run = ONE || KG > 1 ? 1
                                  : run_length<LIST>(likely, nt, (p.kb + 7) / 8,
                                                     MW * NW == 8 ? 256 : 512);
    TileOrder order;
    order.mt = (uint32_t)mt;
    order.nruns = (uint32_t)((nt + run - 1) / run);
    order.high = LIST ? (uint32_t)(likely < 32 ? 1 : likely < 64 ? 2 : 4) : 8;
    int64_t blocks = mt * order.nruns;
    if (LIST) // whole groups, the same number for every XCD
        blocks = ((mt + order.high - 1) / order.high + 7) / 8 * 8 * order.high * order.nruns;
    order.blocks = (uint32_t)blocks;
    return launch_blocks(mx4_tile_kernel<T, LIST, WM, WN, MW, NW, KG, ONE>, blocks,
                         64 * MW * NW * KG, stream, p, order, run);
}

template <typename T, bool LIST, int KS>
static hipError_t direct_as(const Mx4Product &p, int64_t mt, hipStream_t stream)
{
    const int64_t nt = (p.n + 16ll * 8 / KS - 1) / (16 * 8 / KS);
    return launch_blocks(mx4_direct_kernel<T, LIST, KS>, nt * mt, 512, stream, p, (uint32_t)nt);
}

template <typename T, bool LIST>
static hipError_t product_of(const Mx4Product &p, hipStream_t stream)
{
    const int64_t mt = LIST ? most_list_tiles(p.m, p.nlist, 16) : (p.m + 15) / 16;
    switch (mx4_kernel_of(LIST, p.m, p.n, p.kb, p.nlist, p.arows, p.order != nullptr)) {
    case kMx4Direct1: return direct_as<T, LIST, 1>(p, mt, stream);
    case kMx4Direct4: return direct_as<T, LIST, 4>(p, mt, stream);
    case kMx4Direct8: return direct_as<T, LIST, 8>(p, mt, stream);
    case kMx4Shared: return tiles_as<T, LIST, 1, 1, 2, 2, 2>(p, stream);
    case kMx4Small: return tiles_as<T, LIST, 1, 1, 2, 4>(p, stream);
    case kMx4Middle: return tiles_as<T, LIST, 2, 2, 2, 2>(p, stream);
    case kMx4Large: return tiles_as<T, LIST, 4, 2, 2, 4>(p, stream);
    case kMx4One:
        if constexpr (!LIST)
            return tiles_as<T, false, 1, 1, 2, 4, 1, true>(p, stream);
    }
    return hipErrorInvalidValue;
}

template <typename T>
static hipError_t product_as(const Mx4Product &p, hipStream_t stream)
{
    return p.offsets ? product_of<T, true>(p, stream) : product_of<T, false>(p, stream);
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

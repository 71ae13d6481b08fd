// Products of rows sorted by list with their list's own matrix, and the gradient of
// the matrices.
#include "list_direct.hpp"
#include "list_tiles.hpp"

namespace ivfpq {

template <typename T, int FORM>
static hipError_t rows_as(const ListJob &p, hipStream_t stream)
{
    if constexpr (sizeof(T) == 2) {
        if (copies_fit<FORM>(p)) {
            switch (copy_tile(p.rows, p.nlist, p.n, p.kdim, true)) {
            case 0: return launch_copies<T, T, FORM, 64, 4, 1, 1, 1, 4>(p, stream);
            case 1: return launch_copies<T, T, FORM, 64, 4, 1, 2, 2, 2>(p, stream);
            case 2: return launch_copies<T, T, FORM, 64, 2, 1, 2, 2, 2>(p, stream);
            case 3: return launch_copies<T, T, FORM, 64, 4, 2, 2, 2, 2>(p, stream);
            case 4: return launch_copies<T, T, FORM, 64, 2, 2, 2, 2, 2>(p, stream);
            default: return launch_copies<T, T, FORM, 64, 2, 4, 2, 2, 4>(p, stream);
            }
        }
    }
    if constexpr (FORM == kRowsAlong) {
        // Few 16 x 32 tiles: their waves share the contraction.  float32, one list of 128
        // rows, 1024 x 1024 (256 tiles): 14 us, in 64 x 64 tiles 21; 8 lists of 2 rows, 2049
        // x 2049 (325): 41 and 57; 64 lists of 4 rows, 1024 x 1024 (1536): 80 and 57.
        // bfloat16, one list of 1025 x 1025, 64 rows (132): 10 and 12; 128 rows (264): 17
        // and 12.
        if (count_tiles<FORM>(p, 16, 32) <= (sizeof(T) == 4 ? 400 : 256) && !any_tiny<FORM>(p))
            return launch_direct<T, kRowsAlong, 1, 1, 4, 2>(p, stream);
    }
    constexpr int KS = sizeof(T) == 4 ? 16 : 32;
    // Larger tiles where lists fill them and there are enough.  float32, 64 lists of
    // 1024 x 1024, 64 rows each: 109 us in 64 x 64 tiles, 117 in 128 x 128; 512: 482 and
    // 381.  8 lists of 1025 x 1025, bfloat16, 512 rows each (324 tiles): 49 and 46; 2048: 139
    // and 117.
    if (p.rows > 64 * p.nlist && count_tiles<FORM>(p, 128, 128) > 512)
        return launch_tiles<T, T, FORM, KS, 2, 2, 2, 2>(p, stream);
    // 64 x 64 tiles, two a CU; in 16 bits 64 x 128 by eight waves where those would take a
    // second turn (of which two fit a CU as well).  Both ways through 16 lists of 1281 x 1281,
    // 128 rows each: 98 us and 81; 8 lists of 1025 x 1025, 64 rows each (204 tiles): 26 and
    // 31.
    if constexpr (sizeof(T) == 2)
        if (count_tiles<FORM>(p, 64, 64) > 512)
            return launch_tiles<T, T, FORM, 2 * KS, 1, 1, 2, 4>(p, stream);
    return launch_tiles<T, T, FORM, 2 * KS, 1, 1, 2, 2>(p, stream);
}

template <typename T>
static hipError_t product_as(const ListJob &p, bool transposed, hipStream_t stream)
{
    return transposed ? rows_as<T, kRowsAcross>(p, stream) : rows_as<T, kRowsAlong>(p, stream);
}

hipError_t launch_list_product(const ListProduct &q, int type, hipStream_t stream)
{
    ListJob p;
    p.a = q.x;
    p.arows = q.arows;
    p.kdim = q.d;
    p.b = q.matrices;
    p.n = q.n;
    p.nlist = q.nlist;
    p.offsets = q.offsets;
    p.order = q.order;
    p.k = FastDiv((uint32_t)q.k);
    p.rows = q.rows;
    p.out = q.out;
    switch (type) {
    case kF32: return product_as<float>(p, q.transposed, stream);
    case kBF16: return product_as<__bf16>(p, q.transposed, stream);
    default: return product_as<_Float16>(p, q.transposed, stream);
    }
}

template <typename T, typename TO>
static hipError_t gradient_as(const ListJob &p, int size, hipStream_t stream)
{
    constexpr int KS = sizeof(T) == 4 ? 16 : 32;
    if constexpr (sizeof(T) == 2) {
        if (copies_fit<kGradient>(p))
            return size == 256 ? launch_copies<T, TO, kGradient, 64, 2, 4, 2, 2, 4>(p, stream)
                               : launch_copies<T, TO, kGradient, 64, 2, 2, 2, 2, 2>(p, stream);
    }
    // 64 x 64 tiles where larger ones leave CUs empty, float32 up to one tile a CU, 16-bit
    // up to two: 256 rows a list, float32, 8 lists of 512 x 512 (128 tiles): 16 us in 64 x
    // 64, 22 in 128 x 128; 16 lists (256): 26 and 24; bfloat16, 16 lists of 513 x 513
    // (400): 22 and 21; 16 of 1025 x 1025 (1296): 51 and 48.
    return count_tiles<kGradient>(p, 128, 128) * p.splits > (sizeof(T) == 4 ? 192 : 512)
               ? launch_tiles<T, TO, kGradient, KS, 2, 2, 2, 2>(p, stream)
               : launch_tiles<T, TO, kGradient, 32, 1, 1, 2, 2>(p, stream);
}

// The parts' sums, in their order, to the output's type; a thread four of them.
template <typename TO>
__global__ __launch_bounds__(256) void list_join_kernel(const float *__restrict__ parts,
                                                        int64_t count, int splits,
                                                        TO *__restrict__ out, int64_t block0)
{
    typedef float F4 __attribute__((ext_vector_type(4), aligned(4)));
    typedef TO V4 __attribute__((ext_vector_type(4), aligned(sizeof(TO))));
    const int64_t at = ((block0 + blockIdx.x) * 256 + threadIdx.x) * 4;
    if (at >= count)
        return;
    if (at + 4 <= count) {
        F4 sum = *reinterpret_cast<const F4 *>(parts + at);
        for (int s = 1; s < splits; ++s)
            sum += *reinterpret_cast<const F4 *>(parts + s * count + at);
        V4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            v[i] = (TO)sum[i];
        *reinterpret_cast<V4 *>(out + at) = v;
    } else {
        for (int64_t i = at; i < count; ++i) {
            float sum = parts[i];
            for (int s = 1; s < splits; ++s)
                sum += parts[s * count + i];
            out[i] = (TO)sum;
        }
    }
}

template <typename TO>
static hipError_t join_parts(const float *parts, int64_t count, int splits, void *out,
                             hipStream_t stream)
{
    const int64_t blocks = (count + 1023) / 1024, most = most_blocks(256);
    for (int64_t b = 0; b < blocks; b += most)
        hipLaunchKernelGGL(list_join_kernel<TO>,
                           dim3((unsigned)(blocks - b < most ? blocks - b : most)), dim3(256), 0,
                           stream, parts, count, splits, static_cast<TO *>(out), b);
    return hipGetLastError();
}

template <typename T>
static hipError_t gradient_to(ListJob p, int size, int out_type, void *ws, hipStream_t stream)
{
    if (p.splits > 1) {
        void *out = p.out;
        p.out = ws;
        if (hipError_t e = gradient_as<T, float>(p, size, stream))
            return e;
        const int64_t count = (int64_t)p.nlist * p.m * p.n;
        return out_type == kF32
                   ? join_parts<float>(static_cast<float *>(ws), count, p.splits, out, stream)
                   : join_parts<T>(static_cast<float *>(ws), count, p.splits, out, stream);
    }
    return out_type == kF32 ? gradient_as<T, float>(p, size, stream)
                            : gradient_as<T, T>(p, size, stream);
}

// The lists in descending order of length, by eighths of a power of two, so that no long
// one is left for the end.
__global__ __launch_bounds__(1024) void list_size_kernel(const int32_t *offsets, int nlist,
                                                         int64_t rows, int32_t *order)
{
    constexpr int CLASSES = 256;
    __shared__ int at[CLASSES];
    auto class_of = [&](int e) {
        const int64_t n = part_begin(offsets, nlist, rows, e + 2) -
                          part_begin(offsets, nlist, rows, e + 1);
        const uint32_t v = n > 0 ? (uint32_t)n : 0u;
        if (v < 8)
            return CLASSES - 1 - (int)v;
        const int top = 31 - __builtin_clz(v);
        return CLASSES - 1 - ((top - 2) * 8 + (int)(v >> (top - 3) & 7));
    };
    for (int c = threadIdx.x; c < CLASSES; c += 1024)
        at[c] = 0;
    __syncthreads();
    for (int e = threadIdx.x; e < nlist; e += 1024)
        atomicAdd(&at[class_of(e)], 1);
    __syncthreads();
    if (threadIdx.x < 64) { // exclusive sums, four classes a lane
        int c[4], sum = 0;
        for (int i = 0; i < 4; ++i) {
            c[i] = at[threadIdx.x * 4 + i];
            sum += c[i];
        }
        int before = (int)wave_inclusive_sum((uint32_t)sum) - sum;
        for (int i = 0; i < 4; ++i) {
            at[threadIdx.x * 4 + i] = before;
            before += c[i];
        }
    }
    __syncthreads();
    // which list of a class comes first depends on the run; no result does
    for (int e = threadIdx.x; e < nlist; e += 1024)
        order[atomicAdd(&at[class_of(e)], 1)] = e;
}

// Whether sorting the lists by length is worth a launch (64 lists, 32,768 rows, 2048 x
// 2048, lengths as 1 / i: 524 us, the lists by length 370).
static bool by_size(int64_t rows, int n, int d, int nlist)
{
    return nlist > 1 && rows * n >= ((int64_t)1 << 33) / d;
}

size_t list_gradient_bytes(int64_t rows, int n, int d, int nlist)
{
    const int splits = gradient_share(rows, nlist, n, d).splits;
    if (splits > 1)
        return (size_t)splits * nlist * n * d * 4;
    return by_size(rows, n, d, nlist) ? (size_t)nlist * 4 : 0;
}

hipError_t launch_list_gradient(const ListGradient &q, int type, int out_type, hipStream_t stream)
{
    ListJob p;
    p.a = q.grad;
    p.m = q.n;
    p.b = q.x;
    p.arows = q.arows;
    p.n = q.d;
    p.nlist = q.nlist;
    p.offsets = q.offsets;
    p.order = q.order;
    p.k = FastDiv((uint32_t)q.k);
    p.rows = q.rows;
    p.out = q.out;
    const GradientShare share = gradient_share(q.rows, q.nlist, q.n, q.d);
    p.splits = share.splits;
    if (p.splits == 1 && by_size(q.rows, q.n, q.d, q.nlist)) {
        int32_t *order = static_cast<int32_t *>(q.ws);
        hipLaunchKernelGGL(list_size_kernel, dim3(1), dim3(1024), 0, stream, q.offsets, q.nlist,
                           q.rows, order);
        p.by_size = order;
    }
    switch (type) {
    case kF32: return gradient_to<float>(p, share.size, out_type, q.ws, stream);
    case kBF16: return gradient_to<__bf16>(p, share.size, out_type, q.ws, stream);
    default: return gradient_to<_Float16>(p, share.size, out_type, q.ws, stream);
    }
}

} // namespace ivfpq

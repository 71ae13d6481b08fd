// Products of rows sorted by list with their list's own matrix, and the gradient of
// the matrices.
#include "list_direct.hpp"
#include "list_tiles.hpp"

namespace ivfpq {

static bool small_tiles(const ListJob &p)
{
    const int64_t mt = (p.rows + 127) / 128 + (p.rows < p.nlist ? p.rows : p.nlist) / 2;
    return mt * ((p.n + 127) / 128) <= 512;
}

template <typename T, int FORM>
static hipError_t rows_as(const ListJob &p, hipStream_t stream)
{
    if constexpr (FORM == kRowsAlong) {
        if (p.rows <= 4 * p.nlist && !any_tiny<FORM>(p))
            return launch_direct<T, kRowsAlong, 1, 1, 4, 2>(p, stream);
    }
    if constexpr (std::is_same<T, float>::value)
        return small_tiles(p) ? launch_tiles<T, T, FORM, 32, 1, 1, 2, 2>(p, stream)
                              : launch_tiles<T, T, FORM, 16, 2, 2, 2, 2>(p, stream);
    else if (copies_fit<FORM>(p))
        return launch_copies<T, T, FORM, 64, 2, 4, 2, 2, 4>(p, stream);
    else
        return small_tiles(p) ? launch_tiles<T, T, FORM, 64, 1, 1, 2, 2>(p, stream)
                              : launch_tiles<T, T, FORM, 32, 2, 2, 2, 2>(p, stream);
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
static hipError_t gradient_as(const ListJob &p, hipStream_t stream)
{
    if constexpr (sizeof(T) == 2)
        if (copies_fit<kGradient>(p))
            return launch_copies<T, TO, kGradient, 64, 2, 4, 2, 2, 4>(p, stream);
    constexpr int KS = std::is_same<T, float>::value ? 16 : 32;
    if ((int64_t)p.nlist * ((p.n + 127) / 128) * ((p.m + 127) / 128) <= 512)
        return launch_tiles<T, TO, kGradient, 32, 1, 1, 2, 2>(p, stream);
    return launch_tiles<T, TO, kGradient, KS, 2, 2, 2, 2>(p, stream);
}

template <typename T>
static hipError_t gradient_to(const ListJob &p, int out_type, hipStream_t stream)
{
    return out_type == kF32 ? gradient_as<T, float>(p, stream) : gradient_as<T, T>(p, stream);
}

size_t list_gradient_bytes(int64_t, int, int, int) { return 0; }

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
    switch (type) {
    case kF32: return gradient_as<float, float>(p, stream);
    case kBF16: return gradient_to<__bf16>(p, out_type, stream);
    default: return gradient_to<_Float16>(p, out_type, stream);
    }
}

} // namespace ivfpq

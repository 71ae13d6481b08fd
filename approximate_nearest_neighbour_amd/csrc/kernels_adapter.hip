// Rows times one shared matrix, plus each row's own low-rank product.
//
// y[t] = W x[t] + s[a] U[a] (D[a] x[t]), a the list (adapter) of row t, in two
// launches: the hidden rows h[t] = s[a] D[a] x[t], a product per list of the sorted
// rows, then the shared product with the contraction continued over the hidden rows:
// after the chunks of x and W come, for each list among a tile's rows, chunks of
// that list's hidden rows (the other rows zero) and its up matrix.  So the adapters
// add to sums that are still in registers.
//
// Hidden rows of 16-bit types are kept as two parts, h = high + low, side by side,
// and multiplied with the same up matrix twice: rounded once more to 16 bits they
// would add an error as large as the result's own rounding.  float32 hidden
// rows are float32.
#include "list_direct.hpp"
#include "list_tiles.hpp"

namespace ivfpq {

static int hidden_part(int r) { return (r + 7) / 8 * 8; }

// Hidden rows are short and their contraction long, so they take the kernel of few rows,
// of as many columns at once as they have.
template <typename T>
static hipError_t hidden_as(const ListJob &p, hipStream_t stream)
{
    if (any_tiny<kHidden>(p))
        return launch_tiles<T, float, kHidden, 32, 2, 1, 2, 2, true>(p, stream);
    const bool few = p.rows <= 16 * p.nlist;
    if constexpr (sizeof(T) == 4) {
        return few ? launch_direct<T, kHidden, 1, 1, 8, 2>(p, stream)
                   : launch_direct<T, kHidden, 2, 2, 8, 1>(p, stream);
    } else {
        if (few)
            return p.r <= 16 ? launch_direct<T, kHidden, 1, 1, 8, 2>(p, stream)
                             : launch_direct<T, kHidden, 1, 4, 8, 1>(p, stream);
        return p.r <= 16 ? launch_direct<T, kHidden, 4, 1, 8, 1>(p, stream)
                         : launch_direct<T, kHidden, 2, 4, 8, 1>(p, stream);
    }
}

template <typename T>
static hipError_t adapter_as(const AdapterProduct &q, hipStream_t stream)
{
    constexpr int KS = std::is_same<T, float>::value ? 16 : 32;
    ListJob p;
    p.a = q.x;
    p.rows = p.arows = q.t;
    p.kdim = q.d;
    p.nlist = q.nlist;
    p.offsets = q.offsets;
    p.order = q.order;
    p.pos = q.pos;
    p.scales = q.scales;
    p.up = q.up;
    p.r = q.r;
    p.rp = hidden_part(q.r);
    p.width = sizeof(T) == 4 ? p.rp : 2 * p.rp;
    p.hidden = q.ws;
    p.row_list = reinterpret_cast<int32_t *>(static_cast<T *>(q.ws) + q.t * p.width);
    p.b = q.down;
    p.n = q.r;
    if (hipError_t e = hidden_as<T>(p, stream))
        return e;
    p.b = q.w;
    p.n = q.n;
    p.out = q.out;
    // Few rows, or rows that the copies cannot read and too few tiles for all CUs.
    const bool copies = sizeof(T) == 2 && copies_fit<kAdapter>(p);
    const int64_t middle = count_tiles<kAdapter>(p, 128, 128);
    if (!any_tiny<kAdapter>(p) && (p.rows <= 128 || (!copies && middle <= 64))) {
        if (p.rows <= 16)
            return launch_direct<T, kAdapter, 1, 1, 8, 2>(p, stream);
        if (p.rows <= 32)
            return launch_direct<T, kAdapter, 2, 1, 8, 2>(p, stream);
        return launch_direct<T, kAdapter, 2, 2, 8, 1>(p, stream);
    }
    if constexpr (sizeof(T) == 2) {
        if (copies) {
            if (middle <= 64)
                return launch_copies<T, T, kAdapter, 64, 4, 1, 1, 1, 4>(p, stream);
            if (middle <= 128)
                return launch_copies<T, T, kAdapter, 64, 4, 1, 2, 2, 2>(p, stream);
            if (middle <= 256)
                return launch_copies<T, T, kAdapter, 64, 2, 1, 2, 2, 2>(p, stream);
            if (3 * ((count_tiles<kAdapter>(p, 256, 256) + 255) / 256) <= (middle + 255) / 256)
                return launch_copies<T, T, kAdapter, 64, 2, 4, 2, 2, 4>(p, stream);
            return launch_copies<T, T, kAdapter, 64, 2, 2, 2, 2, 2>(p, stream);
        }
    }
    return middle <= 512 ? launch_tiles<T, T, kAdapter, 2 * KS, 1, 1, 2, 2>(p, stream)
                         : launch_tiles<T, T, kAdapter, KS, 2, 2, 2, 2>(p, stream);
}

size_t adapter_bytes(int64_t t, int r)
{
    // hidden rows, 32 bits a value in either form, and the rows' lists
    return (size_t)t * ((size_t)hidden_part(r) * 4 + 4);
}

hipError_t launch_adapter(const AdapterProduct &p, int type, hipStream_t stream)
{
    switch (type) {
    case kF32: return adapter_as<float>(p, stream);
    case kBF16: return adapter_as<__bf16>(p, stream);
    default: return adapter_as<_Float16>(p, stream);
    }
}

} // namespace ivfpq

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

// Hidden rows are short and their contraction long, so they take the kernel of few rows: in
// 16 x 16 blocks, whose eight waves share the contraction, up to a workgroup a CU; from
// there on in 32 x 32, which read the operands half as often; from four such blocks a
// CU on, if the copies fit, in copied tiles of 64 x 64.  bfloat16, d = 4096, the whole
// call with 1024 columns, rank 64: 1024 rows of one list (256 blocks) 34 us, 43 and 40;
// 2048 of 16 lists (544) 64, 50 and 55; 8192 of 16 lists (2080) 161, 123 and 97.
template <typename T>
static hipError_t hidden_as(const ListJob &p, hipStream_t stream)
{
    if (any_tiny<kHidden>(p))
        return launch_tiles<T, float, kHidden, 32, 2, 1, 2, 2, true>(p, stream);
    const int64_t blocks = count_tiles<kHidden>(p, 16, 16);
    if (blocks <= 256)
        return launch_direct<T, kHidden, 1, 1, 8, 2>(p, stream);
    if constexpr (sizeof(T) == 2)
        if (blocks > 1024 && copies_fit<kHidden>(p))
            return launch_copies<T, float, kHidden, 64, 4, 1, 1, 2, 2>(p, stream);
    return launch_direct<T, kHidden, 2, 2, 8, 1>(p, stream);
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
    const bool copies = sizeof(T) == 2 && copies_fit<kAdapter>(p);
    const int64_t middle = count_tiles<kAdapter>(p, 128, 128);
    // Few rows: blocks whose waves share the contraction, the largest that still make a
    // workgroup a CU.  16 rows of 4096 x 4096: 26 us in 16 x 16 blocks, 29 in 32 x 32, 44 in
    // copied 32 x 128 tiles; 64 rows: 53, 33 and 44; 128: 90, 53 and 43; 32 rows of 11,008 x
    // 4096: 73, 57 and 86.  Where the copies do not fit, up to two workgroups a CU: 256
    // rows of 2048 x 2048 in float32 58 us, in 64 x 64 tiles 71; 512 rows: 99 and 74.
    const int64_t blocks = count_tiles<kAdapter>(p, 32, 32);
    if (!any_tiny<kAdapter>(p) && (p.rows <= 32 || blocks <= (copies ? 256 : 512))) {
        if (p.rows <= 16 || count_tiles<kAdapter>(p, 16, 16) <= 256)
            return launch_direct<T, kAdapter, 1, 1, 8, 2>(p, stream);
        if (count_tiles<kAdapter>(p, 32, 16) <= 256)
            return launch_direct<T, kAdapter, 2, 1, 8, 2>(p, stream);
        return launch_direct<T, kAdapter, 2, 2, 8, 1>(p, stream);
    }
    if constexpr (sizeof(T) == 2) {
        if (copies) {
            switch (copy_tile(p.rows, p.nlist, p.n, p.kdim, false)) {
            case 0: return launch_copies<T, T, kAdapter, 64, 4, 1, 1, 1, 4>(p, stream);
            case 1: return launch_copies<T, T, kAdapter, 64, 4, 1, 2, 2, 2>(p, stream);
            case 2: return launch_copies<T, T, kAdapter, 64, 2, 1, 2, 2, 2>(p, stream);
            case 3: return launch_copies<T, T, kAdapter, 64, 4, 2, 2, 2, 2>(p, stream);
            case 4: return launch_copies<T, T, kAdapter, 64, 2, 2, 2, 2, 2>(p, stream);
            default: return launch_copies<T, T, kAdapter, 64, 2, 4, 2, 2, 4>(p, stream);
            }
        }
    }
    // In float32 tiles of 64 x 64 or 128 x 128: 2048 x 2048, 1024 rows (128 of the larger)
    // 92 us and 131, 2048 rows (256) 152 and 139.  In 16 bits of 64 x 64, or of 64 x 128 by
    // eight waves where those would take more than a turn of two a CU: 2001 x 2001, 2048 rows
    // 93 us and 82, 4096 167 and 146 (128 x 128 tiles: 190).
    if constexpr (sizeof(T) == 4) {
        if (middle > 192)
            return launch_tiles<T, T, kAdapter, KS, 2, 2, 2, 2>(p, stream);
    } else {
        if (count_tiles<kAdapter>(p, 64, 64) > 512)
            return launch_tiles<T, T, kAdapter, 2 * KS, 1, 1, 2, 4>(p, stream);
    }
    return launch_tiles<T, T, kAdapter, 2 * KS, 1, 1, 2, 2>(p, stream);
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

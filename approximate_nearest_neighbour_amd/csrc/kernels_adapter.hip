// Rows times one shared matrix, plus each row's own low-rank product.
//
// y[t] = W x[t] + s[a] U[a] (D[a] x[t]), a the list (adapter) of row t, in two
// launches: the hidden rows h[t] = s[a] D[a] x[t], a product per list of the sorted
// rows, then the shared product, whose tiles begin (those of few rows end) with the
// adapters' products, so that both add to sums in registers.
//
// Hidden rows are float32: those of 16-bit types in three bfloat16 parts, which hold all 24
// bits of a float32 value of 2^-110 or more, each multiplied with the same up matrix.  Two
// parts lose 8 bits, which show where W x and the adapter cancel; binary16 parts lose
// what leaves binary16's range, below 2^-14 bit by bit and above 65504 all.  Binary16 up
// matrices are split in two bfloat16 parts on their way into the matrix instructions.
// 8192 rows through 4096 x 4096, rank 64: 275 us in bfloat16, 294 in binary16 (with two
// parts of the rows' type 273 and 284).
#include "list_direct.hpp"
#include "list_tiles.hpp"

namespace ivfpq {

// Values of a hidden row, and of all hidden rows: whole steps and blocks (HiddenPlace).
static int hidden_width(int r) { return (r + 15) / 16 * 16; }
static size_t hidden_values(int64_t t, int r)
{
    return (size_t)((t + 31) / 32 * 32) * (size_t)hidden_width(r);
}

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
    p.rp = hidden_width(q.r);
    p.hidden = q.ws;
    p.row_list = reinterpret_cast<int32_t *>(
        static_cast<typename HiddenPlace<T>::E *>(q.ws) +
        hidden_values(q.t, q.r) * HiddenPlace<T>::PARTS);
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
    // workgroup a CU.  16 rows of 4096 x 4096: 24 us in 16 x 16 blocks, 29 in 32 x 32, 35 in
    // copied 32 x 128 tiles; 64 rows: 53, 34 and 37; 128: 87, 51 and 35; 32 rows of 11,008 x
    // 4096: 72, 56 and 69.  Where the copies do not fit: 128 rows of 2048 x 2048 in float32
    // (256 blocks of 32 x 32) 39 us, in 64 x 64 tiles 53; 192 rows 57 and 53; binary16, rank
    // 7, 256 rows of 1001 x 777 (256 blocks) 21.8 and 21.3, 301 rows 29.4 and 21.4.
    const int64_t blocks = count_tiles<kAdapter>(p, 32, 32);
    if (!any_tiny<kAdapter>(p) && (p.rows <= 32 || blocks <= 256)) {
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
    // 77 us and 98, 2048 rows (256) 131 and 114.  In 16 bits of 64 x 64, or of 64 x 128 by
    // eight waves where those would take more than a turn of two a CU: 2001 x 2001, 512 rows
    // (256 of the smaller) 30 us and 35, 2048 rows 65 and 55, 4096 116 and 96.
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
    // hidden rows, 32 bits a value or three times 16, and the rows' lists
    return hidden_values(t, r) * 6 + (size_t)t * 4;
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

// Products of few rows: bound by the matrices' bytes, which go from memory straight to
// registers.
//
// A wave forms 16 RT rows by 16 CT columns with 16 x 16 x 32 matrix instructions; KW of a
// workgroup's eight waves share the contraction of the same columns out between them
// and join their sums through LDS, in the waves' order.  The contraction comes in
// units of 64 values, of which lane group g (16 lanes) has values 16 g to 16 g + 15 of
// its row: whole lines of memory for 16-bit rows.  Two turns of TURN units are under
// way, one of them while the other is multiplied.  Rows may begin at any address.
//
// 32 rows of 4096 x 4096 with their adapters: 20 us for the shared product (34 MB, which
// partly stay in the caches), 10 for the hidden rows of rank 16: there a chain of search,
// row numbers, loads and join.
//
// An adapter's hidden rows are multiplied with the up matrices after the shared ones:
// the lists of the tile's rows are dealt to the KW waves.  A lane's results are of one
// row, and keep what they were where the list is not the row's.
#pragma once

#include "list_tiles.hpp"

namespace ivfpq {

template <typename E>
__device__ __forceinline__ f32x4 mfma16_small(s16x8 a, s16x8 b, f32x4 c)
{
    typedef E V __attribute__((ext_vector_type(8)));
    if constexpr (std::is_same<E, __bf16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, a),
                                                       __builtin_bit_cast(V, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, a),
                                                      __builtin_bit_cast(V, b), c, 0, 0, 0);
}

// The list of each row of a tile (-1: none), and these lists each once, ascending:
// segs[0 .. segs[TM]).
template <int TM, int THREADS>
__device__ __forceinline__ void find_lists(const ListJob &p, const PartTile &tile, int *tile_list,
                                           int *segs)
{
    const int tid = (int)threadIdx.x, lane = lane_id();
    for (int i = tid; i < TM; i += THREADS) {
        const int64_t row = tile.p0 + i;
        int e = -1;
        if (row < tile.p1 && (uint32_t)p.pos[row] < (uint64_t)p.rows) {
            e = p.row_list[row];
            e = (uint32_t)e < (uint32_t)p.nlist ? e : -1;
        }
        tile_list[i] = e;
    }
    lds_barrier();
    if (tid < 64) {
        int last = -1, found = 0;
        for (;;) { // at most TM times
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
    lds_barrier();
}

template <typename T, bool ODD, int FORM, int RT, int CT, int KW, int TURN>
__global__ __launch_bounds__(512) void list_direct_kernel(ListJob p)
{
    static_assert(FormOf<FORM>::B_ALONG, "rows along the contraction");
    using E = typename Parts<T>::E;
    constexpr int NP = Parts<T>::N, TM = 16 * RT, GROUPS = 8 / KW, UNIT = 64;
    __shared__ f32x4 part[KW > 1 ? 8 : 1][RT * CT][64];
    __shared__ int segs[FORM == kAdapter ? TM + 1 : 1];
    __shared__ int tile_list[FORM == kAdapter ? TM : 1];

    const int lane = lane_id(), r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t block = p.block0 + blockIdx.x;
    const int64_t mt = block / p.nt;
    const int cols = FORM == kHidden ? p.r : p.n;
    const int n0 = ((int)(block - mt * p.nt) * GROUPS + wave / KW) * 16 * CT;
    PartTile tile{0, mt * TM, min(mt * TM + TM, p.rows)};
    if constexpr (FORM != kAdapter)
        tile = find_part(p.offsets, p.nlist, p.rows, mt, TM, p.by_row);
    if (tile.p0 >= tile.p1)
        return;
    tile.p0 = uniform(tile.p0);
    tile.p1 = uniform(tile.p1);
    const bool listed = FORM == kAdapter || (tile.e >= 0 && tile.e < p.nlist);
    if (FORM == kHidden && !listed) {
        no_list_rows(p, tile, n0 == 0, (int)threadIdx.x, 512);
        return;
    }

    f32x4 acc[RT][CT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
            acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    int64_t arow[RT]; // rows past the tile's end repeat its last one; they are not stored
    bool there[RT];
    if (listed) {
        const T *a = static_cast<const T *>(p.a), *b = static_cast<const T *>(p.b);
#pragma unroll
        for (int i = 0; i < RT; ++i) {
            const int64_t row = min(tile.p0 + i * 16 + r, tile.p1 - 1);
            const int64_t from = FORM == kAdapter ? row : source_row(p, row);
            there[i] = from >= 0;
            arow[i] = max(from, (int64_t)0) * p.kdim;
        }
        const int64_t list = FORM == kAdapter ? 0 : tile.e;
        int64_t brow[CT]; // columns past the last repeat it; they are not stored
#pragma unroll
        for (int j = 0; j < CT; ++j)
            brow[j] = (list * cols + min(n0 + j * 16 + r, cols - 1)) * p.kdim;
        using Values = Eight<T, ODD>;
        struct Turn {
            Values a[TURN][2][RT], b[TURN][2][CT];
        };
        const int units = (p.kdim + UNIT - 1) / UNIT, whole = p.kdim / UNIT;
        auto load = [&](Turn &t, int u0) { // units u0 and u0 + KW, whole ones
#pragma unroll
            for (int u = 0; u < TURN; ++u) {
                const int64_t at = (int64_t)min(u0 + u * KW, whole - 1) * UNIT + g * 16;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < CT; ++j)
                        t.b[u][h][j].read(b + brow[j] + at + h * 8);
#pragma unroll
                    for (int i = 0; i < RT; ++i)
                        t.a[u][h][i].read(a + arow[i] + at + h * 8);
                }
            }
        };
        auto product = [&](const s16x8 (&oa)[NP], const s16x8 (&ob)[NP], f32x4 &c) {
#pragma unroll
            for (int sum = NP - 1; sum >= 0; --sum)
#pragma unroll
                for (int q = 0; q <= sum; ++q)
                    c = mfma16_small<E>(ob[sum - q], oa[q], c);
        };
        auto products = [&](const Values (&xa)[RT], const Values (&xb)[CT]) {
            s16x8 ob[CT][NP];
#pragma unroll
            for (int j = 0; j < CT; ++j)
                operands_of(xb[j], ob[j]);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                s16x8 oa[NP];
                operands_of(xa[i], oa);
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    product(oa, ob[j], acc[i][j]);
            }
        };
        auto all_ready = [](auto &x) {
#pragma unroll
            for (auto &v : x)
                v.ready();
        };
        auto multiply = [&](Turn &t, int u0) {
#pragma unroll
            for (int u = 0; u < TURN; ++u) {
                if (u0 + u * KW >= whole)
                    break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    all_ready(t.a[u][h]);
                    all_ready(t.b[u][h]);
                    products(t.a[u][h], t.b[u][h]);
                }
            }
        };
        const int first = wave % KW, step = TURN * KW;
        Turn x, y;
        if (whole > 0)
            load(x, first);
        if constexpr (FORM == kAdapter) // while the first operands are under way
            find_lists<TM, 512>(p, tile, tile_list, segs);
        if (whole > 0) {
            for (int u = first; u < whole; u += 2 * step) {
                load(y, u + step);
                __builtin_amdgcn_sched_barrier(0);
                multiply(x, u);
                load(x, u + 2 * step);
                __builtin_amdgcn_sched_barrier(0);
                multiply(y, u + step);
            }
        }
        if (units > whole && whole % KW == first) { // the rows' end
            const int64_t all_a = p.arows * p.kdim;
            const int64_t all_b = (FORM == kAdapter ? 1 : (int64_t)p.nlist) * cols * p.kdim;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = whole * UNIT + g * 16 + h * 8;
                Values xb[CT], xa[RT];
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    xb[j].template read_near<false>(b, brow[j] + at, all_b);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    xa[i].template read_near<false>(a, arow[i] + at, all_a);
                all_ready(xa);
                all_ready(xb);
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    xb[j].template settle<false>(brow[j] + at, all_b, p.kdim - at);
#pragma unroll
                for (int i = 0; i < RT; ++i)
                    xa[i].template settle<false>(arow[i] + at, all_a, p.kdim - at);
                products(xa, xb);
            }
        }
        if constexpr (FORM == kAdapter) {
            using Place = HiddenPlace<T>;
            const typename Place::E *hidden = static_cast<const typename Place::E *>(p.hidden);
            const T *up = static_cast<const T *>(p.up);
            const int64_t all_up = (int64_t)p.nlist * p.n * p.r;
            const int count = segs[TM];
            constexpr int AHEAD = RT + CT <= 3 ? 4 : 2; // lists under way
            for (int at0 = 0; at0 < p.rp; at0 += 32) {  // 32 values a matrix instruction
                const int at = at0 + g * 8;
                Eight<typename Place::E> h[RT][Place::PARTS];
#pragma unroll
                for (int i = 0; i < RT; ++i)
#pragma unroll
                    for (int q = 0; q < Place::PARTS; ++q)
                        h[i][q].read(hidden + q * 512 +
                                     Place::piece(tile.p0 + i * 16 + r, min(at, p.rp - 8), p.rp));
                for (int s0 = first; s0 < count; s0 += AHEAD * KW) {
                    Values xb[AHEAD][CT];
                    auto up_at = [&](int seg, int j) {
                        return ((int64_t)seg * p.n + min(n0 + j * 16 + r, p.n - 1)) * p.r + at;
                    };
#pragma unroll
                    for (int s = 0; s < AHEAD; ++s) {
                        const int seg = segs[min(s0 + s * KW, count - 1)];
#pragma unroll
                        for (int j = 0; j < CT; ++j)
                            xb[s][j].template read_near<false>(up, up_at(seg, j), all_up);
                    }
                    s16x8 oh[RT][kHiddenParts];
#pragma unroll
                    for (int i = 0; i < RT; ++i) {
#pragma unroll
                        for (int q = 0; q < Place::PARTS; ++q)
                            h[i][q].keep(at < p.rp);
                        if constexpr (Place::PARTS == 1)
                            operands_of(h[i][0], oh[i]);
                        else
#pragma unroll
                            for (int q = 0; q < kHiddenParts; ++q)
                                oh[i][q] = __builtin_bit_cast(s16x8, h[i][q].v);
                    }
#pragma unroll
                    for (int s = 0; s < AHEAD; ++s) {
                        if (s0 + s * KW >= count)
                            break;
                        const int seg = segs[s0 + s * KW];
                        all_ready(xb[s]);
#pragma unroll
                        for (int j = 0; j < CT; ++j) {
                            xb[s][j].template settle<false>(up_at(seg, j), all_up,
                                                            at < p.rp ? p.r - at : 0);
                            s16x8 ou[UpParts<T>::N];
                            UpParts<T>::of(xb[s][j], ou);
#pragma unroll
                            for (int i = 0; i < RT; ++i) {
                                f32x4 d = acc[i][j];
                                // parts whose numbers add to 2, then 1, then 0
#pragma unroll
                                for (int sum = kHiddenParts - 1; sum >= 0; --sum)
#pragma unroll
                                    for (int q = 0; q <= sum; ++q)
                                        if (sum - q < UpParts<T>::N)
                                            d = mfma16_small<__bf16>(ou[sum - q], oh[i][q], d);
                                const bool mine = tile_list[i * 16 + r] == seg;
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    acc[i][j][q] = mine ? d[q] : acc[i][j][q];
                            }
                        }
                    }
                }
            }
        }
    }
    if constexpr (KW > 1) {
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
                part[wave][i * CT + j][lane] = acc[i][j];
        __syncthreads();
        if (wave % KW != 0)
            return;
#pragma unroll
        for (int w = 1; w < KW; ++w)
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int j = 0; j < CT; ++j)
                    acc[i][j] += part[wave + w][i * CT + j][lane];
    }
    // result q of a lane: column 4 g + q, row r
#pragma unroll
    for (int i = 0; i < RT; ++i) {
        const int64_t row = tile.p0 + i * 16 + r;
        if (row >= tile.p1)
            continue;
        int64_t t = -1;
        float scale = 1.f;
        if constexpr (FORM == kHidden) {
            t = source_row(p, row);
            if (t < 0)
                continue;
            if (n0 == 0 && g == 0)
                p.row_list[t] = tile.e;
            scale = p.scales ? p.scales[tile.e] : 1.f;
        }
#pragma unroll
        for (int j = 0; j < CT; ++j) {
            const int n = n0 + j * 16 + 4 * g;
            f32x4 v = acc[i][j];
            if (listed && !there[i])
                v = f32x4{0.f, 0.f, 0.f, 0.f};
            if constexpr (FORM == kHidden) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (n + q < p.rp)
                        HiddenPlace<T>::put(p.hidden, t, n + q, p.rp,
                                            n + q < p.r ? v[q] * scale : 0.f);
            } else {
                typedef T V __attribute__((ext_vector_type(4), aligned(sizeof(T))));
                T *out = static_cast<T *>(p.out) + row * p.n + n;
                if (n + 4 <= p.n) {
                    V w;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        w[q] = (T)v[q];
                    *reinterpret_cast<V *>(out) = w;
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (n + q < p.n)
                            out[q] = (T)v[q];
                }
            }
        }
    }
}

template <typename T, int FORM, int RT, int CT, int KW, int TURN>
hipError_t launch_direct(ListJob p, hipStream_t stream)
{
    constexpr int TM = 16 * RT, TN = 16 * CT * 8 / KW;
    const int cols = FORM == kHidden ? p.rp : p.n;
    p.nt = (uint32_t)((cols + TN - 1) / TN);
    int64_t mt;
    if (FORM == kAdapter) {
        mt = (p.rows + TM - 1) / TM;
    } else {
        p.by_row = slots_by_row(p.rows, p.nlist, TM);
        mt = tile_slots(p.rows, p.nlist, TM);
    }
    const int64_t blocks = mt * p.nt, most = most_blocks(512);
    auto odd = [&](const void *q, int64_t width) {
        return sizeof(T) == 2 && ((reinterpret_cast<uintptr_t>(q) & 2) || width % 2);
    };
    auto kernel = list_direct_kernel<T, false, FORM, RT, CT, KW, TURN>;
    if constexpr (sizeof(T) == 2)
        if (odd(p.a, p.kdim) || odd(p.b, p.kdim) || (FORM == kAdapter && odd(p.up, p.r)))
            kernel = list_direct_kernel<T, true, FORM, RT, CT, KW, TURN>;
    for (int64_t b = 0; b < blocks; b += most) {
        p.block0 = b;
        hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks - b < most ? blocks - b : most)),
                           dim3(512), 0, stream, p);
    }
    return hipGetLastError();
}

} // namespace ivfpq

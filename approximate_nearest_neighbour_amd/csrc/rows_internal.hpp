// Launchers of the row operators, as their entry points call them.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ivfpq {

// Microscaled 4-bit rows: [rows][16 kb] codes and [rows][kb] exponent bytes,
// kb = ceil(d / 32); type is an ivfpq_type.
hipError_t launch_mx4_quantize(const void *x, int type, int64_t rows, int d, int64_t stride,
                               uint8_t *codes, uint8_t *scales, hipStream_t stream);
hipError_t launch_mx4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int d,
                                 int type, void *out, hipStream_t stream);

// out [m][n] = A B^T; with offsets, output row p of list e is A's row
// order[p] / k (or p) times B's matrix e.
struct Mx4Product {
    const uint8_t *a = nullptr, *as = nullptr; // [arows][16 kb], [arows][kb]
    const uint8_t *b = nullptr, *bs = nullptr; // [nlist or 1][n][16 kb], [..][n][kb]
    int64_t m = 0, arows = 0;
    int n = 0, kb = 0;
    void *out = nullptr;
    const int32_t *offsets = nullptr; // [nlist + 1]
    const int32_t *order = nullptr;   // [m] or nullptr
    int nlist = 0, k = 1;
    uint32_t block0 = 0; // number of the launch's first workgroup
};
hipError_t launch_mx4_product(const Mx4Product &p, int type, hipStream_t stream);

// Slots sorted by list, and rows there and back; n = nvec k slots.
constexpr int kMaxRouteLists = (1 << 22) - 1;
size_t route_sort_bytes(int64_t n, int nlist);
hipError_t launch_route_sort(const int32_t *lists, int64_t n, int nlist, void *ws, int32_t *offsets,
                             int32_t *order, int32_t *pos, hipStream_t stream);
hipError_t launch_route_gather(const void *x, int type, int64_t nvec, int d, const int32_t *order,
                               const float *weights, int k, void *rows, hipStream_t stream);
hipError_t launch_route_combine(const void *rows, int type, int64_t nvec, int d, const int32_t *pos,
                                const float *weights, int k, void *out, hipStream_t stream);
hipError_t launch_route_combine_grad(const void *grad, const void *rows, int type, int64_t nvec,
                                     int d, const int32_t *order, const int32_t *pos,
                                     const float *weights, int k, void *d_rows, float *d_weights,
                                     hipStream_t stream);


// Products per list of rows in 16 or 32 bits: out [rows][n], output row p of list e is
// x's row order[p] / k (or p) times matrix e, [n][d] (transposed: [d][n]).
struct ListProduct {
    const void *x = nullptr, *matrices = nullptr;
    void *out = nullptr;
    int64_t arows = 0, rows = 0;
    int d = 0, n = 0, nlist = 0, k = 1;
    bool transposed = false;
    const int32_t *offsets = nullptr, *order = nullptr;
};
hipError_t launch_list_product(const ListProduct &p, int type, hipStream_t stream);

// out [nlist][n][d]: per list, the sum over its rows p of grad[p] (outer) x[order[p] / k].
struct ListGradient {
    const void *grad = nullptr, *x = nullptr;
    void *out = nullptr, *ws = nullptr;
    int64_t arows = 0, rows = 0;
    int d = 0, n = 0, nlist = 0, k = 1;
    const int32_t *offsets = nullptr, *order = nullptr;
};
size_t list_gradient_bytes(int64_t rows, int n, int d, int nlist);
hipError_t launch_list_gradient(const ListGradient &p, int type, int out_type, hipStream_t stream);

// out [t][n] = x w^T, plus for a row of list a scales[a] up[a] (down[a] x).
struct AdapterProduct {
    const void *x = nullptr, *w = nullptr, *down = nullptr, *up = nullptr;
    const float *scales = nullptr;
    void *out = nullptr, *ws = nullptr;
    int64_t t = 0;
    int d = 0, n = 0, nlist = 0, r = 0;
    const int32_t *offsets = nullptr, *order = nullptr, *pos = nullptr;
};
size_t adapter_bytes(int64_t t, int r);
hipError_t launch_adapter(const AdapterProduct &p, int type, hipStream_t stream);

// out [n][d] = scale times row ids[i] of table [rows][d].
hipError_t launch_table_lookup(const void *table, int type, int64_t rows, int d, const int32_t *ids,
                               int64_t n, float scale, void *out, hipStream_t stream);

// out [nlist][d]: scale times the sum of the rows order[p] / k of grad over a list's p.
size_t table_grad_bytes(int64_t n, int d);
hipError_t launch_table_grad(const void *grad, int type, int64_t nvec, int d,
                             const int32_t *offsets, const int32_t *order, int k, int nlist,
                             float scale, int out_type, void *out, void *ws, hipStream_t stream);

} // namespace ivfpq

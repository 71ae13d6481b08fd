// Entry points of the products per list, the adapters and the table rows: argument
// checks on the host, then the kernels on the caller's stream.  Declarations and
// conventions: include/ivfpq.h.
#include "rows_check.hpp"
#include "rows_internal.hpp"

using namespace ivfpq;

namespace {

constexpr int64_t kMaxRows = 0x7FFFFFFF;
constexpr int kMaxLists = 1 << 16; // of products per list
constexpr int kMaxRank = 1 << 12;

bool rows_ok(int64_t n) { return n >= 0 && n <= kMaxRows; }
bool width_ok(int d) { return d >= 1 && d <= kMaxRowDim; }

ivfpq_status null_pointer()
{
    return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
}

// Shapes of a product per list or its gradient.
ivfpq_status check_lists(int type, int64_t arows, int d, int nlist, int n, const void *order, int k,
                         int64_t rows)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (!rows_ok(arows) || !rows_ok(rows) || !width_ok(d) || !width_ok(n))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be in [0, 2^31), d and n in [1, 2^20]");
    if (nlist < 1 || nlist > kMaxLists || k < 1)
        return fail(IVFPQ_E_INVALID_ARG, "nlist must be in [1, 2^16] and k at least 1");
    if (rows > 0 && (order ? arows < 1 : arows < rows))
        return fail(IVFPQ_E_INVALID_ARG, "the gathered operand has too few rows");
    return IVFPQ_OK;
}

} // namespace

extern "C" {

ivfpq_status ivfpq_list_product_ex(const void *rows_dev, int type, int64_t arows, int d,
                                   const void *matrices_dev, int transposed, int nlist, int n,
                                   const int32_t *offsets_dev, const int32_t *order_dev, int k,
                                   int64_t rows, void *out_dev, void *stream)
{
    if (ivfpq_status s = check_lists(type, arows, d, nlist, n, order_dev, k, rows))
        return s;
    if (rows == 0)
        return ok();
    if (!rows_dev || !matrices_dev || !offsets_dev || !out_dev)
        return null_pointer();
    const size_t to = type_size(type);
    if (!aligned(rows_dev, to) || !aligned(matrices_dev, to) || !aligned(out_dev, to))
        return fail(IVFPQ_E_INVALID_ARG, "rows and matrices must be aligned to their type");
    ListProduct p;
    p.x = rows_dev;
    p.matrices = matrices_dev;
    p.out = out_dev;
    p.arows = arows;
    p.rows = rows;
    p.d = d;
    p.n = n;
    p.nlist = nlist;
    p.k = k;
    p.transposed = transposed != 0;
    p.offsets = offsets_dev;
    p.order = order_dev;
    return launched(launch_list_product(p, type, reinterpret_cast<hipStream_t>(stream)),
                    "list product kernel");
}

size_t ivfpq_list_product_grad_bytes(int64_t rows, int n, int d, int nlist)
{
    if (!rows_ok(rows) || !width_ok(d) || !width_ok(n) || nlist < 1 || nlist > kMaxLists)
        return 0;
    return list_gradient_bytes(rows, n, d, nlist);
}

ivfpq_status ivfpq_list_product_grad_ex(const void *grad_dev, const void *rows_dev, int type,
                                        int64_t arows, int d, int nlist, int n,
                                        const int32_t *offsets_dev, const int32_t *order_dev, int k,
                                        int64_t rows, int out_type, void *workspace_dev,
                                        size_t workspace_bytes, void *out_dev, void *stream)
{
    if (ivfpq_status s = check_lists(type, arows, d, nlist, n, order_dev, k, rows))
        return s;
    if (out_type != IVFPQ_F32 && out_type != type)
        return fail(IVFPQ_E_INVALID_ARG, "the output's type must be the rows' or float32");
    const size_t need = list_gradient_bytes(rows, n, d, nlist);
    if (!offsets_dev || !out_dev || (rows > 0 && (!grad_dev || !rows_dev)) ||
        (need > 0 && !workspace_dev))
        return null_pointer();
    const size_t to = type_size(type);
    if (!aligned(grad_dev, to) || !aligned(rows_dev, to) || !aligned(out_dev, type_size(out_type)))
        return fail(IVFPQ_E_INVALID_ARG, "rows and matrices must be aligned to their type");
    if (workspace_bytes < need || !aligned(workspace_dev, 16))
        return fail(IVFPQ_E_INVALID_ARG, "the workspace is too small or not 16-byte aligned");
    ListGradient p;
    p.grad = grad_dev;
    p.x = rows_dev;
    p.out = out_dev;
    p.ws = workspace_dev;
    p.arows = arows;
    p.rows = rows;
    p.d = d;
    p.n = n;
    p.nlist = nlist;
    p.k = k;
    p.offsets = offsets_dev;
    p.order = order_dev;
    return launched(launch_list_gradient(p, type, out_type, reinterpret_cast<hipStream_t>(stream)),
                    "list gradient kernel");
}

size_t ivfpq_adapter_product_bytes(int64_t t, int r)
{
    if (!rows_ok(t) || r < 1 || r > kMaxRank)
        return 0;
    return adapter_bytes(t, r);
}

ivfpq_status ivfpq_adapter_product_ex(const void *rows_dev, int type, int64_t t, int d,
                                      const void *matrix_dev, int n, const void *down_dev,
                                      const void *up_dev, int nlist, int r, const float *scales_dev,
                                      const int32_t *offsets_dev, const int32_t *order_dev,
                                      const int32_t *pos_dev, void *workspace_dev,
                                      size_t workspace_bytes, void *out_dev, void *stream)
{
    if (ivfpq_status s = check_lists(type, t, d, nlist, n, order_dev, 1, t))
        return s;
    if (r < 1 || r > kMaxRank)
        return fail(IVFPQ_E_INVALID_ARG, "r must be in [1, 2^12]");
    if (t == 0)
        return ok();
    if (!rows_dev || !matrix_dev || !down_dev || !up_dev || !offsets_dev || !order_dev ||
        !pos_dev || !workspace_dev || !out_dev)
        return null_pointer();
    const size_t to = type_size(type);
    if (!aligned(rows_dev, to) || !aligned(matrix_dev, to) || !aligned(down_dev, to) ||
        !aligned(up_dev, to) || !aligned(out_dev, to))
        return fail(IVFPQ_E_INVALID_ARG, "rows and matrices must be aligned to their type");
    if (workspace_bytes < adapter_bytes(t, r) || !aligned(workspace_dev, 16))
        return fail(IVFPQ_E_INVALID_ARG, "the workspace is too small or not 16-byte aligned");
    AdapterProduct p;
    p.x = rows_dev;
    p.w = matrix_dev;
    p.down = down_dev;
    p.up = up_dev;
    p.scales = scales_dev;
    p.out = out_dev;
    p.ws = workspace_dev;
    p.t = t;
    p.d = d;
    p.n = n;
    p.nlist = nlist;
    p.r = r;
    p.offsets = offsets_dev;
    p.order = order_dev;
    p.pos = pos_dev;
    return launched(launch_adapter(p, type, reinterpret_cast<hipStream_t>(stream)),
                    "adapter kernels");
}

ivfpq_status ivfpq_table_lookup_ex(const void *table_dev, int type, int64_t rows, int d,
                                   const int32_t *ids_dev, int64_t n, float scale, void *out_dev,
                                   void *stream)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (!rows_ok(rows) || !rows_ok(n) || !width_ok(d))
        return fail(IVFPQ_E_INVALID_ARG, "rows and n must be in [0, 2^31) and d in [1, 2^20]");
    if (n == 0)
        return ok();
    if ((rows > 0 && !table_dev) || !ids_dev || !out_dev)
        return null_pointer();
    if (!aligned(table_dev, type_size(type)) || !aligned(out_dev, type_size(type)))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be aligned to their type");
    return launched(launch_table_lookup(table_dev, type, rows, d, ids_dev, n, scale, out_dev,
                                        reinterpret_cast<hipStream_t>(stream)),
                    "table lookup kernel");
}

size_t ivfpq_table_grad_bytes(int64_t nvec, int d, int k)
{
    if (nvec < 0 || k < 1 || nvec > kMaxRows / k || !width_ok(d))
        return 0;
    return table_grad_bytes(nvec * k, d);
}

ivfpq_status ivfpq_table_grad_ex(const void *grad_dev, int type, int64_t nvec, int d,
                                 const int32_t *offsets_dev, const int32_t *order_dev, int k,
                                 int nlist, float scale, int out_type, void *workspace_dev,
                                 size_t workspace_bytes, void *out_dev, void *stream)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (out_type != IVFPQ_F32 && out_type != type)
        return fail(IVFPQ_E_INVALID_ARG, "the output's type must be the rows' or float32");
    if (k < 1 || nvec < 0 || nvec > kMaxRows / k || !width_ok(d))
        return fail(IVFPQ_E_INVALID_ARG, "need k >= 1, nvec k in [0, 2^31) and d in [1, 2^20]");
    if (nlist < 1 || nlist > kMaxRouteLists)
        return fail(IVFPQ_E_INVALID_ARG, "nlist must be in [1, 2^22)");
    const size_t need = table_grad_bytes(nvec * k, d);
    if (!offsets_dev || !out_dev || (nvec > 0 && (!grad_dev || !order_dev)) ||
        (need > 0 && !workspace_dev))
        return null_pointer();
    if (!aligned(grad_dev, type_size(type)) || !aligned(out_dev, type_size(out_type)))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be aligned to their type");
    if (workspace_bytes < need || !aligned(workspace_dev, 16))
        return fail(IVFPQ_E_INVALID_ARG, "the workspace is too small or not 16-byte aligned");
    return launched(launch_table_grad(grad_dev, type, nvec, d, offsets_dev, order_dev, k, nlist,
                                      scale, out_type, out_dev, workspace_dev,
                                      reinterpret_cast<hipStream_t>(stream)),
                    "table gradient kernels");
}

} // extern "C"

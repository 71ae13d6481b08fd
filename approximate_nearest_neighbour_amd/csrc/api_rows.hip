// Entry points of the 4-bit rows, their products and the list routing: argument
// checks on the host, then the kernels on the caller's stream.  Declarations and
// conventions: include/ivfpq.h.
#include "rows_check.hpp"
#include "rows_internal.hpp"

using namespace ivfpq;

namespace {

// Shape of the routed rows: nvec vectors of d values, k slots each.
ivfpq_status check_route(int64_t nvec, int d, int type, int k)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (d < 1 || d > kMaxRowDim)
        return fail(IVFPQ_E_INVALID_ARG, "d must be in [1, 2^20]");
    if (k < 1 || nvec < 0 || nvec > (int64_t)0x7FFFFFFF / k)
        return fail(IVFPQ_E_INVALID_ARG, "need k >= 1, nvec >= 0 and nvec k < 2^31");
    return IVFPQ_OK;
}

ivfpq_status product(Mx4Product p, int type, int d, hipStream_t stream)
{
    p.kb = (d + 31) / 32;
    if (p.m == 0 || p.n == 0)
        return ok();
    if (!p.a || !p.as || !p.b || !p.bs || !p.out)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (!aligned(p.a, 16) || !aligned(p.b, 16) || !aligned(p.out, type_size(type)))
        return fail(IVFPQ_E_INVALID_ARG, "codes must be 16-byte aligned, the output to its type");
    return launched(launch_mx4_product(p, type, stream), "4-bit product kernel");
}

} // namespace

extern "C" {

ivfpq_status ivfpq_mx4_quantize_ex(const void *rows_dev, int type, int64_t rows, int d,
                                   int64_t stride, uint8_t *codes_dev, uint8_t *scales_dev,
                                   void *stream)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (rows < 0 || rows > (int64_t)0x7FFFFFFF || d < 1 || d > kMaxRowDim || stride < 0)
        return fail(IVFPQ_E_INVALID_ARG,
                    "rows must be in [0, 2^31), d in [1, 2^20] and stride at least 0");
    if (rows == 0)
        return ok();
    if (!rows_dev || !codes_dev || !scales_dev)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (!aligned(rows_dev, type_size(type)) || !aligned(codes_dev, 16))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be aligned to their type, codes to 16 bytes");
    return launched(launch_mx4_quantize(rows_dev, type, rows, d, stride, codes_dev, scales_dev,
                                        reinterpret_cast<hipStream_t>(stream)),
                    "4-bit quantize kernel");
}

ivfpq_status ivfpq_mx4_dequantize_ex(const uint8_t *codes_dev, const uint8_t *scales_dev,
                                     int64_t rows, int d, int type, void *out_dev, void *stream)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (rows < 0 || rows > (int64_t)0x7FFFFFFF || d < 1 || d > kMaxRowDim)
        return fail(IVFPQ_E_INVALID_ARG, "rows must be in [0, 2^31) and d in [1, 2^20]");
    if (rows == 0)
        return ok();
    if (!codes_dev || !scales_dev || !out_dev)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (!aligned(codes_dev, 16) || !aligned(out_dev, type_size(type)))
        return fail(IVFPQ_E_INVALID_ARG, "codes must be 16-byte aligned, the output to its type");
    return launched(launch_mx4_dequantize(codes_dev, scales_dev, rows, d, type, out_dev,
                                          reinterpret_cast<hipStream_t>(stream)),
                    "4-bit dequantize kernel");
}

ivfpq_status ivfpq_mx4_product_ex(const uint8_t *a_codes_dev, const uint8_t *a_scales_dev,
                                  int64_t m, const uint8_t *b_codes_dev,
                                  const uint8_t *b_scales_dev, int64_t n, int d, int type,
                                  void *out_dev, void *stream)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (m < 0 || m > (int64_t)0x7FFFFFFF || n < 0 || n > (int64_t)0x7FFFFFF0 || d < 1 ||
        d > kMaxRowDim || (m / 16 + 1) * (n / 16 + 1) > (int64_t)0x7FFFFFFF)
        return fail(IVFPQ_E_INVALID_ARG,
                    "m and n must be in [0, 2^31), m n below 2^39 and d in [1, 2^20]");
    Mx4Product p;
    p.a = a_codes_dev;
    p.as = a_scales_dev;
    p.b = b_codes_dev;
    p.bs = b_scales_dev;
    p.m = p.arows = m;
    p.n = (int)n;
    p.out = out_dev;
    return product(p, type, d, reinterpret_cast<hipStream_t>(stream));
}

ivfpq_status ivfpq_mx4_list_product_ex(const uint8_t *a_codes_dev, const uint8_t *a_scales_dev,
                                       int64_t arows, const uint8_t *b_codes_dev,
                                       const uint8_t *b_scales_dev, int nlist, int64_t n, int d,
                                       const int32_t *offsets_dev, const int32_t *order_dev, int k,
                                       int64_t rows, int type, void *out_dev, void *stream)
{
    if (!type_ok(type))
        return fail(IVFPQ_E_INVALID_ARG, "type must be an ivfpq_type");
    if (arows < 0 || arows > (int64_t)0x7FFFFFFF || rows < 0 || rows > (int64_t)0x7FFFFFFF ||
        n < 0 || n > (int64_t)0x7FFFFFF0 || d < 1 || d > kMaxRowDim ||
        (rows + 1) * (n / 16 + 1) > (int64_t)1 << 30)
        return fail(IVFPQ_E_INVALID_ARG,
                    "rows and n must be in [0, 2^31), rows n below 2^34 and d in [1, 2^20]");
    if (nlist < 1 || nlist > (1 << 16) || k < 1)
        return fail(IVFPQ_E_INVALID_ARG, "nlist must be in [1, 2^16] and k at least 1");
    if (rows > 0 && n > 0 && !offsets_dev)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (rows > 0 && (order_dev ? arows < 1 : arows < rows))
        return fail(IVFPQ_E_INVALID_ARG, "the first operand has too few rows");
    Mx4Product p;
    p.a = a_codes_dev;
    p.as = a_scales_dev;
    p.b = b_codes_dev;
    p.bs = b_scales_dev;
    p.m = rows;
    p.arows = arows;
    p.n = (int)n;
    p.out = out_dev;
    p.offsets = offsets_dev;
    p.order = order_dev;
    p.nlist = nlist;
    p.k = k;
    return product(p, type, d, reinterpret_cast<hipStream_t>(stream));
}

size_t ivfpq_route_sort_bytes(int64_t nvec, int k, int nlist)
{
    if (k < 1 || nvec < 0 || nvec > (int64_t)0x7FFFFFFF / k || nlist < 1 || nlist > kMaxRouteLists)
        return 0;
    return route_sort_bytes(nvec * k, nlist);
}

ivfpq_status ivfpq_route_sort_ex(const int32_t *lists_dev, int64_t nvec, int k, int nlist,
                                 void *workspace_dev, size_t workspace_bytes, int32_t *offsets_dev,
                                 int32_t *order_dev, int32_t *pos_dev, void *stream)
{
    if (ivfpq_status s = check_route(nvec, 1, IVFPQ_F32, k))
        return s;
    if (nlist < 1 || nlist > kMaxRouteLists)
        return fail(IVFPQ_E_INVALID_ARG, "nlist must be in [1, 2^22)");
    const size_t need = route_sort_bytes(nvec * k, nlist);
    if (!offsets_dev || (nvec > 0 && (!lists_dev || !order_dev || !pos_dev)) ||
        (need > 0 && !workspace_dev))
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (workspace_bytes < need || !aligned(workspace_dev, 16))
        return fail(IVFPQ_E_INVALID_ARG, "the workspace is too small or not 16-byte aligned");
    return launched(launch_route_sort(lists_dev, nvec * k, nlist, workspace_dev, offsets_dev,
                                      order_dev, pos_dev, reinterpret_cast<hipStream_t>(stream)),
                    "route sort kernels");
}

ivfpq_status ivfpq_route_gather_ex(const void *vectors_dev, int type, int64_t nvec, int d,
                                   const int32_t *order_dev, const float *weights_dev, int k,
                                   void *rows_dev, void *stream)
{
    if (ivfpq_status s = check_route(nvec, d, type, k))
        return s;
    if (nvec == 0)
        return ok();
    if (!vectors_dev || !order_dev || !rows_dev)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (!aligned(vectors_dev, type_size(type)) || !aligned(rows_dev, type_size(type)))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be aligned to their type");
    return launched(launch_route_gather(vectors_dev, type, nvec, d, order_dev, weights_dev, k,
                                        rows_dev, reinterpret_cast<hipStream_t>(stream)),
                    "route gather kernel");
}

ivfpq_status ivfpq_route_combine_ex(const void *rows_dev, int type, int64_t nvec, int d,
                                    const int32_t *pos_dev, const float *weights_dev, int k,
                                    void *out_dev, void *stream)
{
    if (ivfpq_status s = check_route(nvec, d, type, k))
        return s;
    if (nvec == 0)
        return ok();
    if (!rows_dev || !pos_dev || !out_dev)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (!aligned(rows_dev, type_size(type)) || !aligned(out_dev, type_size(type)))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be aligned to their type");
    return launched(launch_route_combine(rows_dev, type, nvec, d, pos_dev, weights_dev, k, out_dev,
                                         reinterpret_cast<hipStream_t>(stream)),
                    "route combine kernel");
}

ivfpq_status ivfpq_route_combine_grad_ex(const void *grad_dev, const void *rows_dev, int type,
                                         int64_t nvec, int d, const int32_t *order_dev,
                                         const int32_t *pos_dev, const float *weights_dev, int k,
                                         void *grad_rows_dev, float *grad_weights_dev, void *stream)
{
    if (ivfpq_status s = check_route(nvec, d, type, k))
        return s;
    if (nvec == 0)
        return ok();
    if (!grad_dev || !rows_dev || !order_dev || !pos_dev || !weights_dev || !grad_rows_dev ||
        !grad_weights_dev)
        return fail(IVFPQ_E_INVALID_ARG, "a required device pointer is NULL");
    if (!aligned(grad_dev, type_size(type)) || !aligned(rows_dev, type_size(type)) ||
        !aligned(grad_rows_dev, type_size(type)))
        return fail(IVFPQ_E_INVALID_ARG, "rows must be aligned to their type");
    return launched(launch_route_combine_grad(grad_dev, rows_dev, type, nvec, d, order_dev, pos_dev,
                                              weights_dev, k, grad_rows_dev, grad_weights_dev,
                                              reinterpret_cast<hipStream_t>(stream)),
                    "route combine gradient kernel");
}

} // extern "C"

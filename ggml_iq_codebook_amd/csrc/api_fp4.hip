// api_fp4.hip -- the extern "C" entry points of the 4-bit format and the products
// with it (include/iq_fp4.h): argument validation and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "api_common.hpp"
#include "iq_fp4.h"
#include "layers_args.hpp"
#include "layers_launch.hpp"
#include "overlap.hpp"

using iqk::aligned;
using iqk::array;
using iqk::bad_rows;
using iqk::check_device;
using iqk::from_hip;
using iqk::overlaps;
using iqk::region;
using iqk::run_with_status;
using iqk::value_bytes;

namespace {

// Codes and scales of `rows` rows of `cols` values.
bool bad_groups(int64_t rows, int64_t cols, int64_t ldc, int64_t lds, bool output)
{
    return cols < IQ_GROUP || cols % IQ_GROUP || bad_rows(rows, cols / 2, ldc, output) ||
           bad_rows(rows, cols / IQ_GROUP, lds, output);
}

bool bad_product(int64_t tokens, int64_t rows, int64_t channels, int64_t depth, int64_t ldx,
                 int64_t ldw, int64_t lds, int64_t ldy)
{
    return depth > INT32_MAX / 2 || channels < 1 || channels > INT32_MAX / 2 ||
           tokens > INT32_MAX || rows > INT32_MAX || bad_rows(tokens, depth, ldx, false) ||
           bad_groups(channels, depth, ldw, lds, false) || bad_rows(rows, channels, ldy, true);
}

bool bad_stride(int64_t stride, int32_t experts)
{
    return stride < 0 || (stride > 0 && experts > (INT64_C(1) << 61) / stride);
}

// Whether the output meets the memory of one of the experts' rows: all of it first,
// and only where that meets the output each expert's.
bool meets(const iqk::Region& out, const uint8_t* p, int32_t experts, int64_t stride, int64_t rows,
           int64_t cols, int64_t ld)
{
    if (!overlap(out, array(p, (experts - 1) * stride + (rows - 1) * ld + cols, 1))) return false;
    for (int32_t e = 0; e < experts; ++e)
        if (overlap(out, region(p + e * stride, rows, cols, ld, 1))) return true;
    return false;
}

}  // namespace

extern "C" {

iq_status_t iq_quantize_groups(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t rows,
                               int64_t cols, uint8_t* codes, int64_t ldc, uint8_t* scale,
                               int64_t lds, int32_t* status, hipStream_t stream)
{
    if (bad_rows(rows, cols, ldx, false) || bad_groups(rows, cols, ldc, lds, true))
        return IQ_ERR_SHAPE;
    if (rows && (!x || !codes || !scale)) return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(x, bytes) || (status && !aligned(status, 4))) return IQ_ERR_ARG;
    if (!rows) return IQ_OK;
    if (overlaps({region(codes, rows, cols / 2, ldc, 1), region(scale, rows, cols / IQ_GROUP, lds, 1),
                  array(status, 1, 4)},
                 {region(x, rows, cols, ldx, bytes)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    return run_with_status(status, stream, [&](int32_t* s) {
        return iqk::launch_quantize_groups(dtype, x, ldx, rows, cols, codes, ldc, scale, lds, s,
                                           stream);
    });
}

iq_status_t iq_dequantize_groups(const uint8_t* codes, int64_t ldc, const uint8_t* scale,
                                 int64_t lds, int64_t rows, int64_t cols, iq_dtype_t out_dtype,
                                 void* y, int64_t ldy, hipStream_t stream)
{
    if (bad_groups(rows, cols, ldc, lds, false) || bad_rows(rows, cols, ldy, true))
        return IQ_ERR_SHAPE;
    if (rows && (!codes || !scale || !y)) return IQ_ERR_NULL;
    const int bytes = value_bytes(out_dtype);
    if (!bytes || !aligned(y, bytes)) return IQ_ERR_ARG;
    if (!rows) return IQ_OK;
    if (overlaps({region(y, rows, cols, ldy, bytes)},
                 {region(codes, rows, cols / 2, ldc, 1),
                  region(scale, rows, cols / IQ_GROUP, lds, 1)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    return from_hip(iqk::launch_dequantize_groups(codes, ldc, scale, lds, rows, cols, out_dtype, y,
                                                  ldy, stream));
}

int64_t iq_fp4_linear_workspace(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t tokens,
                                int64_t channels, int64_t depth)
{
    if (tokens < 1 || !value_bytes(dtype) ||
        bad_product(tokens, tokens, channels, depth, ldx, depth / 2, depth / IQ_GROUP, channels))
        return 0;
    return iqk::fp4_workspace(dtype, x, ldx, tokens, tokens, 0, channels, depth);
}

iq_status_t iq_fp4_linear(iq_dtype_t dtype, const void* x, int64_t ldx, const uint8_t* w,
                          int64_t ldw, const uint8_t* w_scale, int64_t lds, int64_t tokens,
                          int64_t channels, int64_t depth, void* y, int64_t ldy, void* workspace,
                          int64_t workspace_bytes, hipStream_t stream)
{
    if (bad_product(tokens, tokens, channels, depth, ldx, ldw, lds, ldy)) return IQ_ERR_SHAPE;
    const int64_t need = iq_fp4_linear_workspace(dtype, x, ldx, tokens, channels, depth);
    if (tokens && (!x || !w || !w_scale || !y || (need && !workspace))) return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(x, bytes) || !aligned(y, bytes) || !aligned(workspace, 16) ||
        workspace_bytes < need)
        return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    if (overlaps({region(y, tokens, channels, ldy, bytes), array(workspace, need, 1)},
                 {region(x, tokens, depth, ldx, bytes), region(w, channels, depth / 2, ldw, 1),
                  region(w_scale, channels, depth / IQ_GROUP, lds, 1)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    const iqk::Fp4Product p = {x, ldx, w, ldw, 0, w_scale, lds, 0, y, ldy, tokens, tokens,
                               (int)channels, (int)depth, (int)dtype, nullptr, nullptr, 0, 1};
    return from_hip(iqk::launch_fp4_product(p, workspace, stream));
}

int64_t iq_fp4_expert_linear_workspace(iq_dtype_t dtype, const void* x, int64_t ldx,
                                       int64_t tokens, int32_t experts, int64_t rows,
                                       int64_t channels, int64_t depth)
{
    if (tokens < 1 || rows < 1 || experts < 1 || experts > IQ_MAX_EXPERTS || !value_bytes(dtype) ||
        bad_product(tokens, rows, channels, depth, ldx, depth / 2, depth / IQ_GROUP, channels))
        return 0;
    return iqk::fp4_workspace(dtype, x, ldx, tokens, rows, experts, channels, depth);
}

iq_status_t iq_fp4_expert_linear(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t tokens,
                                 const int32_t* order, int32_t top_k, const int32_t* offsets,
                                 int32_t experts, int64_t rows, const uint8_t* w, int64_t ldw,
                                 int64_t w_stride, const uint8_t* w_scale, int64_t lds,
                                 int64_t s_stride, int64_t channels, int64_t depth, void* y,
                                 int64_t ldy, void* workspace, int64_t workspace_bytes,
                                 hipStream_t stream)
{
    if (bad_product(tokens, rows, channels, depth, ldx, ldw, lds, ldy) || top_k < 1 ||
        experts < 1 || experts > IQ_MAX_EXPERTS || bad_stride(w_stride, experts) ||
        bad_stride(s_stride, experts) || (rows > 0 && tokens < (order ? 1 : rows)))
        return IQ_ERR_SHAPE;
    const int64_t need = iq_fp4_expert_linear_workspace(dtype, x, ldx, tokens, experts, rows,
                                                        channels, depth);
    if (rows && (!x || !offsets || !w || !w_scale || !y || (need && !workspace)))
        return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(x, bytes) || !aligned(y, bytes) || !aligned(order, 4) ||
        !aligned(offsets, 4) || !aligned(workspace, 16) || workspace_bytes < need)
        return IQ_ERR_ARG;
    if (!rows) return IQ_OK;
    const iqk::Region out[] = {region(y, rows, channels, ldy, bytes), array(workspace, need, 1)};
    if (overlaps(out, {region(x, tokens, depth, ldx, bytes), array(order, rows, 4),
                       array(offsets, (int64_t)experts + 1, 4)}))
        return IQ_ERR_ARG;
    for (const iqk::Region& o : out)
        if (meets(o, w, experts, w_stride, channels, depth / 2, ldw) ||
            meets(o, w_scale, experts, s_stride, channels, depth / IQ_GROUP, lds))
            return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    const iqk::Fp4Product p = {x, ldx, w, ldw, w_stride, w_scale, lds, s_stride, y, ldy, tokens,
                               rows, (int)channels, (int)depth, (int)dtype, order, offsets,
                               experts, top_k};
    return from_hip(iqk::launch_fp4_product(p, workspace, stream));
}

}  // extern "C"

// api_layers.hip -- the extern "C" entry points declared in
// include/iq_layers.h: argument validation and the stream-ordered launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "api_common.hpp"
#include "iq_layers.h"
#include "layers_launch.hpp"
#include "overlap.hpp"

using iqk::aligned;
using iqk::array;
using iqk::check_device;
using iqk::from_hip;
using iqk::overlaps;
using iqk::region;
using iqk::run_with_status;

namespace {

// Bytes per value, 0 for a type these calls do not take.
int value_bytes(iq_dtype_t t)
{
    return t == IQ_DTYPE_F32 ? 4 : (t == IQ_DTYPE_BF16 || t == IQ_DTYPE_F16 ? 2 : 0);
}

// Rows of `cols` values with stride ld: every offset stays below 2^61.
// Outputs may not have rows that overlap (ld >= cols); inputs may.
bool bad_rows(int64_t rows, int64_t cols, int64_t ld, bool output)
{
    if (rows < 0 || cols < 1 || ld < 0 || (output && rows > 1 && ld < cols)) return true;
    const int64_t most = INT64_C(1) << 61;
    return cols > most || (ld > 0 && rows > most / ld);
}

// Places are 32-bit.
bool bad_choices(int64_t tokens, int32_t top_k)
{
    return tokens < 0 || top_k < 1 || tokens > INT32_MAX / top_k;
}

bool bad_product(int64_t tokens, int64_t channels, int64_t depth, int64_t ldx, int64_t ldw,
                 int64_t ldy, int64_t rows)
{
    return depth < 1 || depth > IQ_MAX_INT8_DEPTH || channels < 1 || channels > INT32_MAX / 2 ||
           tokens > INT32_MAX || rows > INT32_MAX || bad_rows(tokens, depth, ldx, false) ||
           bad_rows(channels, depth, ldw, false) || bad_rows(rows, channels, ldy, true);
}

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// The codes of iq_int8_linear: rows that start on 16 bytes.
int64_t code_stride(int64_t depth) { return round_up(depth, 16); }

iqk::Route route(iq_dtype_t dtype, int64_t tokens, int64_t width, const int32_t* position,
                 int32_t top_k, const int32_t* offsets, int32_t experts)
{
    return {tokens, tokens * top_k, width, position, top_k, offsets + experts,
            iqk::streams(tokens * top_k, width, value_bytes(dtype))};
}

// One tensor of a routing call: [tokens][width], or [tokens * top_k][width]
// where it is sorted.  The output comes last.
struct Rows {
    const void* p;
    int64_t ld;
    bool sorted;
    bool output;
};

template <int kN>
iq_status_t route_args(iq_dtype_t dtype, int64_t tokens, int64_t width, int32_t top_k,
                       int32_t experts, const int32_t* position, const int32_t* offsets,
                       const Rows (&tensors)[kN])
{
    if (bad_choices(tokens, top_k) || experts < 1 || experts > IQ_MAX_EXPERTS)
        return IQ_ERR_SHAPE;
    for (const Rows& t : tensors)
        if (bad_rows(t.sorted ? tokens * top_k : tokens, width, t.ld, t.output))
            return IQ_ERR_SHAPE;
    if (tokens) {
        if (!position || !offsets) return IQ_ERR_NULL;
        for (const Rows& t : tensors)
            if (!t.p) return IQ_ERR_NULL;
    }
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(position, 4) || !aligned(offsets, 4)) return IQ_ERR_ARG;
    for (const Rows& t : tensors)
        if (!aligned(t.p, bytes)) return IQ_ERR_ARG;
    return IQ_OK;
}

// Whether the last of the tensors, the output, or the weights' gradient overlaps
// something else of the call.
template <int kN>
bool route_overlaps(iq_dtype_t dtype, int64_t tokens, int64_t width, int32_t top_k,
                    int32_t experts, const int32_t* position, const int32_t* offsets,
                    const float* weights, const float* weights_grad, const Rows (&tensors)[kN])
{
    const int64_t n = tokens * top_k;
    iqk::Region out[2], in[kN + 2];
    for (int i = 0; i < kN; ++i) {
        const Rows& t = tensors[i];
        (i < kN - 1 ? in[i] : out[0]) =
            region(t.p, t.sorted ? n : tokens, width, t.ld, value_bytes(dtype));
    }
    out[1] = array(weights_grad, n, 4);
    in[kN - 1] = array(position, n, 4);
    in[kN] = array(offsets, (int64_t)experts + 1, 4);
    in[kN + 1] = array(weights, n, 4);
    return overlaps(out, in);
}

}  // namespace

extern "C" {

iq_status_t iq_quantize_rows(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t rows,
                             int64_t cols, int8_t* q, int64_t ldq, float* scale, int32_t* status,
                             hipStream_t stream)
{
    if (rows > INT32_MAX || bad_rows(rows, cols, ldx, false) || bad_rows(rows, cols, ldq, true))
        return IQ_ERR_SHAPE;
    if (rows && (!x || !q || !scale)) return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(x, bytes) || !aligned(scale, 4) || (status && !aligned(status, 4)))
        return IQ_ERR_ARG;
    if (!rows) return IQ_OK;
    if (overlaps({region(q, rows, cols, ldq, 1), array(scale, rows, 4), array(status, 1, 4)},
                 {region(x, rows, cols, ldx, bytes)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    return run_with_status(status, stream, [&](int32_t* s) {
        return iqk::launch_quantize_rows(dtype, x, ldx, rows, cols, q, ldq, scale, s, stream);
    });
}

iq_status_t iq_int8_matmul(const int8_t* x, int64_t ldx, const float* x_scale, const int8_t* w,
                           int64_t ldw, const float* w_scale, int64_t tokens, int64_t channels,
                           int64_t depth, iq_dtype_t out_dtype, void* y, int64_t ldy,
                           hipStream_t stream)
{
    if (bad_product(tokens, channels, depth, ldx, ldw, ldy, tokens)) return IQ_ERR_SHAPE;
    if (tokens && (!x || !x_scale || !w || !w_scale || !y)) return IQ_ERR_NULL;
    const int bytes = value_bytes(out_dtype);
    if (!bytes || !aligned(y, bytes) || !aligned(x_scale, 4) || !aligned(w_scale, 4))
        return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    if (overlaps({region(y, tokens, channels, ldy, bytes)},
                 {region(x, tokens, depth, ldx, 1), array(x_scale, tokens, 4),
                  region(w, channels, depth, ldw, 1), array(w_scale, channels, 4)}))
        return IQ_ERR_ARG;
    int cus = 1;
    const iq_status_t st = check_device(&cus);
    if (st) return st;
    const iqk::Int8Product p = {x,      ldx,    x_scale, w,       ldw,
                                0,      w_scale, y,      ldy,     tokens,
                                tokens, (int)channels,   (int)depth, (int)out_dtype,
                                nullptr, nullptr, 0,     1};
    return from_hip(iqk::launch_int8_product(p, cus, stream));
}

int64_t iq_int8_linear_workspace(int64_t tokens, int64_t channels, int64_t depth)
{
    if (tokens < 1 || tokens > INT32_MAX || channels < 1 || channels > INT32_MAX || depth < 1 ||
        depth > IQ_MAX_INT8_DEPTH || iqk::int8_decode_takes(tokens, channels, depth))
        return 0;
    return tokens * code_stride(depth) + round_up(tokens * 4, 16);
}

iq_status_t iq_int8_linear(iq_dtype_t dtype, const void* x, int64_t ldx, const int8_t* w,
                           int64_t ldw, const float* w_scale, int64_t tokens, int64_t channels,
                           int64_t depth, void* y, int64_t ldy, void* workspace,
                           int64_t workspace_bytes, int32_t* status, hipStream_t stream)
{
    if (bad_product(tokens, channels, depth, ldx, ldw, ldy, tokens)) return IQ_ERR_SHAPE;
    const int64_t need = iq_int8_linear_workspace(tokens, channels, depth);
    if (tokens && (!x || !w || !w_scale || !y || (need && !workspace))) return IQ_ERR_NULL;
    const int bytes = value_bytes(dtype);
    if (!bytes || !aligned(x, bytes) || !aligned(y, bytes) || !aligned(w_scale, 4) ||
        !aligned(workspace, 16) || workspace_bytes < need || (status && !aligned(status, 4)))
        return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    if (overlaps({region(y, tokens, channels, ldy, bytes), array(workspace, need, 1),
                  array(status, 1, 4)},
                 {region(x, tokens, depth, ldx, bytes), region(w, channels, depth, ldw, 1),
                  array(w_scale, channels, 4)}))
        return IQ_ERR_ARG;
    int cus = 1;
    const iq_status_t st = check_device(&cus);
    if (st) return st;
    int8_t* codes = static_cast<int8_t*>(workspace);
    const int64_t ldc = code_stride(depth);
    float* scale = codes ? reinterpret_cast<float*>(codes + tokens * ldc) : nullptr;
    const iqk::Int8Product p = {codes,  ldc,    scale,   w,       ldw,
                                0,      w_scale, y,      ldy,     tokens,
                                tokens, (int)channels,   (int)depth, (int)dtype,
                                nullptr, nullptr, 0,     1};
    return run_with_status(status, stream, [&](int32_t* s) {
        if (iqk::int8_decode_takes(tokens, channels, depth))
            return iqk::launch_int8_decode(p, dtype, x, ldx, s, stream);
        const hipError_t e = iqk::launch_quantize_rows(dtype, x, ldx, tokens, depth, codes, ldc,
                                                       scale, s, stream);
        return e != hipSuccess ? e : iqk::launch_int8_product(p, cus, stream);
    });
}

iq_status_t iq_int8_expert_matmul(const int8_t* x, int64_t ldx, const float* x_scale,
                                  int64_t tokens, const int32_t* order, int32_t top_k,
                                  const int32_t* offsets, int32_t experts, int64_t rows,
                                  const int8_t* w, int64_t ldw, int64_t w_stride,
                                  const float* w_scale, int64_t channels, int64_t depth,
                                  iq_dtype_t out_dtype, void* y, int64_t ldy, hipStream_t stream)
{
    if (bad_product(tokens, channels, depth, ldx, ldw, ldy, rows) || top_k < 1 || experts < 1 ||
        experts > IQ_MAX_EXPERTS || w_stride < 0 ||
        (w_stride > 0 && experts > (INT64_C(1) << 61) / w_stride) || tokens < 0 ||
        (rows > 0 && tokens < (order ? 1 : rows)))
        return IQ_ERR_SHAPE;
    if (rows && (!x || !x_scale || !offsets || !w || !w_scale || !y)) return IQ_ERR_NULL;
    const int bytes = value_bytes(out_dtype);
    if (!bytes || !aligned(y, bytes) || !aligned(x_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(order, 4) || !aligned(offsets, 4))
        return IQ_ERR_ARG;
    if (!rows) return IQ_OK;
    const iqk::Region out = region(y, rows, channels, ldy, bytes);
    if (overlaps({out}, {region(x, tokens, depth, ldx, 1), array(x_scale, tokens, 4),
                         array(order, rows, 4), array(offsets, (int64_t)experts + 1, 4),
                         array(w_scale, experts * channels, 4)}))
        return IQ_ERR_ARG;
    // The weights as a whole first: only where that meets the output, each of them.
    if (overlap(out, array(w, (experts - 1) * w_stride + (channels - 1) * ldw + depth, 1)))
        for (int32_t e = 0; e < experts; ++e)
            if (overlap(out, region(w + e * w_stride, channels, depth, ldw, 1))) return IQ_ERR_ARG;
    int cus = 1;
    const iq_status_t st = check_device(&cus);
    if (st) return st;
    const iqk::Int8Product p = {x,     ldx,     x_scale, w,        ldw,
                                w_stride, w_scale, y,    ldy,      tokens,
                                rows,  (int)channels,    (int)depth, (int)out_dtype,
                                order, offsets, experts, top_k};
    return from_hip(iqk::launch_int8_product(p, cus, stream));
}

int64_t iq_expert_sort_workspace(int64_t choices, int32_t experts)
{
    if (choices < 1 || choices > INT32_MAX || experts < 1 || experts > IQ_MAX_EXPERTS) return 0;
    const int chunks = iqk::expert_sort_plan(choices).chunks;
    return chunks > 1 ? (int64_t)chunks * (experts + 1) * 4 : 0;
}

iq_status_t iq_expert_sort(const void* choice, int32_t choice_bytes, int64_t tokens, int32_t top_k,
                           int32_t experts, int32_t* order, int32_t* position, int32_t* offsets,
                           void* workspace, int64_t workspace_bytes, int32_t* status,
                           hipStream_t stream)
{
    if (bad_choices(tokens, top_k) || experts < 1 || experts > IQ_MAX_EXPERTS) return IQ_ERR_SHAPE;
    const int64_t need = iq_expert_sort_workspace(tokens * top_k, experts);
    if (!offsets || (tokens && (!choice || !order || !position)) || (need && !workspace))
        return IQ_ERR_NULL;
    if ((choice_bytes != 4 && choice_bytes != 8) || !aligned(choice, choice_bytes) ||
        !aligned(order, 4) || !aligned(position, 4) || !aligned(offsets, 4) ||
        !aligned(workspace, 4) || workspace_bytes < need || (status && !aligned(status, 4)))
        return IQ_ERR_ARG;
    const int64_t n = tokens * top_k;
    if (overlaps({array(order, n, 4), array(position, n, 4), array(offsets, (int64_t)experts + 1, 4),
                  array(workspace, need, 1), array(status, 1, 4)},
                 {array(choice, n, choice_bytes)}))
        return IQ_ERR_ARG;
    const iq_status_t st = check_device();
    if (st) return st;
    return run_with_status(status, stream, [&](int32_t* s) {
        return iqk::launch_expert_sort(choice, choice_bytes, n, experts, order, position, offsets,
                                       static_cast<int32_t*>(workspace), s, stream);
    });
}

iq_status_t iq_expert_dispatch(iq_dtype_t dtype, const void* x, int64_t ldx, int64_t tokens,
                               int64_t width, const int32_t* position, int32_t top_k,
                               const int32_t* offsets, int32_t experts, void* sorted, int64_t lds,
                               hipStream_t stream)
{
    const Rows tensors[] = {{x, ldx, false, false}, {sorted, lds, true, true}};
    iq_status_t st = route_args(dtype, tokens, width, top_k, experts, position, offsets, tensors);
    if (st || !tokens) return st;
    if (route_overlaps(dtype, tokens, width, top_k, experts, position, offsets, nullptr, nullptr,
                       tensors))
        return IQ_ERR_ARG;
    st = check_device();
    if (st) return st;
    const iqk::Route r = route(dtype, tokens, width, position, top_k, offsets, experts);
    return from_hip(iqk::launch_expert_dispatch(dtype, r, x, ldx, sorted, lds, stream));
}

iq_status_t iq_expert_dispatch_backward(iq_dtype_t dtype, const void* sorted_grad, int64_t lds,
                                        int64_t tokens, int64_t width, const int32_t* position,
                                        int32_t top_k, const int32_t* offsets, int32_t experts,
                                        void* x_grad, int64_t ldx, hipStream_t stream)
{
    const Rows tensors[] = {{sorted_grad, lds, true, false}, {x_grad, ldx, false, true}};
    iq_status_t st = route_args(dtype, tokens, width, top_k, experts, position, offsets, tensors);
    if (st || !tokens) return st;
    if (route_overlaps(dtype, tokens, width, top_k, experts, position, offsets, nullptr, nullptr,
                       tensors))
        return IQ_ERR_ARG;
    st = check_device();
    if (st) return st;
    const iqk::Route r = route(dtype, tokens, width, position, top_k, offsets, experts);
    return from_hip(iqk::launch_expert_combine(dtype, r, sorted_grad, lds, nullptr, x_grad, ldx,
                                               stream));
}

iq_status_t iq_expert_combine(iq_dtype_t dtype, const void* y, int64_t ldy, int64_t tokens,
                              int64_t width, const int32_t* position, int32_t top_k,
                              const int32_t* offsets, int32_t experts, const float* weights,
                              void* out, int64_t ldo, hipStream_t stream)
{
    const Rows tensors[] = {{y, ldy, true, false}, {out, ldo, false, true}};
    iq_status_t st = route_args(dtype, tokens, width, top_k, experts, position, offsets, tensors);
    if (st) return st;
    if (tokens && !weights) return IQ_ERR_NULL;
    if (!aligned(weights, 4)) return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    if (route_overlaps(dtype, tokens, width, top_k, experts, position, offsets, weights, nullptr,
                       tensors))
        return IQ_ERR_ARG;
    st = check_device();
    if (st) return st;
    const iqk::Route r = route(dtype, tokens, width, position, top_k, offsets, experts);
    return from_hip(iqk::launch_expert_combine(dtype, r, y, ldy, weights, out, ldo, stream));
}

iq_status_t iq_expert_combine_backward(iq_dtype_t dtype, const void* out_grad, int64_t ldo,
                                       const void* y, int64_t ldy, int64_t tokens, int64_t width,
                                       const int32_t* position, int32_t top_k,
                                       const int32_t* offsets, int32_t experts,
                                       const float* weights, void* y_grad, int64_t ldg,
                                       float* weights_grad, hipStream_t stream)
{
    const Rows tensors[] = {{out_grad, ldo, false, false}, {y, ldy, true, false},
                            {y_grad, ldg, true, true}};
    iq_status_t st = route_args(dtype, tokens, width, top_k, experts, position, offsets, tensors);
    if (st) return st;
    if (tokens && (!weights || !weights_grad)) return IQ_ERR_NULL;
    if (!aligned(weights, 4) || !aligned(weights_grad, 4)) return IQ_ERR_ARG;
    if (!tokens) return IQ_OK;
    if (route_overlaps(dtype, tokens, width, top_k, experts, position, offsets, weights,
                       weights_grad, tensors))
        return IQ_ERR_ARG;
    st = check_device();
    if (st) return st;
    const iqk::Route r = route(dtype, tokens, width, position, top_k, offsets, experts);
    return from_hip(iqk::launch_expert_combine_backward(dtype, r, out_grad, ldo, y, ldy, weights,
                                                        y_grad, ldg, weights_grad, stream));
}

}  // extern "C"

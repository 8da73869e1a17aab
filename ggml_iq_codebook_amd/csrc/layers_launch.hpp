// layers_launch.hpp -- host-side launchers of the layer operators, called by
// the entry points in api_layers.hip after argument validation.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch_parts.hpp"

namespace iqk {

hipError_t launch_quantize_rows(int dtype, const void* x, int64_t ldx, int64_t rows, int64_t cols,
                                int8_t* q, int64_t ldq, float* scale, int32_t* status,
                                hipStream_t stream);

// An 8-bit product.  Dense: experts = 0, rows = tokens.  By expert: rows of y
// in the order of their experts, the token of row p being order[p] / top_k
// (p where order is null).
struct Int8Product {
    const int8_t* x;
    int64_t ldx;
    const float* x_scale;
    const int8_t* w;
    int64_t ldw;
    int64_t w_stride;         // from one expert's weight to the next
    const float* w_scale;
    void* y;
    int64_t ldy;
    int64_t tokens;
    int64_t rows;
    int channels;
    int depth;
    int out_dtype;
    const int32_t* order;
    const int32_t* offsets;
    int experts;
    int top_k;
    int64_t first_tile = 0;   // of the launch's part of the tiles
};

hipError_t launch_int8_product(const Int8Product& p, int cus, hipStream_t stream);

// The layer for a few tokens, rounding included, as one launch.  A workgroup has
// 16 channels and rounds all tokens, dealt out in parts of 512 values of which it
// keeps up to kDecodeParts.
constexpr int kDecodeParts = 32;
constexpr int kDecodeChannels = 16;
__host__ __device__ constexpr int decode_stride(int depth)
{
    // Whole pieces of 64, and rows that start on different banks.
    return (depth + 63) / 64 * 64 + 16;
}
// Where one launch pays: its rounding is repeated by every workgroup, so its cost
// goes with the parts and with the rounds of workgroups on the 256 compute
// units of a whole card (not the device's own: the rule also sizes the workspace,
// which has to be the same wherever it is asked).  GPU time, one launch against
// two, us (as calls of their own the second launch adds 3 more):
//   channels x depth, tokens   1            2            4            8
//   1024 x 1024                3.6 / 6.0                              5.0 / 6.4
//   4096 x 4096                7.8 / 10.0   8.8 / 9.8   10.5 / 9.9
//   5632 x 2048                6.3 / 7.8    6.6 / 7.9    9.3 / 8.0
//   4096 x 16384              19.2 / 25.5
//   16384 x 4096              17.4 / 19.7  19.0 / 18.9  21.5 / 19.2
//   32768 x 2048              21.3 / 18.7
inline bool int8_decode_takes(int64_t tokens, int64_t channels, int64_t depth)
{
    const int64_t rounds = (channels + 256 * kDecodeChannels - 1) / (256 * kDecodeChannels);
    return tokens <= 16 && rounds <= 4 &&
           tokens * ((depth + 511) / 512) * rounds <= (tokens == 1 ? kDecodeParts : kDecodeParts / 2);
}
// p.x, p.x_scale are not used; y has the type of x.
hipError_t launch_int8_decode(const Int8Product& p, int dtype, const void* x, int64_t ldx,
                              int32_t* status, hipStream_t stream);

// Routing.  chunks: how many workgroups share the sort of n choices.
struct SortPlan {
    int chunks;
    int64_t per_chunk;
};
SortPlan expert_sort_plan(int64_t n);
hipError_t launch_expert_sort(const void* choice, int choice_bytes, int64_t n, int experts,
                              int32_t* order, int32_t* position, int32_t* offsets,
                              int32_t* counts, int32_t* status, hipStream_t stream);

struct Route {
    int64_t tokens;
    int64_t rows;             // of a sorted tensor
    int64_t width;
    const int32_t* position;
    int top_k;
    const int32_t* kept;      // offsets + experts: the number of kept choices
    bool streaming;           // sorted rows that are written go past the caches
};

// Sorted rows larger than half of the 256 MiB cache in front of HBM push out
// what the next kernels read, and are not there any more themselves when they
// are read: writing them past the caches took the routing of a training step
// (4096 x 8 rows of 4096 bf16 values, forward and gradients) from 317 to 286 us.
// Smaller ones stay where the next kernel finds them.
inline bool streams(int64_t rows, int64_t width, int bytes)
{
    return rows * width * bytes > (INT64_C(128) << 20);
}

hipError_t launch_expert_dispatch(int dtype, const Route& r, const void* x, int64_t ldx,
                                  void* sorted, int64_t lds, hipStream_t stream);
// weights null: all 1 (the gradient of dispatch).
hipError_t launch_expert_combine(int dtype, const Route& r, const void* y, int64_t ldy,
                                 const float* weights, void* out, int64_t ldo,
                                 hipStream_t stream);
hipError_t launch_expert_combine_backward(int dtype, const Route& r, const void* out_grad,
                                          int64_t ldo, const void* y, int64_t ldy,
                                          const float* weights, void* y_grad, int64_t ldg,
                                          float* weights_grad, hipStream_t stream);

}  // namespace iqk

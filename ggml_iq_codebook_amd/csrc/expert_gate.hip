// expert_gate.hip -- the router: each token's experts and their weights from its
// logits, the loss that keeps the experts evenly used, and the gradients of both.
//   p = softmax(l) over the experts;
//   gate: the k largest l, the lowest index where they are equal, with weights
//         p_c, or p_c / (sum of the chosen p) where they are renormalized;
//   loss = E * sum_e (counts_e / C) (1/N) sum_t p_te   (C choices, N live tokens).
//
// kL lanes share a row and keep it in registers; what crosses lanes is a maximum
// or a sum of kL values by lane exchanges (no LDS, no barrier).  A logit of -inf
// is an expert that cannot be chosen, a row of them a token that does not count.
// A row with a NaN or +inf is reported and treated as such a row.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "iq_router.h"
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

constexpr int kThreads = 256;
constexpr float kNone = -__builtin_inff();

// op over the kL lanes of a row, the same result in all of them.
template <int kL, class T, class Op>
__device__ __forceinline__ T across(T v, Op&& op)
{
    if constexpr (kL > 1) v = op(v, quad_xchg<kQuadXor1>(v));
    if constexpr (kL > 2) v = op(v, quad_xchg<kQuadXor2>(v));
    if constexpr (kL > 4) v = op(v, quad_xchg<0x141>(v));     // lane 7 - i of 8
    if constexpr (kL > 8) v = op(v, quad_xchg<0x140>(v));     // lane 15 - i of 16
    if constexpr (kL > 16) v = op(v, __shfl_xor(v, 16));
    return v;
}

template <int kL>
__device__ __forceinline__ float max_across(float v)
{
    return across<kL>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int kL, class T>
__device__ __forceinline__ T sum_across(T v)
{
    return across<kL>(v, [](T a, T b) { return a + b; });
}

// A row of logits: lane `lane` of kL has kC vectors, experts at(c) .. + kN - 1.
template <int kDT, int kL, int kC>
struct LogitRow {
    typedef typename Value<kDT>::raw raw;
    static constexpr int kN = Row<kDT>::kN, kV = kC * kN;
    float v[kV];
    float top;
    // Whether the row is refused (a NaN or +inf); its values are -inf then.
    bool bad;
    __device__ __forceinline__ static int at(int lane, int c) { return (c * kL + lane) * kN; }
    __device__ __forceinline__ static int expert(int lane, int i) { return at(lane, i / kN) + i % kN; }
    __device__ __forceinline__ void load(const Logits& l, int64_t row, int lane)
    {
        const raw* from = static_cast<const raw*>(l.p) + row * l.ld;
        Row<kDT> r[kC];
#pragma unroll
        for (int c = 0; c < kC; ++c) r[c].load(from, at(lane, c), l.experts);
        int wrong = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            v[i] = r[i / kN][i % kN];
            if (expert(lane, i) >= l.experts) v[i] = kNone;
            wrong |= !(v[i] < __builtin_inff());
        }
        bad = across<kL>(wrong, [](int a, int b) { return a | b; }) != 0;
        top = kNone;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            if (bad) v[i] = kNone;
            top = fmaxf(top, v[i]);
        }
        top = max_across<kL>(top);
    }
    __device__ __forceinline__ bool live() const { return top > kNone; }
    // e = exp(v - top) of the lane's values; their sum over the row.  Live rows.
    __device__ __forceinline__ float exps(float (&e)[kV]) const
    {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            e[i] = expf(v[i] - top);
            sum += e[i];
        }
        return sum_across<kL>(sum);
    }
};

template <int kDT, int kL, int kC>
__global__ __launch_bounds__(kThreads) void expert_gate_kernel(Logits l, int64_t first, int top_k,
                                                               bool renormalize,
                                                               int32_t* __restrict__ choice,
                                                               float* __restrict__ weights,
                                                               int32_t* status)
{
    typedef LogitRow<kDT, kL, kC> R;
    const int lane = threadIdx.x % kL;
    const int64_t row = (first + blockIdx.x) * (kThreads / kL) + threadIdx.x / kL;
    if (row >= l.tokens) return;
    R r;
    r.load(l, row, lane);
    if (r.bad && lane == 0) report_generic(status, IQ_ERR_NONFINITE);
    float sum = 0.0f;
    if (!renormalize && r.live()) {
        float e[R::kV];
        sum = r.exps(e);
    }
    int32_t* to_choice = choice + row * top_k;
    float* to_weight = weights + row * top_k;
    int32_t my_choice = -1;
    float my_weight = 0.0f;
    for (int j = 0; j < top_k; ++j) {
        float m = kNone;
#pragma unroll
        for (int i = 0; i < R::kV; ++i) m = fmaxf(m, r.v[i]);
        m = max_across<kL>(m);
        int who = INT32_MAX;
#pragma unroll
        for (int i = R::kV - 1; i >= 0; --i)
            if (r.v[i] == m) who = R::expert(lane, i);
        who = across<kL>(who, [](int a, int b) { return min(a, b); });
        const bool kept = m > kNone;
        const float e = kept ? expf(m - r.top) : 0.0f;
        if (renormalize) sum += e;
#pragma unroll
        for (int i = 0; i < R::kV; ++i)
            if (R::expert(lane, i) == who) r.v[i] = kNone;
        if (j % kL == lane) {
            my_choice = kept ? who : -1;
            my_weight = e;
        }
        // A block of kL choices, one to a lane.
        const int block = j / kL * kL;
        if ((j % kL == kL - 1 || j == top_k - 1) && block + lane <= j) {
            to_choice[block + lane] = my_choice;
            // Where later blocks add to the sum, divided below.
            if (!renormalize || (block == 0 && j == top_k - 1))
                my_weight = my_weight > 0.0f ? my_weight / sum : 0.0f;
            to_weight[block + lane] = my_weight;
        }
    }
    if (renormalize && top_k > kL)
        for (int j = lane; j < top_k; j += kL) {
            const float e = to_weight[j];
            to_weight[j] = e > 0.0f ? e / sum : 0.0f;
        }
}

// The gradient of the logits for the gradient g of the weights w, with
// s = sum_j g_j w_j: renormalized, w_j (g_j - s) at choice j and 0 elsewhere;
// otherwise g_j w_j there, less p_e s everywhere.
template <int kDT, int kL, int kC>
__global__ __launch_bounds__(kThreads) void expert_gate_backward_kernel(
    Logits l, int64_t first, const float* __restrict__ weights_grad,
    const int32_t* __restrict__ choice, const float* __restrict__ weights, int top_k,
    bool renormalize, void* __restrict__ grad, int64_t ldg)
{
    typedef LogitRow<kDT, kL, kC> R;
    typedef typename R::raw raw;
    const int lane = threadIdx.x % kL;
    const int64_t row = (first + blockIdx.x) * (kThreads / kL) + threadIdx.x / kL;
    if (row >= l.tokens) return;
    const int32_t* c = choice + row * top_k;
    const float *g = weights_grad + row * top_k, *w = weights + row * top_k;
    float s = 0.0f;
    for (int j = lane; j < top_k; j += kL)
        if ((uint32_t)c[j] < (uint32_t)l.experts) s += g[j] * w[j];
    s = sum_across<kL>(s);

    float out[R::kV] = {};
    if (!renormalize) {
        R r;
        r.load(l, row, lane);
        if (r.live()) {
            const float factor = -s / r.exps(out);
#pragma unroll
            for (int i = 0; i < R::kV; ++i) out[i] *= factor;
        }
    }
    for (int j = 0; j < top_k; ++j) {
        const int at = c[j];
        if ((uint32_t)at >= (uint32_t)l.experts) continue;
        const float add = renormalize ? w[j] * (g[j] - s) : g[j] * w[j];
#pragma unroll
        for (int i = 0; i < R::kV; ++i)
            if (R::expert(lane, i) == at) out[i] += add;
    }
    raw* to = static_cast<raw*>(grad) + row * ldg;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
        Row<kDT> o;
        o.zero();
#pragma unroll
        for (int i = 0; i < R::kN; ++i) o.set(i, out[k * R::kN + i]);
        o.store(to, R::at(lane, k), l.experts);
    }
}

// ---------------------------------------------------------------------------
// The balance loss
// ---------------------------------------------------------------------------

constexpr int kSumThreads = 512, kSumWaves = kSumThreads / kWave;

// The loss from the sums of the probabilities and the counts in LDS; all threads,
// each with its part of the live tokens.
__device__ __forceinline__ void finish(const double* probability, const int* count, int live,
                                       int experts, float* loss, int32_t* counts, int32_t* tokens)
{
    __shared__ double parts[3][kSumWaves];
    double sum[3] = {0.0, 0.0, (double)live};
    for (int e = threadIdx.x; e < experts; e += kSumThreads) {
        counts[e] = count[e];
        sum[0] += probability[e] * (double)count[e];
        sum[1] += (double)count[e];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int d = kWave / 2; d; d >>= 1) sum[i] += __shfl_xor(sum[i], d);
        if (threadIdx.x % kWave == 0) parts[i][threadIdx.x / kWave] = sum[i];
    }
    __syncthreads();
    if (threadIdx.x) return;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        sum[i] = 0.0;
        for (int w = 0; w < kSumWaves; ++w) sum[i] += parts[i][w];
    }
    *tokens = (int32_t)sum[2];
    // Without choices the sum is 0, without live tokens so is each probability.
    *loss = sum[0] > 0.0 ? (float)(experts * sum[0] / (sum[1] * sum[2])) : 0.0f;
}

// A workgroup's part of the tokens: sums of the probabilities (fp32 over up to 32
// rows a lane, fp64 beyond), counts of the choices and live tokens.  Alone it
// finishes; otherwise its sums go to the workspace.
template <int kDT, int kL, int kC, bool kAlone>
__global__ __launch_bounds__(kSumThreads) void expert_balance_kernel(
    Logits l, const void* __restrict__ choice, int choice_bytes, int top_k, float* loss,
    int32_t* counts, int32_t* tokens, float* sums, int32_t* part_counts, int32_t* part_live,
    int32_t* status)
{
    typedef LogitRow<kDT, kL, kC> R;
    constexpr int kRows = kSumThreads / kL, kMost = kL * R::kV;
    __shared__ double probability[kMost];
    __shared__ double wave_sums[kSumWaves][kMost];
    __shared__ int count[kMost];
    __shared__ int live;
    const int lane = threadIdx.x % kL;
    const int64_t r0 = l.tokens * blockIdx.x / gridDim.x;
    const int64_t r1 = l.tokens * (blockIdx.x + 1) / gridDim.x;
    for (int e = threadIdx.x; e < kMost; e += kSumThreads) count[e] = 0;
    if (threadIdx.x == 0) live = 0;
    __syncthreads();

    for (int64_t i = r0 * top_k + threadIdx.x; i < r1 * top_k; i += kSumThreads) {
        const int64_t c = choice_bytes == 4 ? (int64_t)static_cast<const int32_t*>(choice)[i]
                                            : static_cast<const int64_t*>(choice)[i];
        if ((uint64_t)c < (uint64_t)l.experts)
            atomicAdd(&count[c], 1);
        else if (c != -1)
            report_generic(status, IQ_ERR_INDEX);
    }

    double long_sum[R::kV] = {};
    float sum[R::kV] = {};
    int mine = 0, n = 0;
    for (int64_t row = r0 + threadIdx.x / kL; row < r1; row += kRows) {
        R r;
        r.load(l, row, lane);
        if (r.bad && lane == 0) report_generic(status, IQ_ERR_NONFINITE);
        if (r.live()) {
            float e[R::kV];
            const float inv = 1.0f / r.exps(e);
#pragma unroll
            for (int i = 0; i < R::kV; ++i) sum[i] += e[i] * inv;
            ++mine;
        }
        if (++n % 32 == 0) {
#pragma unroll
            for (int i = 0; i < R::kV; ++i) {
                long_sum[i] += (double)sum[i];
                sum[i] = 0.0f;
            }
        }
    }
    if (lane == 0 && mine) atomicAdd(&live, mine);
#pragma unroll
    for (int i = 0; i < R::kV; ++i) {
        long_sum[i] += (double)sum[i];
#pragma unroll
        for (int d = kL; d < kWave; d <<= 1) long_sum[i] += __shfl_xor(long_sum[i], d);
        if (threadIdx.x % kWave < kL)
            wave_sums[threadIdx.x / kWave][R::expert(lane, i)] = long_sum[i];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < l.experts; e += kSumThreads) {
        double all = 0.0;
#pragma unroll
        for (int i = 0; i < kSumWaves; ++i) all += wave_sums[i][e];
        if constexpr (kAlone) {
            probability[e] = all;
        } else {
            sums[(int64_t)blockIdx.x * l.experts + e] = (float)all;
            part_counts[(int64_t)blockIdx.x * l.experts + e] = count[e];
        }
    }
    if constexpr (kAlone) {
        // A thread reads back what it wrote itself.
        finish(probability, count, threadIdx.x ? 0 : live, l.experts, loss, counts, tokens);
    } else if (threadIdx.x == 0) {
        part_live[blockIdx.x] = live;
    }
}

__global__ __launch_bounds__(kSumThreads) void expert_balance_finish_kernel(
    int experts, int parts, const float* __restrict__ sums, const int32_t* __restrict__ part_counts,
    const int32_t* __restrict__ part_live, float* loss, int32_t* counts, int32_t* tokens)
{
    __shared__ double probability[IQ_MAX_EXPERTS];
    __shared__ int count[IQ_MAX_EXPERTS];
    __shared__ double slice_sums[kSumThreads];
    __shared__ int slice_counts[kSumThreads];
    // Threads beside each other have experts beside each other; slices of threads
    // share the parts.
    const int wide = experts <= 64 ? 64 : (experts <= 128 ? 128 : (experts <= 256 ? 256 : 512));
    const int slices = kSumThreads / wide, slice = threadIdx.x / wide, e = threadIdx.x % wide;
    double sum = 0.0;
    int number = 0, live = 0;
    if (e < experts)
        for (int i = slice; i < parts; i += slices) {
            sum += (double)sums[(int64_t)i * experts + e];
            number += part_counts[(int64_t)i * experts + e];
        }
    for (int i = threadIdx.x; i < parts; i += kSumThreads) live += part_live[i];
    slice_sums[threadIdx.x] = sum;
    slice_counts[threadIdx.x] = number;
    __syncthreads();
    if (threadIdx.x < experts) {
        for (int i = 1; i < slices; ++i) {
            sum += slice_sums[i * wide + e];
            number += slice_counts[i * wide + e];
        }
        probability[e] = sum;
        count[e] = number;
    }
    finish(probability, count, live, experts, loss, counts, tokens);
}

// p (counts_e - sum_j counts_j p_j) E g / (C N) for each row.
template <int kDT, int kL, int kC>
__global__ __launch_bounds__(kThreads) void expert_balance_backward_kernel(
    Logits l, const float* __restrict__ loss_grad, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, void* __restrict__ grad, int64_t ldg)
{
    typedef LogitRow<kDT, kL, kC> R;
    typedef typename R::raw raw;
    const int lane = threadIdx.x % kL;
    float share[R::kV];
    double total = 0.0;
#pragma unroll
    for (int i = 0; i < R::kV; ++i) {
        const int e = R::expert(lane, i);
        const int n = e < l.experts ? counts[e] : 0;
        share[i] = (float)n;
        total += n;
    }
    total = sum_across<kL>(total);
    const int n = *tokens;
    const float scale = total > 0.0 ? (float)(1.0 / total) : 0.0f;
    const float factor = n > 0 ? *loss_grad * (float)l.experts / (float)n : 0.0f;
#pragma unroll
    for (int i = 0; i < R::kV; ++i) share[i] *= scale;

    constexpr int kRows = kThreads / kL;
    for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kL; row < l.tokens;
         row += (int64_t)gridDim.x * kRows) {
        R r;
        r.load(l, row, lane);
        float out[R::kV] = {};
        if (r.live()) {
            const float inv = 1.0f / r.exps(out);
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < R::kV; ++i) {
                out[i] *= inv;
                mean += out[i] * share[i];
            }
            mean = sum_across<kL>(mean);
#pragma unroll
            for (int i = 0; i < R::kV; ++i) out[i] *= (share[i] - mean) * factor;
        }
        raw* to = static_cast<raw*>(grad) + row * ldg;
#pragma unroll
        for (int k = 0; k < kC; ++k) {
            Row<kDT> o;
            o.zero();
#pragma unroll
            for (int i = 0; i < R::kN; ++i) o.set(i, out[k * R::kN + i]);
            o.store(to, R::at(lane, k), l.experts);
        }
    }
}

// How many workgroups share the loss's sums.  The rule sizes the workspace too, so
// it asks nothing of the device.
int balance_parts(int64_t tokens, int experts)
{
    const int64_t rows = experts <= 64 ? 64 : 32;
    return (int)std::min<int64_t>(256, std::max<int64_t>(1, tokens / rows / 4));
}

// body(lanes, vectors) for a number of experts: the lanes of a row and the vectors
// of 16 bytes that each of them has.
template <int kDT, class Body>
hipError_t with_row(int experts, Body&& body)
{
    constexpr int kN = Row<kDT>::kN;
    if (experts <= 32) return body(Int<4>(), Int<8 / kN>());
    if (experts <= 64) return body(Int<8>(), Int<8 / kN>());
    if (experts <= 128) return body(Int<16>(), Int<8 / kN>());
    if (experts <= 256) return body(Int<16>(), Int<16 / kN>());
    return body(Int<32>(), Int<16 / kN>());
}

template <class Body>
hipError_t with_logits(const Logits& l, Body&& body)
{
    return with_dtype(l.dtype, [&](auto dt) {
        return with_row<decltype(dt)::value>(l.experts, [&](auto lanes, auto vectors) {
            return body(dt, lanes, vectors);
        });
    });
}

}  // namespace

hipError_t launch_expert_gate(const Logits& l, int top_k, bool renormalize, int32_t* choice,
                              float* weights, int32_t* status, hipStream_t stream)
{
    return with_logits(l, [&](auto dt, auto lanes, auto vectors) {
        constexpr int kL = decltype(lanes)::value, kRows = kThreads / kL;
        return in_parts((l.tokens + kRows - 1) / kRows, kThreads, [&](int64_t first, dim3 wgs) {
            hipLaunchKernelGGL((expert_gate_kernel<decltype(dt)::value, kL, decltype(vectors)::value>),
                               wgs, dim3(kThreads), 0, stream, l, first, top_k, renormalize, choice,
                               weights, status);
            return hipGetLastError();
        });
    });
}

hipError_t launch_expert_gate_backward(const Logits& l, const float* weights_grad,
                                       const int32_t* choice, const float* weights, int top_k,
                                       bool renormalize, void* grad, int64_t ldg,
                                       hipStream_t stream)
{
    return with_logits(l, [&](auto dt, auto lanes, auto vectors) {
        constexpr int kL = decltype(lanes)::value, kRows = kThreads / kL;
        return in_parts((l.tokens + kRows - 1) / kRows, kThreads, [&](int64_t first, dim3 wgs) {
            hipLaunchKernelGGL((expert_gate_backward_kernel<decltype(dt)::value, kL,
                                                            decltype(vectors)::value>),
                               wgs, dim3(kThreads), 0, stream, l, first, weights_grad, choice,
                               weights, top_k, renormalize, grad, ldg);
            return hipGetLastError();
        });
    });
}

int64_t balance_workspace(int64_t tokens, int experts)
{
    const int64_t parts = balance_parts(tokens, experts);
    return parts > 1 ? parts * (2 * (int64_t)experts + 1) * 4 : 0;
}

hipError_t launch_expert_balance(const Logits& l, const void* choice, int choice_bytes, int top_k,
                                 float* loss, int32_t* counts, int32_t* live, void* workspace,
                                 int32_t* status, hipStream_t stream)
{
    const int parts = balance_parts(l.tokens, l.experts);
    float* sums = static_cast<float*>(workspace);
    int32_t* part_counts = reinterpret_cast<int32_t*>(sums + (int64_t)parts * l.experts);
    int32_t* part_live = part_counts + (int64_t)parts * l.experts;
    const hipError_t e = with_logits(l, [&](auto dt, auto lanes, auto vectors) {
        constexpr int kDT = decltype(dt)::value, kL = decltype(lanes)::value;
        constexpr int kC = decltype(vectors)::value;
        if (parts == 1)
            hipLaunchKernelGGL((expert_balance_kernel<kDT, kL, kC, true>), dim3(1),
                               dim3(kSumThreads), 0, stream, l, choice, choice_bytes, top_k, loss,
                               counts, live, nullptr, nullptr, nullptr, status);
        else
            hipLaunchKernelGGL((expert_balance_kernel<kDT, kL, kC, false>), dim3(parts),
                               dim3(kSumThreads), 0, stream, l, choice, choice_bytes, top_k, loss,
                               counts, live, sums, part_counts, part_live, status);
        return hipGetLastError();
    });
    if (e != hipSuccess || parts == 1) return e;
    hipLaunchKernelGGL(expert_balance_finish_kernel, dim3(1), dim3(kSumThreads), 0, stream,
                       l.experts, parts, sums, part_counts, part_live, loss, counts, live);
    return hipGetLastError();
}

hipError_t launch_expert_balance_backward(const Logits& l, const float* loss_grad,
                                          const int32_t* counts, const int32_t* live, void* grad,
                                          int64_t ldg, hipStream_t stream)
{
    return with_logits(l, [&](auto dt, auto lanes, auto vectors) {
        constexpr int kL = decltype(lanes)::value, kRows = kThreads / kL;
        const int64_t wgs = std::min<int64_t>(2048, (l.tokens + kRows - 1) / kRows);
        hipLaunchKernelGGL((expert_balance_backward_kernel<decltype(dt)::value, kL,
                                                           decltype(vectors)::value>),
                           dim3((unsigned)wgs), dim3(kThreads), 0, stream, l, loss_grad, counts,
                           live, grad, ldg);
        return hipGetLastError();
    });
}

}  // namespace iqk

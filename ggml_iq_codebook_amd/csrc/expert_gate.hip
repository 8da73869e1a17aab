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
//
// The gate takes k turns of a maximum over the row and the lowest index that has it:
// bound by latency for few tokens (4 x 64 fp32, 8 chosen: 3.3 us), by instruction issue
// for many (131072 x 64: 18 us, its bytes 8).  Its gradient and the loss's are a pass
// over the logits (16384 x 64: 5.8 us; 65536 x 256: 23 us, 5.8 TB/s with what the
// last level of caches holds).  The loss's forward pass keeps a column's sum in the lanes
// that have it and asks for the next row while it works on one (65536 x 256: 20.4 us,
// 3.3 TB/s, bound by its exponentials and sums, and by LDS, where the counts by atomics
// and the waves' columns meet on banks in 40 % of its active cycles).
#include <hip/hip_runtime.h>

#include <algorithm>

#include "iq_router.h"
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

constexpr int kThreads = 256;
constexpr float kNone = -__builtin_inff();

// v of the lanes of the other 16 of 32 (kDistance 16) or the other 32 (32): both, of this
// half and of the other, in an order that is the same for all lanes.
template <int kDistance>
__device__ __forceinline__ void both_halves(uint32_t v, uint32_t (&half)[2])
{
    typedef uint32_t v2u __attribute__((ext_vector_type(2)));
    const v2u swapped = __builtin_bit_cast(
        v2u, kDistance == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                             : __builtin_amdgcn_permlane32_swap(v, v, false, false));
    half[0] = swapped[0];
    half[1] = swapped[1];
}
template <int kDistance, class T, class Op>
__device__ __forceinline__ T halves(T v, Op&& op)
{
    static_assert(sizeof(T) == 4 || sizeof(T) == 8, "one or two registers");
    uint32_t u[sizeof(T) / 4], low[2], high[2] = {};
    __builtin_memcpy(u, &v, sizeof(T));
    both_halves<kDistance>(u[0], low);
    if constexpr (sizeof(T) == 8) both_halves<kDistance>(u[1], high);
    T half[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        u[0] = low[i];
        if constexpr (sizeof(T) == 8) u[1] = high[i];
        __builtin_memcpy(&half[i], u, sizeof(T));
    }
    return op(half[0], half[1]);
}

// op over the kL lanes of a row (64: a wave), the same result in all of them.
template <int kL, class T, class Op>
__device__ __forceinline__ T across(T v, Op&& op)
{
    if constexpr (kL > 1) v = op(v, quad_xchg<kQuadXor1>(v));
    if constexpr (kL > 2) v = op(v, quad_xchg<kQuadXor2>(v));
    if constexpr (kL > 4) v = op(v, quad_xchg<0x141>(v));     // lane 7 - i of 8
    if constexpr (kL > 8) v = op(v, quad_xchg<0x140>(v));     // lane 15 - i of 16
    if constexpr (kL > 16) v = halves<16>(v, op);
    if constexpr (kL > 32) v = halves<32>(v, op);
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

// The sum over the rows of a wave, kL lanes each, of what their lanes of one place have.
template <int kL, class T>
__device__ __forceinline__ T sum_rows(T v)
{
    const auto add = [](T a, T b) { return a + b; };
    if constexpr (kL <= 4) v = v + quad_xchg<0x124>(v);       // the lane 4 before, of 16
    if constexpr (kL <= 8) v = v + quad_xchg<0x128>(v);       // the lane 8 before, of 16
    if constexpr (kL <= 16) v = halves<16>(v, add);
    return halves<32>(v, add);
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
    // The row as it is stored, to be asked for ahead.
    struct Stored {
        Row<kDT> r[kC];
        __device__ __forceinline__ void load(const Logits& l, int64_t row, int lane)
        {
            const raw* from = static_cast<const raw*>(l.p) + row * l.ld;
#pragma unroll
            for (int c = 0; c < kC; ++c) r[c].load(from, at(lane, c), l.experts);
        }
    };
    __device__ __forceinline__ void load(const Logits& l, int64_t row, int lane)
    {
        Stored stored;
        stored.load(l, row, lane);
        take(l, stored, lane);
    }
    __device__ __forceinline__ void take(const Logits& l, const Stored& stored, int lane)
    {
        int wrong = 0;
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            v[i] = stored.r[i / kN][i % kN];
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

constexpr int kSumThreads = 1024, kSumWaves = kSumThreads / kWave;

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
        sum[i] = sum_across<kWave>(sum[i]);
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
// finishes; otherwise its sums go to the workspace, rounded to fp32 (2^-24 of a sum of
// positive terms, no more than the probabilities themselves are off, for half of the
// bytes that the finishing workgroups wait for) and added up in fp64 there.
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
    typename R::Stored next;
    if (r0 + threadIdx.x / kL < r1) next.load(l, r0 + threadIdx.x / kL, lane);
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
        r.take(l, next, lane);
        if (row + kRows < r1) next.load(l, row + kRows, lane);
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
        long_sum[i] = sum_rows<kL>(long_sum[i] + (double)sum[i]);
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

// The parts' sums added up.  A workgroup has 16 experts, so that what the parts left,
// which comes from beyond the L2, comes to many compute units; with more than one
// workgroup their shares of the loss are added by the kernel below.
constexpr int kFinishExperts = 16, kFinishThreads = 256;
constexpr int kFinishSlices = kFinishThreads / kFinishExperts;

struct Share {
    double dot, total;                // sum of probability * count, and of counts
};

__device__ __forceinline__ void write_loss(Share s, int live, int experts, float* loss, int32_t* tokens)
{
    *tokens = live;
    *loss = s.dot > 0.0 ? (float)(experts * s.dot / (s.total * live)) : 0.0f;
}

// The live tokens of all parts, in every lane of a wave.
__device__ __forceinline__ int live_tokens(const int32_t* part_live, int parts)
{
    int live = 0;
    for (int i = threadIdx.x % kWave; i < parts; i += kWave) live += part_live[i];
    return sum_across<kWave>(live);
}

__global__ __launch_bounds__(kFinishThreads) void expert_balance_finish_kernel(
    int experts, int parts, const float* __restrict__ sums, const int32_t* __restrict__ part_counts,
    const int32_t* __restrict__ part_live, float* loss, int32_t* counts, int32_t* tokens,
    Share* shares)
{
    __shared__ double slice_sums[kFinishSlices][kFinishExperts];
    __shared__ int slice_counts[kFinishSlices][kFinishExperts];
    const int slice = threadIdx.x / kFinishExperts, at = threadIdx.x % kFinishExperts;
    const int e = blockIdx.x * kFinishExperts + at;
    double sum = 0.0;
    int number = 0;
    if (e < experts) {
#pragma unroll 8
        for (int i = slice; i < parts; i += kFinishSlices) {
            sum += (double)sums[(int64_t)i * experts + e];
            number += part_counts[(int64_t)i * experts + e];
        }
    }
    slice_sums[slice][at] = sum;
    slice_counts[slice][at] = number;
    __syncthreads();
    if (threadIdx.x >= kWave) return;
    Share share = {0.0, 0.0};
    if (threadIdx.x < kFinishExperts && e < experts) {
        sum = 0.0;
        number = 0;
#pragma unroll
        for (int i = 0; i < kFinishSlices; ++i) {
            sum += slice_sums[i][at];
            number += slice_counts[i][at];
        }
        counts[e] = number;
        share = {sum * (double)number, (double)number};
    }
    share.dot = sum_across<kFinishExperts>(share.dot);
    share.total = sum_across<kFinishExperts>(share.total);
    if (gridDim.x > 1) {
        if (threadIdx.x == 0) shares[blockIdx.x] = share;
        return;
    }
    const int live = live_tokens(part_live, parts);
    if (threadIdx.x == 0) write_loss(share, live, experts, loss, tokens);
}

__global__ __launch_bounds__(kWave) void expert_balance_loss_kernel(
    int experts, int parts, const Share* __restrict__ shares, const int32_t* __restrict__ part_live,
    float* loss, int32_t* tokens)
{
    static_assert(IQ_MAX_EXPERTS / kFinishExperts <= kWave, "a lane for every workgroup");
    const int workgroups = (experts + kFinishExperts - 1) / kFinishExperts;
    Share share = {0.0, 0.0};
    if ((int)threadIdx.x < workgroups) share = shares[threadIdx.x];
    share.dot = sum_across<kWave>(share.dot);
    share.total = sum_across<kWave>(share.total);
    const int live = live_tokens(part_live, parts);
    if (threadIdx.x == 0) write_loss(share, live, experts, loss, tokens);
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

// The lanes of a row, as above.
int row_lanes(int experts)
{
    return experts <= 32 ? 4 : (experts <= 64 ? 8 : (experts <= 256 ? 16 : 32));
}

// How many workgroups share the loss's sums: alone what they take at once, otherwise at
// most one for every compute unit of a whole card.  (The rule sizes the workspace too, so
// it asks nothing of the device.)
int balance_parts(int64_t tokens, int experts)
{
    const int64_t rows = kSumThreads / row_lanes(experts);
    return (int)std::min<int64_t>(256, std::max<int64_t>(1, (tokens + rows - 1) / rows));
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

constexpr int64_t kShareBytes = IQ_MAX_EXPERTS / kFinishExperts * (int64_t)sizeof(Share);

int64_t balance_workspace(int64_t tokens, int experts)
{
    const int64_t parts = balance_parts(tokens, experts);
    // The shares of the loss first, then the parts' sums, counts and live tokens.
    return parts > 1 ? kShareBytes + parts * (2 * (int64_t)experts + 1) * 4 : 0;
}

hipError_t launch_expert_balance(const Logits& l, const void* choice, int choice_bytes, int top_k,
                                 float* loss, int32_t* counts, int32_t* live, void* workspace,
                                 int32_t* status, hipStream_t stream)
{
    const int parts = balance_parts(l.tokens, l.experts);
    Share* shares = static_cast<Share*>(workspace);
    float* sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + kShareBytes);
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
    const int wgs = (l.experts + kFinishExperts - 1) / kFinishExperts;
    hipLaunchKernelGGL(expert_balance_finish_kernel, dim3(wgs), dim3(kFinishThreads), 0, stream,
                       l.experts, parts, sums, part_counts, part_live, loss, counts, live, shares);
    const hipError_t f = hipGetLastError();
    if (f != hipSuccess || wgs == 1) return f;
    hipLaunchKernelGGL(expert_balance_loss_kernel, dim3(1), dim3(kWave), 0, stream, l.experts, parts,
                       shares, part_live, loss, live);
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

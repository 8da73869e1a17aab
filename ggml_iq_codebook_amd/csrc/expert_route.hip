// expert_route.hip -- tokens sorted by expert, copied there and brought back
// with the router's weights, and the gradients of both copies.
//
// The sort is a stable counting sort: counts per expert and chunk of choices,
// their sums, then each choice's rank among the equal ones before it.  Nothing
// depends on the order of atomics: they only add counts.  Dropped choices (-1)
// count as one more expert behind the last, so `position` is a permutation of
// all choices and every row of a sorted tensor has exactly one writer.
//
// Bound by latency: 1024 choices of 16 experts 3.7 us, 32768 of 64 experts 8.7 us
// in two launches.
//
// The copies are bound by HBM.  They go token by token: a token's row is read
// once for all its choices (dispatch), or its choices' rows are read and
// summed in registers (combine), 16 bytes a lane, with no intermediate tensor
// and no atomics.  4096 tokens of 4096 bf16 values with 8 choices each: dispatch
// 52 us (5.8 TB/s), combine 56 us and the gradient of dispatch 55 us (5.4 TB/s),
// the gradients of combine 110 us (5.2 TB/s).
#include <hip/hip_runtime.h>

#include "iq_layers.h"
#include "layers_common.hpp"
#include "layers_launch.hpp"

namespace iqk {
namespace {

// ---------------------------------------------------------------------------
// The sort
// ---------------------------------------------------------------------------

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / kWave;
constexpr int kMaxKeys = IQ_MAX_EXPERTS + 1;
static_assert(kMaxKeys <= kSortThreads, "a thread per key");
constexpr int kKeptSteps = 4;         // steps of 64 choices a wave keeps in registers
constexpr int64_t kAloneChoices = (int64_t)kKeptSteps * kSortThreads;
constexpr int kMaxChunks = 256;

// The choice at place i as a key 0..experts, experts where it is dropped.
template <class Choice>
__device__ __forceinline__ int key_of(const Choice* choice, int64_t i, int experts, bool* bad)
{
    const Choice c = choice[i];
    if (c >= 0 && c < (Choice)experts) return (int)c;
    *bad = *bad || c != (Choice)-1;
    return experts;
}

// Counts of a chunk's keys.
template <class Choice>
__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(
    const Choice* __restrict__ choice, int64_t n, int64_t per_chunk, int experts,
    int32_t* __restrict__ counts)
{
    __shared__ int32_t count[kMaxKeys];
    for (int e = threadIdx.x; e <= experts; e += kSortThreads) count[e] = 0;
    __syncthreads();
    const int64_t first = blockIdx.x * per_chunk;
    const int64_t last = min(first + per_chunk, n);
    bool bad = false;
    for (int64_t i = first + threadIdx.x; i < last; i += kSortThreads)
        atomicAdd(&count[key_of(choice, i, experts, &bad)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= experts; e += kSortThreads)
        counts[(int64_t)blockIdx.x * (experts + 1) + e] = count[e];
}

// The lanes of a wave that hold the same key (of the live ones), found bit by
// bit.
__device__ __forceinline__ uint64_t same_key(int key, bool live, int bits)
{
    uint64_t same = __ballot(live);
    for (int b = 0; b < bits; ++b) {
        const uint64_t set = __ballot((key >> b) & 1);
        same &= ((key >> b) & 1) ? set : ~set;
    }
    return same;
}

// Places a chunk's choices.  Each wave takes a consecutive part of the chunk,
// so the ranks follow the order of the choices: chunk, wave, step of 64, lane.
// A wave first ranks each choice among the equal ones of its own part, in a row
// of counters of its own; what the keys, chunks and waves before it hold is
// added afterwards.  kKept: the part is at most kKeptSteps steps, and keys and
// ranks stay in registers in between; otherwise they are found again.
template <class Choice, bool kKept>
__global__ __launch_bounds__(kSortThreads) void expert_place_kernel(
    const Choice* __restrict__ choice, int64_t n, int64_t per_chunk, int experts,
    const int32_t* __restrict__ counts, int32_t* __restrict__ order,
    int32_t* __restrict__ position, int32_t* __restrict__ offsets, int32_t* status)
{
    extern __shared__ int32_t shared[];
    const int keys = experts + 1;
    int32_t* before = shared;                     // [waves][keys]: counters, then first places
    int32_t* total = shared + kSortWaves * keys;  // [keys]: over all chunks
    int32_t* start = total + keys;                // [keys]: of the chunks before this one
    __shared__ int32_t wave_sums[kSortWaves];
    const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
    const int64_t first = blockIdx.x * per_chunk;
    const int64_t last = min(first + per_chunk, n);
    const int64_t per_wave = ((per_chunk + kSortThreads - 1) / kSortThreads) * kWave;
    const int64_t wfirst = first + wave * per_wave;
    const int64_t wlast = min(wfirst + per_wave, last);
    const int steps = wlast > wfirst ? (int)((wlast - wfirst + kWave - 1) / kWave) : 0;
    const uint64_t below = (1ull << lane) - 1ull;
    int bits = 0;
    while ((1 << bits) < keys) ++bits;

    int key[kKeptSteps], rank[kKeptSteps];
    bool bad = false;
    if (kKept) {
#pragma unroll
        for (int s = 0; s < kKeptSteps; ++s) {
            const int64_t i = wfirst + s * kWave + lane;
            key[s] = i < wlast ? key_of(choice, i, experts, &bad) : -1;
        }
    }
    for (int i = threadIdx.x; i < (kSortWaves + 2) * keys; i += kSortThreads) shared[i] = 0;
    __syncthreads();

    // One step's rank among the wave's earlier choices of the same key.  All
    // lanes read a counter before its first lane advances it: a wave's LDS
    // accesses are done in order.
    int32_t* mine = before + wave * keys;
    auto rank_of = [&](int k, bool live) {
        const uint64_t same = same_key(k, live, bits);
        const int32_t base = live ? mine[k] : 0;
        const int32_t r = __popcll(same & below);
        __builtin_amdgcn_wave_barrier();
        if (live && r == 0) mine[k] = base + __popcll(same);
        __builtin_amdgcn_wave_barrier();
        return base + r;
    };
    if (kKept) {
#pragma unroll
        for (int s = 0; s < kKeptSteps; ++s)
            if (s < steps) rank[s] = rank_of(max(key[s], 0), key[s] >= 0);
    } else {
        for (int s = 0; s < steps; ++s) {
            const int64_t i = wfirst + (int64_t)s * kWave + lane;
            const bool live = i < wlast;
            rank_of(live ? key_of(choice, i, experts, &bad) : 0, live);
        }
    }
    if (bad) report_generic(status, IQ_ERR_INDEX);
    // The other chunks' counts: several threads a key, each over some chunks.
    if (gridDim.x > 1) {
        const int groups = kSortThreads / keys;
        const int group = threadIdx.x / keys, e = threadIdx.x % keys;
        if (group < groups) {
            int32_t all = 0, prior = 0;
            for (int c = group; c < (int)gridDim.x; c += groups) {
                const int32_t v = counts[(int64_t)c * keys + e];
                all += v;
                prior += c < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&start[e], prior);
        }
    }
    __syncthreads();
    // First place of each key: the sum over the keys before it.
    {
        const int e = threadIdx.x;
        int32_t held[kSortWaves], here = 0;
        if (e < keys) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                held[w] = before[w * keys + e];
                here += held[w];
            }
        }
        const int32_t all = e < keys ? (gridDim.x > 1 ? total[e] : here) : 0;
        int32_t sum = all;
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int32_t up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        if (lane == kWave - 1) wave_sums[wave] = sum;
        __syncthreads();
        if (e < keys) {
            int32_t next = sum - all;
            for (int w = 0; w < wave; ++w) next += wave_sums[w];
            if (blockIdx.x == 0) offsets[e] = next;
            // and of this chunk's waves
            next += start[e];
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) {
                before[w * keys + e] = next;
                next += held[w];
            }
        }
        __syncthreads();
    }
    if (kKept) {
#pragma unroll
        for (int s = 0; s < kKeptSteps; ++s)
            if (key[s] >= 0) {
                const int64_t i = wfirst + s * kWave + lane;
                const int32_t place = mine[key[s]] + rank[s];
                position[i] = place;
                order[place] = (int32_t)i;
            }
    } else {
        for (int s = 0; s < steps; ++s) {
            const int64_t i = wfirst + (int64_t)s * kWave + lane;
            const bool live = i < wlast;
            const int32_t place = rank_of(live ? key_of(choice, i, experts, &bad) : 0, live);
            if (live) {
                position[i] = place;
                order[place] = (int32_t)i;
            }
        }
    }
}

__global__ void no_choices_kernel(int32_t* offsets, int keys)
{
    for (int e = threadIdx.x; e < keys; e += blockDim.x) offsets[e] = 0;
}

// ---------------------------------------------------------------------------
// The copies
// ---------------------------------------------------------------------------

constexpr int kThreads = 256;

// A row is shared by `lanes` threads (a power of two), 16 bytes a lane.

// The place of a token's choice: -1 outside the sorted rows (skipped).
__device__ __forceinline__ int64_t place_of(const Route& r, int64_t token, int j)
{
    const int32_t p = r.position[token * r.top_k + j];
    return p >= 0 && p < r.rows ? p : -1;
}

// This thread's token.  Where a row is shared by whole waves the token is the
// same for all of a wave's lanes, and its places and weights are read as
// scalars, all at once, ahead of the rows.
template <bool kWaves>
__device__ __forceinline__ int64_t token_of(int lanes)
{
    const int in_block = threadIdx.x / lanes;
    return (int64_t)blockIdx.x * (kThreads / lanes) +
           (kWaves ? __builtin_amdgcn_readfirstlane(in_block) : in_block);
}

template <int kDT, bool kWaves, bool kStreaming>
__global__ __launch_bounds__(kThreads) void expert_dispatch_kernel(Route r,
                                                                   const void* __restrict__ x,
                                                                   int64_t ldx,
                                                                   void* __restrict__ sorted,
                                                                   int64_t lds, int lanes)
{
    typedef typename Value<kDT>::raw raw;
    const int64_t token = token_of<kWaves>(lanes);
    if (token >= r.tokens) return;
    const int64_t kept = *r.kept;
    const raw* xr = static_cast<const raw*>(x) + token * ldx;
    for (int64_t at = (int64_t)(threadIdx.x % lanes) * Row<kDT>::kN; at < r.width;
         at += (int64_t)lanes * Row<kDT>::kN) {
        Row<kDT> v, none;
        v.load(xr, at, r.width);
        none.zero();
        for (int j = 0; j < r.top_k; ++j) {
            const int64_t p = place_of(r, token, j);
            if (p < 0) continue;
            raw* to = static_cast<raw*>(sorted) + p * lds;
            if (p < kept)
                v.template store<kStreaming>(to, at, r.width);
            else
                none.template store<kStreaming>(to, at, r.width);
        }
    }
}

// kGroup choices of a token: their places, weights and which of them count.
// `row` is a place that is there in any case (0 where the choice's is not), so
// that rows are loaded without branches between the loads; what the row of a
// choice that does not count holds is left out of every sum.
template <int kGroup>
struct Choices {
    int64_t place[kGroup];
    int64_t row[kGroup];
    float weight[kGroup];
    bool live[kGroup];
    __device__ __forceinline__ Choices(const Route& r, int64_t token, int j0, int64_t kept,
                                       const float* weights)
    {
        int32_t p[kGroup];
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
            const int64_t c = token * r.top_k + min(j0 + g, r.top_k - 1);
            p[g] = r.position[c];
            weight[g] = weights ? weights[c] : 1.0f;
        }
#pragma unroll
        for (int g = 0; g < kGroup; ++g) {
            const bool there = (j0 + g < r.top_k) & (p[g] >= 0) & (p[g] < r.rows);
            place[g] = there ? p[g] : -1;
            live[g] = there & (p[g] < kept);
            row[g] = live[g] ? p[g] : 0;
        }
    }
};

// kWeighted: combine; otherwise the gradient of dispatch.  The rows of kGroup
// choices are on their way at once; the sum keeps the order of the choices.
// Bound by HBM's reads: a row is read once, without keeping it in the caches.
template <int kDT, bool kWeighted, int kGroup, bool kWaves>
__global__ __launch_bounds__(kThreads) void expert_combine_kernel(Route r,
                                                                  const void* __restrict__ y,
                                                                  int64_t ldy,
                                                                  const float* __restrict__ weights,
                                                                  void* __restrict__ out,
                                                                  int64_t ldo, int lanes)
{
    typedef typename Value<kDT>::raw raw;
    constexpr int kN = Row<kDT>::kN;
    const int64_t token = token_of<kWaves>(lanes);
    if (token >= r.tokens) return;
    const int64_t kept = *r.kept;
    raw* to = static_cast<raw*>(out) + token * ldo;
    const int64_t first = (int64_t)(threadIdx.x % lanes) * kN, step = (int64_t)lanes * kN;
    for (int64_t at = first; at < r.width; at += step) {
        float sum[kN] = {};
        for (int j0 = 0; j0 < r.top_k; j0 += kGroup) {
            const Choices<kGroup> c(r, token, j0, kept, kWeighted ? weights : nullptr);
            if (at + kN <= r.width) {
                Row<kDT> v[kGroup];
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    v[g].load_once(static_cast<const raw*>(y) + c.row[g] * ldy + at);
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    if (c.live[g]) {
#pragma unroll
                        for (int i = 0; i < kN; ++i)
                            sum[i] += kWeighted ? c.weight[g] * v[g][i] : v[g][i];
                    }
            } else {
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    if (c.live[g]) {
                        Row<kDT> v;
                        v.load(static_cast<const raw*>(y) + c.row[g] * ldy, at, r.width);
#pragma unroll
                        for (int i = 0; i < kN; ++i)
                            sum[i] += kWeighted ? c.weight[g] * v[i] : v[i];
                    }
            }
        }
        Row<kDT> o;
        o.zero();
#pragma unroll
        for (int i = 0; i < kN; ++i) o.set(i, sum[i]);
        o.store(to, at, r.width);
    }
}

// A token's gradient is scaled into the rows of its choices, and multiplied
// with what those rows held, kGroup choices at a time.  kLanes: a wave or the
// workgroup shares a token.
template <int kDT, int kLanes, bool kStreaming>
__global__ __launch_bounds__(kThreads) void expert_combine_backward_kernel(
    Route r, const void* __restrict__ out_grad, int64_t ldo, const void* __restrict__ y,
    int64_t ldy, const float* __restrict__ weights, void* __restrict__ y_grad, int64_t ldg,
    float* __restrict__ weights_grad)
{
    typedef typename Value<kDT>::raw raw;
    constexpr int kGroup = 4, kN = Row<kDT>::kN;
    __shared__ float parts[kThreads / kWave][kGroup];
    const int64_t token = token_of<true>(kLanes);
    // Tokens beyond the last only occur where a token is a wave's: no barrier then.
    if (token >= r.tokens) return;
    const int lane = threadIdx.x % kLanes;
    const int64_t kept = *r.kept;
    const raw* gr = static_cast<const raw*>(out_grad) + token * ldo;
    for (int j0 = 0; j0 < r.top_k; j0 += kGroup) {
        const Choices<kGroup> c(r, token, j0, kept, weights);
        float dot[kGroup] = {};
        for (int64_t at = (int64_t)lane * kN; at < r.width; at += (int64_t)kLanes * kN) {
            // One choice's part, from its row's vector.
            auto part = [&](int g, const Row<kDT>& grad, const Row<kDT>& v) {
                Row<kDT> d;
                d.zero();
                if (c.live[g]) {
#pragma unroll
                    for (int i = 0; i < kN; ++i) {
                        dot[g] += grad[i] * v[i];
                        d.set(i, c.weight[g] * grad[i]);
                    }
                }
                if (c.place[g] >= 0)
                    d.template store<kStreaming>(static_cast<raw*>(y_grad) + c.place[g] * ldg, at,
                                                 r.width);
            };
            Row<kDT> grad;
            grad.load(gr, at, r.width);
            if (at + kN <= r.width) {
                Row<kDT> v[kGroup];
#pragma unroll
                for (int g = 0; g < kGroup; ++g)
                    v[g].load_once(static_cast<const raw*>(y) + c.row[g] * ldy + at);
#pragma unroll
                for (int g = 0; g < kGroup; ++g) part(g, grad, v[g]);
            } else {
#pragma unroll
                for (int g = 0; g < kGroup; ++g) {
                    Row<kDT> v;
                    v.zero();
                    if (c.live[g])
                        v.load(static_cast<const raw*>(y) + c.row[g] * ldy, at, r.width);
                    part(g, grad, v);
                }
            }
        }
#pragma unroll
        for (int g = 0; g < kGroup; ++g)
#pragma unroll
            for (int d = kWave / 2; d; d >>= 1) dot[g] += __shfl_xor(dot[g], d);
        if (kLanes > kWave) {
            if (threadIdx.x % kWave == 0) {
#pragma unroll
                for (int g = 0; g < kGroup; ++g) parts[threadIdx.x / kWave][g] = dot[g];
            }
            __syncthreads();
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                dot[g] = parts[0][g];
#pragma unroll
                for (int i = 1; i < kThreads / kWave; ++i) dot[g] += parts[i][g];
            }
            __syncthreads();
        }
        if (lane == 0) {
#pragma unroll
            for (int g = 0; g < kGroup; ++g)
                if (j0 + g < r.top_k) weights_grad[token * r.top_k + j0 + g] = dot[g];
        }
    }
}

int lanes_for(int64_t width, int values)
{
    int lanes = 16;
    while (lanes < kThreads && (int64_t)lanes * values < width) lanes *= 2;
    return lanes;
}

// launch(the tokens from `token` on, token, workgroups) for each part of a launch
// that gives a token to `lanes` threads.
template <class Launch>
hipError_t by_tokens(const Route& r, int lanes, Launch&& launch)
{
    const int each = kThreads / lanes;
    return in_parts((r.tokens + each - 1) / each, kThreads, [&](int64_t first, dim3 wgs) {
        const int64_t token = first * each;
        Route part = r;
        part.tokens -= token;
        part.position += token * r.top_k;
        launch(part, token, wgs);
        return hipGetLastError();
    });
}

}  // namespace

// One workgroup while a wave's part fits its registers; beyond, a workgroup per
// 1024 choices, or more where that would be over 256 of them.
SortPlan expert_sort_plan(int64_t n)
{
    SortPlan s;
    s.per_chunk = n <= kAloneChoices ? kAloneChoices : kSortThreads;
    if ((n + s.per_chunk - 1) / s.per_chunk > kMaxChunks)
        s.per_chunk = ((n + kMaxChunks - 1) / kMaxChunks + kSortThreads - 1) / kSortThreads *
                      kSortThreads;
    s.chunks = (int)((n + s.per_chunk - 1) / s.per_chunk);
    if (s.chunks <= 1) s.per_chunk = (n + kSortThreads - 1) / kSortThreads * kSortThreads;
    return s;
}

template <class Choice, bool kKept>
static void place_as(const SortPlan& s, const Choice* choice, int64_t n, int experts,
                     int32_t* order, int32_t* position, int32_t* offsets, int32_t* counts,
                     int32_t* status, hipStream_t stream)
{
    const size_t lds = sizeof(int32_t) * (kSortWaves + 2) * (experts + 1);
    hipLaunchKernelGGL((expert_place_kernel<Choice, kKept>), dim3(s.chunks), dim3(kSortThreads),
                       lds, stream, choice, n, s.per_chunk, experts, counts, order, position,
                       offsets, status);
}

template <class Choice>
static hipError_t sort_as(const void* choice, int64_t n, int experts, int32_t* order,
                          int32_t* position, int32_t* offsets, int32_t* counts, int32_t* status,
                          hipStream_t stream)
{
    const SortPlan s = expert_sort_plan(n);
    const Choice* c = static_cast<const Choice*>(choice);
    if (s.chunks > 1)
        hipLaunchKernelGGL((expert_count_kernel<Choice>), dim3(s.chunks), dim3(kSortThreads), 0,
                           stream, c, n, s.per_chunk, experts, counts);
    if (s.per_chunk <= kAloneChoices)
        place_as<Choice, true>(s, c, n, experts, order, position, offsets, counts, status, stream);
    else
        place_as<Choice, false>(s, c, n, experts, order, position, offsets, counts, status, stream);
    return hipGetLastError();
}

hipError_t launch_expert_sort(const void* choice, int choice_bytes, int64_t n, int experts,
                              int32_t* order, int32_t* position, int32_t* offsets,
                              int32_t* counts, int32_t* status, hipStream_t stream)
{
    if (n == 0) {
        hipLaunchKernelGGL(no_choices_kernel, dim3(1), dim3(kThreads), 0, stream, offsets,
                           experts + 1);
        return hipGetLastError();
    }
    return choice_bytes == 8 ? sort_as<int64_t>(choice, n, experts, order, position, offsets,
                                                counts, status, stream)
                             : sort_as<int32_t>(choice, n, experts, order, position, offsets,
                                                counts, status, stream);
}

hipError_t launch_expert_dispatch(int dtype, const Route& r, const void* x, int64_t ldx,
                                  void* sorted, int64_t lds, hipStream_t stream)
{
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        const int lanes = lanes_for(r.width, Row<kDT>::kN);
        const auto kernel = lanes < kWave ? (r.streaming ? expert_dispatch_kernel<kDT, false, true>
                                                         : expert_dispatch_kernel<kDT, false, false>)
                                          : (r.streaming ? expert_dispatch_kernel<kDT, true, true>
                                                         : expert_dispatch_kernel<kDT, true, false>);
        return by_tokens(r, lanes, [&](const Route& part, int64_t token, dim3 wgs) {
            hipLaunchKernelGGL(kernel, wgs, dim3(kThreads), 0, stream, part,
                               static_cast<const typename Value<kDT>::raw*>(x) + token * ldx, ldx,
                               sorted, lds, lanes);
        });
    });
}

template <int kDT, bool kWeighted, int kGroup, bool kWaves>
static hipError_t combine_as(const Route& r, const void* y, int64_t ldy, const float* weights,
                             void* out, int64_t ldo, int lanes, hipStream_t stream)
{
    return by_tokens(r, lanes, [&](const Route& part, int64_t token, dim3 wgs) {
        hipLaunchKernelGGL((expert_combine_kernel<kDT, kWeighted, kGroup, kWaves>), wgs,
                           dim3(kThreads), 0, stream, part, y, ldy,
                           kWeighted ? weights + token * r.top_k : nullptr,
                           static_cast<typename Value<kDT>::raw*>(out) + token * ldo, ldo, lanes);
    });
}

// As many rows at once as there are choices, 2, 4 or 8; 4 where lanes of a wave
// work on different tokens.
template <int kDT, bool kWeighted>
static hipError_t combine_with(const Route& r, const void* y, int64_t ldy, const float* weights,
                               void* out, int64_t ldo, hipStream_t stream)
{
    const int lanes = lanes_for(r.width, Row<kDT>::kN);
    if (lanes < kWave)
        return combine_as<kDT, kWeighted, 4, false>(r, y, ldy, weights, out, ldo, lanes, stream);
    if (r.top_k <= 2)
        return combine_as<kDT, kWeighted, 2, true>(r, y, ldy, weights, out, ldo, lanes, stream);
    if (r.top_k <= 4)
        return combine_as<kDT, kWeighted, 4, true>(r, y, ldy, weights, out, ldo, lanes, stream);
    return combine_as<kDT, kWeighted, 8, true>(r, y, ldy, weights, out, ldo, lanes, stream);
}

hipError_t launch_expert_combine(int dtype, const Route& r, const void* y, int64_t ldy,
                                 const float* weights, void* out, int64_t ldo, hipStream_t stream)
{
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        return weights ? combine_with<kDT, true>(r, y, ldy, weights, out, ldo, stream)
                       : combine_with<kDT, false>(r, y, ldy, weights, out, ldo, stream);
    });
}

hipError_t launch_expert_combine_backward(int dtype, const Route& r, const void* out_grad,
                                          int64_t ldo, const void* y, int64_t ldy,
                                          const float* weights, void* y_grad, int64_t ldg,
                                          float* weights_grad, hipStream_t stream)
{
    return with_dtype(dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        // Two vectors a lane of a wave at most, else the workgroup.
        const bool by_wave = r.width <= 2 * kWave * Row<kDT>::kN;
        const auto kernel =
            by_wave ? (r.streaming ? expert_combine_backward_kernel<kDT, kWave, true>
                                   : expert_combine_backward_kernel<kDT, kWave, false>)
                    : (r.streaming ? expert_combine_backward_kernel<kDT, kThreads, true>
                                   : expert_combine_backward_kernel<kDT, kThreads, false>);
        return by_tokens(r, by_wave ? kWave : kThreads,
                         [&](const Route& part, int64_t token, dim3 wgs) {
            hipLaunchKernelGGL(kernel, wgs, dim3(kThreads), 0, stream, part,
                               static_cast<const typename Value<kDT>::raw*>(out_grad) + token * ldo,
                               ldo, y, ldy, weights + token * r.top_k, y_grad, ldg,
                               weights_grad + token * r.top_k);
        });
    });
}

}  // namespace iqk

// fp4_linear.hip -- products with 4-bit weights whose groups of 32 share a power
// of two, dense or with a weight per expert:
//   y[t][n] = sum_k x[t][k] * value(w[n][k]).
//
// The weight's values are exact in bf16, so the matrix cores take them as they
// are.  bf16 activations are an operand as they come; fp32 ones are split into
// three bf16 parts (v = hi + mid + lo exactly), each multiplied in turn.  fp16
// activations are an operand of fp16 products while the weight's scales are in
// fp16's range, 2^-23 .. 2^13, and split into two bf16 parts where one is not.
// Every product is exact that way, and only the fp32 sums and the one rounding of
// the result differ from the formula.  (The parts of fp32 values below 2^-110 reach
// below bf16's smallest number, 2^-133, and are cut there.)  Where a scale reaches
// beyond fp32, what was summed up in several parts is summed up again with care.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "expert_tiles.hpp"
#include "fp4_common.hpp"
#include "fp4_sizes.hpp"
#include "layers_launch.hpp"
#include "row_codes.hpp"

namespace iqk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

constexpr int kPiece = 128;           // depth of a step: four groups, 64 bytes of codes a row

__device__ __forceinline__ v4f mfma16(v8bf a, v8bf b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 16 bytes at any alignment.
__device__ __forceinline__ v4u load16(const uint8_t* from)
{
    v4u v;
    __builtin_memcpy(&v, from, 16);
    return v;
}

__device__ __forceinline__ v4f mfma16(v8h a, v8h b, v4f c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Parts in which activations wait in LDS: fp32 is split on the way there, the others
// come as they are.
template <int kDT>
constexpr int kStaged = kDT == IQ_DTYPE_F32 ? 3 : 1;

// bf16 parts that a type is split into.
template <int kDT>
constexpr int kSplit = kDT == IQ_DTYPE_BF16 ? 1 : (kDT == IQ_DTYPE_F16 ? 2 : 3);

// 8 activations as operands.  hi is v cut to 8 significant bits, mid what is
// left cut likewise, lo the rest; of a NaN or an infinity hi is all.
template <int kDT>
__device__ __forceinline__ void split_values(const typename Value<kDT>::raw (&r)[8],
                                             v8bf (&part)[kSplit<kDT>])
{
    if constexpr (kDT == IQ_DTYPE_BF16) {
        part[0] = __builtin_bit_cast(v8bf, r);
    } else {
        constexpr int kN = kSplit<kDT>;
        uint32_t u[kN][8], top = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float left = Value<kDT>::load(r[i]);
            top = max(top, __float_as_uint(left) & 0x7fffffffu);
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                u[k][i] = __float_as_uint(left);
                left = left - __uint_as_float(u[k][i] & 0xffff0000u);
            }
        }
        if constexpr (kDT == IQ_DTYPE_F16) {
            // Without a branch, which costs a kernel registers.
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t bits = u[0][i] & 0x7fffffffu;
                u[0][i] = bits > 0x7f800000u ? 0x7fc00000u : u[0][i];
                u[1][i] = bits >= 0x7f800000u ? 0u : u[1][i];
            }
        } else if (top >= 0x7f800000u) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (finite_f32(Value<kDT>::load(r[i]))) continue;
                // A NaN whose payload is in the bits that are cut stays one.
                u[0][i] |= u[0][i] & 0xffffu ? 0x400000u : 0u;
#pragma unroll
                for (int k = 1; k < kN; ++k) u[k][i] = 0u;
            }
        }
        // The upper halves of two words.
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = __builtin_amdgcn_perm(u[k][2 * i + 1], u[k][2 * i], 0x07060302u);
            part[k] = __builtin_bit_cast(v8bf, w);
        }
    }
}

// Whether the values of a lane's groups are exact in fp16: scales within its range, or
// zeros only (NaN where the scale is).
template <int kN>
__device__ __forceinline__ bool exact_in_f16(const v4u (&word)[kN], const uint32_t (&byte)[kN])
{
    bool exact = true;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
        const v4u w = word[i];
        exact &= byte[i] - kLowF16 <= kHighF16 - kLowF16 ||
                 ((w.x | w.y | w.z | w.w) & 0x77777777u) == 0u;
    }
    return exact;
}

// The scale bytes g0 .. g0 + 15 of a row that ends before, that of 1 beyond its end.
__device__ __forceinline__ v4u last_scales(const uint8_t* row, int g0, int groups)
{
    unsigned __int128 v = 0;
    constexpr uint32_t kOnes = 0x7f7f7f7fu;
    if (g0 >= groups) return v4u{kOnes, kOnes, kOnes, kOnes};
    if (groups >= 16) {
        v = __builtin_bit_cast(unsigned __int128, load16(row + groups - 16)) >> 8 * (g0 + 16 - groups);
    } else {
#pragma unroll 1
        for (int i = 0; i < groups - g0; ++i) v |= (unsigned __int128)row[g0 + i] << 8 * i;
    }
    v |= __builtin_bit_cast(unsigned __int128, v4u{kOnes, kOnes, kOnes, kOnes}) << 8 * (groups - g0);
    return __builtin_bit_cast(v4u, v);
}

// A tile whose rows, the same for all lanes, are kept in scalar registers: the sums below need
// them late, and a few vector registers more would cost some kernels a workgroup of the compute
// unit.  (There are below 2^31 rows.)
__device__ __forceinline__ Tile rows_in_scalars(Tile t)
{
    t.row0 = __builtin_amdgcn_readfirstlane((int)t.row0);
    t.row_end = __builtin_amdgcn_readfirstlane((int)t.row_end);
    return t;
}

// The lanes of the wave whose groups may have infinite values.  (A lane mask is kept in scalar
// registers.)
template <int kN>
__device__ __forceinline__ uint64_t may_be_infinite(const uint32_t (&byte)[kN])
{
    uint32_t top = byte[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) top = max(top, byte[i]);
    return __ballot(top >= kInfinite);
}

// Sums over the depths begin .. end - 1 of a weight with infinite values, for 16 kFC
// channels from `channel` on and kFT rows of activations for each of 16 lanes.  An infinite
// value meets the first part of an activation only, which is 0 where the activation is: the
// others are 0 where the first is all, and 0 times infinity is NaN.  Nothing is asked for
// ahead, and with the sums done before a product takes 2 to 4 times as long (2048 x 4096 x
// 4096 of fp32 activations 616 us, 151 where the weight is finite).
template <int kDT, int kFC, int kFT>
__device__ __forceinline__ void sum_with_infinities(const Fp4Product& p, int expert, int channel,
                                                    const typename Value<kDT>::raw* const (&from)[kFT],
                                                    int begin, int end, v4f (&acc)[kFC][kFT])
{
    constexpr int kS = kSplit<kDT>;
    const int lane = threadIdx.x % kWave, quarter = lane / 16;
#pragma unroll
    for (int i = 0; i < kFC; ++i)
#pragma unroll
        for (int j = 0; j < kFT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
    for (int at = begin; at < end; at += kGroup) {
        v8bf a[kFC], rest[kFC];
#pragma unroll
        for (int i = 0; i < kFC; ++i) {
            const int64_t n = min(channel + 16 * i + lane % 16, p.channels - 1);
            const uint32_t byte = p.scale[expert * p.s_stride + n * p.lds + at / kGroup];
            uint32_t word;
            __builtin_memcpy(&word, p.w + expert * p.w_stride + n * p.ldw + at / 2 + 4 * quarter, 4);
            a[i] = values_of(word, group_scale(byte));
            rest[i] = values_of(finite_codes(word, byte), group_scale(byte));
        }
#pragma unroll
        for (int j = 0; j < kFT; ++j) {
            typename Value<kDT>::raw r[8];
            v8bf part[kS];
            __builtin_memcpy(r, from[j] + at + 8 * quarter, sizeof(r));
            split_values<kDT>(r, part);
#pragma unroll
            for (int q = kS - 1; q >= 0; --q)
#pragma unroll
                for (int i = 0; i < kFC; ++i) acc[i][j] = mfma16(q ? rest[i] : a[i], part[q], acc[i][j]);
        }
    }
}

// What the wave's lanes have written to LDS is there for its other lanes, and what they have
// read may be written over.  A wave's LDS accesses are done in order, so this is for the
// compiler, which must not move one across.
__device__ __forceinline__ void order_in_wave()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 4 consecutive channels of one row of y, in its type.
template <int kDT>
__device__ __forceinline__ void store_channels(const Fp4Product& p, int64_t row, int channel, v4f f)
{
    typedef typename Value<kDT>::raw raw;
    raw* to = static_cast<raw*>(p.y) + row * p.ldy + channel;
    raw v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = Value<kDT>::store(f[i]);
    if (channel + 4 <= p.channels) {
        __builtin_memcpy(to, v, sizeof(v));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (channel + i < p.channels) to[i] = v[i];
    }
}

template <int kDT, int kRows, int kChannels, int kThreads>
__device__ __forceinline__ void store_zeros(const Fp4Product& p, const Tile& t)
{
    for (int i = threadIdx.x; i < kRows * (kChannels / 4); i += kThreads) {
        const int64_t row = t.row0 + i / (kChannels / 4);
        const int channel = t.channel_tile * kChannels + i % (kChannels / 4) * 4;
        if (row < t.row_end && channel < p.channels)
            store_channels<kDT>(p, row, channel, v4f{0.0f, 0.0f, 0.0f, 0.0f});
    }
}

// A handful of rows: a workgroup takes 16 kFC channels of kTok rows, and its waves share
// the depth in blocks of 4 steps.  A block of the weight is asked for while the one
// before is multiplied.  The activations, few of them, are split into their parts once
// by the lanes together, and every lane takes its operand from there: as operands
// straight from memory, 16 / kTok times as many would be loaded and split (one token
// through 4096 x 4096: bf16 5.4 us that way and 3.9 as it is, fp16 10.7 and 4.2, fp32
// 11.5 and 4.7).  Bound by latency, then by HBM: the weight's 9 MB in 4.7 us, waited for
// singly; 16 tokens, 2 of 16 experts of 1536 x 4096 47 MB in 16 us.
template <int kDT, int kTok, int kFC, int kWaves, bool kExperts>
__global__ __launch_bounds__(kWaves* kWave) void fp4_few_kernel(Fp4Product p, int channel_tiles)
{
    typedef typename Value<kDT>::raw raw;
    constexpr int kN = kStaged<kDT>, kChannels = 16 * kFC, kThreads = kWaves * kWave;
    constexpr int kFT = (kTok + 15) / 16;
    constexpr int kBlock = 4;
    // Steps whose activations are staged at once, 8 values each to a lane kX times.
    constexpr int kSub = kTok <= 2 ? 4 : (kTok == 4 ? 2 : 1);
    constexpr int kUnits = kSub * kPiece / 8, kX = kTok * kUnits / kWave;
    constexpr int kRow = kSub * kPiece + 8;           // rows start on different banks
    union Shared {
        uint16_t x[kWaves][kN][kTok][kRow];
        float sums[kWaves][kTok][kChannels];
    };
    __shared__ __align__(16) Shared shared;
    const Tile t = kExperts ? rows_in_scalars(expert_tile<kTok>(p, channel_tiles))
                            : dense_tile<kTok>(p, channel_tiles);
    if (t.expert == -2) return;
    if (t.expert == -1) {
        store_zeros<kDT, kTok, kChannels, kThreads>(p, t);
        return;
    }
    const int lane = threadIdx.x % kWave, quarter = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int channel0 = t.channel_tile * kChannels;
    const int groups = p.depth / kGroup;
    const int steps = (groups + 3) / 4;
    const int first = (int)((int64_t)steps * wave / kWaves);
    const int last = (int)((int64_t)steps * (wave + 1) / kWaves);

    // Beyond the last group, whose activations are zeros: its codes, with scale 1.
    const uint8_t *w[kFC], *scale[kFC];
#pragma unroll
    for (int i = 0; i < kFC; ++i) {
        const int64_t n = min(channel0 + 16 * i + lane % 16, p.channels - 1);
        w[i] = p.w + t.expert * p.w_stride + n * p.ldw;
        scale[i] = p.scale + t.expert * p.s_stride + n * p.lds;
    }
    v4u codes[2][kBlock][kFC], scales[2][kFC];
    auto fetch = [&](int b, int s) {
#pragma unroll
        for (int i = 0; i < kFC; ++i) {
#pragma unroll
            for (int j = 0; j < kBlock; ++j)
                if (s + j < last)
                    codes[b][j][i] = load16(w[i] + min(4 * (s + j) + quarter, groups - 1) * (kGroup / 2));
            if (s < last)
                scales[b][i] = 4 * s + 16 <= groups ? load16(scale[i] + 4 * s)
                                                    : last_scales(scale[i], 4 * s, groups);
        }
    };
    fetch(0, first);

    const raw* from[kX];
#pragma unroll
    for (int i = 0; i < kX; ++i) {
        const int64_t row = min(t.row0 + (i * kWave + lane) / kUnits, t.row_end - 1);
        from[i] = static_cast<const raw*>(p.x) + (kExperts ? token_of(p, row) : row) * p.ldx;
    }
    Chunk<kDT, true> held[kX];
    auto fetch_x = [&](int s) {
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int at = s * kPiece + (i * kWave + lane) % kUnits * 8;
            held[i].load(from[i], at, p.depth);
        }
    };
    auto stage_x = [&]() {
#pragma unroll
        for (int i = 0; i < kX; ++i) {
            const int unit = i * kWave + lane;
            v8bf part[kN];
            raw r[8];
            __builtin_memcpy(r, held[i].r, sizeof(r));
            if constexpr (kN > 1)
                split_values<kDT>(r, part);
            else
                part[0] = __builtin_bit_cast(v8bf, r);
#pragma unroll
            for (int q = 0; q < kN; ++q)
                *reinterpret_cast<v8bf*>(&shared.x[wave][q][unit / kUnits][unit % kUnits * 8]) = part[q];
        }
    };
    v4f acc[kFC][kFT] = {};
    uint64_t infinite = 0u;
    auto multiply = [&](int in_sub, const v4u (&word)[kFC], const v4u (&scales_of)[kFC], int j) {
        uint32_t byte[kFC];
#pragma unroll
        for (int i = 0; i < kFC; ++i) byte[i] = scales_of[i][j] >> 8 * quarter & 0xffu;
        if constexpr (kSplit<kDT> > 1) infinite |= may_be_infinite(byte);
        auto operand = [&](int f, int q, int k) {
            return *reinterpret_cast<const v8bf*>(
                &shared.x[wave][q][(16 * f + lane % 16) % kTok][in_sub * kPiece + 32 * quarter + 8 * k]);
        };
        if constexpr (kDT == IQ_DTYPE_F16) {
            if (__all(exact_in_f16(word, byte))) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    v8h b[kFT];
#pragma unroll
                    for (int f = 0; f < kFT; ++f) b[f] = __builtin_bit_cast(v8h, operand(f, 0, k));
#pragma unroll
                    for (int i = 0; i < kFC; ++i) {
                        const v8h a = half_values_of(word[i][k], group_scale(byte[i]));
#pragma unroll
                        for (int f = 0; f < kFT; ++f) acc[i][f] = mfma16(a, b[f], acc[i][f]);
                    }
                }
                return;
            }
        }
        constexpr int kS = kSplit<kDT>;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v8bf b[kFT][kS];
#pragma unroll
            for (int f = 0; f < kFT; ++f) {
                if constexpr (kS > kN) {
                    raw r[8];
                    const v8bf v = operand(f, 0, k);
                    __builtin_memcpy(r, &v, sizeof(r));
                    split_values<kDT>(r, b[f]);
                } else {
#pragma unroll
                    for (int q = 0; q < kS; ++q) b[f][q] = operand(f, q, k);
                }
            }
#pragma unroll
            for (int i = 0; i < kFC; ++i) {
                const v8bf a = values_of(word[i][k], group_scale(byte[i]));
#pragma unroll
                for (int f = 0; f < kFT; ++f)
#pragma unroll
                    for (int q = kS - 1; q >= 0; --q) acc[i][f] = mfma16(a, b[f][q], acc[i][f]);
            }
        }
    };
    if (first < last) fetch_x(first);
    for (int s0 = first; s0 < last; s0 += 2 * kBlock) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int s1 = s0 + h * kBlock;
            if (s1 >= last) break;
            fetch(1 - h, s1 + kBlock);
#pragma unroll
            for (int j = 0; j < kBlock; ++j) {
                const int s = s1 + j;
                if (s >= last) break;
                if (j % kSub == 0) {
                    order_in_wave();
                    stage_x();
                    order_in_wave();
                    if (s + kSub < last) fetch_x(s + kSub);
                }
                multiply(j % kSub, codes[h][j], scales[h], j);
            }
        }
    }

    if (kSplit<kDT> > 1 && __builtin_expect(infinite != 0u, 0)) {
        const raw* rows[kFT];
#pragma unroll
        for (int f = 0; f < kFT; ++f) {
            const int64_t row = min(t.row0 + (16 * f + lane % 16) % kTok, t.row_end - 1);
            rows[f] = static_cast<const raw*>(p.x) + (kExperts ? token_of(p, row) : row) * p.ldx;
        }
        sum_with_infinities<kDT>(p, t.expert, channel0, rows, first * kPiece,
                                 min(last * kPiece, p.depth), acc);
    }
    __syncthreads();
    if (lane % 16 < kTok) {
#pragma unroll
        for (int i = 0; i < kFC; ++i)
#pragma unroll
            for (int f = 0; f < kFT; ++f)
                *reinterpret_cast<v4f*>(&shared.sums[wave][16 * f + lane % 16][16 * i + 4 * quarter]) =
                    acc[i][f];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kTok * kChannels; i += kThreads) {
        const int64_t row = t.row0 + i / kChannels;
        const int channel = channel0 + i % kChannels;
        if (row >= t.row_end || channel >= p.channels) continue;
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) sum += shared.sums[v][i / kChannels][i % kChannels];
        static_cast<raw*>(p.y)[row * p.ldy + channel] = Value<kDT>::store(sum);
    }
}

// ---------------------------------------------------------------------------
// Many rows
// ---------------------------------------------------------------------------

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void global_void;

// 16 bytes a lane from global memory into LDS at `to` + 16 * lane.
__device__ __forceinline__ void copy_to_lds(const uint16_t* from, uint16_t* to)
{
    __builtin_amdgcn_global_load_lds((global_void*)(uintptr_t)from, (lds_void*)to, 16, 0, 0);
}

// The same from base + offset + step bytes, with the offset of the lane's own; zeros where
// it is kBeyond.  (The host's pass over this file does not know the type of a buffer.)
constexpr uint32_t kBeyond = 0xffffffffu;
__device__ __forceinline__ void copy_to_lds(const uint16_t* base, uint32_t offset, int step,
                                            uint16_t* to)
{
#ifdef __HIP_DEVICE_COMPILE__
    const __amdgpu_buffer_rsrc_t buffer = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint16_t*>(base), 0, kBeyond - 1, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer, (lds_void*)to, 16, offset, step, 0, 0);
#endif
}

// Waits until at most kLeft of this wave's loads are under way and all its LDS
// reads have arrived, then for the other waves.  The wait is the compiler's own
// instruction, so that it knows which registers have their values.
template <int kLeft>
__device__ __forceinline__ void wait_and_meet()
{
    static_assert(kLeft < 64, "vmcnt holds 6 bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kLeft & 15) | 7 << 4 | (kLeft >> 4) << 14);
    asm volatile("s_barrier" ::: "memory");
}

__device__ const uint16_t kZeros[8] __attribute__((aligned(16))) = {};

// x in rows of ldx values that start on 16 bytes and have `width` of them: 16-bit
// activations as they are where they do, others as split_kernel lays them out, the
// three bf16 parts of each piece of fp32 one after another.
struct Parts {
    const uint16_t* x;
    int64_t ldx;
    int width;
};

// kWT x kWC waves share a tile of kRows rows of y by kChannels channels, each a
// part of kRows/kWT by kChannels/kWC, in steps of 128 of the depth.  The activations
// go through a ring of kStages buffers in LDS that direct copies fill kStages - 1
// steps ahead.  The weight comes step by step through registers into two buffers of
// codes (any alignment), its scales 8 steps at a time, and becomes bf16 where it is
// multiplied, four instructions for 8 values.
//
// Of eight waves, two on a SIMD, the second half runs half a step behind (ping-pong): on
// each SIMD one wave multiplies while the other reads its operands.  A step is two
// barriers long.  Four waves go together, a step a barrier, and it is other workgroups
// of the compute unit that fill the gaps.
//
// 128 x 256 at 4096^3 in bf16: 114 us waited for singly, 1210 TFLOP/s, the matrix cores 54 %
// busy, and what they wait for LDS reads and conversions; a library product of the unpacked
// weight 97 to 104.  On the way there: the weight straight to registers each step 260 us (a
// load that touches 16 rows takes 75 cycles to issue), through LDS in steps of 64 of the depth
// 147, of 128 128, copies by a buffer's 32-bit offsets 124.  Smaller tiles fill the card where
// there are few: 1021 x 2049 x 1568 in bf16 takes 18.7 us with 32 x 64.
template <int kDT, int kRows, int kChannels, int kWT, int kWC, int kStages, bool kExperts>
__global__ __launch_bounds__(kWT* kWC* kWave, kWT* kWC / 4) void fp4_tile_kernel(Fp4Product p,
                                                                               Parts parts,
                                                                               int channel_tiles)
{
    typedef typename Value<kDT>::raw raw;
    constexpr int kWaves = kWT * kWC, kThreads = kWaves * kWave;
    constexpr bool kPingPong = kWaves == 8;
    constexpr int kFT = kRows / kWT / 16, kFC = kChannels / kWC / 16;
    constexpr int kParts = kStaged<kDT>;
    constexpr int kRowsPerLoad = 4;   // of 256 bytes each
    constexpr int kLoads = kRows / kRowsPerLoad / kWaves;
    // Groups of a step, 16 bytes of codes each, and a thread's part of them.
    constexpr int kGroups = kPiece / kGroup, kCodes = kChannels * kGroups / kThreads;
    // Scales come for more steps at once, 16 groups to a thread: what they cost is the
    // cache lines they are spread over.
    constexpr int kScales = 32, kScaleThreads = kChannels * kScales / 16;
    constexpr int kScaleRow = kScales / 4 + 1;        // words: rows start on different banks
    static_assert(kLoads * kRowsPerLoad * kWaves == kRows && kFT > 0 && kFC > 0 &&
                  kCodes * kThreads == kChannels * kGroups && kScaleThreads <= kThreads, "tile");
    struct Staged {
        uint16_t x[kStages][kRows * kPiece];
        v4u codes[2][kChannels * kGroups];
        uint32_t scales[2][kChannels * kScaleRow];
    };
    __shared__ __align__(1024) Staged staged;

    const Tile t = kExperts ? rows_in_scalars(expert_tile<kRows>(p, channel_tiles))
                            : dense_tile<kRows>(p, channel_tiles);
    if (t.expert == -2) return;
    if (t.expert == -1) {
        store_zeros<kDT, kRows, kChannels, kThreads>(p, t);
        return;
    }
    const int lane = threadIdx.x % kWave, quarter = lane / 16;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wt = wave % kWT, wc = wave / kWT;

    // Staged rows in pieces of 16 bytes, piece k of a lane's group q in slot
    // (4 k + q) ^ (row % 16).  A read of 16 bytes a lane takes 16 lanes at a time, four
    // neighbours each of different rows and quarters of the wave: with q in the low bits
    // they meet different banks (with 4 q + k two and two meet, 39 % more LDS cycles:
    // 4096^3 120 us against 117).  Rows beyond the last repeat it: their results are not stored.
    auto column = [&](int i) {
        const int c = (lane % 16) ^ ((wave * kLoads + i) * kRowsPerLoad + lane / 16) % 16;
        return (c % 4 * 4 + c / 4) * 8;
    };
    // Dense rows by 32-bit offsets into a buffer that begins at the tile's first row,
    // where an offset beyond its end reads zeros; gathered rows by addresses.
    const uint16_t* from[kExperts ? kLoads : 1];
    uint32_t near[kExperts ? 1 : kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int r = (wave * kLoads + i) * kRowsPerLoad + lane / 16;
        const int64_t row = min(t.row0 + r, t.row_end - 1);
        if constexpr (kExperts)
            from[i] = parts.x + token_of(p, row) * parts.ldx + column(i);
        else
            near[i] = ((uint32_t)(row - t.row0) * (uint32_t)parts.ldx + column(i)) * 2;
    }
    const uint16_t* x0 = parts.x + (kExperts ? 0 : t.row0 * parts.ldx);
    // Steps beyond the last are zeros.
    auto fetch = [&](int b, int step) {
        const int at = step * kPiece;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const bool here = at + column(i) < parts.width;
            uint16_t* to = &staged.x[b][(wave * kLoads + i) * 512];
            if constexpr (kExperts)
                copy_to_lds(here ? from[i] + at : kZeros, to);
            else
                copy_to_lds(x0, here ? near[i] : kBeyond, at * 2, to);
        }
    };

    const int groups = p.depth / kGroup;
    const int channel0 = t.channel_tile * kChannels;
    const uint8_t* w = p.w + t.expert * p.w_stride + (int64_t)channel0 * p.ldw;
    const uint8_t* scale = p.scale + t.expert * p.s_stride + (int64_t)channel0 * p.lds;
    // Row r's group g of a step in slot g ^ slot(r).
    auto slot = [](int r) { return r / 2 % kGroups; };
    v4u codes[kCodes];
    auto fetch_codes = [&](int piece) {
#pragma unroll
        for (int i = 0; i < kCodes; ++i) {
            const int q = i * kThreads + threadIdx.x, r = q / kGroups;
            const int n = min(r, p.channels - 1 - channel0);
            const int g = min(piece * kGroups + ((q % kGroups) ^ slot(r)), groups - 1);
            codes[i] = load16(w + ((uint32_t)n * (uint32_t)p.ldw + g * (kGroup / 2)));
        }
    };
    auto store_codes = [&](int b) {
#pragma unroll
        for (int i = 0; i < kCodes; ++i) staged.codes[b][i * kThreads + threadIdx.x] = codes[i];
    };
    // Groups beyond the last, whose activations are zeros, have the scale 1.
    v4u scales = {};
    auto fetch_scales = [&](int turn) {
        if (threadIdx.x >= kScaleThreads) return;
        const int n = min((int)threadIdx.x / 2, p.channels - 1 - channel0);
        const uint8_t* s = scale + (uint32_t)n * (uint32_t)p.lds;
        const int g0 = turn * kScales + threadIdx.x % 2 * 16;
        if (g0 + 16 <= groups)
            scales = load16(s + g0);
        else
            scales = last_scales(s, g0, groups);
    };
    auto store_scales = [&](int b) {
        if (threadIdx.x >= kScaleThreads) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            staged.scales[b][threadIdx.x / 2 * kScaleRow + threadIdx.x % 2 * 4 + i] = scales[i];
    };

    v4f acc[kFC][kFT] = {};
    v8bf x[4][kFT];
    v4u word[kFC];
    uint32_t byte[kFC];
    // The ring's buffer b, and the weight of step `piece` of the depth.
    auto read = [&](int b, int piece) {
#pragma unroll
        for (int i = 0; i < kFC; ++i) {
            const int r = (wc * kFC + i) * 16 + lane % 16;
            word[i] = staged.codes[piece % 2][r * kGroups + (quarter ^ slot(r))];
            byte[i] = reinterpret_cast<const uint8_t*>(
                &staged.scales[4 * piece / kScales % 2][r * kScaleRow])[4 * piece % kScales + quarter];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < kFT; ++j) {
                const int r = (wt * kFT + j) * 16 + lane % 16;
                x[k][j] = *reinterpret_cast<const v8bf*>(
                    &staged.x[b][r * kPiece + ((4 * k + quarter) ^ (lane % 16)) * 8]);
            }
    };
    // The products of one kind of operand, the next one's conversions among those of one.
    auto multiply_as = [&](auto&& operand, auto&& activations) {
        auto a = operand(0), next = a;
#pragma unroll
        for (int f = 0; f < 4 * kFC; ++f) {
            if (f + 1 < 4 * kFC) next = operand(f + 1);
#pragma unroll
            for (int j = 0; j < kFT; ++j)
                acc[f % kFC][j] = mfma16(a, activations(f / kFC, j), acc[f % kFC][j]);
            a = next;
            constexpr int kEach = kFT >= 4 ? 1 : 4 / kFT;
#pragma unroll
            for (int i = 0; i < 4 / kEach; ++i) {
                __builtin_amdgcn_sched_group_barrier(0x008, kFT * kEach / 4, 0);
                __builtin_amdgcn_sched_group_barrier(0x002, kEach, 0);
            }
        }
    };
    // fp16 activations are multiplied as fp16 as long as the weight is exact in it.
    bool exact = true;
    uint64_t infinite = 0u;
    auto multiply = [&](auto in_f16, int of_part) {
        if constexpr (kSplit<kDT> > 1 && !in_f16)
            if (of_part == 0) infinite |= may_be_infinite(byte);
        auto weight = [&](int f) { return values_of(word[f % kFC][f / kFC], group_scale(byte[f % kFC])); };
        if constexpr (kDT != IQ_DTYPE_F16) {
            multiply_as(weight, [&](int k, int j) { return x[k][j]; });
        } else if constexpr (in_f16) {
            exact &= exact_in_f16(word, byte);
            multiply_as([&](int f) { return half_values_of(word[f % kFC][f / kFC],
                                                           group_scale(byte[f % kFC])); },
                        [&](int k, int j) { return __builtin_bit_cast(v8h, x[k][j]); });
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int j = 0; j < kFT; ++j) {
                    raw r[8];
                    v8bf part[kSplit<kDT>];
                    __builtin_memcpy(r, &x[k][j], sizeof(r));
                    split_values<kDT>(r, part);
#pragma unroll
                    for (int q = kSplit<kDT> - 1; q >= 0; --q)
#pragma unroll
                        for (int i = 0; i < kFC; ++i)
                            acc[i][j] = mfma16(weight(k * kFC + i), part[q], acc[i][j]);
                    __builtin_amdgcn_sched_barrier(0);  // one at a time, for want of registers
                }
        }
    };

    const int pieces = (groups + 3) / 4;
    auto run = [&](auto in_f16) {
        fetch_codes(0);
        fetch_scales(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) fetch(i, i);
        __builtin_amdgcn_sched_barrier(0);
        store_codes(0);
        store_scales(0);
        fetch_scales(1);
        fetch_codes(1);
        constexpr int kLeft = (kStages - 2) * kLoads;
        constexpr int kTurn = kScales / kGroups;
        int buffer = 0;
        auto store_weight = [&](int piece) {
            store_codes((piece + 1) % 2);
            if (piece % kTurn == 0) store_scales((piece / kTurn + 1) % 2);
        };
        // A step of the depth is one of each part of the activations.  The one kStages - 1
        // ahead goes into the buffer of the one before, and with the first part the weight two
        // steps ahead is asked for.
        auto fetch_ahead = [&](int piece, int part) {
            fetch(buffer == 0 ? kStages - 1 : buffer - 1, piece * kParts + part + kStages - 1);
            buffer = buffer + 1 == kStages ? 0 : buffer + 1;
            if (part == 0) {
                __builtin_amdgcn_sched_barrier(0);
                if (piece % kTurn == 0) fetch_scales(piece / kTurn + 2);
                fetch_codes(piece + 2);
            }
        };
        if constexpr (kPingPong) {
            const bool late = wave >= kWaves / 2;
            wait_and_meet<kLeft + kCodes>();
            if (late) asm volatile("s_barrier" ::: "memory");
            for (int piece = 0; piece < pieces; ++piece) {
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    // The weight's step before, whose buffer this is, was read before the last
                    // barrier, as both halves read the step before.
                    if (part == 0) store_weight(piece);
                    read(buffer, piece);
                    fetch_ahead(piece, part);
                    // The next step has to be there.  The weight's codes were asked for behind
                    // the copies of the step kStages - 1 behind its first part's.
                    if (part <= kStages - 2)
                        wait_and_meet<kLeft + kCodes>();
                    else
                        wait_and_meet<kLeft>();
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_setprio(1);
                    multiply(in_f16, part);
                    __builtin_amdgcn_s_setprio(0);
                    __builtin_amdgcn_sched_barrier(0);
                    asm volatile("s_barrier" ::: "memory");
                }
            }
            if (!late) asm volatile("s_barrier" ::: "memory");
        } else {
            for (int piece = 0; piece < pieces; ++piece) {
#pragma unroll
                for (int part = 0; part < kParts; ++part) {
                    // This step has to be there, and the others are done with the one before.
                    // The codes last asked for are behind the copies of the step kStages - 1
                    // behind this weight's first part's, or the weight's before.
                    if (part == 0 ? kParts < kStages : part < kStages)
                        wait_and_meet<kLeft + kCodes>();
                    else
                        wait_and_meet<kLeft>();
                    if (part == 0) store_weight(piece);
                    const int b = buffer;
                    fetch_ahead(piece, part);
                    read(b, piece);
                    multiply(in_f16, part);
                }
            }
        }
    };
    run(std::bool_constant<kDT == IQ_DTYPE_F16>());
    if constexpr (kDT == IQ_DTYPE_F16) {
        // Otherwise all is done again with bf16 parts: 2048 x 4096 x 4096 61 us, with scales
        // out of range everywhere 244.
        wait_and_meet<0>();
        if (__builtin_expect(!__syncthreads_and(exact), 0)) {
#pragma unroll
            for (int i = 0; i < kFC; ++i)
#pragma unroll
                for (int j = 0; j < kFT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
            run(std::false_type());
        }
    }

    if (kSplit<kDT> > 1 && __builtin_expect(infinite != 0u, 0)) {
        const raw* rows[kFT];
#pragma unroll
        for (int j = 0; j < kFT; ++j) {
            const int64_t row = min(t.row0 + (wt * kFT + j) * 16 + lane % 16, t.row_end - 1);
            rows[j] = static_cast<const raw*>(p.x) + (kExperts ? token_of(p, row) : row) * p.ldx;
        }
        sum_with_infinities<kDT>(p, t.expert, channel0 + wc * kFC * 16, rows, 0, p.depth, acc);
    }

    // Results through LDS, as the matrix instructions leave them (4 channels of a row
    // to a lane), and out as whole rows of the wave's channels, 16 bytes a lane.
    wait_and_meet<0>();
    constexpr int kN = 16 / (int)sizeof(raw);
    constexpr int kRow = kFC * 16 + kN;               // rows start on different banks
    constexpr int kLanes = kFC * 16 / kN;             // lanes to a row
    static_assert(kWaves * 16 * kRow * (int)sizeof(raw) <= (int)sizeof(staged), "results fit");
    raw* mine = reinterpret_cast<raw*>(&staged) + wave * 16 * kRow;
    const int wave_channel = channel0 + wc * kFC * 16;
#pragma unroll
    for (int j = 0; j < kFT; ++j) {
        const int64_t row0 = t.row0 + (wt * kFT + j) * 16;
#pragma unroll
        for (int i = 0; i < kFC; ++i) {
            raw o[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) o[v] = Value<kDT>::store(acc[i][j][v]);
            __builtin_memcpy(__builtin_assume_aligned(mine + lane % 16 * kRow + i * 16 + 4 * quarter,
                                                      4 * sizeof(raw)),
                             o, sizeof(o));
        }
        order_in_wave();
#pragma unroll
        for (int s = 0; s < (16 * kLanes + kWave - 1) / kWave; ++s) {
            const int r = (s * kWave + lane) / kLanes, c = (s * kWave + lane) % kLanes * kN;
            const int channel = wave_channel + c;
            if (r >= 16 || row0 + r >= t.row_end || channel >= p.channels) continue;
            raw o[kN];
            __builtin_memcpy(o, __builtin_assume_aligned(mine + r * kRow + c, 16), 16);
            raw* to = static_cast<raw*>(p.y) + (row0 + r) * p.ldy + channel;
            if (channel + kN <= p.channels) {
                __builtin_memcpy(to, o, 16);
            } else {
#pragma unroll
                for (int v = 0; v < kN; ++v)
                    if (channel + v < p.channels) to[v] = o[v];
            }
        }
        order_in_wave();
    }
}

// Activations padded to whole pieces with zeros, fp32 split into its parts: row t,
// piece c, part q from out[t][(c * kN + q) * 128].
template <int kDT>
__global__ __launch_bounds__(256) void split_kernel(const void* __restrict__ x, int64_t ldx,
                                                    int64_t tokens, int depth, int64_t first,
                                                    int per_row, uint16_t* __restrict__ out)
{
    typedef typename Value<kDT>::raw raw;
    constexpr int kN = kStaged<kDT>;
    const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;   // 8 values each
    const int64_t row = i / per_row;
    if (row >= tokens) return;
    const int at = (int)(i - row * per_row) * 8;
    raw r[8] = {};
    if (at < depth)
        __builtin_memcpy(r, static_cast<const raw*>(x) + row * ldx + at, sizeof(r));
    v8bf part[kN];
    if constexpr (kN > 1)
        split_values<kDT>(r, part);
    else
        part[0] = __builtin_bit_cast(v8bf, r);
    uint16_t* to = out + (row * per_row * 8 + at / kPiece * kPiece) * kN + at % kPiece;
#pragma unroll
    for (int q = 0; q < kN; ++q) *reinterpret_cast<v8bf*>(to + q * kPiece) = part[q];
}

// Strides up to which the tile kernel's 32-bit offsets reach all of its rows.
constexpr int64_t kNear = INT64_C(1) << 22;

// Every expert (and the dropped rows) may end in a tile that is not full.
int64_t workgroups(const Fp4Product& p, int rows, int channel_tiles)
{
    const int64_t row_tiles = p.experts ? std::min(p.rows, p.rows / rows + p.experts + 1)
                                        : (p.rows + rows - 1) / rows;
    return row_tiles * channel_tiles;
}

// Whether the activations can be copied to LDS as they are: rows that start on 16
// bytes, 256 of them within the reach of 32-bit offsets.
bool direct(int dtype, const void* x, int64_t ldx, int64_t tokens)
{
    return dtype != IQ_DTYPE_F32 && reinterpret_cast<uintptr_t>(x) % 16 == 0 &&
           (ldx % 8 == 0 || tokens == 1) && ldx <= kNear;
}

template <int kDT, int kRows, int kChannels, int kWT, int kWC, int kStages, bool kExperts>
hipError_t launch_tiles(const Fp4Product& p, const Parts& parts, hipStream_t stream)
{
    const int channel_tiles = (p.channels + kChannels - 1) / kChannels;
    Fp4Product part = p;
    return in_parts(workgroups(p, kRows, channel_tiles), kWT * kWC * kWave,
                    [&](int64_t first, dim3 wgs) {
        part.first_tile = first;
        hipLaunchKernelGGL((fp4_tile_kernel<kDT, kRows, kChannels, kWT, kWC, kStages, kExperts>),
                           wgs, dim3(kWT * kWC * kWave), 0, stream, part, parts, channel_tiles);
        return hipGetLastError();
    });
}

template <int kDT>
hipError_t launch_split(const Fp4Product& p, void* workspace, Parts* parts, hipStream_t stream)
{
    const int per_row = (p.depth + kPiece - 1) / kPiece * (kPiece / 8);
    uint16_t* out = static_cast<uint16_t*>(workspace);
    const int width = per_row * 8 * kStaged<kDT>;
    *parts = {out, width, width};
    return in_parts((p.tokens * per_row + 255) / 256, 256, [&](int64_t first, dim3 wgs) {
        hipLaunchKernelGGL(split_kernel<kDT>, wgs, dim3(256), 0, stream, p.x, p.ldx, p.tokens,
                           p.depth, first, per_row, out);
        return hipGetLastError();
    });
}

template <int kDT, int kTok, int kFC, int kWaves, bool kExperts>
hipError_t launch_few(const Fp4Product& p, hipStream_t stream)
{
    const int channel_tiles = (p.channels + 16 * kFC - 1) / (16 * kFC);
    Fp4Product part = p;
    return in_parts(workgroups(p, kTok, channel_tiles), kWaves * kWave,
                    [&](int64_t first, dim3 wgs) {
        part.first_tile = first;
        hipLaunchKernelGGL((fp4_few_kernel<kDT, kTok, kFC, kWaves, kExperts>), wgs,
                           dim3(kWaves * kWave), 0, stream, part, channel_tiles);
        return hipGetLastError();
    });
}

template <int kDT>
hipError_t launch_dense(int size, const Fp4Product& p, const Parts& x, hipStream_t stream)
{
    switch (size) {
    case size_key(1, 16, 8): return launch_few<kDT, 1, 1, 8, false>(p, stream);
    case size_key(4, 16, 8): return launch_few<kDT, 4, 1, 8, false>(p, stream);
    case size_key(8, 16, 8): return launch_few<kDT, 8, 1, 8, false>(p, stream);
    case size_key(16, 16, 8): return launch_few<kDT, 16, 1, 8, false>(p, stream);
    case size_key(16, 32, 8):
        // The 16-bit types have a faster one always.
        if constexpr (kDT == IQ_DTYPE_F32) return launch_few<kDT, 16, 2, 8, false>(p, stream);
        break;
    case size_key(32, 32, 8):
        // The parts of 32 rows of fp32 do not fit LDS.
        if constexpr (kDT != IQ_DTYPE_F32) return launch_few<kDT, 32, 2, 8, false>(p, stream);
        break;
    case size_key(32, 64, 4): return launch_tiles<kDT, 32, 64, 1, 4, 2, false>(p, x, stream);
    case size_key(32, 128, 4): return launch_tiles<kDT, 32, 128, 1, 4, 2, false>(p, x, stream);
    case size_key(64, 128, 4): return launch_tiles<kDT, 64, 128, 1, 4, 2, false>(p, x, stream);
    case size_key(128, 256, 8): return launch_tiles<kDT, 128, 256, 2, 4, 3, false>(p, x, stream);
    default: break;
    }
    return launch_few<kDT, 16, 1, 4, false>(p, stream);
}

template <int kDT>
hipError_t launch_experts(int size, const Fp4Product& p, const Parts& x, hipStream_t stream)
{
    switch (size) {
    case size_key(1, 16, 4): return launch_few<kDT, 1, 1, 4, true>(p, stream);
    case size_key(4, 16, 4): return launch_few<kDT, 4, 1, 4, true>(p, stream);
    case size_key(8, 16, 4): return launch_few<kDT, 8, 1, 4, true>(p, stream);
    case size_key(8, 32, 4):
        // fp16 has a faster one always.
        if constexpr (kDT != IQ_DTYPE_F16) return launch_few<kDT, 8, 2, 4, true>(p, stream);
        break;
    case size_key(32, 64, 4): return launch_tiles<kDT, 32, 64, 1, 4, 2, true>(p, x, stream);
    case size_key(32, 128, 4): return launch_tiles<kDT, 32, 128, 1, 4, 2, true>(p, x, stream);
    case size_key(64, 128, 4): return launch_tiles<kDT, 64, 128, 1, 4, 2, true>(p, x, stream);
    case size_key(128, 256, 8): return launch_tiles<kDT, 128, 256, 2, 4, 3, true>(p, x, stream);
    default: break;
    }
    return launch_few<kDT, 16, 2, 4, true>(p, stream);
}

// 0: the kernel of few rows, whatever its size, where the depth is beyond the reach of
// the tile kernel's offsets.
int choose_size(int dtype, int64_t rows, int64_t channels, int64_t depth, int experts)
{
    const int size = fp4_size(dtype, rows, channels, depth, experts);
    return is_tile(size) && depth > kNear / 4 ? 0 : size;
}

}  // namespace

int64_t fp4_workspace(int dtype, const void* x, int64_t ldx, int64_t tokens, int64_t rows,
                      int experts, int64_t channels, int64_t depth)
{
    if (!is_tile(choose_size(dtype, rows, channels, depth, experts)) ||
        direct(dtype, x, ldx, tokens))
        return 0;
    return tokens * ((depth + kPiece - 1) / kPiece * kPiece) * 2 *
           (dtype == IQ_DTYPE_F32 ? kStaged<IQ_DTYPE_F32> : 1);
}

hipError_t launch_fp4_product(const Fp4Product& p, void* workspace, hipStream_t stream)
{
    int size = choose_size(p.dtype, p.rows, p.channels, p.depth, p.experts);
    // So too where the weight's rows are too far apart.
    if (is_tile(size) && (p.ldw > kNear || p.lds > kNear)) size = 0;
    return with_dtype(p.dtype, [&](auto dt) {
        constexpr int kDT = decltype(dt)::value;
        Parts x = {static_cast<const uint16_t*>(p.x), p.ldx, p.depth};
        if (is_tile(size) && !direct(p.dtype, p.x, p.ldx, p.tokens)) {
            const hipError_t e = launch_split<kDT>(p, workspace, &x, stream);
            if (e != hipSuccess) return e;
        }
        return p.experts ? launch_experts<kDT>(size, p, x, stream)
                         : launch_dense<kDT>(size, p, x, stream);
    });
}

}  // namespace iqk

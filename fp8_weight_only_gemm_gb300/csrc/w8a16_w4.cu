// Products with 4-bit weights and group scales, for a few tokens.
//
// Mathematics.  C[m][n] = sum_g s[n][g] * ( sum_{k in g} A[m][k] (code[n][k] - z[n][g]) ).
// Codes become operands of the tensor cores exactly, products add in FP32, a group's sum is
// scaled once, in FP32: no weight is rounded. Bytes are HBM's to bound (0.5 a weight and the
// scales); the integer pipe, at one instruction in two cycles, bounds the decoding, so the two
// kernels below spend as few integer operations on a word of eight codes as they can.
//
// Layout. m16n8k16 with 16 weight rows as M and 8 columns as N. A lane's 32-bit word holds 8
// codes of a row, and masks take the pairs (k, k + 4) out of it; the order of a
// contraction's index being free, the activations are paired the same way, and weights never
// move between lanes.
//
// Work. K goes in stages of 256; a CTA takes the rows of a tile and a contiguous range of
// stages. Codes are copied by TMA, whole boxes, into rings. (Bulk copies of a row a lane are
// issued lane by lane and cost a warp some 400 instructions a stage.)
// The sums of a CTA's warps, and those of the CTAs of a cluster that share the rows, are added
// in a fixed order.
//   1 or 2 tokens (w4_stream_kernel). Every warp has a ring and a part of K of its own. The bits of
//     a nibble, as FP16, are the subnormal number c 2^-24 (or 16 c 2^-24 four bits higher): four
//     masks and a shift decode a word. The activations become FP16, times a power of two that
//     puts the largest of a chunk of 32 at 2^14 (exact down to 2^-24 of it), and a sixteenth of
//     that where the codes come times 16. The zero point leaves the product: with S = sum c a,
//     T = sum a, sum (c - z) a = S - z T. Columns that tokens leave unused take other chunks of K
//     (the operand is zero outside a column's own), so 8 (4) chunks need one set of sums and one
//     folding.
//   more (w4_tile_kernel). 128 rows a CTA; its 8 warps share the activations, as they are.
//     Nibbles are placed under the exponent of 128 (BF16) or 1024 (FP16), and 128 + z (1024 + z)
//     is subtracted, exactly. From 9 tokens on the pairs are (k, k + 1): two more operations a
//     word, for none on the activations.
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "w8a16_cluster.cuh"
#include "w8a16_kv.cuh"

namespace w8a16 {
namespace {

__device__ DeviceStatus g_w4_status;

constexpr uint32_t kStageK = 256;             // codes of a row per stage: 128 bytes
constexpr uint32_t kChunks = kStageK / 32;    // of 32 codes: a word a lane of a quad
constexpr uint32_t kMaxSplit = 8;             // CTAs of a cluster (portable size)

struct W4Args {
    const uint16_t* A;
    const uint8_t* W;
    const uint8_t* scale;      // FP32 or the activation type
    const uint8_t* zeros;      // or NULL: 8
    uint16_t* C;
    uint32_t lda, ldc, M, N, K;
    uint32_t scale_bytes;      // 4 or 2
    uint32_t split;            // CTAs of a cluster
    uint32_t early;            // weights may be read before the dependency wait
    uint64_t timeout_ns;       // limit of an in-kernel wait
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// A box at (x, y) without a cache hint.
__device__ __forceinline__ void box_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, uint32_t x, uint32_t y) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
                 : "memory");
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
    return mbar_wait(bar, parity, globaltimer_ns() + timeout_ns, abort_flag, &g_w4_status, 1);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
    return __all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity) || wait_slow(bar, parity, timeout_ns, abort_flag));
}

// (w4_stream_kernel) The weight operands of 32 codes of rows g and g + 8 (words at w, w + 1024: 128-byte rows):
// pairs (0,4) and 16 (1,5) | (2,6) and 16 (3,7), in units of 2^-24.
__device__ __forceinline__ void weights32(const uint8_t* w, uint32_t (&f0)[4], uint32_t (&f1)[4]) {
#pragma unroll
    for (uint32_t r = 0; r < 2; ++r) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(w + 1024 * r), h = q >> 8;
        f0[r] = q & 0x000F000Fu, f0[2 + r] = q & 0x00F000F0u;
        f1[r] = h & 0x000F000Fu, f1[2 + r] = h & 0x00F000F0u;
    }
}
// The activation operand of 8 consecutive values, times du.x, and their sum.
template <bool F16>
__device__ __forceinline__ float acts8(const uint4& v, float down, uint32_t (&b)[4]) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = unpack2<F16>(x[e]);
        f[2 * e] = y.x, f[2 * e + 1] = y.y;
    }
    const float odd = down * 0.0625f;
    b[0] = pack2<true>(f[0] * down, f[4] * down), b[1] = pack2<true>(f[1] * odd, f[5] * odd);
    b[2] = pack2<true>(f[2] * down, f[6] * down), b[3] = pack2<true>(f[3] * odd, f[7] * odd);
    return ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
}
template <bool F16>
__device__ __forceinline__ float amax8(const uint4& v) {
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    float mx = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 y = unpack2<F16>(x[e]);
        mx = max3(mx, fabsf(y.x), fabsf(y.y));
    }
    return mx;
}
// 2^(14 - E) for the exponent E of mx, and 2^(E - 14); both normal (tiny maxima keep fewer bits).
__device__ __forceinline__ float2 down_up(float mx) {
    const uint32_t E = min(max(__float_as_uint(mx) >> 23, 16u), 254u);
    return make_float2(__uint_as_float((268u - E) << 23), __uint_as_float((E - 14u) << 23));
}
template <bool F16>
__device__ __forceinline__ float scale_of(const W4Args& p, size_t at) {
    return p.scale_bytes == 4 ? *reinterpret_cast<const float*>(p.scale + 4 * at)
                              : unpack2<F16>(*reinterpret_cast<const uint16_t*>(p.scale + 2 * at)).x;
}
// acc + s (part up 2^24 - z sum), part in units of 2^-24
__device__ __forceinline__ float fold(float acc, float part, float up, float sum, float2 sz) {
    return fmaf(sz.x, fmaf(part * 16777216.f, up, -sz.y * sum), acc);
}

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        mma_f16(d, a, b0, b1);
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (w4_tile_kernel) 8 codes -> code - z. zb: (128 + z) twice in BF16, (1024 + z) twice in FP16.
// NATURAL: pairs (0,1) (2,3) (4,5) (6,7), else (0,4) (1,5) (2,6) (3,7).
template <bool F16, bool NATURAL>
__device__ __forceinline__ void decode8(uint32_t q, uint32_t zb, uint32_t (&o)[4]) {
    const uint32_t odd = q >> 4;   // byte j: code 2 j + 1 low
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t y = NATURAL ? prmt(q, odd, i == 0 ? 0x4400u : i == 1 ? 0x5511u : i == 2 ? 0x6622u : 0x7733u) : q >> (4 * i);
        const uint32_t x = (y & 0x000F000Fu) | (F16 ? 0x64006400u : 0x43004300u);
        if constexpr (F16) asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x), "r"(zb));
        else asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x), "r"(zb));
    }
}

// ------------------------------------------------------------- 1 or 2 tokens --
constexpr uint32_t kSwWarps = 4, kSwThreads = 32 * kSwWarps, kSwRows = 32, kSwStages = 3;
constexpr uint32_t kSwBox = kSwRows * 128, kSwAPitch = kStageK * 2 + 64;   // (no bank is hit twice)
constexpr uint32_t kSwRedPitch = kSwRows + 4;
constexpr uint32_t sw_smem_bytes(uint32_t mp) { return 1024 + kSwWarps * kSwStages * (kSwBox + mp * kSwAPitch); }

// MP tokens: column slot MP + m sums, for token m, the chunks that are slot modulo 8 / MP.
template <bool F16, uint32_t MP, uint32_t G>
__global__ void __launch_bounds__(kSwThreads, 4) w4_stream_kernel(const W4Args p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap) {
    constexpr uint32_t kSlots = 8 / MP, kFolds = MP;
    static_assert(kSlots >= G / 32, "a folding's chunks of one column share a group");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kSwWarps][kSwStages];
    __shared__ int abort_flag;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t rank = blockIdx.x % p.split, n0 = blockIdx.x / p.split * kSwRows;
    const uint32_t stages = (p.K + kStageK - 1) / kStageK, groups = p.K / G;
    const uint32_t s_begin = static_cast<uint32_t>(static_cast<uint64_t>(rank) * stages / p.split),
                   s_end = static_cast<uint32_t>(static_cast<uint64_t>(rank + 1) * stages / p.split);
    uint8_t* const boxes = smem + warp * kSwStages * kSwBox;
    uint8_t* const acts = smem + kSwWarps * kSwStages * kSwBox + warp * kSwStages * MP * kSwAPitch;
    const uint16_t* const a_row = p.A + static_cast<size_t>(min(lane, p.M - 1)) * p.lda;

    if (lane == 0) {
        for (uint32_t i = 0; i < kSwStages; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();

    const uint32_t first = s_begin + warp, mine = first < s_end ? (s_end - first + kSwWarps - 1) / kSwWarps : 0;
    const auto k_of = [&](uint32_t i) { return (first + i * kSwWarps) * kStageK; };
    const auto copy_weights = [&](uint32_t i) {   // (the barrier expects the activations' bytes too)
        if (i >= mine || lane != 0) return;
        const uint32_t k0 = k_of(i), at = i % kSwStages, bar = smem_u32(&full[warp][at]);
        mbar_arrive_expect_tx(bar, kSwBox + MP * min(kStageK, p.K - k0) * 2);
        box_load(smem_u32(boxes) + at * kSwBox, &map_w, bar, k0 / 2, n0);
    };
    const auto copy_acts = [&](uint32_t i) {
        if (i >= mine || lane >= MP) return;
        const uint32_t k0 = k_of(i), at = i % kSwStages;
        bulk_copy(smem_u32(acts) + (at * MP + lane) * kSwAPitch, a_row + k0, min(kStageK, p.K - k0) * 2, smem_u32(&full[warp][at]));
    };
    // Scales and zero points of rows 8 r + g and of columns 2 c + e's groups, asked for a stage ahead:
    // with two tokens both columns have the same slot, and so has a group of 64 or more with one.
    constexpr uint32_t kCols = MP == 1 && G == 32 ? 2 : 1;
    float sc[kFolds][4][kCols];
    uint32_t zp[kFolds][4][kCols];
    uint32_t p_at[4];   // of the row's groups
#pragma unroll
    for (uint32_t r = 0; r < 4; ++r) p_at[r] = min(n0 + 8 * r + g, p.N - 1);
    const bool pairs = groups % 2 == 0 && reinterpret_cast<uintptr_t>(p.scale) % 8 == 0;   // column pairs in one load
    const auto load_params = [&](uint32_t i) {
        if (i >= mine) return;
        const uint32_t g0 = k_of(i) / G;
#pragma unroll
        for (uint32_t f = 0; f < kFolds; ++f) {
            const uint32_t at = min(g0 + (f * kSlots + 2 * c / MP) * 32 / G, groups - kCols);
            if (kCols == 1 || pairs) {
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    const size_t from = static_cast<size_t>(p_at[r]) * groups + at;
                    if constexpr (kCols == 1) sc[f][r][0] = scale_of<F16>(p, from);
                    else {
                        const float2 v = p.scale_bytes == 4 ? *reinterpret_cast<const float2*>(p.scale + 4 * from)
                                                            : unpack2<F16>(*reinterpret_cast<const uint32_t*>(p.scale + 2 * from));
                        sc[f][r][0] = v.x, sc[f][r][kCols - 1] = v.y;
                    }
                    if (p.zeros) {
#pragma unroll
                        for (uint32_t e = 0; e < kCols; ++e) zp[f][r][e] = p.zeros[from + e];
                    }
                }
            } else {
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r)
#pragma unroll
                    for (uint32_t e = 0; e < kCols; ++e) {
                        const size_t from = static_cast<size_t>(p_at[r]) * groups + min(g0 + 2 * c + e, groups - 1);
                        sc[f][r][e] = scale_of<F16>(p, from);
                        zp[f][r][e] = p.zeros ? p.zeros[from] : 8u;
                    }
            }
        }
    };
#pragma unroll
    for (uint32_t f = 0; f < kFolds; ++f)
#pragma unroll
        for (uint32_t r = 0; r < 4; ++r)
#pragma unroll
            for (uint32_t e = 0; e < kCols; ++e) zp[f][r][e] = 8u;
#pragma unroll 1
    for (uint32_t i = 0; i < kSwStages - 1; ++i) copy_weights(i);
    load_params(0);
    if (p.early) grid_dependency_wait();
#pragma unroll 1
    for (uint32_t i = 0; i < kSwStages - 1; ++i) copy_acts(i);

    const uint32_t slot = g / MP;   // of this lane's column of the operand
    float acc[2][4] = {};
#pragma unroll 1
    for (uint32_t i = 0; i < mine; ++i) {
        const uint32_t at = i % kSwStages;
        if (!wait_warp(smem_u32(&full[warp][at]), (i / kSwStages) & 1, p.timeout_ns, &abort_flag)) break;
        // the slot before this one has been read by all lanes: the next copies may overwrite it
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        copy_weights(i + kSwStages - 1);
        copy_acts(i + kSwStages - 1);
        float2 cur[kFolds][4][kCols];
#pragma unroll
        for (uint32_t f = 0; f < kFolds; ++f)
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r)
#pragma unroll
                for (uint32_t e = 0; e < kCols; ++e) cur[f][r][e] = make_float2(sc[f][r][e], static_cast<float>(zp[f][r][e]));
        load_params(i + 1);
        const uint32_t chunks = (p.K - k_of(i)) / 32;   // past them activations and codes are 0
        const uint8_t* w = boxes + at * kSwBox + g * 128 + 4 * c;
        const uint8_t* a = acts + (at * MP + g % MP) * kSwAPitch + 16 * c;
#pragma unroll
        for (uint32_t f = 0; f < kFolds; ++f) {
            const uint32_t mine_ch = f * kSlots + slot;   // this lane's chunk
            const uint4 v = mine_ch < chunks ? *reinterpret_cast<const uint4*>(a + 64 * mine_ch) : make_uint4(0, 0, 0, 0);
            float mx = amax8<F16>(v);
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            const float2 du = down_up(fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2)));
            uint32_t b[4];
            float sum = acts8<F16>(v, du.x, b);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            float part[2][4] = {};
#pragma unroll
            for (uint32_t j = 0; j < kSlots; ++j) {
                const bool on = j == slot;
                const uint32_t b0 = on ? b[0] : 0u, b1 = on ? b[1] : 0u, b2 = on ? b[2] : 0u, b3 = on ? b[3] : 0u;
#pragma unroll
                for (uint32_t t = 0; t < 2; ++t) {
                    uint32_t f0[4], f1[4];
                    weights32(w + 2048 * t + (((f * kSlots + j) ^ g) << 4), f0, f1);
                    mma_f16(part[t], f0, b0, b1);
                    mma_f16(part[t], f1, b2, b3);
                }
            }
#pragma unroll
            for (uint32_t e = 0; e < 2; ++e) {   // column 2 c + e: its sum and scale are with lanes 4 (2 c + e) ..
                const float s = __shfl_sync(0xFFFFFFFFu, sum, 4 * (2 * c + e)), up = __shfl_sync(0xFFFFFFFFu, du.y, 4 * (2 * c + e));
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r)
                    acc[r / 2][2 * (r % 2) + e] = fold(acc[r / 2][2 * (r % 2) + e], part[r / 2][2 * (r % 2) + e], up, s, cur[f][r][kCols == 2 ? e : 0]);
            }
        }
    }

    // ---- sums of the warps and slots, then of the cluster's CTAs, in order
    __syncthreads();   // every warp is done with its ring, which the sums reuse
    float* const red = reinterpret_cast<float*>(smem);                // [warp][8 columns][kSwRedPitch]
    float* const sums = red + kSwWarps * 8 * kSwRedPitch;             // [token][kSwRedPitch]
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[(warp * 8 + 2 * c + (e & 1)) * kSwRedPitch + 16 * t + 8 * (e >> 1) + g] = acc[t][e];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < p.M * kSwRows; i += kSwThreads) {
        const uint32_t m = i / kSwRows, r = i % kSwRows;
        float v = 0.f;
#pragma unroll 8
        for (uint32_t w = 0; w < kSwWarps * kSlots; ++w) v += red[(w * MP + m) * kSwRedPitch + r];
        if (p.split > 1) sums[m * kSwRedPitch + r] = v;
        else if (n0 + r < p.N) p.C[static_cast<size_t>(m) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
    }
    if (p.split == 1) return;
    cluster_sync_all();
    for (uint32_t i = threadIdx.x + rank * kSwThreads; i < p.M * kSwRows; i += kSwThreads * p.split) {
        const uint32_t m = i / kSwRows, r = i % kSwRows;
        float v = 0.f;
        for (uint32_t q = 0; q < p.split; ++q) v += ld_dsmem_f32(smem_u32(sums + m * kSwRedPitch + r), q);
        if (n0 + r < p.N) p.C[static_cast<size_t>(m) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
    }
    cluster_sync_all();   // no CTA leaves while another still reads its sums
}

// --------------------------------------------------------------- more tokens --
// Warp (wn, wk): rows 32 wn of the tile's 128, half wk (4 chunks) of every stage's K. The rings
// are the CTA's: a box of codes, and one of 32 values of K of the tokens for each chunk (64-byte
// rows, with the 64-byte swizzle: no bank is hit twice), filled by a lane of warp 0 when all warps
// have read a slot.
constexpr uint32_t kTwThreads = 256, kTwRows = 128, kTwStages = 3, kTwBox = kTwRows * 128, kTwRedPitch = kTwRows + 4;
constexpr uint32_t tw_stage_bytes(uint32_t tok) { return kTwBox + tok * kStageK * 2; }
constexpr uint32_t tw_red_bytes(uint32_t tok) { return 2 * tok * kTwRedPitch * 4; }   // halves of K; the first becomes the CTA's sums
constexpr uint32_t tw_smem_bytes(uint32_t tok) {
    return 1024 + (kTwStages * tw_stage_bytes(tok) > tw_red_bytes(tok) ? kTwStages * tw_stage_bytes(tok) : tw_red_bytes(tok));
}

template <bool F16, uint32_t NT, uint32_t G>
__global__ void __launch_bounds__(kTwThreads, 2)
    w4_tile_kernel(const W4Args p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a) {
    constexpr uint32_t kTok = 8 * NT, kHalfGroups = kStageK / G / 2, kFold = G / 32, kStageBytes = tw_stage_bytes(kTok);
    constexpr bool kNatural = NT > 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kTwStages], empty[kTwStages];
    __shared__ int abort_flag;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, wn = warp & 3, wk = warp >> 2;
    const uint32_t rank = blockIdx.x % p.split, n0 = blockIdx.x / p.split * kTwRows, m0 = blockIdx.y * kTok;
    const uint32_t stages = (p.K + kStageK - 1) / kStageK, groups = p.K / G;
    const uint32_t s_begin = static_cast<uint32_t>(static_cast<uint64_t>(rank) * stages / p.split),
                   n_stages = static_cast<uint32_t>(static_cast<uint64_t>(rank + 1) * stages / p.split) - s_begin;
    const uint32_t tokens = min(kTok, p.M - m0), k_begin = s_begin * kStageK;
    const size_t row = min(n0 + 32 * wn + lane, p.N - 1);   // whose scales this lane loads

    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kTwStages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&empty[i]), 8);
        }
        abort_flag = 0;
        fence_barrier_init();
    }
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();

    const auto copy_weights = [&](uint32_t i) {   // (the barrier expects the activations' bytes too)
        const uint32_t bar = smem_u32(&full[i % kTwStages]);
        mbar_arrive_expect_tx(bar, kStageBytes);
        box_load(smem_u32(smem) + i % kTwStages * kStageBytes, &map_w, bar, (k_begin + i * kStageK) / 2, n0);
    };
    const auto copy_acts = [&](uint32_t i) {
        const uint32_t bar = smem_u32(&full[i % kTwStages]), to = smem_u32(smem) + i % kTwStages * kStageBytes + kTwBox;
#pragma unroll 1
        for (uint32_t ch = 0; ch < kChunks; ++ch) box_load(to + ch * kTok * 64, &map_a, bar, k_begin + i * kStageK + 32 * ch, m0);
    };
    // scales and zero points of this lane's row, of the groups of the warp's half, a stage ahead
    float sc[kHalfGroups];
    uint32_t zp[kHalfGroups];
    const auto load_params = [&](uint32_t i) {
        if (i >= n_stages) return;
        const uint32_t g0 = (k_begin + i * kStageK) / G + wk * kHalfGroups;
#pragma unroll
        for (uint32_t q = 0; q < kHalfGroups; ++q) {   // past the end of K activations are 0
            const size_t at = row * groups + min(g0 + q, groups - 1);
            sc[q] = scale_of<F16>(p, at);
            if (p.zeros) zp[q] = p.zeros[at];
        }
    };
#pragma unroll
    for (uint32_t q = 0; q < kHalfGroups; ++q) zp[q] = 8u;
    const uint32_t ahead = min(n_stages, kTwStages);
    if (threadIdx.x == 0)
        for (uint32_t i = 0; i < ahead; ++i) copy_weights(i);
    load_params(0);
    if (p.early) grid_dependency_wait();
    if (threadIdx.x == 0)
        for (uint32_t i = 0; i < ahead; ++i) copy_acts(i);

    float acc[2][NT][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.f;
#pragma unroll 1
    for (uint32_t i = 0; i < n_stages; ++i) {
        const uint32_t at = i % kTwStages, parity = (i / kTwStages) & 1;
        float cs[kHalfGroups];
        uint32_t cz[kHalfGroups];
#pragma unroll
        for (uint32_t q = 0; q < kHalfGroups; ++q) {
            cs[q] = sc[q];
            // 128 + z in BF16 (0x4300 + z), 1024 + z in FP16 (0x6400 + z), twice
            cz[q] = ((F16 ? 0x6400u : 0x4300u) + zp[q]) * 0x10001u;
        }
        load_params(i + 1);
        if (!wait_warp(smem_u32(&full[at]), parity, p.timeout_ns, &abort_flag)) break;
        const uint8_t* const w = smem + at * kStageBytes + (32 * wn + g) * 128 + 4 * c;
        const uint8_t* const a = smem + at * kStageBytes + kTwBox + 4 * wk * kTok * 64 + g * 64 + ((c ^ (g >> 1 & 3)) << 4);
#pragma unroll
        for (uint32_t q = 0; q < kHalfGroups; ++q) {
            uint32_t z[4];
            float f[4];
#pragma unroll
            for (uint32_t r = 0; r < 4; ++r) z[r] = __shfl_sync(0xFFFFFFFFu, cz[q], 8 * r + g), f[r] = __shfl_sync(0xFFFFFFFFu, cs[q], 8 * r + g);
            float part[2][NT][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n) part[t][n][0] = part[t][n][1] = part[t][n][2] = part[t][n][3] = 0.f;
#pragma unroll
            for (uint32_t ch = q * kFold; ch < (q + 1) * kFold; ++ch) {
                uint32_t x[4][4];
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) decode8<F16, kNatural>(*reinterpret_cast<const uint32_t*>(w + 1024 * r + (((4 * wk + ch) ^ g) << 4)), z[r], x[r]);
                uint32_t f0[2][4], f1[2][4];
#pragma unroll
                for (uint32_t t = 0; t < 2; ++t)
#pragma unroll
                    for (uint32_t r = 0; r < 2; ++r) f0[t][r] = x[2 * t + r][0], f0[t][2 + r] = x[2 * t + r][1], f1[t][r] = x[2 * t + r][2], f1[t][2 + r] = x[2 * t + r][3];
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n) {
                    uint4 b = *reinterpret_cast<const uint4*>(a + (ch * kTok + 8 * n) * 64);
                    if constexpr (!kNatural) b = make_uint4(prmt(b.x, b.z, 0x5410), prmt(b.x, b.z, 0x7632), prmt(b.y, b.w, 0x5410), prmt(b.y, b.w, 0x7632));
#pragma unroll
                    for (uint32_t t = 0; t < 2; ++t) {
                        mma_16816<F16>(part[t][n], f0[t], b.x, b.y);
                        mma_16816<F16>(part[t][n], f1[t], b.z, b.w);
                    }
                }
            }
#pragma unroll
            for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
                for (uint32_t r = 0; r < 4; ++r) {
                    acc[r / 2][n][2 * (r % 2)] = fmaf(f[r], part[r / 2][n][2 * (r % 2)], acc[r / 2][n][2 * (r % 2)]);
                    acc[r / 2][n][2 * (r % 2) + 1] = fmaf(f[r], part[r / 2][n][2 * (r % 2) + 1], acc[r / 2][n][2 * (r % 2) + 1]);
                }
        }
        // this slot has been read by all lanes of the warp; the one before it is refilled once all warps
        // are past it (by then most are, and warp 0 has a stage of its own left)
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[at]));
        if (warp == 0 && i > 0 && i - 1 + kTwStages < n_stages) {
            if (!wait_warp(smem_u32(&empty[(i - 1) % kTwStages]), ((i - 1) / kTwStages) & 1, p.timeout_ns, &abort_flag)) break;
            if (lane == 0) {
                copy_weights(i - 1 + kTwStages);
                copy_acts(i - 1 + kTwStages);
            }
            __syncwarp();
        }
    }

    // ---- sums of the halves, then of the cluster's CTAs, in order
    __syncthreads();   // every warp is done with the rings, which the sums reuse
    float* const red = reinterpret_cast<float*>(smem);   // [half][token][kTwRedPitch]
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wk * kTok + 8 * n + 2 * c + (e & 1)) * kTwRedPitch + 32 * wn + 16 * t + 8 * (e >> 1) + g] = acc[t][n][e];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < tokens * kTwRows; i += kTwThreads) {
        const uint32_t m = i / kTwRows, r = i % kTwRows;
        const float v = red[m * kTwRedPitch + r] + red[(kTok + m) * kTwRedPitch + r];
        if (p.split > 1) red[m * kTwRedPitch + r] = v;   // this thread's own element
        else if (n0 + r < p.N) p.C[static_cast<size_t>(m0 + m) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
    }
    if (p.split == 1) return;
    cluster_sync_all();
    for (uint32_t i = threadIdx.x + rank * kTwThreads; i < tokens * kTwRows; i += kTwThreads * p.split) {
        const uint32_t m = i / kTwRows, r = i % kTwRows;
        float v = 0.f;
        for (uint32_t q = 0; q < p.split; ++q) v += ld_dsmem_f32(smem_u32(red + m * kTwRedPitch + r), q);
        if (n0 + r < p.N) p.C[static_cast<size_t>(m0 + m) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
    }
    cluster_sync_all();   // no CTA leaves while another still reads its sums
}

// Launches `kernel` on clusters of a.split CTAs along x, as a programmatic dependent.
cudaError_t launch_clusters(void (*kernel)(const W4Args, const CUtensorMap, const CUtensorMap), const W4Args& a, const CUtensorMap& map_w,
                            const CUtensorMap& map_a, dim3 grid, uint32_t threads, uint32_t smem, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, map_w, map_a);
}

// CTAs per row tile: as many as the GPU holds at once, each with `least` stages or more.
uint32_t choose_split(uint64_t tiles, uint64_t slots, uint32_t stages, uint32_t least) {
    uint32_t split = 1;
    while (split < kMaxSplit && tiles * (split + 1) <= slots && stages >= least * (split + 1)) ++split;
    return split;
}

// The descriptors of a launch; false with a message.
struct Maps {
    CUtensorMap w, a;
    bool make(const W4Args& p, uint32_t rows, uint32_t tokens, std::string* err) {
        std::memset(&a, 0, sizeof a);
        return tensor_map_2d(p.W, p.N, p.K / 2, p.K / 2, 1, rows, 128, &w, err) &&
               (tokens == 0 || tensor_map_2d(p.A, p.M, p.K, 2ull * p.lda, 2, tokens, 32, &a, err));
    }
};

template <bool F16, uint32_t MP, uint32_t G>
cudaError_t launch_stream(W4Args a, int sms, cudaStream_t s, std::string* err) {
    const uint32_t tiles = (a.N + kSwRows - 1) / kSwRows, smem = sw_smem_bytes(MP);
    const uint32_t fit = 228u * 1024 / (smem + 1024), resident = fit < 4 ? fit : 4;
    // a stage a warp at least
    a.split = choose_split(tiles, static_cast<uint64_t>(sms) * resident, (a.K + kStageK - 1) / kStageK, kSwWarps);
    Maps m;
    if (!m.make(a, kSwRows, 0, err)) return cudaErrorInvalidValue;
    return launch_clusters(w4_stream_kernel<F16, MP, G>, a, m.w, m.a, dim3(tiles * a.split, 1, 1), kSwThreads, smem, s);
}
template <bool F16, uint32_t NT, uint32_t G>
cudaError_t launch_tile(W4Args a, int sms, cudaStream_t s, std::string* err) {
    const uint32_t tiles = (a.N + kTwRows - 1) / kTwRows, tok_tiles = (a.M + 8 * NT - 1) / (8 * NT);
    a.split = choose_split(static_cast<uint64_t>(tiles) * tok_tiles, 2ull * sms, (a.K + kStageK - 1) / kStageK, 2);
    Maps m;
    if (!m.make(a, kTwRows, 8 * NT, err)) return cudaErrorInvalidValue;
    return launch_clusters(w4_tile_kernel<F16, NT, G>, a, m.w, m.a, dim3(tiles * a.split, tok_tiles, 1), kTwThreads, tw_smem_bytes(8 * NT), s);
}
template <bool F16, uint32_t G>
cudaError_t launch_tokens(const W4Args& a, int sms, cudaStream_t s, std::string* err) {
    return a.M == 1    ? launch_stream<F16, 1, G>(a, sms, s, err)
           : a.M == 2  ? launch_stream<F16, 2, G>(a, sms, s, err)
           : a.M <= 8  ? launch_tile<F16, 1, G>(a, sms, s, err)
           : a.M <= 16 ? launch_tile<F16, 2, G>(a, sms, s, err)
                       : launch_tile<F16, 4, G>(a, sms, s, err);
}
template <bool F16>
cudaError_t launch_group(const W4Args& a, uint32_t group, int sms, cudaStream_t s, std::string* err) {
    return group == 32   ? launch_tokens<F16, 32>(a, sms, s, err)
           : group == 64 ? launch_tokens<F16, 64>(a, sms, s, err)
                         : launch_tokens<F16, 128>(a, sms, s, err);
}

}  // namespace

int launch_w4(const W4Operands& o, int sms, uint64_t timeout_ns, uint32_t flags, cudaStream_t s, std::string* err) {
    const W4Args a{static_cast<const uint16_t*>(o.A), static_cast<const uint8_t*>(o.W), static_cast<const uint8_t*>(o.scale),
                   static_cast<const uint8_t*>(o.zeros), static_cast<uint16_t*>(o.C), o.lda, o.ldc, o.M, o.N, o.K,
                   o.scale_f32 ? 4u : 2u, 1, flags & W8A16_FLAG_PDL ? 1u : 0u, timeout_ns};
    const cudaError_t e = o.act_dtype == W8A16_ACT_F16 ? launch_group<true>(a, o.group, sms, s, err) : launch_group<false>(a, o.group, sms, s, err);
    if (e != cudaSuccess) {
        cudaGetLastError();
        if (err->empty()) *err = std::string("4-bit product launch failed: ") + cudaGetErrorString(e);
        return W8A16_ERR_LAUNCH;
    }
    return W8A16_OK;
}

cudaError_t w4_status_read(StatusWord* out, bool clear, cudaStream_t s) {
    DeviceStatus st;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&st, g_w4_status, sizeof st, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    out->code = st.code;
    out->where = st.where;
    out->detail = st.detail;
    if (clear) {
        const DeviceStatus zero{0, 0, 0};
        e = cudaMemcpyToSymbolAsync(g_w4_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace w8a16

// Products with 4-bit weights and group scales, for a few tokens.
//
// Mathematics.  C[m][n] = sum_g s[n][g] * ( sum_{k in g} A[m][k] (code[n][k] - z[n][g]) ).
// Codes become operands of the tensor cores exactly, products add in FP32, a group's sum is
// scaled once, in FP32: no weight is rounded. Bytes are HBM's to bound (0.5 a weight and the
// scales); the integer pipe, at one instruction in two cycles, bounds the decoding, so the three
// kernels below spend as few integer operations on a word of eight codes as they can.
//
// Layout (of the two kernels on mma.sync). m16n8k16 with 16 weight rows as M and 8 columns as N. A lane's 32-bit word holds 8
// codes of a row, and masks take the pairs (k, k + 4) out of it; the order of a
// contraction's index being free, the activations are paired the same way, and weights never
// move between lanes.
//
// Work. A CTA takes the rows of a tile and a contiguous range of K's stages; where tiles alone do
// not fill the GPU, the CTAs of a cluster share K. Codes are copied by TMA, whole boxes, into rings.
// (Bulk copies of a row a lane are issued lane by lane and cost a warp some 400 instructions a
// stage.) The sums of a CTA's warps, and those of a cluster's CTAs, are added in a fixed order.
//   1 or 2 tokens (w4_stream_kernel). Every warp has a ring and a part of K of its own. The bits of
//     a nibble, as FP16, are the subnormal number c 2^-24 (or 16 c 2^-24 four bits higher): four
//     masks and a shift decode a word. The activations become FP16, times a power of two that
//     puts the largest of a chunk of 32 at 2^14, and a sixteenth of that where the codes come times 16, the
//     odd elements (exact down to 2^-27 of the largest for BF16, whose 8 bits end at FP16's 2^-24, and 2^-24 for
//     FP16; 2^-31 and 2^-28 for even ones). The zero point leaves the product: with S = sum c a,
//     T = sum a, sum (c - z) a = S - z T. Columns that tokens leave unused take other chunks of K
//     (the operand is zero outside a column's own), so 8 (4) chunks need one set of sums and one
//     folding.
//   3 to 8, and more of a small product (w4_rows_kernel). The columns are the tokens, so a warp
//     would normalise a chunk of activations for 32 rows only: they stay as they are and codes
//     become code - z, exactly (nibbles under the exponent of 128 in BF16, 1024 in FP16; 128 + z,
//     1024 + z comes off).
//   more (w4_tc_kernel). m16n8k16 would be issued once for every 8 tokens: tcgen05 instead, 128 rows
//     of decoded weights in TMEM against 16 or 32 tokens.
// Where the steps are (us, BF16, 32-bit scales, zero points, groups of 128):
//                        1024x4096   4096x4096   12288x4096   28672x8192   (N x K)
//     2 tokens  stream      3.1         5.4         10.4         32.7
//               rows        3.5         6.7         13.3         37.1
//     8 tokens  rows        3.8         7.1         13.8         40.4
//               tc          6.1         8.7         18.0         46.3
//     16        rows        4.4         7.5         18.9         59.4
//               tc          6.4         9.1         18.2         47.4
// (12288 rows are 1.3 rounds of tiles there.)
// Bound by: the stream of bytes at large sizes (28672x8192, one token: 132 MB in 33 us, 4.1 TB/s with groups
// of 32, 4.6 with groups of 128), the time to the first bytes and the join at small ones. What
// counts for it is bytes in flight: rings of 192 KB an SM without a barrier between warps stream
// twice as fast as rings of 96 KB behind a CTA's barriers did. With more tokens (14336x5120, 32
// tokens: 21.7 us) decoding, the products' hand-over and the folding take turns: a copy of the
// kernel took 4.5 us less without the decoding, 2.2 without the join, 10 in all with neither these
// nor products.
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
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
    return mbar_wait_for(bar, parity, timeout_ns, abort_flag, &g_w4_status, 1);
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
// The cluster's (2 or more) CTAs each hold sums [token][ROWS + 4] at `sums`, of TOK tokens at most:
// adds them in rank order, each CTA a share of the elements, and writes C's rows m0 .. and columns
// n0 ... All peers are read at once: a load from one takes as long as from eight. C is written after
// the last arrival, whose release would otherwise wait for the stores.
template <bool F16, uint32_t ROWS, uint32_t THREADS, uint32_t TOK>
__device__ __forceinline__ void join_cluster(const W4Args& p, const float* sums, uint32_t rank, uint32_t m0, uint32_t tokens, uint32_t n0) {
    constexpr uint32_t kIters = ((TOK * (ROWS / 4) + 1) / 2 + THREADS - 1) / THREADS;
    cluster_sync_all();
    const uint32_t items = tokens * (ROWS / 4), share = (items + p.split - 1) / p.split, end = min(items, (rank + 1) * share);
    uint32_t out[kIters][2];
#pragma unroll
    for (uint32_t it = 0; it < kIters; ++it) {
        const uint32_t i = rank * share + it * THREADS + threadIdx.x;
        if (i >= end) continue;
        const uint32_t at = smem_u32(sums + i / (ROWS / 4) * (ROWS + 4) + i % (ROWS / 4) * 4);
        float4 v[kMaxSplit];
#pragma unroll
        for (uint32_t q = 0; q < kMaxSplit; ++q)
            if (q < p.split) v[q] = ld_dsmem_v4f32(at, q);
        float4 x = v[0];
#pragma unroll
        for (uint32_t q = 1; q < kMaxSplit; ++q)
            if (q < p.split) x.x += v[q].x, x.y += v[q].y, x.z += v[q].z, x.w += v[q].w;
        out[it][0] = pack2<F16>(x.x, x.y), out[it][1] = pack2<F16>(x.z, x.w);
    }
    __syncwarp();
    cluster_arrive_release();
#pragma unroll
    for (uint32_t it = 0; it < kIters; ++it) {
        const uint32_t i = rank * share + it * THREADS + threadIdx.x;
        if (i >= end) continue;
        const uint32_t r = i % (ROWS / 4) * 4;
        uint16_t* const c = p.C + static_cast<size_t>(m0 + i / (ROWS / 4)) * p.ldc + n0 + r;
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e)
            if (n0 + r + e < p.N) c[e] = static_cast<uint16_t>(out[it][e / 2] >> (16 * (e & 1)));
    }
    cluster_wait();   // no CTA leaves while another still reads its sums
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
            const uint32_t at = min(g0 + (f * kSlots + 2 * c / MP) * 32 / G, groups - kCols);   // (past the end of K sums are 0)
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
        if (!wait_warp(smem_u32(&full[warp][at]), (i / kSwStages) & 1, p.timeout_ns, &abort_flag)) {
            ring_drain<kSwStages>(full[warp], i, min(i + kSwStages - 1, mine), p.timeout_ns, &g_w4_status, 3);
            break;
        }
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
    join_cluster<F16, kSwRows, kSwThreads, MP>(p, sums, rank, 0, p.M, n0);
}

// --------------------------------------------- 3 to 8 tokens, and small products --
// As the kernel above, a ring of codes and a part of K for every warp; fragments of the
// activations are loaded from global memory a stage ahead. 32 rows a warp and four stages of 4 KB on
// 3 CTAs an SM; 64 rows and two stages of 8 KB read the activations half as often and took 0.97 (BF16)
// and 0.88 (FP16) of the time at 28672x8192 and 8 tokens, but 1.3 at 1024x4096.
constexpr uint32_t kRwWarps = 4, kRwThreads = 32 * kRwWarps, kRwTiles = 2, kRwRows = 16 * kRwTiles;
constexpr uint32_t kRwBox = kRwRows * 128, kRwRedPitch = kRwRows + 4;
template <uint32_t NT>
struct RwCfg {
    static constexpr uint32_t kTok = 8 * NT, kStages = NT == 1 ? 4 : 6, kResident = NT == 1 ? 3 : 2, kSmem = 1024 + kRwWarps * kStages * kRwBox;
    static_assert((kRwWarps + 1) * kTok * kRwRedPitch * 4 <= kSmem - 1024, "the sums reuse the rings");
};

// Scales and zero points of COUNT consecutive groups from `at`; `wide`: they are aligned to be read at once.
template <bool F16, uint32_t COUNT>
__device__ __forceinline__ void load_run(const W4Args& p, size_t at, uint32_t valid, bool wide, float (&sc)[COUNT], uint32_t (&zp)[(COUNT + 3) / 4]) {
    if (wide) {
        if (p.scale_bytes == 4) {
            if constexpr (COUNT >= 4) {
#pragma unroll
                for (uint32_t i = 0; i < COUNT / 4; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(p.scale + 4 * (at + 4 * i));
                    sc[4 * i] = v.x, sc[4 * i + 1] = v.y, sc[4 * i + 2] = v.z, sc[4 * i + 3] = v.w;
                }
            } else if constexpr (COUNT == 2) {
                const float2 v = *reinterpret_cast<const float2*>(p.scale + 4 * at);
                sc[0] = v.x, sc[1] = v.y;
            } else {
                sc[0] = *reinterpret_cast<const float*>(p.scale + 4 * at);
            }
        } else {
            if constexpr (COUNT >= 4) {
#pragma unroll
                for (uint32_t i = 0; i < COUNT / 4; ++i) {
                    const uint2 v = *reinterpret_cast<const uint2*>(p.scale + 2 * (at + 4 * i));
                    const float2 a = unpack2<F16>(v.x), b = unpack2<F16>(v.y);
                    sc[4 * i] = a.x, sc[4 * i + 1] = a.y, sc[4 * i + 2] = b.x, sc[4 * i + 3] = b.y;
                }
            } else if constexpr (COUNT == 2) {
                const float2 v = unpack2<F16>(*reinterpret_cast<const uint32_t*>(p.scale + 2 * at));
                sc[0] = v.x, sc[1] = v.y;
            } else {
                sc[0] = scale_of<F16>(p, at);
            }
        }
        if (p.zeros) {
            if constexpr (COUNT >= 4) {
#pragma unroll
                for (uint32_t i = 0; i < COUNT / 4; ++i) zp[i] = *reinterpret_cast<const uint32_t*>(p.zeros + at + 4 * i);
            } else if constexpr (COUNT == 2) {
                zp[0] = *reinterpret_cast<const uint16_t*>(p.zeros + at);
            } else {
                zp[0] = p.zeros[at];
            }
        }
        return;
    }
#pragma unroll
    for (uint32_t i = 0; i < COUNT; ++i) {   // past the end of K sums are 0: the row's last scale does
        const size_t from = at + min(i, valid - 1);
        sc[i] = scale_of<F16>(p, from);
        if (p.zeros) zp[i / 4] = (i % 4 ? zp[i / 4] : 0u) | static_cast<uint32_t>(p.zeros[from]) << (8 * (i % 4));
    }
}
// Whether every run of COUNT groups that starts at a multiple of COUNT is whole and aligned.
template <uint32_t COUNT>
__device__ __forceinline__ bool runs_wide(const W4Args& p, uint32_t groups) {
    return groups % COUNT == 0 && reinterpret_cast<uintptr_t>(p.scale) % (COUNT >= 4 ? 4 * p.scale_bytes : COUNT * p.scale_bytes) == 0;
}

// 8 codes -> (code - z), pairs (0,4) (1,5) (2,6) (3,7).
template <bool F16>
__device__ __forceinline__ void decode_pairs(uint32_t q, uint32_t z, uint32_t (&o)[4]) {
    if constexpr (F16) {   // 1024 + c, and 1024 + 16 c for what stands four bits higher
        const uint32_t h = q >> 8, za = (0xE400u + z) * 0x10001u, zb = (0xD400u + 16u * z) * 0x10001u, one = 0x3C003C00u, sixteenth = 0x2C002C00u;
        const uint32_t x[4] = {(q & 0x000F000Fu) | 0x64006400u, (q & 0x00F000F0u) | 0x64006400u, (h & 0x000F000Fu) | 0x64006400u, (h & 0x00F000F0u) | 0x64006400u};
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(x[i]), "r"(i & 1 ? sixteenth : one), "r"(i & 1 ? zb : za));
    } else {
        const uint32_t zb = (0x4300u + z) * 0x10001u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = (q >> (4 * i) & 0x000F000Fu) | 0x43004300u;
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x), "r"(zb));
        }
    }
}

template <bool F16, uint32_t NT, uint32_t G>
__global__ void __launch_bounds__(kRwThreads, RwCfg<NT>::kResident) w4_rows_kernel(const W4Args p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap) {
    constexpr uint32_t kGroups = kStageK / G, kGroupChunks = G / 32, kRwStages = RwCfg<NT>::kStages, kTok = RwCfg<NT>::kTok;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[kRwWarps][kRwStages];
    __shared__ int abort_flag;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint32_t rank = blockIdx.x % p.split, n0 = blockIdx.x / p.split * kRwRows, m0 = blockIdx.y * kTok,
                   tokens = min(kTok, p.M - m0);
    const uint32_t stages = (p.K + kStageK - 1) / kStageK, groups = p.K / G;
    const uint32_t s_begin = static_cast<uint32_t>(static_cast<uint64_t>(rank) * stages / p.split),
                   s_end = static_cast<uint32_t>(static_cast<uint64_t>(rank + 1) * stages / p.split);
    uint8_t* const boxes = smem + warp * kRwStages * kRwBox;
    const uint16_t* a_row[NT];
#pragma unroll
    for (uint32_t n = 0; n < NT; ++n) a_row[n] = p.A + static_cast<size_t>(min(m0 + 8 * n + g, p.M - 1)) * p.lda + 8 * c;

    if (lane == 0) {
        for (uint32_t i = 0; i < kRwStages; ++i) mbar_init(smem_u32(&full[warp][i]), 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) abort_flag = 0;
    if (!p.early) grid_dependency_wait();
    __syncthreads();

    const uint32_t first = s_begin + warp, mine = first < s_end ? (s_end - first + kRwWarps - 1) / kRwWarps : 0;
    const auto k_of = [&](uint32_t i) { return (first + i * kRwWarps) * kStageK; };
    const auto copy_weights = [&](uint32_t i) {
        if (i >= mine || lane != 0) return;
        const uint32_t at = i % kRwStages, bar = smem_u32(&full[warp][at]);
        mbar_arrive_expect_tx(bar, kRwBox);
        box_load(smem_u32(boxes) + at * kRwBox, &map_w, bar, k_of(i) / 2, n0);
    };
    uint4 acts[NT][kChunks];
    const auto load_acts = [&](uint32_t i) {
        if (i >= mine) return;
        const uint32_t k0 = k_of(i), chunks = (p.K - k0) / 32;
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (uint32_t ch = 0; ch < kChunks; ++ch) acts[n][ch] = ch < chunks ? *reinterpret_cast<const uint4*>(a_row[n] + k0 + 32 * ch) : make_uint4(0, 0, 0, 0);
    };
    // scales and zero points of the tile's row `lane`, a stage ahead
    const bool wide = runs_wide<kGroups>(p, groups);
    float sc[kGroups];
    uint32_t zp[(kGroups + 3) / 4];
    const size_t p_row = static_cast<size_t>(min(n0 + lane, p.N - 1)) * groups;
    const auto load_params = [&](uint32_t i) {
        if (i >= mine) return;
        const uint32_t g0 = k_of(i) / G;
        load_run<F16, kGroups>(p, p_row + g0, min(kGroups, groups - g0), wide, sc, zp);
    };
#pragma unroll
    for (uint32_t q = 0; q < (kGroups + 3) / 4; ++q) zp[q] = 0x08080808u;
#pragma unroll 1
    for (uint32_t i = 0; i < kRwStages; ++i) copy_weights(i);
    load_params(0);
    if (p.early) grid_dependency_wait();
    load_acts(0);

    float acc[kRwTiles][NT][4] = {};
#pragma unroll 1
    for (uint32_t i = 0; i < mine; ++i) {
        const uint32_t at = i % kRwStages;
        uint4 b[NT][kChunks];
        float cs[kGroups];
        uint32_t cz[(kGroups + 3) / 4];
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (uint32_t ch = 0; ch < kChunks; ++ch) b[n][ch] = acts[n][ch];
#pragma unroll
        for (uint32_t q = 0; q < kGroups; ++q) cs[q] = sc[q];
#pragma unroll
        for (uint32_t q = 0; q < (kGroups + 3) / 4; ++q) cz[q] = zp[q];
        load_params(i + 1);
        load_acts(i + 1);
        if (!wait_warp(smem_u32(&full[warp][at]), (i / kRwStages) & 1, p.timeout_ns, &abort_flag)) {
            ring_drain<kRwStages>(full[warp], i, min(i + kRwStages, mine), p.timeout_ns, &g_w4_status, 3);
            break;
        }
        const uint8_t* const w = boxes + at * kRwBox + g * 128 + 4 * c;
#pragma unroll
        for (uint32_t q = 0; q < kGroups; ++q) {
            float part[kRwTiles][NT][4] = {};
            uint32_t z[kRwTiles][2];
#pragma unroll
            for (uint32_t t = 0; t < kRwTiles; ++t)
#pragma unroll
                for (uint32_t r = 0; r < 2; ++r)
                    z[t][r] = __shfl_sync(0xFFFFFFFFu, cz[q / 4] >> (8 * (q % 4)), 16 * t + 8 * r + g) & 0xFFu;
#pragma unroll
            for (uint32_t ch = q * kGroupChunks; ch < (q + 1) * kGroupChunks; ++ch) {
                uint32_t y[NT][4];
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n) {
                    const uint4 v = b[n][ch];
                    y[n][0] = prmt(v.x, v.z, 0x5410), y[n][1] = prmt(v.x, v.z, 0x7632), y[n][2] = prmt(v.y, v.w, 0x5410), y[n][3] = prmt(v.y, v.w, 0x7632);
                }
#pragma unroll
                for (uint32_t t = 0; t < kRwTiles; ++t) {
                    uint32_t x[2][4];
#pragma unroll
                    for (uint32_t r = 0; r < 2; ++r) decode_pairs<F16>(*reinterpret_cast<const uint32_t*>(w + 2048 * t + 1024 * r + ((ch ^ g) << 4)), z[t][r], x[r]);
                    const uint32_t f0[4] = {x[0][0], x[1][0], x[0][1], x[1][1]}, f1[4] = {x[0][2], x[1][2], x[0][3], x[1][3]};
#pragma unroll
                    for (uint32_t n = 0; n < NT; ++n) {
                        mma_16816<F16>(part[t][n], f0, y[n][0], y[n][1]);
                        mma_16816<F16>(part[t][n], f1, y[n][2], y[n][3]);
                    }
                }
            }
#pragma unroll
            for (uint32_t t = 0; t < kRwTiles; ++t)
#pragma unroll
                for (uint32_t r = 0; r < 2; ++r) {
                    const float f = __shfl_sync(0xFFFFFFFFu, cs[q], 16 * t + 8 * r + g);
#pragma unroll
                    for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
                        for (uint32_t e = 2 * r; e < 2 * r + 2; ++e) acc[t][n][e] = fmaf(f, part[t][n][e], acc[t][n][e]);
                }
        }
        // all lanes have read the slot: it may be overwritten
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        copy_weights(i + kRwStages);
    }

    // Dependents come in only now: on the SMs whose CTAs were done first they took part of what the rest
    // runs on (12288x4096, 8 tokens, call behind call: 12.9 us against 11.2).
    grid_launch_dependents();
    // ---- sums of the warps, then of the cluster's CTAs, in order
    __syncthreads();   // every warp is done with its ring, which the sums reuse
    float* const red = reinterpret_cast<float*>(smem);                       // [warp][token][kRwRedPitch]
    float* const sums = red + kRwWarps * kTok * kRwRedPitch;             // [token][kRwRedPitch]
#pragma unroll
    for (uint32_t t = 0; t < kRwTiles; ++t)
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[(warp * kTok + 8 * n + 2 * c + (e & 1)) * kRwRedPitch + 16 * t + 8 * (e >> 1) + g] = acc[t][n][e];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < tokens * kRwRows; i += kRwThreads) {
        const uint32_t m = i / kRwRows, r = i % kRwRows;
        float v = 0.f;
#pragma unroll
        for (uint32_t w = 0; w < kRwWarps; ++w) v += red[(w * kTok + m) * kRwRedPitch + r];
        if (p.split > 1) sums[m * kRwRedPitch + r] = v;
        else if (n0 + r < p.N) p.C[static_cast<size_t>(m0 + m) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
    }
    if (p.split > 1) join_cluster<F16, kRwRows, kRwThreads, kTok>(p, sums, rank, m0, tokens, n0);
}

// --------------------------------------------------------------- more tokens --
// D[row][token] of a chunk of kCk values of K (no more than a group) is one run of tcgen05.mma
// with the decoded weights in TMEM as A (lane = weight row, column j = values 2 j and 2 j + 1)
// and the activations, as TMA wrote them, as B. Warps 0-3 decode, a thread a row, and add
// scale * D to the row's sums; warp 4 copies and issues. Two slots of TMEM: while a chunk's
// product runs the next one is decoded, and a slot is free again once its sums have been read. The
// two chunks of a group of 128 add to one D, which is read once.
constexpr uint32_t kTcThreads4 = 160, kTcRows4 = 128, kTcStageK = 128, kTcWBytes = kTcRows4 * kTcStageK / 2, kTcResident = 4;
constexpr uint32_t kTcTmemCols = 128, kTcRedPitch = kTcRows4 + 4;
template <uint32_t NT, uint32_t G>
struct TcCfg {
    static constexpr uint32_t kTok = NT;                                  // the product's columns
    static constexpr uint32_t kCk = G < 64 ? G : 64, kPerStage = kTcStageK / kCk, kACols = kCk / 2;
    static constexpr uint32_t kStageGroups = kTcStageK / G;
    static constexpr bool kWhole = G == kTcStageK;                        // a stage is a group: its chunks share a product
    static constexpr uint32_t kActBytes = kTok * 128;                       // 64 values of K
    static constexpr uint32_t kStageBytes = kTcWBytes + 2 * kActBytes;
    static constexpr uint32_t kStages = NT > 16 ? 3 : 4;
    static constexpr uint32_t kSmem = 1024 + kStages * kStageBytes;
    static_assert(2 * (kACols + kTok) <= kTcTmemCols && kPerStage % 2 == 0 && (!kWhole || kPerStage == 2), "slots");
    static_assert(kTok * kTcRedPitch * 4 <= kStages * kStageBytes, "the sums reuse the ring");
    static_assert(kTcResident * (kSmem + 2048) <= 228 * 1024, "CTAs of an SM");
};

// 8 codes of a row -> (code - z), pairs (0,1) (2,3) (4,5) (6,7). The bits of a nibble go under the
// exponent of 128 (BF16) or, the even one of a pair, 1024 and the odd one, times 16, 1024 (FP16: no
// shift); what comes off is exact in both.
template <bool F16>
__device__ __forceinline__ uint32_t zero_operand(uint32_t z) {
    return F16 ? (0xE400u + z) | (0xD400u + 16u * z) << 16    // -(1024 + z), -(64 + z)
               : (0x4300u + z) * 0x10001u;                    // 128 + z
}
template <bool F16>
__device__ __forceinline__ void decode_row8(uint32_t q, uint32_t zb, uint32_t* o) {
    const uint32_t odd = F16 ? 0x64646464u : q >> 4;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        if constexpr (F16) {
            const uint32_t x = prmt(q, odd, 0x4040u + 0x0101u * i) & 0x64F0640Fu;
            asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[i]) : "r"(x), "r"(0x2C003C00u), "r"(zb));   // (1/16, 1)
        } else {
            const uint32_t x = (prmt(q, odd, 0x4400u + 0x1111u * i) & 0x000F000Fu) | 0x43004300u;
            asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x), "r"(zb));
        }
    }
}

template <bool F16, uint32_t NT, uint32_t G>
__global__ void __launch_bounds__(kTcThreads4, kTcResident)
    w4_tc_kernel(const W4Args p, const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a) {
    using C = TcCfg<NT, G>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ uint64_t full[C::kStages], a_full[2], d_full[2], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 4) {   // first of all: the SM starts no other CTA until the permit is back (0.5 us a CTA)
        tmem_alloc(smem_u32(&tmem_slot), kTcTmemCols);
        tmem_relinquish();
    } else if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_a);
        for (uint32_t i = 0; i < C::kStages; ++i) mbar_init(smem_u32(&full[i]), 1);
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&a_full[i]), 4);
            mbar_init(smem_u32(&d_full[i]), 1);
        }
        mbar_init(smem_u32(&drain), 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    const uint32_t rank = blockIdx.x % p.split, n0 = blockIdx.x / p.split * kTcRows4, m0 = blockIdx.y * C::kTok;
    const uint32_t stages = (p.K + kTcStageK - 1) / kTcStageK, groups = p.K / G;
    const uint32_t s_begin = static_cast<uint32_t>(static_cast<uint64_t>(rank) * stages / p.split),
                   n_stages = static_cast<uint32_t>(static_cast<uint64_t>(rank + 1) * stages / p.split) - s_begin;
    const uint32_t tokens = min(C::kTok, p.M - m0), k_begin = s_begin * kTcStageK;

    if (!p.early) grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_slot;
    uint64_t acc[C::kTok / 2] = {};   // FP32 pairs

    if (warp == 4) {
        // The whole warp goes through the loop, on broadcast addresses, and one elected lane issues: so
        // descriptors are formed in uniform registers (a lane of its own took 430 cycles for 4 products).
        const uint32_t base = __shfl_sync(0xFFFFFFFFu, smem_u32(smem), 0), tmu = __shfl_sync(0xFFFFFFFFu, tm, 0);
        const uint64_t desc = smem_desc_kmajor_sw128(base + kTcWBytes);
        const bool elected = elect_one();
        const auto copy_weights = [&](uint32_t s) {   // (the barrier expects the activations' bytes too)
            const uint32_t bar = smem_u32(&full[s % C::kStages]);
            mbar_arrive_expect_tx(bar, C::kStageBytes);
            box_load(base + s % C::kStages * C::kStageBytes, &map_w, bar, (k_begin + s * kTcStageK) / 2, n0);
        };
        const auto copy_acts = [&](uint32_t s) {
            const uint32_t bar = smem_u32(&full[s % C::kStages]), to = base + s % C::kStages * C::kStageBytes + kTcWBytes;
            box_load(to, &map_a, bar, k_begin + s * kTcStageK, m0);
            box_load(to + C::kActBytes, &map_a, bar, k_begin + s * kTcStageK + 64, m0);
        };
        const uint32_t ahead = min(n_stages, C::kStages);
        if (elected)
            for (uint32_t s = 0; s < ahead; ++s) copy_weights(s);
        if (p.early) grid_dependency_wait();
        if (elected)
            for (uint32_t s = 0; s < ahead; ++s) copy_acts(s);
        __syncwarp();
        constexpr uint32_t kIdesc = idesc_bf16_f32(128, C::kTok) & ~(F16 ? (1u << 7 | 1u << 10) : 0u);
        uint32_t issued = ahead;   // stages
        bool ok = true;
        uint32_t s = 0;
#pragma unroll 1
        for (; ok && s < n_stages; ++s) {
            const uint32_t at = s % C::kStages;
#pragma unroll
            for (uint32_t j = 0; j < C::kPerStage; ++j) {
                const uint32_t i = s * C::kPerStage + j, slot = j & 1;
                ok = ok && wait_warp(smem_u32(&a_full[slot]), (i >> 1) & 1, p.timeout_ns, &abort_flag);
                if (j == 0) ok = ok && wait_warp(smem_u32(&full[at]), (s / C::kStages) & 1, p.timeout_ns, &abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t k = j * C::kCk;
                const uint64_t b = desc + at * (C::kStageBytes >> 4) + ((k / 64 * C::kActBytes + k % 64 * 2) >> 4);
                const uint32_t tA = tmu + slot * C::kACols, tD = tmu + 2 * C::kACols + (C::kWhole ? s & 1 : slot) * C::kTok;
                if (elected) {
#pragma unroll
                    for (uint32_t e = 0; e < C::kCk / 16; ++e) tc_mma_a_tmem(tD, tA + 8 * e, b + 2 * e, kIdesc, e || (C::kWhole && j) ? 1u : 0u);
                    tc_commit(smem_u32(&d_full[slot]));
                }
                __syncwarp();
                // The stage before this one has been decoded; once its last product is done it is refilled.
                if (j == 0 && s > 0 && issued < n_stages) {
                    ok = wait_warp(smem_u32(&d_full[1]), ((i - 1) >> 1) & 1, p.timeout_ns, &abort_flag);
                    if (!ok) break;
                    if (elected) {
                        copy_weights(issued);
                        copy_acts(issued);
                    }
                    ++issued;
                    __syncwarp();
                }
            }
        }
        // Nothing of this CTA's is in flight when it leaves: products, and (after a wait that gave up) copies.
        if (elected) {
            int none = 0;   // not the abort flag, which may be raised: these waits have their own limit
            tc_commit(smem_u32(&drain));
            mbar_wait_for(smem_u32(&drain), 0, p.timeout_ns, &none, &g_w4_status, 2);
            if (!ok) ring_drain<C::kStages>(full, s > 0 ? s - 1 : 0, issued, p.timeout_ns, &g_w4_status, 3);
        }
        __syncwarp();
    } else {
        const uint32_t row = threadIdx.x, lanes = (warp * 32) << 16;
        const size_t p_row = static_cast<size_t>(min(n0 + row, p.N - 1)) * groups;
        const bool wide = runs_wide<C::kStageGroups>(p, groups);
        float sc[C::kStageGroups];
        uint32_t zp = 0x08080808u;
        const auto load_params = [&](uint32_t s) {   // a stage ahead
            if (s >= n_stages) return;
            const uint32_t g0 = (k_begin + s * kTcStageK) / G;
            uint32_t z[1] = {zp};
            load_run<F16, C::kStageGroups>(p, p_row + g0, min(C::kStageGroups, groups - g0), wide, sc, z);
            zp = z[0];
        };
        load_params(0);
        if (p.early) grid_dependency_wait();   // the limit of the waits below starts behind the previous kernel: they are for its outputs
        float f[2] = {};   // scales of the products in flight
        const auto done = [&](uint32_t i, uint32_t slot) {   // the product of chunk i, in this slot
            const bool ok = wait_warp(smem_u32(&d_full[slot]), (i >> 1) & 1, p.timeout_ns, &abort_flag);
            tc_fence_after();
            return ok;
        };
        const auto fold = [&](uint32_t slot, float scale) {   // sums += scale * D
            const uint64_t ff = pack_f32x2(scale, scale);
#pragma unroll
            for (uint32_t t = 0; t < C::kTok; t += 16) {
                float d[2][8];
                const uint32_t tD = tm + 2 * C::kACols + slot * C::kTok + lanes + t;
                tmem_ld_32x32b_x8(tD, d[0]);
                tmem_ld_32x32b_x8(tD + 8, d[1]);
                tc_wait_ld();
#pragma unroll
                for (uint32_t e = 0; e < 8; ++e)
                    acc[t / 2 + e] = fma_f32x2(ff, pack_f32x2(d[e / 4][e % 4 * 2], d[e / 4][e % 4 * 2 + 1]), acc[t / 2 + e]);
            }
        };
        bool ok = true;
#pragma unroll 1
        for (uint32_t s = 0; ok && s < n_stages; ++s) {
            const uint32_t at = s % C::kStages;
            float cs[C::kStageGroups];
            uint32_t cz[C::kStageGroups];
#pragma unroll
            for (uint32_t q = 0; q < C::kStageGroups; ++q) cs[q] = sc[q], cz[q] = zero_operand<F16>(zp >> (8 * q) & 0xFFu);
            load_params(s + 1);
            ok = wait_warp(smem_u32(&full[at]), (s / C::kStages) & 1, p.timeout_ns, &abort_flag);
            const uint8_t* const w = smem + at * C::kStageBytes + row * 64;
#pragma unroll
            for (uint32_t j = 0; j < C::kPerStage; ++j) {
                const uint32_t i = s * C::kPerStage + j, slot = j & 1, q = j * C::kCk / G;
                uint4 v = *reinterpret_cast<const uint4*>(w + (((j * C::kCk / 32) ^ (row >> 1 & 3)) << 4));
                if (i >= 2) ok = ok && done(i - 2, slot);
                if (!ok) break;
                if (!C::kWhole && i >= 2) fold(slot, f[slot]);
                if (C::kWhole && j == 1 && s > 0) fold(s & 1 ^ 1, f[0]);
                const uint32_t tA = tm + slot * C::kACols + lanes;
#pragma unroll
                for (uint32_t h = 0; h < C::kCk / 32; ++h) {
                    if (h > 0) v = *reinterpret_cast<const uint4*>(w + (((j * C::kCk / 32 + h) ^ (row >> 1 & 3)) << 4));
                    uint32_t o[16];
                    decode_row8<F16>(v.x, cz[q], o);
                    decode_row8<F16>(v.y, cz[q], o + 4);
                    decode_row8<F16>(v.z, cz[q], o + 8);
                    decode_row8<F16>(v.w, cz[q], o + 12);
                    tmem_st_32x32b_x16(tA + 16 * h, o);
                }
                if (!C::kWhole || j == 1) f[C::kWhole ? 0 : slot] = cs[q];
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&a_full[slot]));
            }
        }
        if (n_stages > 0) {   // the last two chunks
            const uint32_t n = n_stages * C::kPerStage;
            ok = ok && done(n - 2, 0);
            if (!C::kWhole && ok) fold(0, f[0]);
            ok = ok && done(n - 1, 1);
            if (ok) fold(C::kWhole ? n_stages & 1 ^ 1 : 1, f[C::kWhole ? 0 : 1]);
        }
    }

    // ---- the rows' sums, then those of the cluster's CTAs, in order
    tc_fence_before();
    __syncthreads();   // products and copies are done: the sums reuse the ring, and TMEM goes back before any wait for a peer
    tc_fence_after();
    if (warp == 4) tmem_dealloc(tm, kTcTmemCols);
    // Dependents come in here (every CTA has had its TMEM): let in at the start they take the places of CTAs that
    // are done (28672x8192, 32 tokens: 60 us for 50), not before the end 12288x4096 takes 20 for 18.
    grid_launch_dependents();
    float* const red = reinterpret_cast<float*>(smem);   // [token][kTcRedPitch]
    if (warp < 4) {
#pragma unroll
        for (uint32_t t = 0; t < C::kTok; t += 2) {
            const float2 x = unpack_f32x2(acc[t / 2]);
            red[t * kTcRedPitch + threadIdx.x] = x.x, red[(t + 1) * kTcRedPitch + threadIdx.x] = x.y;
        }
    }
    if (p.split > 1) {
        join_cluster<F16, kTcRows4, kTcThreads4, C::kTok>(p, red, rank, m0, tokens, n0);
        return;
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < tokens * kTcRows4; i += kTcThreads4) {
        const uint32_t m = i / kTcRows4, r = i % kTcRows4;
        if (n0 + r < p.N) p.C[static_cast<size_t>(m0 + m) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(red[m * kTcRedPitch + r], 0.f));
    }
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
    cfg.numAttrs = a.split > 1 ? 2 : 1;   // (a cluster of one CTA starts 11 ns after another: 600 CTAs in 0.7 us, 0.1 without)
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
    bool make(const W4Args& p, uint32_t rows, uint32_t bytes, uint32_t tokens, uint32_t ks, std::string* err) {
        std::memset(&a, 0, sizeof a);
        return tensor_map_2d(p.W, p.N, p.K / 2, p.K / 2, 1, rows, bytes, &w, err) &&
               (tokens == 0 || tensor_map_2d(p.A, p.M, p.K, 2ull * p.lda, 2, tokens, ks, &a, err));
    }
};

template <bool F16, uint32_t MP, uint32_t G>
cudaError_t launch_stream(W4Args a, int sms, cudaStream_t s, std::string* err) {
    const uint32_t tiles = (a.N + kSwRows - 1) / kSwRows, smem = sw_smem_bytes(MP);
    const uint32_t fit = 228u * 1024 / (smem + 1024), resident = fit < 4 ? fit : 4;
    // a stage a warp at least
    a.split = choose_split(tiles, static_cast<uint64_t>(sms) * resident, (a.K + kStageK - 1) / kStageK, kSwWarps);
    Maps m;
    if (!m.make(a, kSwRows, 128, 0, 0, err)) return cudaErrorInvalidValue;
    return launch_clusters(w4_stream_kernel<F16, MP, G>, a, m.w, m.a, dim3(tiles * a.split, 1, 1), kSwThreads, smem, s);
}
template <bool F16, uint32_t NT, uint32_t G>
cudaError_t launch_rows(W4Args a, int sms, cudaStream_t s, std::string* err) {
    const uint32_t tiles = (a.N + kRwRows - 1) / kRwRows, tok_tiles = (a.M + 8 * NT - 1) / (8 * NT);
    a.split = choose_split(static_cast<uint64_t>(tiles) * tok_tiles, static_cast<uint64_t>(sms) * RwCfg<NT>::kResident, (a.K + kStageK - 1) / kStageK, kRwWarps);
    Maps m;
    if (!m.make(a, kRwRows, 128, 0, 0, err)) return cudaErrorInvalidValue;
    return launch_clusters(w4_rows_kernel<F16, NT, G>, a, m.w, m.a, dim3(tiles * a.split, tok_tiles, 1), kRwThreads, RwCfg<NT>::kSmem, s);
}
template <bool F16, uint32_t NT, uint32_t G>
cudaError_t launch_tc(W4Args a, int sms, cudaStream_t s, std::string* err) {
    using C = TcCfg<NT, G>;
    const uint32_t tiles = (a.N + kTcRows4 - 1) / kTcRows4, tok_tiles = (a.M + NT - 1) / NT;
    a.split = choose_split(static_cast<uint64_t>(tiles) * tok_tiles, static_cast<uint64_t>(kTcResident) * sms, (a.K + kTcStageK - 1) / kTcStageK, 2);
    Maps m;
    if (!m.make(a, kTcRows4, kTcStageK / 2, C::kTok, 64, err)) return cudaErrorInvalidValue;
    return launch_clusters(w4_tc_kernel<F16, NT, G>, a, m.w, m.a, dim3(tiles * a.split, tok_tiles, 1), kTcThreads4, C::kSmem, s);
}
// More than 8 tokens by w4_rows_kernel, in tiles of 16: one tile where the rows' tiles run at once and the
// product is small, more where it is smaller still. us, rows against tc (BF16, 32-bit scales, zero
// points, groups of 128):
//   16 tokens: 256x8192 4.4, 8.9; 4096x4096 7.5, 9.1; 6144x4096 10.8, 10.6; 9728x4096 13.6, 16.7; 4096x14336 21.4,
//     23.3; past the rule 8192x8192 21.7, 19.5; 5120x13824 36.0, 24.0; 12288x4096 (a second round of tiles) 18.9, 18.2
//   32: 256x8192 5.1, 9.7; 1024x4096 5.2, 7.0; 4096x2048 6.7, 7.4; 2044x5632 9.2, 9.9 (groups of 32: 10.1, 12.8); past
//     it 4096x4096 10.5, 10.1; 4096x8192 19.7, 16.3
//   64: 1024x4096 7.3, 8.3; past it 4096x2048 12.0, 9.3
bool small_for_rows(const W4Args& a, int sms) {
    const uint64_t weights = static_cast<uint64_t>(a.N) * a.K, tok_tiles = (a.M + 15) / 16;
    if (tok_tiles > 1) return tok_tiles <= 65535 && weights < (3ull << 23) && weights * tok_tiles < 3ull << 23;
    return (a.N + kRwRows - 1) / kRwRows <= static_cast<uint64_t>(sms) * RwCfg<2>::kResident && weights < 1ull << 26;
}
template <bool F16, uint32_t G>
cudaError_t launch_tokens(const W4Args& a, int sms, cudaStream_t s, std::string* err) {
    return a.M == 1    ? launch_stream<F16, 1, G>(a, sms, s, err)
           : a.M == 2  ? launch_stream<F16, 2, G>(a, sms, s, err)
           : a.M <= 8  ? launch_rows<F16, 1, G>(a, sms, s, err)
           : small_for_rows(a, sms) ? launch_rows<F16, 2, G>(a, sms, s, err)
           : a.M <= 16 ? launch_tc<F16, 16, G>(a, sms, s, err)
                       : launch_tc<F16, 32, G>(a, sms, s, err);
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

// Products with 4-bit weights and group scales, for a few tokens.
//
// Mathematics.  C[m][n] = sum_g s[n][g] * ( sum_{k in g} A[m][k] (code[n][k] - z[n][g]) ).
// The integers code - z lie in [-15, 15] and are exact in BF16 and FP16, so the inner
// sums are exact products added in FP32 on the tensor cores, and the group's scale is
// applied once per group in FP32: no weight is ever rounded.
//
// Layout. m16n8k16 products with 16 weight rows as M and 8 tokens as N, 32 rows a
// warp. A 32-bit word holds 8 codes; masking it (and its shifts by 4, 8, 12) against
// 0x000F000F and placing the nibbles under the exponent of 128 (BF16) or 1024 (FP16)
// gives the pairs (k, k+4) as 128 + code, from which 128 + z is subtracted exactly.
// The order of a contraction's index is free, so the activations are paired the same way
// (two byte permutations per pair of words) and the weights never move between lanes.
//
// Work. A CTA takes 64 (or 128) weight rows and a contiguous range of 256-K stages; W, A,
// scales and zeros of a stage are copied asynchronously into a ring. Its 8 warps split
// rows and the stage's K; their sums, and those of the CTAs of a cluster that share the
// rows, are added in a fixed order. Bound by HBM: 0.5 byte a weight plus the scales.
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "w8a16_cluster.cuh"
#include "w8a16_kv.cuh"

namespace w8a16 {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kStageK = 256;             // codes of a row per stage: 128 bytes
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
};

template <uint32_t NT, uint32_t G>
struct W4Cfg {
    static constexpr uint32_t kWN = NT == 1 ? 2 : 4, kWK = 8 / kWN;    // warps along rows and along a stage's K
    static constexpr uint32_t kRows = 32 * kWN;
    static constexpr uint32_t kTok = 8 * NT;
    static constexpr uint32_t kStages = NT == 2 ? 3 : 4;
    static constexpr uint32_t kGroups = kStageK / G;                    // per stage
    static constexpr uint32_t kWarpK = kStageK / kWK;                   // codes of a row per warp and stage
    // scale words per row: FP32 aligned; 16-bit and zero bytes in the aligned words that cover them
    static constexpr uint32_t kScaleWords = kGroups;                    // >= kGroups / 2 + 1
    static constexpr uint32_t kZeroWords = kGroups / 4 + 2;
    static constexpr uint32_t kWBytes = kRows * kStageK / 2, kABytes = kTok * kStageK * 2;
    static constexpr uint32_t kSBytes = kRows * kScaleWords * 4, kZBytes = kRows * kZeroWords * 4;
    static constexpr uint32_t kStageBytes = kWBytes + kABytes + kSBytes + kZBytes;
    static constexpr uint32_t kRedPitch = kRows + 4;
    static constexpr uint32_t kRedBytes = kWK * kTok * kRedPitch * 4;
    static constexpr uint32_t kSmem = kStages * kStageBytes > kRedBytes ? kStages * kStageBytes : kRedBytes;
    static constexpr uint32_t kCtasPerSm = NT == 1 ? 3 : NT == 2 ? 2 : 1;
    static_assert(kGroups >= 2, "16-bit scale words");
};

__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, uint32_t bytes, uint32_t piece) {
    if (piece == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 codes -> code - z as pairs (k0,k4) (k1,k5) (k2,k6) (k3,k7). zb: (128 + z) twice in
// BF16, or (1024 + z) twice in FP16.
template <bool F16>
__device__ __forceinline__ void decode8(uint32_t q, uint32_t zb, uint32_t (&o)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = ((q >> (4 * i)) & 0x000F000Fu) | (F16 ? 0x64006400u : 0x43004300u);
        if constexpr (F16) asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x), "r"(zb));
        else asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(x), "r"(zb));
    }
}

template <bool F16, uint32_t NT, uint32_t G>
__global__ void __launch_bounds__(kThreads, (W4Cfg<NT, G>::kCtasPerSm)) w4_kernel(const W4Args p) {
    using C = W4Cfg<NT, G>;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const uint32_t wn = warp % C::kWN, wk = warp / C::kWN;
    const uint32_t rank = blockIdx.x % p.split, tile = blockIdx.x / p.split;
    const uint32_t n0 = tile * C::kRows, m0 = blockIdx.y * C::kTok;
    const uint32_t stages = (p.K + kStageK - 1) / kStageK;
    const uint32_t s_begin = static_cast<uint32_t>(static_cast<uint64_t>(rank) * stages / p.split),
                   s_end = static_cast<uint32_t>(static_cast<uint64_t>(rank + 1) * stages / p.split);
    const uint32_t groups = p.K / G;
    const uint32_t tokens = min(C::kTok, p.M - m0);
    const uint32_t base = smem_u32(smem);

    if (!p.early) grid_dependency_wait();

    const auto copy_weights = [&](uint32_t s) {
        if (s < s_end) {
            const uint32_t slot = base + (s - s_begin) % C::kStages * C::kStageBytes;
#pragma unroll
            for (uint32_t i = tid; i < C::kRows * 8; i += kThreads) {   // 16-byte chunks, xor-swizzled by row
                const uint32_t r = i >> 3, ch = i & 7;
                const uint32_t k = s * kStageK + ch * 32;
                const bool take = n0 + r < p.N && k < p.K;
                const uint8_t* src = take ? p.W + static_cast<size_t>(n0 + r) * (p.K / 2) + k / 2 : p.W;
                copy_async(slot + r * 128 + ((ch ^ (r & 7)) << 4), src, take ? 16u : 0u, 16);
            }
            // scales and zeros: the aligned words that cover a row's groups of this stage
            const uint32_t g0 = s * C::kGroups;
            const uint32_t sw = p.scale_bytes == 4 ? C::kGroups : C::kGroups / 2 + 1;
            for (uint32_t i = tid; i < C::kRows * sw; i += kThreads) {
                const uint32_t r = i / sw, w = i % sw;
                const size_t first = (static_cast<size_t>(n0 + r) * groups + g0) * p.scale_bytes;
                const size_t at = (first & ~static_cast<size_t>(3)) + 4 * w;
                const size_t end = (static_cast<size_t>(n0 + r) * groups + min(g0 + C::kGroups, groups)) * p.scale_bytes;
                const uint32_t bytes = n0 + r < p.N && at < end ? static_cast<uint32_t>(min(end - at, static_cast<size_t>(4))) : 0u;
                copy_async(slot + C::kWBytes + C::kABytes + (r * C::kScaleWords + w) * 4, bytes ? p.scale + at : p.scale, bytes, 4);
            }
            if (p.zeros) {
                constexpr uint32_t zw = C::kZeroWords;
                for (uint32_t i = tid; i < C::kRows * zw; i += kThreads) {
                    const uint32_t r = i / zw, w = i % zw;
                    const size_t first = static_cast<size_t>(n0 + r) * groups + g0;
                    const size_t at = (first & ~static_cast<size_t>(3)) + 4 * w;
                    const size_t end = static_cast<size_t>(n0 + r) * groups + min(g0 + C::kGroups, groups);
                    const uint32_t bytes = n0 + r < p.N && at < end ? static_cast<uint32_t>(min(end - at, static_cast<size_t>(4))) : 0u;
                    copy_async(slot + C::kWBytes + C::kABytes + C::kSBytes + (r * zw + w) * 4, bytes ? p.zeros + at : p.zeros, bytes, 4);
                }
            }
        }
    };
    const auto copy_acts = [&](uint32_t s) {
        if (s < s_end) {
            const uint32_t slot = base + (s - s_begin) % C::kStages * C::kStageBytes + C::kWBytes;
            for (uint32_t i = tid; i < C::kTok * 32; i += kThreads) {   // tokens past M: zero
                const uint32_t t = i >> 5, ch = i & 31;
                const uint32_t k = s * kStageK + ch * 8;
                const bool take = t < tokens && k < p.K;
                const uint16_t* src = take ? p.A + static_cast<size_t>(m0 + t) * p.lda + k : p.A;
                copy_async(slot + t * 512 + ((ch ^ ((t & 1) << 2)) << 4), src, take ? 16u : 0u, 16);
            }
        }
    };
    if (p.early) {
        for (uint32_t i = 0; i < C::kStages - 1; ++i) copy_weights(s_begin + i);
        grid_dependency_wait();
        for (uint32_t i = 0; i < C::kStages - 1; ++i) {
            copy_acts(s_begin + i);
            cp_async_commit();   // the first group holds all weights: stages then complete in order
        }
    } else {
        for (uint32_t i = 0; i < C::kStages - 1; ++i) {
            copy_weights(s_begin + i);
            copy_acts(s_begin + i);
            cp_async_commit();
        }
    }
    grid_launch_dependents();

    float acc[2][NT][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n) acc[t][n][0] = acc[t][n][1] = acc[t][n][2] = acc[t][n][3] = 0.f;

    for (uint32_t s = s_begin; s < s_end; ++s) {
        cp_async_wait_group<C::kStages - 2>();
        __syncthreads();   // the stage has landed for everyone, and the slot refilled below is free
        copy_weights(s + C::kStages - 1);
        copy_acts(s + C::kStages - 1);
        cp_async_commit();
        const uint8_t* slot = smem + (s - s_begin) % C::kStages * C::kStageBytes;
        const uint8_t* sa = slot + C::kWBytes;
        const uint8_t* ss = sa + C::kABytes;
        const uint8_t* sz = ss + C::kSBytes;
        constexpr uint32_t kBlocks = C::kWarpK / 32;                    // 32-code chunks of the warp
        constexpr uint32_t kPerGroup = G / 32 < kBlocks ? G / 32 : kBlocks;
#pragma unroll
        for (uint32_t b0 = 0; b0 < kBlocks; b0 += kPerGroup) {
            const uint32_t ch0 = wk * kBlocks + b0, gi = ch0 * 32 / G;   // the group within the stage
            float sc[4];
            uint32_t zb[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t row = wn * 32 + 8 * r + g;
                const size_t first = static_cast<size_t>(n0 + row) * groups + s * C::kGroups;
                if (p.scale_bytes == 4) {
                    sc[r] = *reinterpret_cast<const float*>(ss + (row * C::kScaleWords + gi) * 4);
                } else {
                    const uint32_t h = *reinterpret_cast<const uint16_t*>(ss + row * C::kScaleWords * 4 + ((first * 2) & 3) + 2 * gi);
                    sc[r] = unpack2<F16>(h).x;
                }
                const uint32_t z = p.zeros ? sz[row * C::kZeroWords * 4 + (first & 3) + gi] : 8u;
                // 128 + z in BF16 (0x4300 + z), 1024 + z in FP16 (0x6400 + z): z sits in the low mantissa bits
                zb[r] = ((F16 ? 0x6400u : 0x4300u) + z) * 0x10001u;
            }
            float part[2][NT][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n) part[t][n][0] = part[t][n][1] = part[t][n][2] = part[t][n][3] = 0.f;
#pragma unroll
            for (uint32_t b = 0; b < kPerGroup; ++b) {
                const uint32_t ch = ch0 + b;
                uint32_t w[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const uint32_t row = wn * 32 + 8 * r + g;
                    decode8<F16>(*reinterpret_cast<const uint32_t*>(slot + row * 128 + ((ch ^ (row & 7)) << 4) + 4 * c), zb[r], w[r]);
                }
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n) {
                    const uint32_t tok = 8 * n + g, ach = 4 * ch + c;
                    const uint4 a = *reinterpret_cast<const uint4*>(sa + tok * 512 + ((ach ^ ((tok & 1) << 2)) << 4));
                    const uint32_t x0 = prmt(a.x, a.z, 0x5410), x1 = prmt(a.x, a.z, 0x7632), x2 = prmt(a.y, a.w, 0x5410),
                                   x3 = prmt(a.y, a.w, 0x7632);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        const uint32_t f0[4] = {w[2 * t][0], w[2 * t + 1][0], w[2 * t][1], w[2 * t + 1][1]};
                        const uint32_t f1[4] = {w[2 * t][2], w[2 * t + 1][2], w[2 * t][3], w[2 * t + 1][3]};
                        mma_16816<F16>(part[t][n], f0, x0, x1);
                        mma_16816<F16>(part[t][n], f1, x2, x3);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[t][n][e] = fmaf(sc[2 * t + (e >> 1)], part[t][n][e], acc[t][n][e]);
        }
    }
    cp_async_wait_group<0>();
    __syncthreads();

    // ---- sums of the warps along K, then of the cluster's CTAs, in order
    float* red = reinterpret_cast<float*>(smem);   // [kWK][kTok][kRedPitch]
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (uint32_t n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                red[(wk * C::kTok + 8 * n + 2 * c + (e & 1)) * C::kRedPitch + wn * 32 + 16 * t + 8 * (e >> 1) + g] = acc[t][n][e];
    __syncthreads();
    const auto cta_sum = [&](uint32_t tok, uint32_t r) {
        float v = red[tok * C::kRedPitch + r];
#pragma unroll
        for (uint32_t w = 1; w < C::kWK; ++w) v += red[(w * C::kTok + tok) * C::kRedPitch + r];
        return v;
    };
    if (p.split == 1) {
        for (uint32_t i = tid; i < tokens * C::kRows; i += kThreads) {
            const uint32_t tok = i / C::kRows, r = i % C::kRows;
            if (n0 + r < p.N) p.C[static_cast<size_t>(m0 + tok) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(cta_sum(tok, r), 0.f));
        }
        return;
    }
    for (uint32_t i = tid; i < tokens * C::kRows; i += kThreads) {
        const uint32_t tok = i / C::kRows, r = i % C::kRows;
        red[tok * C::kRedPitch + r] = cta_sum(tok, r);   // each thread reads and writes its own elements
    }
    cluster_sync_all();
    for (uint32_t i = tid + rank * kThreads; i < tokens * C::kRows; i += kThreads * p.split) {
        const uint32_t tok = i / C::kRows, r = i % C::kRows;
        float v = 0.f;
        for (uint32_t q = 0; q < p.split; ++q) v += ld_dsmem_f32(base + (tok * C::kRedPitch + r) * 4, q);
        if (n0 + r < p.N) p.C[static_cast<size_t>(m0 + tok) * p.ldc + n0 + r] = static_cast<uint16_t>(pack2<F16>(v, 0.f));
    }
    cluster_sync_all();   // no CTA leaves while another still reads its sums
}

template <bool F16, uint32_t NT, uint32_t G>
cudaError_t launch(W4Args a, int sms, bool early, cudaStream_t s) {
    using C = W4Cfg<NT, G>;
    cudaError_t e = cudaFuncSetAttribute(w4_kernel<F16, NT, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    const uint32_t tiles = (a.N + C::kRows - 1) / C::kRows, tok_tiles = (a.M + C::kTok - 1) / C::kTok;
    const uint32_t stages = (a.K + kStageK - 1) / kStageK;
    // as many CTAs per row tile as fill the GPU once, each with at least two stages
    const uint64_t slots = static_cast<uint64_t>(sms) * C::kCtasPerSm;
    uint32_t split = 1;
    while (split < kMaxSplit && static_cast<uint64_t>(tiles) * tok_tiles * (split + 1) <= slots && stages >= 2 * (split + 1)) ++split;
    a.split = split;
    a.early = early;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(tiles * split, tok_tiles, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, w4_kernel<F16, NT, G>, a);
}

template <bool F16, uint32_t NT>
cudaError_t launch_group(const W4Args& a, uint32_t group, int sms, bool early, cudaStream_t s) {
    return group == 32   ? launch<F16, NT, 32>(a, sms, early, s)
           : group == 64 ? launch<F16, NT, 64>(a, sms, early, s)
                         : launch<F16, NT, 128>(a, sms, early, s);
}
template <bool F16>
cudaError_t launch_tokens(const W4Args& a, uint32_t group, int sms, bool early, cudaStream_t s) {
    return a.M <= 8    ? launch_group<F16, 1>(a, group, sms, early, s)
           : a.M <= 16 ? launch_group<F16, 2>(a, group, sms, early, s)
                       : launch_group<F16, 4>(a, group, sms, early, s);
}

}  // namespace

int launch_w4(const W4Operands& o, int sms, uint32_t flags, cudaStream_t s, std::string* err) {
    const W4Args a{static_cast<const uint16_t*>(o.A), static_cast<const uint8_t*>(o.W), static_cast<const uint8_t*>(o.scale),
                   static_cast<const uint8_t*>(o.zeros), static_cast<uint16_t*>(o.C), o.lda, o.ldc, o.M, o.N, o.K,
                   o.scale_f32 ? 4u : 2u, 1, 0};
    const bool early = (flags & W8A16_FLAG_PDL) != 0;
    const cudaError_t e = o.act_dtype == W8A16_ACT_F16 ? launch_tokens<true>(a, o.group, sms, early, s)
                                                       : launch_tokens<false>(a, o.group, sms, early, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        *err = std::string("4-bit product launch failed: ") + cudaGetErrorString(e);
        return W8A16_ERR_LAUNCH;
    }
    return W8A16_OK;
}

}  // namespace w8a16

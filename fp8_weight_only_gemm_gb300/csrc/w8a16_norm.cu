// The norms around a block with its gate, its residual scale and the quantiser of the next
// product's activations, one pass over a row:
//     t = norm(x; post_weight, post_bias)  or  x
//     h = residual + scale * gate * t
//     y = norm(h; weight, bias),  in the activations' type or as E4M3 codes with a scale per 128 of K
// RMS norm: x / sqrt(mean(x^2) + eps) * w. Layer norm: (x - mean) / sqrt(mean((x - mean)^2) + eps) * w + b,
// with the mean taken first: squares of values far from 0 would cancel.
//
// Work. Everything between the loads and the stores is FP32 in registers: a row belongs to as many warps as hold
// it in VPT vectors of 8 elements a thread, x and residual are read once and all at once, h and y are written once.
// y comes from h before its rounding. A group of 128 is 16 lanes' vectors, so its maximum is four shuffles.
// A row's sums cross its warps through shared memory, one barrier a sum.
//
// Bound by: many rows, by HBM: 8192 of 8192 with both norms take 92 us, 5.8 TB/s, 87 % of a copy's rate. Rows brought into a ring
// ahead of a block that goes through them took 138: blocks of a row each have more rows under way. Fewer, shorter and quantised rows
// stay further from it (4096 of 4096 with both norms 25.5 us, 79 %; 4096 of 5120 with an FP32 residual, quantised, 52.7, 66 %; 1974 of 4048, two
// layer norms, 21, 46 %; 2145 of 1672, the same, 9.6, 34 %): a block holds one row, and no load runs under the barriers of its sums, two for a
// layer norm. One token of 4096: 1.8 us, the launch and one chain of loads and sums.
#include <cuda_runtime.h>

#include <cstring>
#include <string>
#include <type_traits>

#include "w8a16_kv.cuh"

namespace w8a16 {
namespace {

constexpr uint32_t kWarpRows = 8;    // rows of a block whose rows are a warp each

struct NormArgs {
    w8a16_norm_t n;
    uint32_t vectors;     // of a row: H / 8
    uint32_t gate_every;  // rows that share a gate row
    bool early;           // weights may be asked for before the previous kernel is done
};

// 8 elements as FP32, two a register pair: all arithmetic is on pairs.
struct Eight {
    uint64_t p[4];
};
template <bool F16>
__device__ __forceinline__ Eight unpack8(const uint4& q) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    Eight v;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<F16>(w[e]);
        v.p[e] = pack_f32x2(f.x, f.y);
    }
    return v;
}
__device__ __forceinline__ uint4 load16(const void* p) { return *reinterpret_cast<const uint4*>(p); }
// What is read once stays out of L1: the weights are there.
__device__ __forceinline__ uint4 load_once(const void* p) {
    uint4 q;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "l"(p) : "memory");
    return q;
}
// Elements from `at` on, of the activations' type or FP32.
template <bool F16>
__device__ __forceinline__ Eight load8(const void* base, bool f32, int64_t at) {
    if (!f32) return unpack8<F16>(load16(static_cast<const uint16_t*>(base) + at));
    const ulonglong2* const from = reinterpret_cast<const ulonglong2*>(static_cast<const float*>(base) + at);
    const ulonglong2 a = from[0], b = from[1];
    return {{a.x, a.y, b.x, b.y}};
}
template <bool F16>
__device__ __forceinline__ void store8(void* base, bool f32, int64_t at, const Eight& v) {
    if (f32) {
        ulonglong2* const to = reinterpret_cast<ulonglong2*>(static_cast<float*>(base) + at);
        to[0] = make_ulonglong2(v.p[0], v.p[1]), to[1] = make_ulonglong2(v.p[2], v.p[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_f32x2(v.p[e]);
            w[e] = pack2<F16>(f.x, f.y);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ uint64_t both(float x) { return pack_f32x2(x, x); }

// The sum over a row's threads, for all of them. WARP: the row is one warp's. `turn`: alternates between the two
// halves of `sh`, so that one barrier a sum is enough.
template <bool WARP>
__device__ __forceinline__ float row_sum(float x, float (&sh)[2][32], uint32_t& turn) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    if constexpr (WARP) return x;
    float* const at = sh[turn];
    turn ^= 1;
    const uint32_t warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0) at[threadIdx.x >> 5] = x;
    __syncthreads();
    x = (threadIdx.x & 31) < warps ? at[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
    return x;
}

// The row's 1 / sqrt(mean square + eps) and, layer norm, v <- v - mean, v being this thread's vectors of it (0 past its end).
template <bool LAYER, bool WARP, uint32_t VPT>
__device__ __forceinline__ float moments(const NormArgs& p, Eight (&v)[VPT], uint32_t tid, uint32_t threads, float (&sh)[2][32], uint32_t& turn) {
    const float inv_h = 1.f / static_cast<float>(p.n.H);
    const uint64_t one = both(1.f);
    if constexpr (LAYER) {
        uint64_t s = 0;
#pragma unroll
        for (uint32_t i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) s = fma_f32x2(v[i].p[e], one, s);
        const float2 f = unpack_f32x2(s);
        const uint64_t less = both(-row_sum<WARP>(f.x + f.y, sh, turn) * inv_h);
#pragma unroll
        for (uint32_t i = 0; i < VPT; ++i)
            if (tid + i * threads < p.vectors)
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i].p[e] = fma_f32x2(v[i].p[e], one, less);
    }
    uint64_t s = 0;
#pragma unroll
    for (uint32_t i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fma_f32x2(v[i].p[e], v[i].p[e], s);
    const float2 f = unpack_f32x2(s);
    return rsqrtf(row_sum<WARP>(f.x + f.y, sh, turn) * inv_h + p.n.eps);
}

// Four codes of x times f.
__device__ __forceinline__ uint32_t encode4(const float* x, float f) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1] * f), "f"(x[0] * f));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x[3] * f), "f"(x[2] * f));
    return a | (static_cast<uint32_t>(b) << 16);
}
// The codes of 8 quotients y / s, each rounded to FP32 first, with s = mx / 448 and mx the largest |y| of the group. Products with the
// reciprocal 1 / s, itself off by 2^-24, taken 2^-21 smaller and 2^-21 larger: their own rounding and the quotient's included
// (2^-24 each) they lie on both sides of it, and codes are monotone, so where the two have one code it is the quotient's. Where they
// have not (a quotient next to the middle between two codes) and where s has few bits or none, it is divided. A scale of 0: codes 0; NaN
// stays NaN. (us, 4096 rows of 5120 with an FP32 residual 52, with a division for each value 55; 8192 of 8192 90 and 111.)
__device__ __forceinline__ uint2 encode8(float (&y)[8], float mx, float s) {
    const float inv = __frcp_rn(s), below = inv * (1.f - 0x1p-21f), above = inv * (1.f + 0x1p-21f);
    uint2 codes = make_uint2(encode4(y, below), encode4(y + 4, below));
    if (__builtin_expect(mx < 1e-30f || codes.x != encode4(y, above) || codes.y != encode4(y + 4, above), 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = s > 0.f || y[e] != y[e] ? __fdiv_rn(y[e], s) : 0.f;
        codes = make_uint2(encode4(y, 1.f), encode4(y + 4, 1.f));
    }
    return codes;
}

// WARP: a warp a row, kWarpRows rows a block. Else a block of up to MAXT threads a row. RF32: the residual is FP32.
template <bool F16, bool RF32, bool LAYER, bool WARP, uint32_t VPT, uint32_t MAXT>
__global__ void __launch_bounds__(MAXT) norm_kernel(const NormArgs p) {
    __shared__ float sh[2][32];
    const uint32_t threads = WARP ? 32u : blockDim.x, tid = WARP ? threadIdx.x & 31u : threadIdx.x;
    const uint32_t m = WARP ? blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    if (p.early) {
        const uint32_t bytes = p.n.weight_f32 ? 4u : 2u;
        const void* const all[4] = {p.n.weight, p.n.bias, p.n.post_weight, p.n.post_bias};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            for (uint32_t at = 8 * bytes * tid; all[k] != nullptr && at < bytes * p.n.H; at += 8 * bytes * threads)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const uint8_t*>(all[k]) + at));
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (m >= p.n.M) return;   // whole warps
    uint32_t turn = 0;

    // x and residual as they lie in memory, all asked for at once
    uint4 xq[VPT], rq[VPT][RF32 ? 2 : 1];
    const uint16_t* const x = static_cast<const uint16_t*>(p.n.x) + static_cast<int64_t>(m) * p.n.x_stride;
    const uint8_t* const res = static_cast<const uint8_t*>(p.n.residual) + static_cast<int64_t>(m) * p.n.residual_stride * (RF32 ? 4 : 2);
#pragma unroll
    for (uint32_t i = 0; i < VPT; ++i) {
        const uint32_t at = tid + i * threads;
        xq[i] = at < p.vectors ? load_once(x + 8 * at) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (uint32_t i = 0; i < VPT; ++i) {
        const uint32_t at = tid + i * threads;
        const bool there = at < p.vectors && p.n.residual != nullptr;
#pragma unroll
        for (uint32_t k = 0; k < (RF32 ? 2 : 1); ++k)
            rq[i][k] = there ? load_once(res + static_cast<size_t>(at) * (RF32 ? 32 : 16) + 16 * k) : make_uint4(0, 0, 0, 0);
    }
    Eight v[VPT];
#pragma unroll
    for (uint32_t i = 0; i < VPT; ++i) v[i] = unpack8<F16>(xq[i]);
    // The norm's factor of x comes last where no bias stands between: one with the residual's scale.
    const bool post = p.n.post_weight != nullptr, wf32 = p.n.weight_f32 != 0;
    const float r1 = post ? moments<LAYER, WARP, VPT>(p, v, tid, threads, sh, turn) : 1.f;
    const uint64_t factor = both(p.n.post_bias != nullptr ? p.n.scale : r1 * p.n.scale);
    const int64_t gate_row = p.n.gate != nullptr ? static_cast<int64_t>(m / p.gate_every) * p.n.gate_stride : 0;
#pragma unroll
    for (uint32_t i = 0; i < VPT; ++i) {
        const uint32_t at = tid + i * threads;
        if (at >= p.vectors) continue;
        if (post) {
            const Eight w = load8<F16>(p.n.post_weight, wf32, 8ll * at);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i].p[e] = mul_f32x2(v[i].p[e], w.p[e]);
            if (p.n.post_bias != nullptr) {
                const Eight b = load8<F16>(p.n.post_bias, wf32, 8ll * at);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i].p[e] = fma_f32x2(v[i].p[e], both(r1), b.p[e]);
            }
        }
        if (p.n.gate != nullptr) {
            const Eight g = load8<F16>(p.n.gate, false, gate_row + 8 * at);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[i].p[e] = mul_f32x2(v[i].p[e], g.p[e]);
        }
        Eight r;
        if constexpr (RF32) {
            const uint32_t w[8] = {rq[i][0].x, rq[i][0].y, rq[i][0].z, rq[i][0].w, rq[i][1].x, rq[i][1].y, rq[i][1].z, rq[i][1].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) r.p[e] = pack_f32x2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
        } else {
            r = unpack8<F16>(rq[i][0]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[i].p[e] = fma_f32x2(v[i].p[e], factor, r.p[e]);
        if (p.n.residual_out != nullptr) store8<F16>(p.n.residual_out, RF32, static_cast<int64_t>(m) * p.n.residual_out_stride + 8 * at, v[i]);
    }
    if (p.n.weight == nullptr) return;
    const uint64_t r2 = both(moments<LAYER, WARP, VPT>(p, v, tid, threads, sh, turn));
#pragma unroll
    for (uint32_t i = 0; i < VPT; ++i) {
        const uint32_t at = tid + i * threads;
        if (at < p.vectors) {
            const Eight w = load8<F16>(p.n.weight, wf32, 8ll * at);
            if (p.n.bias != nullptr) {
                const Eight b = load8<F16>(p.n.bias, wf32, 8ll * at);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i].p[e] = fma_f32x2(mul_f32x2(v[i].p[e], w.p[e]), r2, b.p[e]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[i].p[e] = mul_f32x2(mul_f32x2(v[i].p[e], r2), w.p[e]);
            }
        }
        if (p.n.out_scale == nullptr) {
            if (at < p.vectors) store8<F16>(p.n.out, false, static_cast<int64_t>(m) * p.n.out_stride + 8 * at, v[i]);
            continue;
        }
        // a group's 16 lanes are all there or all past the row (H is a multiple of 128 here)
        float y[8], mx = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = unpack_f32x2(v[i].p[e]);
            y[2 * e] = f.x, y[2 * e + 1] = f.y;
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        if (at >= p.vectors) continue;
        const float s = __fdiv_rn(mx, 448.f);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.n.out) + static_cast<int64_t>(m) * p.n.out_stride + 8 * at) = encode8(y, mx, s);
        if ((at & 15u) == 0) p.n.out_scale[static_cast<int64_t>(at / 16) * p.n.out_scale_stride + m] = s;
    }
}

template <bool F16, bool RF32, bool LAYER>
cudaError_t launch(const NormArgs& p, cudaStream_t s) {
    const uint32_t warps = (p.vectors + 31) / 32;   // that hold a row in a vector a thread
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // us, of bf16 rows: a row a warp up to 512 elements: 8192 of 512 7.3, a block a row 8.8; 16384 of 256 6.8 and 16.9.
    if (warps <= 2 && p.n.M > 1) {
        cfg.gridDim = dim3((p.n.M + kWarpRows - 1) / kWarpRows, 1, 1);
        cfg.blockDim = dim3(32 * kWarpRows, 1, 1);
        return cudaLaunchKernelEx(&cfg, warps == 1 ? norm_kernel<F16, RF32, LAYER, true, 1, 32 * kWarpRows> : norm_kernel<F16, RF32, LAYER, true, 2, 32 * kWarpRows>, p);
    }
    // One vector a thread up to 5120 elements (4096 of 5120 with an FP32 residual: 53 and, with four, 54.5; of 4096 38 and 47), and for
    // no more rows than two an SM, where the shortest chain counts (one row of 8192: 3.1 and 4.8; 300 6.3 and 9.9). Else
    // four: 8192 of 8192 89, with one 106.
    cfg.gridDim = dim3(p.n.M, 1, 1);
    const bool one = warps <= 20 || (p.n.M <= 304 && warps <= 32);
    cfg.blockDim = dim3(32 * (one ? warps : (warps + 3) / 4), 1, 1);
    return cudaLaunchKernelEx(&cfg, one ? norm_kernel<F16, RF32, LAYER, false, 1, 1024> : warps <= 32 ? norm_kernel<F16, RF32, LAYER, false, 4, 256>
                                                                                     : norm_kernel<F16, RF32, LAYER, false, 4, 1024>, p);
}

}  // namespace

int launch_norm(const w8a16_norm_t& n, uint32_t flags, cudaStream_t s, std::string* err) {
    const NormArgs p{n, n.H / 8, n.gate != nullptr ? n.M / n.gate_rows : 1, (flags & W8A16_FLAG_PDL) != 0};
    const auto pick = [&](auto f16, auto rf32) {
        constexpr bool F = decltype(f16)::value, R = decltype(rf32)::value;
        return n.kind == W8A16_NORM_LAYER ? launch<F, R, true>(p, s) : launch<F, R, false>(p, s);
    };
    const std::true_type yes;
    const std::false_type no;
    const cudaError_t e = n.act_dtype == W8A16_ACT_F16 ? (n.residual_f32 ? pick(yes, yes) : pick(yes, no))
                                                       : (n.residual_f32 ? pick(no, yes) : pick(no, no));
    if (e != cudaSuccess) {
        cudaGetLastError();
        *err = std::string("norm launch failed: ") + cudaGetErrorString(e);
        return W8A16_ERR_LAUNCH;
    }
    return W8A16_OK;
}

}  // namespace w8a16

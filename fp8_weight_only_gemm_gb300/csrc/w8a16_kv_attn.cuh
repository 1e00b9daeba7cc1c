// What the two attention kernels over the paged cache share.
#pragma once

#include "w8a16_kv.cuh"

namespace w8a16 {

struct AttnArgs {
    w8a16_kv_cache_t c;
    w8a16_kv_batch_t b;
    w8a16_heads_t q, out;
    float* ws;
    float scale_log2;       // softmax scale times log2(e)
    uint32_t group;         // query heads per key/value head
    uint32_t page_shift;
    uint32_t ctas;          // of the attention kernel
    uint32_t tile_rows;     // query rows of an item (the kernel for few rows)
    uint64_t timeout_ns;    // limit of an in-kernel wait
};

// Smaller page scales count as this one.
constexpr float kMinScale = 8.673617379884035e-19f;   // 2^-60

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// a / b: the 64-bit division takes some 400 cycles, few calls need it.
__device__ __forceinline__ uint64_t divide(uint64_t a, uint64_t b) {
    return ((a | b) >> 32) == 0 ? static_cast<uint64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b)) : a / b;
}

// The CTAs that get work (no more than there are units, so that none between the
// first and the last CTA of an item is empty), the first unit of CTA c's range, and the
// CTA that holds unit u.
__device__ __forceinline__ uint64_t active_ctas(uint64_t units, uint32_t ctas) {
    return units < ctas ? units : ctas;
}
__device__ __forceinline__ uint64_t first_unit(uint64_t c, uint64_t units, uint64_t ctas) { return divide(c * units, ctas); }
__device__ __forceinline__ uint32_t cta_of(uint64_t u, uint64_t units, uint64_t ctas) {
    return static_cast<uint32_t>(divide((u + 1) * ctas - 1, units));
}

// What CTA c's range begins in, written by it at the head of the workspace for the launch
// that joins split items: `parts` > 0 where it is the first range to begin inside an item,
// whose parts are then those of CTAs c - 1 (at `slot`) and c .. c + parts - 2 (their first
// slots).
struct Boundary {
    uint32_t parts, slot;
    int32_t first, count;    // the sequence's rows
    uint32_t h, tile;        // the item's head and row tile
};
// After them, `parts` alone (a multiple of 4 of them, and where the slots begin).
__host__ __device__ constexpr uint64_t parts_at(uint32_t ctas) { return (ctas * sizeof(Boundary) + 15) / 16 * 4; }
__host__ __device__ constexpr uint64_t boundary_floats(uint32_t ctas) { return parts_at(ctas) + (ctas + 3) / 4 * 4; }
__device__ __forceinline__ void write_boundary(float* ws, uint64_t u0, uint64_t item_first, uint32_t item_units, const Seq& s,
                                               uint32_t h, uint32_t tile, uint64_t total, uint64_t ctas) {
    Boundary b{0, 0, s.first, s.count, h, tile};
    const uint32_t c = blockIdx.x;
    if (c < ctas && u0 != item_first) {
        const uint64_t before = first_unit(c - 1, total, ctas);
        if (before <= item_first) {
            b.parts = cta_of(item_first + item_units - 1, total, ctas) - c + 2;
            b.slot = before == item_first ? 2 * (c - 1) : 2 * (c - 1) + 1;   // that CTA's first part, or its last
        }
    }
    reinterpret_cast<Boundary*>(ws)[c] = b;
    reinterpret_cast<uint32_t*>(ws + parts_at(gridDim.x))[c] = b.parts;
}

// The CTA of the k-th boundary with parts (from 0), or 0 if there are fewer; for all of a block. A thread looks at 4.
template <uint32_t THREADS>
__device__ __forceinline__ uint32_t split_boundary(const AttnArgs& p, uint32_t k) {
    __shared__ uint32_t sh_count[THREADS / 32];
    __shared__ uint32_t sh_c;
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t* const parts = reinterpret_cast<const uint32_t*>(p.ws + parts_at(p.ctas));
    if (threadIdx.x == 0) sh_c = 0;
    for (uint32_t base = 0; base < p.ctas; base += 4 * THREADS) {
        const uint32_t c0 = base + 4 * threadIdx.x;
        uint32_t has = 0;
        if (c0 < p.ctas) {   // (past the last one: whatever is there is masked; CTA 0 begins no item inside)
            const uint4 v = *reinterpret_cast<const uint4*>(parts + c0);
            has = ((v.x ? 1u : 0u) | (v.y ? 2u : 0u) | (v.z ? 4u : 0u) | (v.w ? 8u : 0u)) & (p.ctas - c0 < 4 ? (1u << (p.ctas - c0)) - 1u : 15u);
        }
        const uint32_t n = __popc(has);
        uint32_t before = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xFFFFFFFFu, before, o);
            if (lane >= static_cast<uint32_t>(o)) before += x;
        }
        __syncthreads();
        if (lane == 31) sh_count[warp] = before;
        before -= n;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (uint32_t w = 0; w < THREADS / 32; ++w) {
            if (w < warp) before += sh_count[w];
            all += sh_count[w];
        }
        if (k >= before && k < before + n) {
            for (uint32_t i = k - before; i; --i) has &= has - 1;
            sh_c = c0 + __ffs(has) - 1;
        }
        if (k < all) break;
        k -= all;
    }
    __syncthreads();
    return sh_c;
}

// Zeros in the rows of sequences without keys.
__device__ __forceinline__ void zero_keyless(const AttnArgs& p) {
    for (uint32_t b = blockIdx.x; b < p.b.batch; b += gridDim.x) {
        const Seq s = sequence(p.b, p.c.page_size, b);
        if (s.bad || s.len > 0) continue;
        const uint32_t per_head = p.c.head_dim / 8, per_row = p.out.heads * per_head;
        for (uint64_t i = threadIdx.x; i < static_cast<uint64_t>(s.count) * per_row; i += blockDim.x) {
            const uint32_t n = static_cast<uint32_t>(i / per_row), h = static_cast<uint32_t>(i % per_row) / per_head,
                           d = static_cast<uint32_t>(i % per_head) * 8;
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(s.first + static_cast<int>(n)) * p.out.token_stride +
                                      static_cast<int64_t>(h) * p.out.head_stride + d) = make_uint4(0, 0, 0, 0);
        }
    }
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The row scale of a query: softmax scale times 2^(E - 7) for its largest element's
// exponent E, and the two factors f1 f2 = 2^(7 - E) that bring the row to [2^7, 2^8)
// (two: E reaches -133 for BF16 subnormals). What reaches the logits is its product with a page's
// key scale (2^-60 and more), and only that has to be in FP32's range: a row scale below 2^-60 is
// kept times -2^64, and its sign tells logit_factor. A row with a non-finite element gets a NaN scale.
struct RowScale {
    float scale, f1, f2;
};
__device__ __forceinline__ RowScale row_scale_of(float amax, bool bad, float scale_log2) {
    if (bad) return {__uint_as_float(0x7FC00000u), 0.f, 0.f};
    const int E = amax > 0.f ? ilogbf(amax) : 7;
    const int a = (7 - E) / 2, b = 7 - E - a;
    const auto pow2 = [](int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); };
    const float scale = scale_log2 * pow2(-a) * pow2(-b);
    return {scale < kMinScale ? -(scale_log2 * pow2(64 - a) * pow2(-b)) : scale, pow2(a), pow2(b)};
}
// Logit per unit of score of a row and page. Never 0, so that a masked score (-inf) stays one (where
// the smallest normal number shows in it, all logits are below 2^-75).
__device__ __forceinline__ float logit_factor(float ks, float row_scale) {
    constexpr float kTwoToMinus64 = 5.421010862427522e-20f, kSmallest = 1.1754943508222875e-38f;
    return fmaf(row_scale < 0.f ? ks * kTwoToMinus64 : ks, fabsf(row_scale), kSmallest);
}

// The kernel for many query rows per key/value head (w8a16_kv_attn_tc.cu).
bool kv_attn_tc_applies(uint32_t head_dim, uint32_t rows_per_head);
uint64_t kv_attn_tc_ws_bytes(uint32_t head_dim, int sms);
cudaError_t launch_kv_attn_tc(AttnArgs p, bool f16, int sms, cudaStream_t s);

}  // namespace w8a16

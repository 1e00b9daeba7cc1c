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
    uint64_t timeout_ns;    // limit of an in-kernel wait
};

// Smaller page scales count as this one.
constexpr float kMinScale = 8.673617379884035e-19f;   // 2^-60

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The CTAs that get work (no more than there are units, so that none between the
// first and the last CTA of an item is empty), the first unit of CTA c's range, and the
// CTA that holds unit u.
__device__ __forceinline__ uint64_t active_ctas(uint64_t units, uint32_t ctas) {
    return units < ctas ? units : ctas;
}
__device__ __forceinline__ uint64_t first_unit(uint64_t c, uint64_t units, uint64_t ctas) { return c * units / ctas; }
__device__ __forceinline__ uint32_t cta_of(uint64_t u, uint64_t units, uint64_t ctas) {
    return static_cast<uint32_t>(((u + 1) * ctas - 1) / units);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The row scale of a query: softmax scale times 2^(E - 7) for its largest element's
// exponent E, and the two factors f1 f2 = 2^(7 - E) that bring the row to [2^7, 2^8)
// (two: E reaches -133 for BF16 subnormals). A row with a non-finite element gets a NaN scale.
struct RowScale {
    float scale, f1, f2;
};
__device__ __forceinline__ RowScale row_scale_of(float amax, bool bad, float scale_log2) {
    if (bad) return {__uint_as_float(0x7FC00000u), 0.f, 0.f};
    const int E = amax > 0.f ? ilogbf(amax) : 7;
    const int a = (7 - E) / 2, b = 7 - E - a;
    const auto pow2 = [](int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); };
    return {scale_log2 * pow2(-a) * pow2(-b), pow2(a), pow2(b)};
}

// The kernel for many query rows per key/value head (w8a16_kv_attn_tc.cu).
bool kv_attn_tc_applies(uint32_t head_dim, uint32_t rows_per_head);
uint64_t kv_attn_tc_ws_bytes(uint32_t head_dim, int sms);
cudaError_t launch_kv_attn_tc(AttnArgs p, bool f16, int sms, cudaStream_t s);

}  // namespace w8a16

// What the paged-cache kernels share: where a sequence's tokens lie, and the
// activation types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "w8a16_device.cuh"

namespace w8a16 {

// Rows of sequence b in q, k and v, [first, first + count), and its length with them.
// `bad`: row offsets outside [0, tokens], running backwards or of more than max_q
// rows, or a length past the table's pages; count and len are then 0.
struct Seq {
    int first, count, len;
    bool bad;
};
__device__ __forceinline__ Seq sequence(const w8a16_kv_batch_t& bt, uint32_t page_size, uint32_t b) {
    int lo = static_cast<int>(b * bt.max_q), hi = lo + static_cast<int>(bt.max_q);
    if (bt.cu_q != nullptr) {
        lo = bt.cu_q[b];
        hi = bt.cu_q[b + 1];
    }
    const int len = bt.lens[b];
    const bool bad = lo < 0 || hi < lo || hi > static_cast<int>(bt.tokens) || hi - lo > static_cast<int>(bt.max_q) ||
                     len > static_cast<int>(bt.max_pages * page_size);
    return bad ? Seq{0, 0, 0, true} : Seq{lo, hi - lo, len, false};
}

// The sequence that holds row n (the last b with cu_q[b] <= n).
__device__ __forceinline__ uint32_t seq_of_row(const w8a16_kv_batch_t& bt, uint32_t n) {
    if (bt.cu_q == nullptr) return n / bt.max_q;
    uint32_t lo = 0, hi = bt.batch;   // cu_q[lo] <= n < cu_q[hi]
    while (hi - lo > 1) {
        const uint32_t mid = (lo + hi) / 2;
        if (bt.cu_q[mid] <= static_cast<int>(n)) lo = mid;
        else hi = mid;
    }
    return lo;
}

// Two BF16 or FP16 values of a 32-bit word as FP32, and back (round to nearest even).
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (F16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four E4M3 codes as two FP16 pairs (exact).
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

}  // namespace w8a16

// Appending to the 8-bit paged cache: rotate the new keys (and queries), choose the
// page scales, encode E4M3.
//
// Mathematics. A rotated pair is (a cos - b sin, b cos + a sin), each product and sum
// rounded once in FP32. The scale of a page and head is the smallest power of two s
// with amax <= 448 s: E4M3 is a floating format, so a power of two costs no mantissa
// bit against amax/448, division by it is exact, and when a later token needs a
// larger scale the codes already held keep their values (their exponents shift) but
// for those pushed under 2^-6 s, which round once more. Scales only grow while a
// page fills, so no chain of tokens can round a code twice in its normal range.
//
// Work. One item per (sequence, touched page, head, K or V): pass 1 takes the
// maximum over the item's new tokens, pass 2 rotates again and encodes. A thread
// holds two 8-element chunks of a token (the two halves of eight rotary pairs in
// the half layout, 16 consecutive elements in the interleaved one), so every load is
// 16 bytes, every store 8 or 16. Queries are independent tasks of 16 elements, in blocks of
// their own behind the items', two a thread.
//
// Bound by: a few tokens, by two dependent loads behind the launch, length -> page -> codes (48
// sequences, one token: 2.8 us device time); prompts by HBM, where 28 us for 138 MB (4 sequences of 1501
// tokens, 64 query heads) are 4.9 TB/s. A thread's query elements are asked for before the token's
// position is known: with one task a thread, found by 64-bit divisions, and asked for after it,
// that took 33 us; four tasks a thread take 31.6.
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "w8a16_kv.cuh"

namespace w8a16 {
namespace {

__device__ DeviceStatus g_kv_append_status;

constexpr uint32_t kThreads = 128, kQueryTasks = 2;
constexpr int kMinScaleExp = -60;

struct AppendArgs {
    w8a16_kv_cache_t c;
    w8a16_kv_batch_t b;
    w8a16_heads_t k, v, q, q_out;
    w8a16_rope_t rope;
    uint32_t pages_per_seq;   // most pages that one sequence's new tokens touch
    uint32_t items;           // batch * pages_per_seq * kv_heads * 2
    uint32_t item_blocks;
    uint32_t token_blocks;    // of a token's queries
};

// The smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8), at least 2^-60.
__device__ __forceinline__ float page_scale(float amax) {
    const uint32_t bits = __float_as_uint(amax);
    int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(e, 127 + kMinScaleExp);   // subnormal and zero maxima included
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

__device__ __forceinline__ uint32_t e4m3_byte_nan_patch(float x, uint32_t code) {
    return fabsf(x) <= 3.4028235e38f ? code : 0x7Fu;   // NaN and infinity
}

__device__ __forceinline__ uint32_t encode4(const float* x, float inv) {
    uint16_t a, b;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1] * inv), "f"(x[0] * inv));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(x[3] * inv), "f"(x[2] * inv));
    uint32_t w = a | (static_cast<uint32_t>(b) << 16);
    const float m = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    const bool nan = (x[0] != x[0]) | (x[1] != x[1]) | (x[2] != x[2]) | (x[3] != x[3]);
    if (__builtin_expect(nan || m > 3.4028235e38f, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w = (w & ~(0xFFu << (8 * i))) | (e4m3_byte_nan_patch(x[i], (w >> (8 * i)) & 0xFFu) << (8 * i));
    }
    return w;
}

// Where the two chunks of task i of a head begin.
struct Chunks {
    uint32_t a, b;
    bool rotated;
};
__device__ __forceinline__ Chunks chunks_of(uint32_t rotary_dim, bool interleaved, uint32_t i) {
    if (16 * i >= rotary_dim) return {16 * i, 16 * i + 8, false};
    if (interleaved) return {16 * i, 16 * i + 8, true};
    return {8 * i, rotary_dim / 2 + 8 * i, true};
}

__device__ __forceinline__ void rotate(float& lo, float& hi, float c, float s) {
    const float a = lo, b = hi;
    lo = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    hi = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// The 16 values of a task, from its chunks' words, rotated for `pos`.
template <bool F16>
__device__ __forceinline__ void rotated(const uint4& qa, const uint4& qb, const w8a16_rope_t& r, const Chunks& ch, uint32_t i, int pos,
                                        float (&x)[16]) {
    const uint32_t wa[4] = {qa.x, qa.y, qa.z, qa.w}, wb[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 a = unpack2<F16>(wa[e]), b = unpack2<F16>(wb[e]);
        x[2 * e] = a.x;
        x[2 * e + 1] = a.y;
        x[8 + 2 * e] = b.x;
        x[8 + 2 * e + 1] = b.y;
    }
    if (!ch.rotated) return;
    const size_t row = static_cast<size_t>(pos) * (r.rotary_dim / 2) + 8 * i;
    const float4 c0 = *reinterpret_cast<const float4*>(r.cos + row), c1 = reinterpret_cast<const float4*>(r.cos + row)[1];
    const float4 s0 = *reinterpret_cast<const float4*>(r.sin + row), s1 = reinterpret_cast<const float4*>(r.sin + row)[1];
    const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate(x[2 * e], x[2 * e + 1], c[e], s[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate(x[e], x[8 + e], c[e], s[e]);
    }
}
template <bool F16>
__device__ __forceinline__ void load_rotated(const uint16_t* head, const w8a16_rope_t& r, const Chunks& ch, uint32_t i,
                                             int pos, float (&x)[16]) {
    rotated<F16>(*reinterpret_cast<const uint4*>(head + ch.a), *reinterpret_cast<const uint4*>(head + ch.b), r, ch, i, pos, x);
}

// Up to kQueryTasks tasks (16 elements of a query head) of token n a thread, `first` and every
// kThreads-th after it; they are asked for before the token's position is known.
template <bool F16>
__device__ __forceinline__ void rotate_queries(const AppendArgs& p, uint32_t n, uint32_t first) {
    const uint32_t per_head = p.c.head_dim / 16, tasks = p.q.heads * per_head;
    const uint16_t* const src = static_cast<const uint16_t*>(p.q.ptr) + static_cast<int64_t>(n) * p.q.token_stride;
    uint16_t* const dst = static_cast<uint16_t*>(p.q_out.ptr) + static_cast<int64_t>(n) * p.q_out.token_stride;
    uint4 qa[kQueryTasks], qb[kQueryTasks];
    Chunks ch[kQueryTasks];
    uint32_t h[kQueryTasks], i[kQueryTasks];
#pragma unroll
    for (uint32_t u = 0; u < kQueryTasks; ++u) {
        const uint32_t task = first + u * kThreads;
        h[u] = task / per_head, i[u] = task % per_head;
        ch[u] = chunks_of(p.rope.rotary_dim, p.rope.interleaved, i[u]);
        if (task >= tasks) continue;
        const uint16_t* const head = src + static_cast<int64_t>(h[u]) * p.q.head_stride;
        qa[u] = *reinterpret_cast<const uint4*>(head + ch[u].a), qb[u] = *reinterpret_cast<const uint4*>(head + ch[u].b);
    }
    const Seq seq = sequence(p.b, p.c.page_size, seq_of_row(p.b, n));
    const int t = static_cast<int>(n) - seq.first;
    if (t < 0 || t >= seq.count) return;   // rows that no sequence claims (a bad one: reported by its items)
    const int pos = seq.len - seq.count + t;
#pragma unroll
    for (uint32_t u = 0; u < kQueryTasks; ++u) {
        if (first + u * kThreads >= tasks) break;
        if (pos < 0) ch[u].rotated = false;   // padding: passed through
        if (ch[u].rotated && pos >= static_cast<int>(p.rope.rows)) {
            record_failure(&g_kv_append_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(pos));
            continue;
        }
        float x[16];
        rotated<F16>(qa[u], qb[u], p.rope, ch[u], i[u], pos, x);
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack2<F16>(x[2 * e], x[2 * e + 1]);
        uint16_t* const head = dst + static_cast<int64_t>(h[u]) * p.q_out.head_stride;
        *reinterpret_cast<uint4*>(head + ch[u].a) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(head + ch[u].b) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// TPI threads per item: 32 (a warp, kThreads / 32 items a block) or kThreads.
template <bool F16, uint32_t TPI>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs p) {
    __shared__ uint32_t warp_max[kThreads / 32];
    grid_dependency_wait();     // k, v, q and the cache may be the previous kernel's
    grid_launch_dependents();
    if (blockIdx.x >= p.item_blocks) {
        const uint32_t at = blockIdx.x - p.item_blocks;
        rotate_queries<F16>(p, at / p.token_blocks, at % p.token_blocks * (kThreads * kQueryTasks) + threadIdx.x);
        return;
    }
    const uint32_t lane = threadIdx.x % TPI;
    uint32_t item = blockIdx.x * (kThreads / TPI) + threadIdx.x / TPI;
    if (item >= p.items) return;   // whole warps
    const bool is_v = item & 1u;
    item >>= 1;
    const uint32_t h = item % p.c.kv_heads;
    item /= p.c.kv_heads;
    const uint32_t j = item % p.pages_per_seq, b = item / p.pages_per_seq;

    const Seq seq = sequence(p.b, p.c.page_size, b);
    if (seq.bad) {
        if (lane == 0) record_failure(&g_kv_append_status, W8A16_STATUS_BAD_INDEX, b);
        return;
    }
    const int first = seq.len - seq.count;                    // position of the first new token
    const int begin = max(first, 0);
    const int P = static_cast<int>(p.c.page_size);
    const int page = begin / P + static_cast<int>(j);
    const int lo = max(begin, page * P), hi = min(seq.len, (page + 1) * P);   // this item's positions
    if (lo >= hi) return;
    const int phys = p.b.page_table[static_cast<int64_t>(b) * p.b.page_table_stride + page];
    if (phys < 0 || phys >= static_cast<int>(p.c.num_pages)) {
        if (lane == 0) record_failure(&g_kv_append_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(phys));
        return;
    }
    const uint32_t rot = is_v ? 0u : p.rope.rotary_dim;
    if (p.rope.rotary_dim != 0 && hi > static_cast<int>(p.rope.rows)) {   // keys and values alike
        if (lane == 0) record_failure(&g_kv_append_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(hi - 1));
        return;
    }
    const w8a16_heads_t& src = is_v ? p.v : p.k;
    const uint16_t* x0 = static_cast<const uint16_t*>(src.ptr) + static_cast<int64_t>(h) * src.head_stride;
    uint8_t* codes = static_cast<uint8_t*>(is_v ? p.c.v_codes : p.c.k_codes) +
                     static_cast<int64_t>(phys) * p.c.page_stride + static_cast<int64_t>(h) * p.c.head_stride;
    float* scale_at = (is_v ? p.c.v_scale : p.c.k_scale) + static_cast<int64_t>(phys) * p.c.scale_page_stride +
                      static_cast<int64_t>(h) * p.c.scale_head_stride;
    const bool old_tokens = lo > page * P;
    const float old = old_tokens ? *scale_at : 0.f;
    const uint32_t per_token = p.c.head_dim / 16;
    const uint32_t tasks = static_cast<uint32_t>(hi - lo) * per_token;

    float amax = 0.f;
    for (uint32_t task = lane; task < tasks; task += TPI) {
        const uint32_t i = task % per_token;
        const int pos = lo + static_cast<int>(task / per_token);
        float x[16];
        load_rotated<F16>(x0 + static_cast<int64_t>(seq.first + pos - first) * src.token_stride, p.rope,
                          chunks_of(rot, p.rope.interleaved, i), i, pos, x);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float a = fabsf(x[e]);
            if (a <= 3.4028235e38f) amax = fmaxf(amax, a);
        }
    }
    uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));   // |x| orders as its bits
    if constexpr (TPI > 32) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = bits;
        __syncthreads();
#pragma unroll
        for (uint32_t w = 0; w < kThreads / 32; ++w) bits = max(bits, warp_max[w]);
    }
    const float scale = fmaxf(page_scale(__uint_as_float(bits)), old);
    const float inv = __frcp_rn(scale);   // exact for a power of two

    for (uint32_t task = lane; task < tasks; task += TPI) {
        const uint32_t i = task % per_token;
        const int pos = lo + static_cast<int>(task / per_token);
        const Chunks ch = chunks_of(rot, p.rope.interleaved, i);
        float x[16];
        load_rotated<F16>(x0 + static_cast<int64_t>(seq.first + pos - first) * src.token_stride, p.rope, ch, i, pos, x);
        uint8_t* dst = codes + static_cast<int64_t>(pos - page * P) * p.c.token_stride;
        *reinterpret_cast<uint2*>(dst + ch.a) = make_uint2(encode4(x, inv), encode4(x + 4, inv));
        *reinterpret_cast<uint2*>(dst + ch.b) = make_uint2(encode4(x + 8, inv), encode4(x + 12, inv));
    }
    // older tokens of the page: rewritten where the scale has grown
    if (old_tokens && scale != old) {
        const float ratio = __fdiv_rn(old, scale);
        const uint32_t olds = static_cast<uint32_t>(lo - page * P) * per_token;
        for (uint32_t task = lane; task < olds; task += TPI) {
            uint4* at = reinterpret_cast<uint4*>(codes + static_cast<int64_t>(task / per_token) * p.c.token_stride) +
                        task % per_token;
            const uint4 q = *at;
            uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t l, g;
                e4m3x4_to_f16x4(w[e], l, g);
                const float2 u = unpack2<true>(l), v = unpack2<true>(g);
                const float y[4] = {u.x, u.y, v.x, v.y};
                w[e] = encode4(y, ratio);
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (lane == 0) *scale_at = scale;
}

}  // namespace

int launch_kv_append(const w8a16_kv_cache_t& c, const w8a16_kv_batch_t& b, uint32_t act_dtype, const w8a16_heads_t& k,
                     const w8a16_heads_t& v, const w8a16_heads_t& q, const w8a16_heads_t& q_out,
                     const w8a16_rope_t& rope, cudaStream_t s, std::string* err) {
    AppendArgs p{c, b, k, v, q, q_out, rope, 0, 0, 0, 0};
    p.pages_per_seq = (b.max_q + c.page_size - 2) / c.page_size + 1;
    const uint64_t items = 2ull * b.batch * p.pages_per_seq * c.kv_heads;
    // A warp per item where a page's new tokens have a task a lane at most, else a block. us, warp against
    // block (8 heads of 128, 32 query heads): 48 sequences of 1 token (8 tasks) 2.8 3.2; 1 of 5 (40) 3.5
    // 2.7; 48 of 5 4.5 4.2; 1 of 8 3.5 2.8; 32 of 16 7.6 4.3; 4 of 1500 41.9 27.9.
    const bool wide = static_cast<uint64_t>(b.max_q < c.page_size ? b.max_q : c.page_size) * (c.head_dim / 16) > 32;
    const uint64_t item_blocks = wide ? items : (items + kThreads / 32 - 1) / (kThreads / 32);
    p.token_blocks = (q.heads * (c.head_dim / 16) + kThreads * kQueryTasks - 1) / (kThreads * kQueryTasks);
    const uint64_t q_blocks = q.ptr ? static_cast<uint64_t>(b.tokens) * p.token_blocks : 0;
    if (items > 0x7FFFFFFFull || item_blocks + q_blocks > 0x7FFFFFFFull) {
        *err = "cache append: too many pages or queries for one launch";
        return W8A16_ERR_RANGE;
    }
    p.items = static_cast<uint32_t>(items);
    p.item_blocks = static_cast<uint32_t>(item_blocks);
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(static_cast<unsigned>(item_blocks + q_blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool f16 = act_dtype == W8A16_ACT_F16;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, wide ? (f16 ? kv_append_kernel<true, kThreads> : kv_append_kernel<false, kThreads>)
                                                        : (f16 ? kv_append_kernel<true, 32> : kv_append_kernel<false, 32>),
                                             p);
    if (e != cudaSuccess) {
        cudaGetLastError();
        *err = std::string("cache append launch failed: ") + cudaGetErrorString(e);
        return W8A16_ERR_LAUNCH;
    }
    return W8A16_OK;
}

cudaError_t kv_append_status_read(StatusWord* out, bool clear, cudaStream_t s) {
    DeviceStatus st;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&st, g_kv_append_status, sizeof st, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    out->code = st.code;
    out->where = st.where;
    out->detail = st.detail;
    if (clear) {
        const DeviceStatus zero{0, 0, 0};
        e = cudaMemcpyToSymbolAsync(g_kv_append_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace w8a16

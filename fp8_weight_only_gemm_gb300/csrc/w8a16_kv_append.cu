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
// that took 33 us; four tasks a thread take 31.6. Several axes: a token's positions are one more load in that chain
// (one sequence, one token: 3.6 us a call for 2.9), and 4 sequences of 1369 tokens take 29.6 us for one axis's 25.5, the axes dealt in turn
// or in blocks that end inside a chunk; in blocks of whole chunks 27.0. Large pages and few heads are far from memory's time: an item is a page of a
// head for 128 threads, each with several tasks that it rotates twice (2 sequences of 149 tokens, pages of 128: 17.3 us for 13.5 MB; 2
// of 1351, 8 heads of 64: 12.6 for 14.6).
#include <cuda_runtime.h>

#include <cstring>
#include <string>
#include <type_traits>

#include "w8a16_kv.cuh"

namespace w8a16 {
namespace {

__device__ DeviceStatus g_kv_append_status;

constexpr uint32_t kThreads = 128, kQueryTasks = 2;
constexpr int kMinScaleExp = -60;

// The positions of tokens with several axes: `axes` rows, and of each chunk of 8 rotary pairs their axes, two bits each.
struct Axes {
    const int32_t* positions;
    int64_t stride;
    uint32_t axes;
    uint16_t of_pairs[16];
};
struct AppendArgs {
    w8a16_kv_cache_t c;
    w8a16_kv_batch_t b;
    w8a16_heads_t k, v, q, q_out;
    w8a16_rope_t rope;
    uint32_t pages_per_seq;   // most pages that one sequence's new tokens touch
    uint32_t items;           // batch * pages_per_seq * kv_heads * 2
    uint32_t item_blocks;
    uint32_t token_blocks;    // of a token's queries
    Axes axes;
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

// The rows of the rotary table for a token: its position, or that of each axis.
template <bool AXES>
struct Rows {
    int pos[AXES ? 4 : 1];
};
// Of row n of the call, at `pos` in its sequence. false: outside the table (they are 0 then, and may be used); `bad` is one that is.
template <bool AXES>
__device__ __forceinline__ bool rows_of(const AppendArgs& p, uint32_t n, int pos, Rows<AXES>& r, int& bad) {
    if constexpr (!AXES) {
        r.pos[0] = pos;
        return true;   // the callers look at the last position
    } else {
        bool good = true;
#pragma unroll
        for (uint32_t a = 0; a < 4; ++a) {
            r.pos[a] = a < p.axes.axes ? p.axes.positions[a * p.axes.stride + n] : 0;
            if (static_cast<uint32_t>(r.pos[a]) >= p.rope.rows) good = false, bad = r.pos[a], r.pos[a] = 0;
        }
        return good;
    }
}
__device__ __forceinline__ void load_row8(const float* from, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(from), b = reinterpret_cast<const float4*>(from)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Several axes: the cosines and sines of a token, pair by pair from the rows of their axes, for the threads of a block whose
// tasks are all of that token. Rows outside the table count as 0 here. (Each task for itself, as keys still do, it was 35 us for
// 4 sequences of 1369 tokens whose axes are dealt in turn over the pairs, 30 now; where a chunk of pairs mixes axes, wide loads
// of every axis's row are slower than an element each, 42 for 35, and keys gathered page by page wait for it, 47.)
struct Gathered {
    float cos[kThreads], sin[kThreads];
};
__device__ __forceinline__ void gather(const AppendArgs& p, uint32_t n, Gathered& g) {
    const uint32_t half = p.rope.rotary_dim / 2, pair = threadIdx.x;   // at most 128
    if (pair < half) {
        const uint32_t axis = (p.axes.of_pairs[pair / 8] >> (2 * (pair % 8))) & 3u;
        uint32_t row = static_cast<uint32_t>(p.axes.positions[axis * p.axes.stride + n]);
        if (row >= p.rope.rows) row = 0;
        const size_t from = static_cast<size_t>(row) * half + pair;
        g.cos[pair] = p.rope.cos[from], g.sin[pair] = p.rope.sin[from];
    }
}

// The 16 values of a task, from its chunks' words, rotated for its token's rows (cs: gathered ones of its token).
template <bool F16, bool AXES>
__device__ __forceinline__ void rotated(const AppendArgs& p, const uint4& qa, const uint4& qb, const Chunks& ch, uint32_t i, const Rows<AXES>& rows,
                                        float (&x)[16], const float* cs = nullptr) {
    const w8a16_rope_t& r = p.rope;
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
    float c[8], s[8];
    if constexpr (!AXES) {
        const size_t row = static_cast<size_t>(rows.pos[0]) * (r.rotary_dim / 2) + 8 * i;
        load_row8(r.cos + row, c);
        load_row8(r.sin + row, s);
    } else {
        const uint32_t of = p.axes.of_pairs[i];
        const auto at = [&](uint32_t axis) {
            const int lo = axis & 1u ? rows.pos[1] : rows.pos[0], hi = axis & 1u ? rows.pos[3] : rows.pos[2];
            return static_cast<size_t>(axis & 2u ? hi : lo) * (r.rotary_dim / 2) + 8 * i;
        };
        if (cs != nullptr) {
            load_row8(cs + 8 * i, c);
            load_row8(cs + kThreads + 8 * i, s);
        } else if (of == (of & 3u) * 0x5555u) {   // pairs of one axis
            const size_t row = at(of & 3u);
            load_row8(r.cos + row, c);
            load_row8(r.sin + row, s);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const size_t row = at((of >> (2 * e)) & 3u) + e;
                c[e] = r.cos[row], s[e] = r.sin[row];
            }
        }
    }
    if (r.interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate(x[2 * e], x[2 * e + 1], c[e], s[e]);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) rotate(x[e], x[8 + e], c[e], s[e]);
    }
}
template <bool F16, bool AXES>
__device__ __forceinline__ void load_rotated(const AppendArgs& p, const uint16_t* head, const Chunks& ch, uint32_t i, const Rows<AXES>& rows,
                                             float (&x)[16], const float* cs = nullptr) {
    rotated<F16, AXES>(p, *reinterpret_cast<const uint4*>(head + ch.a), *reinterpret_cast<const uint4*>(head + ch.b), ch, i, rows, x, cs);
}

// Up to kQueryTasks tasks (16 elements of a query head) of token n a thread, `first` and every
// kThreads-th after it; they are asked for before the token's position is known.
template <bool F16, bool AXES>
__device__ __forceinline__ void rotate_queries(const AppendArgs& p, uint32_t n, uint32_t first, Gathered& g) {
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
    Rows<AXES> rows{};
    int bad = pos;
    const bool good = pos < 0 || rows_of<AXES>(p, n, pos, rows, bad);
    if (AXES ? !good : p.rope.rotary_dim != 0 && pos >= static_cast<int>(p.rope.rows)) {   // the block's one token: skipped whole
        if (threadIdx.x == 0) record_failure(&g_kv_append_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(bad));
        return;
    }
    if constexpr (AXES) {
        if (pos >= 0) gather(p, n, g);
        __syncthreads();
    }
#pragma unroll
    for (uint32_t u = 0; u < kQueryTasks; ++u) {
        if (first + u * kThreads >= tasks) break;
        if (pos < 0) ch[u].rotated = false;   // padding: passed through
        float x[16];
        rotated<F16, AXES>(p, qa[u], qb[u], ch[u], i[u], rows, x, AXES ? g.cos : nullptr);
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack2<F16>(x[2 * e], x[2 * e + 1]);
        uint16_t* const head = dst + static_cast<int64_t>(h[u]) * p.q_out.head_stride;
        *reinterpret_cast<uint4*>(head + ch[u].a) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4*>(head + ch[u].b) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// TPI threads per item: 32 (a warp, kThreads / 32 items a block) or kThreads.
template <bool F16, uint32_t TPI, bool AXES>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs p) {
    __shared__ uint32_t warp_max[kThreads / 32];
    __shared__ __align__(16) char gathered[AXES ? sizeof(Gathered) : 16];
    Gathered& g = *reinterpret_cast<Gathered*>(gathered);
    grid_dependency_wait();     // k, v, q and the cache may be the previous kernel's
    grid_launch_dependents();
    if (blockIdx.x >= p.item_blocks) {
        const uint32_t at = blockIdx.x - p.item_blocks;
        rotate_queries<F16, AXES>(p, at / p.token_blocks, at % p.token_blocks * (kThreads * kQueryTasks) + threadIdx.x, g);
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
    if (!AXES && p.rope.rotary_dim != 0 && hi > static_cast<int>(p.rope.rows)) {   // keys and values alike
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

    bool good = true;   // of the tokens that this lane has looked at: their rows of the table are there
    int bad = 0;
    if constexpr (AXES)
        for (int t = lo + static_cast<int>(lane); t < hi; t += static_cast<int>(TPI)) {
            Rows<AXES> rows;
            good = rows_of<AXES>(p, static_cast<uint32_t>(seq.first + t - first), t, rows, bad) && good;
        }
    // What each of the new tokens' tasks does, with its rotated values.
    const auto each = [&](auto&& use) {
            for (uint32_t task = lane; task < tasks; task += TPI) {
                const uint32_t i = task % per_token;
                const int pos = lo + static_cast<int>(task / per_token), n = seq.first + pos - first;
                const Chunks ch = chunks_of(rot, p.rope.interleaved, i);
                Rows<AXES> rows{};
                if (!AXES || !is_v) rows_of<AXES>(p, static_cast<uint32_t>(n), pos, rows, bad);
                float x[16];
                load_rotated<F16, AXES>(p, x0 + static_cast<int64_t>(n) * src.token_stride, ch, i, rows, x);
                use(pos, ch, x);
            }
    };
    float amax = 0.f;
    each([&](int, const Chunks&, const float (&x)[16]) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const float a = fabsf(x[e]);
            if (a <= 3.4028235e38f) amax = fmaxf(amax, a);
        }
    });
    uint32_t bits = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax));   // |x| orders as its bits
    if constexpr (AXES) {   // keys and values alike; 0xFFFFFFFF is no finite maximum's
        if (__any_sync(0xFFFFFFFFu, !good)) bits = 0xFFFFFFFFu;
    }
    if constexpr (TPI > 32) {
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = bits;
        __syncthreads();
#pragma unroll
        for (uint32_t w = 0; w < kThreads / 32; ++w) bits = max(bits, warp_max[w]);
    }
    if (AXES && bits == 0xFFFFFFFFu) {
        if (!good) record_failure(&g_kv_append_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(bad));
        return;
    }
    const float scale = fmaxf(page_scale(__uint_as_float(bits)), old);
    const float inv = __frcp_rn(scale);   // exact for a power of two

    each([&](int pos, const Chunks& ch, const float (&x)[16]) {
        uint8_t* dst = codes + static_cast<int64_t>(pos - page * P) * p.c.token_stride;
        *reinterpret_cast<uint2*>(dst + ch.a) = make_uint2(encode4(x, inv), encode4(x + 4, inv));
        *reinterpret_cast<uint2*>(dst + ch.b) = make_uint2(encode4(x + 8, inv), encode4(x + 12, inv));
    });
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
                     const w8a16_rope_t& rope, const w8a16_rope_axes_t* axes, cudaStream_t s, std::string* err) {
    AppendArgs p{c, b, k, v, q, q_out, rope, 0, 0, 0, 0, {}};
    if (axes) {
        p.axes.positions = axes->positions, p.axes.stride = axes->axis_stride, p.axes.axes = axes->axes;
        for (uint32_t i = 0; i < rope.rotary_dim / 2; ++i) p.axes.of_pairs[i / 8] |= static_cast<uint16_t>(axes->pair_axis[i] << (2 * (i % 8)));
    }
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
    const auto pick = [&](auto with_axes) {
        constexpr bool A = decltype(with_axes)::value;
        return wide ? (f16 ? kv_append_kernel<true, kThreads, A> : kv_append_kernel<false, kThreads, A>)
                    : (f16 ? kv_append_kernel<true, 32, A> : kv_append_kernel<false, 32, A>);
    };
    const cudaError_t e = cudaLaunchKernelEx(&cfg, axes ? pick(std::true_type{}) : pick(std::false_type{}), p);
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

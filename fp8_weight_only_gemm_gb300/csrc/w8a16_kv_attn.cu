// Attention over the 8-bit paged cache, a few query rows per key/value head.
//
// Mathematics. For a row with query q at position p, over the keys j <= p:
//     o = sum_j w_j v_j / sum_j w_j,   w_j = exp(c ks_j (q . k_j)),   v_j = vs_j V_j
// with E4M3 codes k_j, V_j and the page scales ks_j, vs_j. One pass keeps a running
// maximum m of y_j = log2(e) c ks_j (q . k_j) + log2(vs_j), the sum l and the
// unnormalised output in FP32:
//     P_j = 2^(y_j - m + 7),   O += P_j V_j,   l += P_j / vs_j.
// m moves only when a y exceeds it by more than 8 (few steps do after the first; moving it
// means rescaling O). The value scale is part of the maximum, so P_j <= 2^15 whatever the
// scales are, and P is rounded once, to FP16: 11 bits, with 2^-31 of the largest weight
// still representable (l adds the rounded P where they have these bits). Both products run on FP16 operands: E4M3 converts to FP16 exactly
// (one instruction for two codes), and the query row is multiplied by a power of two
// that puts its largest element in [2^7, 2^8), so BF16 queries are exact too down to
// 2^-21 of their row's maximum. A non-finite query makes its row's outputs NaN.
//
// Layout. The products are m16n8k16 with the cache as M: S^T = K Q^T for 16 keys and 8
// query rows (the G query heads of one key/value head times the call's tokens), O^T = V^T P^T,
// so up to 8 rows waste nothing, and 9 to 16 use each converted operand twice. The order of a
// contraction's index and of an output's rows is free, and both are chosen so that every
// thread reads 16 consecutive codes of a key (16, or DP / 8, of a value): only P is
// transposed between the products (movmatrix). A warp's step is 16 keys, copied by the bulk
// copy engine into a ring of its own: two copies where a page's tokens are contiguous,
// else one a row.
//
// Work. The units (64 keys of one sequence, key/value head and 16-row tile) of the whole
// call, in that order, are split over the grid in equal contiguous ranges, so ragged
// lengths balance; the lengths are read on the device and the launch depends on none
// (it can be captured in a graph). The four warps of a CTA take 16 keys of each unit and
// join their (m, l, O) at the end of a range's part of an item; an item split
// between CTAs goes through the workspace in FP32 and a second, dependent kernel joins
// its parts in a fixed order: the result depends on nothing but the arguments.
//
// Bound by: long caches, by HBM. 32 sequences up to 8191 take 67 us for 342 MB (5.1 TB/s, 76 % of a
// plain copy's rate), one of 131000 55 us for 268 MB (4.9 TB/s); the loop over units alone runs at a
// copy's rate, the rest is the schedule (4 us to the first codes: lengths, page, codes are
// loads that wait for one another), the spread of the CTAs' ends and the join. Short ones
// (1000 tokens: 9.0 us) are that latency. Small heads with few rows a key (16 sequences of some 1000,
// five tokens, heads of 64: 22 us for 43 MB) are bound by instructions and by the fixed work of an
// item, 2 to 3 us a CTA. Rows: one tile of 8 if they fit, as a second doubles the products.
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "w8a16_kv_attn.cuh"

namespace w8a16 {
namespace {

__device__ DeviceStatus g_kv_attn_status;

constexpr uint32_t kWarps = 4, kThreads = 32 * kWarps;
constexpr uint32_t kMaxRows = 16;              // query rows of a tile: 8 NR
constexpr uint32_t kStepKeys = 16;             // keys of a warp's step (MMA M of the first product, K of the second)
constexpr uint32_t kUnitKeys = kWarps * kStepKeys;
constexpr uint32_t kStopped = 0x80000000u;
constexpr float kPBits = 7.f, kRise = 8.f;     // P = 2^(y - m + 7); m moves when exceeded by 8
constexpr float kNormalP = 6.103515625e-05f;   // 2^-14: above it FP16 keeps 11 bits

// DP: the head size rounded up to 64, 128 or 256. NR: tiles of 8 query rows, 1 or 2.
template <uint32_t DP, uint32_t NR>
struct Cfg {
    static constexpr uint32_t kRows = 8 * NR;
    static constexpr uint32_t kStages = 3;
    static constexpr uint32_t kCtasPerSm = DP >= 256 ? 2 : NR == 2 ? 3 : 4;   // by registers, and shared memory for 256
    static constexpr uint32_t kKChunks = DP / 64;             // 16-byte chunks of a key row per thread
    static constexpr uint32_t kVBytes = DP / 8;               // bytes of a value row per thread
    static constexpr uint32_t kVPiece = kVBytes < 16 ? kVBytes : 16;
    static constexpr uint32_t kVPieces = kVBytes / kVPiece;
    static constexpr uint32_t kStageBytes = 2 * kStepKeys * DP;
    static constexpr uint32_t kSmem = kWarps * kStages * kStageBytes;   // (rows of the head's own size, at most DP)
    static_assert(kStages * kStageBytes >= kRows * DP * 4, "a warp's outputs fit its ring");
};
constexpr uint32_t kMostCtasPerSm = 4;

// Workspace: slot (cta, which) = [kMaxRows][DP] outputs, [kMaxRows] maxima, [kMaxRows] sums.
__host__ __device__ constexpr uint32_t slot_floats(uint32_t dp) { return kMaxRows * dp + 2 * kMaxRows; }

// ------------------------------------------------------------ the schedule --
struct Items {
    uint32_t tiles;   // row tiles
    uint32_t units;   // per item
};
__device__ __forceinline__ Items items_of(const AttnArgs& p, const Seq& s) {
    const uint32_t len = static_cast<uint32_t>(max(s.len, 0));
    return {(static_cast<uint32_t>(s.count) * p.group + p.tile_rows - 1) / p.tile_rows, (len + kUnitKeys - 1) / kUnitKeys};
}
__device__ __forceinline__ uint64_t seq_units(const AttnArgs& p, uint32_t b, bool report) {
    const Seq s = sequence(p.b, p.c.page_size, b);
    if (s.bad && report) record_failure(&g_kv_attn_status, W8A16_STATUS_BAD_INDEX, b);
    const Items it = items_of(p, s);
    return static_cast<uint64_t>(it.tiles) * it.units * p.c.kv_heads;
}

// Units of all sequences (every thread gets the sum). `mine`, `before`: of sequence threadIdx.x and
// ahead of it, where there are no more sequences than threads.
__device__ __forceinline__ uint64_t count_units(const AttnArgs& p, uint64_t* sh, uint64_t& mine, uint64_t& before) {
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    mine = 0;
    for (uint32_t i = threadIdx.x; i < p.b.batch; i += kThreads) mine += seq_units(p, i, blockIdx.x == 0);
    uint64_t inc = mine;   // inclusive scan of the warp, then of the block
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= static_cast<uint32_t>(o)) inc += t;
    }
    if (lane == 31) sh[warp] = inc;
    __syncthreads();
    uint64_t all = 0;
    before = inc - mine;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) {
        if (w < warp) before += sh[w];
        all += sh[w];
    }
    return all;
}

// The sequence that holds unit `at` (below the total), and its first unit: of the counts already there, or,
// for more sequences than threads, in blocks of them.
__device__ __forceinline__ void find_unit(const AttnArgs& p, uint64_t at, uint64_t* sh, uint64_t mine, uint64_t before, uint32_t& b,
                                          uint64_t& base) {
    uint64_t run = 0;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.b.batch <= kThreads) {
        if (at >= before && at < before + mine) {
            sh[kWarps] = before;
            sh[kWarps + 1] = threadIdx.x;
        }
        __syncthreads();
    }
    for (uint32_t i0 = 0; p.b.batch > kThreads && i0 < p.b.batch; i0 += kThreads) {
        const uint32_t i = i0 + threadIdx.x;
        const uint64_t v = i < p.b.batch ? seq_units(p, i, false) : 0;
        __syncthreads();    // sh has been read
        uint64_t inc = v;   // inclusive scan of the warp, then of the block
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint64_t t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= static_cast<uint32_t>(o)) inc += t;
        }
        if (lane == 31) sh[warp] = inc;
        __syncthreads();
        uint64_t off = run, total = run;
#pragma unroll
        for (uint32_t w = 0; w < kWarps; ++w) {
            if (w < warp) off += sh[w];
            total += sh[w];
        }
        if (at >= off + inc - v && at < off + inc) {
            sh[kWarps] = off + inc - v;
            sh[kWarps + 1] = i;
        }
        __syncthreads();
        if (at < total) break;
        run = total;
    }
    base = sh[kWarps];
    b = static_cast<uint32_t>(sh[kWarps + 1]);
    __syncthreads();
}

// ------------------------------------------------------------- primitives --
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag) {
    return mbar_wait_for(bar, parity, timeout_ns, abort_flag, &g_kv_attn_status, 1);
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// ----------------------------------------------------------------- kernel --
template <bool F16, uint32_t DP, uint32_t NR>
__global__ void __launch_bounds__(kThreads, (Cfg<DP, NR>::kCtasPerSm)) kv_attn_kernel(const AttnArgs p) {
    using C = Cfg<DP, NR>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t sh[2 * kWarps];
    __shared__ float sh_m[kWarps][C::kRows], sh_l[kWarps][C::kRows];
    __shared__ uint64_t full[kWarps][C::kStages];
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kWarps * C::kStages; ++i) mbar_init(smem_u32(&full[0][0] + i), 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    grid_dependency_wait();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    uint64_t mine, before;
    const uint64_t total = count_units(p, sh, mine, before), ctas = active_ctas(total, p.ctas);
    zero_keyless(p);
    if (blockIdx.x >= ctas) {
        if (threadIdx.x == 0) write_boundary(p.ws, 0, 0, 0, Seq{}, 0, 0, total, ctas);
        return;
    }
    float* const slots = p.ws + boundary_floats(p.ctas);
    uint64_t u = first_unit(blockIdx.x, total, ctas);
    const uint64_t u_end = first_unit(blockIdx.x + 1, total, ctas);
    uint32_t b;
    uint64_t base;
    find_unit(p, u, sh, mine, before, b, base);

    uint8_t* const ring = smem + warp * C::kStages * C::kStageBytes;
    float* const merge = reinterpret_cast<float*>(ring);
    const uint32_t D = p.c.head_dim;
    const uint32_t ts = static_cast<uint32_t>(p.c.token_stride);   // at most 2^22: a page's tokens within 32 bits
    uint32_t k_at[C::kKChunks], v_at[C::kVPieces];   // this thread's bytes of a step: chunks past the head repeat its last
#pragma unroll
    for (uint32_t i = 0; i < C::kKChunks; ++i) k_at[i] = g * D + min(i * 64 + c * 16, D - 16);
#pragma unroll
    for (uint32_t i = 0; i < C::kVPieces; ++i) v_at[i] = (kStepKeys + 2 * c) * D + min(g * C::kVPiece + i * 8 * C::kVPiece, D - C::kVPiece);
    uint32_t taken = 0;   // steps of this warp so far; kStopped once a wait has given up
    bool first_part = true;

    while (u < u_end) {
        Seq seq = sequence(p.b, p.c.page_size, b);
        Items it = items_of(p, seq);
        uint64_t n_b = static_cast<uint64_t>(it.tiles) * it.units * p.c.kv_heads;
        while (u >= base + n_b) {   // the next sequence with work
            base += n_b;
            seq = sequence(p.b, p.c.page_size, ++b);
            it = items_of(p, seq);
            n_b = static_cast<uint64_t>(it.tiles) * it.units * p.c.kv_heads;
        }
        const uint64_t in_seq = u - base;
        const uint32_t item = static_cast<uint32_t>(divide(in_seq, it.units));
        const uint32_t unit0 = static_cast<uint32_t>(in_seq - static_cast<uint64_t>(item) * it.units);
        const uint32_t nunits = static_cast<uint32_t>(min(static_cast<uint64_t>(it.units - unit0), u_end - u));
        const uint32_t h = item / it.tiles, row0 = (item % it.tiles) * C::kRows;
        const uint32_t nrows = static_cast<uint32_t>(seq.count) * p.group;
        const int before = seq.len - seq.count + 1;   // keys that the sequence's first token sees
        // keys that any row, and every row, of the tile sees
        const int tile_end = before + static_cast<int>((min(row0 + C::kRows, nrows) - 1) / p.group),
                  tile_min = before + static_cast<int>(row0 / p.group);

        // ---- this warp's steps: 16 keys of each unit
        const int key0 = static_cast<int>(unit0 * kUnitKeys + warp * kStepKeys);
        const uint32_t nsteps = taken == kStopped ? 0u : static_cast<uint32_t>(max(0, min(static_cast<int>(nunits), (tile_end - key0 + static_cast<int>(kUnitKeys) - 1) / static_cast<int>(kUnitKeys))));
        // Lane l holds what step l (mod 32) of a batch of 32 needs; a batch is asked for kStages - 1
        // steps before its first use, and its scales are first touched there.
        int meta_page = 0;
        float meta_k = 1.f, meta_v = 1.f, cur_k = 1.f, cur_lv = 0.f, cur_iv = 1.f;
        const auto load_meta = [&](uint32_t step) {
            const int key = key0 + static_cast<int>((step + lane) * kUnitKeys);
            meta_page = 0;
            meta_k = meta_v = 1.f;
            if (step + lane < nsteps) {
                const int page = p.b.page_table[static_cast<int64_t>(b) * p.b.page_table_stride + (key >> p.page_shift)];
                if (static_cast<uint32_t>(page) >= p.c.num_pages) {   // page 0 instead
                    record_failure(&g_kv_attn_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(page));
                } else {
                    const int64_t at = static_cast<int64_t>(page) * p.c.scale_page_stride + static_cast<int64_t>(h) * p.c.scale_head_stride;
                    meta_page = page;
                    meta_k = p.c.k_scale[at];
                    meta_v = p.c.v_scale[at];
                }
            }
        };
        // This lane's source: K for lane 0 (or lanes 0-15, a row each), V for lane 1 (or 16-31).
        // Keys past the last one repeat it: their scores are masked, and their values are as finite as
        // those that they repeat (where rows see different keys: see below).
        const auto issue = [&](uint32_t step) {
            if (step >= nsteps) return;
            if ((step & 31u) == 0u) load_meta(step);
            const int page = __shfl_sync(0xFFFFFFFFu, meta_page, step & 31u);
            const int key = key0 + static_cast<int>(step * kUnitKeys);
            const uint32_t at = (taken + step) % C::kStages, slot = smem_u32(ring) + at * C::kStageBytes, bar = smem_u32(&full[warp][at]);
            const bool block = ts == D && tile_end - key >= static_cast<int>(kStepKeys);
            const uint8_t* src = static_cast<const uint8_t*>((block ? lane & 1u : lane & 16u) ? p.c.v_codes : p.c.k_codes) +
                                 static_cast<int64_t>(h) * p.c.head_stride + static_cast<int64_t>(page) * p.c.page_stride +
                                 static_cast<uint32_t>(key & static_cast<int>(p.c.page_size - 1)) * ts;
            if (lane == 0) mbar_arrive_expect_tx(bar, 2 * kStepKeys * D);
            __syncwarp();
            if (block) {
                if (lane < 2) bulk_copy(slot + lane * kStepKeys * D, src, kStepKeys * D, bar);
            } else {
                bulk_copy(slot + lane * D, src + min(lane & 15u, static_cast<uint32_t>(tile_end - key - 1)) * ts, D, bar);
            }
        };
#pragma unroll 1
        for (uint32_t s = 0; s < C::kStages - 1; ++s) issue(s);

        // ---- the query tile: row 8 t + g of it, FP16, each times 2^(7 - exponent of its maximum)
        uint32_t qf[NR][C::kKChunks][4][2];
        float row_scale[NR][2];   // of rows 8 t + 2 c + e
        int row_end[NR][2];       // keys that they see
#pragma unroll
        for (uint32_t t = 0; t < NR; ++t) {
            const uint32_t row = row0 + 8 * t + g;
            const bool real = row < nrows;
            const uint16_t* src = static_cast<const uint16_t*>(p.q.ptr) +
                                  static_cast<int64_t>(seq.first + static_cast<int>(real ? row / p.group : 0)) * p.q.token_stride +
                                  static_cast<int64_t>(h * p.group + (real ? row % p.group : 0)) * p.q.head_stride;
            uint32_t raw[C::kKChunks][8];
#pragma unroll
            for (uint32_t i = 0; i < C::kKChunks; ++i) {
                const uint32_t d = i * 64 + c * 16;
                uint4 a = make_uint4(0, 0, 0, 0), e = a;
                if (real && d < D) {
                    a = *reinterpret_cast<const uint4*>(src + d);
                    e = *reinterpret_cast<const uint4*>(src + d + 8);
                }
                raw[i][0] = a.x, raw[i][1] = a.y, raw[i][2] = a.z, raw[i][3] = a.w;
                raw[i][4] = e.x, raw[i][5] = e.y, raw[i][6] = e.z, raw[i][7] = e.w;
            }
            float mx = 0.f;
            bool finite = true;
#pragma unroll
            for (uint32_t i = 0; i < C::kKChunks; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 x = unpack2<F16>(raw[i][k]);
                    finite = finite && fabsf(x.x) <= 3.4028235e38f && fabsf(x.y) <= 3.4028235e38f;
                    mx = fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            const bool bad = (__ballot_sync(0xFFFFFFFFu, !finite) >> (4 * g) & 15u) != 0u;   // by the row's four lanes
            const RowScale rs = row_scale_of(mx, bad, p.scale_log2);
            // a padding row is one that sees no key: it is zero whatever its query holds
            const float mine = bad && before + static_cast<int>(row / p.group) <= 0 ? 0.f : rs.scale;
#pragma unroll
            for (uint32_t e = 0; e < 2; ++e) {
                row_scale[t][e] = __shfl_sync(0xFFFFFFFFu, mine, 4 * (2 * c + e));
                const uint32_t r = row0 + 8 * t + 2 * c + e;
                row_end[t][e] = r < nrows ? before + static_cast<int>(r / p.group) : 0x7FFFFFFF;
            }
#pragma unroll
            for (uint32_t i = 0; i < C::kKChunks; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 x = unpack2<F16>(raw[i][k]);
                    qf[t][i][k >> 1][k & 1] = bad ? 0u : pack2<true>(x.x * rs.f1 * rs.f2, x.y * rs.f1 * rs.f2);
                }
        }

        // O^T: tile mt, rows 2 mt and 2 mt + 1 of this thread's 2 DP / 16 dims
        float o[NR][DP / 16][4];
#pragma unroll
        for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
            for (uint32_t n = 0; n < DP / 16; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
        float m[NR][2], l[NR][2];   // of rows 8 t + 2 c + e; l: this lane's keys
#pragma unroll
        for (uint32_t t = 0; t < NR; ++t) m[t][0] = m[t][1] = -INFINITY, l[t][0] = l[t][1] = 0.f;

#pragma unroll 1
        for (uint32_t step = 0; step < nsteps; ++step) {
            const uint32_t at = (taken + step) % C::kStages, parity = ((taken + step) / C::kStages) & 1;
            if (!__all_sync(0xFFFFFFFFu, mbar_try_wait(smem_u32(&full[warp][at]), parity) ||
                                             wait_slow(smem_u32(&full[warp][at]), parity, p.timeout_ns, &abort_flag))) {
                ring_drain<C::kStages>(full[warp], taken + step, taken + min(step + C::kStages - 1, nsteps), p.timeout_ns, &g_kv_attn_status, 2);
                taken = kStopped - nsteps;   // the phases no longer count: no steps of later items
                break;
            }
            if ((step & 31u) == 0u) {   // the batch of 32 that the copies have reached
                cur_k = meta_k < kMinScale ? kMinScale : meta_k;
                const float v = meta_v < kMinScale ? kMinScale : meta_v;
                cur_lv = __log2f(v);
                cur_iv = __frcp_rn(v);
            }
            // the slot before this one has been read by all lanes: the next copies may overwrite it
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            issue(step + C::kStages - 1);
            const int key = key0 + static_cast<int>(step * kUnitKeys);
            const float ks = __shfl_sync(0xFFFFFFFFu, cur_k, step & 31u), lv = __shfl_sync(0xFFFFFFFFu, cur_lv, step & 31u),
                        iv = __shfl_sync(0xFFFFFFFFu, cur_iv, step & 31u);
            const uint8_t* slot = ring + at * C::kStageBytes;

            // ---- scores of keys g, g + 8 and rows 2 c, 2 c + 1; two chains of products each
            float s[NR][4], s2[NR][4];
#pragma unroll
            for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[t][e] = s2[t][e] = 0.f;
#pragma unroll
            for (uint32_t i = 0; i < C::kKChunks; ++i) {
                const uint4 w0 = *reinterpret_cast<const uint4*>(slot + k_at[i]), w1 = *reinterpret_cast<const uint4*>(slot + 8 * D + k_at[i]);
                const uint32_t x0[4] = {w0.x, w0.y, w0.z, w0.w}, x1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t a[4];
                    e4m3x4_to_f16x4(x0[k], a[0], a[2]);
                    e4m3x4_to_f16x4(x1[k], a[1], a[3]);
#pragma unroll
                    for (uint32_t t = 0; t < NR; ++t) mma_f16(k & 1 ? s2[t] : s[t], a, qf[t][i][k][0], qf[t][i][k][1]);
                }
            }
            // ---- weights
            const bool edge = key + static_cast<int>(kStepKeys) > tile_min;
            float f[NR][2], mx[NR][2];
            bool rise = false;
#pragma unroll
            for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    s[t][e] += s2[t][e];
                    s[t][2 + e] += s2[t][2 + e];
                    f[t][e] = logit_factor(ks, row_scale[t][e]);
                    if (edge) {
                        if (key + static_cast<int>(g) >= row_end[t][e]) s[t][e] = -INFINITY;
                        if (key + 8 + static_cast<int>(g) >= row_end[t][e]) s[t][2 + e] = -INFINITY;
                    }
                    // f > 0: the largest score gives the largest y = score f + log2(vs)
                    float x = fmaxf(s[t][e], s[t][2 + e]);
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
                    mx[t][e] = fmaf(x, f[t][e], lv);
                    rise = rise || mx[t][e] > m[t][e] + kRise;
                }
            if (__any_sync(0xFFFFFFFFu, rise)) {
                // a running maximum is exceeded by more than 2^8: it moves, sums and outputs are rescaled
#pragma unroll
                for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float m_new = fmaxf(m[t][e], mx[t][e]);
                        const float a = m[t][e] == -INFINITY ? 0.f : ex2(m[t][e] - m_new);
                        l[t][e] *= a;
#pragma unroll
                        for (uint32_t n = 0; n < DP / 16; ++n) {
                            o[t][n][e] *= a;
                            o[t][n][2 + e] *= a;
                        }
                        m[t][e] = m_new;
                    }
            }
            uint32_t pb[NR][2];   // P^T as the second product's operand: keys 2 c.. of row g
#pragma unroll
            for (uint32_t t = 0; t < NR; ++t) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float d = m[t][e] == -INFINITY ? 0.f : lv - m[t][e] + kPBits;
                    y[e] = ex2(fmaf(s[t][e], f[t][e], d));
                    y[2 + e] = ex2(fmaf(s[t][2 + e], f[t][e], d));
                }
                // The sum takes the weights as they were rounded: where one key has most of it, the rounding
                // cancels. Small ones as they are: a page with a small scale has small P and large P / vs.
                const uint32_t w0 = pack2<true>(y[0], y[1]), w1 = pack2<true>(y[2], y[3]);
                const float2 r0 = unpack2<true>(w0), r1 = unpack2<true>(w1);
                const auto kept = [](float x, float rounded) { return x > kNormalP ? rounded : x; };
                l[t][0] = fmaf(kept(y[0], r0.x) + kept(y[2], r1.x), iv, l[t][0]);
                l[t][1] = fmaf(kept(y[1], r0.y) + kept(y[3], r1.y), iv, l[t][1]);
                pb[t][0] = transpose8x8(w0);
                pb[t][1] = transpose8x8(w1);
            }
            // ---- outputs
            uint32_t vw[4][C::kVBytes / 4];   // keys 2 c, 2 c + 1, 8 + 2 c, 9 + 2 c
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                for (uint32_t i = 0; i < C::kVPieces; ++i) {
                    const uint8_t* from = slot + (8 * (j >> 1) + (j & 1)) * D + v_at[i];
                    if constexpr (C::kVPiece == 16) {
                        const uint4 w = *reinterpret_cast<const uint4*>(from);
                        vw[j][4 * i] = w.x, vw[j][4 * i + 1] = w.y, vw[j][4 * i + 2] = w.z, vw[j][4 * i + 3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(from);
                        vw[j][0] = w.x, vw[j][1] = w.y;
                    }
                }
            if (edge && seq.count > 1) {
                // keys that some rows do not see: a NaN value there must not reach them through 0 * NaN.
                // The NaN codes leave the product, and a product of indicators (value is NaN, row sees key)
                // marks the outputs that are NaN.
                uint32_t any = 0;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                    for (uint32_t i = 0; i < C::kVBytes / 4; ++i) any |= e4m3_nan_flags(vw[j][i]);
                if (__any_sync(0xFFFFFFFFu, any != 0u)) {
                    uint32_t seen[NR][2];
#pragma unroll
                    for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            seen[t][k] = transpose8x8(pack2<true>(key + 8 * k + static_cast<int>(g) < row_end[t][0] ? 1.f : 0.f,
                                                                  key + 8 * k + static_cast<int>(g) < row_end[t][1] ? 1.f : 0.f));
#pragma unroll
                    for (uint32_t i = 0; i < C::kVBytes / 4; ++i) {
                        uint32_t ind[4];
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j) {
                            const uint32_t nan = (e4m3_nan_flags(vw[j][i]) >> 7) * 0xFFu;   // 0xFF where NaN
                            ind[j] = nan & 0x38383838u;                                     // E4M3 1.0
                            vw[j][i] &= ~nan;
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t sel = half ? 0x7362u : 0x5140u;
                            uint32_t a[4];
                            e4m3x4_to_f16x4(prmt(ind[0], ind[1], sel), a[0], a[1]);
                            e4m3x4_to_f16x4(prmt(ind[2], ind[3], sel), a[2], a[3]);
#pragma unroll
                            for (uint32_t t = 0; t < NR; ++t) {
                                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(hit, a, seen[t][0], seen[t][1]);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    if (hit[e] > 0.f) o[t][2 * i + half][e] = __uint_as_float(0x7FC00000u);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (uint32_t i = 0; i < C::kVBytes / 4; ++i)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x7362u : 0x5140u;   // (key, key + 1) byte pairs of two dims
                    uint32_t a[4];
                    e4m3x4_to_f16x4(prmt(vw[0][i], vw[1][i], sel), a[0], a[1]);
                    e4m3x4_to_f16x4(prmt(vw[2][i], vw[3][i], sel), a[2], a[3]);
#pragma unroll
                    for (uint32_t t = 0; t < NR; ++t) mma_f16(o[t][2 * i + half], a, pb[t][0], pb[t][1]);
                }
        }
        taken += nsteps;

        // ---- join the warps' parts. Word i of a value row piece holds dims 4 i .. 4 i + 3 of it: tile
        // 2 i + half, elements e and 2 + e are dims 4 i + 2 half and + 1 of row 2 c + e.
#pragma unroll
        for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[t][e] += __shfl_xor_sync(0xFFFFFFFFu, l[t][e], 4);
                l[t][e] += __shfl_xor_sync(0xFFFFFFFFu, l[t][e], 8);
                l[t][e] += __shfl_xor_sync(0xFFFFFFFFu, l[t][e], 16);
                if (g == 0) {
                    sh_m[warp][8 * t + 2 * c + e] = m[t][e];
                    sh_l[warp][8 * t + 2 * c + e] = l[t][e];
                }
            }
        __syncwarp();   // every lane is done with its ring slots, which `merge` reuses
#pragma unroll
        for (uint32_t t = 0; t < NR; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (uint32_t i = 0; i < C::kVBytes / 4; ++i) {
                    const uint32_t d = (4 * i / C::kVPiece) * 8 * C::kVPiece + g * C::kVPiece + 4 * i % C::kVPiece;
                    *reinterpret_cast<float4*>(merge + (8 * t + 2 * c + e) * DP + d) =
                        make_float4(o[t][2 * i][e], o[t][2 * i][2 + e], o[t][2 * i + 1][e], o[t][2 * i + 1][2 + e]);
                }
        __syncthreads();
        const bool whole = nunits == it.units;
        if (first_part && threadIdx.x == 0) write_boundary(p.ws, u, u - unit0, it.units, seq, h, item % it.tiles, total, ctas);
        float* const slot_ws = slots + (static_cast<uint64_t>(blockIdx.x) * 2 + (first_part ? 0 : 1)) * slot_floats(DP);
#pragma unroll 1
        for (uint32_t i = threadIdx.x; i < C::kRows * DP / 4; i += kThreads) {
            const uint32_t r = i / (DP / 4), d = (i % (DP / 4)) * 4;
            if (row0 + r >= nrows || d >= D) continue;
            float mm = sh_m[0][r];
#pragma unroll
            for (uint32_t w = 1; w < kWarps; ++w) mm = fmaxf(mm, sh_m[w][r]);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float ll = 0.f;
#pragma unroll
            for (uint32_t w = 0; w < kWarps; ++w) {
                const float a = sh_m[w][r] == -INFINITY ? 0.f : ex2(sh_m[w][r] - mm);
                const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + w * C::kStages * C::kStageBytes) + r * DP + d);
                acc.x = fmaf(a, x.x, acc.x);
                acc.y = fmaf(a, x.y, acc.y);
                acc.z = fmaf(a, x.z, acc.z);
                acc.w = fmaf(a, x.w, acc.w);
                ll = fmaf(a, sh_l[w][r], ll);
            }
            if (whole) {
                const float inv = ll == 0.f ? 0.f : 1.f / ll;   // a row that sees no key is zero
                const uint32_t row = row0 + r;
                uint16_t* dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(seq.first + static_cast<int>(row / p.group)) * p.out.token_stride +
                                static_cast<int64_t>(h * p.group + row % p.group) * p.out.head_stride + d;
                *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<F16>(acc.x * inv, acc.y * inv), pack2<F16>(acc.z * inv, acc.w * inv));
            } else {
                *reinterpret_cast<float4*>(slot_ws + r * DP + d) = acc;
                if (d == 0) {
                    slot_ws[kMaxRows * DP + r] = mm;
                    slot_ws[kMaxRows * DP + kMaxRows + r] = ll;
                }
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();   // the rings and sh_* are free again
        first_part = false;
        u += nunits;
        // The join's blocks come in only now: let in at the start they, and behind them the next call's CTAs,
        // took the places of CTAs that were done early (32 sequences to 8191: 81 us a call instead of 68).
        if (u >= u_end) grid_launch_dependents();
    }
}

template <uint32_t V>
__device__ __forceinline__ void load_dims(const float* from, float (&x)[V]) {
    if constexpr (V == 2) {
        const float2 t = *reinterpret_cast<const float2*>(from);
        x[0] = t.x, x[1] = t.y;
    } else {
#pragma unroll
        for (uint32_t k = 0; k < V; k += 4) {
            const float4 t = *reinterpret_cast<const float4*>(from + k);
            x[k] = t.x, x[k + 1] = t.y, x[k + 2] = t.z, x[k + 3] = t.w;
        }
    }
}
// Joins the parts of split items, in an order that their number alone decides: a block for the k-th
// split item and a row, whose warps take parts in turn, 8 in flight each. It is bound by the latency
// of three loads, one after another. (A warp for all parts of a row: 72 us instead of 54 for one
// sequence of 131000 tokens, whose items have 77 parts each, 12.4 for 9.6 at 1000; for 128 sequences
// of 1000, whose items have 2, 78 for 70. 8 warps a row: 79 there.)
template <bool F16, uint32_t DP>
__global__ void __launch_bounds__(kThreads) kv_attn_join_kernel(const AttnArgs p) {
    __shared__ float sh_m[kWarps], sh_l[kWarps];
    __shared__ __align__(16) float sh_acc[kWarps][DP];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y;
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t c = split_boundary<kThreads>(p, blockIdx.x);
    if (c == 0) return;   // fewer items are split
    const Boundary b = reinterpret_cast<const Boundary*>(p.ws)[c];
    const uint32_t row = b.tile * p.tile_rows + r;
    if (row >= static_cast<uint32_t>(b.count) * p.group) return;
    const float* const slots = p.ws + boundary_floats(p.ctas);
    constexpr uint32_t V = DP / 32, kAtOnce = 8;
    float m = -INFINITY, l = 0.f, acc[V] = {};
    for (uint32_t i0 = warp; i0 < b.parts; i0 += kWarps * kAtOnce) {
        float x[kAtOnce][V], mi[kAtOnce], li[kAtOnce];
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            const uint32_t i = i0 + kWarps * j;
            mi[j] = -INFINITY, li[j] = 0.f;
#pragma unroll
            for (uint32_t e = 0; e < V; ++e) x[j][e] = 0.f;
            if (i < b.parts) {
                const float* const s = slots + static_cast<uint64_t>(i == 0 ? b.slot : 2 * (c + i - 1)) * slot_floats(DP);
                mi[j] = s[kMaxRows * DP + r], li[j] = s[kMaxRows * DP + kMaxRows + r];
                load_dims<V>(s + r * DP + V * lane, x[j]);
            }
        }
        float top = m;
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) top = fmaxf(top, mi[j]);
        const float keep = m == -INFINITY ? 0.f : ex2(m - top);
        l *= keep;
#pragma unroll
        for (uint32_t e = 0; e < V; ++e) acc[e] *= keep;
        m = top;
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            const float a = mi[j] == -INFINITY ? 0.f : ex2(mi[j] - m);   // (0 times NaN: a query that is not finite)
            l = fmaf(a, li[j], l);
#pragma unroll
            for (uint32_t e = 0; e < V; ++e) acc[e] = fmaf(a, x[j][e], acc[e]);
        }
    }
#pragma unroll
    for (uint32_t e = 0; e < V; ++e) sh_acc[warp][V * lane + e] = acc[e];
    if (lane == 0) sh_m[warp] = m, sh_l[warp] = l;
    __syncthreads();
    const uint32_t d = 2 * threadIdx.x;
    if (d >= p.c.head_dim) return;
    float top = sh_m[0];
#pragma unroll
    for (uint32_t w = 1; w < kWarps; ++w) top = fmaxf(top, sh_m[w]);
    float x0 = 0.f, x1 = 0.f, sum = 0.f;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) {
        const float a = sh_m[w] == -INFINITY ? 0.f : ex2(sh_m[w] - top);
        sum = fmaf(a, sh_l[w], sum);
        x0 = fmaf(a, sh_acc[w][d], x0), x1 = fmaf(a, sh_acc[w][d + 1], x1);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* const dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(b.first + static_cast<int>(row / p.group)) * p.out.token_stride +
                          static_cast<int64_t>(b.h * p.group + row % p.group) * p.out.head_stride;
    *reinterpret_cast<uint32_t*>(dst + d) = pack2<F16>(x0 * inv, x1 * inv);
}

template <bool F16, uint32_t DP, uint32_t NR>
cudaError_t launch(AttnArgs p, int sms, cudaStream_t s) {
    using C = Cfg<DP, NR>;
    p.tile_rows = C::kRows;
    p.ctas = static_cast<uint32_t>(sms) * C::kCtasPerSm;
    cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<F16, DP, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(p.ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv_attn_kernel<F16, DP, NR>, p);
    if (e != cudaSuccess || p.ctas < 2) return e;
    const uint64_t rows = static_cast<uint64_t>(p.b.max_q) * p.group;   // of an item, at most
    const uint32_t item_rows = static_cast<uint32_t>(rows < C::kRows ? rows : C::kRows);
    cfg.dynamicSmemBytes = 0;
    const uint64_t items = static_cast<uint64_t>(p.b.batch) * p.c.kv_heads * ((rows + C::kRows - 1) / C::kRows);
    cfg.gridDim = dim3(static_cast<uint32_t>(items < p.ctas ? items : p.ctas - 1), item_rows, 1);   // no more are split
    return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<F16, DP>, p);
}
template <bool F16, uint32_t DP>
cudaError_t launch_rows(const AttnArgs& p, int sms, cudaStream_t s) {
    return p.b.max_q * static_cast<uint64_t>(p.group) <= 8 ? launch<F16, DP, 1>(p, sms, s) : launch<F16, DP, 2>(p, sms, s);
}
template <bool F16>
cudaError_t launch_dim(const AttnArgs& p, int sms, cudaStream_t s) {
    return p.c.head_dim <= 64 ? launch_rows<F16, 64>(p, sms, s) : p.c.head_dim <= 128 ? launch_rows<F16, 128>(p, sms, s) : launch_rows<F16, 256>(p, sms, s);
}

}  // namespace

uint64_t kv_attn_ws_bytes(uint32_t head_dim, uint32_t rows_per_head, int sms) {
    if (kv_attn_tc_applies(head_dim, rows_per_head)) return kv_attn_tc_ws_bytes(head_dim, sms);
    const uint32_t ctas = static_cast<uint32_t>(sms) * kMostCtasPerSm, dp = head_dim <= 64 ? 64u : head_dim <= 128 ? 128u : 256u;
    return 4 * boundary_floats(ctas) + 8ull * ctas * slot_floats(dp);
}

int launch_kv_attn(const w8a16_kv_cache_t& c, const w8a16_kv_batch_t& b, uint32_t act_dtype, const w8a16_heads_t& q,
                   const w8a16_heads_t& out, float softmax_scale, void* ws, int sms, uint64_t timeout_ns, cudaStream_t s,
                   std::string* err) {
    AttnArgs p{c, b, q, out, static_cast<float*>(ws), softmax_scale * 1.4426950408889634f, q.heads / c.kv_heads, 0, 0, 0, timeout_ns};
    while ((1u << p.page_shift) < c.page_size) ++p.page_shift;
    const bool f16 = act_dtype == W8A16_ACT_F16;
    const cudaError_t e = kv_attn_tc_applies(c.head_dim, b.max_q * p.group)
                              ? launch_kv_attn_tc(p, f16, sms, s)
                              : f16 ? launch_dim<true>(p, sms, s) : launch_dim<false>(p, sms, s);
    if (e != cudaSuccess) {
        cudaGetLastError();
        *err = std::string("cache attention launch failed: ") + cudaGetErrorString(e);
        return W8A16_ERR_LAUNCH;
    }
    return W8A16_OK;
}

cudaError_t kv_attn_status_read(StatusWord* out, bool clear, cudaStream_t s) {
    DeviceStatus st;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&st, g_kv_attn_status, sizeof st, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    out->code = st.code;
    out->where = st.where;
    out->detail = st.detail;
    if (clear) {
        const DeviceStatus zero{0, 0, 0};
        e = cudaMemcpyToSymbolAsync(g_kv_attn_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace w8a16

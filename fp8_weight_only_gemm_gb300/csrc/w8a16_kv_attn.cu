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
// still representable. Both products run on FP16 operands: E4M3 converts to FP16 exactly
// (one instruction for two codes), and the query row is multiplied by a power of two
// that puts its largest element in [2^7, 2^8), so BF16 queries are exact too down to
// 2^-21 of their row's maximum. A non-finite query makes its row's outputs NaN.
//
// Layout. The products are m16n8k16 with 16 query rows (the G query heads of one
// key/value head times the call's tokens) as M. The order of a contraction's index and of
// an output's columns is free, and both are chosen so that every thread reads 16
// consecutive codes of a key (16, or DP / 8, of a value) and nobody else reads them: a
// thread copies its own fragments with cp.async into a slot of its own, a ring that
// needs no barrier at all.
//
// Work. The units (64 keys of one sequence, key/value head and 16-row tile) of the whole
// call, in that order, are split over the grid in equal contiguous ranges, so ragged
// lengths balance; the lengths are read on the device and the launch depends on none
// (it can be captured in a graph). The four warps of a CTA take 16 keys of each unit and
// join their (m, l, O) at the end of a range's part of an item; an item split
// between CTAs goes through the workspace in FP32 and a second, dependent kernel joins
// its parts in key order: the result depends on nothing but the arguments.
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "w8a16_kv_attn.cuh"

namespace w8a16 {
namespace {

__device__ DeviceStatus g_kv_attn_status;

constexpr uint32_t kWarps = 4, kThreads = 32 * kWarps;
constexpr uint32_t kRows = 16;                 // query rows of a tile (MMA M)
constexpr uint32_t kStepKeys = 16;             // keys of a warp's step (two n8 tiles; MMA K of the second product)
constexpr uint32_t kUnitKeys = kWarps * kStepKeys;
constexpr float kPBits = 7.f, kRise = 8.f;     // P = 2^(y - m + 7); m moves when exceeded by 8

template <uint32_t DP>
struct Cfg {
    static constexpr uint32_t kStages = DP >= 256 ? 3 : 4;
    static constexpr uint32_t kCtasPerSm = DP >= 256 ? 2 : 3;
    static constexpr uint32_t kKChunks = DP / 64;             // 16-byte chunks of a key row per thread
    static constexpr uint32_t kVBytes = DP / 8;               // bytes of a value row per thread
    static constexpr uint32_t kVPiece = kVBytes < 16 ? kVBytes : 16;
    static constexpr uint32_t kVPieces = kVBytes / kVPiece;
    static constexpr uint32_t kStageBytes = 2 * kStepKeys * DP;
    static constexpr uint32_t kSmem = kWarps * kStages * kStageBytes;
    static_assert(kStages * kStageBytes >= kRows * DP * 4, "a warp's outputs fit its ring");
};

// Workspace: slot (cta, which) = [kRows][DP] outputs, [kRows] maxima, [kRows] sums.
__host__ __device__ constexpr uint32_t slot_floats(uint32_t dp) { return kRows * dp + 2 * kRows; }

// ------------------------------------------------------------ the schedule --
struct Items {
    uint32_t tiles;   // row tiles
    uint32_t units;   // per item
};
__device__ __forceinline__ Items items_of(const AttnArgs& p, const Seq& s) {
    const uint32_t len = static_cast<uint32_t>(max(s.len, 0));
    return {(static_cast<uint32_t>(s.count) * p.group + kRows - 1) / kRows, (len + kUnitKeys - 1) / kUnitKeys};
}
__device__ __forceinline__ uint64_t seq_units(const AttnArgs& p, uint32_t b, bool report) {
    const Seq s = sequence(p.b, p.c.page_size, b);
    if (s.bad && report) record_failure(&g_kv_attn_status, W8A16_STATUS_BAD_INDEX, b);
    const Items it = items_of(p, s);
    return static_cast<uint64_t>(it.tiles) * it.units * p.c.kv_heads;
}

// Units of all sequences (every thread gets the sum).
__device__ __forceinline__ uint64_t count_units(const AttnArgs& p, uint64_t* sh) {
    uint64_t x = 0;
    for (uint32_t i = threadIdx.x; i < p.b.batch; i += kThreads) x += seq_units(p, i, blockIdx.x == 0);
    x = warp_sum(x);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kWarps; ++w) all += sh[w];
    __syncthreads();
    return all;
}

// The sequence that holds unit `at` (below the total), and its first unit.
__device__ __forceinline__ void find_unit(const AttnArgs& p, uint64_t at, uint64_t* sh, uint32_t& b, uint64_t& base) {
    uint64_t run = 0;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (uint32_t i0 = 0; i0 < p.b.batch; i0 += kThreads) {
        const uint32_t i = i0 + threadIdx.x;
        const uint64_t v = i < p.b.batch ? seq_units(p, i, false) : 0;
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
// A piece of 16 or 8 bytes global -> shared, or zeros (from an address that is read nothing of).
template <uint32_t PIECE>
__device__ __forceinline__ void copy_piece(uint32_t dst, const void* src) {
    if constexpr (PIECE == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
template <uint32_t PIECE>
__device__ __forceinline__ void fill_piece(uint32_t dst, const void* src, const void* safe, bool take) {
    const void* from = take ? src : safe;
    const uint32_t bytes = take ? PIECE : 0u;
    if constexpr (PIECE == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(from), "r"(bytes) : "memory");
}

// ----------------------------------------------------------------- kernel --
template <bool F16, uint32_t DP>
__global__ void __launch_bounds__(kThreads, Cfg<DP>::kCtasPerSm) kv_attn_kernel(const AttnArgs p) {
    using C = Cfg<DP>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t sh[2 * kWarps];
    __shared__ float sh_m[kWarps][kRows], sh_l[kWarps][kRows];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const uint64_t total = count_units(p, sh), ctas = active_ctas(total, p.ctas);
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
    find_unit(p, u, sh, b, base);

    const uint32_t ring = smem_u32(smem) + warp * C::kStages * C::kStageBytes;
    float* const merge = reinterpret_cast<float*>(smem + warp * C::kStages * C::kStageBytes);
    const uint32_t D = p.c.head_dim;
    const uint32_t ts = static_cast<uint32_t>(p.c.token_stride);   // below 2^22: a page's tokens within 32 bits
    uint32_t k_dim[C::kKChunks], v_dim[C::kVPieces];
#pragma unroll
    for (uint32_t i = 0; i < C::kKChunks; ++i) k_dim[i] = min(i * 64 + c * 16, D - 16);
#pragma unroll
    for (uint32_t i = 0; i < C::kVPieces; ++i) v_dim[i] = min(g * C::kVPiece + i * 8 * C::kVPiece, D - C::kVPiece);
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
        const uint32_t item = static_cast<uint32_t>(in_seq / it.units);
        const uint32_t unit0 = static_cast<uint32_t>(in_seq % it.units);
        const uint32_t nunits = static_cast<uint32_t>(min(static_cast<uint64_t>(it.units - unit0), u_end - u));
        const uint32_t h = item / it.tiles, row0 = (item % it.tiles) * kRows;
        const uint32_t nrows = static_cast<uint32_t>(seq.count) * p.group;

        // ---- the query tile: rows g and g + 8 of it, FP16, each times 2^(7 - exponent of its maximum)
        uint32_t qf[C::kKChunks][4][4];
        float row_scale[2];
        int row_end[2];   // keys that the row sees
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t row = row0 + g + 8 * r;
            const bool real = row < nrows;
            const uint32_t t = real ? row / p.group : 0, head = h * p.group + (real ? row % p.group : 0);
            row_end[r] = real ? seq.len - seq.count + static_cast<int>(t) + 1 : 0x7FFFFFFF;
            const uint16_t* src = static_cast<const uint16_t*>(p.q.ptr) +
                                  static_cast<int64_t>(seq.first + static_cast<int>(t)) * p.q.token_stride +
                                  static_cast<int64_t>(head) * p.q.head_stride;
            uint32_t raw[C::kKChunks][8];
            float mx = 0.f;
            bool finite = true;
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
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 x = unpack2<F16>(raw[i][k]);
                    finite = finite && fabsf(x.x) <= 3.4028235e38f && fabsf(x.y) <= 3.4028235e38f;
                    mx = fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y)));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
            int bad = !finite;
            bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 1);
            bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, 2);
            const RowScale rs = row_scale_of(mx, bad, p.scale_log2);
            // kept above 0, so that a masked score (-inf) stays one: below 2^-66 all logits are 0 anyway
            row_scale[r] = bad ? rs.scale : fmaxf(rs.scale, kMinRowScale);
#pragma unroll
            for (uint32_t i = 0; i < C::kKChunks; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    float2 x = unpack2<F16>(raw[i][k]);
                    if (bad) x = make_float2(0.f, 0.f);   // the row's scale is NaN
                    qf[i][k >> 1][(k & 1) * 2 + r] = pack2<true>(x.x * rs.f1 * rs.f2, x.y * rs.f1 * rs.f2);
                }
        }
        int tile_end, tile_min;   // keys any row, and every row, of the tile sees
        {
            const uint32_t last = min(row0 + kRows, nrows) - 1;
            tile_end = seq.len - seq.count + static_cast<int>(last / p.group) + 1;
            tile_min = seq.len - seq.count + static_cast<int>(row0 / p.group) + 1;
        }

        // ---- this warp's steps: 16 keys of each unit
        const int key0 = static_cast<int>(unit0 * kUnitKeys + warp * kStepKeys);
        // Lane l holds what step l (mod 32) of a batch of 32 needs; a batch is asked for 32 - kStages + 1
        // steps before its first use, and its scales are first touched there.
        int meta_page = -1;
        float meta_k = 1.f, meta_v = 1.f, cur_k = 1.f, cur_lv = 0.f, cur_iv = 1.f;
        const auto load_meta = [&](uint32_t step) {
            const int key = key0 + static_cast<int>((step + lane) * kUnitKeys);
            meta_page = -1;
            meta_k = meta_v = 1.f;
            if (step + lane < nunits && key < tile_end) {
                const int page = p.b.page_table[static_cast<int64_t>(b) * p.b.page_table_stride + (key >> p.page_shift)];
                if (static_cast<uint32_t>(page) >= p.c.num_pages) {
                    record_failure(&g_kv_attn_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(page));
                } else {
                    const int64_t at = static_cast<int64_t>(page) * p.c.scale_page_stride + static_cast<int64_t>(h) * p.c.scale_head_stride;
                    meta_page = page;
                    meta_k = p.c.k_scale[at];
                    meta_v = p.c.v_scale[at];
                }
            }
        };
        // Chunks past the head repeat its last one (their queries are zero, their outputs are not stored).
        const uint8_t* const k_head = static_cast<const uint8_t*>(p.c.k_codes) + static_cast<int64_t>(h) * p.c.head_stride;
        const uint8_t* const v_head = static_cast<const uint8_t*>(p.c.v_codes) + static_cast<int64_t>(h) * p.c.head_stride;
        const auto issue = [&](uint32_t step) {
            if (step < nunits) {
                if ((step & 31u) == 0u) load_meta(step);
                const int page = __shfl_sync(0xFFFFFFFFu, meta_page, step & 31u);
                const int key = key0 + static_cast<int>(step * kUnitKeys);
                const uint32_t slot = ring + (step % C::kStages) * C::kStageBytes + lane * 16, vslot = ring + (step % C::kStages) * C::kStageBytes + kStepKeys * DP + lane * C::kVPiece;
                const int64_t off = static_cast<int64_t>(page) * p.c.page_stride +
                                    static_cast<uint32_t>(key & static_cast<int>(p.c.page_size - 1)) * ts;
                const uint8_t *kp = k_head + off, *vp = v_head + off;
                if (page >= 0 && tile_end - key >= static_cast<int>(kStepKeys)) {
#pragma unroll
                    for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
                        for (uint32_t i = 0; i < C::kKChunks; ++i)
                            copy_piece<16>(slot + (j * C::kKChunks + i) * 512, kp + ((8 * j + g) * ts + k_dim[i]));
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                        for (uint32_t i = 0; i < C::kVPieces; ++i)
                            copy_piece<C::kVPiece>(vslot + (j * C::kVPieces + i) * 32 * C::kVPiece,
                                                   vp + ((8 * (j >> 1) + 2 * c + (j & 1)) * ts + v_dim[i]));
                } else {
                    const int left = page < 0 ? 0 : tile_end - key;   // keys of the step that exist; the others are zero filled
#pragma unroll 1
                    for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
                        for (uint32_t i = 0; i < C::kKChunks; ++i)
                            fill_piece<16>(slot + (j * C::kKChunks + i) * 512, kp + ((8 * j + g) * ts + k_dim[i]), p.c.k_codes,
                                           static_cast<int>(8 * j + g) < left);
#pragma unroll 1
                    for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                        for (uint32_t i = 0; i < C::kVPieces; ++i)
                            fill_piece<C::kVPiece>(vslot + (j * C::kVPieces + i) * 32 * C::kVPiece,
                                                   vp + ((8 * (j >> 1) + 2 * c + (j & 1)) * ts + v_dim[i]), p.c.v_codes,
                                                   static_cast<int>(8 * (j >> 1) + 2 * c + (j & 1)) < left);
                }
            }
            cp_async_commit();
        };

        float o[DP / 8][4];
#pragma unroll
        for (uint32_t n = 0; n < DP / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

#pragma unroll
        for (uint32_t s = 0; s < C::kStages - 1; ++s) issue(s);
        for (uint32_t step = 0; step < nunits; ++step) {
            cp_async_wait_group<C::kStages - 2>();
            if ((step & 31u) == 0u) {   // the batch of 32 that the copies have reached
                cur_k = meta_k < kMinScale ? kMinScale : meta_k;
                const float v = meta_v < kMinScale ? kMinScale : meta_v;
                cur_lv = __log2f(v);
                cur_iv = __frcp_rn(v);
            }
            issue(step + C::kStages - 1);
            const int key = key0 + static_cast<int>(step * kUnitKeys);
            if (key >= tile_end) continue;
            const float ks = __shfl_sync(0xFFFFFFFFu, cur_k, step & 31u), lv = __shfl_sync(0xFFFFFFFFu, cur_lv, step & 31u),
                        iv = __shfl_sync(0xFFFFFFFFu, cur_iv, step & 31u);
            const uint8_t* slot = smem + warp * C::kStages * C::kStageBytes + (step % C::kStages) * C::kStageBytes;

            // ---- scores
            float s[2][4];
#pragma unroll
            for (uint32_t j = 0; j < 2; ++j) {
                s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
                for (uint32_t i = 0; i < C::kKChunks; ++i) {
                    const uint4 w = *reinterpret_cast<const uint4*>(slot + ((j * C::kKChunks + i) * 32 + lane) * 16);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16x4(ww[k], b0, b1);
                        mma_f16(s[j], qf[i][k], b0, b1);
                    }
                }
            }
            // ---- weights
            const bool edge = key + static_cast<int>(kStepKeys) > tile_min;
            uint32_t pf[4];
            float f[2], mx[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                f[r] = ks * row_scale[r];
                if (edge) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (key + 8 * j + 2 * static_cast<int>(c) + e >= row_end[r]) s[j][2 * r + e] = -INFINITY;
                }
                // f > 0: the largest score gives the largest y = score f + log2(vs)
                mx[r] = fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1]));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 1));
                mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], 2));
                mx[r] = fmaf(mx[r], f[r], lv);
            }
            if (__any_sync(0xFFFFFFFFu, mx[0] > m[0] + kRise || mx[1] > m[1] + kRise)) {
                // a running maximum is exceeded by more than 2^8: it moves, sums and outputs are rescaled
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float m_new = fmaxf(m[r], mx[r]);
                    const float a = m[r] == -INFINITY ? 0.f : ex2(m[r] - m_new);
                    l[r] *= a;
#pragma unroll
                    for (uint32_t n = 0; n < DP / 8; ++n) {
                        o[n][2 * r] *= a;
                        o[n][2 * r + 1] *= a;
                    }
                    m[r] = m_new;
                }
            }
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const float t = m[r] == -INFINITY ? 0.f : lv - m[r] + kPBits;
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = ex2(fmaf(s[e >> 1][2 * r + (e & 1)], f[r], t));
                l[r] = fmaf((y[0] + y[1]) + (y[2] + y[3]), iv, l[r]);
                pf[r] = pack2<true>(y[0], y[1]);
                pf[2 + r] = pack2<true>(y[2], y[3]);
            }
            // ---- outputs
            const uint8_t* vslot = slot + kStepKeys * DP;
            uint32_t vw[4][C::kVBytes / 4];
#pragma unroll
            for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                for (uint32_t i = 0; i < C::kVPieces; ++i) {
                    const uint8_t* at = vslot + ((j * C::kVPieces + i) * 32 + lane) * C::kVPiece;
                    if constexpr (C::kVPiece == 16) {
                        const uint4 w = *reinterpret_cast<const uint4*>(at);
                        vw[j][4 * i] = w.x, vw[j][4 * i + 1] = w.y, vw[j][4 * i + 2] = w.z, vw[j][4 * i + 3] = w.w;
                    } else {
                        const uint2 w = *reinterpret_cast<const uint2*>(at);
                        vw[j][0] = w.x, vw[j][1] = w.y;
                    }
                }
            if (edge && seq.count > 1) {
                // keys that some rows do not see: a NaN value there must not reach them through 0 * NaN.
                // The NaN codes leave the product, and a product of indicators (row sees key, value is
                // NaN) marks the outputs that are NaN.
                uint32_t any = 0;
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j)
#pragma unroll
                    for (uint32_t i = 0; i < C::kVBytes / 4; ++i) any |= e4m3_nan_flags(vw[j][i]);
                if (__any_sync(0xFFFFFFFFu, any != 0u)) {
                    uint32_t seen[4];
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const int k0 = key + 8 * j + 2 * static_cast<int>(c);
                            seen[2 * j + r] = pack2<true>(k0 < row_end[r] ? 1.f : 0.f, k0 + 1 < row_end[r] ? 1.f : 0.f);
                        }
#pragma unroll
                    for (uint32_t i = 0; i < C::kVBytes / 4; ++i) {
                        uint32_t ind[4];
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j) {
                            const uint32_t full = (e4m3_nan_flags(vw[j][i]) >> 7) * 0xFFu;   // 0xFF where NaN
                            ind[j] = full & 0x38383838u;                                     // E4M3 1.0
                            vw[j][i] &= ~full;
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t sel = half ? 0x7362u : 0x5140u;
                            uint32_t a0, a1, c0, c1;
                            e4m3x4_to_f16x4(prmt(ind[0], ind[1], sel), a0, a1);
                            e4m3x4_to_f16x4(prmt(ind[2], ind[3], sel), c0, c1);
                            float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(t0, seen, a0, c0);
                            mma_f16(t1, seen, a1, c1);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if (t0[e] > 0.f) o[4 * i + 2 * half][e] = __uint_as_float(0x7FC00000u);
                                if (t1[e] > 0.f) o[4 * i + 2 * half + 1][e] = __uint_as_float(0x7FC00000u);
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
                    uint32_t a0, a1, c0, c1;
                    e4m3x4_to_f16x4(prmt(vw[0][i], vw[1][i], sel), a0, a1);
                    e4m3x4_to_f16x4(prmt(vw[2][i], vw[3][i], sel), c0, c1);
                    mma_f16(o[4 * i + 2 * half], pf, a0, c0);
                    mma_f16(o[4 * i + 2 * half + 1], pf, a1, c1);
                }
        }
        cp_async_wait_group<0>();

        // ---- join the warps' parts. Output column n of tile 4 i + e holds dim
        // n * kVPiece + (4 i + e) % kVPiece of piece (4 i + e) / kVPiece (8 kVPiece dims each).
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
            l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
            if (c == 0) {
                sh_m[warp][g + 8 * r] = m[r];
                sh_l[warp][g + 8 * r] = l[r];
            }
        }
        __syncwarp();   // every lane is done with its ring slots, which `merge` reuses
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (uint32_t i = 0; i < C::kVPieces; ++i)
#pragma unroll
                    for (uint32_t k = 0; k < C::kVPiece; k += 4)
                        *reinterpret_cast<float4*>(merge + (g + 8 * r) * DP + i * 8 * C::kVPiece + (2 * c + e) * C::kVPiece + k) =
                            make_float4(o[i * C::kVPiece + k][2 * r + e], o[i * C::kVPiece + k + 1][2 * r + e],
                                        o[i * C::kVPiece + k + 2][2 * r + e], o[i * C::kVPiece + k + 3][2 * r + e]);
        __syncthreads();
        const bool whole = nunits == it.units;
        if (first_part && threadIdx.x == 0) write_boundary(p.ws, u, u - unit0, it.units, seq, h, item % it.tiles, total, ctas);
        float* slot_ws = slots + (static_cast<uint64_t>(blockIdx.x) * 2 + (first_part ? 0 : 1)) * slot_floats(DP);
        for (uint32_t i = threadIdx.x; i < kRows * DP / 4; i += kThreads) {
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
                    slot_ws[kRows * DP + r] = mm;
                    slot_ws[kRows * DP + kRows + r] = ll;
                }
            }
        }
        __syncthreads();   // the rings and sh_* are free again
        first_part = false;
        u += nunits;
    }
}

// Joins the parts of split items in key order: a block per boundary between CTAs' ranges and
// kWarps rows, a warp a row, the parts' loads in flight together.
template <bool F16, uint32_t DP>
__global__ void __launch_bounds__(kThreads) kv_attn_join_kernel(const AttnArgs p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t c = blockIdx.x + 1, lane = threadIdx.x & 31, r = blockIdx.y * kWarps + (threadIdx.x >> 5);
    const Boundary b = reinterpret_cast<const Boundary*>(p.ws)[c];
    const uint32_t row = b.tile * kRows + r;
    if (b.parts == 0 || row >= static_cast<uint32_t>(b.count) * p.group) return;
    const float* const slots = p.ws + boundary_floats(p.ctas);
    const auto slot = [&](uint32_t i) { return slots + static_cast<uint64_t>(i == 0 ? b.slot : 2 * (c + i - 1)) * slot_floats(DP); };
    float m = -INFINITY;
    for (uint32_t i = lane; i < b.parts; i += 32) m = fmaxf(m, slot(i)[kRows * DP + r]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    constexpr uint32_t V = DP / 32;   // consecutive dims of a lane
    float acc[V] = {}, l = 0.f;
#pragma unroll 8
    for (uint32_t i = 0; i < b.parts; ++i) {
        const float* s = slot(i);
        const float mi = s[kRows * DP + r];
        const float a = mi == -INFINITY ? 0.f : ex2(mi - m);
        l = fmaf(a, s[kRows * DP + kRows + r], l);
        float x[V];
        if constexpr (V == 2) {
            const float2 t = *reinterpret_cast<const float2*>(s + r * DP + 2 * lane);
            x[0] = t.x, x[1] = t.y;
        } else {
#pragma unroll
            for (uint32_t k = 0; k < V; k += 4) {
                const float4 t = *reinterpret_cast<const float4*>(s + r * DP + V * lane + k);
                x[k] = t.x, x[k + 1] = t.y, x[k + 2] = t.z, x[k + 3] = t.w;
            }
        }
#pragma unroll
        for (uint32_t k = 0; k < V; ++k) acc[k] = fmaf(a, x[k], acc[k]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(b.first + static_cast<int>(row / p.group)) * p.out.token_stride +
                    static_cast<int64_t>(b.h * p.group + row % p.group) * p.out.head_stride;
#pragma unroll
    for (uint32_t k = 0; k < V; k += 2)
        if (V * lane + k < p.c.head_dim) *reinterpret_cast<uint32_t*>(dst + V * lane + k) = pack2<F16>(acc[k] * inv, acc[k + 1] * inv);
}

template <bool F16, uint32_t DP>
cudaError_t launch(const AttnArgs& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kv_attn_kernel<F16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP>::kSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(p.ctas, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = Cfg<DP>::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kv_attn_kernel<F16, DP>, p);
    if (e != cudaSuccess) return e;
    if (p.ctas < 2) return cudaSuccess;
    const uint64_t rows = static_cast<uint64_t>(p.b.max_q) * p.group;   // of an item, at most
    cfg.gridDim = dim3(p.ctas - 1, (static_cast<uint32_t>(rows < kRows ? rows : kRows) + kWarps - 1) / kWarps, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_attn_join_kernel<F16, DP>, p);
}

uint32_t padded_dim(uint32_t d) { return d <= 64 ? 64u : d <= 128 ? 128u : 256u; }
uint32_t grid_ctas(uint32_t dp, int sms) { return static_cast<uint32_t>(sms) * (dp == 256 ? Cfg<256>::kCtasPerSm : Cfg<128>::kCtasPerSm); }

}  // namespace

uint64_t kv_attn_ws_bytes(uint32_t head_dim, uint32_t rows_per_head, int sms) {
    if (kv_attn_tc_applies(head_dim, rows_per_head)) return kv_attn_tc_ws_bytes(head_dim, sms);
    const uint32_t dp = padded_dim(head_dim);
    return 4 * boundary_floats(grid_ctas(dp, sms)) + 8ull * grid_ctas(dp, sms) * slot_floats(dp);
}

int launch_kv_attn(const w8a16_kv_cache_t& c, const w8a16_kv_batch_t& b, uint32_t act_dtype, const w8a16_heads_t& q,
                   const w8a16_heads_t& out, float softmax_scale, void* ws, int sms,
                   uint64_t timeout_ns, cudaStream_t s, std::string* err) {
    AttnArgs p{c, b, q, out, static_cast<float*>(ws), softmax_scale * 1.4426950408889634f, q.heads / c.kv_heads, 0, 0, timeout_ns};
    while ((1u << p.page_shift) < c.page_size) ++p.page_shift;
    const uint32_t dp = padded_dim(c.head_dim);
    p.ctas = grid_ctas(dp, sms);
    const bool f16 = act_dtype == W8A16_ACT_F16;
    const cudaError_t e = kv_attn_tc_applies(c.head_dim, b.max_q * p.group) ? launch_kv_attn_tc(p, f16, sms, s)
                          : dp == 64    ? (f16 ? launch<true, 64>(p, s) : launch<false, 64>(p, s))
                          : dp == 128 ? (f16 ? launch<true, 128>(p, s) : launch<false, 128>(p, s))
                                      : (f16 ? launch<true, 256>(p, s) : launch<false, 256>(p, s));
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

// Attention over the 8-bit paged cache for many query rows per key/value head (prompt
// chunks): the mathematics of w8a16_kv_attn_few.cuh on the 5th-generation tensor cores.
//
// Work. An item is 256 query rows (two tiles of 128; the G query heads of a key/value head
// times the call's tokens) of one sequence and head, a unit 128 keys of it, with the
// keys that no row of the item sees left out. The units of the whole call are split
// over one CTA per SM in equal contiguous ranges; split items are joined through the
// workspace by a second launch, in a fixed order.
//
// Bound by: the hand-over between the softmax warps and the products. 1024 tokens on 8192 (32 query heads of
// 128 on 8): 141 us, 0.91 PFLOP/s, 49 % of a library product's rate; the tensor pipe is busy for
// 41 % of the kernel's 138 us: each tile's scores, weights and
// outputs follow one another, and two tiles do not fill the gaps that a third, for
// which TMEM has no room, would (a tile's next scores come 1100 cycles after its last weights, of some 4600 a unit).
//
// An item's begin and end cost some two units each: its query rows come by asynchronous copies under the last unit of the
// item before (loaded and scaled a row a thread from memory, 10000 to 20000 cycles), and outputs are turned in shared
// memory, so that neighbouring lanes write one row (a row a thread: 7000 cycles an item, 3000 now).
//
// Windows and prefixes (SpanMode): as in w8a16_kv_attn_few.cuh, the keys of an item's rows come in groups of 16 without those between
// sinks and window. A chunk of 2048 tokens, window 1024 (32 heads on 8): 68 us, 0.51 PFLOP/s, 27 %, of which an item's begin and
// end are half: its keys are 9 units. The prefix pass of 64 sequences on 16384 takes 88 of the 152 SMs, and 48 us with the sequences' own
// keys (48 MB) beside it and the join: its units (256 rows, 128 keys) as long as a chunk's, its start 8 us.
//
// A CTA. Warp 13 looks the units' pages and scales up, four units at a time, into a ring.
// Warps 8-11 read a unit's E4M3 codes into registers a unit ahead, convert them to
// FP16 (exact) and write the K and V tiles, [128 keys][DP] in 128-byte swizzled rows, two
// stages each; the same layout serves K as a K-major operand and V, whose contraction
// runs along its rows, as an MN-major one. One thread of warp 12 issues the products, S = Q K^T
// (M = 128 rows, N = 64 keys) and O += P V with P read from TMEM. Warps 0-3 and 4-7 own a
// row tile each, a thread a row, so no reduction crosses threads. A unit's softmax goes in
// two blocks of 64 keys, and O's products of the first run under the softmax of the second.
// (S in N = 64 products, with a buffer each, would let a tile's softmax run on without a
// pause, but they take 80 cycles for the 64 that N = 128 takes for twice the columns: the
// A operand is read from shared memory again, and that is what these products wait for.)
// A thread reads its 64 scores from TMEM, and only where their maximum exceeds the row's
// running one by more than 8 is that moved and O rescaled; P (at most 2^15, FP16) overwrites
// the first columns of S.
//
// TMEM: S of tile t at columns 128 t, P of its blocks at 128 t and 128 t + 64, O at 256 + DP t.
#include <cuda_runtime.h>

#include <cstring>
#include <string>

#include "w8a16_cluster.cuh"
#include "w8a16_kv_attn.cuh"

namespace w8a16 {
namespace {

__device__ DeviceStatus g_kv_attn_tc_status;

constexpr uint32_t kTile = 128;                // rows of a tile, and keys of a unit
constexpr uint32_t kItemRows = 2 * kTile;
constexpr uint32_t kSoftmaxWarps = 8, kConvWarps = 4;
constexpr uint32_t kIssueWarp = kSoftmaxWarps + kConvWarps, kLookWarp = kIssueWarp + 1;
constexpr uint32_t kThreads = 32 * (kLookWarp + 1);
constexpr uint32_t kWarpsAll = kThreads / 32;
constexpr uint32_t kBlockKeys = 64;            // keys of a P
constexpr uint32_t kStages = 2;
constexpr uint32_t kRing = 8, kLook = 4;        // units whose pages and scales are held, and looked up at a time
constexpr float kPBits = 7.f, kRise = 8.f;     // P = 2^(y - m + 7); m moves when exceeded by 8
constexpr uint32_t kChunk = 256;               // sequences whose unit counts are held at a time
constexpr uint32_t kNanWords = 64;             // of the map of those groups of 16 keys in whose values clean_tile found a NaN
// The bit there of group i of a CTA with `units` units, eight groups each: one a group, where there are bits enough.
__device__ __forceinline__ uint32_t nan_bit(uint32_t i, uint32_t units) { return i / (8 * units / (32 * kNanWords) + 1); }

constexpr uint32_t kTurnBytes = 32 * 64;        // 64 bytes of a warp's 32 rows

template <uint32_t DP>
struct Cfg {
    static constexpr uint32_t kTileBytes = kTile * DP * 2;          // an FP16 tile
    static constexpr uint32_t kHalfBytes = kTile * 128;             // a 64-column block of a tile
    static constexpr uint32_t kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes;
    static constexpr uint32_t kTail = kV + kStages * kTileBytes;    // barriers, scales
    static constexpr uint32_t kTurn = kTail + 2048;                 // the softmax warps' transposes of outputs
    static constexpr uint32_t kSmem = 1024 + kTurn + kSoftmaxWarps * kTurnBytes;
};
struct Look {   // a unit, by its 8 groups of 16 keys
    int64_t offset[8];                 // of the group's codes
    float ks[8], lv[8], iv[8];         // K scale, log2 and reciprocal of the V scale
    int last;                          // row of the last key there is
    int edge;                          // some rows do not see all keys
};
struct Tail {
    uint64_t qfull[2], kfull[kStages], kempty[kStages], vfull[kStages], vempty[kStages], sfull[2], pfull[2][2], odone[2][2], drain;
    uint64_t lfull[kRing], lempty[kRing];
    uint32_t tmem;
    int abort_flag;
    int nan_seen;
    uint32_t nan_groups[kNanWords];
    Look look[kRing];
};
static_assert(sizeof(Tail) <= 2048, "barrier block");

enum Wait : unsigned { kWaitQ = 1, kWaitK, kWaitV, kWaitKFree, kWaitVFree, kWaitS, kWaitP, kWaitO, kWaitDrain, kWaitLook, kWaitLookFree };

// ------------------------------------------------------------ the schedule --
// Keys that the last row of row block rb sees, and the units of its item.
__device__ __forceinline__ int block_end(const Seq& s, uint32_t group, uint32_t rb) {
    const uint32_t rows = static_cast<uint32_t>(s.count) * group;
    return s.len - s.count + static_cast<int>((min((rb + 1) * kItemRows, rows) - 1) / group) + 1;
}
// Keys that its first row sees.
__device__ __forceinline__ int edge_key(const Seq& s, uint32_t group, uint32_t rb) {
    return s.len - s.count + static_cast<int>(rb * kItemRows / group) + 1;
}
// But for kFull: its groups of 16 keys.
template <SpanMode MODE>
__device__ __forceinline__ Groups block_groups(const AttnArgs& p, const Seq& s, uint32_t rb) {
    return groups_of<MODE>(p, edge_key(s, p.group, rb), MODE == kPrefix ? p.span.lower : block_end(s, p.group, rb));
}
template <SpanMode MODE>
__device__ __forceinline__ uint32_t block_units(const AttnArgs& p, const Seq& s, uint32_t rb) {
    if constexpr (MODE != kFull) return max(1, (block_groups<MODE>(p, s, rb).count + 7) / 8);
    return max(1, (block_end(s, p.group, rb) + static_cast<int>(kTile) - 1) / static_cast<int>(kTile));
}
__device__ __forceinline__ uint32_t seq_blocks(const Seq& s, uint32_t group) {
    return s.len <= 0 ? 0u : (static_cast<uint32_t>(s.count) * group + kItemRows - 1) / kItemRows;
}

// Windows and suffix passes: items of much the same length go whole to the CTAs, some more to one than to another, rather than
// split where the units divide evenly: a split costs the join's launch, and an item's part that is read and written again, some
// kSplitCost units' time. (us, whole and split, 32 query heads on 8: a chunk of 2048 tokens, window 1024, 68 and 74, window 200 39 and
// 47; a chunk of 1024, window 1024, 38 and 50; 2 sequences of 500 tokens on 3000 shared 102 and 131.)
constexpr uint32_t kSplitCost = 7;
// What decides it: the row blocks of the sequences, and the most units of one.
struct Blocks {
    uint32_t of[kChunk], most;
};

// Units per key/value head of up to kChunk sequences from b0, a warp per sequence.
template <uint32_t WARPS, SpanMode MODE>
__device__ __forceinline__ uint32_t chunk_units(const AttnArgs& p, uint32_t b0, uint64_t* sh, bool report, Blocks* blocks = nullptr) {
    const uint32_t count = min(kChunk, p.b.batch - b0);
    for (uint32_t i = threadIdx.x >> 5; i < count; i += WARPS) {
        const Seq s = attn_sequence<MODE>(p, b0 + i);
        if (s.bad && report && (threadIdx.x & 31) == 0) record_failure(&g_kv_attn_tc_status, W8A16_STATUS_BAD_INDEX, b0 + i);
        const uint32_t nb = seq_blocks(s, p.group);
        uint64_t n = 0;
        uint32_t most = 0;
        for (uint32_t rb = threadIdx.x & 31; rb < nb; rb += 32) {
            const uint32_t units = block_units<MODE>(p, s, rb);
            n += units, most = max(most, units);
        }
        n = warp_sum(n);
        if ((threadIdx.x & 31) == 0) sh[i] = n;
        if constexpr (MODE == kWindow || MODE == kSuffix) {
            if (blocks != nullptr) {
                most = __reduce_max_sync(0xFFFFFFFFu, most);
                if ((threadIdx.x & 31) == 0) blocks->of[i] = nb, atomicMax(&blocks->most, most);
            }
        }
    }
    __syncthreads();
    return count;
}

// An item of the schedule: its sequence, head, row block, first unit (in the whole call's
// order) and unit count.
struct Item {
    uint64_t first;
    Seq s;
    uint32_t b, h, rb, n;
};
template <SpanMode MODE>
__device__ __forceinline__ void next_item(const AttnArgs& p, Item& it) {
    it.first += it.n;
    if constexpr (MODE == kPrefix) {
        if (++it.rb == p.span.pass.tiles) it.rb = 0, ++it.h;
        return;
    }
    if (++it.rb == seq_blocks(it.s, p.group)) {
        it.rb = 0;
        if (++it.h == p.c.kv_heads) {
            it.h = 0;
            do it.s = attn_sequence<MODE>(p, ++it.b);
            while (seq_blocks(it.s, p.group) == 0);   // asked for only where units are left
        }
    }
    it.n = block_units<MODE>(p, it.s, it.rb);
}
// Leaves the counts of the first kChunk sequences in sh.
template <uint32_t WARPS, SpanMode MODE>
__device__ __noinline__ uint64_t total_units(const AttnArgs& p, uint64_t* sh, bool report, Blocks* blocks) {
    uint64_t n = 0;
    for (uint32_t b0 = (p.b.batch - 1) / kChunk * kChunk;; b0 -= kChunk) {
        const uint32_t count = chunk_units<WARPS, MODE>(p, b0, sh, report, blocks);
        uint64_t x = 0;   // a warp's lanes share the sum
        for (uint32_t i = threadIdx.x & 31; i < count; i += 32) x += sh[i];
        n += warp_sum(x);
        if (b0 == 0) break;
        __syncthreads();
    }
    return n * p.c.kv_heads;
}
// kPrefix: all items are alike.
__device__ __forceinline__ Item prefix_item(const AttnArgs& p, uint64_t u) {
    const PrefixPass& s = p.span.pass;
    const uint32_t i = static_cast<uint32_t>(divide(u, s.units));
    return {static_cast<uint64_t>(i) * s.units, attn_sequence<kPrefix>(p, 0), 0, i / s.tiles, i % s.tiles, s.units};
}
// The item that holds unit u (below the total); sh as total_units left it. whole: the u-th item; sh counts items.
template <uint32_t WARPS, SpanMode MODE>
__device__ __noinline__ Item find_item(const AttnArgs& p, uint64_t u, uint64_t* sh, bool whole) {
    Item it{};
    uint64_t base = 0;
    for (uint32_t b0 = 0; b0 < p.b.batch; b0 += kChunk) {
        if (b0) {
            __syncthreads();
            chunk_units<WARPS, MODE>(p, b0, sh, false);
        }
        const uint32_t count = min(kChunk, p.b.batch - b0);
        for (uint32_t i = 0; i < count; ++i) {
            const uint64_t n = sh[i] * p.c.kv_heads;
            if (u < base + n) {
                it.s = attn_sequence<MODE>(p, b0 + i);
                it.b = b0 + i;
                it.h = static_cast<uint32_t>(divide(u - base, sh[i]));
                uint64_t rest = u - base - it.h * sh[i];
                const uint32_t lane = threadIdx.x & 31, nb = seq_blocks(it.s, p.group);
                for (uint32_t r0 = 0;; r0 += 32) {   // the row block that holds it, 32 at a time
                    const uint32_t mine = r0 + lane < nb ? (whole ? 1u : block_units<MODE>(p, it.s, r0 + lane)) : 0u;
                    uint64_t inc = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint64_t x = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                        if (lane >= static_cast<uint32_t>(o)) inc += x;
                    }
                    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, rest < inc);
                    if (hit) {
                        const int at = __ffs(hit) - 1;
                        it.rb = r0 + at;
                        it.n = __shfl_sync(0xFFFFFFFFu, mine, at);
                        it.first = u - (rest - (__shfl_sync(0xFFFFFFFFu, inc, at) - it.n));
                        if (whole) it.n = block_units<MODE>(p, it.s, it.rb);
                        return it;
                    }
                    rest -= __shfl_sync(0xFFFFFFFFu, inc, 31);
                }
            }
            base += n;
        }
    }
    return it;
}

// ------------------------------------------------------------- primitives --
// FP16 operands, FP32 sums; B_MN: B is MN-major (its contraction runs along smem rows).
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t m, uint32_t n, bool b_mn) {
    return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// MN-major operand of 128-byte swizzled rows: 8-row groups (along the contraction) 1024
// bytes apart, 64-element column blocks kHalfBytes apart.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t block_bytes) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(block_bytes >> 4) << 16;     // leading byte offset: next 64 columns
    d |= static_cast<uint64_t>(1024 >> 4) << 32;            // stride byte offset: next 8 rows
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// 8 columns of a warp's lanes, times f.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&v)[8], float f) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "f"(v[0] * f),
                 "f"(v[1] * f), "f"(v[2] * f), "f"(v[3] * f), "f"(v[4] * f), "f"(v[5] * f), "f"(v[6] * f), "f"(v[7] * f)
                 : "memory");
}

// A wait that gives up `timeout_ns` after it began, and tells the warp as one. (What is
// rarely run is kept out of line: the loops' code has to stay in the instruction cache.)
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag, unsigned what) {
    return mbar_wait_for(bar, parity, timeout_ns, abort_flag, &g_kv_attn_tc_status, what);
}
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag, unsigned what) {
    if (mbar_try_wait(bar, parity)) return true;
    return wait_slow(bar, parity, timeout_ns, abort_flag, what);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint64_t timeout_ns, volatile int* abort_flag, unsigned what) {
    return __all_sync(0xFFFFFFFFu, wait_one(bar, parity, timeout_ns, abort_flag, what));
}

// 16 codes -> 32 bytes of FP16.
__device__ __forceinline__ void convert16(const uint4& q, uint4& lo, uint4& hi) {
    e4m3x4_to_f16x4(q.x, lo.x, lo.y);
    e4m3x4_to_f16x4(q.y, lo.z, lo.w);
    e4m3x4_to_f16x4(q.z, hi.x, hi.y);
    e4m3x4_to_f16x4(q.w, hi.z, hi.w);
}
// NaN values (FP16) that this lane has stored to a V tile: 0 for the products, marked in the
// outputs at the end (mark_nan). For units where some rows do not see all keys: there 0 * NaN
// would reach them. But for kFull, whose marking reads all such keys again, the groups that held one are noted: `group` is
// that of the warp's first keys, of a CTA with `units` units.
template <bool NOTED>
__device__ __noinline__ void clean_tile(uint8_t* even, uint8_t* odd, uint32_t chunks, uint32_t halves, uint32_t half_bytes, Tail* tl, uint32_t group = 0,
                                        uint32_t units = 0) {
    for (uint32_t i = 0; i < 2 * chunks; ++i) {
        uint16_t* at = reinterpret_cast<uint16_t*>((i & 1 ? odd : even) + i / 2 % halves * half_bytes + i / 2 / halves * 1024);
        for (int e = 0; e < 8; ++e)
            if ((at[e] & 0x7FFF) > 0x7C00) {
                at[e] = 0;
                if constexpr (NOTED) {
                    const uint32_t bit = nan_bit(group + i / 2 / halves / 2, units);   // (8 keys a step)
                    atomicOr(&tl->nan_groups[bit / 32], 1u << bit % 32);
                }
                *static_cast<volatile int*>(&tl->nan_seen) = 1;
            }
    }
}

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 32 scores of a row, columns `first` on: those of keys from `end` on are masked.
__device__ __forceinline__ void mask_scores(uint32_t (&v)[32], int first, int end) {
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (first + e >= end) v[e] = 0xFF800000u;
}
// The others: those that are not below `end`, and neither below `sinks` nor from `lo` on.
__device__ __forceinline__ void mask_span(uint32_t (&v)[32], int first, int end, int lo, int sinks) {
    const auto below = [&](int x) { return x <= first ? 0u : x >= first + 32 ? 0xFFFFFFFFu : (1u << (x - first)) - 1u; };
    const uint32_t seen = below(end) & (below(sinks) | ~below(lo));
#pragma unroll
    for (int e = 0; e < 32; ++e)
        if (!(seen >> e & 1u)) v[e] = 0xFF800000u;
}
// Their largest y = score f + log2(vs) (f = logit_factor > 0: that of the largest score);
// ks, lv (and iv): of the two groups of 16 keys.
__device__ __forceinline__ float score_max(const uint32_t (&v)[32], const float* ks, const float* lv, float rowf) {
    float y = -INFINITY;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; e += 2) mx = max3(mx, __uint_as_float(v[16 * g + e]), __uint_as_float(v[16 * g + e + 1]));
        y = fmaxf(y, fmaf(mx, logit_factor(ks[g], rowf), lv[g]));
    }
    return y;
}
// Their weights 2^(y - rc) as FP16 pairs; returns l + the sum of weight / vs.
__device__ __forceinline__ float score_weights(const uint32_t (&v)[32], const float* ks, const float* lv, const float* iv, float rowf,
                                               float rc, float l, uint32_t (&pk)[16]) {
    const uint64_t one = pack_f32x2(1.f, 1.f);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        const float f = logit_factor(ks[g], rowf), d = lv[g] - rc;
        const uint64_t ff = pack_f32x2(f, f), dd = pack_f32x2(d, d);
        uint64_t s2 = pack_f32x2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
            const float2 y = unpack_f32x2(fma_f32x2(pack_f32x2(__uint_as_float(v[16 * g + e]), __uint_as_float(v[16 * g + e + 1])), ff, dd));
            const float a = ex2(y.x), b = ex2(y.y);
            s2 = fma_f32x2(pack_f32x2(a, b), one, s2);
            pk[8 * g + e / 2] = pack2<true>(a, b);
        }
        const float2 s = unpack_f32x2(s2);
        l = fmaf(s.x + s.y, iv[g], l);
    }
    return l;
}

// NaN values of the keys [lo, hi), which the products at the causal edge left out, marked
// in the outputs (or this range's part of them) of a row that sees these keys.
__device__ __noinline__ void mark_nan(const AttnArgs& p, uint32_t b, uint32_t h, int lo, int hi, uint16_t* dst, float* part) {
    for (int key = lo; key < hi; ++key) {
        const int page = p.b.page_table[static_cast<int64_t>(b) * p.b.page_table_stride + (key >> p.page_shift)];
        if (page < 0 || page >= static_cast<int>(p.c.num_pages)) continue;
        const uint8_t* v = static_cast<const uint8_t*>(p.c.v_codes) + static_cast<int64_t>(page) * p.c.page_stride +
                           static_cast<int64_t>(h) * p.c.head_stride +
                           static_cast<int64_t>(key & static_cast<int>(p.c.page_size - 1)) * p.c.token_stride;
        for (uint32_t d = 0; d < p.c.head_dim; ++d)
            if ((v[d] & 0x7F) == 0x7F) {
                if (dst) dst[d] = 0x7FC0u;   // a NaN in BF16 and in FP16
                else part[d * kItemRows] = __uint_as_float(0x7FC00000u);
            }
    }
}

// But for kFull: the same of the keys of an item's units [j0, j0 + cnt) that a row sees whose keys end at row_end; marks lie `stride`
// floats apart. Only the groups that clean_tile found a NaN in are read again, 16 codes a load (the other warps wait meanwhile, and a
// prefix that some rows end in goes through clean_tile whole): `unit0` is the CTA's number of the first unit, of `units`.
template <SpanMode MODE>
__device__ __noinline__ void mark_nan_span(const AttnArgs& p, const Tail* tl, uint32_t unit0, uint32_t units, uint32_t b, uint32_t h, const Groups& span,
                                           uint32_t j0, uint32_t cnt, int row_end, uint16_t* dst, float* part, uint32_t stride) {
    const int lo = row_lo<MODE>(p, row_end);
    const auto found = [&](uint32_t bit) { return (static_cast<const volatile uint32_t*>(tl->nan_groups)[bit / 32] >> bit % 32 & 1u) != 0; };
    uint64_t marked[2] = {0, 0};   // dims, 64 each
    const uint32_t pieces = p.c.head_dim / 16;
    for (uint32_t v = 8 * j0; v < min(8 * (j0 + cnt), static_cast<uint32_t>(span.count)); ++v) {
        if (!found(nan_bit(8 * (unit0 - j0) + v, units))) continue;
        const int first = group_key(span, static_cast<int>(v));
        const int page = p.b.page_table[static_cast<int64_t>(b) * p.b.page_table_stride + (first >> p.page_shift)];
        if (page < 0 || page >= static_cast<int>(p.c.num_pages)) continue;
        const uint8_t* codes = static_cast<const uint8_t*>(p.c.v_codes) + static_cast<int64_t>(page) * p.c.page_stride +
                               static_cast<int64_t>(h) * p.c.head_stride +
                               static_cast<int64_t>(first & static_cast<int>(p.c.page_size - 1)) * p.c.token_stride;
#pragma unroll 1
        for (int key = first; key < first + 16; ++key, codes += p.c.token_stride) {
            if (key >= row_end || (key < lo && key >= sinks_of<MODE>(p))) continue;
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half) {
                uint32_t any = 0;
#pragma unroll
                for (uint32_t c = 4 * half; c < 4 * half + 4; ++c) {
                    const uint4 q = c < pieces ? __ldg(reinterpret_cast<const uint4*>(codes) + c) : make_uint4(0, 0, 0, 0);
                    any |= e4m3_nan_flags(q.x) | e4m3_nan_flags(q.y) | e4m3_nan_flags(q.z) | e4m3_nan_flags(q.w);
                }
                if (any == 0) continue;
#pragma unroll 1
                for (uint32_t e = 0; e < 64 && 64 * half + e < p.c.head_dim; ++e) {
                    const uint32_t d = 64 * half + e;
                    if ((codes[d] & 0x7F) != 0x7F || (marked[half] >> e & 1u)) continue;
                    marked[half] |= 1ull << e;
                    if (dst) dst[d] = 0x7FC0u;   // a NaN in BF16 and in FP16
                    else part[d * stride] = __uint_as_float(0x7FC00000u);
                }
            }
        }
    }
}
// kPrefix: the CTAs that take part where the suffix pass runs beside this one: by the time of a unit here (256 rows, 128
// keys) to that of one there (64 keys of a sequence and head, read once), some kUnitCost, where an item's begin and end
// count as kOwnItem units there. us with costs of 5 and 0, 4 and 0, 8 and 4 (heads of 128, 8 but where it says otherwise): 64 sequences on 16384
// with 150 to 600 keys of their own 47.7 49.8 47.7; 16 on 8000 (75 to 300) 27.8 23.6 23.6; 32 on 10000 (2 heads, 100 to 400)
// 35.2 35.0 35.0; 16 of 5 tokens on 4001 (16 heads of 64, 75 to 300) 22.6 20.4 20.4; 64 on 2000 (4 heads, 25 to 100) 19.7 21.1
// 20.7; 24 of 2 tokens on 3000 (heads of 64, 15 to 60) 19.6 19.6 18.3.
constexpr uint32_t kUnitCost = 8, kOwnItem = 4;
// ragged: as prefix_is_ragged.
__device__ __forceinline__ bool seq_is_ragged(const AttnArgs& p, const Seq& s) {
    return s.count > 0 && s.len > 0 && max(s.len - s.count, 0) + 1 < p.span.lower;
}
// seen: keys that some row sees, at most.
__device__ __forceinline__ int seq_end(const Seq& s) { return s.count > 0 ? s.len : 0; }
__device__ __noinline__ uint32_t prefix_share(const AttnArgs& p, uint64_t* sh, bool& ragged, int& seen) {
    const uint32_t rows = p.span.rows.max_q * p.group <= 8 ? 8u : 16u;
    uint64_t n = 0;
    bool any = false;
    int end = 0;
    for (uint32_t b = threadIdx.x; b < p.span.rows.batch; b += blockDim.x) {
        const Seq s = sequence(p.span.rows, p.c.page_size, b);
        any = any || seq_is_ragged(p, s);
        end = max(end, seq_end(s));
        if (s.len > p.span.lower)
            n += static_cast<uint64_t>((static_cast<uint32_t>(s.count) * p.group + rows - 1) / rows) * ((s.len - p.span.lower + 63) / 64 + kOwnItem);
    }
    n = warp_sum(n);
    end = __reduce_max_sync(0xFFFFFFFFu, end);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = n, sh[kWarpsAll + (threadIdx.x >> 5)] = end;
    ragged = __syncthreads_or(any) != 0;
    n = 0;
    for (uint32_t w = 0; w < kWarpsAll; ++w) n += sh[w], end = max(end, static_cast<int>(sh[kWarpsAll + w]));
    seen = end;
    const uint64_t here = p.span.pass.total * kUnitCost, share = divide(here * p.ctas, here + n * p.c.kv_heads);
    return PrefixPass::even(min(static_cast<uint64_t>(p.span.pass.ctas), max(share, static_cast<uint64_t>(p.ctas / 4))),
                            static_cast<uint64_t>(p.span.pass.tiles) * p.c.kv_heads);
}
// kPrefix: whether a row that sees keys at all sees fewer than the prefix holds; for a warp.
__device__ __noinline__ bool prefix_is_ragged(const AttnArgs& p, int& seen) {
    bool ragged = false;
    seen = 0;
    for (uint32_t b = threadIdx.x & 31; b < p.span.rows.batch; b += 32) {
        const Seq s = sequence(p.span.rows, p.c.page_size, b);
        ragged = ragged || seq_is_ragged(p, s);
        seen = max(seen, seq_end(s));
    }
    seen = __reduce_max_sync(0xFFFFFFFFu, seen);
    return __any_sync(0xFFFFFFFFu, ragged) != 0;
}

// ----------------------------------------------------------------- kernel --
template <bool F16, uint32_t DP, SpanMode MODE>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_tc_kernel(const AttnArgs p) {
    using C = Cfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t sh_units[kChunk];
    __shared__ Blocks sh_blocks;
    uint8_t* const smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    Tail* const tl = reinterpret_cast<Tail*>(smem + C::kTail);
    const uint32_t sbase = smem_u32(smem);
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    volatile int* const abort_flag = &tl->abort_flag;
    const uint64_t tmo = p.timeout_ns;

    if (warp == kIssueWarp) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(&tl->qfull[i]), 4);
                mbar_init(smem_u32(&tl->kfull[i]), kConvWarps);
                mbar_init(smem_u32(&tl->vfull[i]), kConvWarps);
                mbar_init(smem_u32(&tl->kempty[i]), 1);
                mbar_init(smem_u32(&tl->vempty[i]), 1);
                mbar_init(smem_u32(&tl->sfull[i]), 2);   // the products' completion, and the issuer's own arrival
                for (int k = 0; k < 2; ++k) {
                    mbar_init(smem_u32(&tl->pfull[i][k]), 4);
                    mbar_init(smem_u32(&tl->odone[i][k]), 2);
                }
            }
            for (uint32_t i = 0; i < kRing; ++i) {
                mbar_init(smem_u32(&tl->lfull[i]), 1);
                mbar_init(smem_u32(&tl->lempty[i]), 1);
            }
            mbar_init(smem_u32(&tl->drain), 1);
            sh_blocks.most = 0;
            tl->abort_flag = 0;
            tl->nan_seen = 0;
            for (uint32_t i = 0; MODE != kFull && i < kNanWords; ++i) tl->nan_groups[i] = 0;
            fence_barrier_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(&tl->tmem), 512);
        tmem_relinquish();
    }
    grid_dependency_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tl->tmem;

    constexpr bool kMayBeWhole = MODE == kWindow || MODE == kSuffix;
    Blocks* const blocks = kMayBeWhole && p.b.batch <= kChunk ? &sh_blocks : nullptr;
    const uint64_t total = MODE == kPrefix ? p.span.pass.total : total_units<kWarpsAll, MODE>(p, sh_units, blockIdx.x == 0, blocks);
    zero_keyless<MODE>(p);
    uint64_t ctas = active_ctas(total, p.ctas);
    bool ragged = false;
    int seen = 0;
    if constexpr (MODE == kPrefix) {
        ctas = p.span.pass.ctas;
        grid_launch_dependents();   // a suffix pass runs beside this one, on the SMs that are left
        if (p.span.pass.taken != nullptr) {
            ctas = prefix_share(p, sh_units, ragged, seen);
            if (blockIdx.x == 0 && threadIdx.x == 0) *p.span.pass.taken = static_cast<uint32_t>(ctas);
        }
    }
    bool whole_items = false;
    uint64_t items = 0;
    if constexpr (kMayBeWhole) {
        if (blocks != nullptr) {
            for (uint32_t i = lane; i < p.b.batch; i += 32) items += blocks->of[i];
            items = warp_sum(items) * p.c.kv_heads;
            whole_items = divide(items + p.ctas - 1, p.ctas) * blocks->most <= divide(total, p.ctas) + kSplitCost;
            if (whole_items) {
                ctas = active_ctas(items, p.ctas);
                __syncthreads();   // sh_units has been read
                for (uint32_t i = threadIdx.x; i < p.b.batch; i += kThreads) sh_units[i] = blocks->of[i];
                __syncthreads();
            }
        }
    }
    const bool works = blockIdx.x < ctas;
    uint64_t u0 = works ? first_unit(blockIdx.x, whole_items ? items : total, ctas) : 0,
             u_end = works ? first_unit(blockIdx.x + 1, whole_items ? items : total, ctas) : 0;
    float* const slots = p.ws + boundary_floats(p.ctas);
    if (MODE != kPrefix && !works && threadIdx.x == 0) write_boundary(p.ws, Boundary{});
    if (works) {
        Item it;
        if constexpr (MODE == kPrefix) it = prefix_item(p, u0);
        else it = find_item<kWarpsAll, MODE>(p, u0, sh_units, whole_items);
        if (kMayBeWhole && whole_items) {   // from items to the units of this CTA's, counted from its first one's
            const uint64_t n = u_end - u0;
            it.first = u0 = 0;
            u_end = it.n;
            Item next = it;
            for (uint64_t i = 1; i < n; ++i) {
                next_item<MODE>(p, next);
                u_end += next.n;
            }
        }
        if (MODE != kPrefix && threadIdx.x == 0) write_boundary(p.ws, whole_items ? Boundary{} : boundary_of(u0, it.first, it.n, it.s, it.h, it.rb, total, ctas));
        uint64_t u = u0;

        if (warp < kSoftmaxWarps) {
            // ------------------------------------------------------------ softmax
            const uint32_t t = warp / 4, row = (warp % 4) * 32 + lane;      // row of the tile
            const uint32_t lanes = ((warp % 4) * 32) << 16;
            const uint32_t tS = tm + t * kTile + lanes, tO = tm + 2 * kTile + t * DP + lanes;
            uint32_t blocks = 0;   // of this tile
            bool first_part = true, fetched = false, ok = true;
            // Asks for the warp's 32 query rows of an item, as they are, into its place in the Q tile. A row's 16-byte pieces are
            // neighbouring lanes', so a copy touches few lines (a row a thread, 32 lines a load, took 10000 cycles an item).
            constexpr uint32_t kPieces = DP / 8, kRowsAtOnce = 32 / kPieces, kSteps = 32 / kRowsAtOnce;
            const uint32_t piece = lane % kPieces, in_step = lane / kPieces;
            uint8_t* const qs = smem + C::kQ + t * C::kTileBytes + (piece / 8) * C::kHalfBytes + (warp % 4) * 32 * 128;
            const auto qs_at = [&](uint32_t from) { return reinterpret_cast<uint4*>(qs + from * 128 + (((piece % 8) ^ (from & 7)) << 4)); };
            const auto fetch = [&](const Item& x) {
                const uint32_t R = static_cast<uint32_t>(x.s.count) * p.group, r0 = x.rb * kItemRows + t * kTile + (warp % 4) * 32;
                const uint32_t r = min(r0 + lane, R - 1);
                const uint64_t mine = reinterpret_cast<uint64_t>(static_cast<const uint16_t*>(p.q.ptr) +
                                                                 static_cast<int64_t>(x.s.first + static_cast<int>(r / p.group)) * p.q.token_stride +
                                                                 static_cast<int64_t>(x.h * p.group + r % p.group) * p.q.head_stride);
#pragma unroll 4
                for (uint32_t s = 0; s < kSteps; ++s) {
                    const uint32_t from = s * kRowsAtOnce + in_step;
                    const auto* const src = reinterpret_cast<const uint16_t*>(__shfl_sync(0xFFFFFFFFu, mine, from));
                    uint4* const to = qs_at(from);
                    if (r0 + from < R && 8 * piece < p.c.head_dim) cp_async_16(smem_u32(to), src + 8 * piece);
                    else *to = make_uint4(0, 0, 0, 0);
                }
                cp_async_commit();
            };
            while (ok && u < u_end) {
                const uint32_t j0 = static_cast<uint32_t>(u - it.first);
                const uint32_t cnt = static_cast<uint32_t>(min(static_cast<uint64_t>(it.n - j0), u_end - u));
                const uint32_t R = static_cast<uint32_t>(it.s.count) * p.group;
                const uint32_t tile_row0 = it.rb * kItemRows + t * kTile;
                if (tile_row0 < R) {
                    if (!fetched) fetch(it);   // (first of all: what else an item's begin needs is loaded beside it)
                    fetched = false;
                    // the query row, FP16, times 2^(7 - exponent of its maximum), 128-byte swizzled
                    const uint32_t r = tile_row0 + row;
                    const bool real = r < R;
                    const uint32_t tok = real ? r / p.group : 0, head = it.h * p.group + (real ? r % p.group : 0);
                    int row_end = real ? it.s.len - it.s.count + static_cast<int>(tok) + 1 : 0x7FFFFFFF;
                    const uint32_t r_w = min(tile_row0 + (warp % 4) * 32, R - 1);
                    int warp_min = it.s.len - it.s.count + static_cast<int>(r_w / p.group) + 1;
                    // but for kFull: in the order of the item's groups, where the row's keys begin and end, and where the last row's begin
                    int v_lo = 0, v_end = 0, v_warp_lo = 0;
                    Groups span{};
                    if constexpr (MODE != kFull) {
                        if (MODE == kPrefix) {
                            if (real) row_end = prefix_row_end(p, tok);
                            warp_min = __reduce_min_sync(0xFFFFFFFFu, row_end);
                        }
                        span = block_groups<MODE>(p, it.s, it.rb);
                        const int last = it.s.len - it.s.count + static_cast<int>(min(tile_row0 + (warp % 4) * 32 + 31, R - 1) / p.group) + 1;
                        v_lo = row_lo<MODE>(p, real ? row_end : 0) - 16 * span.skip;
                        v_end = row_end - 16 * span.skip;
                        v_warp_lo = row_lo<MODE>(p, last) - 16 * span.skip;
                        warp_min -= 16 * span.skip;
                    }
                    // Each row times 2^(7 - exponent of its maximum), in place: a thread a row, whose 16-byte pieces the swizzle puts
                    // on other banks than its neighbours'. (Magnitudes order as their bits do, those that are not finite above.)
                    cp_async_wait_group<0>();
                    __syncwarp();
                    uint8_t* const qrow = smem + C::kQ + t * C::kTileBytes + row * 128;
                    const auto piece_at = [&](uint32_t k) { return reinterpret_cast<uint4*>(qrow + (k / 8) * C::kHalfBytes + (((k % 8) ^ (row & 7)) << 4)); };
                    uint32_t m2 = 0;
#pragma unroll
                    for (uint32_t k = 0; k < DP / 8; ++k) {
                        const uint4 a = *piece_at(k);
                        m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu), __vmaxu2(a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu)));
                    }
                    const uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
                    const RowScale rs = row_scale_of(unpack2<F16>(top).x, top >= (F16 ? 0x7C00u : 0x7F80u), p.scale_log2);
                    float rowf = rs.scale;
#pragma unroll 1
                    for (uint32_t k0 = 0; k0 < DP / 8; k0 += 4) {
                        uint4 a[4];
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) a[k] = *piece_at(k0 + k);
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            uint32_t w[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 x = unpack2<F16>(w[e]);
                                w[e] = rs.f1 == 0.f ? 0u : pack2<true>(x.x * rs.f1 * rs.f2, x.y * rs.f1 * rs.f2);   // (0: a row that is not finite)
                            }
                            *piece_at(k0 + k) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    // a padding row is one that sees no key: it is zero whatever its query holds
                    if (rowf != rowf && row_end <= 0) rowf = 0.f;
                    fence_proxy_async_smem();
                    tc_fence_before();   // the previous item's reads of O come before this one's products
                    __syncwarp();
                    if (lane == 0) mbar_arrive(smem_u32(&tl->qfull[t]));
                    const uint32_t unit0 = static_cast<uint32_t>(u - u0);   // the CTA's units, those of both tiles

                    float ref = -INFINITY, l = 0.f;
#pragma unroll 1
                    for (uint32_t j = 0; j < 2 * cnt; ++j, ++blocks) {
                        const uint32_t half = j & 1, tB = tS + half * kBlockKeys;
                        if (half == 0) {
                            if (!(ok = wait_warp(smem_u32(&tl->sfull[t]), (blocks >> 1) & 1, tmo, abort_flag, kWaitS))) break;
                            tc_fence_after();
                            if (j + 2 == 2 * cnt && u + cnt < u_end) {   // the item's products have read the tile: the next one's rows
                                Item next = it;
                                next_item<MODE>(p, next);
                                fetched = next.rb * kItemRows + t * kTile < static_cast<uint32_t>(next.s.count) * p.group;
                                if (fetched) fetch(next);
                            }
                        }
                        const Look& look = tl->look[(unit0 + j / 2) % kRing];
                        const int key0 = static_cast<int>(j0 * kTile + j * kBlockKeys);
                        // ---- the row's 64 scores, and the largest y = score ks rowf + log2(vs)
                        uint32_t v[2][32];
                        tmem_ld32(tB, v[0]);
                        tmem_ld32(tB + 32, v[1]);
                        tc_wait_ld();
                        if constexpr (MODE != kFull) {
                            if (key0 + static_cast<int>(kBlockKeys) > warp_min || (key0 < v_warp_lo && key0 + static_cast<int>(kBlockKeys) > sinks_of<MODE>(p))) {
                                mask_span(v[0], key0, v_end, v_lo, sinks_of<MODE>(p));
                                mask_span(v[1], key0 + 32, v_end, v_lo, sinks_of<MODE>(p));
                            }
                        } else if (key0 + static_cast<int>(kBlockKeys) > warp_min) {
                            mask_scores(v[0], 0, row_end - key0);
                            mask_scores(v[1], 32, row_end - key0);
                        }
                        const float *ks = look.ks + 4 * half, *lv = look.lv + 4 * half, *iv = look.iv + 4 * half;
                        const float ymax = fmaxf(score_max(v[0], ks, lv, rowf), score_max(v[1], ks + 2, lv + 2, rowf));
                        if (__any_sync(0xFFFFFFFFu, ymax > ref + kRise)) {
                            // the maximum moves: the sum and, once the products so far are in it, O are rescaled
                            const float m_new = fmaxf(ref, ymax);
                            const float a = ref == -INFINITY ? 0.f : ex2(ref - m_new);
                            l *= a;
                            ref = m_new;
                            if (j > 0) {
                                if (!(ok = wait_warp(smem_u32(&tl->odone[t][half ^ 1]), ((blocks - 1) >> 1) & 1, tmo, abort_flag, kWaitO))) break;
                                tc_fence_after();
#pragma unroll 1
                                for (uint32_t d = 0; d < DP; d += 8) {
                                    float o[8];
                                    tmem_ld_32x32b_x8(tO + d, o);
                                    tc_wait_ld();
                                    tmem_st8(tO + d, o, a);
                                }
                            }
                        }
                        const float rc = ref == -INFINITY ? 0.f : ref - kPBits;
#pragma unroll
                        for (int ch = 0; ch < 2; ++ch) {
                            uint32_t pk[16];
                            l = score_weights(v[ch], ks + 2 * ch, lv + 2 * ch, iv + 2 * ch, rowf, rc, l, pk);
                            tmem_st_32x32b_x16(tB + 16 * ch, pk);
                        }
                        tc_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(&tl->pfull[t][half]));
                    }
                    // The last unit's products. Each half has a barrier of its own, whose phases are the tile's
                    // units: a parity tells one phase from the next only, and when both of these products end
                    // before they are first asked for, the phases of one shared barrier would be taken for others.
                    const uint32_t last = ((blocks >> 1) - 1) & 1;
                    ok = ok && wait_warp(smem_u32(&tl->odone[t][0]), last, tmo, abort_flag, kWaitO) &&
                         wait_warp(smem_u32(&tl->odone[t][1]), last, tmo, abort_flag, kWaitO);
                    if (!ok) break;
                    tc_fence_after();
                    // ---- outputs, or this range's part of them ([d][row], coalesced over rows)
                    const bool whole = cnt == it.n;
                    float* slot = slots + (static_cast<uint64_t>(blockIdx.x) * 2 + (first_part ? 0 : 1)) * ((DP + 2) * kItemRows);
                    const bool none = l == 0.f;   // a row that sees no key is zero
                    const float inv = none ? 0.f : 1.f / l;
                    float* put = nullptr;   // kPrefix: the row's record, or its place in this CTA's slot
                    if constexpr (MODE != kFull) {
                        if (MODE == kPrefix) {
                            const uint64_t at = static_cast<uint64_t>(tok) * p.q.heads + head;
                            put = whole ? record_row(p.span.record, at, DP) : slot + (t * kTile + row) * DP;
                            if (!whole) {
                                slot[DP * kItemRows + t * kTile + row] = ref;
                                slot[(DP + 1) * kItemRows + t * kTile + row] = l;
                            } else if (real) {
                                *reinterpret_cast<float2*>(record_max(p, p.span.record, at, DP)) = make_float2(ref, l);
                            }
                        }
                    }
                    uint16_t* dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(it.s.first + static_cast<int>(tok)) * p.out.token_stride +
                                    static_cast<int64_t>(head) * p.out.head_stride;
                    // Rows that go out whole are turned through shared memory, 64 bytes of each at a time, so that neighbouring
                    // lanes write one row's pieces.
                    uint8_t* const turn = smem + C::kTurn + warp * kTurnBytes;
                    const auto pass = [&](const uint4* q, uint64_t to, uint32_t byte0, uint32_t bytes) {   // `to`: of this lane's row, or 0
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) *reinterpret_cast<uint4*>(turn + lane * 64 + ((k ^ (lane >> 1 & 3)) << 4)) = q[k];
                        __syncwarp();
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            const uint32_t from = 8 * k + lane / 4, byte = byte0 + 16 * (lane % 4);
                            const uint64_t row_to = __shfl_sync(0xFFFFFFFFu, to, from);
                            if (row_to != 0 && byte < bytes)
                                *reinterpret_cast<uint4*>(row_to + byte) = *reinterpret_cast<const uint4*>(turn + from * 64 + (((lane % 4) ^ (from >> 1 & 3)) << 4));
                        }
                        __syncwarp();
                    };
                    if (MODE == kPrefix || whole) {
                        PrefixRow px{};
                        if (MODE == kSuffix && real) px = prefix_row(p, static_cast<uint32_t>(it.s.first) + tok, head, DP);
                        const uint64_t to = !real ? 0 : reinterpret_cast<uint64_t>(MODE == kPrefix ? static_cast<void*>(put) : static_cast<void*>(dst));
#pragma unroll 1
                        for (uint32_t d = 0; d < DP; d += 32) {
                            uint32_t o[32];
                            __syncwarp();   // (rows differ in what they add)
                            tmem_ld32(tO + d, o);
                            tc_wait_ld();
                            if (none) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = 0u;
                            }
                            uint4 q[8];
                            if constexpr (MODE == kPrefix) {
#pragma unroll
                                for (int e = 0; e < 32; e += 4) q[e / 4] = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                                pass(q, to, 4 * d, 4 * p.c.head_dim);
                                pass(q + 4, to, 4 * d + 64, 4 * p.c.head_dim);
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; e += 8) {
                                    float x[8], f = inv;
#pragma unroll
                                    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(o[e + k]);
                                    if constexpr (MODE == kSuffix) {
                                        float m8 = ref, l8 = l;
                                        if (real) add_prefix<8>(p, px, DP, d + e, m8, l8, x);
                                        f = l8 == 0.f ? 0.f : 1.f / l8;
                                    }
                                    q[e / 8] = make_uint4(pack2<F16>(x[0] * f, x[1] * f), pack2<F16>(x[2] * f, x[3] * f), pack2<F16>(x[4] * f, x[5] * f),
                                                          pack2<F16>(x[6] * f, x[7] * f));
                                }
                                pass(q, to, 2 * d, 2 * p.c.head_dim);
                            }
                        }
                    } else {
#pragma unroll 1
                        for (uint32_t d = 0; d < DP; d += 32) {
                            uint32_t o[32];
                            tmem_ld32(tO + d, o);
                            tc_wait_ld();
                            if (none) {
#pragma unroll
                                for (int e = 0; e < 32; ++e) o[e] = 0u;
                            }
#pragma unroll
                            for (int e = 0; e < 32; ++e) slot[(d + e) * kItemRows + t * kTile + row] = __uint_as_float(o[e]);
                        }
                    }
                    if (!whole && !(MODE != kFull && put != nullptr)) {
                        slot[DP * kItemRows + t * kTile + row] = ref;
                        slot[(DP + 1) * kItemRows + t * kTile + row] = l;
                    }
                    if constexpr (MODE != kFull) {
                        if (*static_cast<volatile int*>(&tl->nan_seen) != 0 && real)
                            mark_nan_span<MODE>(p, tl, unit0, static_cast<uint32_t>(u_end - u0), it.b, it.h, span, j0, cnt, row_end,
                                                whole && put == nullptr ? dst : nullptr, put != nullptr ? put : slot + t * kTile + row,
                                                put != nullptr ? 1u : kItemRows);
                    } else if (*static_cast<volatile int*>(&tl->nan_seen) != 0 && real)
                        mark_nan(p, it.b, it.h,
                                 max(static_cast<int>(j0 * kTile), edge_key(it.s, p.group, it.rb) / static_cast<int>(kTile) * static_cast<int>(kTile)),
                                 min(row_end, static_cast<int>((j0 + cnt) * kTile)), whole ? dst : nullptr, slot + t * kTile + row);
                }
                first_part = false;
                u += cnt;
                if (u < u_end) next_item<MODE>(p, it);
            }
            cp_async_wait_group<0>();   // after a wait that gave up
        } else if (warp == kIssueWarp) {
            // ------------------------------------------------------- products
            // The whole warp goes through the loops, on broadcast counts, and one elected lane issues:
            // so descriptors are formed in uniform registers. (A lane of its own formed them in
            // ordinary ones and took longer over each product than the tensor core.)
            constexpr uint32_t idS = idesc_f16(kTile, kTile, false), idO = idesc_f16(kTile, DP, true);
            constexpr uint32_t kBlockDesc = (kBlockKeys * 128) >> 4;   // descriptors count 16 bytes
            const uint32_t tmu = __shfl_sync(0xFFFFFFFFu, tm, 0), sb = __shfl_sync(0xFFFFFFFFu, sbase, 0);
            const uint64_t desc_q = smem_desc_kmajor_sw128(sb + C::kQ), desc_k = smem_desc_kmajor_sw128(sb + C::kK),
                           desc_v = smem_desc_mn_sw128(sb + C::kV, C::kHalfBytes);
            const bool elected = elect_one();
            const auto scores = [&](uint32_t t, uint32_t unit) {   // S of the CTA's unit
                const uint64_t q0 = desc_q + t * (C::kTileBytes >> 4), k0 = desc_k + unit % kStages * (C::kTileBytes >> 4);
                if (elected) {
#pragma unroll
                    for (uint32_t k = 0; k < DP / 16; ++k) {
                        const uint32_t off = ((k / 4) * C::kHalfBytes + (k % 4) * 32) >> 4;
                        mma_ss(tmu + t * kTile, q0 + off, k0 + off, idS, k > 0);
                    }
                    tc_commit(smem_u32(&tl->sfull[t]));
                    mbar_arrive(smem_u32(&tl->sfull[t]));
                }
            };
            const auto outputs = [&](uint32_t t, uint32_t unit, uint32_t half, bool add) {   // O += P V of half a unit
                const uint64_t v0 = desc_v + unit % kStages * (C::kTileBytes >> 4) + half * kBlockDesc;
                if (elected) {
#pragma unroll
                    for (uint32_t k = 0; k < kBlockKeys / 16; ++k)
                        tc_mma_a_tmem(tmu + 2 * kTile + t * DP, tmu + t * kTile + half * kBlockKeys + 8 * k, v0 + k * (2048 >> 4), idO, add || k > 0);
                    tc_commit(smem_u32(&tl->odone[t][half]));
                    mbar_arrive(smem_u32(&tl->odone[t][half]));
                }
            };
            bool ok = true;
            uint32_t unit = 0;                            // the CTA's units so far
            uint32_t nq0 = 0, nq1 = 0, np0 = 0, np1 = 0;  // items and units of each tile so far
            while (ok && u < u_end) {
                const uint32_t cnt = __shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(min(it.first + it.n - u, u_end - u)), 0);
                const uint32_t tiles = __shfl_sync(0xFFFFFFFFu, static_cast<uint32_t>(it.s.count) * p.group > it.rb * kItemRows + kTile ? 2u : 1u, 0);
                ok = wait_warp(smem_u32(&tl->kfull[unit % kStages]), (unit / kStages) & 1, tmo, abort_flag, kWaitK) &&
                     wait_warp(smem_u32(&tl->qfull[0]), nq0++ & 1, tmo, abort_flag, kWaitQ) &&
                     (tiles == 1 || wait_warp(smem_u32(&tl->qfull[1]), nq1++ & 1, tmo, abort_flag, kWaitQ));
                if (!ok) break;
                tc_fence_after();
                scores(0, unit);
                if (tiles == 2) scores(1, unit);
                if (elected) tc_commit(smem_u32(&tl->kempty[unit % kStages]));
#pragma unroll 1
                for (uint32_t j = 0; j < cnt; ++j, ++unit) {
                    // the first half's products of both tiles
                    ok = wait_warp(smem_u32(&tl->vfull[unit % kStages]), (unit / kStages) & 1, tmo, abort_flag, kWaitV) &&
                         wait_warp(smem_u32(&tl->pfull[0][0]), np0 & 1, tmo, abort_flag, kWaitP);
                    if (!ok) break;
                    tc_fence_after();
                    outputs(0, unit, 0, j > 0);
                    if (tiles == 2) {
                        if (!(ok = wait_warp(smem_u32(&tl->pfull[1][0]), np1 & 1, tmo, abort_flag, kWaitP))) break;
                        tc_fence_after();
                        outputs(1, unit, 0, j > 0);
                    }
                    // the second half's, each followed by the next unit's S over P, which the products
                    // ahead of it in order have then read
                    const bool next = j + 1 < cnt;
                    ok = (!next || wait_warp(smem_u32(&tl->kfull[(unit + 1) % kStages]), ((unit + 1) / kStages) & 1, tmo, abort_flag, kWaitK)) &&
                         wait_warp(smem_u32(&tl->pfull[0][1]), np0++ & 1, tmo, abort_flag, kWaitP);
                    if (!ok) break;
                    tc_fence_after();
                    outputs(0, unit, 1, true);
                    if (next) scores(0, unit + 1);
                    if (tiles == 2) {
                        if (!(ok = wait_warp(smem_u32(&tl->pfull[1][1]), np1++ & 1, tmo, abort_flag, kWaitP))) break;
                        tc_fence_after();
                        outputs(1, unit, 1, true);
                        if (next) scores(1, unit + 1);
                    }
                    if (elected) {   // the unit's V, and what was looked up for it, are done with
                        tc_commit(smem_u32(&tl->vempty[unit % kStages]));
                        tc_commit(smem_u32(&tl->lempty[unit % kRing]));
                        if (next) tc_commit(smem_u32(&tl->kempty[(unit + 1) % kStages]));
                    }
                }
                u += cnt;
                if (ok && u < u_end) next_item<MODE>(p, it);
            }
            // every product issued ends before TMEM is released
            if (elected) {
                tc_commit(smem_u32(&tl->drain));
                volatile int never = 0;
                mbar_wait_for(smem_u32(&tl->drain), 0, tmo, &never, &g_kv_attn_tc_status, kWaitDrain);
            }
        } else if (warp == kLookWarp) {
            // ------------------------------------------------- pages and scales
            // lane 8 q + g: group g of the q-th of the next kLook units
            const uint32_t q = lane / 8, g = lane % 8;
            // The item's keys: it_end; the units with keys that some row does not see: from it_edge on and, but for kFull, below it_lo.
            // There it_end, it_edge and it_lo are in the order of its groups, of which the first it_head come without it_skip.
            if (MODE == kPrefix && p.span.pass.taken == nullptr) ragged = prefix_is_ragged(p, seen);
            int it_end = 0, it_edge = 0, it_lo = 0, it_head = 0, it_skip = 0;
            const auto enter = [&] {
                it_end = block_end(it.s, p.group, it.rb);
                it_edge = edge_key(it.s, p.group, it.rb);
                if constexpr (MODE != kFull) {
                    const Groups g = block_groups<MODE>(p, it.s, it.rb);
                    it_lo = row_lo<MODE>(p, it_end) - 16 * g.skip;
                    it_edge = MODE == kPrefix ? (ragged ? 0 : p.span.lower) : it_edge - 16 * g.skip;
                    it_head = g.head, it_skip = g.skip;
                    it_end = g.count == 0 ? 0 : g.end - 16 * g.skip;
                }
            };
            enter();
            uint32_t i = 0;   // the CTA's units so far
            bool ok = true;
#pragma unroll 1
            while (ok && u < u_end) {
                const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(kLook), u_end - u));
                int key0 = 0, end = 0, edge = 0, head = 0, skip = 0;
                uint32_t b = 0, h = 0;
#pragma unroll 1
                for (uint32_t k = 0; k < n; ++k, ++u) {
                    if (u >= it.first + it.n) {
                        next_item<MODE>(p, it);
                        enter();
                    }
                    if (k == q) {
                        key0 = static_cast<int>(u - it.first) * static_cast<int>(kTile);
                        end = it_end;
                        edge = (MODE != kFull || it.s.count > 1) && key0 + static_cast<int>(kTile) > it_edge;
                        if constexpr (MODE != kFull) {
                            edge = edge || (key0 < it_lo && key0 + static_cast<int>(kTile) > sinks_of<MODE>(p));
                            head = it_head, skip = it_skip;
                        }
                        b = it.b;
                        h = it.h;
                    }
                }
                int key = key0 + 16 * static_cast<int>(g);
                const bool there = q < n && key < end;
                if (MODE != kFull && key >= 16 * head) key += 16 * skip;
                int page = -1;
                if (there) {
                    page = p.b.page_table[static_cast<int64_t>(b) * p.b.page_table_stride + (key >> p.page_shift)];
                    if (static_cast<uint32_t>(page) >= p.c.num_pages) {
                        record_failure(&g_kv_attn_tc_status, W8A16_STATUS_BAD_INDEX, static_cast<uint32_t>(page));
                        page = -1;
                    }
                }
                float sk = 1.f, sv = 1.f;
                if (page >= 0) {
                    const int64_t at = static_cast<int64_t>(page) * p.c.scale_page_stride + static_cast<int64_t>(h) * p.c.scale_head_stride;
                    sk = p.c.k_scale[at];
                    sv = p.c.v_scale[at];
                    if (sk < kMinScale) sk = kMinScale;
                    if (sv < kMinScale) sv = kMinScale;
                }
                // (past all rows' ends, where nothing need have been written: masked scores have no weight, but with a scale that is not finite)
                if (MODE == kPrefix && key >= seen) sk = sv = 1.f;
                for (uint32_t k = 0; k < n && ok; ++k)
                    ok = wait_warp(smem_u32(&tl->lempty[(i + k) % kRing]), (((i + k) / kRing) & 1) ^ 1, tmo, abort_flag, kWaitLookFree);
                if (!ok) break;
                if (q < n) {
                    Look& look = tl->look[(i + q) % kRing];
                    look.offset[g] = static_cast<int64_t>(max(page, 0)) * p.c.page_stride + static_cast<int64_t>(h) * p.c.head_stride +
                                     static_cast<int64_t>(key & static_cast<int>(p.c.page_size - 1)) * p.c.token_stride;
                    look.ks[g] = sk;
                    look.lv[g] = __log2f(sv);
                    look.iv[g] = __frcp_rn(sv);
                    if (g == 0) {
                        look.last = max(end - 1 - key0, 0);
                        look.edge = edge;
                    }
                }
                __syncwarp();
                if (lane < n) mbar_arrive(smem_u32(&tl->lfull[(i + lane) % kRing]));
                i += n;
            }
        } else {
            // --------------------------------------------- codes -> FP16 tiles
            // A warp takes 32 keys, 8 rows x 4 chunks of 16 codes at a time: 64 contiguous bytes a
            // row from memory, and the eight lanes of a store phase hold one unit of eight rows,
            // which the swizzle spreads over all banks.
            constexpr uint32_t CH = DP / 16, kHalves = DP / 64;
            const uint32_t cw = warp - kSoftmaxWarps, lrow = lane & 7, lch = lane >> 3;
            const uint32_t off0 = min(16 * lch, p.c.head_dim - 16), off1 = min(64 + 16 * lch, p.c.head_dim - 16);
            const uint32_t st0 = (cw * 32 + lrow) * 128 + (((2 * lch) ^ lrow) << 4), st1 = (cw * 32 + lrow) * 128 + (((2 * lch + 1) ^ lrow) << 4);
            const uint32_t units = static_cast<uint32_t>(u_end - u0);
            // Rows past the last key, and chunks past the head, repeat the last ones: their scores are
            // masked and their queries and outputs are not there, and their values are as finite as
            // those that they repeat (in a unit where rows see different keys: after clean_tile).
            int64_t row[4];   // this lane's rows of 8 of the unit being loaded
            const auto load_codes = [&](const void* codes, uint4 (&c)[CH]) {
#pragma unroll
                for (uint32_t i = 0; i < CH; ++i)   // L2 only: the few KB of L1 beside the tiles are for what is used again
                    c[i] = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(codes) + row[i / kHalves] + (i % kHalves ? off1 : off0)));
            };
            const auto store_tile = [&](uint32_t tile, const uint4 (&c)[CH]) {
#pragma unroll
                for (uint32_t i = 0; i < CH; ++i) {
                    uint4 lo, hi;
                    convert16(c[i], lo, hi);
                    uint8_t* at = smem + tile + (i % kHalves) * C::kHalfBytes + i / kHalves * 1024;
                    *reinterpret_cast<uint4*>(at + st0) = lo;
                    *reinterpret_cast<uint4*>(at + st1) = hi;
                }
            };
            const auto signal = [&](uint64_t* bar) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(bar));
            };
            // step i: store unit i (codes in registers), load unit i + 1's
            uint4 kq[CH], vq[CH];
            int edge = 0, next_edge = 0;
#pragma unroll 1
            for (uint32_t i = 0xFFFFFFFFu; i + 1 <= units; ++i) {
                const uint32_t st = i % kStages, parity = ((i / kStages) & 1) ^ 1;
                const bool have = i != 0xFFFFFFFFu, more = i + 1 < units;
                if (have) {
                    if (!wait_warp(smem_u32(&tl->kempty[st]), parity, tmo, abort_flag, kWaitKFree)) break;
                    store_tile(C::kK + st * C::kTileBytes, kq);
                    signal(&tl->kfull[st]);
                }
                if (more) {
                    if (!wait_warp(smem_u32(&tl->lfull[(i + 1) % kRing]), ((i + 1) / kRing) & 1, tmo, abort_flag, kWaitLook)) break;
                    const Look& look = tl->look[(i + 1) % kRing];
                    const int last = look.last;
                    next_edge = look.edge;
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k) {
                        const int r = min(static_cast<int>(32 * cw + 8 * k + lrow), last);
                        row[k] = look.offset[r >> 4] + static_cast<int64_t>(r & 15) * p.c.token_stride;
                    }
                    load_codes(p.c.k_codes, kq);
                }
                if (have) {
                    if (!wait_warp(smem_u32(&tl->vempty[st]), parity, tmo, abort_flag, kWaitVFree)) break;
                    store_tile(C::kV + st * C::kTileBytes, vq);
                    if constexpr (MODE != kFull) {   // a window begins and ends in any item: mostly there is nothing to clean
                        uint32_t nan = 0;
#pragma unroll
                        for (uint32_t k = 0; k < CH; ++k) nan |= e4m3_nan_flags(vq[k].x) | e4m3_nan_flags(vq[k].y) | e4m3_nan_flags(vq[k].z) | e4m3_nan_flags(vq[k].w);
                        edge = edge && nan != 0u;
                    }
                    if (edge) {
                        uint8_t* const even = smem + C::kV + st * C::kTileBytes + st0;
                        uint8_t* const odd = smem + C::kV + st * C::kTileBytes + st1;
                        if constexpr (MODE != kFull) clean_tile<true>(even, odd, CH, kHalves, C::kHalfBytes, tl, 8 * i + 2 * cw, units);
                        else clean_tile<false>(even, odd, CH, kHalves, C::kHalfBytes, tl);
                    }
                    signal(&tl->vfull[st]);
                }
                if (more) load_codes(p.c.v_codes, vq);
                edge = next_edge;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssueWarp) tmem_dealloc(tm, 512);
    if (MODE != kPrefix) grid_launch_dependents();   // late: the join's blocks beside working CTAs cost them 7 % (160 us against 149)
}

// Joins the parts of split items, in an order that their number and the rows' alone decide: a block
// for the k-th split item and 16 dims, a thread a row; where there are 128 rows or fewer, 256 /
// rows threads take a row's parts in turn. Two parts are in flight at a time.
constexpr uint32_t kJoinThreads = kItemRows, kJoinDims = 16;
template <bool F16, SpanMode MODE>
__global__ void __launch_bounds__(kJoinThreads, 4) kv_attn_tc_join_kernel(const AttnArgs p, uint32_t dp) {
    __shared__ float sh_m[kJoinThreads], sh_l[kJoinThreads], sh_acc[kJoinDims][kJoinThreads];
    grid_dependency_wait();
    // (a block for each boundary where most have parts; elsewhere one for each item)
    const uint32_t c = gridDim.x == p.ctas - 1 ? blockIdx.x + 1 : split_boundary<kJoinThreads>(p, blockIdx.x), d0 = blockIdx.y * kJoinDims;
    const Boundary b = reinterpret_cast<const Boundary*>(p.ws)[c];
    if (b.parts == 0) return;   // (of CTA 0 too: fewer items are split)
    const uint32_t rows = min(static_cast<uint32_t>(b.count) * p.group - b.tile * kItemRows, kItemRows);
    const uint32_t lanes = rows <= 32 ? 32u : rows <= 64 ? 64u : rows <= 128 ? 128u : 256u, turns = kJoinThreads / lanes;
    const uint32_t row = threadIdx.x % lanes, turn = threadIdx.x / lanes;
    const uint64_t stride = static_cast<uint64_t>(dp + 2) * kItemRows;
    const float* const slots = p.ws + boundary_floats(p.ctas);
    constexpr uint32_t kAtOnce = 2;
    float m = -INFINITY, l = 0.f, acc[kJoinDims] = {};
    for (uint32_t i0 = turn; i0 < b.parts; i0 += turns * kAtOnce) {
        float x[kAtOnce][kJoinDims], mi[kAtOnce], li[kAtOnce];
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            const uint32_t i = i0 + turns * j;
            mi[j] = -INFINITY, li[j] = 0.f;
#pragma unroll
            for (uint32_t d = 0; d < kJoinDims; ++d) x[j][d] = 0.f;
            if (i < b.parts && row < rows) {
                const float* const s = slots + (i == 0 ? b.slot : 2ull * (c + i - 1)) * stride + row;
                mi[j] = s[dp * kItemRows], li[j] = s[(dp + 1) * kItemRows];
#pragma unroll
                for (uint32_t d = 0; d < kJoinDims; ++d) x[j][d] = s[(d0 + d) * kItemRows];
            }
        }
        float top = m;
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) top = fmaxf(top, mi[j]);
        const float keep = m == -INFINITY ? 0.f : ex2(m - top);
        l *= keep;
#pragma unroll
        for (uint32_t d = 0; d < kJoinDims; ++d) acc[d] *= keep;
        m = top;
#pragma unroll
        for (uint32_t j = 0; j < kAtOnce; ++j) {
            const float a = mi[j] == -INFINITY ? 0.f : ex2(mi[j] - m);   // (0 times NaN: a query that is not finite)
            l = fmaf(a, li[j], l);
#pragma unroll
            for (uint32_t d = 0; d < kJoinDims; ++d) acc[d] = fmaf(a, x[j][d], acc[d]);
        }
    }
    if (turns > 1) {
        sh_m[threadIdx.x] = m, sh_l[threadIdx.x] = l;
#pragma unroll
        for (uint32_t d = 0; d < kJoinDims; ++d) sh_acc[d][threadIdx.x] = acc[d];
        __syncthreads();
        if (turn > 0) return;
        float top = m;
        for (uint32_t t = 1; t < turns; ++t) top = fmaxf(top, sh_m[t * lanes + row]);
        const float keep = m == -INFINITY ? 0.f : ex2(m - top);
        l *= keep;
#pragma unroll
        for (uint32_t d = 0; d < kJoinDims; ++d) acc[d] *= keep;
        for (uint32_t t = 1; t < turns; ++t) {
            const uint32_t at = t * lanes + row;
            const float a = sh_m[at] == -INFINITY ? 0.f : ex2(sh_m[at] - top);
            l = fmaf(a, sh_l[at], l);
#pragma unroll
            for (uint32_t d = 0; d < kJoinDims; ++d) acc[d] = fmaf(a, sh_acc[d][at], acc[d]);
        }
        m = top;
    }
    if (row >= rows) return;
    const uint32_t r = b.tile * kItemRows + row;
    if constexpr (MODE != kFull) {
        if (MODE == kSuffix)
            add_prefix<kJoinDims>(p, prefix_row(p, static_cast<uint32_t>(b.first) + r / p.group, b.h * p.group + r % p.group, dp), dp, d0, m, l, acc);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(b.first + static_cast<int>(r / p.group)) * p.out.token_stride +
                    static_cast<int64_t>(b.h * p.group + r % p.group) * p.out.head_stride + d0;
#pragma unroll
    for (uint32_t d = 0; d < kJoinDims; d += 8)
        *reinterpret_cast<uint4*>(dst + d) = make_uint4(pack2<F16>(acc[d] * inv, acc[d + 1] * inv), pack2<F16>(acc[d + 2] * inv, acc[d + 3] * inv),
                                                        pack2<F16>(acc[d + 4] * inv, acc[d + 5] * inv), pack2<F16>(acc[d + 6] * inv, acc[d + 7] * inv));
}

template <bool F16, uint32_t DP, SpanMode MODE>
cudaError_t launch(const AttnArgs& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kv_attn_tc_kernel<F16, DP, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP>::kSmem);
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
    e = cudaLaunchKernelEx(&cfg, kv_attn_tc_kernel<F16, DP, MODE>, p);
    if (e != cudaSuccess || p.ctas < 2 || MODE == kPrefix) return e;
    const uint64_t items = static_cast<uint64_t>(p.b.batch) * p.c.kv_heads * ((static_cast<uint64_t>(p.b.max_q) * p.group + kItemRows - 1) / kItemRows);
    cfg.gridDim = dim3(static_cast<uint32_t>(items < p.ctas ? items : p.ctas - 1), p.c.head_dim / kJoinDims, 1);   // no more are split
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_attn_tc_join_kernel<F16, MODE>, p, DP);
}

}  // namespace

// Heads above 128 leave no room in TMEM for two row tiles' outputs. Rows: this kernel's time hardly
// depends on them up to 128, the other's goes with tiles of 16. us, that one against this one, 8 heads of 128:
//                             20 rows      32          40          64          128
//     1 sequence of 1000     12.7 16.8  12.9 16.9   13.0 17.2   14.3 17.3   20.3 18.7
//     1 of 16000             30.0 35.1  30.7 35.3   33.0 36.3   44.2 36.6   70.2 40.7
//     16 of 2000             50.2 62.2  52.7 62.5   68.6 62.6   89.8 63.2    150 65.7
//     32 of 8000              243  243   248  245    353  245    466  247    898  250
bool kv_attn_tc_applies(uint32_t head_dim, uint32_t rows_per_head) { return head_dim <= 128 && rows_per_head > 32; }

uint64_t kv_attn_tc_ws_bytes(uint32_t head_dim, int sms) {
    return 4 * boundary_floats(static_cast<uint32_t>(sms)) + 8ull * static_cast<uint32_t>(sms) * ((head_dim <= 64 ? 64u : 128u) + 2) * kItemRows;
}

PrefixPass kv_attn_tc_prefix_pass(const AttnArgs& p, int sms) {
    PrefixPass s;
    s.rows = s.slot_rows = kItemRows;
    s.tiles = (p.b.tokens * p.group + kItemRows - 1) / kItemRows;
    s.units = (static_cast<uint32_t>(p.span.lower) + kTile - 1) / kTile;
    s.total = static_cast<uint64_t>(s.tiles) * s.units * p.c.kv_heads;
    s.taken = nullptr;
    s.joined = false;
    s.ctas = PrefixPass::even(s.total < static_cast<uint64_t>(sms) ? s.total : static_cast<uint64_t>(sms), static_cast<uint64_t>(s.tiles) * p.c.kv_heads);
    s.slots = p.ws + boundary_floats(static_cast<uint32_t>(sms));
    return s;
}
template <SpanMode MODE>
static cudaError_t launch_dim(const AttnArgs& p, bool f16, cudaStream_t s) {
    if (p.c.head_dim <= 64) return f16 ? launch<true, 64, MODE>(p, s) : launch<false, 64, MODE>(p, s);
    return f16 ? launch<true, 128, MODE>(p, s) : launch<false, 128, MODE>(p, s);
}
cudaError_t launch_kv_attn_tc(AttnArgs p, bool f16, SpanMode mode, int sms, cudaStream_t s) {
    p.ctas = static_cast<uint32_t>(sms);
    return mode == kFull     ? launch_dim<kFull>(p, f16, s)
           : mode == kWindow ? launch_dim<kWindow>(p, f16, s)
           : mode == kPrefix ? launch_dim<kPrefix>(p, f16, s)
                             : launch_dim<kSuffix>(p, f16, s);
}

cudaError_t kv_attn_tc_status_read(StatusWord* out, bool clear, cudaStream_t s) {
    DeviceStatus st;
    cudaError_t e = cudaMemcpyFromSymbolAsync(&st, g_kv_attn_tc_status, sizeof st, 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return e;
    out->code = st.code;
    out->where = st.where;
    out->detail = st.detail;
    if (clear) {
        const DeviceStatus zero{0, 0, 0};
        e = cudaMemcpyToSymbolAsync(g_kv_attn_tc_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    return e;
}

}  // namespace w8a16

// Attention over the 8-bit paged cache for many query rows per key/value head (prompt
// chunks): the mathematics of w8a16_kv_attn.cu on the 5th-generation tensor cores.
//
// Work. An item is 256 query rows (two tiles of 128; the G query heads of a key/value head
// times the call's tokens) of one sequence and head, a unit 128 keys of it, with the
// keys that no row of the item sees left out. The units of the whole call are split
// over one CTA per SM in equal contiguous ranges; split items are joined through the
// workspace by a second launch, in a fixed order.
//
// Bound by: the hand-over between the softmax warps and the products. 1024 tokens on 8192 (32 query heads of
// 128 on 8): 150 us, 0.86 PFLOP/s, 46 % of a library product's rate; the tensor pipe is busy for
// 37 % of the kernel's 146 us and the exponentials for 20 %: each tile's scores, weights and
// outputs follow one another, and two tiles do not fill the gaps that a third, for
// which TMEM has no room, would.
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

template <uint32_t DP>
struct Cfg {
    static constexpr uint32_t kTileBytes = kTile * DP * 2;          // an FP16 tile
    static constexpr uint32_t kHalfBytes = kTile * 128;             // a 64-column block of a tile
    static constexpr uint32_t kQ = 0, kK = 2 * kTileBytes, kV = kK + kStages * kTileBytes;
    static constexpr uint32_t kTail = kV + kStages * kTileBytes;    // barriers, scales
    static constexpr uint32_t kSmem = 1024 + kTail + 2048;
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
__device__ __forceinline__ uint32_t block_units(const Seq& s, uint32_t group, uint32_t rb) {
    return max(1, (block_end(s, group, rb) + static_cast<int>(kTile) - 1) / static_cast<int>(kTile));
}
__device__ __forceinline__ uint32_t seq_blocks(const Seq& s, uint32_t group) {
    return s.len <= 0 ? 0u : (static_cast<uint32_t>(s.count) * group + kItemRows - 1) / kItemRows;
}

// Units per key/value head of up to kChunk sequences from b0, a warp per sequence.
template <uint32_t WARPS>
__device__ __forceinline__ uint32_t chunk_units(const AttnArgs& p, uint32_t b0, uint64_t* sh, bool report) {
    const uint32_t count = min(kChunk, p.b.batch - b0);
    for (uint32_t i = threadIdx.x >> 5; i < count; i += WARPS) {
        const Seq s = sequence(p.b, p.c.page_size, b0 + i);
        if (s.bad && report && (threadIdx.x & 31) == 0) record_failure(&g_kv_attn_tc_status, W8A16_STATUS_BAD_INDEX, b0 + i);
        const uint32_t nb = seq_blocks(s, p.group);
        uint64_t n = 0;
        for (uint32_t rb = threadIdx.x & 31; rb < nb; rb += 32) n += block_units(s, p.group, rb);
        n = warp_sum(n);
        if ((threadIdx.x & 31) == 0) sh[i] = n;
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
__device__ __forceinline__ void next_item(const AttnArgs& p, Item& it) {
    it.first += it.n;
    if (++it.rb == seq_blocks(it.s, p.group)) {
        it.rb = 0;
        if (++it.h == p.c.kv_heads) {
            it.h = 0;
            do it.s = sequence(p.b, p.c.page_size, ++it.b);
            while (seq_blocks(it.s, p.group) == 0);   // asked for only where units are left
        }
    }
    it.n = block_units(it.s, p.group, it.rb);
}
// Leaves the counts of the first kChunk sequences in sh.
template <uint32_t WARPS>
__device__ __noinline__ uint64_t total_units(const AttnArgs& p, uint64_t* sh, bool report) {
    uint64_t n = 0;
    for (uint32_t b0 = (p.b.batch - 1) / kChunk * kChunk;; b0 -= kChunk) {
        const uint32_t count = chunk_units<WARPS>(p, b0, sh, report);
        uint64_t x = 0;   // a warp's lanes share the sum
        for (uint32_t i = threadIdx.x & 31; i < count; i += 32) x += sh[i];
        n += warp_sum(x);
        if (b0 == 0) break;
        __syncthreads();
    }
    return n * p.c.kv_heads;
}
// The item that holds unit u (below the total); sh as total_units left it.
template <uint32_t WARPS>
__device__ __noinline__ Item find_item(const AttnArgs& p, uint64_t u, uint64_t* sh) {
    Item it{};
    uint64_t base = 0;
    for (uint32_t b0 = 0; b0 < p.b.batch; b0 += kChunk) {
        if (b0) {
            __syncthreads();
            chunk_units<WARPS>(p, b0, sh, false);
        }
        const uint32_t count = min(kChunk, p.b.batch - b0);
        for (uint32_t i = 0; i < count; ++i) {
            const uint64_t n = sh[i] * p.c.kv_heads;
            if (u < base + n) {
                it.s = sequence(p.b, p.c.page_size, b0 + i);
                it.b = b0 + i;
                it.h = static_cast<uint32_t>((u - base) / sh[i]);
                uint64_t rest = (u - base) % sh[i];
                const uint32_t lane = threadIdx.x & 31, nb = seq_blocks(it.s, p.group);
                for (uint32_t r0 = 0;; r0 += 32) {   // the row block that holds it, 32 at a time
                    const uint32_t mine = r0 + lane < nb ? block_units(it.s, p.group, r0 + lane) : 0u;
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
// would reach them.
__device__ __noinline__ void clean_tile(uint8_t* even, uint8_t* odd, uint32_t chunks, uint32_t halves, uint32_t half_bytes, Tail* tl) {
    for (uint32_t i = 0; i < 2 * chunks; ++i) {
        uint16_t* at = reinterpret_cast<uint16_t*>((i & 1 ? odd : even) + i / 2 % halves * half_bytes + i / 2 / halves * 1024);
        for (int e = 0; e < 8; ++e)
            if ((at[e] & 0x7FFF) > 0x7C00) {
                at[e] = 0;
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

// ----------------------------------------------------------------- kernel --
template <bool F16, uint32_t DP>
__global__ void __launch_bounds__(kThreads, 1) kv_attn_tc_kernel(const AttnArgs p) {
    using C = Cfg<DP>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t sh_units[kChunk];
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
            tl->abort_flag = 0;
            tl->nan_seen = 0;
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

    const uint64_t total = total_units<kWarpsAll>(p, sh_units, blockIdx.x == 0);
    zero_keyless(p);
    const uint64_t ctas = active_ctas(total, p.ctas);
    const bool works = blockIdx.x < ctas;
    const uint64_t u0 = works ? first_unit(blockIdx.x, total, ctas) : 0, u_end = works ? first_unit(blockIdx.x + 1, total, ctas) : 0;
    float* const slots = p.ws + boundary_floats(p.ctas);
    if (!works && threadIdx.x == 0) write_boundary(p.ws, 0, 0, 0, Seq{}, 0, 0, total, ctas);
    if (works) {
        Item it = find_item<kWarpsAll>(p, u0, sh_units);
        if (threadIdx.x == 0) write_boundary(p.ws, u0, it.first, it.n, it.s, it.h, it.rb, total, ctas);
        uint64_t u = u0;

        if (warp < kSoftmaxWarps) {
            // ------------------------------------------------------------ softmax
            const uint32_t t = warp / 4, row = (warp % 4) * 32 + lane;      // row of the tile
            const uint32_t lanes = ((warp % 4) * 32) << 16;
            const uint32_t tS = tm + t * kTile + lanes, tO = tm + 2 * kTile + t * DP + lanes;
            uint32_t blocks = 0;   // of this tile
            bool first_part = true, ok = true;
            while (ok && u < u_end) {
                const uint32_t j0 = static_cast<uint32_t>(u - it.first);
                const uint32_t cnt = static_cast<uint32_t>(min(static_cast<uint64_t>(it.n - j0), u_end - u));
                const uint32_t R = static_cast<uint32_t>(it.s.count) * p.group;
                const uint32_t tile_row0 = it.rb * kItemRows + t * kTile;
                if (tile_row0 < R) {
                    // the query row, FP16, times 2^(7 - exponent of its maximum), 128-byte swizzled
                    const uint32_t r = tile_row0 + row;
                    const bool real = r < R;
                    const uint32_t tok = real ? r / p.group : 0, head = it.h * p.group + (real ? r % p.group : 0);
                    const int row_end = real ? it.s.len - it.s.count + static_cast<int>(tok) + 1 : 0x7FFFFFFF;
                    const uint32_t r_w = min(tile_row0 + (warp % 4) * 32, R - 1);
                    const int warp_min = it.s.len - it.s.count + static_cast<int>(r_w / p.group) + 1;
                    const uint16_t* src = static_cast<const uint16_t*>(p.q.ptr) +
                                          static_cast<int64_t>(it.s.first + static_cast<int>(tok)) * p.q.token_stride +
                                          static_cast<int64_t>(head) * p.q.head_stride;
                    float rowf;
                    {
                        uint32_t w[DP / 2];   // the whole row: its loads are in flight together
#pragma unroll
                        for (uint32_t d = 0; d < DP; d += 8) {
                            uint4 a = make_uint4(0, 0, 0, 0);
                            if (real && d < p.c.head_dim) a = *reinterpret_cast<const uint4*>(src + d);
                            w[d / 2] = a.x, w[d / 2 + 1] = a.y, w[d / 2 + 2] = a.z, w[d / 2 + 3] = a.w;
                        }
                        float mx = 0.f;
                        bool bad = false;
#pragma unroll
                        for (uint32_t e = 0; e < DP / 2; ++e) {
                            const float2 x = unpack2<F16>(w[e]);
                            bad = bad || !(fabsf(x.x) <= 3.4028235e38f) || !(fabsf(x.y) <= 3.4028235e38f);
                            mx = fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y)));
                        }
                        const RowScale rs = row_scale_of(mx, bad, p.scale_log2);
                        // a padding row is one that sees no key: it is zero whatever its query holds
                        rowf = bad && row_end <= 0 ? 0.f : rs.scale;
#pragma unroll
                        for (uint32_t un = 0; un < DP / 8; ++un) {
                            uint32_t o[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 x = unpack2<F16>(w[4 * un + e]);
                                o[e] = bad ? 0u : pack2<true>(x.x * rs.f1 * rs.f2, x.y * rs.f1 * rs.f2);
                            }
                            *reinterpret_cast<uint4*>(smem + C::kQ + t * C::kTileBytes + (un / 8) * C::kHalfBytes + row * 128 +
                                                      (((un % 8) ^ (row & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
                        }
                    }
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
                        }
                        const Look& look = tl->look[(unit0 + j / 2) % kRing];
                        const int key0 = static_cast<int>(j0 * kTile + j * kBlockKeys);
                        // ---- the row's 64 scores, and the largest y = score ks rowf + log2(vs)
                        uint32_t v[2][32];
                        tmem_ld32(tB, v[0]);
                        tmem_ld32(tB + 32, v[1]);
                        tc_wait_ld();
                        if (key0 + static_cast<int>(kBlockKeys) > warp_min) {
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
                    const auto norm = [&](uint32_t x) { return __uint_as_float(x) * inv; };
                    uint16_t* dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(it.s.first + static_cast<int>(tok)) * p.out.token_stride +
                                    static_cast<int64_t>(head) * p.out.head_stride;
#pragma unroll 1
                    for (uint32_t d = 0; d < DP; d += 32) {
                        uint32_t o[32];
                        tmem_ld32(tO + d, o);
                        tc_wait_ld();
                        if (none) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = 0u;
                        }
                        if (whole) {
                            if (real) {
#pragma unroll
                                for (int e = 0; e < 32; e += 8)
                                    if (d + e < p.c.head_dim)
                                        *reinterpret_cast<uint4*>(dst + d + e) =
                                            make_uint4(pack2<F16>(norm(o[e]), norm(o[e + 1])),
                                                       pack2<F16>(norm(o[e + 2]), norm(o[e + 3])),
                                                       pack2<F16>(norm(o[e + 4]), norm(o[e + 5])),
                                                       pack2<F16>(norm(o[e + 6]), norm(o[e + 7])));
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) slot[(d + e) * kItemRows + t * kTile + row] = __uint_as_float(o[e]);
                        }
                    }
                    if (!whole) {
                        slot[DP * kItemRows + t * kTile + row] = ref;
                        slot[(DP + 1) * kItemRows + t * kTile + row] = l;
                    }
                    if (*static_cast<volatile int*>(&tl->nan_seen) != 0 && real)
                        mark_nan(p, it.b, it.h,
                                 max(static_cast<int>(j0 * kTile), edge_key(it.s, p.group, it.rb) / static_cast<int>(kTile) * static_cast<int>(kTile)),
                                 min(row_end, static_cast<int>((j0 + cnt) * kTile)), whole ? dst : nullptr, slot + t * kTile + row);
                }
                first_part = false;
                u += cnt;
                if (u < u_end) next_item(p, it);
            }
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
                if (ok && u < u_end) next_item(p, it);
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
            int it_end = block_end(it.s, p.group, it.rb), it_edge = edge_key(it.s, p.group, it.rb);
            uint32_t i = 0;   // the CTA's units so far
            bool ok = true;
#pragma unroll 1
            while (ok && u < u_end) {
                const uint32_t n = static_cast<uint32_t>(min(static_cast<uint64_t>(kLook), u_end - u));
                int key0 = 0, end = 0, edge = 0;
                uint32_t b = 0, h = 0;
#pragma unroll 1
                for (uint32_t k = 0; k < n; ++k, ++u) {
                    if (u >= it.first + it.n) {
                        next_item(p, it);
                        it_end = block_end(it.s, p.group, it.rb);
                        it_edge = edge_key(it.s, p.group, it.rb);
                    }
                    if (k == q) {
                        key0 = static_cast<int>(u - it.first) * static_cast<int>(kTile);
                        end = it_end;
                        edge = it.s.count > 1 && key0 + static_cast<int>(kTile) > it_edge;
                        b = it.b;
                        h = it.h;
                    }
                }
                const int key = key0 + 16 * static_cast<int>(g);
                int page = -1;
                if (q < n && key < end) {
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
                    if (edge) clean_tile(smem + C::kV + st * C::kTileBytes + st0, smem + C::kV + st * C::kTileBytes + st1, CH, kHalves, C::kHalfBytes, tl);
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
    grid_launch_dependents();   // late: the join's blocks beside working CTAs cost them 7 % (160 us against 149)
}

// Joins the parts of split items, in an order that their number and the rows' alone decide: a block
// for the k-th split item and 16 dims, a thread a row; where there are 128 rows or fewer, 256 /
// rows threads take a row's parts in turn. Two parts are in flight at a time.
constexpr uint32_t kJoinThreads = kItemRows, kJoinDims = 16;
template <bool F16>
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
    }
    if (row >= rows) return;
    const uint32_t r = b.tile * kItemRows + row;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = static_cast<uint16_t*>(p.out.ptr) + static_cast<int64_t>(b.first + static_cast<int>(r / p.group)) * p.out.token_stride +
                    static_cast<int64_t>(b.h * p.group + r % p.group) * p.out.head_stride + d0;
#pragma unroll
    for (uint32_t d = 0; d < kJoinDims; d += 8)
        *reinterpret_cast<uint4*>(dst + d) = make_uint4(pack2<F16>(acc[d] * inv, acc[d + 1] * inv), pack2<F16>(acc[d + 2] * inv, acc[d + 3] * inv),
                                                        pack2<F16>(acc[d + 4] * inv, acc[d + 5] * inv), pack2<F16>(acc[d + 6] * inv, acc[d + 7] * inv));
}

template <bool F16, uint32_t DP>
cudaError_t launch(const AttnArgs& p, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(kv_attn_tc_kernel<F16, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DP>::kSmem);
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
    e = cudaLaunchKernelEx(&cfg, kv_attn_tc_kernel<F16, DP>, p);
    if (e != cudaSuccess || p.ctas < 2) return e;
    const uint64_t items = static_cast<uint64_t>(p.b.batch) * p.c.kv_heads * ((static_cast<uint64_t>(p.b.max_q) * p.group + kItemRows - 1) / kItemRows);
    cfg.gridDim = dim3(static_cast<uint32_t>(items < p.ctas ? items : p.ctas - 1), p.c.head_dim / kJoinDims, 1);   // no more are split
    cfg.blockDim = dim3(kJoinThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, kv_attn_tc_join_kernel<F16>, p, DP);
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

cudaError_t launch_kv_attn_tc(AttnArgs p, bool f16, int sms, cudaStream_t s) {
    p.ctas = static_cast<uint32_t>(sms);
    if (p.c.head_dim <= 64) return f16 ? launch<true, 64>(p, s) : launch<false, 64>(p, s);
    return f16 ? launch<true, 128>(p, s) : launch<false, 128>(p, s);
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

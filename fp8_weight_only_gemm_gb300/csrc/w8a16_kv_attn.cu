// Attention over the 8-bit paged cache: the kernel for few query rows a head (w8a16_kv_attn_few.cuh) for all keys and for
// windows, and the choice between it and the one for many (w8a16_kv_attn_tc.cu).
#include "w8a16_kv_attn_few.cuh"

namespace w8a16 {

template cudaError_t launch_kv_attn_few<kFull>(const AttnArgs&, bool, int, cudaStream_t);
template cudaError_t launch_kv_attn_few<kWindow>(const AttnArgs&, bool, int, cudaStream_t);
extern template cudaError_t launch_kv_attn_few<kPrefix>(const AttnArgs&, bool, int, cudaStream_t);   // w8a16_kv_attn_prefix.cu
extern template cudaError_t launch_kv_attn_few<kSuffix>(const AttnArgs&, bool, int, cudaStream_t);

namespace {

// Whether the sequences' own keys behind a prefix go to the kernel for many rows. The one for few runs beside the prefix pass. us, few and
// many, 8 heads of 128: 4 sequences of 12 tokens (48 rows a head), 600 keys behind 3000, 24 and 95; 16 of them, 700 behind 1000, 57 and 64; 2 of 16
// (64), 2000 behind 3000, 33 and 52; 16 of them, 2000 behind 500, 95 and 90; 16 of 32 (128), 700 behind 1000, 125 and 58. The host knows
// rows, not lengths: where sequences with 33 to 64 rows a head have long keys of their own behind a short prefix this is the slower side
// (32 of 16 tokens, 7500 behind 512: 549, and 248 without a shared prefix; 16, 2000 behind 500: 109 and 63).
constexpr uint32_t kSuffixFewRows = 64;
bool suffix_tc_applies(uint32_t head_dim, uint32_t rows_per_head) { return rows_per_head > kSuffixFewRows && kv_attn_tc_applies(head_dim, rows_per_head); }
// Parts of a prefix item that it adds to its rows by itself; more are joined by a launch in between, on all SMs: an item's rows
// are one SM's to read. us, with that launch and without: 4 sequences of 24 tokens on 3000 (5 parts) 53 and 72; 2 of 30 on 8000 (19)
// 52 and 102; 1 of 96 on 14696 (12) 47 and 66; none has it at 3 and fewer.
constexpr uint32_t kPartsInPlace = 3;
// The kernel for the number of query rows a key/value head.
template <SpanMode MODE>
cudaError_t launch_rule(AttnArgs p, bool f16, int sms, cudaStream_t s) {
    p.group_inv = group_inverse(p.group, p.b.max_q);
    if (MODE == kSuffix ? suffix_tc_applies(p.c.head_dim, p.b.max_q * p.group) : kv_attn_tc_applies(p.c.head_dim, p.b.max_q * p.group)) return launch_kv_attn_tc(p, f16, MODE, sms, s);
    return launch_kv_attn_few<MODE>(p, f16, sms, s);
}
int launched(cudaError_t e, std::string* err) {
    if (e == cudaSuccess) return W8A16_OK;
    cudaGetLastError();
    *err = std::string("cache attention launch failed: ") + cudaGetErrorString(e);
    return W8A16_ERR_LAUNCH;
}

}  // namespace

namespace {
uint64_t few_ws_bytes(uint32_t head_dim, int sms) {
    const uint32_t ctas = static_cast<uint32_t>(sms) * kMostCtasPerSm, dp = head_dim <= 64 ? 64u : head_dim <= 128 ? 128u : 256u;
    return 4 * boundary_floats(ctas) + 8ull * ctas * slot_floats(dp);
}
}  // namespace
uint64_t kv_attn_ws_bytes(uint32_t head_dim, uint32_t rows_per_head, int sms) {
    return kv_attn_tc_applies(head_dim, rows_per_head) ? kv_attn_tc_ws_bytes(head_dim, sms) : few_ws_bytes(head_dim, sms);
}

int launch_kv_attn(const w8a16_kv_cache_t& c, const w8a16_kv_batch_t& b, uint32_t act_dtype, const w8a16_heads_t& q,
                   const w8a16_heads_t& out, float softmax_scale, void* ws, int sms, uint64_t timeout_ns, cudaStream_t s,
                   std::string* err) {
    AttnArgs p{c, b, q, out, static_cast<float*>(ws), softmax_scale * 1.4426950408889634f, q.heads / c.kv_heads, 0, 0, 0, 0, timeout_ns, {}};
    while ((1u << p.page_shift) < c.page_size) ++p.page_shift;
    return launched(launch_rule<kFull>(p, act_dtype == W8A16_ACT_F16, sms, s), err);
}

namespace {
// Where the parts of a prefix call's workspace begin: the suffix pass's, the prefix pass's, the records of both, the suffix
// rows' parts and the number of CTAs that the prefix pass takes.
struct PrefixWs {
    uint64_t prefix, record, own, parts, taken, bytes;
};
PrefixWs prefix_ws(uint32_t head_dim, uint32_t rows_per_head, uint32_t tokens, uint32_t heads, uint32_t group, int sms) {
    const auto aligned = [](uint64_t n) { return (n + 255) / 256 * 256; };
    const uint32_t dp = head_dim <= 64 ? 64u : head_dim <= 128 ? 128u : 256u;
    PrefixWs w;
    const bool tc = suffix_tc_applies(head_dim, rows_per_head);
    w.prefix = aligned(tc ? kv_attn_tc_ws_bytes(head_dim, sms) : few_ws_bytes(head_dim, sms));
    w.record = w.prefix + aligned(kv_attn_ws_bytes(head_dim, tokens * group, sms));
    const uint64_t rows = static_cast<uint64_t>(tokens) * heads;
    w.own = w.record + aligned(4 * rows * (dp + 2));
    w.parts = w.own + (tc ? 0 : aligned(4 * rows * (dp + 2)));
    w.taken = w.parts + (tc ? 0 : aligned(16 * rows));
    w.bytes = w.taken + 16;
    return w;
}
}  // namespace

uint64_t kv_attn_span_ws_bytes(uint32_t head_dim, uint32_t rows_per_head, bool prefix, uint32_t tokens, uint32_t heads, uint32_t group, int sms) {
    return prefix ? prefix_ws(head_dim, rows_per_head, tokens, heads, group, sms).bytes : kv_attn_ws_bytes(head_dim, rows_per_head, sms);
}

int launch_kv_attn_span(const w8a16_kv_cache_t& c, const w8a16_kv_batch_t& b, uint32_t act_dtype, const w8a16_heads_t& q,
                        const w8a16_heads_t& out, const w8a16_kv_span_t& span, float softmax_scale, void* ws, int sms, uint64_t timeout_ns,
                        cudaStream_t s, std::string* err) {
    AttnArgs p{c, b, q, out, static_cast<float*>(ws), softmax_scale * 1.4426950408889634f, q.heads / c.kv_heads, 0, 0, 0, 0, timeout_ns, {}};
    while ((1u << p.page_shift) < c.page_size) ++p.page_shift;
    const bool f16 = act_dtype == W8A16_ACT_F16;
    if (!span.prefix_pages) {
        p.span.window = static_cast<int>(span.window), p.span.sinks = static_cast<int>(span.sinks);
        return launched(launch_rule<kWindow>(p, f16, sms, s), err);
    }
    const PrefixWs w = prefix_ws(c.head_dim, b.max_q * p.group, b.tokens, q.heads, p.group, sms);
    uint8_t* const base = static_cast<uint8_t*>(ws);
    p.span.lower = static_cast<int>(span.prefix_len);
    p.span.record = reinterpret_cast<float*>(base + w.record);
    p.span.rows = b;
    p.span.own = reinterpret_cast<float*>(base + w.own);
    p.span.parts = reinterpret_cast<uint4*>(base + w.parts);
    AttnArgs first = p;
    first.ws = reinterpret_cast<float*>(base + w.prefix);
    first.b.page_table = span.prefix_pages, first.b.page_table_stride = 0, first.b.max_pages = span.num_prefix_pages;
    first.b.cu_q = nullptr, first.b.batch = 1, first.b.max_q = b.tokens;
    p.span.pass = kv_attn_tc_applies(c.head_dim, b.tokens * p.group) ? kv_attn_tc_prefix_pass(first, sms) : kv_attn_few_prefix_pass(first, sms);
    // a suffix pass on the kernel for few rows runs beside it
    if (kv_attn_tc_applies(c.head_dim, b.tokens * p.group) && !suffix_tc_applies(c.head_dim, b.max_q * p.group))
        p.span.pass.taken = reinterpret_cast<uint32_t*>(base + w.taken);
    first.span.pass = p.span.pass;
    int rc = launched(launch_rule<kPrefix>(first, f16, sms, s), err);
    if (rc) return rc;
    const uint64_t items = static_cast<uint64_t>(p.span.pass.tiles) * c.kv_heads;
    if (suffix_tc_applies(c.head_dim, b.max_q * p.group) && p.span.pass.ctas > kPartsInPlace * items) {
        rc = launched(launch_kv_attn_prefix_parts(p, s), err);
        if (rc) return rc;
        p.span.pass.joined = true;
    }
    return launched(launch_rule<kSuffix>(p, f16, sms, s), err);
}

cudaError_t kv_attn_status_read(StatusWord* out, bool clear, cudaStream_t s) { return status_read(out, clear, s); }

}  // namespace w8a16

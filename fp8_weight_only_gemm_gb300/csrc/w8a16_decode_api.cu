// C entries of the decode-step operators around the GEMM: the paged 8-bit cache's
// append and attention, and the product with 4-bit weights. All checks run on the host before any device work;
// what only device memory tells (lengths, page numbers) the kernels check.
#include <cuda_runtime.h>

#include <new>
#include <string>

#include "w8a16_internal.h"

namespace {

using w8a16::api_fail;
using w8a16::api_ok;

std::string u(uint64_t v) { return std::to_string(v); }
bool misaligned(const void* p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// No C++ exception leaves a C entry: the messages allocate.
template <typename F>
int guarded(F&& f) noexcept {
    try {
        return f();
    } catch (...) {
        return W8A16_ERR_ARG;
    }
}

int check_act(const char* who, uint32_t act_dtype) {
    if (act_dtype != W8A16_ACT_BF16 && act_dtype != W8A16_ACT_F16)
        return api_fail(W8A16_ERR_ARG, std::string(who) + ": unknown activation type " + u(act_dtype));
    return W8A16_OK;
}

int check_cache(const char* who, const w8a16_kv_cache_t* c) {
    const std::string w(who);
    if (!c) return api_fail(W8A16_ERR_NULL, w + ": NULL cache");
    if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale)
        return api_fail(W8A16_ERR_NULL, w + ": NULL cache pointer");
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16)
        return api_fail(W8A16_ERR_ARG, w + ": head_dim=" + u(c->head_dim) + " must be a multiple of 16 in 16..256");
    if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
        return api_fail(W8A16_ERR_ARG, w + ": page_size=" + u(c->page_size) + " must be a power of two in 16..256");
    if (c->kv_heads < 1 || c->kv_heads > 65535)
        return api_fail(W8A16_ERR_ARG, w + ": kv_heads=" + u(c->kv_heads) + " must be in 1..65535");
    if (c->num_pages < 1 || c->num_pages > 0x7FFFFFFFu)
        return api_fail(W8A16_ERR_RANGE, w + ": num_pages=" + u(c->num_pages) + " must be in 1..2^31-1");
    if (misaligned(c->k_codes, 16) || misaligned(c->v_codes, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4))
        return api_fail(W8A16_ERR_ALIGN, w + ": cache codes need 16-byte alignment, scales 4");
    if (c->page_stride % 16 || c->head_stride % 16 || c->token_stride % 16)
        return api_fail(W8A16_ERR_ALIGN, w + ": cache strides must be multiples of 16 bytes");
    if (c->page_stride < 0 || c->head_stride < 0 || c->token_stride < 0 || c->token_stride > 1 << 22)
        return api_fail(W8A16_ERR_RANGE, w + ": cache strides must not be negative, token_stride at most 2^22 bytes");
    return W8A16_OK;
}

int check_batch(const char* who, const w8a16_kv_cache_t* c, const w8a16_kv_batch_t* b) {
    const std::string w(who);
    if (!b) return api_fail(W8A16_ERR_NULL, w + ": NULL batch");
    if (b->batch < 1 || b->tokens < 1 || b->max_q < 1)
        return api_fail(W8A16_ERR_M_ZERO, w + ": no sequences or tokens (batch=" + u(b->batch) + ", tokens=" + u(b->tokens) +
                                              ", max_q=" + u(b->max_q) + ")");
    if (!b->page_table || !b->lens) return api_fail(W8A16_ERR_NULL, w + ": NULL page_table or lens");
    if (misaligned(b->page_table, 4) || misaligned(b->lens, 4) || misaligned(b->cu_q, 4))
        return api_fail(W8A16_ERR_ALIGN, w + ": page_table, lens and cu_q need 4-byte alignment");
    if (b->batch > 0x7FFFFFFFu || b->tokens > 0x7FFFFFFFu || b->max_q > b->tokens)
        return api_fail(W8A16_ERR_RANGE, w + ": batch=" + u(b->batch) + ", tokens=" + u(b->tokens) +
                                             " must be below 2^31 and max_q=" + u(b->max_q) + " at most tokens");
    if (!b->cu_q && static_cast<uint64_t>(b->batch) * b->max_q != b->tokens)
        return api_fail(W8A16_ERR_ARG, w + ": without cu_q, tokens=" + u(b->tokens) + " must be batch=" + u(b->batch) +
                                           " times max_q=" + u(b->max_q));
    if (b->max_pages < 1 || static_cast<uint64_t>(b->max_pages) * c->page_size > 0x7FFFFF00ull)
        return api_fail(W8A16_ERR_RANGE, w + ": max_pages=" + u(b->max_pages) + " pages of " + u(c->page_size) +
                                             " must hold 1..2^31-256 tokens");
    return W8A16_OK;
}

int check_heads(const char* who, const char* name, const w8a16_heads_t* h, uint32_t heads) {
    const std::string w = std::string(who) + ": " + name;
    if (!h || !h->ptr) return api_fail(W8A16_ERR_NULL, w + " is NULL");
    if (heads ? h->heads != heads : h->heads < 1 || h->heads > 1u << 20)
        return api_fail(W8A16_ERR_ARG, w + " has " + u(h->heads) + " heads" + (heads ? ", not " + u(heads) : ""));
    if (misaligned(h->ptr, 16) || h->token_stride % 8 || h->head_stride % 8)
        return api_fail(W8A16_ERR_ALIGN, w + " needs 16-byte alignment and strides that are multiples of 8 elements");
    return W8A16_OK;
}

// Query rows that share a key/value head, which the kernels count in 31 bits; 0 with an error where there are more.
uint32_t rows_per_head(const char* who, uint32_t max_q, uint32_t heads, uint32_t kv_heads) {
    const uint64_t r = static_cast<uint64_t>(max_q) * (heads / kv_heads);
    if (r <= 0x7FFFFFFFu) return static_cast<uint32_t>(r);
    api_fail(W8A16_ERR_RANGE, std::string(who) + ": max_q=" + u(max_q) + " rows of " + u(heads / kv_heads) +
                                  " query heads a key/value head must be below 2^31 in all");
    return 0;
}

}  // namespace

extern "C" {

int w8a16_kv_append(const w8a16_kv_cache_t* cache, const w8a16_kv_batch_t* batch, uint32_t act_dtype,
                    const w8a16_heads_t* k, const w8a16_heads_t* v, const w8a16_heads_t* q, const w8a16_heads_t* q_out,
                    const w8a16_rope_t* rope, w8a16_stream_t stream) {
    return guarded([&] {
        const char* who = "w8a16_kv_append";
        int rc = check_cache(who, cache);
        if (!rc) rc = check_batch(who, cache, batch);
        if (!rc) rc = check_act(who, act_dtype);
        if (!rc) rc = check_heads(who, "k", k, cache->kv_heads);
        if (!rc) rc = check_heads(who, "v", v, cache->kv_heads);
        if (rc) return rc;
        w8a16_heads_t qi{}, qo{};
        if (q && q->ptr) {
            rc = check_heads(who, "q", q, 0);
            if (!rc) rc = check_heads(who, "q_out", q_out, q->heads);
            if (rc) return rc;
            qi = *q;
            qo = *q_out;
        } else if (q_out && q_out->ptr) {
            return api_fail(W8A16_ERR_NULL, std::string(who) + ": q_out without q");
        }
        if (!rope) return api_fail(W8A16_ERR_NULL, std::string(who) + ": NULL rope");
        if (rope->rotary_dim % 16 || rope->rotary_dim > cache->head_dim)
            return api_fail(W8A16_ERR_ARG, std::string(who) + ": rotary_dim=" + u(rope->rotary_dim) +
                                               " must be a multiple of 16, at most head_dim=" + u(cache->head_dim));
        if (rope->rotary_dim) {
            if (!rope->cos || !rope->sin) return api_fail(W8A16_ERR_NULL, std::string(who) + ": NULL cos or sin");
            if (misaligned(rope->cos, 16) || misaligned(rope->sin, 16))
                return api_fail(W8A16_ERR_ALIGN, std::string(who) + ": cos and sin need 16-byte alignment");
            if (rope->rows < 1 || rope->rows > 0x7FFFFFFFu)
                return api_fail(W8A16_ERR_RANGE, std::string(who) + ": rope rows=" + u(rope->rows) + " must be in 1..2^31-1");
        }
        int sms = 0;
        rc = w8a16::api_device(&sms);
        if (rc) return rc;
        std::string err;
        rc = w8a16::launch_kv_append(*cache, *batch, act_dtype, *k, *v, qi, qo, *rope,
                                     reinterpret_cast<cudaStream_t>(stream), &err);
        return rc ? api_fail(rc, err) : api_ok();
    });
}

uint64_t w8a16_kv_attention_workspace_bytes(const w8a16_kv_cache_t* cache, uint32_t batch, uint32_t max_q, uint32_t heads) {
    uint64_t bytes = 0;
    guarded([&] {
        const char* who = "w8a16_kv_attention_workspace_bytes";
        int rc = check_cache(who, cache);
        if (!rc && (batch < 1 || max_q < 1 || heads < 1 || heads % cache->kv_heads))
            rc = api_fail(W8A16_ERR_ARG, std::string(who) + ": batch, max_q and heads must be positive, heads=" + u(heads) +
                                             " a multiple of kv_heads=" + u(cache->kv_heads));
        int sms = 0;
        if (rc) return rc;
        const uint32_t rows = rows_per_head(who, max_q, heads, cache->kv_heads);
        if (rows == 0) return static_cast<int>(W8A16_ERR_RANGE);
        rc = w8a16::api_device(&sms);
        if (rc) return rc;
        bytes = w8a16::kv_attn_ws_bytes(cache->head_dim, rows, sms);
        return api_ok();
    });
    return bytes;
}

int w8a16_kv_attention(const w8a16_kv_cache_t* cache, const w8a16_kv_batch_t* batch, uint32_t act_dtype,
                       const w8a16_heads_t* q, const w8a16_heads_t* out, float softmax_scale, void* workspace,
                       uint64_t workspace_bytes, w8a16_stream_t stream) {
    return guarded([&] {
        const char* who = "w8a16_kv_attention";
        int rc = check_cache(who, cache);
        if (!rc) rc = check_batch(who, cache, batch);
        if (!rc) rc = check_act(who, act_dtype);
        if (!rc) rc = check_heads(who, "q", q, 0);
        if (!rc) rc = check_heads(who, "out", out, q->heads);
        if (rc) return rc;
        if (q->heads % cache->kv_heads)
            return api_fail(W8A16_ERR_ARG, std::string(who) + ": " + u(q->heads) + " query heads do not divide among " +
                                               u(cache->kv_heads) + " key/value heads");
        if (!(softmax_scale > 0.f) || softmax_scale > 1e30f)
            return api_fail(W8A16_ERR_ARG, std::string(who) + ": softmax_scale must be positive and finite");
        const uint32_t rows = rows_per_head(who, batch->max_q, q->heads, cache->kv_heads);
        if (rows == 0) return static_cast<int>(W8A16_ERR_RANGE);
        int sms = 0;
        rc = w8a16::api_device(&sms);
        if (rc) return rc;
        const uint64_t need = w8a16::kv_attn_ws_bytes(cache->head_dim, rows, sms);
        if (!workspace || workspace_bytes < need)
            return api_fail(W8A16_ERR_ARG, std::string(who) + ": needs a workspace of " + u(need) + " bytes, got " +
                                               u(workspace ? workspace_bytes : 0));
        if (misaligned(workspace, 16)) return api_fail(W8A16_ERR_ALIGN, std::string(who) + ": the workspace must be 16-byte aligned");
        std::string err;
        uint64_t timeout_ns = 0;
        rc = w8a16::api_timeout(&timeout_ns);
        if (rc) return rc;
        rc = w8a16::launch_kv_attn(*cache, *batch, act_dtype, *q, *out, softmax_scale, workspace, sms, timeout_ns,
                                   reinterpret_cast<cudaStream_t>(stream), &err);
        return rc ? api_fail(rc, err) : api_ok();
    });
}

int w8a16_gemm_w4(const void* A, uint32_t a_row_stride, uint32_t act_dtype, const void* W, const void* scale,
                  uint32_t scale_dtype, const void* zeros, uint32_t group, void* C, uint32_t c_row_stride, uint32_t M,
                  uint32_t N, uint32_t K, uint32_t flags, w8a16_stream_t stream) {
    return guarded([&] {
        const std::string who("w8a16_gemm_w4");
        if (flags & ~static_cast<uint32_t>(W8A16_FLAG_PDL)) return api_fail(W8A16_ERR_ARG, who + ": unknown flag bits " + u(flags));
        if (M < 1) return api_fail(W8A16_ERR_M_ZERO, who + ": m=0 has no rows to compute");
        if (group != 32 && group != 64 && group != 128)
            return api_fail(W8A16_ERR_ARG, who + ": group=" + u(group) + " must be 32, 64 or 128");
        if (K < group || K % group)
            return api_fail(W8A16_ERR_K_BLOCK, who + ": K=" + u(K) + " must be a positive multiple of group=" + u(group));
        if (a_row_stride < K || c_row_stride < N)
            return api_fail(W8A16_ERR_PITCH, who + ": row pitches (a=" + u(a_row_stride) + ", c=" + u(c_row_stride) +
                                                 ") must cover k=" + u(K) + " and n=" + u(N));
        if (a_row_stride % 8)
            return api_fail(W8A16_ERR_A_PITCH_ALIGN, who + ": a_row_stride=" + u(a_row_stride) + " must be a multiple of 8");
        if (N < 1) return api_fail(W8A16_ERR_N_ZERO, who + ": n=0 has no columns to compute");
        if (M > 65535u * 32u || N > 0x7FFFFFFFu / 8 || K > 0x7FFFFFFFu)
            return api_fail(W8A16_ERR_RANGE, who + ": M=" + u(M) + ", N=" + u(N) + " or K=" + u(K) + " is out of range");
        int rc = check_act(who.c_str(), act_dtype);
        if (rc) return rc;
        if (scale_dtype != W8A16_W4_SCALE_F32 && scale_dtype != W8A16_W4_SCALE_ACT)
            return api_fail(W8A16_ERR_ARG, who + ": unknown scale type " + u(scale_dtype));
        if (!A || !W || !scale || !C) return api_fail(W8A16_ERR_NULL, who + ": NULL operand pointer");
        if (misaligned(A, 16) || misaligned(W, 16) || misaligned(scale, 4) || misaligned(zeros, 4) || misaligned(C, 2))
            return api_fail(W8A16_ERR_ALIGN, who + ": alignment (A and W need 16 bytes, scale and zeros 4, C 2)");
        int sms = 0;
        rc = w8a16::api_device(&sms);
        if (rc) return rc;
        uint64_t timeout_ns = 0;
        rc = w8a16::api_timeout(&timeout_ns);
        if (rc) return rc;
        std::string err;
        rc = w8a16::launch_w4({A, W, scale, zeros, C, a_row_stride, c_row_stride, M, N, K, group, act_dtype,
                               scale_dtype == W8A16_W4_SCALE_F32},
                              sms, timeout_ns, flags, reinterpret_cast<cudaStream_t>(stream), &err);
        return rc ? api_fail(rc, err) : api_ok();
    });
}

}  // extern "C"

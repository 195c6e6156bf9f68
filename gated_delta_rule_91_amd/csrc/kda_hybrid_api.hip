// kda_hybrid_api.hip -- the C ABI of the operators beside KDA (declared in
// include/kda_hybrid.h).  As in kda_api.hip every entry point validates its
// arguments synchronously, before any launch, and launches on the caller's
// stream; nothing here allocates or keeps state.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "kda_checks.hpp"
#include "kda_hybrid.h"
#include "kda_hybrid_internal.hpp"

using namespace kda;

namespace {

// log2 of a page size, or -1 where it is none
int page_shift(int32_t page_size) {
    for (int s = 4; s <= 8; ++s)
        if (page_size == (1 << s)) return s;
    return -1;
}

constexpr float kLog2e = 1.4426950408889634f;

bool ok_io(kda_dtype t) { return t == KDA_F32 || t == KDA_BF16; }

// a * b, or INT64_MAX where that does not fit (a, b >= 0)
int64_t mul_sat(int64_t a, int64_t b) {
    int64_t r;
    return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}

kda_status check_cache(const kda_cache4* c) {
    if (!c || c->pages < 0 || c->heads <= 0 || page_shift(c->page_size) < 0 || c->d <= 0)
        return KDA_ERR_INVALID_ARGUMENT;
    if (c->d != 64 && c->d != 128) return KDA_ERR_UNSUPPORTED;
    // element offsets are 64-bit; a token slot and a (page, head) index have to fit too
    if (mul_sat(mul_sat(c->pages, c->heads), (int64_t)c->page_size * c->d) > ((int64_t)1 << 50))
        return KDA_ERR_UNSUPPORTED;
    const bool any = c->pages > 0;
    if (!ok_ptr(c->k, any) || !ok_ptr(c->k_scale, any) || !ok_ptr(c->v, any) || !ok_ptr(c->v_scale, any))
        return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

Cache4Args cache_args(const kda_cache4* c) {
    Cache4Args a = {};
    a.pages = c->pages; a.page_shift = page_shift(c->page_size); a.heads = c->heads;
    a.k = static_cast<uint8_t*>(c->k); a.k_scale = static_cast<uint8_t*>(c->k_scale);
    a.v = static_cast<uint8_t*>(c->v); a.v_scale = static_cast<uint8_t*>(c->v_scale);
    return a;
}

// append and read share their checks
kda_status check_rows(const kda_cache4* c, int64_t tokens, kda_dtype io, const void* k, const void* v,
                      const int64_t* slot_map) {
    kda_status st = check_cache(c);
    if (st != KDA_OK) return st;
    if (tokens < 0 || !ok_io(io)) return KDA_ERR_INVALID_ARGUMENT;
    // rows are 32-bit in the kernels, and so are the threads of a launch: d / 8 a row, whole workgroups
    if (tokens > INT32_MAX || mul_sat(mul_sat(tokens + 31, c->heads), c->d / 8) > UINT32_MAX) return KDA_ERR_UNSUPPORTED;
    const bool any = tokens > 0;
    if (!ok_ptr(k, any) || !ok_ptr(v, any) || !ok_elem(slot_map, any, 8)) return KDA_ERR_INVALID_ARGUMENT;
    return KDA_OK;
}

kda_status check_attention(const kda_cache4* c, const kda_cache4_attention_problem* p) {
    kda_status st = check_cache(c);
    if (st != KDA_OK) return st;
    if (!p || p->n_seq < 0 || p->tokens < 0 || p->heads <= 0 || p->max_pages < 0 || p->max_q < 1 || p->max_len < 0 ||
        !ok_io(p->io_dtype) || !isfinite(p->scale) || p->heads % c->heads != 0)
        return KDA_ERR_INVALID_ARGUMENT;
    // row tiles, (row, head) pairs and positions are 32-bit in the kernels, which step
    // through the positions in tiles of up to 128 tokens and look one tile ahead
    if (p->n_seq > (1 << 24) || mul_sat(p->tokens, p->heads) > (1 << 30) ||
        mul_sat(p->n_seq, p->heads) > (1 << 30) || mul_sat(p->max_pages, c->page_size) > INT32_MAX - 256)
        return KDA_ERR_UNSUPPORTED;
    // the kernels multiply scores by scale * log2(e), which has to be a normal number or 0
    const float factor = fabsf(p->scale) * kLog2e;
    if (p->scale != 0.0f && !(factor >= FLT_MIN && factor <= FLT_MAX)) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

Cache4AttentionArgs attention_args(const kda_cache4* c, const kda_cache4_attention_problem* p) {
    Cache4AttentionArgs a = {};
    a.c = cache_args(c);
    a.n_seq = p->n_seq; a.tokens = p->tokens; a.heads = p->heads; a.group = p->heads / c->heads;
    a.max_pages = c->pages > 0 ? p->max_pages : 0;   // a cache without pages counts no tokens
    a.max_q = p->max_q; a.max_len = p->max_len;
    a.to_log2 = p->scale == 0.0f ? 1.0f : fabsf(p->scale) * kLog2e;
    a.sign = p->scale < 0.0f ? -1.0f : (p->scale == 0.0f ? 0.0f : 1.0f);
    return a;
}

bool no_rows(const kda_cache4_attention_problem* p) { return p->n_seq == 0 || p->tokens == 0; }
bool fits(const kda_cache4* c, const kda_cache4_attention_problem* p) {
    return no_rows(p) || cache4_attention_fits(p->io_dtype == KDA_BF16, c->d, attention_args(c, p));
}

kda_status check_recurrence(const kda_recurrence_problem* p) {
    if (!p || p->batch < 0 || p->seqlen < 0 || p->width <= 0 || p->n_seq < -1 || !ok_io(p->io_dtype))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!(p->log_alpha_min < 0.0f)) return KDA_ERR_INVALID_ARGUMENT;
    const bool packed = p->n_seq >= 0;
    if (packed && p->batch != 1) return KDA_ERR_INVALID_ARGUMENT;
    // token indices are 32-bit, and so are the threads of a launch; elements are 64-bit
    if (p->seqlen > (1 << 30) || p->width > (1 << 30) || p->batch > (1 << 24) || p->n_seq > (1 << 24) ||
        mul_sat(mul_sat(p->batch, p->seqlen), p->width) > ((int64_t)1 << 40) ||
        mul_sat(packed ? p->n_seq : p->batch, p->width) > ((int64_t)1 << 38) ||
        // threads of a launch: 1024 for 128 tokens x 128 channels
        mul_sat(mul_sat(p->batch, (p->seqlen + 127) / 128), (p->width + 127) / 128) > UINT32_MAX / 1024)
        return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

bool packed(const kda_recurrence_problem* p) { return p->n_seq >= 0; }
int64_t sequences(const kda_recurrence_problem* p) { return packed(p) ? p->n_seq : p->batch; }
bool any_tokens(const kda_recurrence_problem* p) { return p->batch > 0 && p->seqlen > 0; }

bool ok_offsets(const kda_recurrence_problem* p, const int32_t* cu) {
    return packed(p) ? ok_elem(cu, true, 4) : cu == nullptr;
}

RecurrenceArgs recurrence_args(const kda_recurrence_problem* p, const void* x, const float* log_alpha, const void* g,
                               const float* state_in, const int32_t* cu, void* workspace) {
    RecurrenceArgs a = {};
    a.B = p->batch; a.T = p->seqlen; a.D = p->width; a.n_seq = sequences(p); a.cu_seqlens = cu;
    a.floor_ = p->log_alpha_min;
    a.x = x; a.log_alpha = log_alpha; a.g = g; a.state_in = state_in;
    a.ws = static_cast<char*>(workspace);
    return a;
}

kda_status recurrence_forward(const kda_recurrence_problem* p, const void* x, const float* log_alpha, const void* g,
                              const float* state_in, const int32_t* cu, void* out, float* state_out, void* workspace,
                              size_t workspace_bytes, bool keep, void* stream) {
    kda_status st = check_recurrence(p);
    if (st != KDA_OK) return st;
    const bool any = any_tokens(p);
    const size_t need = recurrence_workspace_bytes(p->batch, p->seqlen, p->width, keep);
    if (!ok_ptr(x, any) || !ok_ptr(log_alpha, any) || !ok_opt_ptr(g) || !ok_opt_ptr(state_in) || !ok_offsets(p, cu) ||
        !ok_ptr(out, any) || !ok_opt_ptr(state_out) || !ok_ptr(workspace, need > 0))
        return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (sequences(p) == 0 || (!any && !state_out)) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    RecurrenceArgs a = recurrence_args(p, x, log_alpha, g, state_in, cu, workspace);
    a.out = out; a.state_out = state_out; a.keep = keep;
    return hip_status(launch_recurrence(p->io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

}  // namespace

extern "C" {

kda_status kda_plan_requests(int64_t n_req, int64_t tokens, int32_t page_size, int32_t max_pages,
                             const int32_t* past_lens, const int32_t* new_lens, int32_t* block_table, int64_t n_free,
                             const int32_t* free_pages, int32_t* cu_seqlens, int32_t* total_lens, int64_t* slot_map,
                             int32_t* pages_taken, void* stream) {
    const int shift = page_shift(page_size);
    if (n_req < 0 || tokens < 0 || shift < 0 || max_pages < 0 || n_free < 0) return KDA_ERR_INVALID_ARGUMENT;
    if (n_req > kPlanMaxRequests || tokens > INT32_MAX || n_free > INT32_MAX || mul_sat(n_req, max_pages) > INT32_MAX)
        return KDA_ERR_UNSUPPORTED;
    const bool any = n_req > 0;
    if (!ok_elem(past_lens, any, 4) || !ok_elem(new_lens, any, 4) || !ok_elem(block_table, any && max_pages > 0, 4) ||
        !ok_elem(free_pages, n_free > 0, 4) || !ok_elem(cu_seqlens, true, 4) || !ok_elem(total_lens, any, 4) ||
        !ok_elem(slot_map, tokens > 0, 8) || !ok_elem(pages_taken, true, 4))
        return KDA_ERR_INVALID_ARGUMENT;
    const kda_status st = device_ready();
    if (st != KDA_OK) return st;
    PlanArgs a = {};
    a.n_req = (int)n_req; a.tokens = tokens; a.page_shift = shift; a.max_pages = max_pages;
    a.past_lens = past_lens; a.new_lens = new_lens; a.block_table = block_table; a.n_free = n_free;
    a.free_pages = free_pages; a.cu_seqlens = cu_seqlens; a.total_lens = total_lens; a.slot_map = slot_map;
    a.pages_taken = pages_taken;
    return hip_status(launch_plan(a, (hipStream_t)stream));
}

kda_status kda_cache4_append(const kda_cache4* c, int64_t tokens, kda_dtype io_dtype, const void* k, const void* v,
                             const int64_t* slot_map, void* stream) {
    kda_status st = check_rows(c, tokens, io_dtype, k, v, slot_map);
    if (st != KDA_OK) return st;
    if (tokens == 0 || c->pages == 0) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    Cache4RowsArgs a = {};
    a.c = cache_args(c); a.tokens = tokens; a.slot_map = slot_map; a.k_in = k; a.v_in = v;
    return hip_status(launch_cache4_append(io_dtype == KDA_BF16, c->d, a, (hipStream_t)stream));
}

kda_status kda_cache4_read(const kda_cache4* c, int64_t tokens, kda_dtype io_dtype, const int64_t* slot_map, void* k,
                           void* v, void* stream) {
    kda_status st = check_rows(c, tokens, io_dtype, k, v, slot_map);
    if (st != KDA_OK) return st;
    if (tokens == 0) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    Cache4RowsArgs a = {};
    a.c = cache_args(c); a.tokens = tokens; a.slot_map = slot_map; a.k_out = k; a.v_out = v;
    return hip_status(launch_cache4_read(io_dtype == KDA_BF16, c->d, a, (hipStream_t)stream));
}

size_t kda_cache4_attention_workspace_size(const kda_cache4* c, const kda_cache4_attention_problem* p) {
    if (check_attention(c, p) != KDA_OK || no_rows(p) || !fits(c, p)) return 0;
    return cache4_attention_workspace_bytes(p->io_dtype == KDA_BF16, c->d, attention_args(c, p));
}

kda_status kda_cache4_attention(const kda_cache4* c, const kda_cache4_attention_problem* p, const void* q,
                                const int32_t* block_table, const int32_t* total_lens, const int32_t* cu_seqlens,
                                const void* g, void* out, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st = check_attention(c, p);
    if (st != KDA_OK) return st;
    if (!cu_seqlens && p->tokens != p->n_seq) return KDA_ERR_INVALID_ARGUMENT;
    if (!fits(c, p)) return KDA_ERR_UNSUPPORTED;
    if (no_rows(p)) return KDA_OK;
    const size_t need = kda_cache4_attention_workspace_size(c, p);
    if (!ok_ptr(q, true) || !ok_elem(block_table, p->max_pages > 0, 4) || !ok_elem(total_lens, true, 4) ||
        (cu_seqlens && !ok_elem(cu_seqlens, true, 4)) || !ok_opt_ptr(g) || !ok_ptr(out, true) ||
        !ok_ptr(workspace, need > 0))
        return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (out == q) return KDA_ERR_INVALID_ARGUMENT;       // several workgroups read a row of q
    if ((st = device_ready()) != KDA_OK) return st;
    Cache4AttentionArgs a = attention_args(c, p);
    a.q = q; a.g = g; a.out = out; a.block_table = block_table; a.total_lens = total_lens; a.cu_seqlens = cu_seqlens;
    return hip_status(launch_cache4_attention(p->io_dtype == KDA_BF16, c->d, a, static_cast<char*>(workspace),
                                              (hipStream_t)stream));
}

size_t kda_recurrence_workspace_size(const kda_recurrence_problem* p) {
    if (check_recurrence(p) != KDA_OK) return 0;
    return recurrence_workspace_bytes(p->batch, p->seqlen, p->width, false);
}

size_t kda_recurrence_backward_workspace_size(const kda_recurrence_problem* p) {
    if (check_recurrence(p) != KDA_OK) return 0;
    return recurrence_workspace_bytes(p->batch, p->seqlen, p->width, true);
}

kda_status kda_recurrence_prefill(const kda_recurrence_problem* p, const void* x, const float* log_alpha,
                                  const void* g, const float* state_in, const int32_t* cu_seqlens, void* out,
                                  float* state_out, void* workspace, size_t workspace_bytes, void* stream) {
    return recurrence_forward(p, x, log_alpha, g, state_in, cu_seqlens, out, state_out, workspace, workspace_bytes,
                              false, stream);
}

kda_status kda_recurrence_prefill_for_backward(const kda_recurrence_problem* p, const void* x,
                                               const float* log_alpha, const void* g, const float* state_in,
                                               const int32_t* cu_seqlens, void* out, float* state_out,
                                               void* workspace, size_t workspace_bytes, void* stream) {
    return recurrence_forward(p, x, log_alpha, g, state_in, cu_seqlens, out, state_out, workspace, workspace_bytes,
                              true, stream);
}

kda_status kda_recurrence_backward(const kda_recurrence_problem* p, const void* x, const float* log_alpha,
                                   const void* g, const float* state_in, const int32_t* cu_seqlens,
                                   const void* d_out, const float* d_state, void* dx, float* dlog_alpha, void* dg,
                                   float* d_state_in, void* workspace, size_t workspace_bytes, void* stream) {
    kda_status st = check_recurrence(p);
    if (st != KDA_OK) return st;
    const bool any = any_tokens(p);
    const size_t need = recurrence_workspace_bytes(p->batch, p->seqlen, p->width, true);
    if (!ok_ptr(x, any) || !ok_ptr(log_alpha, any) || !ok_opt_ptr(g) || !ok_opt_ptr(state_in) ||
        !ok_offsets(p, cu_seqlens) || !ok_opt_ptr(d_out) || !ok_opt_ptr(d_state) || !ok_ptr(dx, any) ||
        !ok_ptr(dlog_alpha, any) || !ok_ptr(dg, any && g != nullptr) || !ok_opt_ptr(d_state_in) ||
        !ok_ptr(workspace, need > 0))
        return KDA_ERR_INVALID_ARGUMENT;
    if (workspace_bytes < need) return KDA_ERR_WORKSPACE_TOO_SMALL;
    if (sequences(p) == 0 || (!any && !d_state_in)) return KDA_OK;
    if ((st = device_ready()) != KDA_OK) return st;
    RecurrenceArgs a = recurrence_args(p, x, log_alpha, g, state_in, cu_seqlens, workspace);
    a.d_out = d_out; a.d_state = d_state; a.dx = dx; a.dlog_alpha = dlog_alpha; a.dg = dg; a.d_state_in = d_state_in;
    return hip_status(launch_recurrence_backward(p->io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

kda_status kda_recurrence_step(int64_t N, int64_t width, kda_dtype io_dtype, float log_alpha_min, const void* x,
                               const float* log_alpha, const void* g, float* state, void* out, void* stream) {
    if (N < 0 || width <= 0 || !ok_io(io_dtype) || !(log_alpha_min < 0.0f)) return KDA_ERR_INVALID_ARGUMENT;
    if (mul_sat(N, width) > ((int64_t)1 << 33)) return KDA_ERR_UNSUPPORTED;      // threads of a launch, four elements each
    const bool any = N > 0;
    if (!ok_ptr(x, any) || !ok_ptr(log_alpha, any) || !ok_opt_ptr(g) || !ok_ptr(state, any) || !ok_ptr(out, any))
        return KDA_ERR_INVALID_ARGUMENT;
    if (!any) return KDA_OK;
    const kda_status st = device_ready();
    if (st != KDA_OK) return st;
    RecurrenceStepArgs a = {};
    a.n = N * width; a.floor_ = log_alpha_min; a.x = x; a.log_alpha = log_alpha; a.g = g; a.state = state; a.out = out;
    return hip_status(launch_recurrence_step(io_dtype == KDA_BF16, a, (hipStream_t)stream));
}

}  // extern "C"

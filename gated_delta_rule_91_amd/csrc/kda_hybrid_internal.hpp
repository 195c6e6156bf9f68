// kda_hybrid_internal.hpp -- host-side launch entry points of the operators
// beside KDA (plan, 4-bit cache, attention over it, recurrence).  Arguments
// were validated by kda_hybrid_api.hip before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int64_t kPlanMaxRequests = 8192;   // both prefix sums of a plan lie in LDS

struct PlanArgs {
    int n_req;
    int64_t tokens;
    int page_shift;          // log2(page_size)
    int max_pages;
    const int32_t* past_lens;
    const int32_t* new_lens;
    int32_t* block_table;
    int64_t n_free;
    const int32_t* free_pages;
    int32_t* cu_seqlens;
    int32_t* total_lens;
    int64_t* slot_map;
    int32_t* pages_taken;
};

struct Cache4Args {
    int64_t pages;
    int page_shift;
    int heads;
    uint8_t* k;
    uint8_t* k_scale;
    uint8_t* v;
    uint8_t* v_scale;
};

struct Cache4RowsArgs {      // append (k, v read) and read (k, v written)
    Cache4Args c;
    int64_t tokens;
    const int64_t* slot_map;
    const void* k_in;
    const void* v_in;
    void* k_out;
    void* v_out;
};

struct Cache4AttentionArgs {
    Cache4Args c;
    int64_t n_seq, tokens;
    int heads, group;        // query heads, and how many of them share a key/value head
    int max_pages;
    int64_t max_q, max_len;
    const void* q;
    const void* g;           // or null
    void* out;
    const int32_t* block_table;
    const int32_t* total_lens;
    const int32_t* cu_seqlens;   // or null: one query a sequence
    // Scores are formed in powers of two, with the sign of the scale in the
    // queries, so that the largest product is the largest score.  to_log2 is not
    // 0, which would make NaN of a masked score's -inf: a scale of 0 is in the
    // queries too.  (Formed in the kernel, they cost the prompts' form registers
    // that it spills.)
    float to_log2, sign;
};

struct RecurrenceArgs {
    int64_t B, T, D;
    int64_t n_seq;               // sequences of a packed batch; with cu_seqlens
    const int32_t* cu_seqlens;   // or null (uniform rows)
    float floor_;
    const void* x;
    const float* log_alpha;
    const void* g;               // or null
    const float* state_in;       // or null
    void* out;
    float* state_out;            // or null
    const void* d_out;           // or null
    const float* d_state;        // or null
    void* dx;
    float* dlog_alpha;
    void* dg;                    // with g
    float* d_state_in;           // or null
    bool keep;                   // forward: leave the state entering every tile in ws
    char* ws;
};

struct RecurrenceStepArgs {
    int64_t n;                   // sequences x channels
    float floor_;
    const void* x;
    const float* log_alpha;
    const void* g;               // or null
    float* state;
    void* out;
};

hipError_t launch_plan(const PlanArgs& a, hipStream_t s);
hipError_t launch_cache4_append(bool bf16, int d, const Cache4RowsArgs& a, hipStream_t s);
hipError_t launch_cache4_read(bool bf16, int d, const Cache4RowsArgs& a, hipStream_t s);
// Whether a launch can have as many threads as the problem takes.
bool cache4_attention_fits(bool bf16, int d, const Cache4AttentionArgs& a);
size_t cache4_attention_workspace_bytes(bool bf16, int d, const Cache4AttentionArgs& a);
hipError_t launch_cache4_attention(bool bf16, int d, const Cache4AttentionArgs& a, char* ws, hipStream_t s);
// backward: the workspace of the training pair; else of the prefill alone
size_t recurrence_workspace_bytes(int64_t B, int64_t T, int64_t D, bool backward);
hipError_t launch_recurrence(bool bf16, const RecurrenceArgs& a, hipStream_t s);
hipError_t launch_recurrence_backward(bool bf16, const RecurrenceArgs& a, hipStream_t s);
hipError_t launch_recurrence_step(bool bf16, const RecurrenceStepArgs& a, hipStream_t s);

}  // namespace kda

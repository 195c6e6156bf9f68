// kda_cache4_attention.hip -- causal grouped-query attention over the paged
// 4-bit cache, each sequence by itself.  The kernels, what bounds them and what
// they measured are in kda_cache4_attention.hpp.
#include "kda_cache4_attention.hpp"

namespace kda {

bool cache4_attention_fits(bool bf16, int d, const Cache4AttentionArgs& a) { return attention_fits(bf16, d, a); }

size_t cache4_attention_workspace_bytes(bool bf16, int d, const Cache4AttentionArgs& a) {
    return attention_workspace_bytes(bf16, d, a);
}

hipError_t launch_cache4_attention(bool bf16, int d, const Cache4AttentionArgs& a, char* ws, hipStream_t s) {
    return launch_attention<WHOLE>(bf16, d, a, ws, s);
}

}  // namespace kda

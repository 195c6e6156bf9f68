// kda_cache4_shared.hip -- causal grouped-query attention over the paged 4-bit
// cache for groups of sequences that share their first tokens, which are read and
// converted once for all rows of a group.
//
//   out = (w0 O0 + w1 O1) / (w0 S0 + w1 S1),  w_i = e^(m_i - max(m_0, m_1))
// with maximum m, sum S and weighted values O of a row over the prefix (0) and
// over its own tokens (1).  The prefix is a launch in which a group is one
// sequence with all its rows, which see all of it; the rest a launch in which
// every sequence begins at the end of its prefix.  Both are the kernels of
// kda_cache4_attention.hpp, each in the form that its rows call for.
#include "kda_cache4_attention.hpp"

namespace kda {

namespace {

// What the two launches go by.  All of it lies in the workspace.
struct Groups {
    int32_t* cu;         // [n_groups + 1]: the groups' rows of q
    int32_t* prefix;     // [n_groups]: tokens that all rows of a group see
    int32_t* tables;     // [n_groups]: the first sequence of each
    int32_t* starts;     // [n_seq]: the prefix of each sequence's group
};

// A workgroup has a group, the last one the sequences of none.  The prefix ends
// where the first query of a group's sequences stands at the latest, so that
// no row needs a mask there; a group of one has none.
__global__ __launch_bounds__(256) void kda_cache4_groups_kernel(Cache4SharedArgs args, Groups out) {
    __shared__ int least[4];
    const Cache4AttentionArgs& a = args.a;
    const int n = (int)a.n_seq, G = (int)args.n_groups, j = blockIdx.x, t = threadIdx.x;
    auto bound = [&](int x) { return min(max(x, 0), n); };
    auto row_of = [&](int s) { return a.cu_seqlens ? min(max(a.cu_seqlens[s], 0), (int)a.tokens) : s; };
    if (j == G) {
        const int first = bound(args.group_offsets[0]), last = bound(args.group_offsets[G]);
        for (int s = t; s < first; s += 256) out.starts[s] = 0;
        for (int s = last + t; s < n; s += 256) out.starts[s] = 0;
        return;
    }
    const int s0 = bound(args.group_offsets[j]), s1 = max(bound(args.group_offsets[j + 1]), s0);
    int seen = INT32_MAX;                // tokens before the first query, of the sequence that has the fewest
    for (int s = s0 + t; s < s1; s += 256) {
        int64_t r0 = s, r1 = s + 1;
        if (a.cu_seqlens) seq_bounds(a.cu_seqlens, s, a.tokens, r0, r1);
        if (r1 > r0) seen = min(seen, max(max(a.total_lens[s], 0) - (int)(r1 - r0), 0));
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) seen = min(seen, __shfl_xor(seen, off));
    if ((t & 63) == 0) least[t >> 6] = seen;
    __syncthreads();
    seen = min(min(least[0], least[1]), min(least[2], least[3]));
    int p = min(max(args.prefix_lens[j], 0), min(seen, a.max_pages << a.c.page_shift));
    if (s1 - s0 < 2 || seen == INT32_MAX) p = 0;
    for (int s = s0 + t; s < s1; s += 256) out.starts[s] = p;
    if (t == 0) {
        out.cu[j] = row_of(s0);
        if (j == G - 1) out.cu[G] = row_of(s1);
        out.prefix[j] = p;
        out.tables[j] = min(s0, n - 1);
    }
}

// The launch over the prefixes: a group is one sequence.
PartArgs prefix_args(const Cache4SharedArgs& s, const Groups& g) {
    PartArgs a = {};
    static_cast<Cache4AttentionArgs&>(a) = s.a;
    a.n_seq = s.n_groups;
    a.max_len = s.max_prefix;
    // groups are ragged: about twice the rows of an even share
    const int64_t even = 2 * ((a.tokens + s.n_groups - 1) / s.n_groups);
    a.max_q = even < a.tokens ? even : a.tokens;
    a.g = nullptr;
    a.cu_seqlens = g.cu;
    a.total_lens = g.prefix;
    a.table_rows = g.tables;
    a.tables = (int)s.a.n_seq;
    return a;
}

struct SharedLayout {
    Groups g;
    float* row_o;
    float* row_sums;
    char* parts;         // of one launch after the other
    size_t bytes;
};

SharedLayout lay_out(bool bf16, int d, const Cache4SharedArgs& s, char* ws) {
    SharedLayout l = {};
    size_t used = 0;
    auto take = [&](size_t bytes) {
        char* r = ws ? ws + used : nullptr;
        used += round256(bytes);
        return r;
    };
    const size_t rows = (size_t)s.a.tokens * s.a.heads;
    l.g.cu = reinterpret_cast<int32_t*>(take((s.n_groups + 1) * sizeof(int32_t)));
    l.g.prefix = reinterpret_cast<int32_t*>(take(s.n_groups * sizeof(int32_t)));
    l.g.tables = reinterpret_cast<int32_t*>(take(s.n_groups * sizeof(int32_t)));
    l.g.starts = reinterpret_cast<int32_t*>(take(s.a.n_seq * sizeof(int32_t)));
    l.row_sums = reinterpret_cast<float*>(take(rows * 2 * sizeof(float)));
    l.row_o = reinterpret_cast<float*>(take(rows * d * sizeof(float)));
    const size_t p0 = attention_workspace_bytes(bf16, d, prefix_args(s, l.g)), p1 = attention_workspace_bytes(bf16, d, s.a);
    l.parts = take(p0 > p1 ? p0 : p1);
    l.bytes = used;
    return l;
}

}  // namespace

bool cache4_shared_fits(bool bf16, int d, const Cache4SharedArgs& s) {
    return attention_fits(bf16, d, s.a) && attention_fits(bf16, d, prefix_args(s, Groups{}));
}

size_t cache4_shared_workspace_bytes(bool bf16, int d, const Cache4SharedArgs& s) { return lay_out(bf16, d, s, nullptr).bytes; }

hipError_t launch_cache4_shared(bool bf16, int d, const Cache4SharedArgs& s, char* ws, hipStream_t stream) {
    const SharedLayout l = lay_out(bf16, d, s, ws);
    hipLaunchKernelGGL(kda_cache4_groups_kernel, dim3((unsigned)(s.n_groups + 1)), dim3(256), 0, stream, s, l.g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    PartArgs a = prefix_args(s, l.g);
    a.row_o = l.row_o; a.row_sums = l.row_sums;
    if ((e = launch_attention<PREFIX>(bf16, d, a, l.parts, stream)) != hipSuccess) return e;
    static_cast<Cache4AttentionArgs&>(a) = s.a;
    a.starts = l.g.starts; a.row_o = l.row_o; a.row_sums = l.row_sums;
    return launch_attention<OWN>(bf16, d, a, l.parts, stream);
}

}  // namespace kda

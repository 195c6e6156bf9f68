// kda_cache4_shared.hpp -- causal grouped-query attention over the paged 4-bit
// cache for groups of sequences that share their first tokens, which are read and
// converted once for all rows of a group.  For kda_cache4_shared.hip (bf16) and
// kda_cache4_shared_f32.hip.
//
//   out = (w0 O0 + w1 O1) / (w0 S0 + w1 S1),  w_i = e^(m_i - max(m_0, m_1))
// with maximum m, sum S and weighted values O of a row over the prefix (0) and
// over its own tokens (1).  Over the prefix a group is one sequence with all its
// rows, which see all of it; the rest is every sequence by itself from the end of
// its prefix on.  Both are the body of kda_cache4_attention.hpp, each in the form
// that its rows call for, and workgroups of one launch: neither waits for the
// other, and what each waits for (offsets, tables, its first tiles) passes
// meanwhile.  A second kernel joins what they leave of a row.
//
// 256 requests of one query on 8192 shared tokens and up to 1000 of their own, 32 heads
// over 8 of 128, bf16, take 5 us for the groups, 86 for both sides and 12 for joining;
// two launches for the sides, each with a second kernel for its parts, took 115.  The
// prefix is bound by what prompts are bound by (55 us of it), the rest by HBM (27 us at
// the rate of a copy) and by converting what it reads.
// 4 prompts of 500 on 65536 shared tokens take 5 + 737 + 15, 785 TFLOP/s; 48
// requests in 5 groups on 20000 tokens, 24 heads over 4 of 64, fp32, 4 + 41 + 11.
#pragma once

#include "kda_cache4_attention.hpp"

namespace kda {

namespace {

// What the kernels go by besides the arguments.  All of it lies in the workspace.
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

// A launch's side: its arguments, layout and parts.
struct Side {
    PartArgs a;
    Layout l;
    Parts parts;
};

constexpr int less_of(int x, int y) { return x < y ? x : y; }

// A workgroup's LDS, all of it dynamic: its Room, then what that side has besides.
template <typename Room> constexpr unsigned room_bytes() { return (sizeof(Room) + 15) / 16 * 16; }

// The first workgroups have the prefixes, those of the rest follow as CUs become
// free: 32 sequences behind 8192 tokens take 28.5 us this way, 35.6 with the rest
// first, 48 behind 20000 (24 heads over 4 of 64) 31 and 36, 256 behind 8192 87 and
// 86.  Alternating, which puts one kind on half of the CUs, 33, 51 and 118.
template <typename E, int D, int RP, bool SPLITP, int RO, bool SPLITO, bool ALONE>
__global__ __launch_bounds__(kWaves * 64, (less_of(less_of(waves_of(sizeof(E) == 2, D, RP), waves_of(sizeof(E) == 2, D, RO)), 2))) void kda_cache4_shared_kernel(Side prefix, Side own, unsigned prefix_blocks) {
    typedef Room<D, RP, SPLITP> RoomP;
    typedef Room<D, RO, SPLITO> RoomO;
    extern __shared__ __align__(16) char room[];
    if (blockIdx.x < prefix_blocks)
        attend<E, D, RP, SPLITP, false, PREFIX>(prefix.a, prefix.l, prefix.parts, *reinterpret_cast<RoomP*>(room), room + room_bytes<RoomP>(), blockIdx.x);
    else
        attend<E, D, RO, SPLITO, ALONE, OWN>(own.a, own.l, own.parts, *reinterpret_cast<RoomO*>(room), room + room_bytes<RoomO>(),
                                             blockIdx.x - prefix_blocks);
}

// What one side leaves of a row: an entry of its array, or `count` parts.
struct Share {
    const float *sums_at, *o_at;     // the entry or the first part
    int64_t stride;                  // of the parts; the second is half of it behind the first
    int count;
    __device__ __forceinline__ int64_t place(int i) const { return i == 0 ? 0 : i * stride - stride / 2; }
    __device__ __forceinline__ const float* sums(int i) const { return sums_at + 2 * place(i); }
    template <int D> __device__ __forceinline__ const float* o(int i) const { return o_at + place(i) * D; }
};

// Bounded, so that a workspace that another call writes meanwhile gives wrong
// values but no access outside the arrays.
template <int D>
__device__ __forceinline__ Share share_of(const Side& side, int64_t at, const Row& row, int count) {
    Share x = {&side.a.rows[at].mx, side.a.row_o + at * D, 0, min(count, 1)};
    const int64_t stride = 2 * (int64_t)side.a.c.heads * side.l.rows, places = stride * side.l.groups;
    if (count > 1 && row.first >= 0 && row.first + (count - 1) * stride - stride / 2 < places) {
        x.sums_at = side.parts.sums + 2 * (int64_t)row.first;
        x.o_at = side.parts.o + (int64_t)row.first * D;
        x.stride = stride;
        x.count = count;
    }
    return x;
}

// Joins what the two sides leave, row by row: weights 2^(m_i - max m).  WAVES waves
// take turns at a row's entries, and their sums are joined through LDS in the
// order of the waves.  Latency bounds it: a row's entries tell where its parts are
// (12 us above; found through its sequence, group and cuts it took 19).
template <typename E, int D, int WAVES>
__global__ __launch_bounds__((WAVES > kWaves ? WAVES : kWaves) * 64) void kda_cache4_join_kernel(Side prefix, Side own) {
    constexpr int PER = D / 64;
    constexpr int ROWS = WAVES > kWaves ? 1 : kWaves / WAVES;      // rows of a workgroup at a time
    __shared__ __align__(16) float acc[ROWS * WAVES][D];
    const PartArgs& a = own.a;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), turn = wave % WAVES;
    const int64_t rows = a.tokens * a.heads;
    // rows before the first sequence and behind the last have nothing
    const int first = a.cu_seqlens ? a.cu_seqlens[0] : 0, last = a.cu_seqlens ? a.cu_seqlens[a.n_seq] : INT32_MAX;
    for (int64_t id = (int64_t)blockIdx.x * ROWS + wave / WAVES; id < rows; id += (int64_t)gridDim.x * ROWS) {
        const int row = (int)(id / a.heads);
        if (row < first || row >= last) continue;
        const Row mine = a.rows[id], shared = prefix.a.rows[id];
        if (mine.count == 0) continue;
        const Share o_ = share_of<D>(own, id, mine, abs(mine.count)), p_ = share_of<D>(prefix, id, shared, mine.count < 0 ? 0 : max(shared.count, 0));
        const int before = p_.count, count = before + o_.count;
        auto sums = [&](int i) {
            return i < count ? *reinterpret_cast<const f32x2*>(i < before ? p_.sums(i) : o_.sums(i - before)) : f32x2{-INFINITY, 0.f};
        };
        typedef typename std::conditional<PER == 2, f32x2, float>::type OV;
        auto part = [&](int i) { return *reinterpret_cast<const OV*>((i < before ? p_.template o<D>(i) : o_.template o<D>(i - before)) + lane * PER); };

        // the first entries are on their way while their weights are found
        constexpr int AHEAD = 8;
        f32x2 ms = sums(lane);
        OV x[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) x[k] = part(min(turn + k * WAVES, count - 1));
        E gate[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) gate[e] = a.g ? reinterpret_cast<const E*>(a.g)[id * D + lane * PER + e] : (E)0.f;
        float mx = ms[0];
        for (int i = lane + 64; i < count; i += 64) mx = fmaxf(mx, sums(i)[0]);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
        float sum = 0.f;
        OV o = OV(0.f);
        for (int i0 = 0; i0 < count; i0 += 64) {
            if (i0 > 0) ms = sums(i0 + lane);
            const float w = ms[0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ms[0] - mx);
            sum += w * ms[1];
            auto weight = [&](int k) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), k)); };
            const int most = min(count - i0, 64);
#pragma unroll
            for (int q = 0; q < AHEAD; ++q) {
                const int k = turn + q * WAVES - i0;
                if (k >= 0 && k < most) o += weight(k) * x[q];
            }
#pragma unroll 8
            for (int k = turn + max(AHEAD * WAVES - i0, 0); k < most; k += WAVES) o += weight(k) * part(i0 + k);
        }
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) sum += __shfl_xor(sum, off);
        if constexpr (WAVES > 1) {
            *reinterpret_cast<OV*>(&acc[wave][lane * PER]) = o;
            __syncthreads();
            if (turn == 0) {
#pragma unroll
                for (int k = 1; k < WAVES; ++k) o += *reinterpret_cast<const OV*>(&acc[wave + k][lane * PER]);
            }
            __syncthreads();
            if (turn != 0) continue;
        }
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            float y;
            if constexpr (PER == 2) y = o[e];
            else y = o;
            y = sum == 0.f ? 0.f : y / sum;
            if (a.g) y *= sigmoidf_(to_f32(gate[e]));
            reinterpret_cast<E*>(a.out)[id * D + lane * PER + e] = from_f32<E>(y);
        }
    }
}

// The prefixes' side: a group is one sequence.
Cache4AttentionArgs prefix_args(const Cache4SharedArgs& s) {
    Cache4AttentionArgs a = s.a;
    a.n_seq = s.n_groups;
    a.max_len = s.max_prefix;
    // groups are ragged: about twice the rows of an even share
    const int64_t even = 2 * ((a.tokens + s.n_groups - 1) / s.n_groups);
    a.max_q = even < a.tokens ? even : a.tokens;
    static const int32_t packed = 0;     // a layout goes by whether there are offsets
    a.cu_seqlens = &packed;
    a.g = nullptr;
    return a;
}

struct SharedLayout {
    Plan prefix, own;
    Groups g;
    float* row_o[2];
    Row* rows[2];
    char* parts[2];      // of the prefixes' side, of the other
    size_t bytes;
};

SharedLayout lay_out(bool bf16, int d, const Cache4SharedArgs& s, char* ws) {
    SharedLayout l = {};
    const Cache4AttentionArgs pa = prefix_args(s);
    l.prefix = plan_of(bf16, d, pa, PREFIX);
    l.own = plan_of(bf16, d, s.a, OWN);
    size_t used = 0;
    auto take = [&](size_t bytes) {
        char* r = ws ? ws + used : nullptr;
        used += round256(bytes);
        return r;
    };
    auto ints = [&](int64_t n) { return reinterpret_cast<int32_t*>(take((size_t)n * sizeof(int32_t))); };
    l.g.cu = ints(s.n_groups + 1);
    l.g.prefix = ints(s.n_groups);
    l.g.tables = ints(s.n_groups);
    l.g.starts = ints(s.a.n_seq);
    const size_t rows = (size_t)s.a.tokens * s.a.heads;
    for (int i = 0; i < 2; ++i) {
        l.rows[i] = reinterpret_cast<Row*>(take(rows * sizeof(Row)));
        l.row_o[i] = reinterpret_cast<float*>(take(rows * d * sizeof(float)));
    }
    l.parts[0] = take(attention_workspace_bytes(bf16, d, pa, PREFIX));
    l.parts[1] = take(attention_workspace_bytes(bf16, d, s.a, OWN));
    l.bytes = used;
    return l;
}

template <typename E, int D, int RP, bool SPLITP, int RO, bool SPLITO, bool ALONE>
hipError_t launch_sides(const Side& prefix, const Side& own, const SharedLayout& l, hipStream_t s) {
    const int64_t prefix_blocks = workgroups(l.prefix) * own.a.c.heads, blocks = prefix_blocks + workgroups(l.own) * own.a.c.heads;
    const unsigned lds0 = room_bytes<Room<D, RP, SPLITP>>() + dynamic_lds(l.prefix, D), lds1 = room_bytes<Room<D, RO, SPLITO>>() + dynamic_lds(l.own, D);
    hipLaunchKernelGGL((kda_cache4_shared_kernel<E, D, RP, SPLITP, RO, SPLITO, ALONE>), dim3((unsigned)blocks), dim3(kWaves * 64), lds0 > lds1 ? lds0 : lds1, s,
                       prefix, own, (unsigned)prefix_blocks);
    return hipGetLastError();
}

template <typename E, int D, int RP, bool SPLITP>
hipError_t launch_own(const Side& prefix, const Side& own, const SharedLayout& l, hipStream_t s) {
    constexpr int MANY = rows_r(sizeof(E) == 2);
    if (!l.own.splitw) return launch_sides<E, D, RP, SPLITP, MANY, false, false>(prefix, own, l, s);
    if (l.own.alone) return launch_sides<E, D, RP, SPLITP, 1, true, true>(prefix, own, l, s);
    return launch_sides<E, D, RP, SPLITP, 2, true, false>(prefix, own, l, s);
}

template <typename E, int D>
hipError_t launch_shared(const Cache4SharedArgs& s, char* ws, hipStream_t stream) {
    constexpr bool bf16 = sizeof(E) == 2;
    const SharedLayout l = lay_out(bf16, D, s, ws);
    hipLaunchKernelGGL(kda_cache4_groups_kernel, dim3((unsigned)(s.n_groups + 1)), dim3(256), 0, stream, s, l.g);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    Side prefix = {}, own = {};
    static_cast<Cache4AttentionArgs&>(prefix.a) = prefix_args(s);
    prefix.a.cu_seqlens = l.g.cu;
    prefix.a.total_lens = l.g.prefix;
    prefix.a.table_rows = l.g.tables;
    prefix.a.tables = (int)s.a.n_seq;
    prefix.l = l.prefix.l;
    prefix.parts = parts_at(prefix.a, l.prefix, D, l.parts[0]);
    static_cast<Cache4AttentionArgs&>(own.a) = s.a;
    own.a.starts = l.g.starts;
    own.l = l.own.l;
    own.parts = parts_at(own.a, l.own, D, l.parts[1]);
    prefix.a.row_o = l.row_o[0]; prefix.a.rows = l.rows[0];
    own.a.row_o = l.row_o[1]; own.a.rows = l.rows[1];
    if (!l.prefix.splitw) e = launch_own<E, D, rows_r(bf16), false>(prefix, own, l, stream);
    else e = launch_own<E, D, 2, true>(prefix, own, l, stream);
    if (e != hipSuccess) return e;
    // Where a row has many parts, several waves share them, as where
    // kda_cache4_attention.hip joins them: 8 where rows are few, 4 where there are
    // waves enough.  240 rows take 6.0 us with 8 and 9.2 with 4 (28.5 with 1), 1152
    // 9.7 and 6.2, 2048 15.8 and 10.
    constexpr int SOME = 4;
    const int64_t rows = s.a.tokens * s.a.heads;
    const bool many = l.prefix.l.slots * 8 <= l.prefix.l.groups, few = rows <= 512;
    const int64_t turns = many ? rows : (rows + kWaves - 1) / kWaves;
    const dim3 grid((unsigned)(turns < (1 << 20) ? turns : (1 << 20)));
    if (many && few) hipLaunchKernelGGL((kda_cache4_join_kernel<E, D, kWideWaves>), grid, dim3(kWideWaves * 64), 0, stream, prefix, own);
    else if (many) hipLaunchKernelGGL((kda_cache4_join_kernel<E, D, SOME>), grid, dim3(SOME * 64), 0, stream, prefix, own);
    else hipLaunchKernelGGL((kda_cache4_join_kernel<E, D, 1>), grid, dim3(kWaves * 64), 0, stream, prefix, own);
    return hipGetLastError();
}

}  // namespace

}  // namespace kda

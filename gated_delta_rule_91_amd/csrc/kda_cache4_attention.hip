// kda_cache4_attention.hip -- causal grouped-query attention over the paged
// 4-bit cache.
//
//   out = sum_t e^(s_t - m) V_t / sum_t e^(s_t - m),  s_t = scale q . K_t,
//   m = max s_t, kept as a running maximum and sum in fp32.
//
// A wave takes 32 (few rows) or 64 (many) tokens of one key/value head at a
// time, against 16 R rows; a row is a (query, head of the group) pair, so the
// heads that share keys share their loads.  With lane = 16 g + n:
//  * S^T = K Q^T.  A operand: token n of 16, its channels [D/4 g, D/4 g + D/4),
//    D/32 steps of 8 channels; one scale byte covers them.  B operand: the row
//    n with the same channels.
//  * The result holds row n's scores of 4 tokens a half: as they lie these are
//    the B operand of O^T = V^T P^T, no exchange between lanes.  Maximum and
//    sum of a row are in-lane, then two exchanges over g.
//  * V^T as A operand needs 8 tokens of one channel a lane.  A lane takes, for
//    its 8 tokens, the word with the channels D/16 n + j: conversion gives
//    channel pairs of one token, a byte permute pairs the tokens, and j runs
//    over the MFMAs.  O^T then holds D/4 consecutive channels of row n.
// 4-bit values times their power of two are exact in bf16.  bf16 queries are
// exact too and the probabilities round once to bf16, which is half a step each
// and the size of the output's own rounding (1.8e-3 of the values against 64
// bits, where probabilities in fp32 leave 1.7e-3); their sum is taken before
// that, in fp32.  fp32 queries and probabilities are taken in three bf16 parts,
// which together hold 24 bits.
//
// Few rows (decode; at most split_max_rows of a sequence and head): the four waves
// of a workgroup take turns at the 32-token tiles, each through LDS of its own,
// and join their results.  Bound by the cache's bytes and by what a block costs
// at its ends: 256 ragged contexts of up to 8192 tokens, 32 heads over 8 of
// 128, take 74 us + 5 us for joining the parts where the bytes alone take 66 at
// the rate of a copy (5 us go into dealing out the work); 64 contexts of 32768
// take 396 us, 5.8 TB/s.  Loaded in the order of the operands, without LDS, the
// first took 92.
// Many rows (prompts): each wave has rows of its own, 64 tokens at a time are
// converted once for all four waves, and operands come from LDS.  Bound by the
// vector unit's work on the scores beside the products: 4 prompts of up to 1000
// tokens at the end of contexts of up to 8192, the same heads, take 197 us + 20
// us for the parts, the matrix units busy a quarter of it.  16 rows a wave
// instead of 32 took 320 us, 48 or 64 (one workgroup a CU) 306 and 289.  In fp32
// the ragged contexts take 98 us + 5, the prompts 413 + 19.
// Sequences are ragged and a query's tokens grow along a prompt, so work is
// dealt out by tokens: the row blocks' tokens lie end to end in units of 128,
// and each workgroup takes the same number of units, which may end one block,
// hold several and begin another.  What a workgroup has of a block that it
// does not hold whole is a part; a second kernel joins the parts.
#include <type_traits>

#include "kda_common.hpp"
#include "kda_hybrid_internal.hpp"

namespace kda {

namespace {

constexpr int kWaves = 4;
// The running maximum moves only when a score passes it by this much (in
// powers of two): probabilities then stay below 2^8 and the rescaling of the
// sums is rare.
constexpr float kSlack = 8.f;

typedef uint32_t u32x1 __attribute__((ext_vector_type(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 128;         // tokens that are dealt out at once
// Units that a block counts for beside its own, as beginning one costs: the
// 256 ragged contexts above take 83 us with 2, 77 with 3, 82 with 6, the
// prompts 195, 201 and 204.
constexpr int kBlockCost = 4;
constexpr int kMaxDealt = 4096;    // row blocks whose prefix sums lie in LDS; more fill the card as they are
// Units that can be dealt out: a workgroup's end, at most a unit for each of
// the workgroups (768) past all of them, is a 32-bit number too.
constexpr int kMaxUnits = INT32_MAX - 1024;

// How the work is laid out (host and kernels).
struct Layout {
    int rows;        // rows of a block
    int slots;       // upper bound of row blocks over all sequences
    int per_seq;     // without offsets: row blocks of each sequence
    int groups;      // workgroups of a key/value head that units are dealt to; 0: a block each
    bool by_slot;    // where a block's cut is found: at its slot, else at the workgroup it begins in
};

// Workgroup w has two parts at most, 2 w of a block that began before it and
// 2 w + 1 of one that begins in it and goes on.  Part i of row r of a block and
// key/value head h is at (i * heads + h) * rows + r.  The second kernel finds
// the blocks that several workgroups have by their cuts, of which there are
// as many as slots or workgroups, whichever are fewer.
struct Cut {
    int row0;        // first row of q of its sequence
    int n_rows;      // (query, head) rows of its sequence, 0: there is no such block
    int begin;       // its first one of them
    int from, last;  // first and last workgroup that have a part of it
};
struct Parts {
    Cut* cut;        // [slots or groups]
    float* sums;     // maximum and sum
    float* o;        // D channels
};

struct Block {
    int s;           // sequence
    int row0;        // its first query's row of q
    int n_rows;      // (query, head of the group) pairs of the sequence
    int total;       // tokens that count (at most what the table holds)
    int first;       // position of the first query, may be negative
    int begin;       // first pair of this block
    bool any;
};

// What sequence s is.
__device__ __forceinline__ void sequence_of(const Cache4AttentionArgs& a, int s, Block& b) {
    int64_t r0 = s, r1 = s + 1;
    if (a.cu_seqlens) seq_bounds(a.cu_seqlens, s, a.tokens, r0, r1);
    const int total = max(a.total_lens[s], 0), queries = (int)(r1 - r0);
    b.s = s;
    b.row0 = (int)r0;
    b.n_rows = queries * a.group;
    b.first = total - queries;
    b.total = min(total, a.max_pages << a.c.page_shift);
}

// Row blocks of sequence s with offsets begin at slot floor(cu[s] G / rows) + s,
// which leaves each its ceil(m G / rows) slots and can be searched: the first
// term, of an offset.
__device__ __forceinline__ int first_slot(const Cache4AttentionArgs& a, const Layout& l, int offset) {
    const int c = min(max(offset, 0), (int)a.tokens);
    return (int)((uint32_t)c * (uint32_t)a.group / (uint32_t)l.rows);
}

// The sequence of a slot (n_seq or more: none); cu: the offsets, or a copy of them.
__device__ __forceinline__ int sequence_at(const Cache4AttentionArgs& a, const Layout& l, const int32_t* cu, int slot) {
    if (!a.cu_seqlens) return l.per_seq == 1 ? slot : (int)((uint32_t)slot / (uint32_t)l.per_seq);
    int lo = 0, hi = (int)a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first_slot(a, l, cu[mid]) + mid <= slot) lo = mid; else hi = mid;
    }
    return lo;
}

// The row block of a slot of sequence s.
__device__ __forceinline__ Block block_of(const Cache4AttentionArgs& a, const Layout& l, int s, int slot) {
    Block b = {};
    if (s >= a.n_seq) return b;             // more slots than row blocks
    sequence_of(a, s, b);
    const int at = slot - (a.cu_seqlens ? first_slot(a, l, a.cu_seqlens[s]) + s : s * l.per_seq);
    b.any = at >= 0 && (int64_t)at * l.rows < b.n_rows;
    b.begin = b.any ? at * l.rows : 0;
    return b;
}

// Tokens that row r of a sequence sees.
__device__ __forceinline__ int end_of(const Cache4AttentionArgs& a, const Block& b, int r) {
    if (r >= b.n_rows) return 0;
    const int i = (int)((uint32_t)r / (uint32_t)a.group);
    return min(max(b.first + i + 1, 0), b.total);
}

// Index of (row of q, head) of row r.
__device__ __forceinline__ int place_of(const Cache4AttentionArgs& a, int row0, int kvh, int r) {
    const int i = (int)((uint32_t)r / (uint32_t)a.group);
    return (row0 + i) * a.heads + kvh * a.group + (r - i * a.group);
}

// before[i]: units that the row blocks before i count for, i <= slots; returns
// those of all.  A block with rows has one of its own at least, though its
// output may be zeros.  of[i]: the sequence of slot i.  cu: LDS for n_seq + 1
// offsets, which are searched there.
__device__ int deal_out(const Cache4AttentionArgs& a, const Layout& l, int32_t* before, uint16_t* of, int32_t* cu) {
    __shared__ int32_t part[kWaves];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    if (a.cu_seqlens) {
        for (int i = t; i <= (int)a.n_seq; i += kWaves * 64) cu[i] = a.cu_seqlens[i];
        __syncthreads();
    }
    int sum = 0;
    for (int base = 0; base < l.slots; base += kWaves * 64) {
        int c = 0;
        if (base + t < l.slots) {
            const int s = sequence_at(a, l, cu, base + t);
            const Block b = block_of(a, l, s, base + t);
            of[base + t] = (uint16_t)s;
            if (b.any) c = max((end_of(a, b, min(b.begin + l.rows, b.n_rows) - 1) + kUnit - 1) / kUnit, 1) + kBlockCost;
        }
        int in = c;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int u = __shfl_up(in, off);
            if (lane >= off) in += u;
        }
        if (lane == 63) part[wave] = in;
        __syncthreads();
        int ahead = sum;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            if (w < wave) ahead += part[w];
            sum += part[w];
        }
        if (base + t < l.slots) before[base + t] = ahead + in - c;
        __syncthreads();
    }
    if (t == 0) before[l.slots] = sum;
    __syncthreads();
    return sum;
}

// Whether values with this scale may be Inf or NaN.
__device__ __forceinline__ bool is_odd(float scale) { return (__float_as_uint(scale) >> 23) >= 253u; }

__device__ __forceinline__ float scale_bits(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 channels of a word, times their scale.
__device__ __forceinline__ bf16x8 eight_of(uint32_t w, float scale) {
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

__device__ __forceinline__ uint32_t bits_of(bf16x2 x) { return __builtin_bit_cast(uint32_t, x); }

// Channels (2 I, 2 I + 1) of 8 tokens as two operands: lo and hi.
template <int I>
__device__ __forceinline__ void two_channels(const uint32_t (&w)[8], const float (&s)[8], bf16x8& lo, bf16x8& hi) {
    uint32_t p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = bits_of(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[e], s[e], I));
    u32x4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        a[e] = __builtin_amdgcn_perm(p[2 * e + 1], p[2 * e], 0x05040100u);
        b[e] = __builtin_amdgcn_perm(p[2 * e + 1], p[2 * e], 0x07060302u);
    }
    lo = __builtin_bit_cast(bf16x8, a);
    hi = __builtin_bit_cast(bf16x8, b);
}

// The larger of two, NaN if one is: one instruction for three of them, where
// fmaxf first quiets each.  A row with a NaN score is NaN whatever its maximum.
__device__ __forceinline__ float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }

// The largest over the four lanes with the same n.
__device__ __forceinline__ float over_g(float x) {
    const uint32_t b = __float_as_uint(x);
    const auto p = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    const uint32_t c = __float_as_uint(larger(__uint_as_float(p[0]), __uint_as_float(p[1])));
    const auto q = __builtin_amdgcn_permlane16_swap(c, c, false, false);
    return larger(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// x in PARTS bf16 parts whose sum holds 8 PARTS bits of it.
template <int PARTS>
__device__ __forceinline__ void parts_of(float x, __bf16 (&p)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
        p[i] = (__bf16)x;
        x -= (float)p[i];
    }
}

// One 32-token tile as loaded: keys, values and scales of both 16-token halves.
template <int D>
struct Tile {
    uint32_t k[2][D / 32];
    uint32_t ks[2];
    uint32_t v[2][4];
    uint32_t vs[2][D / 32];     // scales of 4 tokens, D/32 bytes each
    bool ok[2];                 // the half's page exists
};

// The block table of a sequence, 64 entries at a time in the lanes of a wave,
// so that a tile's pages cost no memory access.
struct Pages {
    const int32_t* table;
    int most, shift, base, mine;
    __device__ __forceinline__ Pages(const Cache4AttentionArgs& a, int64_t s, int t)
        : table(a.block_table + s * a.max_pages), most(a.max_pages), shift(a.c.page_shift) { fill(t >> shift); }
    __device__ __forceinline__ void fill(int first) {
        base = first;
        const int i = first + (int)(threadIdx.x & 63);
        mine = i < most ? table[i] : -1;
    }
    __device__ __forceinline__ int of(int t) {
        const int i = t >> shift;
        if ((uint32_t)(i - base) > 63u) fill(i);
        return __builtin_amdgcn_readlane(mine, i - base);
    }
};

// The first row of 16 tokens in the cache's arrays.  Tokens whose page does
// not exist read page 0 (there is one: a cache without pages counts no tokens)
// and are masked.
__device__ __forceinline__ int64_t cache_row(const Cache4AttentionArgs& a, Pages& pages, int kvh, int t, bool& ok) {
    const int page = pages.of(t);
    ok = page >= 0 && page < a.c.pages;
    return (((int64_t)(ok ? page : 0) * a.c.heads + kvh) << a.c.page_shift) + (t & ((1 << a.c.page_shift) - 1));
}

template <int D>
__device__ __forceinline__ void keys_at(const Cache4AttentionArgs& a, int64_t row, int lane, uint32_t (&k)[D / 32], uint32_t& ks) {
    const uint32_t g = lane >> 4, n = lane & 15;
    const uint8_t* kp = a.c.k + row * (D / 2);
    const uint32_t ko = n * (D / 2) + g * (D / 8);
    if constexpr (D == 128) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(kp + ko);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = w[j];
    } else {
        const u32x2 w = *reinterpret_cast<const u32x2*>(kp + ko);
        k[0] = w[0]; k[1] = w[1];
    }
    ks = (a.c.k_scale + row * (D / 32))[n * (D / 32) + g * (D / 32) / 4];
}

template <int D>
__device__ __forceinline__ void values_at(const Cache4AttentionArgs& a, int64_t row, int lane, uint32_t (&v)[4], uint32_t (&vs)[D / 32]) {
    const uint32_t g = lane >> 4, n = lane & 15;
    const uint8_t *vp = a.c.v + row * (D / 2), *sp = a.c.v_scale + row * (D / 32);
    const uint32_t vo = 4 * g * (D / 2) + (D == 128 ? 4 * n : 4 * (n >> 1)), vso = 4 * g * (D / 32);
    if constexpr (D == 128) {
        const u32x4 z = *reinterpret_cast<const u32x4*>(sp + vso);
#pragma unroll
        for (int j = 0; j < 4; ++j) vs[j] = z[j];
    } else {
        const u32x2 z = *reinterpret_cast<const u32x2*>(sp + vso);
        vs[0] = z[0]; vs[1] = z[1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint32_t*>(vp + vo + i * (D / 2));
}

// 32 tokens of one key/value head as they lie in memory: 16 bytes a lane for
// each KB of keys and values, 4 bytes a lane for all scales.
template <int D>
struct Raw {
    u32x4 k[D / 64], v[D / 64];
    uint32_t scales;
    int ok;                     // which halves' pages exist
};

template <int D>
__device__ __forceinline__ void load_raw(const Cache4AttentionArgs& a, Pages& pages, int kvh, int t0, int lane, Raw<D>& x) {
    int64_t row[2];
    x.ok = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        bool ok;
        row[u] = cache_row(a, pages, kvh, t0 + 16 * u, ok);
        x.ok |= ok << u;
    }
    if constexpr (D == 128) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            x.k[u] = *reinterpret_cast<const u32x4*>(a.c.k + row[u] * (D / 2) + (uint32_t)(16 * lane));
            x.v[u] = *reinterpret_cast<const u32x4*>(a.c.v + row[u] * (D / 2) + (uint32_t)(16 * lane));
        }
    } else {
        const int64_t at = (lane < 32 ? row[0] : row[1]) * (D / 2) + 16 * (lane & 31);
        x.k[0] = *reinterpret_cast<const u32x4*>(a.c.k + at);
        x.v[0] = *reinterpret_cast<const u32x4*>(a.c.v + at);
    }
    // scales of the keys of both halves, then of the values: D/8 lanes each
    constexpr int N = D / 8;
    const uint8_t* p = lane & (2 * N) ? a.c.v_scale : a.c.k_scale;
    const int64_t at = (lane & N ? row[1] : row[0]) * (D / 32) + 4 * (lane & (N - 1));
    x.scales = *reinterpret_cast<const uint32_t*>(p + at);
}

// A wave's staging area in LDS: loads that follow memory take a quarter of the
// cache lookups that loads in operand order do (each of whose lanes has a row
// of its own), and the operands are read from here.  Token r of a half has its
// 16-byte chunk c at chunk c ^ (r / 4 mod chunks) of row r, and operand row m
// is token m / 4 + 4 (m mod 4): both so that the lanes of a read lie in
// different banks.  A result row 4 g + v then is token g + 4 v.
template <int D>
struct Stage {
    static constexpr int CH = D / 32, HALF = 16 * CH * 16, V = 2 * HALF, SC = 4 * HALF, SH = 16 * (D / 32);
    static constexpr int BYTES = SC + 4 * SH;
    char* at;
    int lane;
    __device__ __forceinline__ int chunk(int r, int c) const { return (r * CH + (c ^ ((r >> 2) & (CH - 1)))) * 16; }
    __device__ __forceinline__ void put(const Raw<D>& x) const {
        if constexpr (D == 128) {
            const int to = chunk(lane >> 2, lane & 3);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                *reinterpret_cast<u32x4*>(at + u * HALF + to) = x.k[u];
                *reinterpret_cast<u32x4*>(at + V + u * HALF + to) = x.v[u];
            }
        } else {
            const int to = (lane >> 5) * HALF + chunk((lane >> 1) & 15, lane & 1);
            *reinterpret_cast<u32x4*>(at + to) = x.k[0];
            *reinterpret_cast<u32x4*>(at + V + to) = x.v[0];
        }
        if (lane < D / 2) *reinterpret_cast<u32x1*>(at + SC + 4 * lane) = u32x1{x.scales};
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // Before the next put: all lanes have read.
    __device__ __forceinline__ void done() const {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
    // The words and the scale of this lane's key operands, of half u.
    __device__ __forceinline__ void key(int u, uint32_t (&k)[D / 32], float& scale) const {
        const int g = lane >> 4, n = lane & 15, r = (n >> 2) + 4 * (n & 3);
        if constexpr (D == 128) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(at + u * HALF + chunk(r, g));
#pragma unroll
            for (int j = 0; j < 4; ++j) k[j] = w[j];
        } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(at + u * HALF + chunk(r, g >> 1) + 8 * (g & 1));
            k[0] = w[0]; k[1] = w[1];
        }
        scale = scale_bits(*reinterpret_cast<const uint8_t*>(at + SC + u * SH + r * (D / 32) + (D == 128 ? g : g >> 1)));
    }
    // The word and scale of this lane's channel group for its token 4 u + v.
    __device__ __forceinline__ void value(int u, int v, uint32_t& w, uint32_t& scale) const {
        const int g = lane >> 4, n = lane & 15, r = g + 4 * v;
        if constexpr (D == 128) {
            w = (*reinterpret_cast<const u32x1*>(at + V + u * HALF + chunk(r, n >> 2) + 4 * (n & 3)))[0];
        } else {
            w = (*reinterpret_cast<const u32x1*>(at + V + u * HALF + chunk(r, n >> 3) + 4 * ((n >> 1) & 3)))[0];
            w >>= 16 * (n & 1);
        }
        scale = *reinterpret_cast<const uint8_t*>(at + SC + 2 * SH + u * SH + r * (D / 32) + (D == 128 ? n >> 2 : n >> 3));
    }
};

// The keys of 16 tokens, as a tile's first half.
template <int D>
__device__ __forceinline__ void load_keys(const Cache4AttentionArgs& a, Pages& pages, int kvh, int t0, int lane, Tile<D>& x) {
    bool ok;
    keys_at<D>(a, cache_row(a, pages, kvh, t0, ok), lane, x.k[0], x.ks[0]);
}

template <int D>
__device__ __forceinline__ void load_values(const Cache4AttentionArgs& a, Pages& pages, int kvh, int t0, int lane, Tile<D>& x) {
#pragma unroll
    for (int u = 0; u < 2; ++u) values_at<D>(a, cache_row(a, pages, kvh, t0 + 16 * u, x.ok[u]), lane, x.v[u], x.vs[u]);
}

// The words and scales of this lane's channel group for its 8 tokens; those at
// or past `end`, or without a page, are zeros, whatever memory holds there.
template <int D>
__device__ __forceinline__ void values_of(const Tile<D>& x, int t0, int end, int lane, uint32_t (&w)[8], float (&s)[8]) {
    const int g = lane >> 4, n = lane & 15;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            uint32_t b, c;
            if constexpr (D == 128) {
                b = x.vs[u][v] >> (8 * (n >> 2));
                c = x.v[u][v];
            } else {
                b = x.vs[u][v >> 1] >> (16 * (v & 1) + 8 * (n >> 3));
                c = x.v[u][v] >> (16 * (n & 1));
            }
            const bool in = x.ok[u] && t0 + 16 * u + 4 * g + v < end;
            w[4 * u + v] = in ? c : 0u;
            s[4 * u + v] = scale_bits(in ? b & 255u : 127u);
        }
}

// Bytes of two tiles of 64 tokens as operands.
__host__ __device__ constexpr int shared_tiles(int d) { return 2 * 64 * d * 2 * 2; }

// Waves per SIMD that registers are kept for, and so workgroups per CU that work
// is dealt to: what fits without spilling.  (With 3 instead of 2 in bf16 and
// D = 128, R = 1, 56 bytes of spills: 64 contexts of 32768 tokens took 417 us
// instead of 396, of 2048 36 instead of 30; with 2 instead of 3 and D = 64, 256
// contexts of 4096 take 147 instead of 134.  With 3 instead of 2 in fp32 and
// D = 64, R = 1, 56 bytes too: two contexts of up to 131072 tokens, 24 heads over
// 4, take 20.3 us and 8.8 for the parts instead of 19.8 and 6.0.)
constexpr int waves_of(bool bf16, int d, int r) {
    if (bf16) return r == 1 && d == 64 ? 3 : 2;
    return r == 2 && d == 128 ? 1 : 2;
}

template <typename E, int D, int R, bool SPLITW>
__global__ __launch_bounds__(kWaves * 64, (waves_of(sizeof(E) == 2, D, R))) void kda_cache4_attention_kernel(Cache4AttentionArgs a, Layout l, Parts parts) {
    constexpr int PARTS = sizeof(E) == 2 ? 1 : 3;
    constexpr int KS = D / 32;          // MFMA steps over the channels
    constexpr int VJ = D / 16;          // MFMAs of a value tile
    constexpr int PER = D / 4;          // channels of a lane's result
    constexpr int ROWS = 16 * R;        // rows of a wave
    constexpr int LD = D + 4;
    __shared__ __align__(16) float so[SPLITW ? kWaves : 1][SPLITW ? ROWS : 1][LD], sm[kWaves][ROWS], ss[kWaves][ROWS];
    // many rows: the converted tiles, two of 64 tokens in turn; then the prefix sums
    extern __shared__ __align__(16) char dynamic[];
    int32_t* before = reinterpret_cast<int32_t*>(dynamic + (SPLITW ? 0 : shared_tiles(D)));
    uint16_t* of = reinterpret_cast<uint16_t*>(before + l.slots + 1);
    static_assert((SPLITW ? sizeof(so) : shared_tiles(D)) >= (kMaxDealt + 1) * sizeof(int32_t), "the offsets lie there for a while");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, n = lane & 15;

    // key/value heads alternate fastest, so workgroups that share keys and
    // values lie on one XCD where there are 8 heads
    const int kvh = (int)(blockIdx.x % a.c.heads), group = (int)(blockIdx.x / a.c.heads);
    int slot = group;
    int at = 0, stop = 1, each = 1;     // this workgroup's units
    if (l.groups > 0) {
        const int all = deal_out(a, l, before, of, reinterpret_cast<int32_t*>(SPLITW ? reinterpret_cast<char*>(so) : dynamic));
        each = max((all + l.groups - 1) / l.groups, 1);
        if (kvh == 0 && !l.by_slot) {
            if (threadIdx.x == 0) parts.cut[group] = Cut{};
        } else if (kvh == 0 && group == 0) {
            for (int i = threadIdx.x; i < l.slots; i += kWaves * 64)
                if (before[i] == before[i + 1]) parts.cut[i] = Cut{};      // the others have a workgroup that writes them
        }
        at = (int)min((int64_t)group * each, (int64_t)all);
        stop = min(at + each, all);
        int lo = 0, hi = l.slots;  // the last block that begins at or before `at`: empty ones lie before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before[mid] <= at) lo = mid; else hi = mid;
        }
        slot = __builtin_amdgcn_readfirstlane(lo);
        at = __builtin_amdgcn_readfirstlane(at);
        stop = __builtin_amdgcn_readfirstlane(stop);
    }

    for (; at < stop; ++slot) {
        const Block b = block_of(a, l, l.groups > 0 ? __builtin_amdgcn_readfirstlane(of[slot]) : sequence_at(a, l, a.cu_seqlens, slot), slot);
        const int n_rows = b.n_rows;
        int lo = 0, lim = b.total, part = -1;
        if (l.groups > 0) {
            // the block's own units are [p0, p1)
            const int p0 = __builtin_amdgcn_readfirstlane(before[slot]) + kBlockCost, p1 = __builtin_amdgcn_readfirstlane(before[slot + 1]);
            const int from = max(at, p0), to = min(stop, p1);
            at = max(at, min(stop, p1));
            if (to <= from) continue;       // no rows, or the next workgroup has them all
            lo = (from - p0) * kUnit;
            lim = min(b.total, (to - p0) * kUnit);
            const bool begins = from == p0, goes_on = to < p1;
            if (!begins || goes_on) part = 2 * group + (begins ? 1 : 0);
            if (begins && (goes_on || l.by_slot) && kvh == 0 && threadIdx.x == 0)
                parts.cut[l.by_slot ? slot : group] = goes_on ? Cut{b.row0, n_rows, b.begin, group, (p1 - 1) / each} : Cut{};
        } else {
            at = stop;
            if (!b.any) continue;
        }
        const int row0 = b.begin + (SPLITW ? 0 : wave * ROWS);
        const int last = min(row0 + ROWS, n_rows) - 1;          // may lie before row0: nothing for this wave
        const int hi = last < row0 ? lo : min(end_of(a, b, last), lim);
        const int all_see = end_of(a, b, row0);                  // the first row sees the fewest

        // queries: row n of each 16, channels [PER g, PER g + PER)
        bf16x8 q[R][KS][PARTS];
        int end[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int row = row0 + 16 * r + n;
            end[r] = end_of(a, b, row);
            const E* p = reinterpret_cast<const E*>(a.q) + (int64_t)place_of(a, b.row0, kvh, row < n_rows ? row : 0) * D + PER * g;
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if constexpr (PARTS == 1) {
                        q[r][j][0][e] = (__bf16)(a.sign * to_f32(p[8 * j + e]));
                    } else {
                        __bf16 s[PARTS];
                        parts_of<PARTS>(a.sign * p[8 * j + e], s);
#pragma unroll
                        for (int i = 0; i < PARTS; ++i) q[r][j][i][e] = s[i];
                    }
                }
        }

        f32x4 o[R][VJ];
        float m[R], sum[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            sum[r] = 0.f;
#pragma unroll
            for (int j = 0; j < VJ; ++j) o[r][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        Pages pages(a, b.s, lo);

        // The running maxima, of N scores of a lane for each row tile.
        auto raise = [&](const auto& y) {
            constexpr int N = sizeof(y[0]) / sizeof(float);
            float top[R];
            bool more = false;
#pragma unroll
            for (int r = 0; r < R; ++r) {
                top[r] = y[r][0];
#pragma unroll
                for (int e = 1; e < N; ++e) top[r] = larger(top[r], y[r][e]);
                top[r] = over_g(top[r]) * a.to_log2;
                more = more || top[r] > m[r] + kSlack;
            }
            if (__any(more)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float mn = fmaxf(m[r], top[r]);
                    const float f = mn == -INFINITY ? 1.f : __builtin_amdgcn_exp2f(m[r] - mn);
                    sum[r] *= f;
#pragma unroll
                    for (int j = 0; j < VJ; ++j) o[r][j] *= f;
                    m[r] = mn;
                }
            }
        };
        // 8 scores into probabilities of row tile r, whose sum is kept.
        auto weigh = [&](int r, const float* y, bf16x8 (&p)[PARTS]) {
            const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = __builtin_amdgcn_exp2f(fmaf(y[e], a.to_log2, -base));
                sum[r] += z;
                if constexpr (PARTS == 1) {
                    p[0][e] = (__bf16)z;
                } else {
                    __bf16 s[PARTS];
                    parts_of<PARTS>(z, s);
#pragma unroll
                    for (int i = 0; i < PARTS; ++i) p[i][e] = s[i];
                }
            }
        };
        // Whether stop - 1 is the last token that this lane's row of row tile r sees
        // of the 32 from t0 on.
        auto ends_at = [&](int r, int t0, int stop) { return min(min(end[r], hi), t0 + 32) == stop; };
        // to + values x probabilities, where the row counts.
        auto product = [&](f32x4& to, bf16x8 value, const bf16x8 (&p)[PARTS], bool counts) {
            f32x4 sum = to;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(value, p[i], sum, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < 4; ++v) to[v] = counts ? sum[v] : to[v];
        };

        if constexpr (SPLITW) {
            // 32 staged tokens; ALL: every row sees all of them
            const Stage<D> stage = {reinterpret_cast<char*>(&so[wave][0][0]), lane};
            static_assert(Stage<D>::BYTES <= (int)sizeof(so[0]), "a wave stages where its results go later");
            auto run = [&](auto all, int ok, int t0) {
                constexpr bool ALL = decltype(all)::value;
                float y[R][8];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    uint32_t kw[KS];
                    float ks;
                    stage.key(u, kw, ks);
                    f32x4 acc[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        const bf16x8 k = eight_of(kw[j], ks);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int i = 0; i < PARTS; ++i) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[r][j][i], acc[r], 0, 0, 0);
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int t = t0 + 16 * u + g + 4 * v;
                        const bool in = ALL || ((ok >> u & 1) && t < hi);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            y[r][4 * u + v] = acc[r][v];
                            if constexpr (!ALL) {
                                if (!in || t >= end[r]) y[r][4 * u + v] = -INFINITY;
                            }
                        }
                    }
                }
                raise(y);
                bf16x8 p[R][PARTS];
#pragma unroll
                for (int r = 0; r < R; ++r) weigh(r, y[r], p[r]);

                uint32_t w[8];
                float s[8];
                // the values of tokens before `stop`; the others are zeros, whatever memory holds there
                auto values = [&](int stop) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            uint32_t c, b;
                            stage.value(u, v, c, b);
                            if constexpr (!ALL) {
                                const bool in = (ok >> u & 1) && t0 + 16 * u + g + 4 * v < stop;
                                c = in ? c : 0u;
                                b = in ? b : 127u;
                            }
                            w[4 * u + v] = c;
                            s[4 * u + v] = scale_bits(b);
                        }
                };
                auto accumulate = [&](auto counts) {
                    auto pair = [&](auto I) {
                        bf16x8 c[2];
                        two_channels<decltype(I)::value>(w, s, c[0], c[1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int r = 0; r < R; ++r) product(o[r][2 * decltype(I)::value + h], c[h], p[r], counts(r));
                    };
                    pair(std::integral_constant<int, 0>{});
                    pair(std::integral_constant<int, 1>{});
                    if constexpr (VJ == 8) {
                        pair(std::integral_constant<int, 2>{});
                        pair(std::integral_constant<int, 3>{});
                    }
                };
                values(hi);
                if constexpr (ALL) {
                    accumulate([](int) { return true; });
                } else {
                    bool odd = false;       // a value that is no number, which some rows do not see
#pragma unroll
                    for (int e = 0; e < 8; ++e) odd = odd || is_odd(s[e]);
                    const bool apart = __any(odd);
                    // Where apart, the rows of one end at a time, with the tokens behind
                    // it cleared: 0 times NaN would reach rows that do not see it.
                    for (int stop = apart ? t0 + 1 : t0 + 32;; ++stop) {
                        if (apart) values(min(stop, hi));
                        accumulate([&](int r) { return !apart || ends_at(r, t0, stop); });
                        if (stop == t0 + 32) break;
                    }
                }
                stage.done();
            };
            // the next tile is on its way while one is worked on
            constexpr int STEP = 32 * kWaves;
            const int plain = min(all_see, hi) - 32;       // last tile that every row sees
            int t0 = lo + 32 * wave;
            if (t0 < hi) {
                Raw<D> x;
                load_raw<D>(a, pages, kvh, t0, lane, x);
                auto turn = [&] {           // stages one tile, sends for the next
                    const int ok = x.ok;
                    stage.put(x);
                    t0 += STEP;
                    if (t0 < hi) load_raw<D>(a, pages, kvh, t0, lane, x);
                    return ok;
                };
                do {
                    while (t0 <= plain && x.ok == 3) {
                        const int ok = turn();
                        run(std::true_type{}, ok, t0 - STEP);
                    }
                    if (t0 >= hi) break;
                    const int ok = turn();
                    run(std::false_type{}, ok, t0 - STEP);
                } while (t0 < hi);
            }
        } else {
            // 64 tokens at a time for all waves, as operands in LDS: [k | v] operands of
            // 64 lanes x 16 bytes.  Wave w converts the keys of its 16 tokens and half
            // of the channels of the values of 32, while the last 64 tokens' are used.
            constexpr int KB = 4 * KS, OPS = KB + 2 * VJ;
            __shared__ int odd[2][2];       // whether values of 32 tokens were left out (see below)
            bf16x8* ops = reinterpret_cast<bf16x8*>(dynamic);
            const int half = wave >> 1;
            const int hi_all = min(end_of(a, b, min(b.begin + l.rows, n_rows) - 1), lim), see_all = end_of(a, b, b.begin);
            Tile<D> x;                      // the values of 32 tokens; the keys of 16 in its first half
            int ok = 0, ok_next = 0;        // which 16 tokens have a page
            auto fetch = [&](int T0) {
                ok_next = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int page = pages.of(T0 + 16 * u);
                    ok_next |= (page >= 0 && page < a.c.pages && T0 + 16 * u < hi_all) << u;
                }
                load_keys<D>(a, pages, kvh, T0 + 16 * wave, lane, x);
                load_values<D>(a, pages, kvh, T0 + 32 * half, lane, x);
            };
            auto convert = [&](int T0, int buf) {
                bf16x8* to = ops + buf * OPS * 64 + lane;
#pragma unroll
                for (int j = 0; j < KS; ++j) to[(wave * KS + j) * 64] = eight_of(x.k[0][j], scale_bits(x.ks[0]));
                uint32_t w[8];
                float s[8];
                values_of<D>(x, T0 + 32 * half, hi_all, lane, w, s);
                // Values that are no numbers, of tokens that some rows do not see, are
                // left out, as 0 times NaN would reach those rows; the others get them
                // one end at a time.
                const bool partly = T0 + 64 > see_all;
                bool some = false;
                if (partly) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const bool no = is_odd(s[e]);
                        some = some || no;
                        if (no) { w[e] = 0; s[e] = 1.f; }
                    }
                }
                if ((wave & 1) == 0) {
                    const bool any = __any(some);
                    if (lane == 0) odd[buf][half] = any;
                }
                auto pair = [&](auto I) {
                    two_channels<decltype(I)::value>(w, s, to[(KB + half * VJ + 2 * decltype(I)::value) * 64], to[(KB + half * VJ + 2 * decltype(I)::value + 1) * 64]);
                };
                if constexpr (VJ == 8) {
                    if ((wave & 1) == 0) { pair(std::integral_constant<int, 0>{}); pair(std::integral_constant<int, 1>{}); }
                    else { pair(std::integral_constant<int, 2>{}); pair(std::integral_constant<int, 3>{}); }
                } else {
                    if ((wave & 1) == 0) pair(std::integral_constant<int, 0>{});
                    else pair(std::integral_constant<int, 1>{});
                }
            };
            // What the values that were left out of 32 tokens add, to the rows of one
            // end at a time.
            auto add_odd = [&](const bf16x8 (&p)[R][PARTS], int t0) {
                Tile<D> z;
                load_values<D>(a, pages, kvh, t0, lane, z);
#pragma unroll 1
                for (int stop = t0 + 1; stop <= t0 + 32; ++stop) {
                    uint32_t w[8];
                    float s[8];
                    values_of<D>(z, t0, min(stop, hi_all), lane, w, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (!is_odd(s[e])) { w[e] = 0; s[e] = 1.f; }
                    auto pair = [&](auto I) {
                        bf16x8 c[2];
                        two_channels<decltype(I)::value>(w, s, c[0], c[1]);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int r = 0; r < R; ++r) product(o[r][2 * decltype(I)::value + h], c[h], p[r], ends_at(r, t0, stop));
                    };
                    pair(std::integral_constant<int, 0>{});
                    pair(std::integral_constant<int, 1>{});
                    if constexpr (VJ == 8) {
                        pair(std::integral_constant<int, 2>{});
                        pair(std::integral_constant<int, 3>{});
                    }
                }
            };
            // 64 tokens, of which every row sees all or not
            auto use = [&](bool all, int T0, int buf) {
                const bf16x8* from = ops + buf * OPS * 64 + lane;
                // operands are read a group ahead of their products: left alone the
                // compiler reads each right before its product and waits
                float y[R][16];
                bf16x8 k[2][KS];
#pragma unroll
                for (int j = 0; j < KS; ++j) k[0][j] = from[j * 64];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    if (u < 3) {
#pragma unroll
                        for (int j = 0; j < KS; ++j) k[(u + 1) & 1][j] = from[((u + 1) * KS + j) * 64];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    f32x4 acc[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int j = 0; j < KS; ++j)
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int i = 0; i < PARTS; ++i) acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[u & 1][j], q[r][j][i], acc[r], 0, 0, 0);
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int v = 0; v < 4; ++v) y[r][4 * u + v] = acc[r][v];
                }
                if (!all) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const bool page = ok >> u & 1;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const int t = T0 + 16 * u + 4 * g + v;
                            const bool in = page && t < hi;
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                if (!in || t >= end[r]) y[r][4 * u + v] = -INFINITY;
                        }
                    }
                }
                raise(y);
                bf16x8 p[2][R][PARTS], v[2][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) v[0][j] = from[(KB + j) * 64];
#pragma unroll
                for (int r = 0; r < R; ++r) weigh(r, y[r], p[0][r]);
#pragma unroll
                for (int c = 0; c < 2 * VJ / 4; ++c) {         // four operands at a time
                    if (c + 1 < 2 * VJ / 4) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[(c + 1) & 1][j] = from[(KB + 4 * (c + 1) + j) * 64];
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    const int hh = c / (VJ / 4);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int i = 0; i < PARTS; ++i) {
                                f32x4& to = o[r][4 * c % VJ + j];
                                to = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[c & 1][j], p[hh][r][i], to, 0, 0, 0);
                            }
                    // the second half's exponentials go beside the first half's products
                    if (c == 0) {
#pragma unroll
                        for (int r = 0; r < R; ++r) weigh(r, y[r] + 8, p[1][r]);
                    }
                }
                if (T0 + 64 > see_all) {
                    if (__builtin_amdgcn_readfirstlane(odd[buf][0])) add_odd(p[0], T0);
                    if (__builtin_amdgcn_readfirstlane(odd[buf][1])) add_odd(p[1], T0 + 32);
                }
            };
            const int plain = min(all_see, hi) - 64;       // last tile that every row of the wave sees
            if (lo < hi_all) {
                fetch(lo);
                convert(lo, 0);
                ok = ok_next;
                __syncthreads();
                int buf = 0;
                for (int T0 = lo; T0 < hi_all; T0 += 64, buf ^= 1) {
                    if (T0 + 64 < hi_all) fetch(T0 + 64);
                    if (T0 < hi) use(T0 <= plain && ok == 15, T0, buf);
                    if (T0 + 64 < hi_all) convert(T0 + 64, buf ^ 1);
                    ok = ok_next;
                    __syncthreads();
                }
            }
        }

#pragma unroll
        for (int r = 0; r < R; ++r) {
            sum[r] += __shfl_xor(sum[r], 16);
            sum[r] += __shfl_xor(sum[r], 32);
        }

        // what a row's result becomes: a part, or the output
        auto put = [&](int row, int c0, const float* y, float mx, float sm) {      // channels [c0, c0 + 8) of row
            if (part >= 0) {
                const int64_t i = ((int64_t)part * a.c.heads + kvh) * l.rows + (row - b.begin);
                float* po = parts.o + i * D + c0;
                *reinterpret_cast<f32x4*>(po) = f32x4{y[0], y[1], y[2], y[3]};
                *reinterpret_cast<f32x4*>(po + 4) = f32x4{y[4], y[5], y[6], y[7]};
                if (c0 == 0) { parts.sums[2 * i] = mx; parts.sums[2 * i + 1] = sm; }
                return;
            }
            const int64_t at = place_of(a, b.row0, kvh, row);
            const float f = sm == 0.f ? 0.f : 1.f / sm;
            float z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = y[e] * f;
            if (a.g) {
                const E* gp = reinterpret_cast<const E*>(a.g) + at * D + c0;
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] *= sigmoidf_(to_f32(gp[e]));
            }
            E* op = reinterpret_cast<E*>(a.out) + at * D + c0;
            st4(op, f32x4{z[0], z[1], z[2], z[3]});
            st4(op + 4, f32x4{z[4], z[5], z[6], z[7]});
        };

        if constexpr (!SPLITW) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = row0 + 16 * r + n;
                if (row >= n_rows) continue;
                // element (j, v) of the result is channel PER g + VJ v + j
#pragma unroll
                for (int c = 0; c < PER; c += 8) {
                    float y[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] = o[r][(c + e) % VJ][(c + e) / VJ];
                    put(row, PER * g + c, y, m[r], sum[r]);
                }
            }
        } else {
            // join the waves' results, in their order
            if (g == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) { sm[wave][16 * r + n] = m[r]; ss[wave][16 * r + n] = sum[r]; }
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v)
#pragma unroll
                    for (int j = 0; j < VJ; j += 4)
                        *reinterpret_cast<f32x4*>(&so[wave][16 * r + n][PER * g + VJ * v + j]) =
                            f32x4{o[r][j][v], o[r][j + 1][v], o[r][j + 2][v], o[r][j + 3][v]};
            __syncthreads();
            const int here = min(ROWS, n_rows - row0);
            for (int i = threadIdx.x; i < here * (D / 8); i += kWaves * 64) {
                const int r = i / (D / 8), c0 = i % (D / 8) * 8;
                float mx = -INFINITY, sum_r = 0.f, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, sm[w][r]);
#pragma unroll
                for (int w = 0; w < kWaves; ++w) {
                    const float f = sm[w][r] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(sm[w][r] - mx);
                    sum_r += f * ss[w][r];
                    const f32x4 lo4 = *reinterpret_cast<const f32x4*>(&so[w][r][c0]), hi4 = *reinterpret_cast<const f32x4*>(&so[w][r][c0 + 4]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) { y[e] += f * lo4[e]; y[4 + e] += f * hi4[e]; }
                }
                put(row0 + r, c0, y, mx, sum_r);
            }
            __syncthreads();                // before the next block's results
        }
    }
}

// Joins the parts of the block that begins in a workgroup of the first kernel
// and goes on, row by row: weights 2^(m_i - max m).  WAVES waves take turns at
// the parts of a row, and their sums are joined through LDS in the order of
// the waves.
template <typename E, int D, int WAVES>
__global__ __launch_bounds__((WAVES > kWaves ? WAVES : kWaves) * 64) void kda_cache4_combine_kernel(Cache4AttentionArgs a, Layout l, Parts parts, int chunks) {
    constexpr int PER = D / 64;
    constexpr int ROWS = WAVES > kWaves ? 1 : kWaves / WAVES;      // rows of a workgroup at a time
    __shared__ __align__(16) float acc[ROWS * WAVES][D];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), turn = wave % WAVES;
    // chunks of rows, key/value heads, cuts
    const int chunk = (int)(blockIdx.x % chunks), kvh = (int)(blockIdx.x / chunks % a.c.heads);
    const Cut cut = parts.cut[blockIdx.x / chunks / a.c.heads];
    // bounded, so that a workspace that another call writes meanwhile gives
    // wrong values but no access outside the arrays
    const int w0 = cut.from, rows = min(l.rows, cut.n_rows - cut.begin);
    if (cut.n_rows <= 0 || cut.begin < 0 || w0 < 0 || w0 >= l.groups) return;
    const int count = min(cut.last, l.groups - 1) - w0 + 1;
    if (count < 2) return;
    for (int r = chunk * ROWS + wave / WAVES; r < rows; r += chunks * ROWS) {
        const int64_t stride = 2 * (int64_t)a.c.heads * l.rows;
        const int64_t first = ((int64_t)(2 * w0 + 1) * a.c.heads + kvh) * l.rows + r, rest = first - stride / 2;
        const int64_t at = place_of(a, cut.row0, kvh, cut.begin + r);
        if (at < 0 || at >= a.tokens * a.heads) return;
        auto place = [&](int i) { return i == 0 ? first : rest + i * stride; };
        auto sums = [&](int i) { return i < count ? *reinterpret_cast<const f32x2*>(parts.sums + 2 * place(i)) : f32x2{-INFINITY, 0.f}; };
        typedef typename std::conditional<PER == 2, f32x2, float>::type OV;
        auto part = [&](int i) { return *reinterpret_cast<const OV*>(parts.o + place(i) * D + lane * PER); };

        // the first parts are on their way while their weights are found
        constexpr int AHEAD = 8;
        f32x2 ms = sums(lane);
        OV x[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) x[k] = part(min(turn + k * WAVES, count - 1));
        E gate[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) gate[e] = a.g ? reinterpret_cast<const E*>(a.g)[at * D + lane * PER + e] : (E)0.f;
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
        float y[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            if constexpr (PER == 2) y[e] = o[e];
            else y[e] = o;
            y[e] = sum == 0.f ? 0.f : y[e] / sum;
            if (a.g) y[e] *= sigmoidf_(to_f32(gate[e]));
            reinterpret_cast<E*>(a.out)[at * D + lane * PER + e] = from_f32<E>(y[e]);
        }
    }
}

// Rows of a sequence and head up to which the waves of a workgroup share those
// of a block, of 16 or 32 rows.  64 sequences of 4096 tokens, 8 heads of 128: in
// bf16 32 rows take 78 us this way and 187 as many rows, 64 take 134 and 204, 96
// take 184 and 208; in fp32 32 take 143 and 218, 48 take 264 and 222.
constexpr int split_max_rows(bool bf16) { return bf16 ? 96 : 32; }
// bf16 rows of a wave in the many-rows form; fp32 takes three times the
// registers for its queries
constexpr int rows_r(bool bf16) { return bf16 ? 2 : 1; }

// 4 take 42 us for one head's 50000 tokens instead of 28, 16 take 24 but 22
// instead of 18 for 2 sequences of 4096 and 32 rows.
constexpr int kWideWaves = 8;

struct Plan {
    Layout l;
    bool splitw;
    int r;
};

Plan plan_of(bool bf16, int d, const Cache4AttentionArgs& a) {
    Plan p = {};
    const int64_t rows = a.group * (a.max_q < a.tokens ? a.max_q : a.tokens);
    p.splitw = rows <= split_max_rows(bf16);
    p.r = p.splitw ? (rows <= 16 ? 1 : 2) : rows_r(bf16);
    p.l.rows = p.splitw ? 16 * p.r : 16 * p.r * kWaves;
    p.l.per_seq = (a.group + p.l.rows - 1) / p.l.rows;
    // with or without offsets: enough slots for both
    const int64_t packed = a.tokens * a.group / p.l.rows + a.n_seq, plain = a.n_seq * p.l.per_seq;
    const int64_t slots = packed > plain ? packed : plain;
    p.l.slots = (int)(slots < INT32_MAX ? slots : INT32_MAX);
    // as many workgroups as run at once, but none for less than a unit of
    // every block's longest
    const int64_t cap = (int64_t)a.max_pages << a.c.page_shift;
    const int64_t len = a.max_len < cap ? a.max_len : cap;
    const int64_t units = (int64_t)p.l.slots * ((len + kUnit - 1) / kUnit + kBlockCost);
    // (twice as many groups in the many-rows form: 704 us instead of 686 for
    // 4 x 1000 tokens at the end of 8192)
    int64_t groups = (256 * (p.splitw && waves_of(bf16, d, p.r) == 3 ? 3 : 2) + a.c.heads - 1) / a.c.heads;
    groups = groups < units ? groups : units;
    const bool dealt = p.l.slots <= kMaxDealt && (int64_t)p.l.slots * (cap / kUnit + 1 + kBlockCost) <= kMaxUnits;
    p.l.groups = dealt ? (int)(groups < 1 ? 1 : groups) : 0;
    p.l.by_slot = p.l.slots < p.l.groups;
    return p;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int cuts(const Plan& p) { return p.l.by_slot ? p.l.slots : p.l.groups; }
size_t cut_bytes(const Plan& p) { return round256((size_t)cuts(p) * sizeof(Cut)); }
size_t part_places(const Cache4AttentionArgs& a, const Plan& p) {
    return 2 * (size_t)p.l.groups * (size_t)a.c.heads * (size_t)p.l.rows;
}

template <typename E, int D, int R, bool SPLITW>
hipError_t launch_attention_r(const Cache4AttentionArgs& a, const Plan& p, const Parts& parts, hipStream_t s) {
    const int64_t blocks = (int64_t)(p.l.groups > 0 ? p.l.groups : p.l.slots) * a.c.heads;
    const unsigned lds = (SPLITW ? 0u : (unsigned)shared_tiles(D)) + (p.l.groups > 0 ? (unsigned)(p.l.slots + 1) * (unsigned)(sizeof(int32_t) + sizeof(uint16_t)) : 0u);
    hipLaunchKernelGGL((kda_cache4_attention_kernel<E, D, R, SPLITW>), dim3((unsigned)blocks), dim3(kWaves * 64), lds, s, a, p.l,
                       parts);
    return hipGetLastError();
}

template <typename E, int D>
hipError_t launch_attention_t(const Cache4AttentionArgs& a, char* ws, hipStream_t s) {
    constexpr bool bf16 = sizeof(E) == 2;
    const Plan p = plan_of(bf16, D, a);
    Parts parts = {};
    if (p.l.groups > 0) {
        parts.cut = reinterpret_cast<Cut*>(ws);
        parts.o = reinterpret_cast<float*>(ws + cut_bytes(p));
        parts.sums = parts.o + part_places(a, p) * D;
    }
    hipError_t e;
    if (!p.splitw) e = launch_attention_r<E, D, rows_r(bf16), false>(a, p, parts, s);
    else if (p.r == 1) e = launch_attention_r<E, D, 1, true>(a, p, parts, s);
    else e = launch_attention_r<E, D, 2, true>(a, p, parts, s);
    if (e != hipSuccess || p.l.groups < 2) return e;
    // Where a block has many parts, kWideWaves waves share those of a row:
    // both kernels take 10.7 us instead of 13.3 for one of 4097 tokens (37
    // parts), 16 instead of 18 for 4 of 8192 (16 parts), 28 instead of 112 for
    // one head's 50000; with 4 parts 33 instead of 23 for 8 of 4096, 32 rows.
    const int64_t most = a.group * (a.max_q < a.tokens ? a.max_q : a.tokens);
    const int rows = (int)(most < p.l.rows ? most : p.l.rows);
    const bool wide = p.l.slots * 8 <= p.l.groups;
    const int chunks = wide ? rows : (rows + kWaves - 1) / kWaves;
    const dim3 grid((unsigned)(cuts(p) * a.c.heads * chunks));
    if (wide) hipLaunchKernelGGL((kda_cache4_combine_kernel<E, D, kWideWaves>), grid, dim3(kWideWaves * 64), 0, s, a, p.l, parts, chunks);
    else hipLaunchKernelGGL((kda_cache4_combine_kernel<E, D, 1>), grid, dim3(kWaves * 64), 0, s, a, p.l, parts, chunks);
    return hipGetLastError();
}

}  // namespace

bool cache4_attention_fits(bool bf16, int d, const Cache4AttentionArgs& a) {
    const Plan p = plan_of(bf16, d, a);
    return (int64_t)(p.l.groups > 0 ? p.l.groups : p.l.slots) * a.c.heads <= UINT32_MAX / (kWaves * 64);
}

size_t cache4_attention_workspace_bytes(bool bf16, int d, const Cache4AttentionArgs& a) {
    const Plan p = plan_of(bf16, d, a);
    if (p.l.groups == 0) return 0;
    return cut_bytes(p) + part_places(a, p) * (size_t)(d + 2) * sizeof(float);
}

hipError_t launch_cache4_attention(bool bf16, int d, const Cache4AttentionArgs& a, char* ws, hipStream_t s) {
    if (bf16) return d == 128 ? launch_attention_t<__bf16, 128>(a, ws, s) : launch_attention_t<__bf16, 64>(a, ws, s);
    return d == 128 ? launch_attention_t<float, 128>(a, ws, s) : launch_attention_t<float, 64>(a, ws, s);
}

}  // namespace kda

// kda_recurrence.hip -- a gated linear recurrence per channel, its gradients
// and its single-token step.
//
//   lambda = max(log_alpha, floor),  h_t = e^lambda_t h_(t-1) + x_t,
//   out_t = h_t sigmoid(g_t)
// and in reverse, with dh_t the gradient of h_t:
//   dh_t = d_out_t sigmoid(g_t) + e^lambda_(t+1) dh_(t+1)   (d_state at the end)
//   dx_t = dh_t,  dlog_alpha_t = dh_t e^lambda_t h_(t-1)    (0 where the floor binds)
//   dg_t = d_out_t h_t sigmoid'(g_t),  d_state_in = e^lambda_0 dh_0
//
// Both directions are bound by HBM (10 bytes an element forward, 18 in the
// training pass's backward, with a gate in bf16), so each reads its inputs
// once: a workgroup holds a tile of 128 or 64 tokens x 128 channels in
// registers while the state that enters it is found.  65536 tokens of 4096
// channels take 517 us (5.2 TB/s); 4 x 4096 tokens of 2048 92 us, backward 138
// (3.6 and 4.4 TB/s); 60000 of 256, where the chain of tiles bounds it, 81 and
// 126.  In fp32 the first take 841 us (5.1 TB/s), the second 131 and 182 (4.1 and
// 5.2).  Tiles of 64 tokens forward instead of 128 in bf16: 608 us for the first
// instead of 541 at the time, 100 instead of 91 for the second.
//  * A wave runs its stretch of the tile from nothing: (A, H), the product of
//    its decays and the state it ends with.  A stretch is the map
//    h -> A h + H; maps are joined through LDS.
//  * Every tile publishes its map, then its inclusive state h_out = A h_in + H
//    once h_in is known.  h_in is the last tile's h_out, or follows from an
//    earlier tile's h_out and the maps between, taken in the order of time:
//    the same operations whichever tile was ready, so results do not depend
//    on timing.  A look-back window of kWindow tiles lets the states run ahead
//    that many tiles per exchange between workgroups instead of one.
//  * The waves then run again from their true states and write the outputs.
// A sequence's first token starts its state anew, which makes the maps of its
// tile constant (no h_in): that is all that packed batches add, and uniform
// rows are sequences of their own.  The backward is the same in the other
// direction, with the states that enter the tiles kept by the forward call.
//
// Tiles are taken in the order of time off a counter, so a tile only ever
// waits for tiles that running workgroups have taken before it.
//
// A channel that remembers n tokens multiplies about n factors next to 1, so
// where |lambda| <= 1/16 a step is taken as h + (expm1(lambda) h + x):
// rounding e^lambda itself would cost half a step of fp32 per token, always
// the same way for a constant lambda.  Faster decays take e^lambda h + x, which
// leaves nothing of a large h that is forgotten.
#include "kda_common.hpp"
#include "kda_hybrid_internal.hpp"

namespace kda {

namespace {

// Tokens that a workgroup holds, and that its waves share.
constexpr int kTile = 128, kBackTile = 64;
// Tiles that a look-back reads at once.  With 4, 60000 tokens of 256 channels
// take 108 us instead of 81 (backward 188 instead of 128), with 16 68 (97), but
// the 64K tokens above 8% more than with 8, for its registers (in fp32 880 us
// instead of 838).
constexpr int kWindow = 8;
// Polls after which a wait gives up with NaN: a tenth of a second, where a tile takes
// microseconds.  Only a workspace that another call is using can get there.
constexpr int kMaxPolls = 1 << 17;

// The look-back words of one channel of a tile: the state in the low half,
// above it 0 (nothing yet), kFinal (the state is the tile's last one), or the
// product of the decays with its sign bit set (the tile's map).
constexpr uint32_t kFinal = 0xffffffffu;

template <typename E, int N> struct VecOf { typedef E type __attribute__((ext_vector_type(N))); };
template <typename E> struct VecOf<E, 1> { typedef E type; };
template <int N, typename V> __device__ __forceinline__ float lane_of(V v, int i) {
    if constexpr (N == 1) return to_f32(v);
    else return to_f32(v[i]);
}
// N elements as one access, at any multiple of the element's size: rows of an
// odd width do not keep pairs aligned.
template <typename E, int N>
__device__ __forceinline__ typename VecOf<E, N>::type get(const E* p) {
    typename VecOf<E, N>::type v;
    __builtin_memcpy(&v, p, N * sizeof(E));
    return v;
}
template <typename E, int N>
__device__ __forceinline__ void put(E* p, const float (&x)[N]) {
    typename VecOf<E, N>::type v;
    if constexpr (N == 1) {
        v = from_f32<E>(x[0]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = from_f32<E>(x[i]);
    }
    __builtin_memcpy(p, &v, N * sizeof(E));
}

// The least that a decay counts as: e^lambda of a finite lambda is no 0, so that
// an infinite state stays infinite however fast it decays, while a finite one
// leaves less than 2^-20.  Only lambda = -inf leaves nothing, and NaN of Inf.
constexpr float kLeast = 1.40129846e-45f;        // 2^-149

// One token's decay, of lambda = max(log_alpha, floor): `c` is expm1(lambda)
// where `slow` and e^lambda elsewhere.  expm1 is the Taylor series to the 5th
// power (the rest is below 2^-29 of the value), e^lambda the hardware exp2.
struct Decay {
    float c;
    bool slow;
    __device__ __forceinline__ explicit Decay(float x) {
        float p = 1.f / 120.f;
        p = fmaf(p, x, 1.f / 24.f);
        p = fmaf(p, x, 1.f / 6.f);
        p = fmaf(p, x, 0.5f);
        p = fmaf(p * x, x, x);
        slow = fabsf(x) <= 0.0625f;
        // 0 times -inf is NaN, which the maximum leaves out
        c = slow ? p : fmaxf(__builtin_amdgcn_exp2f(1.4426950408889634f * x), fmaf(0.f, x, kLeast));
    }
    __device__ __forceinline__ Decay(float c_, bool slow_) : c(c_), slow(slow_) {}
    // What expm1(lambda) multiplies: of an infinite state the largest number, as
    // -Inf or NaN beside the state itself would be NaN.  (This and kLeast cost
    // the 64K tokens above 4 us.)
    __device__ __forceinline__ float part(float h) const {
        return slow ? __builtin_amdgcn_fmed3f(h, -3.40282347e38f, 3.40282347e38f) : h;
    }
    // e^lambda h, and e^lambda h + x
    __device__ __forceinline__ float times(float h) const { return fmaf(c, part(h), slow ? h : 0.f); }
    __device__ __forceinline__ float step(float h, float x) const { return fmaf(c, part(h), x) + (slow ? h : 0.f); }
};

// e^sum; next to 1 rounded from 1 + expm1, since the hardware exp2 falls short
// of it there, which a long chain of stretches adds up.
__device__ __forceinline__ float product_of(float sum) {
    const Decay d(sum);
    return d.slow ? 1.f + d.c : d.c;
}

// The product of two decays, which vanishes only where one of them does.
__device__ __forceinline__ float both(float a, float b) { return fmaxf(a * b, fminf(fminf(a, b), kLeast)); }

// The sequence of a token, walked along the tokens of one wave (all of it the
// same in every lane).
struct Walk {
    const int32_t* cu;      // null: one sequence, the whole row
    int n, T;
    int s, first, end;      // sequence s holds tokens [first, end)
    __device__ __forceinline__ void bounds() {
        int64_t b, e;
        seq_bounds(cu, s, T, b, e);
        first = (int)b; end = (int)e;
    }
    // at token t or the next one that has a sequence
    __device__ __forceinline__ Walk(const RecurrenceArgs& a, int row, int t)
        : cu(a.cu_seqlens), n((int)a.n_seq), T((int)a.T), s(row), first(0), end((int)a.T) {
        if (!cu) return;
        // The last sequence that begins at or before t, 64 candidates at a
        // time in the lanes: one load of latency up to 64 sequences, two up
        // to 4096.
        int lo = 0, many = n;
        while (many > 1) {
            const int stride = (many + 63) / 64, at = lo + (int)(threadIdx.x & 63) * stride;
            const bool before = at < lo + many && cu[at] <= t;
            const int k = __popcll(__ballot(before));
            const int next = lo + (k > 0 ? k - 1 : 0) * stride;
            many = min(stride, lo + many - next);
            lo = next;
        }
        s = lo;
        bounds();
    }
    __device__ __forceinline__ void go_to(int s_) {
        if (s == s_) return;
        s = s_;
        bounds();
    }
    // Whether tokens [t, t + n) lie within one sequence, neither its first nor
    // its last token among them.
    __device__ __forceinline__ bool inside(int t, int n) const { return t > first && t + n < end; }
    // The last of sequences [lo, hi) that begins at or before t; lo if none
    // does.  (Not in the lanes: some may have left by then.)
    __device__ __forceinline__ void find(int t, int lo, int hi) {
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t) lo = mid; else hi = mid;
        }
        s = lo;
        bounds();
    }
    // Whether a sequence holds token t, for t going up, and going down.  Mostly
    // the next sequence does; over empty ones, of which there may be any number
    // at one place, it is searched.
    __device__ __forceinline__ bool up(int t) {
        if (cu && t >= end && s + 1 < n) {
            ++s;
            bounds();
            if (t >= end && s + 1 < n) find(t, s, n);
        }
        return t >= first && t < end;
    }
    __device__ __forceinline__ bool down(int t) {
        if (cu && t < first && s > 0) {
            --s;
            bounds();
            if (t < first && s > 0) find(t, 0, s);
        }
        return t >= first && t < end;
    }
};

// The channels [c, c + VEC) of a lane.  Where the width is odd, the second lane
// of all begins one channel early: it and the first compute and write the same
// values of channel 1.  Both are of one wave, which has read what it needs of
// the states before it writes any, as state_out may be state_in.  Lanes behind
// the last channel (in false) work on the last ones, without writing.
struct Channels {
    int64_t c;
    bool in;
};
template <int VEC>
__device__ __forceinline__ Channels channels_of(int64_t D, int64_t block, int lane) {
    static_assert(VEC <= 2, "an odd width shares one channel");
    int64_t c = (block * 64 + lane) * VEC;
    if (VEC == 2 && c > 0 && (D & 1)) --c;
    return Channels{c + VEC <= D ? c : D - VEC, c + VEC <= D};
}

struct TileGrid {
    int64_t tiles;          // per row
    int64_t lanes;          // rows x channel blocks: tiles of one time
    int blocks;             // channel blocks of a row
    __host__ __device__ int64_t total() const { return tiles * lanes; }
};

__device__ __forceinline__ uint64_t word(uint32_t high, float h) { return (uint64_t)high << 32 | __float_as_uint(h); }

// One channel's part of a tile's map, as published.
__device__ __forceinline__ uint64_t map_word(float A, float H) {
    return word(A != A ? 0xffc00000u : __float_as_uint(A) | 0x80000000u, H);
}

__device__ __forceinline__ void publish(uint64_t* p, uint64_t w) {
    __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state that leaves tile i - 1 in the order of the scan, for a lane's
// channel: words + k * stride is its word of tile i - 1 - k, k < i.
__device__ __forceinline__ float look_back(const uint64_t* words, int64_t stride, int64_t i) {
    const int64_t most = i < kWindow ? i : kWindow;
    float h = 0.f;
    bool have = false;
    for (int polls = 0; polls < kMaxPolls; ++polls) {
        uint64_t w[kWindow];
#pragma unroll
        for (int k = 0; k < kWindow; ++k)
            w[k] = k < most ? __hip_atomic_load(const_cast<uint64_t*>(words) + k * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0;
        have = false;
#pragma unroll
        for (int k = kWindow - 1; k >= 0; --k) {           // from the earliest tile on
            const uint32_t high = (uint32_t)(w[k] >> 32);
            const float H = __uint_as_float((uint32_t)w[k]);
            const bool final = high == kFinal;
            h = final ? H : fmaf(__uint_as_float(high & 0x7fffffffu), h, H);
            have = final || (have && high != 0);
        }
        if (__all(have)) return h;
        __builtin_amdgcn_s_sleep(1);
    }
    return have ? h : __uint_as_float(0x7fc00000u);
}

// Where a workgroup works: a tile taken off the counter where tiles wait for
// each other, else its own index.  False: nothing left.
__device__ __forceinline__ bool take_tile(const TileGrid& g, int32_t* counter, int32_t* lds, int64_t& id) {
    id = blockIdx.x;
    if (g.tiles > 1) {
        if (threadIdx.x == 0) *lds = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        id = __builtin_amdgcn_readfirstlane(*lds);
    }
    return id >= 0 && id < g.total();
}

template <typename E, int VEC, int WAVES, bool GATE>
__global__ __launch_bounds__(WAVES * 64, 4) void kda_recurrence_kernel(RecurrenceArgs a, TileGrid grid, int32_t* counter,
                                                                       uint64_t* words, float* keep) {
    constexpr int TPW = kTile / WAVES;
    static_assert(TPW * VEC <= 32 && kBackTile % TPW == 0, "one flag a value; a kept state between waves");
    typedef typename VecOf<E, VEC>::type EV;
    typedef typename VecOf<float, VEC>::type FV;
    __shared__ float sA[WAVES][64 * VEC], sH[WAVES][64 * VEC], sIn[64 * VEC];
    __shared__ int32_t sCut[WAVES], sId;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t id;
    if (!take_tile(grid, counter, &sId, id)) return;
    const int64_t i = id / grid.lanes, row = (id % grid.lanes) / grid.blocks;
    const Channels ch = channels_of<VEC>(a.D, id % grid.blocks, lane);
    const int64_t c = ch.c;
    const int t0 = (int)(i * kTile) + wave * TPW;

    Walk walk(a, (int)row, t0);
    EV x[TPW], g[TPW];
    float d[TPW][VEC];
    const int64_t base = row * a.T;
#pragma unroll
    for (int j = 0; j < TPW; ++j) {
        const int64_t t = t0 + j < (int)a.T ? t0 + j : (int)a.T - 1, at = (base + t) * a.D + c;
        x[j] = get<E, VEC>(reinterpret_cast<const E*>(a.x) + at);
        const FV l = get<float, VEC>(a.log_alpha + at);
        if constexpr (GATE) g[j] = get<E, VEC>(reinterpret_cast<const E*>(a.g) + at);
#pragma unroll
        for (int v = 0; v < VEC; ++v) d[j][v] = lane_of<VEC>(l, v);
    }

    // this wave's map
    float h[VEC], sum[VEC];
    uint32_t slow = 0;
    bool cut = false;
    const int s0 = walk.s;
    const bool plain = walk.inside(t0, TPW);
#pragma unroll
    for (int v = 0; v < VEC; ++v) { h[v] = 0.f; sum[v] = 0.f; }
    auto token = [&](int j, bool start) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float l = fmaxf(d[j][v], a.floor_);
            const Decay k(l);
            sum[v] += l;
            slow |= (uint32_t)k.slow << (j * VEC + v);
            h[v] = k.step(h[v], lane_of<VEC>(x[j], v));
            // state_in is read once: state_out may be the same array
            d[j][v] = start ? h[v] : k.c;
        }
    };
    if (plain) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) token(j, false);
    } else {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int t = t0 + j;
            if (t < (int)a.T && walk.up(t)) {
                if (t == walk.first) {
                    cut = true;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) h[v] = a.state_in ? a.state_in[(int64_t)walk.s * a.D + c + v] : 0.f;
                }
                token(j, t == walk.first);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        sA[wave][lane * VEC + v] = product_of(sum[v]);
        sH[wave][lane * VEC + v] = h[v];
    }
    if (lane == 0) sCut[wave] = cut;
    __syncthreads();

    // The tile's map, and the state that enters it: wave v has channel c + v.
    // (One wave with both took twice the registers beside its tokens: the 64K
    // tokens above 541 us instead of 507.)
    if (wave < VEC) {
        const int at = lane * VEC + wave;
        float A = 1.f, H = 0.f, hin = 0.f;
        bool constant = false;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const bool cw = sCut[w] != 0;
            constant = constant || cw;
            H = cw ? sH[w][at] : fmaf(sA[w][at], H, sH[w][at]);
            A = both(A, sA[w][at]);
        }
        if (grid.tiles > 1) {
            uint64_t* mine = words + (row * grid.tiles + i) * a.D + c + wave;
            const bool tells = ch.in && i + 1 < grid.tiles;
            if (tells) publish(mine, constant ? word(kFinal, H) : map_word(A, H));
            if (i > 0) hin = look_back(mine - a.D, -a.D, i);
            if (tells && !constant) publish(mine, word(kFinal, fmaf(A, hin, H)));
        }
        sIn[at] = hin;
    }
    __syncthreads();

    // again from the true state
    if (!ch.in) return;
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = sIn[lane * VEC + v];
    for (int w = 0; w < wave; ++w) {
        const bool cw = sCut[w] != 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float Hw = sH[w][lane * VEC + v];
            h[v] = cw ? Hw : fmaf(sA[w][lane * VEC + v], h[v], Hw);
        }
    }
    if (a.keep && wave * TPW % kBackTile == 0 && t0 < (int)a.T) {
        const int64_t back_tiles = (a.T + kBackTile - 1) / kBackTile;
#pragma unroll
        for (int v = 0; v < VEC; ++v) keep[(row * back_tiles + t0 / kBackTile) * a.D + c + v] = h[v];
    }
    auto write = [&](int j, bool start) {
        float y[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            h[v] = start ? d[j][v] : Decay(d[j][v], slow >> (j * VEC + v) & 1u).step(h[v], lane_of<VEC>(x[j], v));
            y[v] = h[v];
            if constexpr (GATE) y[v] *= sigmoidf_(lane_of<VEC>(g[j], v));
        }
        put<E, VEC>(reinterpret_cast<E*>(a.out) + (base + t0 + j) * a.D + c, y);
    };
    if (plain) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) write(j, false);
    } else {
        walk.go_to(s0);
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int t = t0 + j;
            if (t < (int)a.T && walk.up(t)) {
                write(j, t == walk.first);
                if (a.state_out && t == walk.end - 1) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a.state_out[(int64_t)walk.s * a.D + c + v] = h[v];
                }
            }
        }
    }
}

template <typename E, int VEC, int WAVES, bool GATE>
__global__ __launch_bounds__(WAVES * 64, 4) void kda_recurrence_backward_kernel(RecurrenceArgs a, TileGrid grid, int32_t* counter,
                                                                                uint64_t* words, const float* keep) {
    constexpr int TPW = kBackTile / WAVES;
    static_assert(TPW * VEC <= 32, "one flag a value");
    typedef typename VecOf<E, VEC>::type EV;
    typedef typename VecOf<float, VEC>::type FV;
    __shared__ float sA[WAVES][64 * VEC], sH[WAVES][64 * VEC], sC[WAVES][64 * VEC], sIn[64 * VEC];
    __shared__ int32_t sFirst[WAVES], sLast[WAVES], sId;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int64_t id;
    if (!take_tile(grid, counter, &sId, id)) return;
    const int64_t i = grid.tiles - 1 - id / grid.lanes, row = (id % grid.lanes) / grid.blocks;
    const Channels ch = channels_of<VEC>(a.D, id % grid.blocks, lane);
    const int64_t c = ch.c;
    const int t0 = (int)(i * kBackTile) + wave * TPW;

    Walk walk(a, (int)row, t0);
    EV x[TPW], g[TPW], o[TPW];
    float d[TPW][VEC];
    const int64_t base = row * a.T;
#pragma unroll
    for (int j = 0; j < TPW; ++j) {
        const int64_t t = t0 + j < (int)a.T ? t0 + j : (int)a.T - 1, at = (base + t) * a.D + c;
        x[j] = get<E, VEC>(reinterpret_cast<const E*>(a.x) + at);
        const FV l = get<float, VEC>(a.log_alpha + at);
        if constexpr (GATE) g[j] = get<E, VEC>(reinterpret_cast<const E*>(a.g) + at);
        o[j] = EV(0);
        if (a.d_out) o[j] = get<E, VEC>(reinterpret_cast<const E*>(a.d_out) + at);
#pragma unroll
        for (int v = 0; v < VEC; ++v) d[j][v] = lane_of<VEC>(l, v);
    }
    float enter[VEC];                             // the state that enters the tile
#pragma unroll
    for (int v = 0; v < VEC; ++v) enter[v] = i > 0 ? keep[(row * grid.tiles + i) * a.D + c + v] : 0.f;

    // this wave's maps, of the state forward and of its gradient in reverse
    float h[VEC], e[VEC], sum[VEC];
    uint32_t slow = 0, free_ = 0;                 // free_: the floor does not bind
    bool first = false, last = false;
    const int s0 = walk.s;
    const bool plain = walk.inside(t0, TPW);
#pragma unroll
    for (int v = 0; v < VEC; ++v) { h[v] = 0.f; e[v] = 0.f; sum[v] = 0.f; }
    auto up = [&](int j) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float l = fmaxf(d[j][v], a.floor_);
            free_ |= (uint32_t)(d[j][v] > a.floor_) << (j * VEC + v);
            const Decay k(l);
            sum[v] += l;
            d[j][v] = k.c;
            slow |= (uint32_t)k.slow << (j * VEC + v);
            h[v] = k.step(h[v], lane_of<VEC>(x[j], v));
        }
    };
    auto down = [&](int j) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float s = GATE ? sigmoidf_(lane_of<VEC>(g[j], v)) : 1.f;
            e[v] = Decay(d[j][v], slow >> (j * VEC + v) & 1u).times(fmaf(lane_of<VEC>(o[j], v), s, e[v]));
        }
    };
    if (plain) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) up(j);
#pragma unroll
        for (int j = TPW - 1; j >= 0; --j) down(j);
    } else {
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int t = t0 + j;
            if (t < (int)a.T && walk.up(t)) {
                if (t == walk.first) {
                    first = true;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) h[v] = a.state_in ? a.state_in[(int64_t)walk.s * a.D + c + v] : 0.f;
                }
                up(j);
            }
        }
    }
    const int s1 = walk.s;
    if (!plain) {
#pragma unroll
        for (int j = TPW - 1; j >= 0; --j) {
            const int t = t0 + j;
            if (t < (int)a.T && walk.down(t)) {
                if (t == walk.end - 1) {
                    last = true;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) e[v] = a.d_state ? a.d_state[(int64_t)walk.s * a.D + c + v] : 0.f;
                }
                down(j);
            }
        }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
        sA[wave][lane * VEC + v] = product_of(sum[v]);
        sH[wave][lane * VEC + v] = h[v];
        sC[wave][lane * VEC + v] = e[v];
    }
    if (lane == 0) { sFirst[wave] = first; sLast[wave] = last; }
    __syncthreads();

    // the tile's map of the gradient, and the gradient that enters it from behind
    if (wave < VEC) {
        const int at = lane * VEC + wave;
        float A = 1.f, C = 0.f, ein = 0.f;
        bool constant = false;
#pragma unroll
        for (int w = WAVES - 1; w >= 0; --w) {
            const bool cw = sLast[w] != 0;
            constant = constant || cw;
            C = cw ? sC[w][at] : fmaf(sA[w][at], C, sC[w][at]);
            A = both(A, sA[w][at]);
        }
        if (grid.tiles > 1) {
            uint64_t* mine = words + (row * grid.tiles + i) * a.D + c + wave;
            const int64_t behind = grid.tiles - 1 - i;
            const bool tells = ch.in && i > 0;
            if (tells) publish(mine, constant ? word(kFinal, C) : map_word(A, C));
            if (behind > 0) ein = look_back(mine + a.D, a.D, behind);
            if (tells && !constant) publish(mine, word(kFinal, fmaf(A, ein, C)));
        }
        sIn[at] = ein;
    }
    __syncthreads();
    if (!ch.in) return;

    // the states before each token
    float before[TPW][VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = enter[v];
    for (int w = 0; w < wave; ++w) {
        const bool cw = sFirst[w] != 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float Hw = sH[w][lane * VEC + v];
            h[v] = cw ? Hw : fmaf(sA[w][lane * VEC + v], h[v], Hw);
        }
    }
    auto again = [&](int j) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            before[j][v] = h[v];
            h[v] = Decay(d[j][v], slow >> (j * VEC + v) & 1u).step(h[v], lane_of<VEC>(x[j], v));
        }
    };
    // the gradients, from the one that enters the wave's stretch from behind
#pragma unroll
    for (int v = 0; v < VEC; ++v) e[v] = sIn[lane * VEC + v];
    for (int w = WAVES - 1; w > wave; --w) {
        const bool cw = sLast[w] != 0;
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const float Cw = sC[w][lane * VEC + v];
            e[v] = cw ? Cw : fmaf(sA[w][lane * VEC + v], e[v], Cw);
        }
    }
    auto write = [&](int j) {
        float dx[VEC], dl[VEC], dg[VEC];
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
            const Decay k(d[j][v], slow >> (j * VEC + v) & 1u);
            const float dy = lane_of<VEC>(o[j], v);
            float s = 1.f;
            if constexpr (GATE) {
                s = sigmoidf_(lane_of<VEC>(g[j], v));
                dg[v] = dy * k.step(before[j][v], lane_of<VEC>(x[j], v)) * s * (1.f - s);
            }
            dx[v] = fmaf(dy, s, e[v]);
            e[v] = k.times(dx[v]);
            dl[v] = free_ >> (j * VEC + v) & 1u ? e[v] * before[j][v] : 0.f;
        }
        const int64_t at = (base + t0 + j) * a.D + c;
        put<E, VEC>(reinterpret_cast<E*>(a.dx) + at, dx);
        put<float, VEC>(a.dlog_alpha + at, dl);
        if constexpr (GATE) put<E, VEC>(reinterpret_cast<E*>(a.dg) + at, dg);
    };
    if (plain) {
#pragma unroll
        for (int j = 0; j < TPW; ++j) again(j);
#pragma unroll
        for (int j = TPW - 1; j >= 0; --j) write(j);
    } else {
        walk.go_to(s0);
#pragma unroll
        for (int j = 0; j < TPW; ++j) {
            const int t = t0 + j;
            if (t < (int)a.T && walk.up(t)) {
                if (t == walk.first) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) h[v] = a.state_in ? a.state_in[(int64_t)walk.s * a.D + c + v] : 0.f;
                }
                again(j);
            }
        }
        walk.go_to(s1);
#pragma unroll
        for (int j = TPW - 1; j >= 0; --j) {
            const int t = t0 + j;
            if (t < (int)a.T && walk.down(t)) {
                if (t == walk.end - 1) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) e[v] = a.d_state ? a.d_state[(int64_t)walk.s * a.D + c + v] : 0.f;
                }
                write(j);
                if (a.d_state_in && t == walk.first) {
#pragma unroll
                    for (int v = 0; v < VEC; ++v) a.d_state_in[(int64_t)walk.s * a.D + c + v] = e[v];
                }
            }
        }
    }
}

// Before a scan: no tile taken, nothing published; and the sequences without
// a token, which no tile sees, pass their state through (to may be from).
__global__ __launch_bounds__(kThreads) void kda_recurrence_begin_kernel(uint64_t* clear, int64_t n_clear, const int32_t* cu,
                                                                        int64_t n_seq, int64_t T, int64_t D,
                                                                        const float* from, float* to) {
    const int64_t step = (int64_t)gridDim.x * kThreads, at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    for (int64_t k = at; k < n_clear; k += step) clear[k] = 0;
    if (!to) return;
    for (int64_t s = blockIdx.x; s < n_seq; s += gridDim.x) {
        int64_t b = 0, e = T;
        if (cu) seq_bounds(cu, s, T, b, e);
        if (e > b) continue;
        for (int64_t c = threadIdx.x; c < D; c += kThreads) to[s * D + c] = from ? from[s * D + c] : 0.f;
    }
}

// N elements from i on (aligned to N of them).
template <typename E, int N>
__device__ __forceinline__ void step_elements(const RecurrenceStepArgs& a, int64_t i) {
    const auto x = get<E, N>(reinterpret_cast<const E*>(a.x) + i);
    const auto l = get<float, N>(a.log_alpha + i), h0 = get<float, N>(a.state + i);
    auto g = x;
    if (a.g) g = get<E, N>(reinterpret_cast<const E*>(a.g) + i);
    float h[N], y[N];
#pragma unroll
    for (int v = 0; v < N; ++v) {
        h[v] = Decay(fmaxf(lane_of<N>(l, v), a.floor_)).step(lane_of<N>(h0, v), lane_of<N>(x, v));
        y[v] = a.g ? h[v] * sigmoidf_(lane_of<N>(g, v)) : h[v];
    }
    put<float, N>(a.state + i, h);
    put<E, N>(reinterpret_cast<E*>(a.out) + i, y);
}

// Bound by HBM, by latency when small (256 x 4096 in bf16 with a gate, 18 MB:
// 5 us): four elements a thread, the last ones one by one.
template <typename E>
__global__ __launch_bounds__(kThreads) void kda_recurrence_step_kernel(RecurrenceStepArgs a) {
    const int64_t i = 4 * ((int64_t)blockIdx.x * kThreads + threadIdx.x);
    if (i + 4 <= a.n) step_elements<E, 4>(a, i);
    else
        for (int64_t k = i; k < a.n; ++k) step_elements<E, 1>(a, k);
}

int64_t tiles_of(int64_t T, int tile) { return (T + tile - 1) / tile; }

// The workspace: the counter (its own 256 bytes), the look-back words, then
// for training the state that enters every tile of the backward.  One tile a
// row needs none.
size_t words_bytes(int64_t B, int64_t T, int64_t D, int tile) {
    return tiles_of(T, tile) > 1 ? ((size_t)(B * tiles_of(T, tile)) * (size_t)D * 8 + 255) / 256 * 256 : 0;
}
constexpr size_t kCounterBytes = 256;

// Tokens of a wave: 16 in bf16, 8 in fp32, whose registers hold half as many
// (16 in fp32 spill with a gate: 978 us instead of 838 for 65536 x 4096; without
// one 37 instead of 38 for 16384 x 515, 29 instead of 32 for 16384 x 512).
template <typename E> constexpr int kForwardWaves = sizeof(E) == 2 ? 8 : 16;
constexpr int kBackwardWaves = 8;

template <typename E, int VEC, bool GATE>
hipError_t launch_scan_v(const RecurrenceArgs& a, bool backward, hipStream_t s) {
    TileGrid g;
    g.tiles = tiles_of(a.T, backward ? kBackTile : kTile);
    g.blocks = (int)((a.D + 64 * VEC - 1) / (64 * VEC));
    g.lanes = a.B * g.blocks;
    int32_t* counter = reinterpret_cast<int32_t*>(a.ws);
    uint64_t* words = reinterpret_cast<uint64_t*>(a.ws + kCounterBytes);
    // behind the words of the backward, of which there are more
    float* keep = reinterpret_cast<float*>(a.ws + kCounterBytes + words_bytes(a.B, a.T, a.D, kBackTile));
    if (backward)
        hipLaunchKernelGGL((kda_recurrence_backward_kernel<E, VEC, kBackwardWaves, GATE>), dim3((unsigned)g.total()),
                           dim3(kBackwardWaves * 64), 0, s, a, g, counter, words, keep);
    else
        hipLaunchKernelGGL((kda_recurrence_kernel<E, VEC, kForwardWaves<E>, GATE>), dim3((unsigned)g.total()),
                           dim3(kForwardWaves<E> * 64), 0, s, a, g, counter, words, keep);
    return hipGetLastError();
}

template <typename E>
hipError_t launch_scan_t(RecurrenceArgs a, bool backward, hipStream_t s) {
    if (a.T <= kBackTile) a.keep = false;      // one tile: entered from state_in alone
    const int tile = backward ? kBackTile : kTile;
    const float* from = backward ? a.d_state : a.state_in;
    float* to = backward ? a.d_state_in : a.state_out;
    const bool empties = to && (a.cu_seqlens || a.T == 0);
    const int64_t n_clear = a.T > tile ? (int64_t)((kCounterBytes + words_bytes(a.B, a.T, a.D, tile)) / 8) : 0;
    if (n_clear > 0 || empties) {
        int64_t blocks = (n_clear + 8 * kThreads - 1) / (8 * kThreads);
        if (empties && a.n_seq > blocks) blocks = a.n_seq;
        blocks = blocks > 2048 ? 2048 : blocks;
        hipLaunchKernelGGL(kda_recurrence_begin_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s,
                           reinterpret_cast<uint64_t*>(a.ws), n_clear, a.cu_seqlens, a.n_seq, a.T, a.D, from,
                           empties ? to : nullptr);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    if (a.B == 0 || a.T == 0) return hipSuccess;
    if (a.D == 1) return a.g ? launch_scan_v<E, 1, true>(a, backward, s) : launch_scan_v<E, 1, false>(a, backward, s);
    return a.g ? launch_scan_v<E, 2, true>(a, backward, s) : launch_scan_v<E, 2, false>(a, backward, s);
}

}  // namespace

size_t recurrence_workspace_bytes(int64_t B, int64_t T, int64_t D, bool backward) {
    const int tile = backward ? kBackTile : kTile;
    if (B == 0 || T <= tile) return 0;
    return kCounterBytes + words_bytes(B, T, D, tile) + (backward ? (size_t)(B * tiles_of(T, tile)) * (size_t)D * sizeof(float) : 0);
}

hipError_t launch_recurrence(bool bf16, const RecurrenceArgs& a, hipStream_t s) {
    return bf16 ? launch_scan_t<__bf16>(a, false, s) : launch_scan_t<float>(a, false, s);
}

hipError_t launch_recurrence_backward(bool bf16, const RecurrenceArgs& a, hipStream_t s) {
    return bf16 ? launch_scan_t<__bf16>(a, true, s) : launch_scan_t<float>(a, true, s);
}

hipError_t launch_recurrence_step(bool bf16, const RecurrenceStepArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)((a.n + 4 * kThreads - 1) / (4 * kThreads)));
    if (bf16) hipLaunchKernelGGL(kda_recurrence_step_kernel<__bf16>, grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL(kda_recurrence_step_kernel<float>, grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace kda

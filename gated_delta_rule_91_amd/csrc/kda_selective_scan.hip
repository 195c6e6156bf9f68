// kda_selective_scan.hip -- a selective state space of N states a channel, its
// gradients and its single-token step.
//
//   delta_t = softplus(dt_t + dt_bias),  a_t[n] = exp(delta_t A[n])
//   h_t[n] = a_t[n] h_(t-1)[n] + delta_t x_t B_t[n]
//   y_t = sum_n C_t[n] h_t[n] + skip x_t,  out_t = y_t silu(z_t)
// and in reverse, with dy_t = d_out_t silu(z_t) and r_t the gradient of h_t that
// comes from later tokens (d_state at the end):
//   dh_t = C_t dy_t + r_t,  r_(t-1) = a_t dh_t
//   dx_t = delta_t sum_n dh_t B_t + skip dy_t
//   ddelta_t = x_t sum_n dh_t B_t + sum_n A r_(t-1) h_(t-1),  ddt = ddelta sigmoid(dt + dt_bias)
//   dA = sum_t delta_t r_(t-1) h_(t-1),  dB_t = sum_d dh_t delta_t x_t,  dC_t = sum_d dy_t h_t
//
// Every channel and state fades at its own speed, so there is no matrix product
// in it: it is bound by the vector unit, by an exponential and some four
// operations for each of N states of an element.  A lane has a channel with all
// its states in registers; B and C, the same for all channels, come through the
// scalar cache as scalar operands.  On average the vector unit is busy 92 to 96% of
// the time forward and 73% backward, where sums over channels and two waves a SIMD
// leave gaps.
//
// 65536 tokens of 2048 channels and 16 states, bf16 with a gate, take 458 us for
// step 1, 11 for step 2 and 542 for step 3 (861 for a call among others, at the
// clock that it has then); 16384 x 515 x 8 in fp32, packed, 27 + 9 + 31.  A training
// pass of 4 x 4096 x 2048 x 16 takes 116 + 9 + 160 forward, where step 3 keeps states,
// and 105 + 11 + 516 + 19 backward.  A step of 256 x 4096 x 16 takes 26 us, 5.5 TB/s.
//
// Time is split into tiles, a wave each, where there are too few channels to
// fill the card:
//  1. each tile's state from nothing, sum_t exp(A sum_(s>t) delta_s) delta_t x_t B_t:
//     taken from the last token back, so that no step depends on the one before;
//  2. the tiles' states are joined in order, h <- exp(A sum delta) h + state;
//  3. each tile runs from its true state and writes the outputs.
// The backward does the same from the other end.  A sequence's first token
// starts its state anew, so a tile that holds one hands on a state of its own.
#include <type_traits>

#include "kda_packed.hpp"
#include "kda_selective_internal.hpp"

namespace kda {

namespace {

constexpr int kScanWaves = 4;
constexpr int kXcds = 8;             // a launch over tiles has a multiple of as many workgroups
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.69314718055994531f;
// A tile whose incoming state does not reach its end has this for its sum of delta.
constexpr float kCut = -1.f;

// How time and channels are split (host and kernels).
struct ScanGrid {
    int tile, tiles;     // tokens of a tile, tiles of a row
    int blocks;          // of 64 channels
};

// Tokens between the states that a forward call keeps for the backward, which
// forms the states between them anew in registers.  With half as many the backward
// takes 508 us instead of 517 for 4 x 4096 x 2048 x 16, but the forward 179 instead of
// 162 and the workspace doubles.
template <int N> constexpr int kKeep = 128 / N;

// The states of sequences without tokens, and their gradients, go through: what
// the workgroups behind those of the tiles do, a wave for each sequence.
template <int N>
__device__ __forceinline__ void pass_through(const SelectiveArgs& a, int64_t block, const float* from, float* to) {
    const int64_t s = block * kScanWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), each = a.D * N;
    if (s >= a.n_seq) return;
    int64_t first = 0, end = a.T;
    if (a.cu_seqlens) seq_bounds(a.cu_seqlens, s, a.T, first, end);
    if (first < end) return;
    for (int64_t i = (threadIdx.x & 63) * 4; i < each; i += 256)
        *reinterpret_cast<f32x4*>(to + s * each + i) = from ? *reinterpret_cast<const f32x4*>(from + s * each + i) : f32x4{0.f, 0.f, 0.f, 0.f};
}

struct Place {
    int row, i, block;   // of batch, tile, channel block
    int t0, t1;
    uint32_t c;          // a lane's channel, the last one where it has none
    bool in;             // whether it has
    bool any;
    int64_t at;          // index of (row, tile, block)
};
// `blocks`: workgroups of the tiles, a multiple of kXcds.
__device__ __forceinline__ Place place_of(const SelectiveArgs& a, const ScanGrid& g, unsigned blocks, int skipped_tiles = 0, int first_tile = 0) {
    // Workgroups go to the XCDs in turn: each XCD gets a stretch of them, so that
    // those of a tile, which read the same rows of B and C, share its L2.
    const int64_t block = (int64_t)(blockIdx.x % kXcds) * (blocks / kXcds) + blockIdx.x / kXcds;
    const int64_t w = block * kScanWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = g.tiles - skipped_tiles;
    Place p;
    p.block = (int)(w % g.blocks);
    const int64_t rest = w / g.blocks;
    p.i = (int)(rest % tiles) + first_tile;
    p.any = rest / tiles < a.B;
    p.row = (int)(rest / tiles);
    p.t0 = p.i * g.tile;
    p.t1 = (int)min((int64_t)p.t0 + g.tile, a.T);
    const int64_t c = (int64_t)p.block * 64 + (threadIdx.x & 63);
    p.in = c < a.D;
    p.c = (uint32_t)min(c, a.D - 1);
    p.at = ((int64_t)p.row * g.tiles + p.i) * g.blocks + p.block;
    return p;
}

// A lane's channel of a token's row, which is the same address in all lanes: a
// scalar base and a 32-bit offset, one for all arrays of a type.  (The empty
// assembly keeps the two apart: else each array gets a 64-bit address a lane.)
template <typename T> using Global = __attribute__((address_space(1))) T;
template <typename T> __device__ __forceinline__ T get_at(const T* row, uint32_t c) {
    const Global<char>* base = (const Global<char>*)row;
    asm("" : "+s"(base));
    return *(const Global<T>*)(base + (uint32_t)(c * sizeof(T)));
}
template <typename T> __device__ __forceinline__ void put_at(T* row, uint32_t c, T x) {
    Global<char>* base = (Global<char>*)row;
    asm("" : "+s"(base));
    *(Global<T>*)(base + (uint32_t)(c * sizeof(T))) = x;
}

// softplus(y) to a few ulps of itself, also where it is next to 0: with e =
// exp(-|y|), max(y, 0) + log(1 + e) = max(y, 0) + 2 atanh(s), s = e / (2 + e) <= 1/3.
// exp takes what the product with log2 e and that number itself lose; atanh(s) =
// s + s^3 p(s^2) with p, of degree 3, through the Chebyshev nodes of [0, 1/9]
// (2^-25.9 of the value at most).
__device__ __forceinline__ float softplus(float y) {
    const float m = __builtin_amdgcn_fmed3f(-fabsf(y), -150.f, 0.f);      // -inf would lose itself; NaN stays in y
    const float t = m * kLog2e, lost = fmaf(m, 1.92596303e-8f, fmaf(m, kLog2e, -t));
    const float e0 = __builtin_amdgcn_exp2f(t), e = fmaf(e0, kLn2 * lost, e0);
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float p = 0.1342574954f;
    p = fmaf(p, q, 0.1411830932f);
    p = fmaf(p, q, 0.2000378072f);
    p = fmaf(p, q, 0.3333331943f);
    return fmaf(2.f, fmaf(p * q, s, s), __builtin_elementwise_maximum(y, 0.f));
}

// One row of B or C, in scalar registers.
typedef const __attribute__((address_space(4))) uint32_t* scalar_words;
template <typename E, int N>
struct Shared {
    static constexpr int WORDS = N * sizeof(E) / 4;
    static constexpr bool AHEAD = WORDS <= 8;      // whether two rows of B and of C fit the scalar registers
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const E* row) {
        const scalar_words p = (scalar_words)(uintptr_t)row;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = p[i];
    }
    // Waits for the row.  Scalar loads come back in any order, so a wait is for
    // all of them.
    __device__ __forceinline__ void wait() {
#pragma unroll
        for (int i = 0; i < WORDS; i += 8) asm volatile("" : "+s"(w[i]));
    }
    __device__ __forceinline__ float operator[](int n) const {
        if constexpr (sizeof(E) == 4) return __uint_as_float(w[n]);
        else return __uint_as_float(n & 1 ? w[n >> 1] & 0xffff0000u : w[n >> 1] << 16);
    }
};

// The rows of a walk along the tokens, the next one sent for behind the wait for
// this one, so that it is there when a token's work is done.
template <typename E, int N>
struct SharedWalk {
    static constexpr bool AHEAD = Shared<E, N>::AHEAD;
    const E* at;
    Shared<E, N> now[AHEAD ? 2 : 1];
    __device__ __forceinline__ explicit SharedWalk(const E* first) : at(first) {
        if constexpr (AHEAD) now[0].load(at);
    }
    // The row of this token, the u-th of an even number; `step` elements further
    // lies the next one's, if there is `more`.
    __device__ __forceinline__ void begin(int u) {
        if constexpr (AHEAD) now[u & 1].wait();
        else now[0].load(at);
    }
    __device__ __forceinline__ void go_on(int u, int step, bool more) {
        if (more) at += step;
        if constexpr (AHEAD) now[(u + 1) & 1].load(at);
    }
    __device__ __forceinline__ const Shared<E, N>& row(int u) const { return now[AHEAD ? u & 1 : 0]; }
};

// A lane's parameters: A in powers of two.
template <int N>
struct Params {
    float A2[N], skip, bias;
    __device__ __forceinline__ Params(const SelectiveArgs& a, uint32_t c) {
#pragma unroll
        for (int n = 0; n < N; ++n) A2[n] = a.A[(int64_t)c * N + n] * kLog2e;
        skip = a.skip ? a.skip[c] : 0.f;
        bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    }
};

// N states of a lane's channel as the caller has them, and as the workspace
// does: [N][64 lanes].
template <int N>
__device__ __forceinline__ void get_state(const float* state, int64_t s, const SelectiveArgs& a, uint32_t c, float (&h)[N]) {
#pragma unroll
    for (int n = 0; n < N; n += 4) {
        const f32x4 x = state ? *reinterpret_cast<const f32x4*>(state + (s * a.D + c) * N + n) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) h[n + i] = x[i];
    }
}
template <int N>
__device__ __forceinline__ void put_state(float* state, int64_t s, const SelectiveArgs& a, uint32_t c, const float (&h)[N]) {
#pragma unroll
    for (int n = 0; n < N; n += 4)
        *reinterpret_cast<f32x4*>(state + (s * a.D + c) * N + n) = f32x4{h[n], h[n + 1], h[n + 2], h[n + 3]};
}
template <int N>
__device__ __forceinline__ void get_kept(const float* at, float (&h)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = at[n * 64 + (threadIdx.x & 63)];
}
template <int N>
__device__ __forceinline__ void put_kept(float* at, const float (&h)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) at[n * 64 + (threadIdx.x & 63)] = h[n];
}

// The parts of a workspace: for each tile its sum of delta and its states, which
// the join replaces by those that enter it; of packed batches the state that
// the last sequence which begins in the tile begins with (state_out may be
// state_in, and is written by another wave); the backward's kept states and sums.
struct ScanWorkspace {
    float* sums;         // [row][tile][block][64]
    float* ends;         // [row][tile][block][N][64]
    float* begins;       // the same
    float* delta;        // [row][T][D], of the tokens that step 1 passes; with a backward of all
    float* keep;         // [row][T / kKeep][block][N][64]
    float* params;       // [row][tile][N + 2][D]: sums for dA, dskip, ddt_bias
    float* shared;       // [block][row][T][2 N]: sums for dB, dC
};

// ---- 1. each tile's state from nothing ------------------------------------------
template <typename E, int N>
__global__ __launch_bounds__(kScanWaves * 64) void kda_selective_local_kernel(SelectiveArgs a, ScanGrid g, ScanWorkspace ws) {
    const Place p = place_of(a, g, gridDim.x, 1);
    if (!p.any) return;
    const Params<N> par(a, p.c);
    float h[N], sum = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] = 0.f;
    Sequences q(a.cu_seqlens, a.n_seq, a.T, p.row, p.t1 - 1);
    // the join hands a uniform row's first tile its state
    const bool begins = a.cu_seqlens && q.first >= p.t0;
    if (q.end <= p.t1 || q.first >= p.t1) {     // the next tile takes nothing from this one
        sum = kCut;
    } else {
        const int b = max(q.first, p.t0);
        const int64_t row = (int64_t)p.row * a.T;
        const E* x = reinterpret_cast<const E*>(a.x) + (row + p.t1 - 1) * a.D;
        const E* dt = reinterpret_cast<const E*>(a.dt) + (row + p.t1 - 1) * a.D;
        constexpr int U = 4;
        E xs[2][U], ds[2][U];
        auto fetch = [&](int t, E (&xv)[U], E (&dv)[U]) {     // tokens t - 1, t - 2, ..., called in that order
#pragma unroll
            for (int u = 0; u < U; ++u) {
                xv[u] = get_at(x, p.c);
                dv[u] = get_at(dt, p.c);
                const int64_t step = t - 1 - u > b ? a.D : 0;
                x -= step;
                dt -= step;
            }
        };
        SharedWalk<E, N> B(reinterpret_cast<const E*>(a.Bm) + (row + p.t1 - 1) * N);
        float* to = ws.delta + (row + p.t1 - 1) * a.D;
        auto tokens = [&](int t, const E (&xv)[U], const E (&dv)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t - 1 - u < b) break;
                B.begin(u);
                B.go_on(u, -N, t - 1 - u > b);
                __builtin_amdgcn_sched_barrier(0);
                const float delta = softplus(to_f32(dv[u]) + par.bias), w = delta * to_f32(xv[u]);
                if (p.in) put_at(to, p.c, delta);
                to -= a.D;
#pragma unroll
                for (int n = 0; n < N; ++n) h[n] = fmaf(__builtin_amdgcn_exp2f(sum * par.A2[n]), w * B.row(u)[n], h[n]);
                sum += delta;
            }
        };
        fetch(p.t1, xs[0], ds[0]);
        for (int t = p.t1; t > b; t -= 2 * U) {
            fetch(t - U, xs[1], ds[1]);
            tokens(t, xs[0], ds[0]);
            if (t - U <= b) break;
            fetch(t - 2 * U, xs[0], ds[0]);
            tokens(t - U, xs[1], ds[1]);
        }
        if (begins) {
            float s[N];
            get_state<N>(a.state_in, q.s, a, p.c, s);
            put_kept<N>(ws.begins + p.at * N * 64, s);
#pragma unroll
            for (int n = 0; n < N; ++n) h[n] = fmaf(__builtin_amdgcn_exp2f(sum * par.A2[n]), s[n], h[n]);
            sum = kCut;
        }
    }
    ws.sums[p.at * 64 + (threadIdx.x & 63)] = sum;
    put_kept<N>(ws.ends + p.at * N * 64, h);
}

// ---- 2. the tiles joined, in their order or from the last to the first -----------
// A workgroup has one state of 64 channels of a row, a wave kJoin tiles at a time,
// all of which are on their way together: their latency is what bounds this.  The
// waves' maps h -> A h + H are joined through LDS.  Tile i's state becomes the one
// that enters it.
constexpr int kJoin = 16;

template <int N, bool BACK, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void kda_selective_join_kernel(SelectiveArgs a, ScanGrid g, ScanWorkspace ws) {
    __shared__ float sA[WAVES][64], sH[WAVES][64];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int n = (int)(blockIdx.x % N), block = (int)(blockIdx.x / N % g.blocks);
    const int64_t row = blockIdx.x / N / g.blocks, c = min((int64_t)block * 64 + lane, a.D - 1);
    const float A2 = a.A[c * N + n] * kLog2e;
    const float* from = BACK ? a.d_state : a.state_in;
    float in = !a.cu_seqlens && from ? from[(row * a.D + c) * N + n] : 0.f;       // enters the tiles of a turn
    auto place = [&](int i) { return (row * g.tiles + (BACK ? g.tiles - 1 - i : i)) * g.blocks + block; };
    const int last = g.tiles - 1;        // has no state of its own: nothing goes on behind it
    for (int first = 0; first <= last; first += WAVES * kJoin) {
        const int i0 = first + wave * kJoin;
        float e[kJoin], f[kJoin];
#pragma unroll
        for (int u = 0; u < kJoin; ++u) {
            const int64_t at = place(min(i0 + u, last - 1));
            e[u] = ws.ends[(at * N + n) * 64 + lane];
            f[u] = ws.sums[at * 64 + lane];
        }
        float A = 1.f, H = 0.f;
#pragma unroll
        for (int u = 0; u < kJoin; ++u) {
            f[u] = f[u] < 0.f ? 0.f : __builtin_amdgcn_exp2f(f[u] * A2);
            A *= f[u];
            H = fmaf(f[u], H, e[u]);
        }
        sA[wave][lane] = A;
        sH[wave][lane] = H;
        __syncthreads();
        float h = in;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            in = fmaf(sA[w][lane], in, sH[w][lane]);
            if (w + 1 == wave) h = in;
        }
#pragma unroll
        for (int u = 0; u < kJoin; ++u) {
            if (i0 + u > last) break;
            ws.ends[(place(i0 + u) * N + n) * 64 + lane] = h;
            h = fmaf(f[u], h, e[u]);
        }
        __syncthreads();                 // before the next turn's maps
    }
}

// ---- 3. each tile from its true state ---------------------------------------------
template <typename E, int N, bool GATE, bool KEEP>
__global__ __launch_bounds__(kScanWaves * 64) void kda_selective_scan_kernel(SelectiveArgs a, ScanGrid g, ScanWorkspace ws, unsigned blocks) {
    if (blockIdx.x >= blocks) {
        pass_through<N>(a, blockIdx.x - blocks, a.state_in, a.state_out);
        return;
    }
    const Place p = place_of(a, g, blocks);
    if (!p.any) return;
    const Params<N> par(a, p.c);
    const int64_t row = (int64_t)p.row * a.T;
    Sequences q(a.cu_seqlens, a.n_seq, a.T, p.row, p.t0);
    do {
        const int b = max(q.first, p.t0), e = min(q.end, p.t1);
        if (b >= e) continue;
        float h[N];
        if (g.tiles > 1 && (!a.cu_seqlens || b > q.first)) get_kept<N>(ws.ends + p.at * N * 64, h);
        else if (q.end > p.t1) get_kept<N>(ws.begins + p.at * N * 64, h);
        else get_state<N>(a.state_in, q.s, a, p.c, h);

        // HAVE: step 1 has left delta
        auto run = [&](auto have) {
            constexpr bool HAVE = decltype(have)::value;
            typedef typename std::conditional<HAVE, float, E>::type DE;
            const int64_t first = (row + b) * a.D;
            const E *x = reinterpret_cast<const E*>(a.x) + first, *z = reinterpret_cast<const E*>(a.z) + first;
            float* deltas = ws.delta + first;
            E* to = reinterpret_cast<E*>(a.out) + first;
            const DE* from;
            if constexpr (HAVE) from = deltas;
            else from = reinterpret_cast<const E*>(a.dt) + first;
            constexpr int U = 4;
            E xs[2][U], zs[2][U];
            DE ds[2][U];
            auto fetch = [&](int t, E (&xv)[U], DE (&dv)[U], E (&zv)[U]) {      // called in the order of the tokens
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    xv[u] = get_at(x, p.c);
                    dv[u] = get_at(from, p.c);
                    if constexpr (GATE) zv[u] = get_at(z, p.c);
                    const int64_t step = t + u + 1 < e ? a.D : 0;
                    x += step;
                    from += step;
                    z += step;
                }
            };
            SharedWalk<E, N> B(reinterpret_cast<const E*>(a.Bm) + (row + b) * N), C(reinterpret_cast<const E*>(a.Cm) + (row + b) * N);
            auto tokens = [&](int t, const E (&xv)[U], const DE (&dv)[U], const E (&zv)[U]) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (t + u >= e) break;
                    B.begin(u);
                    C.begin(u);
                    B.go_on(u, N, t + u + 1 < e);
                    C.go_on(u, N, t + u + 1 < e);
                    __builtin_amdgcn_sched_barrier(0);
                    if constexpr (KEEP) {
                        if ((t + u) % kKeep<N> == 0) {
                            const int64_t kept = (a.T + kKeep<N> - 1) / kKeep<N>;
                            put_kept<N>(ws.keep + ((p.row * kept + (t + u) / kKeep<N>) * g.blocks + p.block) * N * 64, h);
                        }
                    }
                    float delta = to_f32(dv[u]);
                    if constexpr (!HAVE) {
                        delta = softplus(delta + par.bias);
                        if constexpr (KEEP) {
                            if (p.in) put_at(deltas, p.c, delta);
                            deltas += a.D;
                        }
                    }
                    const float xf = to_f32(xv[u]), w = delta * xf;
                    float y[4] = {par.skip * xf, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        h[n] = fmaf(__builtin_amdgcn_exp2f(delta * par.A2[n]), h[n], w * B.row(u)[n]);
                        y[n & 3] = fmaf(C.row(u)[n], h[n], y[n & 3]);
                    }
                    float o = (y[0] + y[1]) + (y[2] + y[3]);
                    if constexpr (GATE) {
                        const float zf = to_f32(zv[u]);
                        o *= zf * sigmoidf_(zf);
                    }
                    if (p.in) put_at(to, p.c, from_f32<E>(o));
                    to += a.D;
                }
            };
            fetch(b, xs[0], ds[0], zs[0]);
            for (int t = b; t < e; t += 2 * U) {
                fetch(t + U, xs[1], ds[1], zs[1]);
                tokens(t, xs[0], ds[0], zs[0]);
                if (t + U >= e) break;
                fetch(t + 2 * U, xs[0], ds[0], zs[0]);
                tokens(t + U, xs[1], ds[1], zs[1]);
            }
        };
        if (q.end > p.t1) run(std::true_type{});
        else run(std::false_type{});
        if (a.state_out && e == q.end && p.in) put_state<N>(a.state_out, q.s, a, p.c, h);
    } while (q.end < p.t1 && q.next());
}

// ---- the backward ------------------------------------------------------------------
// 1. What a tile's tokens give the gradient of the state that enters it:
//    sum_t exp(A sum_(s<=t) delta_s) C_t dy_t.
template <typename E, int N, bool GATE>
__global__ __launch_bounds__(kScanWaves * 64) void kda_selective_local_back_kernel(SelectiveArgs a, ScanGrid g, ScanWorkspace ws) {
    const Place p = place_of(a, g, gridDim.x, 1, 1);
    if (!p.any) return;
    const Params<N> par(a, p.c);
    float r[N], sum = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) r[n] = 0.f;
    Sequences q(a.cu_seqlens, a.n_seq, a.T, p.row, p.t0);
    if (q.first >= p.t0 || q.end <= p.t0) {     // the tile before this one gets nothing from it
        sum = kCut;
    } else {
        const int e = min(q.end, p.t1);
        const bool ends = q.end <= p.t1 && a.cu_seqlens;
        const int64_t row = (int64_t)p.row * a.T;
        const int64_t first = (row + p.t0) * a.D;
        const float* deltas = ws.delta + first;
        const E* z = reinterpret_cast<const E*>(a.z) + first;
        const E* d_out = reinterpret_cast<const E*>(a.d_out ? a.d_out : a.x) + first;      // any that is there
        constexpr int U = 4;
        E gs[2][U], zs[2][U];
        float ds[2][U];
        auto fetch = [&](int t, E (&gv)[U], float (&dv)[U], E (&zv)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                gv[u] = get_at(d_out, p.c);
                dv[u] = get_at(deltas, p.c);
                if constexpr (GATE) zv[u] = get_at(z, p.c);
                const int64_t step = t + u + 1 < e ? a.D : 0;
                d_out += step;
                deltas += step;
                z += step;
            }
        };
        SharedWalk<E, N> C(reinterpret_cast<const E*>(a.Cm) + (row + p.t0) * N);
        auto tokens = [&](int t, const E (&gv)[U], const float (&dv)[U], const E (&zv)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= e) break;
                C.begin(u);
                C.go_on(u, N, t + u + 1 < e);
                __builtin_amdgcn_sched_barrier(0);
                sum += dv[u];
                float dy = a.d_out ? to_f32(gv[u]) : 0.f;
                if constexpr (GATE) {
                    const float zf = to_f32(zv[u]);
                    dy *= zf * sigmoidf_(zf);
                }
#pragma unroll
                for (int n = 0; n < N; ++n) r[n] = fmaf(__builtin_amdgcn_exp2f(sum * par.A2[n]), dy * C.row(u)[n], r[n]);
            }
        };
        fetch(p.t0, gs[0], ds[0], zs[0]);
        for (int t = p.t0; t < e; t += 2 * U) {
            fetch(t + U, gs[1], ds[1], zs[1]);
            tokens(t, gs[0], ds[0], zs[0]);
            if (t + U >= e) break;
            fetch(t + 2 * U, gs[0], ds[0], zs[0]);
            tokens(t + U, gs[1], ds[1], zs[1]);
        }
        if (ends) {
            float s[N];
            get_state<N>(a.d_state, q.s, a, p.c, s);
#pragma unroll
            for (int n = 0; n < N; ++n) r[n] = fmaf(__builtin_amdgcn_exp2f(sum * par.A2[n]), s[n], r[n]);
            sum = kCut;
        }
    }
    ws.sums[p.at * 64 + (threadIdx.x & 63)] = sum;
    put_kept<N>(ws.ends + p.at * N * 64, r);
}

// Sums over the 64 lanes of K values at once: halves of the lanes take halves of
// the values, so that each step adds half as many.  The sum of value k ends in
// the lanes whose bits say k: bit 5 of a lane is the value's highest, and so on.
// halves() is the first step, of values k and k + K / 2; sum_lanes takes its K / 2
// results.
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ float pair_sum(float x, float y, bool upper) {     // lanes of `upper` take y
    return (upper ? y : x) + moved<CTRL>(upper ? x : y);
}
__device__ __forceinline__ float halves(float x, float y) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
__device__ __forceinline__ float quarters(float x, float y) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
    return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}
template <int K>
__device__ __forceinline__ float sum_lanes(float (&v)[K / 2]) {
    static_assert(K == 16 || K == 32 || K == 64, "each lane, or 2 or 4 of them, end with a sum");
    constexpr int HALF_MIRROR = 0x141, ROR8 = 0x128, XOR2 = 0x4e, XOR1 = 0xb1;
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < K / 4; ++i) v[i] = quarters(v[i], v[i + K / 4]);
#pragma unroll
    for (int i = 0; i < K / 8; ++i) v[i] = pair_sum<ROR8>(v[i], v[i + K / 8], lane & 8);
#pragma unroll
    for (int i = 0; i < K / 16; ++i) v[i] = pair_sum<HALF_MIRROR>(v[i], v[i + K / 16], lane & 4);
    if constexpr (K >= 32) {
#pragma unroll
        for (int i = 0; i < K / 32; ++i) v[i] = pair_sum<XOR2>(v[i], v[i + K / 32], lane & 2);
    } else {
        v[0] += moved<XOR2>(v[0]);
    }
    if constexpr (K >= 64) v[0] = pair_sum<XOR1>(v[0], v[1], lane & 1);
    else v[0] += moved<XOR1>(v[0]);
    return v[0];
}

// 2. Each tile from its last token to its first, half of kKeep tokens at a time,
//    whose states are formed anew from the kept one and stay in registers.  All
//    KT tokens at once, or the next turn's loads sent ahead, spill (3444 and 1377 us
//    instead of 517); so do three waves a SIMD (1756), and one wave takes 779.
template <typename E, int N, bool GATE>
__global__ __launch_bounds__(kScanWaves * 64, N == 32 ? 1 : 2) void kda_selective_back_kernel(SelectiveArgs a, ScanGrid g, ScanWorkspace ws, unsigned blocks) {
    if (blockIdx.x >= blocks) {
        pass_through<N>(a, blockIdx.x - blocks, a.d_state, a.d_state_in);
        return;
    }
    constexpr int KT = kKeep<N>, HT = KT / 2;
    const Place p = place_of(a, g, blocks);
    if (!p.any) return;
    const int lane = threadIdx.x & 63;
    const Params<N> par(a, p.c);
    const int64_t row = (int64_t)p.row * a.T, kept = (a.T + KT - 1) / KT, at0 = row * a.D;
    const E* x = reinterpret_cast<const E*>(a.x) + at0;
    const E* dt = reinterpret_cast<const E*>(a.dt) + at0;
    const E* z = reinterpret_cast<const E*>(a.z) + at0;
    const E* d_out = reinterpret_cast<const E*>(a.d_out ? a.d_out : a.x) + at0;      // any that is there
    const float* deltas = ws.delta + at0;
    const E *Bp = reinterpret_cast<const E*>(a.Bm) + row * N, *Cp = reinterpret_cast<const E*>(a.Cm) + row * N;
    float dA[N], dskip = 0.f, dbias = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) dA[n] = 0.f;
    Sequences q(a.cu_seqlens, a.n_seq, a.T, p.row, p.t1 - 1);
    do {
        const int b = max(q.first, p.t0), e = min(q.end, p.t1);
        if (b >= e) continue;
        float r[N];
        if (q.end > p.t1 || (g.tiles > 1 && !a.cu_seqlens)) get_kept<N>(ws.ends + p.at * N * 64, r);
        else get_state<N>(a.d_state, q.s, a, p.c, r);
        for (int te = e; te > b;) {
            const int k = (te - 1) / KT, t0 = max(b, k * KT);
            const int tb = te - t0 > HT ? t0 + HT : t0, m = te - tb;      // the tokens of this turn
            float h[HT + 1][N], delta[HT];
            E xs[HT], ds[HT], zs[HT], gs[HT];
#pragma unroll
            for (int u = 0; u < HT; ++u) {
                const int64_t at = (int64_t)min(tb + u, te - 1) * a.D;
                xs[u] = get_at(x + at, p.c);
                delta[u] = get_at(deltas + at, p.c);
                ds[u] = get_at(dt + at, p.c);
                if constexpr (GATE) zs[u] = get_at(z + at, p.c);
                gs[u] = get_at(d_out + at, p.c);
            }
            if (t0 == k * KT) get_kept<N>(ws.keep + ((p.row * kept + k) * g.blocks + p.block) * N * 64, h[0]);
            else get_state<N>(a.state_in, q.s, a, p.c, h[0]);
            if (tb > t0) {                // over the first half, to the state that the second begins with
                E xf[HT];
                float df[HT];
#pragma unroll
                for (int u = 0; u < HT; ++u) {
                    xf[u] = get_at(x + (int64_t)(t0 + u) * a.D, p.c);
                    df[u] = get_at(deltas + (int64_t)(t0 + u) * a.D, p.c);
                }
#pragma unroll
                for (int u = 0; u < HT; ++u) {
                    Shared<E, N> B;
                    B.load(Bp + (int64_t)(t0 + u) * N);
                    const float w = df[u] * to_f32(xf[u]);
#pragma unroll
                    for (int n = 0; n < N; ++n) h[0][n] = fmaf(__builtin_amdgcn_exp2f(df[u] * par.A2[n]), h[0][n], w * B[n]);
                }
            }
#pragma unroll
            for (int u = 0; u < HT; ++u) {
                if (u >= m) continue;
                Shared<E, N> B;
                B.load(Bp + (int64_t)(tb + u) * N);
                const float w = delta[u] * to_f32(xs[u]);
#pragma unroll
                for (int n = 0; n < N; ++n) h[u + 1][n] = fmaf(__builtin_amdgcn_exp2f(delta[u] * par.A2[n]), h[u][n], w * B[n]);
            }
#pragma unroll
            for (int u = HT - 1; u >= 0; --u) {
                if (u >= m) continue;
                const int t = tb + u;
                Shared<E, N> B, C;
                B.load(Bp + (int64_t)t * N);
                C.load(Cp + (int64_t)t * N);
                const float xf = to_f32(xs[u]), d = delta[u], w = d * xf, go = a.d_out ? to_f32(gs[u]) : 0.f;
                float zf = 0.f, sig = 0.f, dy = go;
                if constexpr (GATE) {
                    zf = to_f32(zs[u]);
                    sig = sigmoidf_(zf);
                    dy = go * (zf * sig);
                }
                // lanes without a channel add nothing to the sums over channels
                const float wv = p.in ? w : 0.f, dyv = p.in ? dy : 0.f;
                float y = GATE ? par.skip * xf : 0.f, du = 0.f, dd = 0.f, v[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const float dh = fmaf(C[n], dy, r[n]);
                    if constexpr (GATE) y = fmaf(C[n], h[u + 1][n], y);
                    v[n] = halves(dh * wv, dyv * h[u + 1][n]);
                    du = fmaf(dh, B[n], du);
                    r[n] = __builtin_amdgcn_exp2f(d * par.A2[n]) * dh;
                    const float back = r[n] * h[u][n];
                    dd = fmaf(back, par.A2[n], dd);
                    dA[n] = fmaf(back, d, dA[n]);
                }
                const float s = sum_lanes<2 * N>(v);
                const float ddt = fmaf(du, xf, dd * kLn2) * sigmoidf_(to_f32(ds[u]) + par.bias);
                const int64_t at = at0 + (int64_t)t * a.D;
                if (p.in) {
                    put_at(reinterpret_cast<E*>(a.dx) + at, p.c, from_f32<E>(fmaf(du, d, par.skip * dy)));
                    put_at(reinterpret_cast<E*>(a.ddt) + at, p.c, from_f32<E>(ddt));
                    if constexpr (GATE) put_at(reinterpret_cast<E*>(a.dz) + at, p.c, from_f32<E>(go * y * (sig * fmaf(zf, 1.f - sig, 1.f))));
                }
                dskip = fmaf(dy, xf, dskip);
                dbias += ddt;
                // value i's sum is in the lanes from 64 / (2 N) i on
                if (lane % (64 / (2 * N)) == 0) ws.shared[((int64_t)p.block * a.B * a.T + row + t) * (2 * N) + lane / (64 / (2 * N))] = s;
            }
            te = tb;
        }
        if (b == q.first && a.d_state_in && p.in) put_state<N>(a.d_state_in, q.s, a, p.c, r);
    } while (q.first > p.t0 && q.previous());
    if (p.in) {
        float* to = ws.params + ((int64_t)p.row * g.tiles + p.i) * (N + 2) * a.D;
#pragma unroll
        for (int n = 0; n < N; ++n) put_at(to + n * a.D, p.c, dA[n]);
        put_at(to + N * a.D, p.c, dskip);
        put_at(to + (N + 1) * a.D, p.c, dbias);
    }
}

// 3. The parameters' gradients: sums over the tiles in their order, 64 channels of
//    one a workgroup, whose waves have every fourth tile.  In 64 bits, as there can
//    be any number.
__device__ __forceinline__ void sum_params(const SelectiveArgs& a, const ScanGrid& g, const float* parts, int64_t count, unsigned block) {
    __shared__ double sum[kScanWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c = (int64_t)(block % g.blocks) * 64 + lane;
    const int j = block / g.blocks;
    float* to = j < a.states ? a.dA + c * a.states + j : (j == a.states ? a.dskip : a.ddt_bias);
    if (!to) return;
    if (j >= a.states) to += c;
    double s = 0.;
    if (c < a.D) {
        const float* from = parts + (int64_t)j * a.D + c;
        const int64_t stride = (a.states + 2) * a.D;
#pragma unroll 8
        for (int64_t i = wave; i < count; i += kScanWaves) s += from[i * stride];
    }
    sum[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= a.D) return;
#pragma unroll
    for (int w = 1; w < kScanWaves; ++w) s += sum[w][lane];
    *to = (float)s;
}

//    dB and dC: sums over the channel blocks in their order, by the workgroups
//    behind those of the parameters.
template <typename E>
__global__ __launch_bounds__(256) void kda_selective_sum_kernel(SelectiveArgs a, ScanGrid g, ScanWorkspace ws, int64_t count) {
    const int N = a.states;
    const unsigned params = (unsigned)g.blocks * (N + 2);
    if (blockIdx.x < params) {
        sum_params(a, g, ws.params, count, blockIdx.x);
        return;
    }
    const int64_t i = (int64_t)(blockIdx.x - params) * 256 + threadIdx.x;
    const int64_t row = i / (2 * N), rows = a.B * a.T;
    const int n = (int)(i - row * 2 * N);
    if (row >= rows) return;
    if (a.cu_seqlens) {                   // tokens of no sequence are left as they are
        int64_t first, end, none;
        seq_bounds(a.cu_seqlens, 0, a.T, first, none);
        seq_bounds(a.cu_seqlens, a.n_seq - 1, a.T, none, end);
        if (row < first || row >= end) return;
    }
    float s = 0.f;
#pragma unroll 8
    for (int b = 0; b < g.blocks; ++b) s += ws.shared[(b * rows + row) * 2 * N + n];
    E* to = reinterpret_cast<E*>(n < N ? a.dB : a.dC);
    to[row * N + (n < N ? n : n - N)] = from_f32<E>(s);
}

// ---- one token -----------------------------------------------------------------------
// Four states a lane, so that a wave reads and writes whole lines of states.
template <typename E, int N>
__global__ __launch_bounds__(256) void kda_selective_step_kernel(SelectiveArgs a) {
    constexpr int L = N / 4;             // lanes of a channel
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, e = i / L, row = e / a.D, c = e - row * a.D;
    if (row >= a.B) return;
    const int n0 = (int)(i % L) * 4;
    f32x4* at = reinterpret_cast<f32x4*>(a.state_out + i * 4);
    const f32x4 A = *reinterpret_cast<const f32x4*>(a.A + c * N + n0), B = ld4(reinterpret_cast<const E*>(a.Bm) + row * N + n0),
                C = ld4(reinterpret_cast<const E*>(a.Cm) + row * N + n0);
    f32x4 h = *at;
    const float x = to_f32(reinterpret_cast<const E*>(a.x)[e]);
    const float delta = softplus(to_f32(reinterpret_cast<const E*>(a.dt)[e]) + (a.dt_bias ? a.dt_bias[c] : 0.f)), w = delta * x;
    float y = 0.f;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        h[n] = fmaf(__builtin_amdgcn_exp2f(delta * (A[n] * kLog2e)), h[n], w * B[n]);
        y = fmaf(C[n], h[n], y);
    }
    *at = h;
#pragma unroll
    for (int off = 1; off < L; off <<= 1) y += __shfl_xor(y, off);
    if (n0 != 0) return;
    if (a.skip) y = fmaf(a.skip[c], x, y);
    if (a.z) {
        const float z = to_f32(reinterpret_cast<const E*>(a.z)[e]);
        y *= z * sigmoidf_(z);
    }
    reinterpret_cast<E*>(a.out)[e] = from_f32<E>(y);
}

// ---- host ------------------------------------------------------------------------------
// Waves that a call is split into, where it has that many.  With 8192, whose states
// take twice the workspace, kernels took 1033 us instead of 1049 for 65536 tokens of
// 2048 channels (16 states, bf16) and 956 instead of 966 for a training pass of 4 x
// 4096; with 16384 1071 and 1007.
constexpr int kWaves = 4096;

ScanGrid scan_grid(const SelectiveArgs& a) {
    ScanGrid g = {};
    g.blocks = (int)((a.D + 63) / 64);
    const int64_t alone = a.B * g.blocks;
    int64_t tiles = alone > 0 ? (kWaves + alone / 2) / alone : 1;
    if (tiles < 1) tiles = 1;
    int64_t tile = (a.T + tiles - 1) / tiles;
    // Joining many tiles takes its time: 65536 tokens of 64 channels take 87 us in
    // tiles of 32, 104 of 64, 163 of 128; 4096 tokens 25 in tiles of 16, 34 of 32.
    int64_t least = 16;
    while (least * least * 64 < a.T) least += 16;
    if (tile < least && tiles > 1) tile = least;
    g.tile = (int)((tile + 15) / 16 * 16);
    if (g.tile < 16) g.tile = 16;
    g.tiles = (int)((a.T + g.tile - 1) / g.tile);
    return g;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
int keep_of(int states) { return 128 / states; }

size_t lay_out(const SelectiveArgs& a, bool backward, char* at, ScanWorkspace& ws) {
    const ScanGrid g = scan_grid(a);
    size_t used = 0;
    auto take = [&](bool wanted, size_t floats) {
        float* r = wanted && at ? reinterpret_cast<float*>(at + used) : nullptr;
        if (wanted) used += round256(floats * sizeof(float));
        return r;
    };
    const size_t tiles = (size_t)a.B * g.tiles, one = (size_t)g.blocks * a.states * 64;
    const bool many = g.tiles > 1;
    ws.sums = take(many, tiles * g.blocks * 64);
    ws.ends = take(many, tiles * one);
    ws.begins = take(many && a.cu_seqlens, tiles * one);
    ws.delta = take(many || backward, (size_t)a.B * a.T * a.D);
    const size_t kept = (size_t)a.B * ((a.T + keep_of(a.states) - 1) / keep_of(a.states));
    ws.keep = take(backward, kept * one);
    ws.params = take(backward, tiles * (a.states + 2) * a.D);
    ws.shared = take(backward, (size_t)g.blocks * a.B * a.T * 2 * a.states);
    return used;
}

unsigned tile_blocks(int64_t waves) {
    const int64_t blocks = (waves + kScanWaves - 1) / kScanWaves;
    return (unsigned)((blocks + kXcds - 1) / kXcds * kXcds);
}

// Workgroups for the sequences that may have no tokens, where their states go
// from one array to another.
unsigned through_blocks(const SelectiveArgs& a, const float* from, const float* to) {
    const bool some = to && from != to && a.n_seq > 0 && (a.cu_seqlens || a.T == 0);
    return some ? (unsigned)((a.n_seq + kScanWaves - 1) / kScanWaves) : 0u;
}

// Two waves have 32 tiles at a time, which is all of them in a training pass of 4 x
// 4096 tokens of 2048 channels (10 us; eight waves 21); eight 128 (16384 tokens of
// 515 channels, 256 tiles: 7 us; two 23).
template <int N, bool BACK>
hipError_t launch_join(const SelectiveArgs& a, const ScanGrid& g, const ScanWorkspace& ws, hipStream_t s) {
    const dim3 grid((unsigned)(a.B * g.blocks * N));
    if (g.tiles <= 4 * kJoin) hipLaunchKernelGGL((kda_selective_join_kernel<N, BACK, 2>), grid, dim3(128), 0, s, a, g, ws);
    else hipLaunchKernelGGL((kda_selective_join_kernel<N, BACK, 8>), grid, dim3(512), 0, s, a, g, ws);
    return hipGetLastError();
}

template <typename E, int N>
hipError_t scan_forward(const SelectiveArgs& a, hipStream_t s) {
    hipError_t e;
    const ScanGrid g = scan_grid(a);
    ScanWorkspace ws;
    lay_out(a, a.keep, a.ws, ws);
    const dim3 block(kScanWaves * 64);
    if (g.tiles > 1) {
        hipLaunchKernelGGL((kda_selective_local_kernel<E, N>), dim3(tile_blocks(a.B * (g.tiles - 1) * g.blocks)), block, 0, s, a, g, ws);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if ((e = launch_join<N, false>(a, g, ws, s)) != hipSuccess) return e;
    }
    const unsigned blocks = tile_blocks(a.B * g.tiles * g.blocks), more = through_blocks(a, a.state_in, a.state_out);
    if (blocks + more == 0) return hipSuccess;
    const auto kernel = a.z ? (a.keep ? kda_selective_scan_kernel<E, N, true, true> : kda_selective_scan_kernel<E, N, true, false>)
                            : (a.keep ? kda_selective_scan_kernel<E, N, false, true> : kda_selective_scan_kernel<E, N, false, false>);
    hipLaunchKernelGGL(kernel, dim3(blocks + more), block, 0, s, a, g, ws, blocks);
    return hipGetLastError();
}

template <typename E, int N>
hipError_t scan_backward(const SelectiveArgs& a, hipStream_t s) {
    hipError_t e;
    const ScanGrid g = scan_grid(a);
    ScanWorkspace ws;
    lay_out(a, true, a.ws, ws);
    const dim3 block(kScanWaves * 64);
    const int64_t waves = a.n_seq > 0 ? a.B * g.tiles * g.blocks : 0;
    if (waves > 0 && g.tiles > 1) {
        hipLaunchKernelGGL((a.z ? kda_selective_local_back_kernel<E, N, true> : kda_selective_local_back_kernel<E, N, false>),
                           dim3(tile_blocks(a.B * (g.tiles - 1) * g.blocks)), block, 0, s, a, g, ws);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        if ((e = launch_join<N, true>(a, g, ws, s)) != hipSuccess) return e;
    }
    const unsigned blocks = tile_blocks(waves), more = through_blocks(a, a.d_state, a.d_state_in);
    if (blocks + more > 0) {
        hipLaunchKernelGGL((a.z ? kda_selective_back_kernel<E, N, true> : kda_selective_back_kernel<E, N, false>), dim3(blocks + more), block, 0, s, a, g, ws,
                           blocks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t rows = waves > 0 ? (a.B * a.T * 2 * N + 255) / 256 : 0;
    hipLaunchKernelGGL((kda_selective_sum_kernel<E>), dim3((unsigned)(g.blocks * (N + 2) + rows)), dim3(256), 0, s, a, g, ws, waves > 0 ? a.B * g.tiles : 0);
    return hipGetLastError();
}

template <typename E, int N>
hipError_t scan_step(const SelectiveArgs& a, hipStream_t s) {
    hipLaunchKernelGGL((kda_selective_step_kernel<E, N>), dim3((unsigned)((a.B * a.D * (N / 4) + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename F>
hipError_t by_states(bool bf16, int states, F&& f) {
    auto typed = [&](auto e) {
        if (states == 8) return f(e, std::integral_constant<int, 8>{});
        if (states == 16) return f(e, std::integral_constant<int, 16>{});
        return f(e, std::integral_constant<int, 32>{});
    };
    return bf16 ? typed(__bf16{}) : typed(float{});
}

}  // namespace

bool selective_scan_fits(const SelectiveArgs& a) {
    const ScanGrid g = scan_grid(a);
    const int64_t most = UINT32_MAX / 256 - kXcds;      // workgroups of 256
    return a.B * g.tiles * g.blocks / kScanWaves + a.n_seq / kScanWaves < most && (g.tiles < 2 || a.B * g.blocks * a.states < most / 2) &&
           a.B * a.T * 2 * a.states / 256 + (int64_t)g.blocks * (a.states + 2) < most;
}

size_t selective_scan_workspace_bytes(const SelectiveArgs& a, bool backward) {
    ScanWorkspace ws;
    return lay_out(a, backward, nullptr, ws);
}

hipError_t launch_selective_scan(bool bf16, const SelectiveArgs& a, hipStream_t s) {
    return by_states(bf16, a.states, [&](auto e, auto n) { return scan_forward<decltype(e), decltype(n)::value>(a, s); });
}

hipError_t launch_selective_scan_backward(bool bf16, const SelectiveArgs& a, hipStream_t s) {
    return by_states(bf16, a.states, [&](auto e, auto n) { return scan_backward<decltype(e), decltype(n)::value>(a, s); });
}

hipError_t launch_selective_scan_step(bool bf16, const SelectiveArgs& a, hipStream_t s) {
    return by_states(bf16, a.states, [&](auto e, auto n) { return scan_step<decltype(e), decltype(n)::value>(a, s); });
}

}  // namespace kda

// kda_short_conv.hip -- a causal convolution over the last few tokens of each
// channel, its gradients and its single-token step.
//
//   y_t = bias + sum_j w_j x_(t - W + 1 + j),  out_t = y_t sigmoid(y_t) or y_t
// and in reverse, with d_t = d_out_t (silu'(y_t) or 1), y_t formed anew from x:
//   dx_p = sum_j w_j d_(p + W - 1 - j)  (+ d_state where p is one of the last
//   W - 1 inputs),  dw_j = sum_t d_t x_(t - W + 1 + j),  dbias = sum_t d_t
//
// All are bound by HBM.  A wave walks along a tile of tokens with 64 vectors of
// 16 bytes of channels and keeps the window of W - 1 inputs in registers, so
// that an input is read once but for the W - 1 before each tile.  65536 tokens of
// 12288 channels in bf16 take 639 us, 5.0 TB/s, as fast as a copy.  A training pass
// of 4 x 4096 x 6144 takes 85 us forward (4.7 TB/s), 144 backward (4.2; fewer
// loads are on their way, as its registers leave three waves a SIMD) and 8 for the
// sums.  A call for a step of 8 x 12288 takes
// 9.5 us, of which 3 on the card.
#include <type_traits>

#include "kda_packed.hpp"
#include "kda_selective_internal.hpp"

namespace kda {

namespace {

constexpr int kConvWaves = 4;

// Channels that a lane has at a time: 16 bytes forward, four backward, whose
// weights, windows and sums take three times the registers (144 us backward for
// 4 x 4096 x 6144 in bf16, 200 with eight).  The last lane of a
// row whose width is no multiple begins early: it and the lane before it
// compute and write the same values.  Rows below one vector go channel by channel.
template <typename E> constexpr int kForward = 16 / sizeof(E);
constexpr int kBackward = 4;

__device__ __forceinline__ int wave_of_block() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// The tile that a wave works on.
struct ConvTile {
    int row, t0, t1;
    int64_t part;        // index of the tile over all rows
    int64_t c;           // a lane's first channel
    bool any;
};
template <int V>
__device__ __forceinline__ ConvTile conv_tile(const ShortConvArgs& a, int tile, int tiles, int chunks) {
    const int64_t w = (int64_t)blockIdx.x * kConvWaves + wave_of_block();
    ConvTile r;
    r.part = w / chunks;
    r.any = r.part < a.B * tiles;
    r.row = (int)(r.part / tiles);
    r.t0 = (int)(r.part % tiles) * tile;
    r.t1 = (int)min((int64_t)r.t0 + tile, a.T);
    const int64_t c = ((w % chunks) * 64 + (threadIdx.x & 63)) * V;
    r.c = min(c, a.D - V);
    return r;
}

// d silu(y) / dy, and silu(y)
__device__ __forceinline__ float silu(float y) { return y * sigmoidf_(y); }
__device__ __forceinline__ float silu_slope(float y) {
    const float s = sigmoidf_(y);
    return s * fmaf(y, 1.f - s, 1.f);
}

// Weights and bias of a lane's channels.
template <int W, int V>
struct Filter {
    float w[W][V], b[V];
    __device__ __forceinline__ Filter(const ShortConvArgs& a, int64_t c) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < W; ++j) w[j][v] = a.weight[(c + v) * W + j];
            b[v] = a.bias ? a.bias[c + v] : 0.f;
        }
    }
};

// The W - 1 inputs before token t of the sequence q of a row that begins at
// element `base`: of x, or of the state.
template <typename E, int W, int V>
__device__ __forceinline__ void window_before(const ShortConvArgs& a, const Sequences& q, int64_t base, int t, int64_t c,
                                              float (&win)[W - 1][V]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int at = t - (W - 1) + j;
        const E* from = nullptr;
        if (at >= q.first) from = reinterpret_cast<const E*>(a.x) + base + (int64_t)at * a.D + c;
        else if (a.state_in) from = reinterpret_cast<const E*>(a.state_in) + ((int64_t)q.s * (W - 1) + (at - q.first + W - 1)) * a.D + c;
        if (from) {
            const auto x = get_channels<E, V>(from);
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = x[v];
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = 0.f;
        }
    }
}

// y of one token, whose input moves into the window.
template <int W, int V>
__device__ __forceinline__ void convolve(const Filter<W, V>& f, float (&win)[W - 1][V], const float (&x)[V], float (&y)[V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = f.b[v];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) s = fmaf(f.w[j][v], win[j][v], s);
        y[v] = fmaf(f.w[W - 1][v], x[v], s);
#pragma unroll
        for (int j = 0; j + 1 < W - 1; ++j) win[j][v] = win[j + 1][v];
        win[W - 2][v] = x[v];
    }
}

// The last W - 1 inputs of every sequence, a channel a thread.  state_out may
// be state_in: a thread reads all that it needs of a state before it writes.
template <typename E, int W>
__device__ __forceinline__ void write_states(const ShortConvArgs& a, int64_t block) {
    const int64_t i = block * 256 + threadIdx.x;
    const int64_t s = i / a.D, c = i % a.D;
    if (s >= a.n_seq) return;
    int64_t first = 0, end = a.T, base = s * a.T * a.D;
    if (a.cu_seqlens) {
        seq_bounds(a.cu_seqlens, s, a.T, first, end);
        base = 0;
    }
    E last[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t at = end - (W - 1) + j;
        last[j] = (E)0.f;
        if (at >= first) last[j] = reinterpret_cast<const E*>(a.x)[base + at * a.D + c];
        else if (a.state_in) last[j] = reinterpret_cast<const E*>(a.state_in)[(s * (W - 1) + (at - first + W - 1)) * a.D + c];
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) reinterpret_cast<E*>(a.state_out)[(s * (W - 1) + j) * a.D + c] = last[j];
}

// The workgroups from `blocks` on write the states.
template <typename E, int W, int V>
__global__ __launch_bounds__(kConvWaves * 64) void kda_short_conv_kernel(ShortConvArgs a, int tile, int tiles, int chunks, unsigned blocks) {
    if (blockIdx.x >= blocks) {
        write_states<E, W>(a, blockIdx.x - blocks);
        return;
    }
    const ConvTile r = conv_tile<V>(a, tile, tiles, chunks);
    if (!r.any) return;
    const int64_t base = (int64_t)r.row * a.T * a.D;
    const Filter<W, V> f(a, r.c);
    Sequences q(a.cu_seqlens, a.n_seq, a.T, r.row, r.t0);
    do {
        const int b = max(q.first, r.t0), e = min(q.end, r.t1);
        if (b >= e) continue;
        float win[W - 1][V];
        window_before<E, W, V>(a, q, base, b, r.c, win);
        const E* x = reinterpret_cast<const E*>(a.x) + base + (int64_t)b * a.D + r.c;
        E* out = reinterpret_cast<E*>(a.out) + base + (int64_t)b * a.D + r.c;
        auto token = [&](const Channels<E, V>& in) {
            float now[V], y[V];
#pragma unroll
            for (int v = 0; v < V; ++v) now[v] = in[v];
            convolve<W, V>(f, win, now, y);
            if (a.silu) {
#pragma unroll
                for (int v = 0; v < V; ++v) y[v] = silu(y[v]);
            }
            put_channels<E, V>(out, y);
            out += a.D;
        };
        constexpr int U = 8;                // tokens on their way together (85 us for 4 x 4096 x 6144, 90 with 4)
        int t = b;
        for (; t + U <= e; t += U) {
            Channels<E, V> in[U];
#pragma unroll
            for (int u = 0; u < U; ++u) in[u] = get_channels<E, V>(x + u * a.D);
            x += U * a.D;
#pragma unroll
            for (int u = 0; u < U; ++u) token(in[u]);
        }
        for (; t < e; ++t) {
            token(get_channels<E, V>(x));
            x += a.D;
        }
    } while (q.end < r.t1 && q.next());
}

// A tile's tokens [b, e) of a sequence need d up to e + W - 2, as dx_p does.
// Walking t from b on, the newest d gives dx of p = t - (W - 1), which before a
// sequence's first token is the gradient of its state.
template <typename E, int W, int V>
__global__ __launch_bounds__(kConvWaves * 64) void kda_short_conv_backward_kernel(ShortConvArgs a, int tile, int tiles, int chunks) {
    const ConvTile r = conv_tile<V>(a, tile, tiles, chunks);
    if (!r.any) return;
    const int64_t base = (int64_t)r.row * a.T * a.D;
    const Filter<W, V> f(a, r.c);
    float dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    Sequences q(a.cu_seqlens, a.n_seq, a.T, r.row, r.t0);
    do {
        const int b = max(q.first, r.t0), e = min(q.end, r.t1);
        if (b >= e) continue;
        float win[W - 1][V], dwin[W - 1][V];        // the inputs and the d before token t
        window_before<E, W, V>(a, q, base, b, r.c, win);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) dwin[j][v] = 0.f;
        const E* x = reinterpret_cast<const E*>(a.x) + base + r.c;
        const E* g = reinterpret_cast<const E*>(a.d_out ? a.d_out : a.x) + base + r.c;       // any that is there
        const bool begins = b == q.first;
        const int behind = q.end - (W - 1);         // the first of the last W - 1 inputs
        // d of a token; OWN: it is one of the tile's
        auto gradient = [&](auto own, const Channels<E, V>& xin, const Channels<E, V>& gin, float (&d)[V]) {
            float now[V], y[V], old[W - 1][V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                now[v] = xin[v];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) old[j][v] = win[j][v];
            }
            convolve<W, V>(f, win, now, y);
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = a.d_out ? gin[v] : 0.f;
            if (a.silu) {
#pragma unroll
                for (int v = 0; v < V; ++v) d[v] *= silu_slope(y[v]);
            }
            if constexpr (decltype(own)::value) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    db[v] += d[v];
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][v] = fmaf(d[v], old[j][v], dw[j][v]);
                    dw[W - 1][v] = fmaf(d[v], now[v], dw[W - 1][v]);
                }
            }
        };
        // the gradient of the input at p = t - (W - 1), from d of token t on; PLAIN: it
        // is one of the tile's, and no state takes part
        auto emit = [&](auto plain, int p, const float (&d)[V]) {
            constexpr bool PLAIN = decltype(plain)::value;
            if (PLAIN || p >= b || begins) {
                float s[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    s[v] = f.w[0][v] * d[v];
#pragma unroll
                    for (int j = 1; j < W; ++j) s[v] = fmaf(f.w[j][v], dwin[W - 1 - j][v], s[v]);
                }
                if (!PLAIN && a.d_state && p >= behind) {
                    const auto more = get_channels<E, V>(reinterpret_cast<const E*>(a.d_state) + ((int64_t)q.s * (W - 1) + (p - behind)) * a.D + r.c);
#pragma unroll
                    for (int v = 0; v < V; ++v) s[v] += more[v];
                }
                if (PLAIN || p >= q.first) put_channels<E, V>(reinterpret_cast<E*>(a.dx) + base + r.c + (int64_t)p * a.D, s);
                else if (a.d_state_in) put_channels<E, V>(reinterpret_cast<E*>(a.d_state_in) + ((int64_t)q.s * (W - 1) + (p - q.first + W - 1)) * a.D + r.c, s);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int j = 0; j + 1 < W - 1; ++j) dwin[j][v] = dwin[j + 1][v];
                dwin[W - 2][v] = d[v];
            }
        };
        // tokens on their way together: 144 us for 4 x 4096 x 6144 in bf16, 178 with 2;
        // 148 with 8 or with the next 4 sent for a turn ahead, which leave two waves a SIMD
        constexpr int U = 4;
        auto group = [&](auto plain, int t) {
            Channels<E, V> xin[U], gin[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = (int64_t)min(t + u, e - 1) * a.D;
                xin[u] = get_channels<E, V>(x + at);
                gin[u] = get_channels<E, V>(g + at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!decltype(plain)::value && t + u >= e) break;
                float d[V];
                gradient(std::true_type{}, xin[u], gin[u], d);
                emit(plain, t + u - (W - 1), d);
            }
        };
        // Most turns need no look at either end: a load that may not be there waits
        // for all that are on their way (163 us without this).
        const int last = min(e, a.d_state ? behind + W - 1 : e) - U;
        for (int t = b; t < e; t += U) {
            if (t >= b + W - 1 && t <= last) group(std::true_type{}, t);
            else group(std::false_type{}, t);
        }
        Channels<E, V> xin[W - 1], gin[W - 1];
#pragma unroll
        for (int u = 0; u < W - 1; ++u) {
            const int64_t at = (int64_t)min(e + u, q.end - 1) * a.D;
            xin[u] = get_channels<E, V>(x + at);
            gin[u] = get_channels<E, V>(g + at);
        }
#pragma unroll
        for (int u = 0; u < W - 1; ++u) {
            float d[V];
            gradient(std::false_type{}, xin[u], gin[u], d);
#pragma unroll
            for (int v = 0; v < V; ++v) d[v] = e + u < q.end ? d[v] : 0.f;
            emit(std::false_type{}, e + u - (W - 1), d);
        }
    } while (q.end < r.t1 && q.next());
    // [tile][weights, bias][channel]
    float* to = a.parts + r.part * (W + 1) * a.D + r.c;
#pragma unroll
    for (int j = 0; j < W; ++j) put_channels<float, V>(to + j * a.D, dw[j]);
    put_channels<float, V>(to + W * a.D, db);
}

// The weights' gradients: sums over the tiles in their order, 64 channels of one
// weight a workgroup, whose waves have every fourth tile.  In 64 bits, as there
// can be any number.  The workgroups behind those pass the gradients of the states
// of sequences without tokens through, a wave for each sequence.
template <typename E, int W>
__global__ __launch_bounds__(256) void kda_short_conv_sum_kernel(ShortConvArgs a, int64_t parts, int blocks, unsigned sums) {
    __shared__ double sum[kConvWaves][64];
    const int lane = threadIdx.x & 63, wave = wave_of_block();
    if (blockIdx.x >= sums) {
        const int64_t s = (int64_t)(blockIdx.x - sums) * kConvWaves + wave, each = (W - 1) * a.D;
        if (s >= a.n_seq) return;
        int64_t first = 0, end = a.T;
        if (a.cu_seqlens) seq_bounds(a.cu_seqlens, s, a.T, first, end);
        if (first < end) return;
        for (int64_t i = s * each + lane; i < (s + 1) * each; i += 64)
            reinterpret_cast<E*>(a.d_state_in)[i] = a.d_state ? reinterpret_cast<const E*>(a.d_state)[i] : (E)0.f;
        return;
    }
    const int64_t c = (int64_t)(blockIdx.x % blocks) * 64 + lane;
    const int j = blockIdx.x / blocks;
    double s = 0.;
    if (c < a.D) {
        const float* from = a.parts + (int64_t)j * a.D + c;
        const int64_t stride = (W + 1) * a.D;
#pragma unroll 8
        for (int64_t i = wave; i < parts; i += kConvWaves) s += from[i * stride];
    }
    sum[wave][lane] = s;
    __syncthreads();
    if (wave != 0 || c >= a.D) return;
#pragma unroll
    for (int w = 1; w < kConvWaves; ++w) s += sum[w][lane];
    if (j < W) a.dweight[c * W + j] = (float)s;
    else a.dbias[c] = (float)s;
}

template <typename E, int W, int V>
__global__ __launch_bounds__(256) void kda_short_conv_step_kernel(ShortConvStepArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, per = a.D / V;
    const int64_t row = i / per, c = (i - row * per) * V;
    if (row >= a.N) return;
    E* state = reinterpret_cast<E*>(a.state) + row * (W - 1) * a.D + c;
    Channels<E, V> in[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) in[j] = get_channels<E, V>(state + j * a.D);
    in[W - 1] = get_channels<E, V>(reinterpret_cast<const E*>(a.x) + row * a.D + c);
    float y[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float s = a.bias ? a.bias[c + v] : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(a.weight[(c + v) * W + j], in[j][v], s);
        y[v] = a.silu ? silu(s) : s;
    }
    put_channels<E, V>(reinterpret_cast<E*>(a.out) + row * a.D + c, y);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) __builtin_memcpy(state + j * a.D, &in[j + 1], sizeof in[j]);
}

struct ConvPlan {
    int tile, tiles, chunks;
    int64_t waves, blocks;
};

// Tokens of a tile: as many as leave the card enough waves, for the inputs
// before each tile are read twice.  (The backward of 4 x 4096 x 6144 takes 144 us
// with tiles of 64 and of 128; with 32 it took 180 where 64 took 161.)
ConvPlan conv_plan(const ShortConvArgs& a, int vec) {
    ConvPlan p = {};
    if (a.D < vec) vec = 1;
    p.chunks = (int)((a.D + 64 * vec - 1) / (64 * vec));
    p.tile = 64;
    while (p.tile > 16 && a.B * ((a.T + p.tile - 1) / p.tile) * p.chunks < 4096) p.tile /= 2;
    p.tiles = (int)((a.T + p.tile - 1) / p.tile);
    p.waves = a.B * p.tiles * p.chunks;
    p.blocks = (p.waves + kConvWaves - 1) / kConvWaves;
    return p;
}

template <typename E, int W>
hipError_t conv_forward(const ShortConvArgs& a, hipStream_t s) {
    const ConvPlan p = conv_plan(a, kForward<E>);
    const unsigned blocks = a.n_seq > 0 ? (unsigned)p.blocks : 0u, states = a.state_out ? (unsigned)((a.n_seq * a.D + 255) / 256) : 0u;
    const auto kernel = a.D >= kForward<E> ? kda_short_conv_kernel<E, W, kForward<E>> : kda_short_conv_kernel<E, W, 1>;
    // a state that is written in place may still be read by the tiles
    const bool apart = a.state_out == a.state_in && blocks > 0 && states > 0;
    if (blocks + states > 0) hipLaunchKernelGGL(kernel, dim3(apart ? blocks : blocks + states), dim3(kConvWaves * 64), 0, s, a, p.tile, p.tiles, p.chunks, blocks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !apart) return e;
    hipLaunchKernelGGL(kernel, dim3(states), dim3(kConvWaves * 64), 0, s, a, p.tile, p.tiles, p.chunks, 0u);
    return hipGetLastError();
}

template <typename E, int W>
hipError_t conv_backward(const ShortConvArgs& a, hipStream_t s) {
    const ConvPlan p = conv_plan(a, kBackward);
    hipError_t e;
    const bool any = p.waves > 0 && a.n_seq > 0;
    if (any) {
        const dim3 grid((unsigned)p.blocks), block(kConvWaves * 64);
        if (a.D >= kBackward) hipLaunchKernelGGL((kda_short_conv_backward_kernel<E, W, kBackward>), grid, block, 0, s, a, p.tile, p.tiles, p.chunks);
        else hipLaunchKernelGGL((kda_short_conv_backward_kernel<E, W, 1>), grid, block, 0, s, a, p.tile, p.tiles, p.chunks);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int blocks = (int)((a.D + 63) / 64);
    const unsigned sums = (unsigned)(blocks * (W + (a.dbias ? 1 : 0)));
    const unsigned through = a.d_state_in && (a.cu_seqlens || a.T == 0) ? (unsigned)((a.n_seq + kConvWaves - 1) / kConvWaves) : 0u;
    hipLaunchKernelGGL((kda_short_conv_sum_kernel<E, W>), dim3(sums + through), dim3(256), 0, s, a, any ? a.B * p.tiles : 0, blocks, sums);
    return hipGetLastError();
}

template <typename E, int W>
hipError_t conv_step(const ShortConvStepArgs& a, hipStream_t s) {
    constexpr int V = kForward<E> / 2;
    if (a.D % V == 0)
        hipLaunchKernelGGL((kda_short_conv_step_kernel<E, W, V>), dim3((unsigned)((a.N * (a.D / V) + 255) / 256)), dim3(256), 0, s, a);
    else
        hipLaunchKernelGGL((kda_short_conv_step_kernel<E, W, 1>), dim3((unsigned)((a.N * a.D + 255) / 256)), dim3(256), 0, s, a);
    return hipGetLastError();
}

template <typename F>
hipError_t by_taps(int taps, F&& f) {
    if (taps == 2) return f(std::integral_constant<int, 2>{});
    if (taps == 3) return f(std::integral_constant<int, 3>{});
    return f(std::integral_constant<int, 4>{});
}

}  // namespace

bool short_conv_fits(const ShortConvArgs& a, bool bf16) {
    const int64_t most = UINT32_MAX / (kConvWaves * 64);
    return conv_plan(a, bf16 ? kForward<__bf16> : kForward<float>).blocks + (a.n_seq * a.D + 255) / 256 <= most &&
           conv_plan(a, kBackward).blocks <= most && (a.D + 63) / 64 * (a.taps + 1) + a.n_seq / kConvWaves < most;
}

size_t short_conv_backward_workspace_bytes(const ShortConvArgs& a, bool) {
    return (size_t)(a.B * conv_plan(a, kBackward).tiles) * (size_t)(a.taps + 1) * (size_t)a.D * sizeof(float);
}

hipError_t launch_short_conv(bool bf16, const ShortConvArgs& a, hipStream_t s) {
    return by_taps(a.taps, [&](auto w) {
        return bf16 ? conv_forward<__bf16, decltype(w)::value>(a, s) : conv_forward<float, decltype(w)::value>(a, s);
    });
}

hipError_t launch_short_conv_backward(bool bf16, const ShortConvArgs& a, hipStream_t s) {
    return by_taps(a.taps, [&](auto w) {
        return bf16 ? conv_backward<__bf16, decltype(w)::value>(a, s) : conv_backward<float, decltype(w)::value>(a, s);
    });
}

hipError_t launch_short_conv_step(bool bf16, const ShortConvStepArgs& a, hipStream_t s) {
    return by_taps(a.taps, [&](auto w) {
        return bf16 ? conv_step<__bf16, decltype(w)::value>(a, s) : conv_step<float, decltype(w)::value>(a, s);
    });
}

}  // namespace kda

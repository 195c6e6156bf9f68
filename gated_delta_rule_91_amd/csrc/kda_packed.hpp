// kda_packed.hpp -- device-side building blocks of the kernels whose waves
// walk along the tokens of packed batches (short convolution, selective scan):
// the sequence of a token, and vectors of channels at any alignment.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_common.hpp"

namespace kda {

// N elements as one access, at any multiple of the element's size: rows of an
// odd width do not keep vectors aligned.
template <typename E, int N> struct Channels {
    E v[N];
    __device__ __forceinline__ float operator[](int i) const { return to_f32(v[i]); }
};
template <typename E, int N>
__device__ __forceinline__ Channels<E, N> get_channels(const E* p) {
    Channels<E, N> x;
    __builtin_memcpy(&x, p, sizeof x);
    return x;
}
template <typename E, int N>
__device__ __forceinline__ void put_channels(E* p, const float (&x)[N]) {
    Channels<E, N> y;
#pragma unroll
    for (int i = 0; i < N; ++i) y.v[i] = from_f32<E>(x[i]);
    __builtin_memcpy(p, &y, sizeof y);
}

// The sequences of a row, walked along the tokens by a whole wave (all of it
// the same in every lane, and all lanes take part).
struct Sequences {
    const int32_t* cu;      // null: one sequence, the whole row
    int n, T;
    int s, first, end;      // sequence s holds tokens [first, end)
    __device__ __forceinline__ void bounds() {
        int64_t b, e;
        seq_bounds(cu, s, T, b, e);
        first = __builtin_amdgcn_readfirstlane((int)b);
        end = __builtin_amdgcn_readfirstlane((int)e);
    }
    // The last sequence of [lo, lo + many) that begins at or before t, 64
    // candidates at a time in the lanes: one load of latency up to 64
    // sequences, two up to 4096.
    __device__ __forceinline__ void find(int t, int lo, int many) {
        while (many > 1) {
            const int stride = (many + 63) / 64, at = lo + (int)(threadIdx.x & 63) * stride;
            const bool before = at < lo + many && cu[at] <= t;
            const int k = __popcll(__ballot(before));
            const int next = lo + (k > 0 ? k - 1 : 0) * stride;
            many = min(stride, lo + many - next);
            lo = next;
        }
        s = __builtin_amdgcn_readfirstlane(lo);
        bounds();
    }
    // at the last sequence that begins at or before t
    __device__ __forceinline__ Sequences(const int32_t* cu_, int64_t n_, int64_t T_, int row, int t)
        : cu(cu_), n((int)n_), T((int)T_), s(row), first(0), end((int)T_) {
        if (cu) find(t, 0, n);
    }
    // On to the next sequence with tokens; false: there is none.  Over empty
    // ones, of which there may be any number at one place, it is searched.
    __device__ __forceinline__ bool next() {
        if (!cu || s + 1 >= n) return false;
        const int at = end;
        ++s;
        bounds();
        if (end <= at && s + 1 < n) find(at, s, n - s);
        return end > at;
    }
    // The same towards the row's begin.
    __device__ __forceinline__ bool previous() {
        if (!cu || s == 0) return false;
        const int at = first;
        --s;
        bounds();
        if (first >= at && s > 0) find(at - 1, 0, s);
        return first < at;
    }
};

}  // namespace kda

// rope.cuh -- what the kernels for rotary positions share: vectors of elements, frequencies
// as fractions of a turn, and the strides of a tensor. P is the C structure of a call
// (llsa_rope_params, llsa_rope_grid_params), whose fields of the same names mean the same.
#pragma once

#include <math.h>

#include <algorithm>

#include "entry.h"
#include "internal.h"

namespace llsa {

constexpr int kRopeMaxPairs = 128;  // d <= 256
constexpr int kRopeThreads = 256;
constexpr double kPi = 3.14159265358979323846;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T>
union Vec {
    uint4 u;
    T e[16 / sizeof(T)];
};

// The scaled frequency of a pair whose own is w.
template <typename P>
double rope_scaled(const P& p, double w) {
    if (p.scaling == LLSA_ROPE_SCALE_LINEAR) w /= p.factor;
    if (p.scaling == LLSA_ROPE_SCALE_WAVELENGTH) {
        const double turns = p.orig_len * w / (2 * kPi);
        const double g = std::min(1.0, std::max(0.0, (turns - p.low) / (p.high - p.low)));
        w *= g + (1 - g) / p.factor;
    }
    return w;
}

// w radians per position as turns, a fraction of 2^64; false where w is no number.
inline bool rope_turns(double w, uint64_t* out) {
    double f = w / (2 * kPi);
    f -= floor(f);
    if (!(f >= 0.0 && f < 1.0)) return false;
    // below 2^-11 the fraction has bits behind 2^-64: rounded there
    *out = (uint64_t)(f * 18446744073709551616.0 + (f < 4.8828125e-4 ? 0.5 : 0.0));
    return true;
}

// The strides of one tensor: the caller's, or the contiguous ones. An output's
// rows must not lie over one another.
template <typename P>
int rope_strides(const long long* given, const P& p, int heads, bool output, long long* out) {
    const long long want = p.dtype == LLSA_DTYPE_BF16 ? 8 : 4;  // elements in 16 bytes
    if (!given || (given[0] == 0 && given[1] == 0 && given[2] == 0)) {
        out[0] = (long long)heads * p.n * p.d;
        out[1] = (long long)p.n * p.d;
        out[2] = p.d;
        return LLSA_OK;
    }
    const int extent[3] = {p.batch, heads, p.n};
    for (int i = 0; i < 3; i++) {
        out[i] = extent[i] > 1 ? given[i] : 0;  // one entry: the stride is never walked
        if (out[i] % want != 0) return LLSA_ERR_ALIGN;
        if (output && extent[i] > 1 && out[i] == 0) return LLSA_ERR_INVALID_ARG;
    }
    return LLSA_OK;
}

}  // namespace llsa

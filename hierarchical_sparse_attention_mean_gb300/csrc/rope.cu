// rope.cu -- rotary positions of q and k in one launch.
//
// Mathematics: pair (x, y) of a token at position p becomes
// A (x cos a - y sin a, x sin a + y cos a), a = p w_i. Both the rotation and
// its gradient (the rotation by -a) are the same pass.
//
// Angles. A far position loses its angle in fp32 (p w at p = 10^6 is good to
// 0.06 rad), so the frequency is held as f = w / 2 pi turns in a 64-bit
// fraction: the integer product p f modulo 2^64 is the turn's fraction itself,
// with no range reduction left to do, and its top 32 bits as a signed number
// of half turns are what sincospif takes, rounded to fp32: 2^-26 turns. The frequency
// comes from double precision and adds up to 2^-54 turns per position (w <= 1).
//
// Bound by HBM: every element is read and written once. The angles depend on
// the token and the pair alone, so a thread takes one 16-byte unit of a token
// (two units a half apart in the half layout) and walks a run of heads with
// its sines and cosines in registers.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "entry.h"
#include "internal.h"

namespace llsa {
namespace {

constexpr int kMaxPairs = 128;  // d <= 256
constexpr int kThreads = 256;
constexpr double kPi = 3.14159265358979323846;

struct RopeArgs {
    const void* in[2];
    void* out[2];
    long long in_stride[2][3], out_stride[2][3];  // batch, head, token (elements)
    const int* pos;
    long long rows;  // batch * n
    int heads[2];    // q, k
    int n, d, rot, axes, width, tile, offset, batched;
    int units;           // threads per token
    int heads_per_thread;
    float amplitude, sign;
    uint64_t freq[kMaxPairs];  // per pair of one segment: turns per position, as a fraction of 2^64
};

enum { kInterleaved = 0, kHalfVector = 1, kHalfScalar = 2 };

// Position of token t of batch entry b on axis a.
__device__ __forceinline__ int position(const RopeArgs& a, long long b, int t, int axis) {
    if (a.pos) return __ldg(a.pos + ((a.batched ? b * a.n : 0) + t) * a.axes + axis);
    if (a.axes == 1) return a.offset + t;
    if (!a.tile) return axis == 0 ? t / a.width : t % a.width;
    int px, py;
    block_patch(t, px, py);
    return axis == 0 ? py : px;
}

__device__ __forceinline__ void turn(const RopeArgs& a, int pos, int pair, float& c, float& s) {
    const uint64_t f = (uint64_t)(long long)pos * a.freq[pair];
    sincospif((float)(int)(uint32_t)(f >> 32) * 4.656612873077393e-10f, &s, &c);  // * 2^-31
    c *= a.amplitude;
    s *= a.amplitude * a.sign;
}

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

// One thread: unit u of one token, for heads h0 .. h0 + heads_per_thread - 1 of
// the q heads followed by the k heads.
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int V = 16 / sizeof(T);
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (idx >= a.rows * a.units) return;
    int u, t;
    long long b;
    if (a.rows * a.units <= 0x7fffffffLL) {  // 64-bit divisions cost more than the rest of the thread's set-up
        const uint32_t i = (uint32_t)idx, row = i / (uint32_t)a.units;
        u = (int)(i - row * a.units);
        b = row / (uint32_t)a.n;
        t = (int)(row - (uint32_t)b * a.n);
    } else {
        const long long row = idx / a.units;
        u = (int)(idx - row * a.units);
        b = row / a.n;
        t = (int)(row - b * a.n);
    }
    const int seg = a.rot / a.axes, half = seg / 2;
    constexpr int P = MODE == kInterleaved ? V / 2 : MODE == kHalfVector ? V : 1;  // pairs of a unit
    float c[P], s[P];
    int col0, col1 = 0;      // first column of the unit's vector(s)
    bool copy = false;       // columns behind rot_dim
    if constexpr (MODE == kInterleaved) {
        col0 = u * V;
        copy = col0 >= a.rot;
#pragma unroll
        for (int i = 0; i < P; i++) {
            const int pr = col0 / 2 + i;  // pair of the head
            c[i] = s[i] = 0.f;
            if (2 * pr < a.rot) {
                const int axis = pr >= half ? 1 : 0;
                turn(a, position(a, b, t, axis), pr - axis * half, c[i], s[i]);
            }
        }
    } else {
        const int per_seg = half / P, turned = per_seg * a.axes;
        if (u < turned) {
            const int axis = u >= per_seg ? 1 : 0;
            const int i0 = (u - axis * per_seg) * P;
            col0 = axis * seg + i0;
            col1 = col0 + half;
            const int pos = position(a, b, t, axis);
#pragma unroll
            for (int i = 0; i < P; i++) turn(a, pos, i0 + i, c[i], s[i]);
        } else {
            copy = true;
            col0 = a.rot + (u - turned) * (MODE == kHalfVector ? V : 1);
        }
    }
    const int total = a.heads[0] + a.heads[1];
    const int h0 = blockIdx.y * a.heads_per_thread, h1 = min(h0 + a.heads_per_thread, total);
    auto place = [&](int h, const T*& in, T*& out) {
        const int w = h >= a.heads[0] ? 1 : 0;
        const int hh = h - w * a.heads[0];
        in = static_cast<const T*>(a.in[w]) + b * a.in_stride[w][0] + hh * a.in_stride[w][1] + t * a.in_stride[w][2];
        out = static_cast<T*>(a.out[w]) + b * a.out_stride[w][0] + hh * a.out_stride[w][1] + t * a.out_stride[w][2];
    };
    if constexpr (MODE == kHalfScalar) {
        for (int h = h0; h < h1; h++) {
            const T* in;
            T* out;
            place(h, in, out);
            if (copy) {
                out[col0] = in[col0];
            } else {
                const float x = to_float(in[col0]), y = to_float(in[col1]);
                out[col0] = from_float<T>(x * c[0] - y * s[0]);
                out[col1] = from_float<T>(x * s[0] + y * c[0]);
            }
        }
    } else {
        // Outputs may be the inputs, so loads do not move over stores by
        // themselves. In fp32 two heads are loaded before the first is stored; in
        // bf16, where a vector is twice the arithmetic, the registers are worth more
        // as occupancy (12 heads x 65,536 tokens 69 us, with two 76, with four 87).
        constexpr int HB = sizeof(T) == 2 ? 1 : 2;
        for (int h = h0; h < h1; h += HB) {
            Vec<T> x[HB], y[HB];
            T* out[HB];
#pragma unroll
            for (int k = 0; k < HB; k++)
                if (h + k < h1) {
                    const T* in;
                    place(h + k, in, out[k]);
                    x[k].u = *reinterpret_cast<const uint4*>(in + col0);
                    if (MODE == kHalfVector && !copy) y[k].u = *reinterpret_cast<const uint4*>(in + col1);
                }
#pragma unroll
            for (int k = 0; k < HB; k++) {
                if (h + k >= h1) break;
                if (!copy) {
#pragma unroll
                    for (int i = 0; i < P; i++) {
                        T& first = x[k].e[MODE == kInterleaved ? 2 * i : i];
                        T& second = MODE == kInterleaved ? x[k].e[2 * i + 1] : y[k].e[i];
                        if (MODE == kInterleaved && col0 + 2 * i >= a.rot) break;  // rot_dim may end inside the vector
                        const float p = to_float(first), q = to_float(second);
                        first = from_float<T>(p * c[i] - q * s[i]);
                        second = from_float<T>(p * s[i] + q * c[i]);
                    }
                    if (MODE == kHalfVector) *reinterpret_cast<uint4*>(out[k] + col1) = y[k].u;
                }
                *reinterpret_cast<uint4*>(out[k] + col0) = x[k].u;
            }
        }
    }
}

// Turns per position of every pair of a segment as fractions of 2^64, and the
// amplitude.
int derive_rope(const llsa_rope_params* p, RopeArgs* a) {
    const int seg = a->rot / a->axes, h = seg / 2;
    double base = p->base, amplitude = 1.0;
    if (p->scaling == LLSA_ROPE_SCALE_BASE) {
        if (seg <= 2) return LLSA_ERR_SHAPE;
        base *= pow(p->factor, (double)seg / (seg - 2));
        if (!isfinite(base) || !(base > 0)) return LLSA_ERR_INVALID_ARG;
    }
    for (int i = 0; i < h; i++) {
        double w = pow(base, -2.0 * i / seg);
        if (p->scaling == LLSA_ROPE_SCALE_LINEAR) w /= p->factor;
        if (p->scaling == LLSA_ROPE_SCALE_WAVELENGTH) {
            const double turns = p->orig_len * w / (2 * kPi);
            const double g = std::min(1.0, std::max(0.0, (turns - p->low) / (p->high - p->low)));
            w *= g + (1 - g) / p->factor;
        }
        double f = w / (2 * kPi);
        f -= floor(f);
        if (!(f >= 0.0 && f < 1.0)) return LLSA_ERR_INVALID_ARG;  // not a number
        // below 2^-11 the fraction has bits behind 2^-64: rounded there
        a->freq[i] = (uint64_t)(f * 18446744073709551616.0 + (f < 4.8828125e-4 ? 0.5 : 0.0));
    }
    // stretched positions ask for sharper scores; the logarithm would turn them flat and at last around below 1
    if (p->scaling == LLSA_ROPE_SCALE_WAVELENGTH && p->factor > 1.0) amplitude = 0.1 * log(p->factor) + 1.0;
    if (p->amplitude != 0.0) amplitude = p->amplitude;
    a->amplitude = (float)amplitude;
    return isfinite(a->amplitude) ? LLSA_OK : LLSA_ERR_INVALID_ARG;
}

int check_rope(const llsa_rope_params* p, int has_pos) {
    if (!p) return LLSA_ERR_INVALID_ARG;
    if (p->batch < 0 || p->heads < 0 || p->kv_heads < 0 || p->n < 0) return LLSA_ERR_INVALID_ARG;
    if (p->dtype != LLSA_DTYPE_BF16 && p->dtype != LLSA_DTYPE_F32) return LLSA_ERR_DTYPE;
    if (p->layout != LLSA_ROPE_HALF && p->layout != LLSA_ROPE_INTERLEAVED) return LLSA_ERR_INVALID_ARG;
    if (p->axes != 1 && p->axes != 2) return LLSA_ERR_INVALID_ARG;
    if (p->token_order != LLSA_ORDER_TILE && p->token_order != LLSA_ORDER_RASTER) return LLSA_ERR_INVALID_ARG;
    if (p->pos_batched != 0 && p->pos_batched != 1) return LLSA_ERR_INVALID_ARG;
    if (p->scaling < LLSA_ROPE_SCALE_NONE || p->scaling > LLSA_ROPE_SCALE_WAVELENGTH) return LLSA_ERR_INVALID_ARG;
    if (!(p->base > 1.0) || isinf(p->base)) return LLSA_ERR_INVALID_ARG;
    if (p->scaling != LLSA_ROPE_SCALE_NONE && (!(p->factor > 0.0) || isinf(p->factor))) return LLSA_ERR_INVALID_ARG;
    if (p->scaling == LLSA_ROPE_SCALE_WAVELENGTH &&
        (p->orig_len < 1 || !(p->low < p->high) || isinf(p->low) || isinf(p->high)))
        return LLSA_ERR_INVALID_ARG;
    if (isnan(p->amplitude) || isinf(p->amplitude)) return LLSA_ERR_INVALID_ARG;
    if (p->d < 8 || p->d > 256 || p->d % 8 != 0) return LLSA_ERR_SHAPE;
    if (p->rot_dim < 0 || p->rot_dim > p->d) return LLSA_ERR_SHAPE;
    const int rot = p->rot_dim ? p->rot_dim : p->d;
    if (rot % (2 * p->axes) != 0) return LLSA_ERR_SHAPE;
    if (has_pos) return LLSA_OK;  // the fields below say where positions come from when none are given
    if (p->axes == 1) {
        if (p->width != 0) return LLSA_ERR_INVALID_ARG;
        if ((long long)p->pos_offset + p->n - 1 > 2147483647LL) return LLSA_ERR_INVALID_ARG;
    } else {
        if (p->pos_offset != 0 || p->width < 1) return LLSA_ERR_INVALID_ARG;
        if (p->token_order == LLSA_ORDER_TILE) {
            long long side = 1;
            while (side < p->width) side *= 4;
            if (side != p->width || side * side != p->n) return LLSA_ERR_SHAPE;
        }
    }
    return LLSA_OK;
}

// The strides of one tensor: the caller's, or the contiguous ones. An output's
// rows must not lie over one another.
int take_strides(const long long* given, const llsa_rope_params* p, int heads, bool output, long long* out) {
    const long long want = p->dtype == LLSA_DTYPE_BF16 ? 8 : 4;  // elements in 16 bytes
    if (!given || (given[0] == 0 && given[1] == 0 && given[2] == 0)) {
        out[0] = (long long)heads * p->n * p->d;
        out[1] = (long long)p->n * p->d;
        out[2] = p->d;
        return LLSA_OK;
    }
    const int extent[3] = {p->batch, heads, p->n};
    for (int i = 0; i < 3; i++) {
        out[i] = extent[i] > 1 ? given[i] : 0;  // one entry: the stride is never walked
        if (out[i] % want != 0) return LLSA_ERR_ALIGN;
        if (output && extent[i] > 1 && out[i] == 0) return LLSA_ERR_INVALID_ARG;
    }
    return LLSA_OK;
}

template <typename T>
int launch_rope(const llsa_rope_params* p, RopeArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    const int half = a.rot / a.axes / 2;
    int mode, units;
    if (p->layout == LLSA_ROPE_INTERLEAVED) {
        mode = kInterleaved;
        units = a.d / V;
    } else if (half % V == 0) {
        mode = kHalfVector;
        units = a.axes * (half / V) + (a.d - a.rot) / V;
    } else {  // halves that are no whole number of 16-byte vectors: one pair, or one column, per thread
        mode = kHalfScalar;
        units = a.rot / 2 + (a.d - a.rot);
    }
    a.units = units;
    const int total = a.heads[0] + a.heads[1];
    const long long threads = a.rows * units;
    // As many heads per thread (the sines are computed once for them) as leave
    // one wave of resident threads (6 heads x 10,785 tokens in fp32 14 us; two waves, 22).
    // 65,535 blocks is the most that the grid's second dimension takes.
    const long long want = (long long)sm_count() * 2048;
    const long long least = (total + 65534) / 65535;
    a.heads_per_thread = (int)std::min<long long>(total, std::max(least, threads * total / want));
    const long long gx = (threads + kThreads - 1) / kThreads;
    const int gy = (total + a.heads_per_thread - 1) / a.heads_per_thread;
    a.heads_per_thread = (total + gy - 1) / gy;  // the same share for all
    if (gx > 2147483647LL) return LLSA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    if (mode == kInterleaved) LLSA_LAUNCH("rope", st, rope_kernel<T, kInterleaved><<<grid, kThreads, 0, st>>>(a));
    else if (mode == kHalfVector) LLSA_LAUNCH("rope", st, rope_kernel<T, kHalfVector><<<grid, kThreads, 0, st>>>(a));
    else LLSA_LAUNCH("rope", st, rope_kernel<T, kHalfScalar><<<grid, kThreads, 0, st>>>(a));
    return LLSA_OK;
}

}  // namespace
}  // namespace llsa

using namespace llsa;

extern "C" int llsa_rope(const llsa_rope_params* p, const llsa_rope_strides* strides, const void* q, const void* k,
                         const int32_t* pos, void* q_out, void* k_out, int inverse, void* stream) {
    CallRange range("llsa_rope");
    LLSA_TRY(check_rope(p, pos != nullptr));
    if (inverse != 0 && inverse != 1) return LLSA_ERR_INVALID_ARG;
    RopeArgs a;
    memset(&a, 0, sizeof(a));
    a.d = p->d;
    a.rot = p->rot_dim ? p->rot_dim : p->d;
    a.axes = p->axes;
    LLSA_TRY(derive_rope(p, &a));
    const long long total = (long long)p->heads + p->kv_heads;
    if (p->batch == 0 || p->n == 0 || total == 0) return LLSA_OK;
    if (total > (1 << 30) || (double)p->batch * p->n * total * p->d > (double)(1LL << 40)) return LLSA_ERR_UNSUPPORTED;
    if (p->heads > 0) LLSA_TRY(check_ptrs({q, q_out}));
    if (p->kv_heads > 0) LLSA_TRY(check_ptrs({k, k_out}));
    if (pos && (reinterpret_cast<uintptr_t>(pos) & 3u)) return LLSA_ERR_ALIGN;
    LLSA_TRY(take_strides(strides ? strides->q : nullptr, p, p->heads, false, a.in_stride[0]));
    LLSA_TRY(take_strides(strides ? strides->k : nullptr, p, p->kv_heads, false, a.in_stride[1]));
    LLSA_TRY(take_strides(strides ? strides->q_out : nullptr, p, p->heads, true, a.out_stride[0]));
    LLSA_TRY(take_strides(strides ? strides->k_out : nullptr, p, p->kv_heads, true, a.out_stride[1]));
    // a tensor may be its own output only if every element goes back to its own place
    if (p->heads > 0 && q == q_out && memcmp(a.in_stride[0], a.out_stride[0], sizeof(a.in_stride[0])) != 0)
        return LLSA_ERR_INVALID_ARG;
    if (p->kv_heads > 0 && k == k_out && memcmp(a.in_stride[1], a.out_stride[1], sizeof(a.in_stride[1])) != 0)
        return LLSA_ERR_INVALID_ARG;
    LLSA_TRY(device_ready());
    a.in[0] = q;
    a.in[1] = k;
    a.out[0] = q_out;
    a.out[1] = k_out;
    a.pos = pos;
    a.rows = (long long)p->batch * p->n;
    a.heads[0] = p->heads;
    a.heads[1] = p->kv_heads;
    a.n = p->n;
    a.width = p->width;
    a.tile = p->token_order == LLSA_ORDER_TILE;
    a.offset = p->pos_offset;
    a.batched = p->pos_batched;
    a.sign = inverse ? -1.0f : 1.0f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return p->dtype == LLSA_DTYPE_BF16 ? launch_rope<__nv_bfloat16>(p, a, st) : launch_rope<float>(p, a, st);
}

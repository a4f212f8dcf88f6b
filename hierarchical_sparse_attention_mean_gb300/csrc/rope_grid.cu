// rope_grid.cu -- rotary positions on up to four axes (time, height, width) of q and k
// in one launch.
//
// Mathematics: pair (x, y) of axis a of a token at position p on that axis becomes
// A (x cos t - y sin t, x sin t + y cos t), t = p step_a w; angles as in rope.cu, a
// 64-bit fraction of a turn times the integer position. Every pair has a frequency and
// an axis of its own in the call's tables, so the three ways of handing columns and
// frequencies to axes are one kernel.
//
// Bound by HBM: every element is read and written once, 2 x 12 heads x 65,536 tokens of 64
// columns (403 MB) in 67 us among others, 6.0 TB/s. A thread takes one vector of a
// token (two a half apart in the half layout) and walks a run of heads with its sines
// and cosines in registers. Segments of unequal axes need not be whole 16-byte vectors:
// the half layout takes the widest vector that divides them all, so that 16 + 24 + 24
// columns of bf16 (halves of 8, 12 and 12) still move 8 bytes at a time. A thread has one head
// in flight: fp32 of 20 packed heads x 2 x 4,095 tokens, half layout, 33.6 us, 73 % of a copy's rate.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "rope.cuh"

namespace llsa {
namespace {

constexpr int kAxes = LLSA_ROPE_MAX_AXES, kThreads = kRopeThreads;

struct GridArgs {
    const void* in[2];
    void* out[2];
    long long in_stride[2][3], out_stride[2][3];  // batch, head, token (elements)
    const int* pos;
    long long rows;  // batch * n
    int heads[2];    // q, k
    int n, d, rot, axes, tile, batched;
    int extent[kAxes], offset[kAxes];
    int first[kAxes + 1];  // first pair of an axis' own segment; one segment of all pairs where the head is one ladder
    int segments;
    int units;             // threads per token
    int heads_per_thread;
    float amplitude, sign;
    uint8_t axis[kRopeMaxPairs];
    uint64_t freq[kRopeMaxPairs];  // turns per position, as a fraction of 2^64
};

// Positions of token t of batch entry b on all axes.
__device__ __forceinline__ void grid_position(const GridArgs& a, long long b, int t, int (&p)[kAxes]) {
    if (a.pos) {
        const int* at = a.pos + ((a.batched ? b * a.n : 0) + t) * a.axes;
#pragma unroll
        for (int i = 0; i < kAxes; i++) p[i] = i < a.axes ? at[i] : 0;
        return;
    }
    uint32_t rest = (uint32_t)t;
    int px = 0, py = 0;
    if (a.tile) {  // the last two axes are a frame in tile order
        uint32_t frame = 1;
#pragma unroll
        for (int i = kAxes - 1; i >= 1; i--)
            if (i == a.axes - 1) frame = (uint32_t)a.extent[i] * (uint32_t)a.extent[i - 1];
        const uint32_t which = rest / frame;
        block_patch((int)(rest - which * frame), px, py);
        rest = which;
    }
#pragma unroll
    for (int i = kAxes - 1; i >= 0; i--) {
        int v = 0;
        if (i < a.axes) {
            if (a.tile && i >= a.axes - 2) {
                v = i == a.axes - 1 ? px : py;
            } else {
                const uint32_t e = (uint32_t)a.extent[i], q = rest / e;
                v = (int)(rest - q * e);
                rest = q;
            }
            v += a.offset[i];
        }
        p[i] = v;
    }
}

__device__ __forceinline__ void grid_turn(const GridArgs& a, const int (&p)[kAxes], int pair, float& c, float& s) {
    const int axis = a.axis[pair];
    int pos = p[0];
#pragma unroll
    for (int i = 1; i < kAxes; i++) pos = axis == i ? p[i] : pos;
    const uint64_t f = (uint64_t)(long long)pos * a.freq[pair];
    sincospif((float)(int)(uint32_t)(f >> 32) * 4.656612873077393e-10f, &s, &c);  // * 2^-31
    c *= a.amplitude;
    s *= a.amplitude * a.sign;
}

template <int BYTES>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

template <>
struct Word<32> { struct type { uint4 a, b; }; };

template <typename T, int W>
union Few {
    typename Word<W * sizeof(T)>::type u;
    T e[W];
    __device__ Few() {}
};

// One thread: unit u of one token, for heads h0 .. h0 + heads_per_thread - 1 of the q
// heads followed by the k heads. W elements per vector; PAIRED: neighbouring columns
// are a pair, else two vectors hold W pairs. T: the inputs' type, O: the outputs'.
template <typename T, typename O, int W, bool PAIRED>
__global__ void __launch_bounds__(kThreads) rope_grid_kernel(const __grid_constant__ GridArgs a) {
    const long long idx = (long long)blockIdx.x * kThreads + threadIdx.x;
    close_ahead();
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
    constexpr int P = PAIRED ? W / 2 : W;  // pairs of a unit
    float c[P], s[P];
    int col0, col1 = 0, first = 0;  // columns of the vector(s), first pair
    bool copy;                      // columns behind the turned ones
    if constexpr (PAIRED) {
        col0 = u * W;
        first = col0 / 2;
        copy = col0 >= a.rot;
    } else {
        const int turned = a.rot / 2 / W;
        copy = u >= turned;
        first = u * W;
        if (copy) {
            col0 = a.rot + (u - turned) * W;
        } else {
            int begin = 0, end = a.first[1];
#pragma unroll
            for (int i = 1; i < kAxes; i++)
                if (i < a.segments && first >= a.first[i]) {
                    begin = a.first[i];
                    end = a.first[i + 1];
                }
            col0 = begin + first;        // 2 * begin + (first - begin)
            col1 = col0 + end - begin;
        }
    }
    if (!copy) {
        int p[kAxes];
        if (a.pos) close_wait();
        grid_position(a, b, t, p);
#pragma unroll
        for (int i = 0; i < P; i++) {
            c[i] = s[i] = 0.f;
            if (!PAIRED || 2 * (first + i) < a.rot) grid_turn(a, p, first + i, c[i], s[i]);
        }
    }
    close_wait();
    const int total = a.heads[0] + a.heads[1];
    const int h0 = blockIdx.y * a.heads_per_thread, h1 = min(h0 + a.heads_per_thread, total);
    auto place = [&](int h, const T*& in, O*& out) {
        const int w = h >= a.heads[0] ? 1 : 0;
        const int hh = h - w * a.heads[0];
        in = static_cast<const T*>(a.in[w]) + b * a.in_stride[w][0] + hh * a.in_stride[w][1] + t * a.in_stride[w][2];
        out = static_cast<O*>(a.out[w]) + b * a.out_stride[w][0] + hh * a.out_stride[w][1] + t * a.out_stride[w][2];
    };
    using V = typename Word<W * sizeof(T)>::type;
    using VO = typename Word<W * sizeof(O)>::type;
    for (int h = h0; h < h1; h++) {
        const T* in;
        O* out;
        place(h, in, out);
        Few<T, W> x, y;
        Few<O, W> xo, yo;
        x.u = *reinterpret_cast<const V*>(in + col0);
        if (!copy && !PAIRED) y.u = *reinterpret_cast<const V*>(in + col1);
        // same type: what is not turned keeps its bits, NaN payloads among them
        if constexpr (sizeof(T) == sizeof(O)) {
            xo.u = x.u;
        } else {
#pragma unroll
            for (int i = 0; i < W; i++) xo.e[i] = from_float<O>(to_float(x.e[i]));
        }
        if (!copy) {
#pragma unroll
            for (int i = 0; i < P; i++) {
                if (PAIRED && col0 + 2 * i >= a.rot) break;  // the turned columns may end inside the vector
                const float f = to_float(x.e[PAIRED ? 2 * i : i]), g = to_float(PAIRED ? x.e[2 * i + 1] : y.e[i]);
                xo.e[PAIRED ? 2 * i : i] = from_float<O>(f * c[i] - g * s[i]);
                (PAIRED ? xo.e[2 * i + 1] : yo.e[i]) = from_float<O>(f * s[i] + g * c[i]);
            }
            if (!PAIRED) *reinterpret_cast<VO*>(out + col1) = yo.u;
        }
        *reinterpret_cast<VO*>(out + col0) = xo.u;
    }
}

int check_grid(const llsa_rope_grid_params* p, bool has_pos) {
    if (!p) return LLSA_ERR_INVALID_ARG;
    if (p->batch < 0 || p->heads < 0 || p->kv_heads < 0 || p->n < 0) return LLSA_ERR_INVALID_ARG;
    if (p->dtype != LLSA_DTYPE_BF16 && p->dtype != LLSA_DTYPE_F32) return LLSA_ERR_DTYPE;
    if (p->out_other != 0 && p->out_other != 1) return LLSA_ERR_INVALID_ARG;
    if (p->layout != LLSA_ROPE_HALF && p->layout != LLSA_ROPE_INTERLEAVED) return LLSA_ERR_INVALID_ARG;
    if (p->span < LLSA_ROPE_SPAN_AXIS || p->span > LLSA_ROPE_SPAN_DEALT) return LLSA_ERR_INVALID_ARG;
    if (p->axes < 1 || p->axes > kAxes) return LLSA_ERR_INVALID_ARG;
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
    int left = p->d;
    for (int i = 0; i < p->axes; i++) {
        if (!(p->step[i] >= 0.0) || isinf(p->step[i])) return LLSA_ERR_INVALID_ARG;
        if (p->columns[i] < 2 || p->columns[i] % 2 != 0 || p->columns[i] > left) return LLSA_ERR_SHAPE;
        left -= p->columns[i];
    }
    if (has_pos) return LLSA_OK;  // the fields below say where positions come from when none are given
    long long tokens = 1;
    for (int i = 0; i < p->axes; i++) {
        if (p->extent[i] < 0) return LLSA_ERR_INVALID_ARG;
        if ((long long)p->offset[i] + p->extent[i] - 1 > 2147483647LL) return LLSA_ERR_INVALID_ARG;
        tokens = p->extent[i] == 0 ? 0 : std::min(tokens * p->extent[i], 1LL << 32);  // enough to be no int
    }
    if (tokens != p->n) return LLSA_ERR_SHAPE;
    if (p->token_order == LLSA_ORDER_TILE && p->n > 0) {
        if (p->axes < 2) return LLSA_ERR_INVALID_ARG;
        const int side_of = p->extent[p->axes - 1];
        long long side = 1;
        while (side < side_of) side *= 4;
        if (side != side_of || p->extent[p->axes - 2] != side_of) return LLSA_ERR_SHAPE;
    }
    return LLSA_OK;
}

// Axis and frequency of every pair, and the amplitude.
int derive_grid(const llsa_rope_grid_params* p, GridArgs* a) {
    int pairs[kAxes], total = 0;
    for (int i = 0; i < p->axes; i++) {
        pairs[i] = p->columns[i] / 2;
        total += pairs[i];
    }
    a->rot = 2 * total;
    a->segments = p->span == LLSA_ROPE_SPAN_AXIS ? p->axes : 1;
    a->first[0] = 0;
    for (int i = 0; i < a->segments; i++) a->first[i + 1] = a->segments == 1 ? total : a->first[i] + pairs[i];
    int taken[kAxes] = {}, axis = 0;
    for (int k = 0; k < total; k++) {
        if (p->span == LLSA_ROPE_SPAN_DEALT) {
            while (taken[axis] == pairs[axis]) axis = (axis + 1) % p->axes;
        } else {
            while (taken[axis] == pairs[axis]) axis++;
        }
        const bool own = p->span == LLSA_ROPE_SPAN_AXIS;  // a ladder of frequencies per axis
        const int place = own ? taken[axis] : k, seg = own ? p->columns[axis] : a->rot;
        double base = p->base;
        if (p->scaling == LLSA_ROPE_SCALE_BASE) {
            if (seg <= 2) return LLSA_ERR_SHAPE;
            base *= pow(p->factor, (double)seg / (seg - 2));
            if (!isfinite(base) || !(base > 0)) return LLSA_ERR_INVALID_ARG;
        }
        double w = rope_scaled(*p, pow(base, -2.0 * place / seg));
        if (p->step[axis] != 0.0) w *= p->step[axis];
        if (!rope_turns(w, &a->freq[k])) return LLSA_ERR_INVALID_ARG;
        a->axis[k] = (uint8_t)axis;
        taken[axis]++;
        if (p->span == LLSA_ROPE_SPAN_DEALT) axis = (axis + 1) % p->axes;
    }
    double amplitude = p->scaling == LLSA_ROPE_SCALE_WAVELENGTH && p->factor > 1.0 ? 0.1 * log(p->factor) + 1.0 : 1.0;
    if (p->amplitude != 0.0) amplitude = p->amplitude;
    a->amplitude = (float)amplitude;
    return isfinite(a->amplitude) ? LLSA_OK : LLSA_ERR_INVALID_ARG;
}

template <typename T, typename O>
int launch_grid(const llsa_rope_grid_params* p, GridArgs& a, cudaStream_t st) {
    constexpr int V = 16 / sizeof(T);
    int w = V;
    if (p->layout == LLSA_ROPE_HALF) {
        int all = 0;  // the bits that any segment's length has
        for (int i = 0; i < a.segments; i++) all |= a.first[i + 1] - a.first[i];
        while (w > 1 && all % w != 0) w /= 2;
        if (w == V / 4) w = 1;  // rare: one pair per thread does for those too
    }
    a.units = p->layout == LLSA_ROPE_INTERLEAVED ? a.d / V : a.rot / 2 / w + (a.d - a.rot) / w;
    const int total = a.heads[0] + a.heads[1];
    const long long threads = a.rows * a.units;
    // As many heads per thread (the sines are computed once for them) as leave about one wave of
    // resident threads: 2,048 per SM with 32 registers, which the interleaved layout has; the
    // half layout's whole vectors take 40 (fp32), 51 (bf16) and 56 (bf16 into fp32), so one and a
    // half to two waves there. 65,535 blocks is the most that the grid's second dimension takes.
    const long long want = (long long)sm_count() * 2048;
    const long long least = (total + 65534) / 65535;
    a.heads_per_thread = (int)std::min<long long>(total, std::max(least, threads * total / want));
    const long long gx = (threads + kThreads - 1) / kThreads;
    const int gy = (total + a.heads_per_thread - 1) / a.heads_per_thread;
    a.heads_per_thread = (total + gy - 1) / gy;  // the same share for all
    if (gx > 2147483647LL) return LLSA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    const bool close = close_first(st);
    if (p->layout == LLSA_ROPE_INTERLEAVED)
        LLSA_LAUNCH("rope_grid", st, launch_close(close, rope_grid_kernel<T, O, V, true>, grid, kThreads, 0, st, a));
    else if (w == V)
        LLSA_LAUNCH("rope_grid", st, launch_close(close, rope_grid_kernel<T, O, V, false>, grid, kThreads, 0, st, a));
    else if (w == V / 2)
        LLSA_LAUNCH("rope_grid", st, launch_close(close, rope_grid_kernel<T, O, V / 2, false>, grid, kThreads, 0, st, a));
    else
        LLSA_LAUNCH("rope_grid", st, launch_close(close, rope_grid_kernel<T, O, 1, false>, grid, kThreads, 0, st, a));
    return LLSA_OK;
}

}  // namespace
}  // namespace llsa

using namespace llsa;

extern "C" int llsa_rope_grid(const llsa_rope_grid_params* p, const llsa_rope_strides* strides, const void* q,
                              const void* k, const int32_t* pos, void* q_out, void* k_out, int inverse, void* stream) {
    CallRange range("llsa_rope_grid");
    LLSA_TRY(check_grid(p, pos != nullptr));
    if (inverse != 0 && inverse != 1) return LLSA_ERR_INVALID_ARG;
    GridArgs a;
    memset(&a, 0, sizeof(a));
    LLSA_TRY(derive_grid(p, &a));
    const long long total = (long long)p->heads + p->kv_heads;
    if (p->batch == 0 || p->n == 0 || total == 0) return LLSA_OK;
    if (total > (1 << 30) || (double)p->batch * p->n * total * p->d > (double)(1LL << 40)) return LLSA_ERR_UNSUPPORTED;
    if (p->heads > 0) LLSA_TRY(check_ptrs({q, q_out}));
    if (p->kv_heads > 0) LLSA_TRY(check_ptrs({k, k_out}));
    if (pos && (reinterpret_cast<uintptr_t>(pos) & 3u)) return LLSA_ERR_ALIGN;
    LLSA_TRY(rope_strides(strides ? strides->q : nullptr, *p, p->heads, false, a.in_stride[0]));
    LLSA_TRY(rope_strides(strides ? strides->k : nullptr, *p, p->kv_heads, false, a.in_stride[1]));
    llsa_rope_grid_params outs = *p;
    if (p->out_other) outs.dtype = p->dtype == LLSA_DTYPE_BF16 ? LLSA_DTYPE_F32 : LLSA_DTYPE_BF16;
    LLSA_TRY(rope_strides(strides ? strides->q_out : nullptr, outs, p->heads, true, a.out_stride[0]));
    LLSA_TRY(rope_strides(strides ? strides->k_out : nullptr, outs, p->kv_heads, true, a.out_stride[1]));
    // a tensor may be its own output only if every element goes back to its own place
    if (p->out_other && ((p->heads > 0 && q == q_out) || (p->kv_heads > 0 && k == k_out))) return LLSA_ERR_INVALID_ARG;
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
    a.d = p->d;
    a.axes = p->axes;
    a.tile = p->token_order == LLSA_ORDER_TILE;
    a.batched = p->pos_batched;
    for (int i = 0; i < p->axes; i++) {
        a.extent[i] = p->extent[i];
        a.offset[i] = p->offset[i];
    }
    a.sign = inverse ? -1.0f : 1.0f;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (p->dtype == LLSA_DTYPE_BF16)
        return p->out_other ? launch_grid<__nv_bfloat16, float>(p, a, st) : launch_grid<__nv_bfloat16, __nv_bfloat16>(p, a, st);
    return p->out_other ? launch_grid<float, __nv_bfloat16>(p, a, st) : launch_grid<float, float>(p, a, st);
}

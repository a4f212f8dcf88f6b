// dense_few.cu -- dense attention, forward and backward, for a handful of query
// rows per key head (single tokens, their shared-key heads, pooling queries): the
// keys and values are read once, on the CUDA cores.
//
// Mathematics, forward: one pass over the keys with the running maximum and sum of the
// softmax, as everywhere; the keys of a slice are split over many blocks, and
// inside a block over warps and groups of lanes, each with its own maximum, sum
// and output, joined at the end in a fixed order.
//
// Bound by HBM: 4 d flops per key and row against 4 d bytes per key (bf16). A group
// of 8 to 32 lanes holds one key, 8 columns per lane, so that a warp reads whole
// rows; several keys per group are in flight before the first is used. The
// tensor-core kernel would leave 120 of its 128 rows empty and wait for a softmax
// of full tiles (12 heads x 65,536 keys, one query: 60 us there, 37 here, 30 at
// HBM's rate; backward 167 and 70, at HBM's rate 59).
#include <algorithm>

#include "dense.h"

namespace llsa {
namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

// Eight values as they lie in memory, and as fp32.
template <typename T>
struct Raw {
    uint4 w[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); i++) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)(sizeof(T) / 2); i++) w[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float* f) const {
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float2 t = __bfloat1622float2(h[i]);
                f[2 * i] = t.x;
                f[2 * i + 1] = t.y;
            }
        } else {
            const float* h = reinterpret_cast<const float*>(w);
#pragma unroll
            for (int i = 0; i < 8; i++) f[i] = h[i];
        }
    }
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}

// What a split writes: o unnormalised [split][slice][R][d], then (maximum, sum)
// pairs [split][slice][R].
template <typename T, int RR, int LANES>
__global__ void __launch_bounds__(kThreads) dense_fwd_few_kernel(DenseArgs a) {
    constexpr int GROUPS = 32 / LANES;
    // keys per group of lanes, in use and in flight (one row: 8 x 4 key heads x 16,383 keys 45.3 us, with half as many 47.2)
    constexpr int U = (sizeof(T) == 2 ? 4 : 2) * (RR == 1 ? 2 : 1);
    __shared__ float sO[kWarps][RR][LANES * 8];
    __shared__ float2 sML[kWarps][RR];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / LANES, col = (lane % LANES) * 8;
    const int slice = blockIdx.x / a.splits, part = blockIdx.x - slice * a.splits;
    const DenseSpan sp = dense_span(a, slice);
    const bool on = col < a.d;
    const float sl2 = a.scale * kDenseLog2e;
    float q[RR][8], acc[RR][8], m[RR], l[RR];
    int kend[RR], most = 0;
#pragma unroll
    for (int r = 0; r < RR; r++) {
        kend[r] = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
        most = max(most, kend[r]);
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) q[r][i] = acc[r][i] = 0.f;
        if (on && kend[r] > 0) {
            load8(static_cast<const T*>(a.q) + ((long long)slice * a.R + r) * a.d + col, q[r]);
#pragma unroll
            for (int i = 0; i < 8; i++) q[r][i] *= sl2;
        }
    }
    const int first = part * a.chunk;
    const int stop = min(most, a.splits > 1 ? first + a.chunk : a.nk);
    const T* k = static_cast<const T*>(a.k) + (long long)slice * a.nk * a.d + col;
    const T* v = static_cast<const T*>(a.v) + (long long)slice * a.nk * a.d + col;
    constexpr int STEP = kWarps * GROUPS;  // keys between a group's keys
    Raw<T> kr[U], vr[U];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int j = j0 + u * STEP;
            if (on && j < stop) {
                kr[u].load(k + (long long)j * a.d);
                vr[u].load(v + (long long)j * a.d);
            } else {
                kr[u].zero();
                vr[u].zero();
            }
        }
    };
    const int mine = first + warp * GROUPS + grp;
    fetch(mine);
    for (int j0 = mine; __any_sync(0xffffffffu, j0 < stop); j0 += U * STEP) {
        Raw<T> kc[U], vc[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            kc[u] = kr[u];
            vc[u] = vr[u];
        }
        fetch(j0 + U * STEP);
        float s[U][RR];
#pragma unroll
        for (int u = 0; u < U; u++) {
            float f[8];
            kc[u].get(f);
#pragma unroll
            for (int r = 0; r < RR; r++) {
                float t = q[r][0] * f[0];
#pragma unroll
                for (int i = 1; i < 8; i++) t = fmaf(q[r][i], f[i], t);
#pragma unroll
                for (int o = 1; o < LANES; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                s[u][r] = j0 + u * STEP < min(kend[r], stop) ? t : -INFINITY;
            }
        }
#pragma unroll
        for (int r = 0; r < RR; r++) {
            float top = m[r];
#pragma unroll
            for (int u = 0; u < U; u++) top = fmaxf(top, s[u][r]);
            const float shift = top == -INFINITY ? 0.f : top;
            const float f = ex2(m[r] - shift);
            m[r] = top;
            l[r] *= f;
#pragma unroll
            for (int i = 0; i < 8; i++) acc[r][i] *= f;
#pragma unroll
            for (int u = 0; u < U; u++) {
                s[u][r] = ex2(s[u][r] - shift);
                l[r] += s[u][r];
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            float f[8];
            vc[u].get(f);
#pragma unroll
            for (int r = 0; r < RR; r++)
#pragma unroll
                for (int i = 0; i < 8; i++) acc[r][i] = fmaf(s[u][r], f[i], acc[r][i]);
        }
    }
    // the groups of a warp, then the warps, in a fixed order
#pragma unroll
    for (int r = 0; r < RR; r++) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[r], o), l2 = __shfl_xor_sync(0xffffffffu, l[r], o);
            const float top = fmaxf(m[r], m2), shift = top == -INFINITY ? 0.f : top;
            const float f1 = ex2(m[r] - shift), f2 = ex2(m2 - shift);
            m[r] = top;
            l[r] = l[r] * f1 + l2 * f2;
#pragma unroll
            for (int i = 0; i < 8; i++) acc[r][i] = acc[r][i] * f1 + __shfl_xor_sync(0xffffffffu, acc[r][i], o) * f2;
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < 8; i++) sO[warp][r][col + i] = acc[r][i];
            if (lane == 0) sML[warp][r] = make_float2(m[r], l[r]);
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < RR * a.d; x += kThreads) {
        const int r = x / a.d, c = x - r * a.d;
        if (r >= a.R) break;
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kWarps; i++) top = fmaxf(top, sML[i][r].x);
        const float shift = top == -INFINITY ? 0.f : top;
        float sum = 0.f, out = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; i++) {
            const float f = ex2(sML[i][r].x - shift);
            sum = fmaf(sML[i][r].y, f, sum);
            out = fmaf(sO[i][r][c], f, out);
        }
        const long long row = (long long)slice * a.R + r;
        if (a.splits > 1) {
            const long long prow = (long long)part * a.slices * a.R + row;
            a.part[prow * a.d + c] = out;
            if (c == 0)
                reinterpret_cast<float2*>(a.part + (long long)a.splits * a.slices * a.R * a.d)[prow] = make_float2(top, sum);
        } else {
            out = sum == 0.f ? 0.f : out / sum;
            if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(a.o_out)[row * a.d + c] = __float2bfloat16_rn(out);
            else static_cast<float*>(a.o_out)[row * a.d + c] = out;
            if (c == 0) a.lse_out[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
        }
    }
}

// Backward: with D = dout . o and l2 = lse log2(e) of every row worked out by each
// block, P = 2^(scale log2(e) q.k - l2) and dS = P (dout.v - D) of a key are
// numbers that its group of lanes shares, dk = scale sum dS q and dv = sum P dout
// leave at once, and dq gathers scale dS k in registers, joined as the forward's
// output. One pass reads k and v and writes dk and dv: 8 d bytes per key (bf16)
// against 10 d flops per row.
template <typename T, int RR, int LANES>
__global__ void __launch_bounds__(kThreads) dense_bwd_few_kernel(const __grid_constant__ DenseArgs a) {
    constexpr int GROUPS = 32 / LANES;
    constexpr int U = (sizeof(T) == 2 ? 4 : 2) / (RR > 2 ? 2 : 1);  // keys per group of lanes, in use and in flight
    __shared__ float sQ[kWarps][RR][LANES * 8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / LANES, col = (lane % LANES) * 8;
    const int slice = blockIdx.x / a.splits, part = blockIdx.x - slice * a.splits;
    const DenseSpan sp = dense_span(a, slice);
    const bool on = col < a.d;
    const float sl2 = a.scale * kDenseLog2e;
    float q[RR][8], g[RR][8], acc[RR][8], nl2[RR], D[RR];
    int kend[RR], most = 0;
#pragma unroll
    for (int r = 0; r < RR; r++) {
        kend[r] = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
        most = max(most, kend[r]);
        nl2[r] = -INFINITY;
        D[r] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) q[r][i] = g[r][i] = acc[r][i] = 0.f;
        if (kend[r] > 0) {
            const long long row = (long long)slice * a.R + r;
            nl2[r] = -__ldg(a.lse + row) * kDenseLog2e;
            if (on) {
                float o[8];
                load8(static_cast<const T*>(a.q) + row * a.d + col, q[r]);
                load8(static_cast<const T*>(a.dout) + row * a.d + col, g[r]);
                load8(static_cast<const T*>(a.o) + row * a.d + col, o);
#pragma unroll
                for (int i = 0; i < 8; i++) D[r] = fmaf(g[r][i], o[i], D[r]);
            }
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) D[r] += __shfl_xor_sync(0xffffffffu, D[r], o);
    }
    const int first = part * a.chunk;
    const int last = a.splits > 1 ? min(a.nk, first + a.chunk) : a.nk, stop = min(most, last);
    const long long base = (long long)slice * a.nk * a.d + col;
    const T *k = static_cast<const T*>(a.k) + base, *v = static_cast<const T*>(a.v) + base;
    T *dk = static_cast<T*>(a.dk) + base, *dv = static_cast<T*>(a.dv) + base;
    constexpr int STEP = kWarps * GROUPS;  // keys between a group's keys
    Raw<T> kr[U], vr[U];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int j = j0 + u * STEP;
            if (on && j < stop) {
                kr[u].load(k + (long long)j * a.d);
                vr[u].load(v + (long long)j * a.d);
            } else {
                kr[u].zero();
                vr[u].zero();
            }
        }
    };
    const int mine = first + warp * GROUPS + grp;
    fetch(mine);
    for (int j0 = mine; __any_sync(0xffffffffu, j0 < last); j0 += U * STEP) {
        Raw<T> kc[U], vc[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            kc[u] = kr[u];
            vc[u] = vr[u];
        }
        fetch(j0 + U * STEP);
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int j = j0 + u * STEP;
            float kf[8], vf[8], ok[8], ov[8];
            kc[u].get(kf);
            vc[u].get(vf);
#pragma unroll
            for (int i = 0; i < 8; i++) ok[i] = ov[i] = 0.f;
#pragma unroll
            for (int r = 0; r < RR; r++) {
                float s = q[r][0] * kf[0], p = g[r][0] * vf[0];
#pragma unroll
                for (int i = 1; i < 8; i++) {
                    s = fmaf(q[r][i], kf[i], s);
                    p = fmaf(g[r][i], vf[i], p);
                }
#pragma unroll
                for (int o = 1; o < LANES; o <<= 1) {
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                    p += __shfl_xor_sync(0xffffffffu, p, o);
                }
                const float w = j < min(kend[r], stop) ? ex2(fmaf(s, sl2, nl2[r])) : 0.f;
                const float ds = w * (p - D[r]) * a.scale;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    ok[i] = fmaf(ds, q[r][i], ok[i]);
                    ov[i] = fmaf(w, g[r][i], ov[i]);
                    acc[r][i] = fmaf(ds, kf[i], acc[r][i]);
                }
            }
            if (on && j < last) {  // keys that no row sees: zeros
                store4(dk + (long long)j * a.d, ok);
                store4(dk + (long long)j * a.d + 4, ok + 4);
                store4(dv + (long long)j * a.d, ov);
                store4(dv + (long long)j * a.d + 4, ov + 4);
            }
        }
    }
    // the groups of a warp, then the warps, in a fixed order
#pragma unroll
    for (int r = 0; r < RR; r++) {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1)
#pragma unroll
            for (int i = 0; i < 8; i++) acc[r][i] += __shfl_xor_sync(0xffffffffu, acc[r][i], o);
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < 8; i++) sQ[warp][r][col + i] = acc[r][i];
        }
    }
    __syncthreads();
    for (int x = threadIdx.x; x < RR * a.d; x += kThreads) {
        const int r = x / a.d, c = x - r * a.d;
        if (r >= a.R) break;
        float out = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; i++) out += sQ[i][r][c];
        const long long at = ((long long)slice * a.R + r) * a.d + c;
        if (a.splits > 1) a.part[(long long)part * a.slices * a.R * a.d + at] = out;
        else if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(a.dq)[at] = __float2bfloat16_rn(out);
        else static_cast<float*>(a.dq)[at] = out;
    }
}

template <typename T, int RR>
int launch_bwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    const long long blocks = (long long)s.slices * a.splits;
    if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
    if (s.d <= 64) LLSA_LAUNCH("dense_bwd_few", st, dense_bwd_few_kernel<T, RR, 8><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    else if (s.d <= 128) LLSA_LAUNCH("dense_bwd_few", st, dense_bwd_few_kernel<T, RR, 16><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    else LLSA_LAUNCH("dense_bwd_few", st, dense_bwd_few_kernel<T, RR, 32><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    return LLSA_OK;
}

template <typename T>
int launch_bwd_rows(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    return s.R <= 1 ? launch_bwd<T, 1>(s, a, st) : s.R <= 2 ? launch_bwd<T, 2>(s, a, st) : launch_bwd<T, 4>(s, a, st);
}

template <typename T, int RR>
int launch(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    const long long blocks = (long long)s.slices * a.splits;
    if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
    if (s.d <= 64) LLSA_LAUNCH("dense_fwd_few", st, dense_fwd_few_kernel<T, RR, 8><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    else if (s.d <= 128) LLSA_LAUNCH("dense_fwd_few", st, dense_fwd_few_kernel<T, RR, 16><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    else LLSA_LAUNCH("dense_fwd_few", st, dense_fwd_few_kernel<T, RR, 32><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    return LLSA_OK;
}

template <typename T>
int launch_rows(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    if (s.R <= 1) return launch<T, 1>(s, a, st);
    if constexpr (sizeof(T) == 4)
        if (s.R > 2) return launch<T, 4>(s, a, st);
    return launch<T, 2>(s, a, st);
}

}  // namespace

// bf16: two rows. 12 heads x 65,536 keys 49 us against 61 on the tensor cores; at four
// rows their kernels are the faster ones, 61 us against 72, and 57 against 91 at 8 x 4 key
// heads x 16,383 keys of 128 columns (256 columns: two rows 100 against 131, four 203).
// fp32: four rows, 68 us against 205 at 64 columns there and 121 against 403 at 128.
bool dense_few_supported(const DenseShape& s) { return s.R > 0 && s.R <= (s.dtype == LLSA_DTYPE_BF16 ? 2 : 4); }

// Parts for two blocks per SM; a part has at least 256 keys, two rounds of its warps' loads.
// Three and four rows, and two in the backward pass, take 155 to 197 registers a thread, so
// that an SM holds one block and the parts run in two rounds: as fast as half as many parts
// or faster (8 x 4 key heads x 16,383 keys of 128 columns, fp32: four rows backward 289 us
// and 315, two rows forward 99 and 129).
DenseSplit dense_few_split(const DenseShape& s) {
    DenseSplit p;
    long long n = 2 * kDenseSms / std::max(1, s.slices);
    n = std::max<long long>(1, std::min<long long>(n, s.nk / 256));
    p.chunk = (int)((s.nk + n - 1) / n);
    p.splits = s.nk > 0 ? (s.nk + p.chunk - 1) / p.chunk : 1;
    return p;
}

// Four rows in either type: 8 x 4 key heads x 16,383 keys at 128 columns 139 us in bf16
// against 255 on the tensor cores (one row 90), fp32 289 against 1,170; bf16 at 256
// columns 272 against 762.
bool dense_few_bwd_supported(const DenseShape& s) { return s.R > 0 && s.R <= 4 && s.nk > 0; }

int launch_dense_few_bwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    return s.dtype == LLSA_DTYPE_BF16 ? launch_bwd_rows<__nv_bfloat16>(s, a, st) : launch_bwd_rows<float>(s, a, st);
}

int launch_dense_few(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    return s.dtype == LLSA_DTYPE_BF16 ? launch_rows<__nv_bfloat16>(s, a, st) : launch_rows<float>(s, a, st);
}

}  // namespace llsa

// diff_few.cu -- differential attention forward for one or two query rows per value head
// (single tokens, pooling queries): both maps' keys and the values are read once, on the
// CUDA cores.
//
// Mathematics: one pass over the keys with a running maximum and sum for each map; a key's
// two weights meet its value while that is in registers. The keys of a slice are split
// over blocks, and inside a block over warps and groups of lanes, each with its own
// maxima, sums and outputs, joined at the end in a fixed order, and the maps' difference
// is formed in fp32 there.
//
// Bound by HBM: 12 d flops per key and row against 8 d bytes per key (bf16). A group of 8 or
// 16 lanes holds one key, 8 columns of each map's key and 16 of the value per lane, and
// the next keys are in flight while these are used.
#include <algorithm>

#include "diff.h"

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
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; i++) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
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

template <typename T, int RR, int LANES>
__global__ void __launch_bounds__(kThreads) diff_few_kernel(const __grid_constant__ DiffArgs f) {
    const DenseArgs& a = f.d;
    constexpr int GROUPS = 32 / LANES;
    constexpr int U = (sizeof(T) == 2 ? 8 : 4) / RR;  // keys per group of lanes in flight
    constexpr int VC = LANES * 8;                     // columns of half a value
    extern __shared__ float sm[];
    float* sO = sm;                                                           // [kWarps][RR][2][2 VC]
    float2* sML = reinterpret_cast<float2*>(sm + kWarps * RR * 2 * 2 * VC);  // [kWarps][RR][2]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int grp = lane / LANES, col = (lane % LANES) * 8;
    const int slice = blockIdx.x / a.splits, part = blockIdx.x - slice * a.splits;
    const DenseSpan sp = dense_span(a, slice);
    const int dv = 2 * a.d;
    const bool on = col < a.d, on1 = col < dv, on2 = VC + col < dv;
    const float sl2 = a.scale * kDenseLog2e;
    float q[RR][2][8], acc[RR][2][16], m[RR][2], l[RR][2];
    int kend[RR], most = 0;
#pragma unroll
    for (int r = 0; r < RR; r++) {
        kend[r] = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
        most = max(most, kend[r]);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            m[r][i] = -INFINITY;
            l[r][i] = 0.f;
#pragma unroll
            for (int c = 0; c < 8; c++) q[r][i][c] = acc[r][i][c] = acc[r][i][c + 8] = 0.f;
            if (on && kend[r] > 0) {
                load8(static_cast<const T*>(a.q) + diff_row(f, slice, i, r) * a.d + col, q[r][i]);
#pragma unroll
                for (int c = 0; c < 8; c++) q[r][i][c] *= sl2;
            }
        }
    }
    const int first = part * a.chunk;
    const int stop = min(most, a.splits > 1 ? first + a.chunk : a.nk);
    const int b = slice / a.kv_heads;
    const T* k0 = static_cast<const T*>(a.k) + ((long long)slice + (long long)b * a.kv_heads) * a.nk * a.d + col;
    const T* k1 = k0 + (long long)a.kv_heads * a.nk * a.d;
    const T* v = static_cast<const T*>(a.v) + (long long)slice * a.nk * dv + col;
    constexpr int STEP = kWarps * GROUPS;  // keys between a group's keys
    Raw<T> kr[U][2], vr[U][2];
    auto fetch = [&](int u, int j) {
        const bool here = j < stop;
        if (here && on) {
            kr[u][0].load(k0 + (long long)j * a.d);
            kr[u][1].load(k1 + (long long)j * a.d);
        } else {
            kr[u][0].zero();
            kr[u][1].zero();
        }
        if (here && on1) vr[u][0].load(v + (long long)j * dv);
        else vr[u][0].zero();
        if (here && on2) vr[u][1].load(v + (long long)j * dv + VC);
        else vr[u][1].zero();
    };
    const int mine = first + warp * GROUPS + grp;
#pragma unroll
    for (int u = 0; u < U; u++) fetch(u, mine + u * STEP);
    // Key after key, and each one's registers take its successor U keys further at once.
    for (int j0 = mine; __any_sync(0xffffffffu, j0 < stop); j0 += U * STEP) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int j = j0 + u * STEP;
            float s[RR][2], x[8];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                kr[u][i].get(x);
#pragma unroll
                for (int r = 0; r < RR; r++) {
                    float t = q[r][i][0] * x[0];
#pragma unroll
                    for (int c = 1; c < 8; c++) t = fmaf(q[r][i][c], x[c], t);
                    s[r][i] = t;
                }
            }
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1)
#pragma unroll
                for (int r = 0; r < RR; r++)
#pragma unroll
                    for (int i = 0; i < 2; i++) s[r][i] += __shfl_xor_sync(0xffffffffu, s[r][i], o);
            bool grow = false;
#pragma unroll
            for (int r = 0; r < RR; r++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    if (j >= min(kend[r], stop)) s[r][i] = -INFINITY;
                    grow |= s[r][i] > m[r][i];
                }
            if (__any_sync(0xffffffffu, grow)) {  // rare behind the first keys
#pragma unroll
                for (int r = 0; r < RR; r++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float top = fmaxf(m[r][i], s[r][i]), g = ex2(m[r][i] - (top == -INFINITY ? 0.f : top));
                        m[r][i] = top;
                        l[r][i] *= g;
#pragma unroll
                        for (int c = 0; c < 16; c++) acc[r][i][c] *= g;
                    }
            }
#pragma unroll
            for (int r = 0; r < RR; r++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    s[r][i] = ex2(s[r][i] - (m[r][i] == -INFINITY ? 0.f : m[r][i]));
                    l[r][i] += s[r][i];
                }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                vr[u][h].get(x);
#pragma unroll
                for (int r = 0; r < RR; r++)
#pragma unroll
                    for (int i = 0; i < 2; i++)
#pragma unroll
                        for (int c = 0; c < 8; c++) acc[r][i][8 * h + c] = fmaf(s[r][i], x[c], acc[r][i][8 * h + c]);
            }
            fetch(u, j + U * STEP);
        }
    }
    // the groups of a warp, then the warps, in a fixed order
#pragma unroll
    for (int r = 0; r < RR; r++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int o = LANES; o < 32; o <<= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, m[r][i], o), l2 = __shfl_xor_sync(0xffffffffu, l[r][i], o);
                const float top = fmaxf(m[r][i], m2), shift = top == -INFINITY ? 0.f : top;
                const float f1 = ex2(m[r][i] - shift), f2 = ex2(m2 - shift);
                m[r][i] = top;
                l[r][i] = l[r][i] * f1 + l2 * f2;
#pragma unroll
                for (int c = 0; c < 16; c++) acc[r][i][c] = acc[r][i][c] * f1 + __shfl_xor_sync(0xffffffffu, acc[r][i][c], o) * f2;
            }
            if (grp == 0) {
                float* to = sO + ((warp * RR + r) * 2 + i) * 2 * VC;
#pragma unroll
                for (int c = 0; c < 8; c++) {
                    to[col + c] = acc[r][i][c];
                    to[VC + col + c] = acc[r][i][8 + c];
                }
                if (lane == 0) sML[(warp * RR + r) * 2 + i] = make_float2(m[r][i], l[r][i]);
            }
        }
    __syncthreads();
    for (int x = threadIdx.x; x < RR * dv; x += kThreads) {
        const int r = x / dv, c = x - r * dv;
        if (r >= a.R) break;
        float out[2];
        const long long row = (long long)slice * a.R + r;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; w++) top = fmaxf(top, sML[(w * RR + r) * 2 + i].x);
            const float shift = top == -INFINITY ? 0.f : top;
            float sum = 0.f, o = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                const float2 ml = sML[(w * RR + r) * 2 + i];
                const float g = ex2(ml.x - shift);
                sum = fmaf(ml.y, g, sum);
                o = fmaf(sO[((w * RR + r) * 2 + i) * 2 * VC + c], g, o);
            }
            if (a.splits > 1) {
                const long long prow = diff_part(a, part, i, row);
                a.part[prow * dv + c] = o;
                if (c == 0) diff_part_ml(a)[prow] = make_float2(top, sum);
            } else {
                out[i] = sum == 0.f ? 0.f : o / sum;
                if (c == 0) a.lse_out[diff_row(f, slice, i, r)] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            }
        }
        if (a.splits > 1) continue;
        const float o = fmaf(-diff_lam(f, diff_head(f, slice, r)), out[1], out[0]);
        if constexpr (sizeof(T) == 2) {
            static_cast<__nv_bfloat16*>(a.o_out)[row * dv + c] = __float2bfloat16_rn(o);
            if (f.o2_out) static_cast<__nv_bfloat16*>(f.o2_out)[row * dv + c] = __float2bfloat16_rn(out[1]);
        } else {
            static_cast<float*>(a.o_out)[row * dv + c] = o;
            if (f.o2_out) static_cast<float*>(f.o2_out)[row * dv + c] = out[1];
        }
    }
}

template <typename T, int RR, int LANES>
int launch_lanes(const DiffArgs& a, cudaStream_t st) {
    const long long blocks = (long long)a.d.slices * a.d.splits;
    if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
    constexpr int smem = kWarps * RR * 2 * (2 * LANES * 8 * (int)sizeof(float) + (int)sizeof(float2));
    static_assert(smem <= 48 * 1024, "shared memory budget");
    LLSA_LAUNCH("diff_few", st, diff_few_kernel<T, RR, LANES><<<(unsigned)blocks, kThreads, smem, st>>>(a));
    return LLSA_OK;
}

template <typename T>
int launch(const DiffShape& s, const DiffArgs& a, cudaStream_t st) {
    if (s.R <= 1) return s.d <= 64 ? launch_lanes<T, 1, 8>(a, st) : launch_lanes<T, 1, 16>(a, st);
    return s.d <= 64 ? launch_lanes<T, 2, 8>(a, st) : launch_lanes<T, 2, 16>(a, st);
}

}  // namespace

bool diff_few_supported(const DiffShape& s) { return s.R > 0 && s.R <= 2 && s.nk > 0; }

// Parts for two blocks per SM; a part has at least 128 keys, a few rounds of its warps' loads.
DenseSplit diff_few_split(const DiffShape& s) {
    DenseSplit p;
    long long n = 2 * kDenseSms / std::max(1, s.slices);
    n = std::max<long long>(1, std::min<long long>(n, s.nk / 128));
    p.chunk = (int)((s.nk + n - 1) / n);
    p.splits = (s.nk + p.chunk - 1) / p.chunk;
    return p;
}

int launch_diff_few(const DiffShape& s, const DiffArgs& a, cudaStream_t st) {
    return s.dtype == LLSA_DTYPE_BF16 ? launch<__nv_bfloat16>(s, a, st) : launch<float>(s, a, st);
}

}  // namespace llsa

// diff_api.cu -- the C entries of differential attention: validation, workspace, choice
// of kernels, the gradient of lam, and the form that serves every call.
//
// That form. With V in halves V_1, V_2 of d columns, map i against half j is a dense
// attention of d columns: o's half j is A_1j - lam A_2j, and since a row's dS is linear in
// dout, dQ_i and dK_i are the sums over j, dV_j the sum over i, of the gradients of the
// four calls with dout_1j = dO_j and dout_2j = -lam dO_j. So the call runs as one dense
// call of four times as many slices on fp32 copies in the workspace, on the kernels for
// fp32, and is rounded once where the four are joined. Per pair of a query and a key it
// takes 16 d operations forward and 40 d backward where 12 d and 20 d are needed.
#include <math.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "diff.h"
#include "entry.h"

namespace llsa {
namespace {

constexpr int kThreads = 256;

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

template <typename T>
__device__ __forceinline__ void load4f(const T* p, float* f) {
    if constexpr (sizeof(T) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        f[0] = __uint_as_float(u.x << 16);
        f[1] = __uint_as_float(u.x & 0xffff0000u);
        f[2] = __uint_as_float(u.y << 16);
        f[3] = __uint_as_float(u.y & 0xffff0000u);
    } else {
        const float4 u = *reinterpret_cast<const float4*>(p);
        f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
    }
}

// The fp32 operands of the four calls: slice ((2 b + i) 2 + j) kv_heads + g.
struct FourArgs {
    DiffArgs a;
    float *q, *k, *v;           // [4 slices][R or nk][d]
    float *o, *dout, *lse;      // of the rows (backward)
    const float *dq, *dk, *dv;  // gradients of the four (backward)
    void *dq_out, *dk_out, *dv_out;
};

struct Place {
    int b, i, j, g;
};
__device__ __forceinline__ Place four_place(const FourArgs& f, long long slice4) {
    const int kv = f.a.d.kv_heads;
    const int g = (int)(slice4 % kv), rest = (int)(slice4 / kv);
    return {rest >> 2, (rest >> 1) & 1, rest & 1, g};
}

// blockIdx.y 0: what has query rows, 1: what has keys. Four values per thread. Q: the type of
// q, k and o2.
template <typename T, typename Q, bool BACKWARD>
__global__ void __launch_bounds__(kThreads) diff_expand_kernel(const __grid_constant__ FourArgs f) {
    const DenseArgs& a = f.a.d;
    const bool keys = blockIdx.y == 1;
    const int rows = keys ? a.nk : a.R, per = a.d / 4;
    const long long n = 4LL * a.slices * rows * per;
    for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < n; x += (long long)gridDim.x * kThreads) {
        const long long row4 = x / per;
        const int c = (int)(x - row4 * per) * 4;
        const long long slice4 = row4 / rows;
        const int r = (int)(row4 - slice4 * rows);
        const Place p = four_place(f, slice4);
        const long long one = (((long long)(2 * p.b + p.i) * a.kv_heads + p.g) * rows + r) * a.d + c;  // in q or k
        const long long slice = (long long)p.b * a.kv_heads + p.g;
        const long long two = (slice * rows + r) * 2 * a.d + p.j * a.d + c;                            // in v, o, dout
        const long long to = row4 * a.d + c;
        float y[4];
        if (keys) {
            load4f(static_cast<const Q*>(a.k) + one, y);
            store4(f.k + to, y);
            load4f(static_cast<const T*>(a.v) + two, y);
            store4(f.v + to, y);
            continue;
        }
        load4f(static_cast<const Q*>(a.q) + one, y);
        store4(f.q + to, y);
        if (!BACKWARD) continue;
        const float lam = diff_lam_row(f.a, (int)slice, r);
        float o[4], o2[4];
        load4f(static_cast<const T*>(a.dout) + two, y);
        load4f(static_cast<const Q*>(f.a.o2) + two, o2);
        if (p.i == 0) load4f(static_cast<const T*>(a.o) + two, o);
#pragma unroll
        for (int e = 0; e < 4; e++) {
            o2[e] = p.i == 0 ? fmaf(lam, o2[e], o[e]) : o2[e];
            y[e] = p.i == 0 ? y[e] : -lam * y[e];
        }
        store4(f.dout + to, y);
        store4(f.o + to, o2);
        if (c == 0) f.lse[row4] = a.lse[diff_row(f.a, (int)slice, p.i, r)];
    }
}

// The four calls' operands at once as the three bf16 planes that the fp32 kernels read:
// blockIdx.y q, k, v, dout. Eight values per thread, for both calls that share them at once
// (dense_qk_slice, dense_v_slice), and dout as it is and times -lam. Bound by HBM: 4 bytes in, 6 or 12 out.
struct PlanesArgs {
    DiffArgs a;
    __nv_bfloat16* out[4];  // plane p of tensor t at out[t] + p * n[t]
    long long n[4];
};

__device__ __forceinline__ void put_planes(__nv_bfloat16* out, long long n, const float* y) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; e++) f[e] = y[e];
#pragma unroll
    for (int p = 0; p < 3; p++) {
        uint32_t w[4];
#pragma unroll
        for (int c = 0; c < 8; c += 2) {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[c], f[c + 1]);
            w[c >> 1] = *reinterpret_cast<uint32_t*>(&h);
            f[c] -= __uint_as_float(w[c >> 1] << 16);
            f[c + 1] -= __uint_as_float(w[c >> 1] & 0xffff0000u);
        }
        *reinterpret_cast<uint4*>(out + p * n) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads) diff_planes_kernel(const __grid_constant__ PlanesArgs f) {
    const DenseArgs& a = f.a.d;
    const int t = blockIdx.y;
    const bool one = t < 2;  // a matrix of d columns per map, or of 2 d for both
    close_wait();
    close_ahead();  // behind the wait: the rows' numbers are worked out beside this, from what was there before
    const int rows = t == 0 || t == 3 ? a.R : a.nk, cols = one ? a.d : 2 * a.d, per = cols / 8;
    const long long total = (long long)a.slices * (one ? 2 : 1) * rows * per;
    for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < total; x += (long long)gridDim.x * kThreads) {
        const long long row = x / per;
        int c = (int)(x - row * per) * 8;
        const long long m = row / rows, outer = m / a.kv_heads;  // outer: 2 b + i, or b
        const int r = (int)(row - m * rows), g = (int)(m - outer * a.kv_heads);
        float y[8];
        if (one) diff_load8(static_cast<const Q*>(t == 0 ? a.q : a.k) + x * 8, y);
        else diff_load8(static_cast<const T*>(t == 2 ? a.v : a.dout) + x * 8, y);
        int j = 0;
        if (!one && c >= a.d) {
            j = 1;
            c -= a.d;
        }
        if (t < 3) {
            put_planes(f.out[t] + (one ? x * 8 : (((2 * outer + j) * a.kv_heads + g) * rows + r) * a.d + c), f.n[t], y);
            continue;
        }
        const long long at = (((4 * outer + j) * a.kv_heads + g) * rows + r) * a.d + c;
        put_planes(f.out[t] + at, f.n[t], y);
        const float lam = diff_lam_row(f.a, (int)m, r);
#pragma unroll
        for (int e = 0; e < 8; e++) y[e] *= -lam;
        put_planes(f.out[t] + at + 2LL * a.kv_heads * rows * a.d, f.n[t], y);
    }
}

// o, o2 and the log-sum-exp of both maps from the four calls' (in f.o and f.lse).
template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads) diff_combine_kernel(const __grid_constant__ FourArgs f) {
    const DenseArgs& a = f.a.d;
    close_wait();
    close_ahead();
    const int per = a.d / 2;  // vectors of 4 of a row of 2 d
    const long long n = (long long)a.slices * a.R * per, step = (long long)a.kv_heads * a.R;
    for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < n; x += (long long)gridDim.x * kThreads) {
        const long long row = x / per;
        const int col = (int)(x - row * per) * 4, j = col >= a.d ? 1 : 0;
        const int slice = (int)(row / a.R), r = (int)(row - (long long)slice * a.R);
        const int b = slice / a.kv_heads, g = slice - b * a.kv_heads;
        const long long first = ((4LL * b + j) * a.kv_heads + g) * a.R + r, second = first + 2 * step;
        const float lam = diff_lam_row(f.a, slice, r);
        float y[4], z[4];
        load4f(f.o + first * a.d + col - j * a.d, y);
        load4f(f.o + second * a.d + col - j * a.d, z);
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] = fmaf(-lam, z[e], y[e]);
        store4(static_cast<T*>(a.o_out) + row * 2 * a.d + col, y);
        if (f.a.o2_out) store4(static_cast<Q*>(f.a.o2_out) + row * 2 * a.d + col, z);
        if (col == 0) {
            a.lse_out[diff_row(f.a, slice, 0, r)] = f.lse[first];
            a.lse_out[diff_row(f.a, slice, 1, r)] = f.lse[second];
        }
    }
}

// dq, dk, dv (blockIdx.y) as sums of two of the four calls' gradients.
template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads) diff_collapse_kernel(const __grid_constant__ FourArgs f) {
    const DenseArgs& a = f.a.d;
    const int which = blockIdx.y, rows = which == 0 ? a.R : a.nk;
    close_wait();
    close_ahead();  // what does not wait behind this may read all but what this writes
    const int per = which == 2 ? a.d / 2 : a.d / 4;
    const long long n = (which == 2 ? 1LL : 2LL) * a.slices * rows * per, step = (long long)a.kv_heads * rows * a.d;
    const float* from = which == 0 ? f.dq : which == 1 ? f.dk : f.dv;
    for (long long x = (long long)blockIdx.x * kThreads + threadIdx.x; x < n; x += (long long)gridDim.x * kThreads) {
        const long long row = x / per;
        int c = (int)(x - row * per) * 4;
        const long long m = row / rows;  // matrix of the output
        const int r = (int)(row - m * rows);
        const long long to = row * 4 * per + c;
        const long long outer = m / a.kv_heads;  // 2 b + i, or b
        const int g = (int)(m - outer * a.kv_heads);
        long long matrix;
        int j = 0;
        if (which == 2) {
            j = c >= a.d ? 1 : 0;
            c -= j * a.d;
            matrix = (4 * outer + j) * a.kv_heads + g;
        } else {
            matrix = 2 * outer * a.kv_heads + g;
        }
        const long long at = (matrix * rows + r) * a.d + c, other = at + (which == 2 ? 2 * step : step);
        float y[4], z[4];
        load4f(from + at, y);
        load4f(from + other, z);
#pragma unroll
        for (int e = 0; e < 4; e++) y[e] += z[e];
        if (which == 2) store4(static_cast<T*>(f.dv_out) + to, y);
        else store4(static_cast<Q*>(which == 0 ? f.dq_out : f.dk_out) + to, y);
    }
}

// ------------------------------------------------------ join of a split --

// o, o2 and lse of every row from the parts of a split over the keys: a block per row, four
// warps per map, each with every fourth part. Rows are few where keys are split, so it is
// the latency of the parts that this costs (a warp per row, part after part: 35 us for 6 rows
// of 50 parts).
constexpr int kJoinSets = kThreads / 64;

template <typename T>
__global__ void __launch_bounds__(kThreads) diff_join_kernel(const __grid_constant__ DiffArgs f) {
    const DenseArgs& a = f.d;
    const long long row = blockIdx.x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = warp & 1, set = warp >> 1, dv = 2 * a.d;
    const int slice = (int)(row / a.R), r = (int)(row - (long long)slice * a.R);
    const float2* ml = diff_part_ml(a);
    close_wait();
    close_ahead();
    __shared__ float4 sums[2][kJoinSets][64];
    float m = -INFINITY, l = 0.f;
    for (int p = lane; p < a.splits; p += 32) m = fmaxf(m, ml[diff_part(a, p, i, row)].x);
    m = warp_max(m);
    const float shift = m == -INFINITY ? 0.f : m;
    for (int p = lane; p < a.splits; p += 32) {
        const float2 x = ml[diff_part(a, p, i, row)];
        l = fmaf(x.y, exp2f(x.x - shift), l);
    }
    l = warp_sum(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float acc[2][4] = {};
    for (int p0 = set; p0 < a.splits; p0 += 32 * kJoinSets) {
        const int mine = p0 + lane * kJoinSets;
        const float w = mine < a.splits ? exp2f(ml[diff_part(a, mine, i, row)].x - shift) * inv : 0.f;
        const int n = min(32, (a.splits - p0 + kJoinSets - 1) / kJoinSets);
#pragma unroll 8
        for (int x = 0; x < n; x++) {
            const float wx = __shfl_sync(0xffffffffu, w, x);
            const float* from = a.part + diff_part(a, p0 + x * kJoinSets, i, row) * dv + lane * 4;
#pragma unroll
            for (int k = 0; k < 2; k++)
                if (lane * 4 + 128 * k < dv) {
                    const float4 y = *reinterpret_cast<const float4*>(from + 128 * k);
                    acc[k][0] = fmaf(wx, y.x, acc[k][0]);
                    acc[k][1] = fmaf(wx, y.y, acc[k][1]);
                    acc[k][2] = fmaf(wx, y.z, acc[k][2]);
                    acc[k][3] = fmaf(wx, y.w, acc[k][3]);
                }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; k++) sums[i][set][lane + 32 * k] = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
    if (set == 0 && lane == 0) a.lse_out[diff_row(f, slice, i, r)] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
    __syncthreads();
    const int c = threadIdx.x * 4;
    if (c >= dv) return;
    const float lam = diff_lam_row(f, slice, r);
    float y[2][4];
#pragma unroll
    for (int i2 = 0; i2 < 2; i2++) {
        float4 t = sums[i2][0][threadIdx.x];
#pragma unroll
        for (int s = 1; s < kJoinSets; s++) {
            const float4 u = sums[i2][s][threadIdx.x];
            t.x += u.x;
            t.y += u.y;
            t.z += u.z;
            t.w += u.w;
        }
        y[i2][0] = t.x, y[i2][1] = t.y, y[i2][2] = t.z, y[i2][3] = t.w;
    }
    if (f.o2_out) store4(static_cast<T*>(f.o2_out) + row * dv + c, y[1]);
#pragma unroll
    for (int e = 0; e < 4; e++) y[0][e] = fmaf(-lam, y[1][e], y[0][e]);
    store4(static_cast<T*>(a.o_out) + row * dv + c, y[0]);
}

// ------------------------------------------------------ per-row numbers --

// The numbers that the backward pass needs of every query row: -lse log2(e) and -D of both
// maps, D_1 = dout . (o + lam o2) and D_2 = dout . o2, and lam. Rows that see no key (and
// the padding to Rp) get -infinity and 0, so that their probabilities are 2^(s - inf) = 0.
// A block per 128 rows, eight lanes per row, four rows each at a time. Bound by HBM: dout,
// o and o2 are read once. FOUR: the same for the four calls of the form above, and D_2 itself.
constexpr int kRowsEach = kDenseRowPad / (kThreads / 8);

// A vector's values as fp32.
__device__ __forceinline__ void unpack(const uint2& v, float* f, const __nv_bfloat16*) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const uint4& v, float* f, const __nv_bfloat16* t) {
    unpack(make_uint2(v.x, v.y), f, t);
    unpack(make_uint2(v.z, v.w), f + 4, t);
}
__device__ __forceinline__ void unpack(const uint4& v, float* f, const float*) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
}

template <typename T, typename Q, bool FOUR>
__global__ void __launch_bounds__(kThreads, 4) diff_rows_kernel(const __grid_constant__ DiffArgs f) {
    const DenseArgs& a = f.d;
    const unsigned per = (unsigned)a.Rp / kDenseRowPad, slice = blockIdx.x / per;
    const int r0 = (int)(blockIdx.x - slice * per) * kDenseRowPad + (threadIdx.x >> 3), part = threadIdx.x & 7;
    if (!FOUR) close_wait();
    const DenseSpan sp = dense_span(a, (int)slice);
    const int dv = 2 * a.d;
    float one[kRowsEach], two[kRowsEach];
    bool on[kRowsEach];
#pragma unroll
    for (int u = 0; u < kRowsEach; u++) {
        const int r = r0 + u * (kThreads / 8);
        on[u] = r < a.R && dense_kend(a, sp, r < a.nq ? r : r % a.nq) > 0;
        one[u] = two[u] = 0.f;
    }
    // vectors as they lie in memory: as fp32 four rows of three would not fit the registers
    using VT = std::conditional_t<sizeof(T) == sizeof(Q), uint4, uint2>;  // of dout and o
    constexpr int E = sizeof(VT) / sizeof(T);                             // elements; o2's vector is 16 bytes in any case
    for (int c = part * E; c < dv; c += 8 * E) {
        VT g[kRowsEach], x[kRowsEach];
        uint4 y[kRowsEach];
        const long long at = ((long long)slice * a.R + r0) * dv + c;
#pragma unroll
        for (int u = 0; u < kRowsEach; u++) {
            g[u] = x[u] = VT{};
            y[u] = uint4{};
            if (on[u]) {
                const long long to = at + (long long)u * (kThreads / 8) * dv;
                g[u] = *reinterpret_cast<const VT*>(static_cast<const T*>(a.dout) + to);
                x[u] = *reinterpret_cast<const VT*>(static_cast<const T*>(a.o) + to);
                y[u] = *reinterpret_cast<const uint4*>(static_cast<const Q*>(f.o2) + to);
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsEach; u++) {
            float p[E], q[E];
            unpack(g[u], p, static_cast<const T*>(nullptr));
            unpack(x[u], q, static_cast<const T*>(nullptr));
#pragma unroll
            for (int e = 0; e < E; e++) one[u] = fmaf(p[e], q[e], one[u]);
            unpack(y[u], q, static_cast<const Q*>(nullptr));
#pragma unroll
            for (int e = 0; e < E; e++) two[u] = fmaf(p[e], q[e], two[u]);
        }
    }
    const long long all = (long long)a.slices * a.Rp;
    close_ahead();
#pragma unroll
    for (int u = 0; u < kRowsEach; u++) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            one[u] += __shfl_xor_sync(0xffffffffu, one[u], o);
            two[u] += __shfl_xor_sync(0xffffffffu, two[u], o);
        }
        if (part != 0) continue;
        const int r = r0 + u * (kThreads / 8);
        const long long idx = (long long)slice * a.Rp + r;
        const float lam = on[u] ? diff_lam(f, diff_head(f, (int)slice, r)) : 0.f;
        const float D[2] = {on[u] ? -fmaf(lam, two[u], one[u]) : 0.f, on[u] ? -two[u] : 0.f};
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float lse = on[u] ? a.lse[diff_row(f, (int)slice, i, r)] : -INFINITY;
            const float l2 = lse == -INFINITY ? -INFINITY : -lse * kDenseLog2e;
            if constexpr (FOUR) {
                // both halves' calls of map i; only the sum of their D counts, weighed as their dout is
                const int b = (int)slice / a.kv_heads, gg = (int)slice - b * a.kv_heads;
                const long long first = ((4LL * b + 2 * i) * a.kv_heads + gg) * a.Rp + r, second = first + (long long)a.kv_heads * a.Rp;
                a.nl2[first] = a.nl2[second] = l2;
                a.nd[first] = i == 0 ? D[0] : -lam * D[1];
                a.nd[second] = 0.f;
            } else {
                a.nl2[i * all + idx] = l2;
                a.nl2[(2 + i) * all + idx] = D[i];
            }
        }
        if (!FOUR && idx == 0 && f.lam_ticket) *f.lam_ticket = 0;
        if constexpr (FOUR) f.d2[idx] = -D[1];
        else a.nl2[4 * all + idx] = lam;
    }
    close_wait();  // FOUR: reads nothing that the kernel before it writes
}

// ------------------------------------------------------ gradient of lam --

// dlam of a head: -sum of dout . o2 over its rows that see a key, in two steps of fixed
// order. Bound by HBM: dout and o2 are read once.
constexpr int kLamRows = 64;    // rows that a block takes at least
constexpr int kLamParts = 512;  // most blocks per head

int lam_parts(const DiffShape& s) {
    const long long rows = (long long)s.batch * s.nq;
    return (int)std::max<long long>(1, std::min<long long>({(rows + kLamRows - 1) / kLamRows, kLamParts, 8LL * kDenseSms / s.heads + 1}));
}

template <typename T, typename Q>
__global__ void __launch_bounds__(kThreads) diff_lam_kernel(const __grid_constant__ DiffArgs f, float* part, int parts) {
    const DenseArgs& a = f.d;
    const int h = blockIdx.x / parts, p = blockIdx.x - h * parts;
    const int G = f.heads / a.kv_heads, g = h / G, batch = a.slices / a.kv_heads;
    const long long rows = (long long)batch * a.nq, first = rows * p / parts, last = rows * (p + 1) / parts;
    const int lanes = a.d / 2;  // vectors of 4 in a row of 2 d: 4 to 64 a row
    float sum = 0.f;
    for (long long x = first * lanes + threadIdx.x; x < last * lanes; x += kThreads) {
        const long long row = x / lanes;
        const int c = (int)(x - row * lanes) * 4;
        const int b = (int)(row / a.nq), t = (int)(row - (long long)b * a.nq);
        const int slice = b * a.kv_heads + g;
        if (dense_kend(a, dense_span(a, slice), t) == 0) continue;
        const long long at = ((long long)slice * a.R + (long long)(h - g * G) * a.nq + t) * 2 * a.d + c;
        float y[4], z[4];
        load4f(static_cast<const T*>(a.dout) + at, y);
        load4f(static_cast<const Q*>(f.o2) + at, z);
#pragma unroll
        for (int e = 0; e < 4; e++) sum = fmaf(y[e], z[e], sum);
    }
    __shared__ float warps[kThreads / 32];
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kThreads / 32; i++) sum += warps[i];
        part[blockIdx.x] = sum;
    }
}

// dlam of a head from d2, `sets` sums of P_2 dP of every row: part p of `parts` of its
// rows to part[h parts + p], or with one part to dlam itself. fresh: the kernel before it writes d2.
constexpr int kLamThreads = 1024;

__global__ void __launch_bounds__(kLamThreads) diff_lam_rows_kernel(const __grid_constant__ DiffArgs f, float* part, int parts, int sets,
                                                                 int fresh, void* out) {
    const DenseArgs& a = f.d;
    const int h = blockIdx.x / parts, p = blockIdx.x - h * parts;
    const int G = f.heads / a.kv_heads, g = h / G, batch = a.slices / a.kv_heads;
    const long long rows = (long long)batch * a.nq, first = rows * p / parts, last = rows * (p + 1) / parts;
    const long long all = (long long)a.slices * a.Rp;
    if (fresh) close_wait();
    close_ahead();
    float sum = 0.f;
    for (long long row = first + threadIdx.x; row < last; row += kLamThreads) {
        const int b = (int)(row / a.nq), t = (int)(row - (long long)b * a.nq);
        const float* from = f.d2 + ((long long)b * a.kv_heads + g) * a.Rp + (long long)(h - g * G) * a.nq + t;
#pragma unroll 4
        for (int i = 0; i < sets; i++) sum += from[i * all];
    }
    __shared__ float warps[kLamThreads / 32];
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = sum;
    __syncthreads();
    close_wait();
    if (threadIdx.x != 0) return;
    for (int i = 1; i < kLamThreads / 32; i++) sum += warps[i];
    if (parts > 1) part[blockIdx.x] = sum;
    else if (f.lam_bf16) static_cast<__nv_bfloat16*>(out)[h] = __float2bfloat16_rn(-sum);
    else static_cast<float*>(out)[h] = -sum;
}

// A warp per head.
__global__ void __launch_bounds__(32) diff_lam_sum_kernel(const float* part, int parts, void* out, int bf16) {
    const int h = blockIdx.x;
    float sum = 0.f;
    for (int p = threadIdx.x; p < parts; p += 32) sum += part[(long long)h * parts + p];
    sum = warp_sum(sum);
    if (threadIdx.x != 0) return;
    if (bf16) static_cast<__nv_bfloat16*>(out)[h] = __float2bfloat16_rn(-sum);
    else static_cast<float*>(out)[h] = -sum;
}

template <typename T, typename Q>
int launch_lam(const DiffShape& s, const DiffArgs& a, void* dlam, float* part, cudaStream_t st) {
    const int parts = lam_parts(s);
    const unsigned blocks = (unsigned)s.heads * parts;
    LLSA_LAUNCH("diff_lam", st, diff_lam_kernel<T, Q><<<blocks, kThreads, 0, st>>>(a, part, parts));
    LLSA_LAUNCH("diff_lam_sum", st, diff_lam_sum_kernel<<<s.heads, 32, 0, st>>>(part, parts, dlam, s.lam_dtype == LLSA_DTYPE_BF16));
    return LLSA_OK;
}

// ------------------------------------------------------------ parameters --

int derive_diff(const llsa_diff_params* p, DiffShape* s) {
    if (!p) return LLSA_ERR_INVALID_ARG;
    if (p->lam_dtype != LLSA_DTYPE_BF16 && p->lam_dtype != LLSA_DTYPE_F32) return LLSA_ERR_DTYPE;
    if (p->qk_fp32 != 0 && p->qk_fp32 != 1) return LLSA_ERR_INVALID_ARG;
    if (p->heads < 0 || p->kv_heads < 0) return LLSA_ERR_INVALID_ARG;
    if (p->d > 128) return LLSA_ERR_SHAPE;
    const int kv = p->kv_heads ? p->kv_heads : p->heads;
    if (p->heads > kDenseMaxExtent / 4 || kv > kDenseMaxExtent / 4) return LLSA_ERR_UNSUPPORTED;
    memset(s, 0, sizeof(*s));
    llsa_dense_params four = {p->batch, 4 * p->heads, 4 * kv, p->nq, p->nk, p->d, p->dtype, p->causal, p->scale};
    LLSA_TRY(derive_dense(&four, &s->four));
    s->batch = p->batch;
    s->heads = p->heads;
    s->kv_heads = kv;
    s->G = s->four.G;
    s->nq = p->nq;
    s->nk = p->nk;
    s->d = p->d;
    s->dtype = p->dtype;
    s->wide = p->qk_fp32 && p->dtype == LLSA_DTYPE_BF16;
    s->lam_dtype = p->lam_dtype;
    s->causal = p->causal;
    s->scale = s->four.scale;
    s->slices = s->four.slices / 4;
    s->R = s->four.R;
    s->Rp = s->four.Rp;
    s->four.dtype = LLSA_DTYPE_F32;
    return LLSA_OK;
}

DiffArgs diff_args(const DiffShape& s) {
    DiffArgs a;
    memset(&a, 0, sizeof(a));
    a.d = dense_args(s.four);
    a.d.slices = s.slices;
    a.d.kv_heads = s.kv_heads;
    a.lam_bf16 = s.lam_dtype == LLSA_DTYPE_BF16;
    a.heads = s.heads;
    return a;
}

// -------------------------------------------------- the form for every call --

size_t four_rows(const DiffShape& s) { return up((size_t)4 * s.slices * s.R * s.d * sizeof(float)); }
size_t four_keys(const DiffShape& s) { return up((size_t)4 * s.slices * s.nk * s.d * sizeof(float)); }
size_t four_lse(const DiffShape& s) { return up((size_t)4 * s.slices * s.R * sizeof(float)); }

// Planes of q (two calls share them) and of dout, and of k or v.
size_t plane_q(const DiffShape& s) { return up((size_t)2 * s.slices * s.R * s.d * 6); }
size_t plane_dout(const DiffShape& s) { return up((size_t)4 * s.slices * s.R * s.d * 6); }
size_t plane_keys(const DiffShape& s) { return up((size_t)2 * s.slices * s.nk * s.d * 6); }
size_t padded_rows(const DiffShape& s) { return up((size_t)s.slices * s.Rp * sizeof(float)); }

// One block per head up to 4,096 of its rows: a second launch costs more than a long loop.
int row_parts(const DiffShape& s) { return (int)std::min<long long>(64, ((long long)s.batch * s.nq + 4095) / 4096); }
size_t row_parts_bytes(const DiffShape& s) { return up((size_t)s.heads * row_parts(s) * sizeof(float)); }

int launch_lam_rows(const DiffShape& s, const DiffArgs& a, int sets, int fresh, float* part, void* dlam, cudaStream_t st) {
    const int parts = row_parts(s);
    LLSA_LAUNCH("diff_lam_rows", st, launch_close(true, diff_lam_rows_kernel, dim3((unsigned)s.heads * parts), kLamThreads, 0, st, a, part, parts, sets,
                                                    fresh, dlam));
    if (parts > 1) LLSA_LAUNCH("diff_lam_sum", st, diff_lam_sum_kernel<<<s.heads, 32, 0, st>>>(part, parts, dlam, a.lam_bf16));
    return LLSA_OK;
}

size_t four_workspace(const DiffShape& s, bool backward) {
    if (!backward && dense_fwd_on_planes(s.four))
        return plane_q(s) + 2 * plane_keys(s) + four_rows(s) + four_lse(s) + up(dense_fwd_parts(s.four));
    if (backward && dense_bwd_on_planes(s.four))
        return plane_q(s) + plane_dout(s) + 2 * plane_keys(s) + four_rows(s) + 2 * four_keys(s) + 9 * padded_rows(s) + row_parts_bytes(s) +
               up(dense_bwd_parts(s.four));
    return backward ? 4 * four_rows(s) + 4 * four_keys(s) + four_lse(s) + up(dense_bwd_workspace(s.four))
                    : 2 * four_rows(s) + 2 * four_keys(s) + four_lse(s) + up(dense_fwd_workspace(s.four));
}

DenseArgs four_args(const DiffShape& s, const DiffArgs& a, const FourArgs& f, bool planes = false) {
    DenseArgs d = a.d;
    d.four = planes;
    d.slices = s.four.slices;
    d.kv_heads = s.four.kv_heads;
    d.q = f.q;
    d.k = f.k;
    d.v = f.v;
    return d;
}

unsigned blocks_for(long long n) { return (unsigned)std::min<long long>((n + kThreads - 1) / kThreads, 16LL * kDenseSms); }

// Planes of q, k, v and (backward) dout, one after the other from `at` on.
template <typename T, typename Q>
int launch_planes(const DiffShape& s, const DiffArgs& a, bool backward, char*& at, void** planes, cudaStream_t st) {
    PlanesArgs f;
    memset(&f, 0, sizeof(f));
    f.a = a;
    const long long nq = 2LL * s.slices * s.R * s.d, nk = 2LL * s.slices * s.nk * s.d;
    for (int t = 0; t < (backward ? 4 : 3); t++) {
        f.out[t] = reinterpret_cast<__nv_bfloat16*>(at);
        f.n[t] = t == 0 ? nq : t == 3 ? 2 * nq : nk;
        planes[t] = at;
        at += t == 0 ? plane_q(s) : t == 3 ? plane_dout(s) : plane_keys(s);
    }
    const dim3 grid((unsigned)std::min<long long>((std::max(nq, nk) / 8 + kThreads - 1) / kThreads, 8LL * kDenseSms), backward ? 4 : 3);
    LLSA_LAUNCH("diff_planes", st, launch_close(close_first(st), diff_planes_kernel<T, Q>, grid, kThreads, 0, st, f));
    return LLSA_OK;
}

template <typename T, typename Q>
int launch_planes_fwd(const DiffShape& s, const DiffArgs& a, void* ws, cudaStream_t st) {
    FourArgs f;
    memset(&f, 0, sizeof(f));
    f.a = a;
    char* at = static_cast<char*>(ws);
    void* planes[4];
    LLSA_TRY((launch_planes<T, Q>(s, a, false, at, planes, st)));
    f.o = reinterpret_cast<float*>(at);
    at += four_rows(s);
    f.lse = reinterpret_cast<float*>(at);
    at += four_lse(s);
    DenseArgs d = four_args(s, a, f, true);
    d.o_out = f.o;
    d.lse_out = f.lse;
    LLSA_TRY(launch_dense_fwd_planes(s.four, d, planes, at, st));
    LLSA_LAUNCH("diff_combine", st,
                launch_close(true, diff_combine_kernel<T, Q>, dim3(blocks_for((long long)s.slices * s.R * (s.d / 2))), kThreads, 0, st, f));
    return LLSA_OK;
}

template <typename T, typename Q>
int launch_planes_bwd(const DiffShape& s, DiffArgs a, void* dq, void* dk, void* dv, void* dlam, void* ws, cudaStream_t st) {
    char* at = static_cast<char*>(ws);
    auto take = [&](size_t bytes) { char* p = at; at += bytes; return reinterpret_cast<float*>(p); };
    void* planes[4];
    LLSA_TRY((launch_planes<T, Q>(s, a, true, at, planes, st)));
    void* const order[4] = {planes[0], planes[3], planes[1], planes[2]};  // q, dout, k, v
    FourArgs f;
    memset(&f, 0, sizeof(f));
    float *gq = take(four_rows(s)), *gk = take(four_keys(s)), *gv = take(four_keys(s));
    a.d.nl2 = take(4 * padded_rows(s));
    a.d.nd = take(4 * padded_rows(s));
    a.d2 = take(padded_rows(s));
    float* part = take(row_parts_bytes(s));
    const long long blocks = (long long)s.slices * (s.Rp / kDenseRowPad);
    if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("diff_rows", st, launch_close(true, diff_rows_kernel<T, Q, true>, dim3((unsigned)blocks), kThreads, 0, st, a));
    f.a = a;
    DenseArgs d = four_args(s, a, f, true);
    d.dq = gq;
    d.dk = gk;
    d.dv = gv;
    LLSA_TRY(launch_dense_bwd_planes(s.four, d, order, at, st));
    f.dq = gq;
    f.dk = gk;
    f.dv = gv;
    f.dq_out = dq;
    f.dk_out = dk;
    f.dv_out = dv;
    const unsigned grid = blocks_for((long long)s.four.slices * std::max(s.R, s.nk) * (s.d / 4));
    LLSA_LAUNCH("diff_collapse", st, launch_close(true, diff_collapse_kernel<T, Q>, dim3(grid, 3), kThreads, 0, st, f));
    return launch_lam_rows(s, a, 1, 0, part, dlam, st);
}

template <typename T, typename Q>
int launch_four_fwd(const DiffShape& s, const DiffArgs& a, void* ws, cudaStream_t st) {
    if (dense_fwd_on_planes(s.four)) return launch_planes_fwd<T, Q>(s, a, ws, st);
    FourArgs f;
    memset(&f, 0, sizeof(f));
    f.a = a;
    char* at = static_cast<char*>(ws);
    auto take = [&](size_t bytes) { char* p = at; at += bytes; return reinterpret_cast<float*>(p); };
    f.q = take(four_rows(s));
    f.o = take(four_rows(s));
    f.k = take(four_keys(s));
    f.v = take(four_keys(s));
    f.lse = take(four_lse(s));
    const dim3 grid(blocks_for((long long)s.four.slices * std::max(s.R, s.nk) * (s.d / 4)), s.nk > 0 ? 2 : 1);
    LLSA_LAUNCH("diff_expand", st, diff_expand_kernel<T, Q, false><<<grid, kThreads, 0, st>>>(f));
    DenseArgs d = four_args(s, a, f);
    d.o_out = f.o;
    d.lse_out = f.lse;
    LLSA_TRY(launch_dense_fwd(s.four, d, at, st));
    LLSA_LAUNCH("diff_combine", st,
                diff_combine_kernel<T, Q><<<blocks_for((long long)s.slices * s.R * (s.d / 2)), kThreads, 0, st>>>(f));
    return LLSA_OK;
}

size_t lam_bytes(const DiffShape& s) { return s.heads ? up((size_t)s.heads * lam_parts(s) * sizeof(float)) : 0; }

template <typename T, typename Q>
int launch_four_bwd(const DiffShape& s, const DiffArgs& a, void* dq, void* dk, void* dv, void* dlam, void* ws, cudaStream_t st) {
    if (dense_bwd_on_planes(s.four)) return launch_planes_bwd<T, Q>(s, a, dq, dk, dv, dlam, ws, st);
    LLSA_TRY((launch_lam<T, Q>(s, a, dlam, static_cast<float*>(ws), st)));
    if (s.R == 0 && s.nk == 0) return LLSA_OK;
    FourArgs f;
    memset(&f, 0, sizeof(f));
    f.a = a;
    char* at = static_cast<char*>(ws) + lam_bytes(s);
    auto take = [&](size_t bytes) { char* p = at; at += bytes; return reinterpret_cast<float*>(p); };
    f.q = take(four_rows(s));
    f.dout = take(four_rows(s));
    f.o = take(four_rows(s));
    float* gq = take(four_rows(s));
    f.k = take(four_keys(s));
    f.v = take(four_keys(s));
    float *gk = take(four_keys(s)), *gv = take(four_keys(s));
    f.lse = take(four_lse(s));
    const dim3 grid(blocks_for((long long)s.four.slices * std::max(s.R, s.nk) * (s.d / 4)), s.nk > 0 ? 2 : 1);
    LLSA_LAUNCH("diff_expand", st, diff_expand_kernel<T, Q, true><<<grid, kThreads, 0, st>>>(f));
    DenseArgs d = four_args(s, a, f);
    d.o = f.o;
    d.lse = f.lse;
    d.dout = f.dout;
    d.dq = gq;
    d.dk = gk;
    d.dv = gv;
    LLSA_TRY(launch_dense_bwd(s.four, d, at, st));
    f.dq = gq;
    f.dk = gk;
    f.dv = gv;
    f.dq_out = dq;
    f.dk_out = dk;
    f.dv_out = dv;
    LLSA_LAUNCH("diff_collapse", st, diff_collapse_kernel<T, Q><<<dim3(grid.x, s.nk > 0 ? 3 : 1), kThreads, 0, st>>>(f));
    return LLSA_OK;
}


// Which kernels take a call.
enum class Path { kFew, kTc, kFour };

Path fwd_path(const DiffShape& s) {
    return s.wide ? Path::kFour : diff_few_supported(s) ? Path::kFew : diff_tc_supported(s) ? Path::kTc : Path::kFour;
}

DenseSplit fwd_split(const DiffShape& s) {
    switch (fwd_path(s)) {
        case Path::kFew: return diff_few_split(s);
        case Path::kTc: return diff_tc_fwd_split(s);
        default: return {1, s.nk};
    }
}

size_t fwd_workspace(const DiffShape& s) {
    if (s.R == 0) return 0;
    return fwd_path(s) == Path::kFour ? four_workspace(s, false) : diff_part_bytes(s, fwd_split(s).splits);
}

int launch_diff_fwd(const DiffShape& s, DiffArgs a, void* ws, cudaStream_t st) {
    const bool bf16 = s.dtype == LLSA_DTYPE_BF16;
    const Path path = fwd_path(s);
    if (path == Path::kFour)
        return s.wide ? launch_four_fwd<__nv_bfloat16, float>(s, a, ws, st)
               : bf16 ? launch_four_fwd<__nv_bfloat16, __nv_bfloat16>(s, a, ws, st)
                      : launch_four_fwd<float, float>(s, a, ws, st);
    const DenseSplit p = fwd_split(s);
    a.d.splits = p.splits;
    a.d.chunk = p.chunk;
    a.d.part = static_cast<float*>(ws);
    LLSA_TRY(path == Path::kFew ? launch_diff_few(s, a, st) : launch_diff_tc_fwd(s, a, st));
    if (p.splits > 1) {
        const unsigned blocks = (unsigned)((long long)s.slices * s.R);  // few: blocks would do without a split otherwise
        if (bf16) LLSA_LAUNCH("diff_join", st, launch_close(true, diff_join_kernel<__nv_bfloat16>, dim3(blocks), kThreads, 0, st, a));
        else LLSA_LAUNCH("diff_join", st, launch_close(true, diff_join_kernel<float>, dim3(blocks), kThreads, 0, st, a));
    }
    return LLSA_OK;
}

Path bwd_path(const DiffShape& s) { return !s.wide && diff_tc_supported(s) ? Path::kTc : Path::kFour; }

// Workspace of the tensor-core backward pass, in order: the rows' numbers, the sums of
// P_2 dP, parts of those over a head's rows, parts of dq, of dk, of dv.
struct TcBwd {
    DenseSplit q, k;
    long long nq, nk;  // elements of dq, and of dk or dv
    size_t stats, d2, lam, dq, dkv;
    size_t bytes() const { return stats + d2 + lam + dq + dkv; }
};

TcBwd tc_bwd(const DiffShape& s) {
    TcBwd t;
    diff_tc_bwd_splits(s, &t.q, &t.k);
    t.nq = 2LL * s.slices * s.R * s.d;
    t.nk = 2LL * s.slices * s.nk * s.d;
    const size_t rows = (size_t)s.slices * s.Rp * sizeof(float);
    t.stats = up(kDiffStats * rows);
    t.d2 = up(4 * t.q.splits * rows);
    t.lam = row_parts_bytes(s);
    t.dq = t.q.splits > 1 ? up(t.q.splits * t.nq * sizeof(float)) : 0;
    t.dkv = t.k.splits > 1 ? up(2 * t.k.splits * t.nk * sizeof(float)) : 0;
    return t;
}

int launch_tc_bwd(const DiffShape& s, DiffArgs a, void* dq, void* dk, void* dv, void* dlam, void* ws, cudaStream_t st) {
    const TcBwd t = tc_bwd(s);
    char* at = static_cast<char*>(ws);
    auto take = [&](size_t bytes) { char* p = at; at += bytes; return reinterpret_cast<float*>(p); };
    a.d.nl2 = take(t.stats);
    a.d2 = take(t.d2);
    float* lam = take(t.lam);
    a.d.dq = dq;
    a.d.dk = dk;
    a.d.dv = dv;
    // Up to 4,096 numbers of a head the last block of dq sums them, which takes the GPU as long as a
    // launch behind it, but not the host (6 heads x 64 tokens, a call among others 34.8 -> 30.4 us).
    const int sets = 4 * t.q.splits;
    const bool last = (long long)s.batch * s.nq * sets <= 4096 && s.heads <= 64;
    if (last) {
        a.lam_ticket = reinterpret_cast<int*>(lam);
        a.dlam = dlam;
        a.lam_pieces = (int)((long long)(s.Rp / kDenseRowPad) * s.slices * t.q.splits);
        a.lam_sets = sets;
    }
    DiffArgs aq = a, ak = a;
    aq.d.splits = t.q.splits;
    aq.d.chunk = t.q.chunk;
    aq.d.part = take(t.dq);
    ak.d.splits = t.k.splits;
    ak.d.chunk = t.k.chunk;
    ak.d.part = take(t.dkv);
    const long long blocks = (long long)s.slices * (s.Rp / kDenseRowPad);
    if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("diff_rows", st, launch_close(close_first(st), diff_rows_kernel<__nv_bfloat16, __nv_bfloat16, false>, dim3((unsigned)blocks), kThreads, 0, st,
                                           a));
    LLSA_TRY(launch_diff_tc_bwd(s, aq, ak, st));
    if (!last) LLSA_TRY(launch_lam_rows(s, a, sets, 1, lam, dlam, st));
    DenseSums sums;
    if (t.q.splits > 1) sums.add(aq.d.part, dq, t.nq, t.q.splits);
    if (t.k.splits > 1) {
        sums.add(ak.d.part, dk, t.nk, t.k.splits);
        sums.add(ak.d.part + t.k.splits * t.nk, dv, t.nk, t.k.splits);
    }
    return launch_dense_sums(s.dtype, sums, st);
}

size_t bwd_workspace(const DiffShape& s) {
    return bwd_path(s) == Path::kTc ? tc_bwd(s).bytes() : (dense_bwd_on_planes(s.four) ? 0 : lam_bytes(s)) + four_workspace(s, true);
}

}  // namespace
}  // namespace llsa

using namespace llsa;

extern "C" {

size_t llsa_diff_workspace_bytes(const llsa_diff_params* p, int op) {
    DiffShape s;
    if (derive_diff(p, &s) != LLSA_OK || s.slices == 0) return 0;
    switch (op) {
        case LLSA_OP_DIFF_FWD: return fwd_workspace(s);
        case LLSA_OP_DIFF_BWD: return bwd_workspace(s);
        default: return 0;
    }
}

int llsa_diff_fwd(const llsa_diff_params* p, const void* q, const void* k, const void* v, const void* lam,
                  const int32_t* q_len, const int32_t* k_len, void* o, void* o2, float* lse, void* ws, size_t ws_bytes,
                  void* stream) {
    CallRange range("llsa_diff_fwd");
    DiffShape s;
    LLSA_TRY(derive_diff(p, &s));
    if (s.slices == 0 || s.R == 0) return LLSA_OK;
    LLSA_TRY(check_ptrs({q, lam, o, lse}));
    if (o2) LLSA_TRY(check_ptrs({o2}));
    if (s.nk > 0) LLSA_TRY(check_ptrs({k, v}));
    LLSA_TRY(dense_check_lens(q_len, k_len));
    const size_t need = fwd_workspace(s);
    if (need > 0 && (!ws || ws_bytes < need)) return LLSA_ERR_WORKSPACE;
    if (need > 0) LLSA_TRY(check_ptrs({ws}));
    LLSA_TRY(device_ready());
    DiffArgs a = diff_args(s);
    a.d.q = q;
    a.d.k = k;
    a.d.v = v;
    a.d.q_len = q_len;
    a.d.k_len = k_len;
    a.d.o_out = o;
    a.d.lse_out = lse;
    a.lam = lam;
    a.o2_out = o2;
    return launch_diff_fwd(s, a, ws, static_cast<cudaStream_t>(stream));
}

int llsa_diff_bwd(const llsa_diff_params* p, const void* q, const void* k, const void* v, const void* lam, const void* o,
                  const void* o2, const float* lse, const void* dout, const int32_t* q_len, const int32_t* k_len, void* dq,
                  void* dk, void* dv, void* dlam, void* ws, size_t ws_bytes, void* stream) {
    CallRange range("llsa_diff_bwd");
    DiffShape s;
    LLSA_TRY(derive_diff(p, &s));
    if (s.heads == 0) return LLSA_OK;
    LLSA_TRY(check_ptrs({lam, dlam}));
    const bool rows = s.slices > 0 && s.R > 0, keys = s.slices > 0 && s.nk > 0;
    if (rows) LLSA_TRY(check_ptrs({q, o, o2, lse, dout, dq}));
    if (keys) LLSA_TRY(check_ptrs({k, v, dk, dv}));
    LLSA_TRY(dense_check_lens(q_len, k_len));
    const size_t need = s.slices > 0 ? bwd_workspace(s) : 0;
    if (need > 0 && (!ws || ws_bytes < need)) return LLSA_ERR_WORKSPACE;
    if (need > 0) LLSA_TRY(check_ptrs({ws}));
    LLSA_TRY(device_ready());
    DiffArgs a = diff_args(s);
    a.d.q = q;
    a.d.k = k;
    a.d.v = v;
    a.d.q_len = q_len;
    a.d.k_len = k_len;
    a.d.o = o;
    a.d.lse = lse;
    a.d.dout = dout;
    a.lam = lam;
    a.o2 = o2;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (s.slices == 0) {  // an empty batch: nothing to add up
        LLSA_LAUNCH("diff_lam_sum", st, diff_lam_sum_kernel<<<s.heads, 32, 0, st>>>(nullptr, 0, dlam, s.lam_dtype == LLSA_DTYPE_BF16));
        return LLSA_OK;
    }
    if (bwd_path(s) == Path::kTc) return launch_tc_bwd(s, a, dq, dk, dv, dlam, ws, st);
    return s.wide                       ? launch_four_bwd<__nv_bfloat16, float>(s, a, dq, dk, dv, dlam, ws, st)
           : s.dtype == LLSA_DTYPE_BF16 ? launch_four_bwd<__nv_bfloat16, __nv_bfloat16>(s, a, dq, dk, dv, dlam, ws, st)
                                        : launch_four_bwd<float, float>(s, a, dq, dk, dv, dlam, ws, st);
}

}  // extern "C"

// dense_simt.cu -- dense attention on the CUDA cores: fp32 behind 128 columns, where the
// three bf16 planes of a tile of 128 rows would fill shared memory by themselves.
//
// Forward: one pass over the keys with the running maximum and sum of the
// softmax. Backward: probabilities recomputed from lse; dq by blocks of query
// rows, dk and dv by blocks of keys, so that every sum has one owner and a
// fixed order.
//
// A block takes BM rows against tiles of BM rows of the other side, 256
// threads as 16 x 16, each with an (BM / 16)^2 piece of the score tile and
// BM / 16 rows of the output. Operands sit in shared memory, rows of
// DP + 4 floats: the 16 rows that a quarter warp reads then fall on distinct
// banks. Bound by shared memory: per 4 columns of d a thread loads 4 vectors for 16
// FMAs (4 heads x 2,048 tokens, d = 256: forward 827 us, 21 TFLOP/s of 80; backward
// 3.0 ms, 14).
#include <algorithm>

#include "dense.h"

namespace llsa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

// BM rows of a [rows][d] matrix from row r0 on into shared memory, zeros where
// valid(row) fails and behind column d.
template <int DP, int BM, typename F>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int r0, int d, F valid) {
    constexpr int C = DP / 4;
    for (int x = threadIdx.x; x < BM * C; x += kThreads) {
        const int r = x / C, c = (x - r * C) * 4;
        float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < d && valid(r0 + r)) f = load4(src + (long long)(r0 + r) * d + c);
        *reinterpret_cast<float4*>(dst + r * (DP + 4) + c) = f;
    }
}

// The same through asynchronous copies: in shared memory after async_wait
// and a barrier.
template <int DP, int BM, typename F>
__device__ __forceinline__ void fetch_tile(float* dst, const float* src, int r0, int d, F valid) {
    constexpr int C = DP / 4;
    for (int x = threadIdx.x; x < BM * C; x += kThreads) {
        const int r = x / C, c = (x - r * C) * 4;
        const bool on = c < d && valid(r0 + r);
        const float* from = on ? src + (long long)(r0 + r) * d + c : src;
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * (DP + 4) + c));
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" :: "r"(to), "l"(from), "r"(on ? 16 : 0) : "memory");
    }
}
__device__ __forceinline__ void async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ void async_wait() { asm volatile("cp.async.wait_group 0;\n" ::: "memory"); }

// Tiles of two streamed operands, one after the other, in two buffers: the next tile
// comes in during this one's work. With one buffer 8 heads x 300 queries x 5,000 keys of
// 256 columns took 1,911 us forward instead of 1,006, and 4 heads x 2,048 tokens 3,677
// backward instead of 2,993 (one block per SM either way).
template <int DP, int BM, typename F>
struct Stream {
    float *x, *y;  // two tiles each
    const float *gx, *gy;
    int d, buf;
    F valid;

    __device__ __forceinline__ void fetch(int r0) {  // into the buffer that is not in use
        fetch_tile<DP, BM>(x + buf * BM * (DP + 4), gx, r0, d, valid);
        fetch_tile<DP, BM>(y + buf * BM * (DP + 4), gy, r0, d, valid);
        async_commit();
    }
    // The tile that was asked for becomes the current one, and the one at `next` (or -1) is asked for.
    __device__ __forceinline__ void turn(int next) {
        async_wait();
        __syncthreads();
        buf ^= 1;
        if (next >= 0) fetch(next);
    }
    __device__ __forceinline__ const float* cx() const { return x + (buf ^ 1) * BM * (DP + 4); }
    __device__ __forceinline__ const float* cy() const { return y + (buf ^ 1) * BM * (DP + 4); }
};

// acc[i][j] = A row (ty * N + i) . B row (tx + 16 j)
template <int N, int DP>
__device__ __forceinline__ void tile_dot(float (&acc)[N][N], const float* A, const float* B, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < N; j++) acc[i][j] = 0.f;
#pragma unroll 4
    for (int k = 0; k < DP; k += 4) {
        float4 x[N], y[N];
#pragma unroll
        for (int i = 0; i < N; i++) x[i] = *reinterpret_cast<const float4*>(A + (ty * N + i) * (DP + 4) + k);
#pragma unroll
        for (int j = 0; j < N; j++) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * (DP + 4) + k);
#pragma unroll
        for (int i = 0; i < N; i++)
#pragma unroll
            for (int j = 0; j < N; j++) {
                acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
            }
    }
}

// acc[i][c] (columns 4 tx + 64 c ..) += sum over the BM entries of P row (ty * N + i) times X's rows
template <int N, int DP, int BM>
__device__ __forceinline__ void tile_acc(float4 (&acc)[N][DP / 64], const float* P, const float* X, int ty, int tx) {
#pragma unroll 2
    for (int k = 0; k < BM; k += 4) {
        float4 p[N];
#pragma unroll
        for (int i = 0; i < N; i++) p[i] = *reinterpret_cast<const float4*>(P + (ty * N + i) * (BM + 4) + k);
#pragma unroll
        for (int c = 0; c < DP / 64; c++)
#pragma unroll
            for (int kk = 0; kk < 4; kk++) {
                const float4 x = *reinterpret_cast<const float4*>(X + (k + kk) * (DP + 4) + 4 * tx + 64 * c);
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const float w = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                    acc[i][c].x = fmaf(w, x.x, acc[i][c].x);
                    acc[i][c].y = fmaf(w, x.y, acc[i][c].y);
                    acc[i][c].z = fmaf(w, x.z, acc[i][c].z);
                    acc[i][c].w = fmaf(w, x.w, acc[i][c].w);
                }
            }
    }
}

template <int N>
__device__ __forceinline__ void store_p(float* P, const float (&v)[N][N], int ty, int tx) {
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < N; j++) P[(ty * N + i) * (16 * N + 4) + tx + 16 * j] = v[i][j];
}

// One row's columns of the result, times f.
template <int DP>
__device__ __forceinline__ void store_row(float* dst, const float4 (&acc)[DP / 64], float f, int d, int tx) {
#pragma unroll
    for (int c = 0; c < DP / 64; c++)
        if (4 * tx + 64 * c < d) {
            const float v[4] = {acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f};
            store4(dst + 4 * tx + 64 * c, v);
        }
}

// ---------------------------------------------------------------- forward --

// Partial results of a split over the keys: o unnormalised [split][slice][R][d],
// then (maximum, sum) pairs [split][slice][R].
template <int DP, int BM>
__global__ void __launch_bounds__(kThreads) dense_fwd_simt_kernel(DenseArgs a) {
    constexpr int N = BM / 16;
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sK = sQ + BM * (DP + 4);
    float* sV = sK + 2 * BM * (DP + 4);
    float* sP = sV + 2 * BM * (DP + 4);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles = (a.R + BM - 1) / BM;
    const int slice = blockIdx.x / tiles, r0 = (blockIdx.x - slice * tiles) * BM, part = blockIdx.y;
    const DenseSpan sp = dense_span(a, slice);
    const float* q = static_cast<const float*>(a.q) + (long long)slice * a.R * a.d;
    const float* k = static_cast<const float*>(a.k) + (long long)slice * a.nk * a.d;
    const float* v = static_cast<const float*>(a.v) + (long long)slice * a.nk * a.d;
    load_tile<DP, BM>(sQ, q, r0, a.d, [&](int r) { return r < a.R; });
    int kend[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int r = r0 + ty * N + i;
        kend[i] = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
    }
    const int j_first = part * a.chunk;
    const int j_last = min(dense_tile_kend(a, sp, r0 % a.nq, BM), a.splits > 1 ? j_first + a.chunk : a.nk);
    const float sl2 = a.scale * kDenseLog2e;
    float m[N], l[N];
    float4 acc[N][DP / 64];
#pragma unroll
    for (int i = 0; i < N; i++) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 64; c++) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto key_ok = [&](int j) { return j < sp.lk; };
    Stream<DP, BM, decltype(key_ok)> stream{sK, sV, k, v, a.d, 0, key_ok};
    if (j_first < j_last) stream.fetch(j_first);
    for (int j0 = j_first; j0 < j_last; j0 += BM) {
        stream.turn(j0 + BM < j_last ? j0 + BM : -1);
        float s[N][N];
        tile_dot<N, DP>(s, sQ, stream.cx(), ty, tx);
#pragma unroll
        for (int i = 0; i < N; i++) {
            float top = m[i];
#pragma unroll
            for (int j = 0; j < N; j++) {
                s[i][j] = j0 + tx + 16 * j < kend[i] ? s[i][j] * sl2 : -INFINITY;
                top = fmaxf(top, s[i][j]);
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const float shift = top == -INFINITY ? 0.f : top;  // no key yet: every weight below is exp2(-inf) = 0
            const float f = exp2f(m[i] - shift);
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < N; j++) {
                s[i][j] = exp2f(s[i][j] - shift);
                sum += s[i][j];
            }
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l[i] = l[i] * f + sum;
#pragma unroll
            for (int c = 0; c < DP / 64; c++) {
                acc[i][c].x *= f;
                acc[i][c].y *= f;
                acc[i][c].z *= f;
                acc[i][c].w *= f;
            }
        }
        store_p<N>(sP, s, ty, tx);
        __syncthreads();
        tile_acc<N, DP, BM>(acc, sP, stream.cy(), ty, tx);
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int r = r0 + ty * N + i;
        if (r >= a.R) continue;
        const long long row = (long long)slice * a.R + r;
        if (a.splits > 1) {
            const long long prow = (long long)part * a.slices * a.R + row;
            store_row<DP>(a.part + prow * a.d, acc[i], 1.f, a.d, tx);
            float2* ml = reinterpret_cast<float2*>(a.part + (long long)a.splits * a.slices * a.R * a.d);
            if (tx == 0) ml[prow] = make_float2(m[i], l[i]);
        } else {
            store_row<DP>(static_cast<float*>(a.o_out) + row * a.d, acc[i], l[i] == 0.f ? 0.f : 1.f / l[i], a.d, tx);
            if (tx == 0) a.lse_out[row] = l[i] == 0.f ? -INFINITY : m[i] * 0.6931471805599453f + logf(l[i]);
        }
    }
}

// --------------------------------------------------------------- backward --

// dq of BM query rows. Partial sums of a split over the keys: [split][slice][R][d].
template <int DP, int BM>
__device__ __forceinline__ void rows_side(const DenseArgs& a, int piece) {
    constexpr int N = BM / 16;
    extern __shared__ float4 smem4[];
    float* sQ = reinterpret_cast<float*>(smem4);
    float* sG = sQ + BM * (DP + 4);
    float* sK = sG + BM * (DP + 4);
    float* sV = sK + 2 * BM * (DP + 4);
    float* sP = sV + 2 * BM * (DP + 4);
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles = (a.R + BM - 1) / BM;
    const int part = piece / (tiles * a.slices), rest = piece - part * (tiles * a.slices);
    const int slice = rest / tiles, r0 = (rest - slice * tiles) * BM;
    const DenseSpan sp = dense_span(a, slice);
    const float* q = static_cast<const float*>(a.q) + (long long)slice * a.R * a.d;
    const float* g = static_cast<const float*>(a.dout) + (long long)slice * a.R * a.d;
    const float* k = static_cast<const float*>(a.k) + (long long)slice * a.nk * a.d;
    const float* v = static_cast<const float*>(a.v) + (long long)slice * a.nk * a.d;
    auto row_ok = [&](int r) { return r < a.R && r % a.nq < sp.lq; };
    load_tile<DP, BM>(sQ, q, r0, a.d, row_ok);
    load_tile<DP, BM>(sG, g, r0, a.d, row_ok);
    int kend[N];
    float nl2[N], nd[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int r = r0 + ty * N + i;
        kend[i] = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
        nl2[i] = r < a.R ? a.nl2[(long long)slice * a.Rp + r] : -INFINITY;
        nd[i] = r < a.R ? a.nd[(long long)slice * a.Rp + r] : 0.f;
    }
    const int j_first = part * a.chunk;
    const int j_last = min(dense_tile_kend(a, sp, r0 % a.nq, BM), a.splits > 1 ? j_first + a.chunk : a.nk);
    const float sl2 = a.scale * kDenseLog2e;
    float4 acc[N][DP / 64];
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int c = 0; c < DP / 64; c++) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto key_ok = [&](int j) { return j < sp.lk; };
    Stream<DP, BM, decltype(key_ok)> stream{sK, sV, k, v, a.d, 0, key_ok};
    if (j_first < j_last) stream.fetch(j_first);
    for (int j0 = j_first; j0 < j_last; j0 += BM) {
        stream.turn(j0 + BM < j_last ? j0 + BM : -1);
        float s[N][N], dp[N][N];
        tile_dot<N, DP>(s, sQ, stream.cx(), ty, tx);
        tile_dot<N, DP>(dp, sG, stream.cy(), ty, tx);
#pragma unroll
        for (int i = 0; i < N; i++)
#pragma unroll
            for (int j = 0; j < N; j++) {
                const float p = exp2f(fmaf(s[i][j], sl2, nl2[i]));
                s[i][j] = j0 + tx + 16 * j < kend[i] ? p * (dp[i][j] + nd[i]) : 0.f;
            }
        store_p<N>(sP, s, ty, tx);
        __syncthreads();
        tile_acc<N, DP, BM>(acc, sP, stream.cx(), ty, tx);
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int r = r0 + ty * N + i;
        if (r >= a.R) continue;
        const long long row = (long long)slice * a.R + r;
        if (a.splits > 1)
            store_row<DP>(a.part + ((long long)part * a.slices * a.R + row) * a.d, acc[i], a.scale, a.d, tx);
        else
            store_row<DP>(static_cast<float*>(a.dq) + row * a.d, acc[i], a.scale, a.d, tx);
    }
}

// dk and dv of BM keys, over the query rows of all heads that share them.
// Partial sums of a split over the rows: dk [split][slice][nk][d], then dv.
template <int DP, int BM>
__device__ __forceinline__ void keys_side(const DenseArgs& a, int piece) {
    constexpr int N = BM / 16;
    extern __shared__ float4 smem4[];
    float* sK = reinterpret_cast<float*>(smem4);
    float* sV = sK + BM * (DP + 4);
    float* sQ = sV + BM * (DP + 4);
    float* sG = sQ + 2 * BM * (DP + 4);
    float* sP = sG + 2 * BM * (DP + 4);  // P^T
    float* sS = sP + BM * (BM + 4);  // dS^T
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int tiles = (a.nk + BM - 1) / BM;
    const int part = piece / (tiles * a.slices), rest = piece - part * (tiles * a.slices);
    const int slice = rest / tiles, j0 = (rest - slice * tiles) * BM;
    const DenseSpan sp = dense_span(a, slice);
    const float* q = static_cast<const float*>(a.q) + (long long)slice * a.R * a.d;
    const float* g = static_cast<const float*>(a.dout) + (long long)slice * a.R * a.d;
    const float* k = static_cast<const float*>(a.k) + (long long)slice * a.nk * a.d;
    const float* v = static_cast<const float*>(a.v) + (long long)slice * a.nk * a.d;
    auto key_ok = [&](int j) { return j < sp.lk; };
    auto row_ok = [&](int r) { return r < a.R && r % a.nq < sp.lq; };
    load_tile<DP, BM>(sK, k, j0, a.d, key_ok);
    load_tile<DP, BM>(sV, v, j0, a.d, key_ok);
    const int r_first = a.splits > 1 ? part * a.chunk : 0;
    const int r_last = a.splits > 1 ? min(a.R, r_first + a.chunk) : a.R;
    const float sl2 = a.scale * kDenseLog2e;
    float4 dk[N][DP / 64], dv[N][DP / 64];
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int c = 0; c < DP / 64; c++) dk[i][c] = dv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto settle = [&](int r0) {  // the first tile from r0 on that sees any of these keys, or -1
        while (r0 < r_last && dense_tile_kend(a, sp, r0 % a.nq, BM) <= j0) r0 += BM;
        return r0 < r_last ? r0 : -1;
    };
    Stream<DP, BM, decltype(row_ok)> stream{sQ, sG, q, g, a.d, 0, row_ok};
    int next = settle(r_first);
    if (next >= 0) stream.fetch(next);
    while (next >= 0) {
        const int r0 = next;
        next = settle(r0 + BM);
        stream.turn(next);
        float s[N][N], dp[N][N];
        tile_dot<N, DP>(s, sK, stream.cx(), ty, tx);
        tile_dot<N, DP>(dp, sV, stream.cy(), ty, tx);
#pragma unroll
        for (int j = 0; j < N; j++) {
            const int r = r0 + tx + 16 * j;
            const int kend = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
            const float nl2 = r < a.R ? a.nl2[(long long)slice * a.Rp + r] : -INFINITY;
            const float nd = r < a.R ? a.nd[(long long)slice * a.Rp + r] : 0.f;
#pragma unroll
            for (int i = 0; i < N; i++) {
                const float p = j0 + ty * N + i < kend ? exp2f(fmaf(s[i][j], sl2, nl2)) : 0.f;
                s[i][j] = p;
                dp[i][j] = p * (dp[i][j] + nd);
            }
        }
        store_p<N>(sP, s, ty, tx);
        store_p<N>(sS, dp, ty, tx);
        __syncthreads();
        tile_acc<N, DP, BM>(dv, sP, stream.cy(), ty, tx);
        tile_acc<N, DP, BM>(dk, sS, stream.cx(), ty, tx);
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int j = j0 + ty * N + i;
        if (j >= a.nk) continue;
        if (j >= sp.lk) {  // zeros, also beside a row that is no number
#pragma unroll
            for (int c = 0; c < DP / 64; c++) dk[i][c] = dv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        const long long row = (long long)slice * a.nk + j;
        if (a.splits > 1) {
            const long long all = (long long)a.slices * a.nk;
            store_row<DP>(a.part + (part * all + row) * a.d, dk[i], a.scale, a.d, tx);
            store_row<DP>(a.part + ((a.splits + part) * all + row) * a.d, dv[i], 1.f, a.d, tx);
        } else {
            store_row<DP>(static_cast<float*>(a.dk) + row * a.d, dk[i], a.scale, a.d, tx);
            store_row<DP>(static_cast<float*>(a.dv) + row * a.d, dv[i], 1.f, a.d, tx);
        }
    }
}

// Pieces of keys first, they are the longer ones; those of rows fill up what they
// leave (12 heads x 64 tokens of 256 columns, with one buffer 94 us in two launches and 55 in one).
template <int DP, int BM>
__global__ void __launch_bounds__(kThreads)
dense_bwd_simt_kernel(const __grid_constant__ DenseArgs aq, const __grid_constant__ DenseArgs ak, int key_pieces) {
    const int piece = blockIdx.x;
    if (piece < key_pieces)
        keys_side<DP, BM>(ak, piece);
    else
        rows_side<DP, BM>(aq, piece - key_pieces);
}

constexpr int kColumns = 256, kRows = 32;  // of a tile

}  // namespace

DenseSplit dense_simt_fwd_split(const DenseShape& s) {  // dq: the same
    return dense_make_split((long long)s.slices * ((s.R + kRows - 1) / kRows), s.nk, kRows, 4);
}
DenseSplit dense_simt_dkv_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.nk + kRows - 1) / kRows), s.R, kRows, 4);
}

int launch_dense_simt_fwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    constexpr int BM = kRows, DP = kColumns, tile = BM * (DP + 4) * 4, p = BM * (BM + 4) * 4, smem = 5 * tile + p;
    static_assert(smem <= 227 * 1024, "shared memory budget");
    const long long blocks = (long long)((s.R + BM - 1) / BM) * s.slices;
    if (blocks > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, a.splits);
    cudaFuncSetAttribute(dense_fwd_simt_kernel<DP, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    LLSA_LAUNCH("dense_fwd_simt", st, dense_fwd_simt_kernel<DP, BM><<<grid, kThreads, smem, st>>>(a));
    return LLSA_OK;
}

int launch_dense_simt_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, cudaStream_t st) {
    constexpr int BM = kRows, DP = kColumns, tile = BM * (DP + 4) * 4, p = BM * (BM + 4) * 4;
    constexpr int smem = 6 * tile + 2 * p;
    static_assert(smem <= 227 * 1024, "shared memory budget");
    const long long pq = (long long)((s.R + BM - 1) / BM) * s.slices * aq.splits;
    const long long pk = (long long)((s.nk + BM - 1) / BM) * s.slices * ak.splits;
    if (pq + pk > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    cudaFuncSetAttribute(dense_bwd_simt_kernel<DP, BM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    LLSA_LAUNCH("dense_bwd_simt", st,
                dense_bwd_simt_kernel<DP, BM><<<(unsigned)(pq + pk), kThreads, smem, st>>>(aq, ak, (int)pk));
    return LLSA_OK;
}

}  // namespace llsa

// dense_keys.cu -- dense attention forward in fp32 against a handful of keys (a short
// conditioning sequence, a few memory tokens): the rows are read once, on the CUDA
// cores, with all keys and values of a slice in shared memory.
//
// Mathematics: one pass over the keys, four at a time, with the running maximum and
// sum of the softmax, everything in fp32.
//
// One to eight lanes share a row, 32 columns each in chunks of four that take turns, so
// that a warp's reads of a key are one row of shared memory and its reads of q whole
// sectors. A block stays with its slice for several tiles of rows. Bound by HBM at a
// few keys and by the FMA pipes and shared memory behind that (4 d operations per
// pair, two columns per instruction). 4 x 32 heads over 8 x 8,378 rows, d = 40: 4 keys
// 75 us, 16 keys 159, at HBM's rate 51; the tensor-core kernel 515, which fills tiles
// of 128 keys and writes planes of everything first.
#include <algorithm>

#include "dense.h"
#include "tc.cuh"

namespace llsa {
namespace {

using namespace tc;

constexpr int kThreads = 256, kChunks = 8, kMostKeys = 40;

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

template <int LPR>
__global__ void __launch_bounds__(kThreads) dense_fwd_keys_kernel(const __grid_constant__ DenseArgs a) {
    constexpr int DP = LPR * kChunks * 4, ROWS = kThreads / LPR;
    extern __shared__ float4 smem4[];
    float* sK = reinterpret_cast<float*>(smem4);  // keys in fours: [nk4][DP], zeros behind the lengths and d
    const int nk4 = (a.nk + 3) & ~3;
    float* sV = sK + nk4 * DP;
    const int slice = blockIdx.x / a.pieces, first = blockIdx.x - slice * a.pieces;  // pieces: blocks per slice
    const DenseSpan sp = dense_span(a, slice);
    for (int x = threadIdx.x; x < nk4 * (DP / 4); x += kThreads) {
        const int j = x / (DP / 4), c = (x - j * (DP / 4)) * 4;
        const bool on = j < sp.lk && c < a.d;
        const long long at = ((long long)slice * a.nk + j) * a.d + c;
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(sK + j * DP + c) = on ? load4(static_cast<const float*>(a.k) + at) : zero;
        *reinterpret_cast<float4*>(sV + j * DP + c) = on ? load4(static_cast<const float*>(a.v) + at) : zero;
    }
    __syncthreads();
    const int sub = threadIdx.x % LPR;
    const float sl2 = a.scale * kDenseLog2e;
    const int tiles = (a.R + ROWS - 1) / ROWS;
    for (int tile = first; tile < tiles; tile += a.pieces) {
        const int r = tile * ROWS + threadIdx.x / LPR;
        const int kend = r < a.R ? dense_kend(a, sp, r < a.nq ? r : r % a.nq) : 0;
        const long long row = (long long)slice * a.R + r;
        uint64_t q[kChunks][2], acc[kChunks][2];
#pragma unroll
        for (int i = 0; i < kChunks; i++) {
            const int c = (i * LPR + sub) * 4;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kend > 0 && c < a.d) f = load4(static_cast<const float*>(a.q) + row * a.d + c);
            q[i][0] = pack2(f.x * sl2, f.y * sl2);
            q[i][1] = pack2(f.z * sl2, f.w * sl2);
            acc[i][0] = acc[i][1] = 0ull;
        }
        float m = -INFINITY, l = 0.f;
        for (int j0 = 0; __any_sync(0xffffffffu, j0 < kend); j0 += 4) {
            float s[4];
#pragma unroll
            for (int u = 0; u < 4; u++) {
                uint64_t t0 = 0ull, t1 = 0ull;
                const ulonglong2* k = reinterpret_cast<const ulonglong2*>(sK + (j0 + u) * DP) + sub;
#pragma unroll
                for (int i = 0; i < kChunks; i++) {  // columns behind d are zeros: a branch would keep the loads apart
                    const ulonglong2 x = k[i * LPR];
                    t0 = fma2(q[i][0], x.x, t0);
                    t1 = fma2(q[i][1], x.y, t1);
                }
                float x0, x1;
                unpack2(add2(t0, t1), x0, x1);
                s[u] = x0 + x1;
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1) s[u] += __shfl_xor_sync(0xffffffffu, s[u], o);
                s[u] = j0 + u < kend ? s[u] : -INFINITY;
            }
            const float top = fmaxf(fmaxf(fmaxf(s[0], s[1]), fmaxf(s[2], s[3])), m);
            const float shift = top == -INFINITY ? 0.f : top;
            if (__any_sync(0xffffffffu, top > m)) {
                const float f = ex2(m - shift);  // 2^-inf = 0 at a row's first keys
                const uint64_t f2 = pack2(f, f);
                l *= f;
#pragma unroll
                for (int i = 0; i < kChunks; i++) {
                    acc[i][0] = mul2(acc[i][0], f2);
                    acc[i][1] = mul2(acc[i][1], f2);
                }
            }
            m = top;
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const float p = ex2(s[u] - shift);
                const uint64_t p2 = pack2(p, p);
                l += p;
                const ulonglong2* v = reinterpret_cast<const ulonglong2*>(sV + (j0 + u) * DP) + sub;
#pragma unroll
                for (int i = 0; i < kChunks; i++) {
                    const ulonglong2 x = v[i * LPR];
                    acc[i][0] = fma2(p2, x.x, acc[i][0]);
                    acc[i][1] = fma2(p2, x.y, acc[i][1]);
                }
            }
        }
        if (r >= a.R) continue;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < kChunks; i++) {
            const int c = (i * LPR + sub) * 4;
            float o[4];
            unpack2(acc[i][0], o[0], o[1]);
            unpack2(acc[i][1], o[2], o[3]);
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] *= inv;
            if (c < a.d) store4(static_cast<float*>(a.o_out) + row * a.d + c, o);
        }
        if (sub == 0) a.lse_out[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <int LPR>
int launch(const DenseShape& s, DenseArgs a, cudaStream_t st) {
    constexpr int DP = LPR * kChunks * 4, ROWS = kThreads / LPR;
    const int smem = ((s.nk + 3) & ~3) * DP * 2 * (int)sizeof(float);
    static_assert(kMostKeys * DP * 2 * 4 <= 227 * 1024, "shared memory budget");
    cudaFuncSetAttribute(dense_fwd_keys_kernel<LPR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * DP * 2 * 4);
    // as many blocks as two rounds of two per SM, each with as many tiles of its slice as that leaves
    const long long tiles = (s.R + ROWS - 1) / ROWS, want = std::max<long long>(1, 4LL * kDenseSms / s.slices);
    a.pieces = (int)std::min(tiles, want);
    const long long blocks = (long long)s.slices * a.pieces;
    if (blocks > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("dense_fwd_keys", st, dense_fwd_keys_kernel<LPR><<<(unsigned)blocks, kThreads, smem, st>>>(a));
    return LLSA_OK;
}

}  // namespace

// Up to where the tensor cores take over: 12 heads x 16,384 rows 48 keys 98 us against 107
// (64 tokens 9.4 against 8.4), 64 keys 123; 2 x 8 heads x 16,384 rows at 128 columns 16 keys
// 140 against 191, 32 keys 255; at 256 columns against the other CUDA-core kernel 32 keys 21
// against 21. In bf16 only four keys and fewer would gain (72 us against 121 at the shape above).
bool dense_keys_supported(const DenseShape& s) {
    const int most = s.d <= 64 ? kMostKeys : s.d <= 128 ? 20 : 32;
    return s.dtype == LLSA_DTYPE_F32 && s.R > 0 && s.nk > 0 && s.nk <= most;
}

int launch_dense_keys(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    return s.d <= 32    ? launch<1>(s, a, st)
           : s.d <= 64  ? launch<2>(s, a, st)
           : s.d <= 128 ? launch<4>(s, a, st)
                        : launch<8>(s, a, st);
}

}  // namespace llsa

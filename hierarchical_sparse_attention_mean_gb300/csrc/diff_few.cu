// diff_few.cu -- differential attention forward for a few query rows per value head (single
// tokens, their shared-value heads, pooling queries): both maps' keys and the values are read
// once per two rows, on the CUDA cores.
//
// Mathematics: one pass over the keys with a running maximum and sum for each map; a key's
// two weights meet its value while that is in registers. The keys of a slice are split
// over blocks, and inside a block over warps and groups of lanes, each with its own
// maxima, sums and outputs, joined at the end in a fixed order, and the maps' difference
// is formed in fp32 there.
//
// Bound by HBM with one row: 12 d flops per key and row against 8 d bytes per key (bf16). Keys
// and values of consecutive tokens lie next to each other, so a stage of 32 KB is three bulk
// copies, and a block per SM keeps six of them in flight: 6 heads x 65,536 keys of 64 columns,
// 201 MB, in 37 us (5.4 TB/s), the join of the parts 5 more; with the loads in registers instead,
// as many as fit, the kernel took 4 more. A group of 8 or 16 lanes takes one key, 8
// columns of each map's key and 16 of the value per lane. Further rows go in pairs, blocks
// side by side that read the same keys: the second pair finds them in L2.
#include <algorithm>

#include "dense_tc.cuh"
#include "diff.h"

namespace llsa {
namespace {

using namespace tc;

// Warps that take keys (one more copies): what hides the latency of a key's chain of
// products, shuffles and exponentials. Two rows take 153 registers a thread.
template <int RR>
constexpr int kFewWarps = RR == 1 ? 16 : 8;
constexpr int kStage = 32 * 1024, kStages = 6;

struct FewBars {
    uint64_t full[kStages], empty[kStages];
    int abort_flag;
};

template <typename T, int RR, int LANES>
__global__ void __launch_bounds__((kFewWarps<RR> + 1) * 32, 1) diff_few_kernel(const __grid_constant__ DiffArgs f) {
    const DenseArgs& a = f.d;
    constexpr int kWarps = kFewWarps<RR>, kThreads = (kWarps + 1) * 32;
    constexpr int GROUPS = 32 / LANES, VC = LANES * 8;      // keys of a warp at a time; columns of half a value
    constexpr int KS = kStage / (4 * VC * (int)sizeof(T));  // keys of a stage
    extern __shared__ __align__(128) unsigned char sm[];
    T* ring = reinterpret_cast<T*>(sm);  // per stage: KS rows of each map's keys, then of the values
    FewBars* bar = reinterpret_cast<FewBars*>(sm + kStages * kStage);
    volatile int* abort_flag = &bar->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    close_wait();
    close_ahead();
    const int slice = blockIdx.x / a.splits, part = blockIdx.x - slice * a.splits;
    const DenseSpan sp = dense_span(a, slice);
    const int dv = 2 * a.d, r0 = blockIdx.y * RR;
    int kend[RR], most = 0;
#pragma unroll
    for (int r = 0; r < RR; r++) {
        kend[r] = r0 + r < a.R ? dense_kend(a, sp, (r0 + r) % a.nq) : 0;
        most = max(most, kend[r]);
    }
    const int first = part * a.chunk;
    const int stop = min(most, a.splits > 1 ? first + a.chunk : a.nk);
    const int n = stop > first ? (stop - first + KS - 1) / KS : 0;  // stages
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; i++) {
            mbar_init(smem_u32(&bar->full[i]), 1);
            mbar_init(smem_u32(&bar->empty[i]), kWarps);
        }
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    const int grp = lane / LANES, col = (lane % LANES) * 8;
    float acc[RR][2][16], m[RR][2], l[RR][2];
    if (warp == kWarps) {
        // ----------------------------------------------------------- copies
        if (lane == 0 && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
            const int b = slice / a.kv_heads;
            const T* k0 = static_cast<const T*>(a.k) + ((long long)slice + (long long)b * a.kv_heads) * a.nk * a.d;
            const T* k1 = k0 + (long long)a.kv_heads * a.nk * a.d;
            const T* v = static_cast<const T*>(a.v) + (long long)slice * a.nk * dv;
            Stage<kStages> s;
            int filled = 0;
            for (; filled < n; filled++, s.next()) {
                if (filled >= kStages && !bar_wait(smem_u32(&bar->empty[s.st]), s.parity ^ 1, abort_flag, a)) break;
                const long long j = first + filled * KS;
                const uint32_t bytes = (uint32_t)(min(KS, stop - (int)j) * a.d * (int)sizeof(T));
                const uint32_t to = smem_u32(sm + s.st * kStage), fb = smem_u32(&bar->full[s.st]);
                mbar_arrive_expect_tx(fb, 4 * bytes);
                bulk_load(to, k0 + j * a.d, bytes, fb);
                bulk_load(to + kStage / 4, k1 + j * a.d, bytes, fb);
                bulk_load(to + kStage / 2, v + j * dv, 2 * bytes, fb);
            }
            // copies still in flight must land before the block exits
            for (int x = max(0, filled - kStages); x < filled; x++) land(smem_u32(&bar->full[x % kStages]), (x / kStages) & 1);
        }
    } else {
        const bool on = col < a.d, on1 = col < dv, on2 = VC + col < dv;
        const float sl2 = a.scale * kDenseLog2e;
        float q[RR][2][8];
#pragma unroll
        for (int r = 0; r < RR; r++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
                m[r][i] = -INFINITY;
                l[r][i] = 0.f;
#pragma unroll
                for (int c = 0; c < 8; c++) q[r][i][c] = acc[r][i][c] = acc[r][i][c + 8] = 0.f;
                if (on && kend[r] > 0) {
                    diff_load8(static_cast<const T*>(a.q) + diff_row(f, slice, i, r0 + r) * a.d + col, q[r][i]);
#pragma unroll
                    for (int c = 0; c < 8; c++) q[r][i][c] *= sl2;
                }
            }
        Stage<kStages> st;
        int last = 0;
        for (int t = 0; t < n; t++, st.next()) {
            if (!warp_wait(smem_u32(&bar->full[st.st]), st.parity, abort_flag, a)) break;
            const T* k0 = ring + (size_t)st.st * (kStage / sizeof(T));
            const T *k1 = k0 + kStage / 4 / sizeof(T), *v = k0 + kStage / 2 / sizeof(T);
            const int j0 = first + t * KS;
#pragma unroll
            for (int x0 = 0; x0 < KS; x0 += kWarps * GROUPS) {
                const int x = x0 + warp * GROUPS + grp, j = j0 + x;
                const bool here = x < KS && j < stop;  // what lies behind it in the stage is of other keys
                float s[RR][2], y[8];
#pragma unroll
                for (int i = 0; i < 2; i++) {
#pragma unroll
                    for (int c = 0; c < 8; c++) y[c] = 0.f;
                    if (here && on) diff_load8((i ? k1 : k0) + x * a.d + col, y);
#pragma unroll
                    for (int r = 0; r < RR; r++) {
                        float u = q[r][i][0] * y[0];
#pragma unroll
                        for (int c = 1; c < 8; c++) u = fmaf(q[r][i][c], y[c], u);
                        s[r][i] = u;
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
                        if (!here || j >= kend[r]) s[r][i] = -INFINITY;
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
#pragma unroll
                    for (int c = 0; c < 8; c++) y[c] = 0.f;
                    if (here && (h ? on2 : on1)) diff_load8(v + x * dv + h * VC + col, y);
#pragma unroll
                    for (int r = 0; r < RR; r++)
#pragma unroll
                        for (int i = 0; i < 2; i++)
#pragma unroll
                            for (int c = 0; c < 8; c++) acc[r][i][8 * h + c] = fmaf(s[r][i], y[c], acc[r][i][8 * h + c]);
                }
            }
            // An arrival right behind loads can overtake the last of them. So a stage is released in
            // the next round, when what was read from it has been used.
            if (t > 0) warp_arrive(smem_u32(&bar->empty[last]), lane);
            last = st.st;
        }
    }
    __syncthreads();  // the ring has been read: its place takes what is joined
    float* sO = reinterpret_cast<float*>(sm);                                 // [kWarps][RR][2][2 VC]
    float2* sML = reinterpret_cast<float2*>(sO + kWarps * RR * 2 * 2 * VC);  // [kWarps][RR][2]
    // the groups of a warp, then the warps, in a fixed order
    if (warp < kWarps) {
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
    }
    __syncthreads();
    for (int x = threadIdx.x; x < RR * dv; x += kThreads) {
        const int r = x / dv, c = x - r * dv;
        if (r0 + r >= a.R) break;
        float out[2];
        const long long row = (long long)slice * a.R + r0 + r;
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
                if (c == 0) a.lse_out[diff_row(f, slice, i, r0 + r)] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
            }
        }
        if (a.splits > 1) continue;
        const float o = fmaf(-diff_lam_row(f, slice, r0 + r), out[1], out[0]);
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
    constexpr int smem = kStages * kStage + (int)sizeof(FewBars);
    static_assert(smem <= 227 * 1024 && kFewWarps<RR> * RR * 2 * (2 * LANES * 8 + 2) * 4 <= kStages * kStage, "shared memory budget");
    cudaFuncSetAttribute(diff_few_kernel<T, RR, LANES>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    LLSA_LAUNCH("diff_few", st, launch_close(close_first(st), diff_few_kernel<T, RR, LANES>, dim3((unsigned)blocks, (a.d.R + RR - 1) / RR),
                                              (kFewWarps<RR> + 1) * 32, smem, st, a));
    return LLSA_OK;
}

template <typename T>
int launch(const DiffShape& s, const DiffArgs& a, cudaStream_t st) {
    if (s.R <= 1) return s.d <= 64 ? launch_lanes<T, 1, 8>(a, st) : launch_lanes<T, 1, 16>(a, st);
    return s.d <= 64 ? launch_lanes<T, 2, 8>(a, st) : launch_lanes<T, 2, 16>(a, st);
}

}  // namespace

// Where this is the faster way, times in us here and there (head columns d = 64):
// bf16 against the tensor cores, which read rows by 128. One row: 8 x 4 heads x 16,383 keys 66
//   and 70, d = 128 109 and 121; 6 heads x 65,536 keys 56 and 60; 16 heads x 16 keys 4.9 and 6.7
//   among others of their kind, x 256 keys 7.8 and 8.7, x 1,024 8.1 and 17.4 (from cold caches the
//   two are closest at 256 keys: 16 heads 13 and 14, 64 heads 16 and 15). A pair of rows is bound by
//   instructions (88 and 70; 156 and 121), and only where the other way needs a split and a join for
//   little work, up to 2^22 key elements that the pairs read, are up to eight rows better off here:
//   4 heads x 2,048 keys 20 and 27.
// fp32 against three planes of every operand, which are written first: 8 x 4 heads x 16,383 keys
//   two rows 109 and 513, four 156 and 574, eight 281 and 640, sixteen 550 and 639; 64 x 16 heads
//   x 64 keys four 101 and 156, eight 187 and 255, sixteen 357 and 261; x 16 keys four 87 and 104,
//   eight 163 and 81.
bool diff_few_supported(const DiffShape& s) {
    if (s.R <= 0 || s.R > 8 || s.nk <= 0) return false;
    if (s.dtype == LLSA_DTYPE_F32) return s.R <= 4 || s.nk >= 64;
    const long long read = (s.R + 1LL) / 2 * s.slices * s.nk;
    return s.R == 1 || (read <= (1 << 22) / s.d && diff_tc_fwd_split(s).splits > 1);
}

// Parts for one block per SM (more, shorter ones cost their beginnings and ends: 6 heads x 65,536
// keys 57 us, 64 with twice as many); a part has at least 128 keys, a few rounds of its warps.
DenseSplit diff_few_split(const DiffShape& s) {
    DenseSplit p;
    long long n = kDenseSms / std::max(1LL, s.slices * ((s.R + 1LL) / 2));
    n = std::max<long long>(1, std::min<long long>(n, s.nk / 128));
    p.chunk = (int)((s.nk + n - 1) / n);
    p.splits = (s.nk + p.chunk - 1) / p.chunk;
    return p;
}

int launch_diff_few(const DiffShape& s, const DiffArgs& a, cudaStream_t st) {
    return s.dtype == LLSA_DTYPE_BF16 ? launch<__nv_bfloat16>(s, a, st) : launch<float>(s, a, st);
}

}  // namespace llsa

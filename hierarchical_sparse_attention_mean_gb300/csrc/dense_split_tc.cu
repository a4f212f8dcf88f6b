// dense_split_tc.cu -- dense attention in fp32 on the tcgen05 tensor cores: forward up
// to 128 columns, backward up to 64 (behind them: dense_split_wide_tc.cu). The
// forward serves bf16 behind 128 columns too, as one plane that is read where it is
// (4 heads x 2,048 tokens, d = 256 34 us, 500 TFLOP/s; 19 x 4,096 390 us, 837; there
// the tensor cores' two products of 64 keys and the softmax between them alternate).
//
// Mathematics. Each fp32 operand x is written as x1 + x2 + x3 with x1 = bf16(x),
// x2 = bf16(x - x1), x3 = bf16(x - x1 - x2): 8 bits and a sign each, so what is
// left of x is at most 2^-26 of it. A product keeps the six terms x1 y1, x1 y2,
// x2 y1, x2 y2, x1 y3, x3 y1; the dropped ones are 2^-25 of it and less, as small
// as fp32's own rounding. Products are exact in fp32 and summed in fp32 in tensor
// memory. Probabilities and dS, computed in fp32 from fp32 scores, are split the
// same way in registers.
//
// Six bf16 products take 6 / 2,250 of the tensor cores' time against 1 / 80 on the
// CUDA cores, whose kernel moreover gets half of that rate (an operand from shared
// memory costs them as much as two of its FMAs). The kernels are bound by the
// tensor cores and the work on the scores between two products: a product of 128 x
// 128 x 64 takes 1,530 clocks, and there is shared memory for one tile of each
// operand. 2 x 8 heads x 1,023 tokens: forward 28 us, backward 95 us with the pass
// before (44 and 115 with a thread per row and the sums' order as it falls; CUDA
// cores 134 and 475).
//
// A pass before writes the three planes of q, k, v (and dout) to the workspace,
// plane by plane, where TMA fetches them as ordinary bf16 tiles of 64 columns
// (zeros behind d), the three planes of a tile in one copy.
#include <algorithm>
#include <type_traits>

#include "dense_split.cuh"

namespace llsa {
namespace {

using namespace tc;

constexpr int kPlane = kTileRows * 128;  // bytes of 128 rows x 64 bf16
constexpr int kTile = 3 * kPlane;
constexpr int BT = kTileRows;

// ----------------------------------------------------------------- planes --

struct PlaneArgs {
    const float* x[4];
    __nv_bfloat16* out[4];  // plane p at out + p * n
    long long n[4];
};

// Eight values per thread, blockIdx.y the tensor. Bound by HBM: 4 bytes in, 6 out (three
// tensors of 2 x 8 x 1,023 x 64 values 6 us of 5).
__global__ void __launch_bounds__(256) dense_planes_kernel(const __grid_constant__ PlaneArgs a) {
    const int t = blockIdx.y;
    const long long n = a.n[t];
    for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (long long)gridDim.x * 2048) {
        float f[8];
        load8(a.x[t] + i, f);
#pragma unroll
        for (int p = 0; p < 3; p++) {
            uint4 u;
            uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                w[c >> 1] = pack_bf16x2(f[c], f[c + 1]);
                f[c] -= __uint_as_float(w[c >> 1] << 16);
                f[c + 1] -= __uint_as_float(w[c >> 1] & 0xffff0000u);
            }
            *reinterpret_cast<uint4*>(a.out[t] + p * n + i) = u;
        }
    }
}

// ---------------------------------------------------------------- forward --

// A block takes 128 query rows against a stream of key and value tiles, of 128 keys
// at 64 columns and 64 keys at 128 columns. S has two buffers, so the next S runs
// beside this one's softmax. Two threads share a row: each reads all of its scores
// for the maximum, then takes half of the weights and half of the output.
// 12 warps of 168 registers at launch = 64,512; at 256 columns the softmax warps take 216
// of them and the others keep 72.
constexpr int kFwdWarps = 8, kFwdThreads = (kFwdWarps + 4) * 32, kFwdRegsSoftmax = 216, kFwdRegsOther = 72;

template <int D, int PL>
struct FwdCfg {
    static constexpr int BN = D == 64 ? 128 : 64, NC = D / 64;
    static constexpr int PQ = BT * D * 2, PK = BN * D * 2, RQ = BT * 128, RK = BN * 128;  // bytes of a plane, of 64 columns of it
    static constexpr int KST = D * PL <= 256 ? 2 : 1;                     // K tiles
    static constexpr int SMEM = PL * (PQ + (KST + 1) * PK) + 1024;
    static constexpr int TM_P = 2 * BN, TM_O = D == 64 ? 448 : 256;       // tensor memory: S at 0 and BN
};

struct FwdBars {
    float l[BT];  // the second half's sum of a row
    uint64_t q_full, k_full[2], k_empty[2], v_full, v_empty, s_full[2], s_free[2], p_full, o_done, drain;
    uint32_t tmem_slot;
    int abort_flag;
};

template <int D, int PL>
__global__ void __launch_bounds__(kFwdThreads, 1)
dense_fwd_split_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                       const __grid_constant__ CUtensorMap mv, const __grid_constant__ DenseArgs a) {
    using C = FwdCfg<D, PL>;
    using T = std::conditional_t<PL == 3, float, __nv_bfloat16>;
    constexpr int BN = C::BN;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *sQ = sm, *sK = sm + PL * C::PQ, *sV = sK + C::KST * PL * C::PK;
    FwdBars* bar = reinterpret_cast<FwdBars*>(sV + PL * C::PK);
    volatile int* abort_flag = &bar->abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(sm) & 1023u) {  // the swizzled layouts need it; the whole block leaves
        if (threadIdx.x == 0) set_status(a.status, LLSA_ERR_TIMEOUT);
        return;
    }
    const DenseWork work = dense_work(a, blockIdx.x, (a.R + BT - 1) / BT);
    const int slice = work.slice, part = work.part;
    const int r0 = (a.causal ? work.blocks - 1 - work.block : work.block) * BT;
    const DenseSpan sp = dense_span(a, slice);
    const int j_first = part * a.chunk;
    const int end = min(dense_tile_kend(a, sp, r0 < a.nq ? r0 : r0 % a.nq, BT), a.splits > 1 ? j_first + a.chunk : a.nk);
    const int n = end > j_first ? (end - j_first + BN - 1) / BN : 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->k_full[i]), 1);
            mbar_init(smem_u32(&bar->k_empty[i]), 1);
            mbar_init(smem_u32(&bar->s_full[i]), 1);
            mbar_init(smem_u32(&bar->s_free[i]), kFwdWarps);
        }
        mbar_init(smem_u32(&bar->q_full), 1);
        mbar_init(smem_u32(&bar->v_full), 1);
        mbar_init(smem_u32(&bar->v_empty), 1);
        mbar_init(smem_u32(&bar->p_full), kFwdWarps);
        mbar_init(smem_u32(&bar->o_done), 1);
        mbar_init(smem_u32(&bar->drain), 1);
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kFwdWarps) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_slot, 0);
    const uint32_t tP = tbase + C::TM_P, tO = tbase + C::TM_O;

    if constexpr (D == 256) {  // half an output row is 128 registers
        if (warp >= kFwdWarps) regs_dec<kFwdRegsOther>();
        else regs_inc<kFwdRegsSoftmax>();
    }
    if (warp > kFwdWarps) {
        // ----------------------------------------------------------- copies
        if (warp <= kFwdWarps + 2 && lane == 0 && n > 0 && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
            const bool keys = warp == kFwdWarps + 1;
            if (keys) load_planes<BT, D, PL>(sQ, &mq, r0, slice, smem_u32(&bar->q_full));
            int t = 0;
            for (; t < n; t++) {
                const int st = keys ? t % C::KST : 0, use = keys ? t / C::KST : t;
                const uint32_t full = smem_u32(keys ? &bar->k_full[st] : &bar->v_full);
                if (use > 0 && !bar_wait(smem_u32(keys ? &bar->k_empty[st] : &bar->v_empty), (use - 1) & 1, abort_flag, a)) break;
                load_planes<BN, D, PL>(keys ? sK + st * PL * C::PK : sV, keys ? &mk : &mv, j_first + t * BN, slice, full);
            }
            // copies still in flight must land before the block exits
            if (keys) land(smem_u32(&bar->q_full), 0);
            if (keys)
                for (int x = max(0, t - C::KST); x < t; x++) land(smem_u32(&bar->k_full[x % C::KST]), (x / C::KST) & 1);
            else if (t > 0)
                land(smem_u32(&bar->v_full), (t - 1) & 1);
        }
    } else if (warp == kFwdWarps) {
        // ------------------------------------------------------- MMA issuer
        const uint32_t leader = elect_lane();
        constexpr uint32_t idS = idesc_bf16(BT, BN, 0, 0), idO = idesc_bf16(BT, D, 0, 1);
        const uint64_t dQ = desc_sw128(smem_u32(sQ), 16, 1024), dK = desc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t dV = desc_sw128(smem_u32(sV), PL * C::RK, 1024);
        auto issue_S = [&](int t) {
            const int b = t & 1, st = t % C::KST;
            if (!warp_wait(smem_u32(&bar->k_full[st]), (t / C::KST) & 1, abort_flag, a)) return false;
            if (t > 1 && !warp_wait(smem_u32(&bar->s_free[b]), ((t >> 1) - 1) & 1, abort_flag, a)) return false;
            tc_fence_after();
            const uint64_t dT = dK + (st * PL * C::PK >> 4);
#pragma unroll
            for (int i = 0; i < kTerms<PL>; i++)
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++)
                    mma_ss(leader, tbase + b * BN, dQ + ((term_a<PL>(i) * C::RQ + (ks / 4) * PL * C::RQ + (ks % 4) * 32) >> 4),
                           dT + ((term_b<PL>(i) * C::RK + (ks / 4) * PL * C::RK + (ks % 4) * 32) >> 4), idS, i > 0 || ks > 0);
            commit(leader, smem_u32(&bar->s_full[b]));
            commit(leader, smem_u32(&bar->k_empty[st]));
            return true;
        };
        bool ok = n > 0 && warp_wait(smem_u32(&bar->q_full), 0, abort_flag, a) && issue_S(0);
        for (int t = 0; t < n && ok; t++) {
            if (t + 1 < n) ok = issue_S(t + 1);
            ok = ok && warp_wait(smem_u32(&bar->p_full), t & 1, abort_flag, a);
            ok = ok && warp_wait(smem_u32(&bar->v_full), t & 1, abort_flag, a);
            if (!ok) break;
            // values behind the last valid key may be anything: their weights are 0, so they must be finite
            const int live = sp.lk - (j_first + t * BN);
            if (live < BN) {
                for (int p = 0; p < PL * C::NC; p++)
                    for (int x = live * 8 + lane; x < BN * 8; x += 32)
                        reinterpret_cast<uint4*>(sV + p * C::RK)[x] = make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
                __syncwarp();
            }
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < kTerms<PL>; i++)
#pragma unroll
                for (int ks = 0; ks < BN / 16; ks++)
                    mma_ts(leader, tO, tP + term_a<PL>(i) * (BN / 2) + ks * 8, dV + ((term_b<PL>(i) * C::RK + ks * 2048) >> 4), idO,
                           i > 0 || ks > 0);
            commit(leader, smem_u32(&bar->o_done));
            commit(leader, smem_u32(&bar->v_empty));
        }
        // no MMA may be in flight when tensor memory is released
        commit(leader, smem_u32(&bar->drain));
        if (lane == 0) land(smem_u32(&bar->drain), 0);
        __syncwarp();
    } else {
        // ------------------------------------------------ softmax, epilogue
        const int lr = (warp & 3) * 32 + lane, half = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int r = r0 + lr;
        int lim = (r < a.R ? dense_kend(a, sp, r < a.nq ? r : r % a.nq) : 0) - j_first;
        const float sl2 = a.scale * kDenseLog2e;
        float m = -INFINITY, l = 0.f, acc[D / 2];  // l: of this half of the keys
#pragma unroll
        for (int i = 0; i < D / 2; i++) acc[i] = 0.f;
        auto take_O = [&](int t) {  // adds the product of tile t to this row's sums
            bar_wait(smem_u32(&bar->o_done), t & 1, abort_flag, a);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < D / 2; c += 32) {
                uint32_t o[32];
                tmem_ld32_nowait(tO + lanes + half * (D / 2) + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i++) acc[c + i] += __uint_as_float(o[i]);
            }
            tc_fence_before();
        };
        for (int t = 0; t < n; t++, lim -= BN) {
            const int b = t & 1;
            const uint32_t tS = tbase + b * BN + lanes;
            bar_wait(smem_u32(&bar->s_full[b]), (t >> 1) & 1, abort_flag, a);
            tc_fence_after();
            const bool cut = __any_sync(0xffffffffu, lim < BN);
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < BN; c += 32) {
                uint32_t s[32];
                tmem_ld32_nowait(tS + c, s);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i++)
                    if (!cut || c + i < lim) top = fmaxf(top, __uint_as_float(s[i]));
            }
            top = fmaxf(m, top * sl2);
            const float f = top > m ? ex2(m - top) : 1.f;  // 2^-inf = 0 at a row's first keys
            m = top;
            l *= f;
            if (t > 0) {  // then the planes of P may be written again
                take_O(t - 1);
#pragma unroll
                for (int i = 0; i < D / 2; i++) acc[i] *= f;
            }
            const float shift = m == -INFINITY ? 0.f : -m;
#pragma unroll
            for (int c0 = 0; c0 < BN / 2; c0 += 32) {
                const int c = half * (BN / 2) + c0;
                uint32_t s[32], p1[16], p2[16], p3[16];
                tmem_ld32_nowait(tS + c, s);
                tmem_wait_ld();
                float sum = 0.f;
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float e[2];
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        e[k] = ex2(fmaf(__uint_as_float(s[i + k]), sl2, shift));
                        if (cut) e[k] = c + i + k < lim ? e[k] : 0.f;
                    }
                    sum += e[0] + e[1];
                    if constexpr (PL == 3) split2(e[0], e[1], p1[i >> 1], p2[i >> 1], p3[i >> 1]);
                    else p1[i >> 1] = pack_bf16x2(e[0], e[1]);
                }
                l += sum;
                tmem_st16(tP + lanes + (c >> 1), p1);
                if constexpr (PL == 3) {
                    tmem_st16(tP + lanes + BN / 2 + (c >> 1), p2);
                    tmem_st16(tP + lanes + BN + (c >> 1), p3);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(smem_u32(&bar->s_free[b]), lane);
            warp_arrive(smem_u32(&bar->p_full), lane);
        }
        if (n > 0) take_O(n - 1);
        if (half == 1) bar->l[lr] = l;
        named_barrier(1, kFwdWarps * 32);
        // both threads of a row need its sum, added in the same order
        if (half == 0) {
            l += bar->l[lr];
            bar->l[lr] = l;
        }
        named_barrier(1, kFwdWarps * 32);
        l = bar->l[lr];
        const long long row = (long long)slice * a.R + r, prow = (long long)part * a.slices * a.R + row;
        const float inv = l == 0.f ? 0.f : a.splits > 1 ? 1.f : 1.f / l;
        if (r < a.R) {
            if (a.splits > 1) store_rowpart<D / 2>(a.part + prow * a.d, acc, inv, half * (D / 2), a.d);
            else store_rowpart<D / 2>(static_cast<T*>(a.o_out) + row * a.d, acc, inv, half * (D / 2), a.d);
            if (half == 0 && a.splits > 1)
                reinterpret_cast<float2*>(a.part + (long long)a.splits * a.slices * a.R * a.d)[prow] = make_float2(m, l);
            else if (half == 0)
                a.lse_out[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kFwdWarps) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// --------------------------------------------------------------- backward --

// As the bf16 kernel, rows and keys in one launch too: 128 stationary rows (X1, X2) =
// (Q, dO) or (K, V) against a stream (Y1, Y2) of the others. Shared memory holds one
// tile of each, so what can overlap is ordered by when a tile comes free: the sums
// over P (keys) free Y2 and those over dS then Y1, whose next tiles come in while
// the tensor cores are at the next product. The elementwise work of an item stays
// in their way. Tensor memory: S at 0 and dP at 128; planes 1 and 2 of dS lie over
// S and those of P over dP, 16 columns over the same 16, so that a warp overwrites
// only what it has read; their planes 3 at 320 and 256, the sums at 384.
constexpr int kBwdWarps = 16, kCols = 32;
// 20 warps of 96 registers at launch = 61,440: the 512 elementwise threads take
// 104 of them, the 128 others keep 64.
constexpr int kBwdThreads = (kBwdWarps + 4) * 32, kRegsElementwise = 104, kRegsOther = 64;
constexpr int kBwdSmem = kTile * 4 + 2 * BT * 4 + 512;

struct BwdBars {
    uint64_t x_full[2], y_full[2], y_empty[2], s_full, dp_full, ds_ready, acc_full, acc_free, drain;
    uint32_t tmem_slot;
    int abort_flag;
};

template <bool KEYS>
__device__ __forceinline__ void bwd_side(const CUtensorMap& mx1, const CUtensorMap& mx2, const CUtensorMap& my1,
                                         const CUtensorMap& my2, const DenseArgs& a, int piece) {
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *sX = sm, *sY = sm + 2 * kTile;
    float* stats = reinterpret_cast<float*>(sm + 4 * kTile);  // KEYS: -l2 and -D of the item's rows
    BwdBars* bar = reinterpret_cast<BwdBars*>(sm + 4 * kTile + 2 * BT * 4);
    volatile int* abort_flag = &bar->abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(sm) & 1023u) {  // the swizzled layouts need it; the whole block leaves
        if (threadIdx.x == 0) set_status(a.status, LLSA_ERR_TIMEOUT);
        return;
    }
    const int extent = KEYS ? a.nk : a.R;
    const DenseWork work = dense_work(a, piece, (extent + BT - 1) / BT);
    const int slice = work.slice, part = work.part;
    const int x0 = (a.causal && !KEYS ? work.blocks - 1 - work.block : work.block) * BT;
    const DenseSpan sp = dense_span(a, slice);
    const int first = a.splits > 1 ? part * a.chunk : 0;
    int stop;
    if constexpr (KEYS) {
        stop = x0 < sp.lk ? (a.splits > 1 ? min(a.R, first + a.chunk) : a.R) : 0;
    } else {
        stop = dense_tile_kend(a, sp, x0 < a.nq ? x0 : x0 % a.nq, BT);
        if (a.splits > 1) stop = min(stop, first + a.chunk);
    }
    Items<KEYS> start(a, sp, x0, first, 0, stop);
    start.start(a);
    const bool any = !start.done();

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->x_full[i]), 1);
            mbar_init(smem_u32(&bar->y_full[i]), 1);
            mbar_init(smem_u32(&bar->y_empty[i]), 1);
        }
        mbar_init(smem_u32(&bar->s_full), 1);
        mbar_init(smem_u32(&bar->dp_full), 1);
        mbar_init(smem_u32(&bar->ds_ready), kBwdWarps);
        mbar_init(smem_u32(&bar->acc_full), 1);
        mbar_init(smem_u32(&bar->acc_free), kBwdWarps);
        mbar_init(smem_u32(&bar->drain), 1);
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kBwdWarps) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_slot, 0);
    const uint32_t tDP = tbase + 128, tP3 = tbase + 256, tS3 = tbase + 320, tAcc = tbase + 384;

    if (warp >= kBwdWarps) {
        regs_dec<kRegsOther>();
        if (warp == kBwdWarps + 1 || warp == kBwdWarps + 2) {
            // ----------------------------------------------------------- copies
            if (lane == 0 && any && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const int k = warp - kBwdWarps - 1;
                load_planes<BT, 64, 3>(sX + k * kTile, k == 0 ? &mx1 : &mx2, x0, slice, smem_u32(&bar->x_full[k]));
                const uint32_t full = smem_u32(&bar->y_full[k]);
                int n = 0;
                for (Items<KEYS> it = start; !it.done(); it.next(a)) {
                    if (n > 0 && !bar_wait(smem_u32(&bar->y_empty[k]), (n - 1) & 1, abort_flag, a)) break;
                    if (KEYS && k == 1) {  // one phase for the tile and the rows' numbers
                        const long long row = (long long)slice * a.Rp + it.pos;
                        load_planes<BT, 64, 3>(sY + kTile, &my2, it.pos, slice, full, 2 * BT * 4);
                        bulk_load(smem_u32(stats), a.nl2 + row, BT * 4, full);
                        bulk_load(smem_u32(stats + BT), a.nd + row, BT * 4, full);
                    } else {
                        load_planes<BT, 64, 3>(sY + k * kTile, k == 0 ? &my1 : &my2, it.pos, slice, full);
                    }
                    n++;
                }
                // copies still in flight must land before the block exits
                land(smem_u32(&bar->x_full[k]), 0);
                if (n > 0) land(full, (n - 1) & 1);
            }
        } else if (warp == kBwdWarps) {
            // ------------------------------------------------------- MMA issuer
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BT, BT, 0, 0), idA = idesc_bf16(BT, 64, 0, 1);
            const uint64_t dX = desc_sw128(smem_u32(sX), 16, 1024), dY = desc_sw128(smem_u32(sY), 16, 1024);
            const uint64_t dM = desc_sw128(smem_u32(sY), kPlane, 1024);  // the streamed tiles read along their rows
            // rows whose P and dS are 0 by the lengths may hold anything: cleared, as they meet those zeros in the sums
            auto clear_rows = [&](unsigned char* tile, const Items<KEYS>& it) {
                if constexpr (KEYS) {
                    if (it.all || it.t0 + BT <= it.sp.lq) return;
                    int t = it.t0 + lane;
                    for (int x = lane; x < BT; x += 32, t += 32)
                        if (t % a.nq >= it.sp.lq)
                            for (int p = 0; p < 3; p++)
                                for (int e = 0; e < 8; e++)
                                    reinterpret_cast<uint4*>(tile + p * kPlane + x * 128)[e] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const int live = it.sp.lk - it.pos;
                    if (live >= BT) return;
                    for (int p = 0; p < 3; p++)
                        for (int x = live * 8 + lane; x < BT * 8; x += 32)
                            reinterpret_cast<uint4*>(tile + p * kPlane)[x] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
            };
            bool ok = any && warp_wait(smem_u32(&bar->x_full[0]), 0, abort_flag, a) &&
                      warp_wait(smem_u32(&bar->x_full[1]), 0, abort_flag, a);
            // S (k 0) or dP (k 1) of item n; what lies over it was used up by sums issued before
            auto issue_tile = [&](const Items<KEYS>& it, int k, int n) {
                if (!warp_wait(smem_u32(&bar->y_full[k]), n & 1, abort_flag, a)) return false;
                if (k == 0 || KEYS) clear_rows(sY + k * kTile, it);  // V only enters dP, which the mask covers
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < 6; i++)
#pragma unroll
                    for (int ks = 0; ks < 4; ks++)
                        mma_ss(leader, tbase + k * 128, dX + ((k * kTile + term_a<3>(i) * kPlane + ks * 32) >> 4),
                               dY + ((k * kTile + term_b<3>(i) * kPlane + ks * 32) >> 4), idS, i > 0 || ks > 0);
                commit(leader, smem_u32(k == 0 ? &bar->s_full : &bar->dp_full));
                if (!KEYS && k == 1) commit(leader, smem_u32(&bar->y_empty[1]));
                return true;
            };
            // acc += (dS or P) (streamed tile k, read along its rows): of every 16 columns at t1 plane 1, then plane 2, 8 words each
            auto issue_sum = [&](uint32_t acc, uint32_t t1, uint32_t t3, int k) {
#pragma unroll
                for (int i = 0; i < 6; i++) {
                    const uint32_t op = term_a<3>(i) == 2 ? t3 : t1 + term_a<3>(i) * 8, step = term_a<3>(i) == 2 ? 8 : 16;
#pragma unroll
                    for (int ks = 0; ks < 8; ks++)
                        mma_ts(leader, acc, op + ks * step, dM + ((k * kTile + term_b<3>(i) * kPlane + ks * 2048) >> 4), idA,
                               i > 0 || ks > 0);
                }
                if (KEYS || k == 0) commit(leader, smem_u32(&bar->y_empty[k]));
            };
            ok = ok && issue_tile(start, 1, 0) && issue_tile(start, 0, 0);
            Items<KEYS> it = start;
            for (int n = 0; ok; n++) {
                ok = warp_wait(smem_u32(&bar->ds_ready), n & 1, abort_flag, a);
                if (ok && n > 0) ok = warp_wait(smem_u32(&bar->acc_free), (n - 1) & 1, abort_flag, a);
                if (!ok) break;
                tc_fence_after();
                if (KEYS) issue_sum(tAcc + 64, tDP, tP3, 1);
                issue_sum(tAcc, tbase, tS3, 0);
                commit(leader, smem_u32(&bar->acc_full));
                it.next(a);
                if (it.done()) break;
                ok = issue_tile(it, 1, n + 1) && issue_tile(it, 0, n + 1);
            }
            // no MMA may be in flight when tensor memory is released
            commit(leader, smem_u32(&bar->drain));
            if (lane == 0) land(smem_u32(&bar->drain), 0);
            __syncwarp();
        }
    } else {
        // ---------------------------------------- elementwise, epilogue
        regs_inc<kRegsElementwise>();
        const int w = warp >> 2, q4 = warp & 3;  // quarter of the columns, of the rows
        const uint32_t lanes = (uint32_t)(q4 * 32) << 16;
        const int x = x0 + q4 * 32 + lane;       // stationary row
        const float sl2 = a.scale * kDenseLog2e;
        float nl2 = 0.f, nd = 0.f;
        int kend = 0;
        if constexpr (!KEYS) {
            nl2 = a.nl2[(long long)slice * a.Rp + x];  // Rp is a multiple of 128
            nd = a.nd[(long long)slice * a.Rp + x];
            kend = x < a.R ? dense_kend(a, sp, x < a.nq ? x : x % a.nq) : 0;
        }
        float acc[KEYS ? 2 : 1][16];  // this row's sums, 16 columns of each
#pragma unroll
        for (int k = 0; k < (KEYS ? 2 : 1); k++)
#pragma unroll
            for (int i = 0; i < 16; i++) acc[k][i] = 0.f;
        auto take_sums = [&](int item) {
            bar_wait(smem_u32(&bar->acc_full), item & 1, abort_flag, a);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < (KEYS ? 2 : 1); k++) {
                float o[16];
                tmem_ld16(tAcc + k * 64 + w * 16 + lanes, o);
#pragma unroll
                for (int i = 0; i < 16; i++) acc[k][i] += o[i];
            }
            tc_fence_before();
            warp_arrive(smem_u32(&bar->acc_free), lane);
        };
        int n = 0;
        for (Items<KEYS> it = start; !it.done(); it.next(a), n++) {
            if (n > 0) take_sums(n - 1);  // while S and dP of this item are made
            bar_wait(smem_u32(&bar->dp_full), n & 1, abort_flag, a);
            if (KEYS) bar_wait(smem_u32(&bar->y_full[1]), n & 1, abort_flag, a);  // the streamed rows' numbers
            bar_wait(smem_u32(&bar->s_full), n & 1, abort_flag, a);
            tc_fence_after();
            const int lim = KEYS ? 0 : kend - it.pos - w * kCols;
            const bool cut = KEYS ? a.causal && (it.t0 + BT > a.nq || dense_kend(a, sp, it.t0) < x0 + BT)
                                  : __any_sync(0xffffffffu, lim < kCols);
            int t = KEYS && cut ? (it.t0 + w * kCols) % a.nq : 0;
#pragma unroll 1  // both at once would spill the sums
            for (int c0 = 0; c0 < kCols; c0 += 16) {
                const uint32_t at = lanes + w * kCols + c0;
                uint32_t s[16], g[16];
                tmem_ld16_nowait(tbase + at, s);
                tmem_ld16_nowait(tDP + at, g);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; c++) {
                    const int col = w * kCols + c0 + c;
                    const float l = KEYS ? stats[col] : nl2, D = KEYS ? stats[BT + col] : nd;
                    float p = ex2(fmaf(__uint_as_float(s[c]), sl2, l));
                    float ds = p * (__uint_as_float(g[c]) + D);
                    if (cut) {
                        const bool out = KEYS ? x > t + sp.lk - sp.lq : c0 + c >= lim;
                        p = out ? 0.f : p;
                        ds = out ? 0.f : ds;
                        if (KEYS && ++t == a.nq) t = 0;
                    }
                    s[c] = __float_as_uint(p);
                    g[c] = __float_as_uint(ds);
                }
#pragma unroll
                for (int k = KEYS ? 0 : 1; k < 2; k++) {  // planes of P, of dS
                    uint32_t p12[16], p3[8];
#pragma unroll
                    for (int c = 0; c < 16; c += 2)
                        split2(__uint_as_float(k == 0 ? s[c] : g[c]), __uint_as_float(k == 0 ? s[c + 1] : g[c + 1]),
                               p12[c >> 1], p12[8 + (c >> 1)], p3[c >> 1]);
                    tmem_st16((k == 0 ? tDP : tbase) + at, p12);
                    tmem_st8((k == 0 ? tP3 : tS3) + lanes + (w * kCols + c0) / 2, p3);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(smem_u32(&bar->ds_ready), lane);
        }
        if (n > 0) take_sums(n - 1);
        // rows without a gradient hold whatever their padding made: zero
        const bool live = any && (KEYS ? x < sp.lk : kend > 0);
        const long long row = (long long)slice * extent + x, all = (long long)a.slices * extent;
#pragma unroll
        for (int k = 0; k < (KEYS ? 2 : 1); k++) {
#pragma unroll
            for (int i = 0; i < 16; i++) acc[k][i] = live ? acc[k][i] : 0.f;
            float* base = a.splits > 1 ? a.part + (k * a.splits + part) * all * a.d
                                       : static_cast<float*>(KEYS ? (k == 0 ? a.dk : a.dv) : a.dq);
            if (x < extent) store_rowpart<16>(base + row * a.d, acc[k], k == 0 ? a.scale : 1.f, w * 16, a.d);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kBwdWarps) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

__global__ void __launch_bounds__(kBwdThreads, 1)
dense_bwd_split_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                       const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                       const __grid_constant__ DenseArgs aq, const __grid_constant__ DenseArgs ak, int key_pieces) {
    const int piece = blockIdx.x;
    if (piece < key_pieces)
        bwd_side<true>(mk, mv, mq, mg, ak, piece);
    else
        bwd_side<false>(mq, mg, mk, mv, aq, piece - key_pieces);
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

// Planes of `n` tensors of sizes q_elems (first `nq` ones) or k_elems, laid out one after the other.
int write_planes(const float* const* x, const long long* elems, int n, void* ws, __nv_bfloat16** planes, cudaStream_t st) {
    PlaneArgs p;
    char* at = static_cast<char*>(ws);
    long long most = 0;
    for (int i = 0; i < 4; i++) {
        p.x[i] = i < n ? x[i] : nullptr;
        p.n[i] = i < n ? elems[i] : 0;
        p.out[i] = reinterpret_cast<__nv_bfloat16*>(at);
        if (i < n) {
            planes[i] = p.out[i];
            at += up((size_t)elems[i] * 6);
            most = std::max(most, elems[i]);
        }
    }
    const dim3 grid((unsigned)std::min<long long>((most + 2047) / 2048, 8LL * kDenseSms), (unsigned)n);
    LLSA_LAUNCH("dense_planes", st, dense_planes_kernel<<<grid, 256, 0, st>>>(p));
    return LLSA_OK;
}

}  // namespace

bool dense_split_supported(const DenseShape& s) {
    return (s.dtype == LLSA_DTYPE_F32 ? s.d <= 128 : s.d > 128) && s.R > 0 && s.nk > 0;
}

DenseSplit dense_split_fwd_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.R + BT - 1) / BT), s.nk, BT, 2);
}
DenseSplit dense_split_dkv_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.nk + BT - 1) / BT), s.R, BT, 2);
}

size_t dense_split_planes(const DenseShape& s, bool backward) {
    if (s.dtype == LLSA_DTYPE_BF16) return 0;  // read as they are
    const size_t q = up((size_t)s.slices * s.R * s.d * 6), k = up((size_t)s.slices * s.nk * s.d * 6);
    return backward ? 2 * q + 2 * k : q + 2 * k;
}

template <int D, int PL>
static int launch_fwd(const DenseShape& s, const DenseArgs& a, const void* const* p, cudaStream_t st) {
    using C = FwdCfg<D, PL>;
    static_assert(C::SMEM <= 227 * 1024 && sizeof(FwdBars) <= 1024, "shared memory budget");
    CUtensorMap mq, mk, mv;
    LLSA_TRY(make_tmap_planes(&mq, p[0], PL, s.slices, s.R, s.d, BT));
    LLSA_TRY(make_tmap_planes(&mk, p[1], PL, s.slices, s.nk, s.d, C::BN));
    LLSA_TRY(make_tmap_planes(&mv, p[2], PL, s.slices, s.nk, s.d, C::BN));
    cudaFuncSetAttribute(dense_fwd_split_kernel<D, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    const long long pieces = (long long)((s.R + BT - 1) / BT) * s.slices * a.splits;
    if (pieces > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("dense_fwd_split", st,
                dense_fwd_split_kernel<D, PL><<<(unsigned)pieces, kFwdThreads, C::SMEM, st>>>(mq, mk, mv, a));
    return LLSA_OK;
}

int launch_dense_split_fwd(const DenseShape& s, const DenseArgs& a, void* ws, cudaStream_t st) {
    if (s.dtype == LLSA_DTYPE_BF16) {
        const void* const x[3] = {a.q, a.k, a.v};
        return launch_fwd<256, 1>(s, a, x, st);
    }
    const float* x[3] = {static_cast<const float*>(a.q), static_cast<const float*>(a.k), static_cast<const float*>(a.v)};
    const long long nq = (long long)s.slices * s.R * s.d, nk = (long long)s.slices * s.nk * s.d;
    const long long elems[3] = {nq, nk, nk};
    __nv_bfloat16* p[3];
    LLSA_TRY(write_planes(x, elems, 3, ws, p, st));
    const void* const y[3] = {p[0], p[1], p[2]};
    return s.d <= 64 ? launch_fwd<64, 3>(s, a, y, st) : launch_fwd<128, 3>(s, a, y, st);
}

int make_dense_split_planes(const DenseShape& s, const DenseArgs& a, void* ws, void** planes, cudaStream_t st) {
    if (s.dtype == LLSA_DTYPE_BF16) {
        const void* const x[4] = {a.q, a.dout, a.k, a.v};
        for (int i = 0; i < 4; i++) planes[i] = const_cast<void*>(x[i]);
        return LLSA_OK;
    }
    const float* x[4] = {static_cast<const float*>(a.q), static_cast<const float*>(a.dout), static_cast<const float*>(a.k),
                         static_cast<const float*>(a.v)};
    const long long nq = (long long)s.slices * s.R * s.d, nk = (long long)s.slices * s.nk * s.d;
    const long long elems[4] = {nq, nq, nk, nk};
    __nv_bfloat16* p[4];
    LLSA_TRY(write_planes(x, elems, 4, ws, p, st));
    for (int i = 0; i < 4; i++) planes[i] = p[i];
    return LLSA_OK;
}

int launch_dense_split_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, void* const* planes,
                           cudaStream_t st) {
    if (s.d > 64) return launch_dense_split_wide_bwd(s, aq, ak, planes, st);
    CUtensorMap mq, mg, mk, mv;
    LLSA_TRY(make_tmap_planes(&mq, planes[0], 3, s.slices, s.R, s.d, BT));
    LLSA_TRY(make_tmap_planes(&mg, planes[1], 3, s.slices, s.R, s.d, BT));
    LLSA_TRY(make_tmap_planes(&mk, planes[2], 3, s.slices, s.nk, s.d, BT));
    LLSA_TRY(make_tmap_planes(&mv, planes[3], 3, s.slices, s.nk, s.d, BT));
    static_assert(kBwdSmem <= 227 * 1024 && sizeof(BwdBars) <= 512, "shared memory budget");
    cudaFuncSetAttribute(dense_bwd_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBwdSmem);
    const long long pq = (long long)((s.R + BT - 1) / BT) * s.slices * aq.splits;
    const long long pk = (long long)((s.nk + BT - 1) / BT) * s.slices * ak.splits;
    if (pq + pk > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("dense_bwd_split", st,
                dense_bwd_split_kernel<<<(unsigned)(pq + pk), kBwdThreads, kBwdSmem, st>>>(mq, mg, mk, mv, aq, ak, (int)pk));
    return LLSA_OK;
}

}  // namespace llsa

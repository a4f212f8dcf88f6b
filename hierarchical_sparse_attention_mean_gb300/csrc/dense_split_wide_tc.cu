// dense_split_wide_tc.cu -- dense attention backward on the tcgen05 tensor cores for
// fp32 at 64 < d <= 128, operands as three bf16 planes and six products per term as
// at d <= 64, and for bf16 at 128 < d <= 256, one plane.
//
// Three kinds of blocks own 128 rows each and stream tiles of 64 rows of the other
// side: dq (X1, X2, Y1, Y2 = Q, dO, K, V) and dk (K, V, Q, dO), which are the same
// pass, and dv (K, -, Q, dO), which needs no dP. dk and dv apart cost S a second
// time; together their sums would be 256 columns per row, half of the registers.
//
// The three planes of X1 and X2 would fill 192 KB, so one buffer A holds them in turn: an
// even item makes S, then dP, and right behind it the next item's dP, for which
// there is a second buffer; the odd item then only wants S. A changes once per item,
// mostly while the threads or the sums are at work. Y1 and Y2 take 48 KB each. Sums
// stay in tensor memory for one item and are carried in registers.
//
// Bound by the chain of an item, about 10,000 clocks: a product of 128 x 64 x 128 is
// 2,285 (S, dP) and 1,536 (sums), and Y1 comes in between the sums and the next S. 4
// heads x 2,048 tokens, d = 128: 268 us (80 TFLOP/s of the 10 d operations per
// pair; CUDA cores 1,065 us). One plane: X1 and X2 lie side by side and the sums stay
// in tensor memory; the same at d = 256 in bf16 141 us (304 TFLOP/s; CUDA cores 3,292
// us), 19 x 4,096 tokens 1,880 us (434).
//
// Roles: warps 0-15 elementwise and epilogue, 16 issues the MMAs, 17 copies A, 18 and
// 19 copy Y1 and Y2. Tensor memory: S at 0, dP at 64 and 160, planes 1 and 2 of dS (dv:
// P) over S, 16 columns over the same 16, plane 3 at 128, the sums at 256.
#include <algorithm>
#include <type_traits>

#include "dense_split.cuh"

namespace llsa {
namespace {

using namespace tc;

constexpr int BT = kTileRows, SN = 64;                   // stationary rows, streamed rows
constexpr int kRegionX = BT * 128, kRegionY = SN * 128;  // bytes of 64 columns of a plane
constexpr int kWarps = 16, kCols = SN / 4;
// 20 warps of 96 registers at launch = 61,440: the 512 elementwise threads take
// 104 of them, the 128 others keep 64.
constexpr int kThreads = (kWarps + 4) * 32, kRegsElementwise = 104, kRegsOther = 64;

// PL planes of D columns: fp32 up to 128 columns in three, bf16 up to 256 in one. One
// plane leaves room for X1 and X2 side by side, and their sums stay in tensor memory.
template <int D, int PL>
struct Cfg {
    static constexpr bool BOTH = PL == 1;
    static constexpr int X = PL * BT * D * 2, Y = PL * SN * D * 2;  // bytes of a tile
    static constexpr int SMEM = (BOTH ? 2 : 1) * X + 2 * Y + 2 * SN * 4 + 512;
};

enum Kind { kDq, kDk, kDv };

__device__ __forceinline__ uint32_t dp_column(int item) { return item & 1 ? 160 : 64; }

struct Bars {
    uint64_t a_full, a_empty, y_full[2], y_empty[2], s_full, dp_full[2], ds_ready, acc_full, acc_free, drain;
    uint32_t tmem_slot;
    int abort_flag;
};

template <Kind KIND, int D, int PL>
__device__ __forceinline__ void wide_side(const CUtensorMap& mx1, const CUtensorMap& mx2, const CUtensorMap& my1,
                                          const CUtensorMap& my2, const DenseArgs& a, int piece) {
    using C = Cfg<D, PL>;
    using T = std::conditional_t<PL == 3, float, __nv_bfloat16>;
    constexpr bool KEYS = KIND != kDq, WITH_DP = KIND != kDv, BOTH = C::BOTH;
    using List = Items<KEYS, SN>;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char *sA = sm, *sY = sm + (BOTH ? 2 : 1) * C::X;
    float* stats = reinterpret_cast<float*>(sY + 2 * C::Y);  // KEYS: -l2 and -D of the item's rows
    Bars* bar = reinterpret_cast<Bars*>(sY + 2 * C::Y + 2 * SN * 4);
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
    List start(a, sp, x0, first, 0, stop);
    start.start(a);
    const bool any = !start.done();

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar->a_full), BOTH && WITH_DP ? 2 : 1);
        mbar_init(smem_u32(&bar->a_empty), 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->y_full[i]), 1);
            mbar_init(smem_u32(&bar->y_empty[i]), 1);
            mbar_init(smem_u32(&bar->dp_full[i]), 1);
        }
        mbar_init(smem_u32(&bar->s_full), 1);
        mbar_init(smem_u32(&bar->ds_ready), kWarps);
        mbar_init(smem_u32(&bar->acc_full), 1);
        mbar_init(smem_u32(&bar->acc_free), kWarps);
        mbar_init(smem_u32(&bar->drain), 1);
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarps) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    tc_fence_before();
    close_wait();
    __syncthreads();
    tc_fence_after();
    close_ahead();  // the block has its tensor memory
    const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_slot, 0);
    const uint32_t t3 = tbase + 128, tAcc = tbase + 256;

    if (warp >= kWarps) {
        regs_dec<kRegsOther>();
        if (warp == kWarps + 1) {
            // ------------------------------------------------------ copies of A
            // X1 and X2 in turn, the next one behind the first product of every item
            if (lane == 0 && any && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const uint32_t full = smem_u32(&bar->a_full);
                const int qk = dense_qk_slice(a, slice), second = KEYS ? dense_v_slice(a, slice) : slice;  // of v or dout
                load_planes<BT, D, PL>(sA, &mx1, x0, qk, full);
                if (BOTH && WITH_DP) load_planes<BT, D, PL>(sA + C::X, &mx2, x0, second, full);
                int n = 0;
                if (WITH_DP && !BOTH)
                    for (List it = start; !it.done(); it.next(a)) {
                        if (!bar_wait(smem_u32(&bar->a_empty), n & 1, abort_flag, a)) break;
                        load_planes<BT, D, PL>(sA, n % 2 == 0 ? &mx2 : &mx1, x0, n % 2 == 0 ? second : qk, full);
                        n++;
                    }
                land(full, n & 1);  // copies still in flight must land before the block exits
            }
        } else if (warp > kWarps + 1) {
            // ------------------------------------------- copies of Y1, of Y2
            if (lane == 0 && any && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const int k = warp - kWarps - 2;
                const uint32_t full = smem_u32(&bar->y_full[k]);
                const int at = k == 0 ? dense_qk_slice(a, slice) : KEYS ? slice : dense_v_slice(a, slice);
                int n = 0;
                for (List it = start; !it.done(); it.next(a)) {
                    if (n > 0 && !bar_wait(smem_u32(&bar->y_empty[k]), (n - 1) & 1, abort_flag, a)) break;
                    if (KEYS && k == 0) {  // one phase for the tile and the rows' numbers
                        const long long row = (long long)slice * a.Rp + it.pos;
                        load_planes<SN, D, PL>(sY, &my1, it.pos, at, full, 2 * SN * 4);
                        bulk_load(smem_u32(stats), a.nl2 + row, SN * 4, full);
                        bulk_load(smem_u32(stats + SN), a.nd + row, SN * 4, full);
                    } else {
                        load_planes<SN, D, PL>(sY + k * C::Y, k == 0 ? &my1 : &my2, it.pos, at, full);
                    }
                    n++;
                }
                if (n > 0) land(full, (n - 1) & 1);
            }
        } else {
            // ------------------------------------------------------- MMA issuer
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BT, SN, 0, 0), idA = idesc_bf16(BT, D, 0, 1);
            const uint64_t dA = desc_sw128(smem_u32(sA), 16, 1024), dY = desc_sw128(smem_u32(sY), 16, 1024);
            const uint64_t dM = desc_sw128(smem_u32(sY), PL * kRegionY, 1024);  // the streamed tiles read along their rows
            // rows whose P and dS are 0 by the lengths may hold anything: cleared, as they meet those zeros in the sums
            auto clear_rows = [&](unsigned char* tile, const List& it) {
                if constexpr (KEYS) {
                    if (it.all || it.t0 + SN <= it.sp.lq) return;
                    int t = it.t0 + lane;
                    for (int x = lane; x < SN; x += 32, t += 32)
                        if (t % a.nq >= it.sp.lq)
                            for (int r = 0; r < PL * D / 64; r++)
                                for (int e = 0; e < 8; e++)
                                    reinterpret_cast<uint4*>(tile + r * kRegionY + x * 128)[e] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const int live = it.sp.lk - it.pos;
                    if (live >= SN) return;
                    for (int r = 0; r < PL * D / 64; r++)
                        for (int x = live * 8 + lane; x < SN * 8; x += 32)
                            reinterpret_cast<uint4*>(tile + r * kRegionY)[x] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
            };
            auto take_y = [&](const List& it, int k, int n) {
                if (!warp_wait(smem_u32(&bar->y_full[k]), n & 1, abort_flag, a)) return false;
                if (KEYS || k == 0) clear_rows(sY + k * C::Y, it);  // V only enters dP, which the mask covers
                return true;
            };
            // S (k 0) or dP (k 1) of item n, of what A holds now
            auto issue_tile = [&](const List& it, int k, int n) {
                if (!take_y(it, k, n)) return false;
                tc_fence_after();
#pragma unroll
                for (int i = 0; i < kTerms<PL>; i++)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ks++)
                        mma_ss(leader, tbase + (k == 0 ? 0 : dp_column(n)), dA + (((BOTH ? k * C::X : 0) + term_a<PL>(i) * kRegionX + (ks / 4) * PL * kRegionX + (ks % 4) * 32) >> 4),
                               dY + ((k * C::Y + term_b<PL>(i) * kRegionY + (ks / 4) * PL * kRegionY + (ks % 4) * 32) >> 4), idS,
                               i > 0 || ks > 0);
                commit(leader, smem_u32(k == 0 ? &bar->s_full : &bar->dp_full[n & 1]));
                if (k == 1) commit(leader, smem_u32(&bar->y_empty[1]));
                return true;
            };
            // sums = (dS or P) (streamed tile k, read along its rows)
            auto issue_sum = [&](int k, bool fresh) {
#pragma unroll
                for (int i = 0; i < kTerms<PL>; i++) {
                    const uint32_t op = term_a<PL>(i) == 2 ? t3 : tbase + term_a<PL>(i) * 8, step = term_a<PL>(i) == 2 ? 8 : 16;
#pragma unroll
                    for (int ks = 0; ks < SN / 16; ks++)
                        mma_ts(leader, tAcc, op + ks * step, dM + ((k * C::Y + term_b<PL>(i) * kRegionY + ks * 2048) >> 4), idA,
                               !fresh || i > 0 || ks > 0);
                }
                commit(leader, smem_u32(&bar->y_empty[0]));
                if (k == 1) commit(leader, smem_u32(&bar->y_empty[1]));
                if (!BOTH) commit(leader, smem_u32(&bar->acc_full));
            };
            bool ok = any && warp_wait(smem_u32(&bar->a_full), 0, abort_flag, a);
            int n = 0;
            for (List it = start; ok && !it.done(); it.next(a), n++) {
                if (!WITH_DP) {
                    ok = issue_tile(it, 0, n) && take_y(it, 1, n);
                } else if (BOTH) {
                    ok = issue_tile(it, 0, n) && issue_tile(it, 1, n);
                } else if (n & 1) {  // its dP is made
                    ok = warp_wait(smem_u32(&bar->a_full), (n + 1) & 1, abort_flag, a) && issue_tile(it, 0, n);
                } else {
                    ok = issue_tile(it, 0, n);
                    if (!ok) break;
                    commit(leader, smem_u32(&bar->a_empty));
                    ok = warp_wait(smem_u32(&bar->a_full), (n + 1) & 1, abort_flag, a) && issue_tile(it, 1, n);
                    List next = it;
                    next.next(a);
                    if (ok && !next.done()) {
                        ok = issue_tile(next, 1, n + 1);
                        if (ok) commit(leader, smem_u32(&bar->a_empty));
                    }
                }
                ok = ok && warp_wait(smem_u32(&bar->ds_ready), n & 1, abort_flag, a);
                if (!BOTH && ok && n > 0) ok = warp_wait(smem_u32(&bar->acc_free), (n - 1) & 1, abort_flag, a);
                if (!ok) break;
                tc_fence_after();
                issue_sum(WITH_DP ? 0 : 1, !BOTH || n == 0);
            }
            if (BOTH && any && ok) commit(leader, smem_u32(&bar->acc_full));
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
        float acc[32];  // !BOTH: this row's sums of 32 columns
#pragma unroll
        for (int i = 0; i < 32; i++) acc[i] = 0.f;
        auto take_sums = [&](int item) {
            bar_wait(smem_u32(&bar->acc_full), item & 1, abort_flag, a);
            tc_fence_after();
            uint32_t o[32];
            tmem_ld32_nowait(tAcc + w * 32 + lanes, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i++) acc[i] += __uint_as_float(o[i]);
            tc_fence_before();
            warp_arrive(smem_u32(&bar->acc_free), lane);
        };
        int n = 0;
        for (List it = start; !it.done(); it.next(a), n++) {
            if (!BOTH && n > 0) take_sums(n - 1);  // while S and dP of this item are made
            if (KEYS) bar_wait(smem_u32(&bar->y_full[0]), n & 1, abort_flag, a);  // the streamed rows' numbers
            bar_wait(smem_u32(&bar->s_full), n & 1, abort_flag, a);
            if (WITH_DP) bar_wait(smem_u32(&bar->dp_full[n & 1]), (n >> 1) & 1, abort_flag, a);
            tc_fence_after();
            const int lim = KEYS ? 0 : kend - it.pos - w * kCols;
            const bool cut = KEYS ? a.causal && (it.t0 + SN > a.nq || dense_kend(a, sp, it.t0) < x0 + BT)
                                  : __any_sync(0xffffffffu, lim < kCols);
            int t = KEYS && cut ? (it.t0 + w * kCols) % a.nq : 0;
            const uint32_t at = lanes + w * kCols;
            uint32_t s[16], g[16], p12[16], p3[8];
            tmem_ld16_nowait(tbase + at, s);
            if (WITH_DP) tmem_ld16_nowait(tbase + dp_column(n) + at, g);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; c++) {
                const int col = w * kCols + c;
                float p = ex2(fmaf(__uint_as_float(s[c]), sl2, KEYS ? stats[col] : nl2));
                if (WITH_DP) p *= __uint_as_float(g[c]) + (KEYS ? stats[SN + col] : nd);
                if (cut) {
                    p = (KEYS ? x > t + sp.lk - sp.lq : c >= lim) ? 0.f : p;
                    if (KEYS && ++t == a.nq) t = 0;
                }
                s[c] = __float_as_uint(p);
            }
            if constexpr (PL == 3) {
#pragma unroll
                for (int c = 0; c < 16; c += 2)
                    split2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]), p12[c >> 1], p12[8 + (c >> 1)], p3[c >> 1]);
                tmem_st16(tbase + at, p12);
                tmem_st8(t3 + lanes + w * kCols / 2, p3);
            } else {
#pragma unroll
                for (int c = 0; c < 16; c += 2) p3[c >> 1] = pack_bf16x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                tmem_st8(tbase + at, p3);
            }
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(smem_u32(&bar->ds_ready), lane);
        }
        // rows without a gradient hold whatever their padding made: zero
        const bool live = any && (KEYS ? x < sp.lk : kend > 0);
        const long long row = (long long)slice * extent + x, all = (long long)a.slices * extent;
        float* part_row = a.part + (((KIND == kDv ? a.splits : 0) + part) * all + row) * a.d;
        T* out_row = static_cast<T*>(KIND == kDq ? a.dq : KIND == kDk ? a.dk : a.dv) + row * a.d;
        if (!BOTH && n > 0) take_sums(n - 1);
        if (BOTH && n > 0) {
            bar_wait(smem_u32(&bar->acc_full), 0, abort_flag, a);
            tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < D / 4; c += 32) {  // this warp's columns
            if (BOTH && n > 0) {
                uint32_t o[32];
                tmem_ld32_nowait(tAcc + w * (D / 4) + c + lanes, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i++) acc[i] = __uint_as_float(o[i]);
            }
#pragma unroll
            for (int i = 0; i < 32; i++) acc[i] = live ? acc[i] : 0.f;
            const float f = KIND == kDv ? 1.f : a.scale;
            if (x < extent) {
                if (a.splits > 1) store_rowpart<32>(part_row, acc, f, w * (D / 4) + c, a.d);
                else store_rowpart<32>(out_row, acc, f, w * (D / 4) + c, a.d);
            }
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarps) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Tensor maps: of 128 rows for A, of 64 for the streamed tiles.
struct Maps {
    CUtensorMap q, g, k, v;
};

template <int D, int PL>
__global__ void __launch_bounds__(kThreads, 1)
dense_bwd_wide_kernel(const __grid_constant__ Maps x, const __grid_constant__ Maps y, const __grid_constant__ DenseArgs aq,
                      const __grid_constant__ DenseArgs ak, int key_pieces) {
    const int piece = blockIdx.x;
    if (piece < key_pieces)
        wide_side<kDk, D, PL>(x.k, x.v, y.q, y.g, ak, piece);
    else if (piece < 2 * key_pieces)
        wide_side<kDv, D, PL>(x.k, x.k, y.q, y.g, ak, piece - key_pieces);
    else
        wide_side<kDq, D, PL>(x.q, x.g, y.k, y.v, aq, piece - 2 * key_pieces);
}

template <int D, int PL>
int launch(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, void* const* planes, cudaStream_t st) {
    using C = Cfg<D, PL>;
    Maps x, y;
    for (int i = 0; i < 2; i++) {
        Maps& m = i == 0 ? x : y;
        const int rows = i == 0 ? BT : SN;
        LLSA_TRY(make_tmap_planes(&m.q, planes[0], PL, dense_plane_slices(aq), s.R, s.d, rows));
        LLSA_TRY(make_tmap_planes(&m.g, planes[1], PL, s.slices, s.R, s.d, rows));
        LLSA_TRY(make_tmap_planes(&m.k, planes[2], PL, dense_plane_slices(aq), s.nk, s.d, rows));
        LLSA_TRY(make_tmap_planes(&m.v, planes[3], PL, dense_plane_slices(aq), s.nk, s.d, rows));
    }
    static_assert(C::SMEM <= 227 * 1024 && sizeof(Bars) <= 512, "shared memory budget");
    cudaFuncSetAttribute(dense_bwd_wide_kernel<D, PL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    const long long pq = (long long)((s.R + BT - 1) / BT) * s.slices * aq.splits;
    const long long pk = (long long)((s.nk + BT - 1) / BT) * s.slices * ak.splits;
    if (pq + 2 * pk > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("dense_bwd_split", st, launch_close(aq.four, dense_bwd_wide_kernel<D, PL>, dim3((unsigned)(pq + 2 * pk)), kThreads,
                                                    C::SMEM, st, x, y, aq, ak, (int)pk));
    return LLSA_OK;
}

}  // namespace

int launch_dense_split_wide_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, void* const* planes,
                                cudaStream_t st) {
    return s.dtype == LLSA_DTYPE_BF16 ? launch<256, 1>(s, aq, ak, planes, st) : launch<128, 3>(s, aq, ak, planes, st);
}

}  // namespace llsa

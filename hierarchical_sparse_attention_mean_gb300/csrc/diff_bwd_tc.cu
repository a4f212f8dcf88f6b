// diff_bwd_tc.cu -- differential attention backward on the tcgen05 tensor cores (bf16, up
// to 64 columns of q and k, 128 of v; TMA fills the rest of the tiles with zeros).
//
// Mathematics, with l2_i = lse_i log2(e), D_1 = dout . o + lam dout . o2 and D_2 = dout . o2
// of every query row from the pass before: P_i = 2^(scale log2(e) q_i.k_i - l2_i),
// dP = dout.v, which both maps share, and
//   rows:  dq_1 = scale sum P_1 (dP - D_1) k_1, dq_2 = -lam scale sum P_2 (dP - D_2) k_2,
//          by blocks that own 128 query rows,
//   keys:  dk_1, dk_2 the same sums over rows, dv = sum (P_1 - lam P_2) dout, by blocks
//          that own 128 keys.
// One product with dout makes dv of both maps. P_1 - lam P_2 and dS are rounded to bf16,
// the type that these products have beside bf16 inputs; statistics, D and sums stay in
// fp32. dlam is summed from P_2 dP in fp32 as the rows go by: from o2, which is rounded, it
// would be 2^-8 of its terms off. Every sum has one owner and a fixed order.
//
// Per 128 x 128 pairs the tensor cores take 1,536 clocks for rows and 2,048 for keys, 28 d
// operations per pair where the 20 d of the mathematics would need dq added up across
// blocks in memory in whatever order they run.
//
// Tensor memory is full and decides the order of the work. Rows: S_1, S_2, dP (128
// columns each) and both dq; dS_i lies over S_i, and the maps take turns, so that one's
// products run beside the other's exponentials. Keys: one place for S_1 and S_2 after
// each other, over which P_1 - lam P_2 is written, dP, over which both dS are, and
// the sums of dv, dk_1, dk_2. The tensor cores run dv, the next S_1, dk_1, the next S_2,
// dk_2, the next dP; the exponentials fall beside dk and dP, dS beside dv.
//
// For keys, the numbers that go with a column (l2, D and lam of its row) come from shared
// memory, which the products of two shared-memory operands keep busy by themselves. There
// the threads read tensor memory as fragments, 8 columns of 4 rows each, and need a
// quarter as many of those numbers as with a row of 32 columns each.
//
// Bound by the chain of a tile: products, exponentials, dS and the moves between tensor memory and
// registers wait for each other, 2,925 clocks per tile pair for rows and 3,785 for keys, where the
// counters have neither the issue slots (39 %) nor the tensor cores (42 %) full.
// 6 heads x 16,384 tokens: 2,150 us (1,342 TFLOP/s of the 28 d), the rows' numbers 31 before that.
// Eight warps of 64 columns took 2,225; two teams of eight warps, a map each, 2,649; a ring of
// single map tiles 2,387; S and dP loaded together 2,244.
//
// All sixteen elementwise warps take a tile together, a thread per row and quarter of the
// columns. Shared memory holds one set of stationary tiles, and every piece of work gets a
// block of its own.
//
// Roles: warps 0-15 elementwise and epilogue, warp 16 issues the MMAs, warps 18 and 19 the
// copies of the two streams.
#include <algorithm>

#include "dense_tc.cuh"
#include "diff.h"

namespace llsa {
namespace {

using namespace tc;

constexpr int kWarps = 16, kCols = 32;  // elementwise warps: a thread takes one row and kCols columns of a tile
// 20 warps of 96 registers at launch = 61,440: the 512 elementwise threads take 112 of
// them, of which 60 bytes a thread spill, and the 128 others keep 32.
constexpr int kThreads = (kWarps + 4) * 32, kRegsElementwise = 112, kRegsOther = 32;
constexpr int BT = kTileRows, D = 64;
constexpr int REGION = BT * 128;   // bytes of 128 rows x 64 columns
constexpr int PAIR = 2 * REGION;   // both maps' tiles of q or k, or a tile of v or dout
constexpr int kStats = kDiffStats;
constexpr int STATS = kStats * BT * 4;

template <bool KEYS>
struct Cfg {
    static constexpr int N1 = KEYS ? 2 : 3, N2 = 2;  // stages of the two streams
    static constexpr int SMEM = (2 + N1 + N2) * PAIR + (KEYS ? N1 * STATS : 0) + 1024;
    static constexpr int TM_DP = KEYS ? 128 : 256, TM_ACC = KEYS ? 256 : 384;  // S of map i at 128 i (rows), at 0 (keys)
};

struct Bars {
    uint64_t x_full, y1_full[3], y1_empty[3], y2_full[2], y2_empty[2];
    uint64_t s_full[2], s_read, dp_full, ready[2], acc_full, drain;
    uint32_t tmem_slot;
    int abort_flag, last;
};

// Piece `id`: 128 stationary rows of a slice against a part of the stream.
template <bool KEYS>
__device__ __forceinline__ void bwd_side(const CUtensorMap& mqk, const CUtensorMap& mgv, const CUtensorMap& syqk,
                                         const CUtensorMap& sygv, const CUtensorMap& zqk, const CUtensorMap& zv, const DiffArgs& f,
                                         int id) {
    using C = Cfg<KEYS>;
    const DenseArgs& a = f.d;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* sX = sm;                    // both maps' q or k, then dout or v
    unsigned char* ring1 = sm + 2 * PAIR;      // both maps' k or q
    unsigned char* ring2 = ring1 + C::N1 * PAIR;  // v or dout
    float* stats = reinterpret_cast<float*>(ring2 + C::N2 * PAIR);
    Bars* bar = reinterpret_cast<Bars*>(ring2 + C::N2 * PAIR + (KEYS ? C::N1 * STATS : 0));
    volatile int* abort_flag = &bar->abort_flag;
    // broadcast, so that the compiler knows these as the same in a whole warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(sm) & 1023u) {  // the swizzled layouts need it; the whole block leaves
        if (threadIdx.x == 0) set_status(a.status, LLSA_ERR_TIMEOUT);
        return;
    }
    const int extent = KEYS ? a.nk : a.R;
    const DenseWork work = dense_work(a, id, (extent + BT - 1) / BT);
    const int slice = work.slice, part = work.part;
    // causal order: the last rows see the most keys, the first keys the most rows; those come first
    const int x0 = (a.causal && !KEYS ? work.blocks - 1 - work.block : work.block) * BT;
    const DenseSpan sp = dense_span(a, slice);
    int pos = a.splits > 1 ? part * a.chunk : 0, stop;
    if constexpr (KEYS) {
        stop = x0 < sp.lk ? (a.splits > 1 ? min(a.R, pos + a.chunk) : a.R) : 0;
    } else {
        stop = dense_tile_kend(a, sp, x0 < a.nq ? x0 : x0 % a.nq, BT);
        if (a.splits > 1) stop = min(stop, pos + a.chunk);
    }
    Items<KEYS> first(a, sp, x0, pos, 0, stop);
    first.start(a);
    const bool any = !first.done();

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar->x_full), 1);
        for (int i = 0; i < 3; i++) {
            mbar_init(smem_u32(&bar->y1_full[i]), 1);
            mbar_init(smem_u32(&bar->y1_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->y2_full[i]), 1);
            mbar_init(smem_u32(&bar->y2_empty[i]), 1);
            mbar_init(smem_u32(&bar->s_full[i]), 1);
            mbar_init(smem_u32(&bar->ready[i]), kWarps);
        }
        mbar_init(smem_u32(&bar->s_read), kWarps);
        mbar_init(smem_u32(&bar->dp_full), 1);
        mbar_init(smem_u32(&bar->acc_full), 1);
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
    const int m0 = diff_matrix(a, slice, 0), m1 = m0 + a.kv_heads;

    if (warp >= kWarps) {
        regs_dec<kRegsOther>();
        if (warp >= kWarps + 2) {
            // ----------------------------------------------------------- copies
            if (lane == 0 && any && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const bool one = warp == kWarps + 2;  // the stream of q or k
                const int ns = one ? C::N1 : C::N2;
                unsigned char* ring = one ? ring1 : ring2;
                uint64_t* full = one ? bar->y1_full : bar->y2_full;
                uint64_t* empty = one ? bar->y1_empty : bar->y2_empty;
                const uint32_t fx = smem_u32(&bar->x_full);
                if (one) {
                    mbar_arrive_expect_tx(fx, 2 * PAIR);
                    tma_load_3d(smem_u32(sX), &mqk, 0, x0, m0, fx);
                    tma_load_3d(smem_u32(sX + REGION), &mqk, 0, x0, m1, fx);
                    tma_load_3d(smem_u32(sX + PAIR), &mgv, 0, x0, slice, fx);
                    tma_load_3d(smem_u32(sX + PAIR + REGION), &mgv, 64, x0, slice, fx);
                }
                int st = 0, n = 0;
                uint32_t parity = 1;  // of the release that the stage's next use waits for
                for (Items<KEYS> it = first; !it.done(); it.next(a)) {
                    if (n >= ns && !bar_wait(smem_u32(&empty[st]), parity, abort_flag, a)) break;
                    const uint32_t fb = smem_u32(&full[st]);
                    const bool with_stats = KEYS && one;
                    mbar_arrive_expect_tx(fb, PAIR + (with_stats ? STATS : 0));
                    unsigned char* to = ring + st * PAIR;
                    tma_load_3d(smem_u32(to), one ? &syqk : &sygv, 0, it.pos, one ? m0 : slice, fb);
                    tma_load_3d(smem_u32(to + REGION), one ? &syqk : &sygv, one ? 0 : 64, it.pos, one ? m1 : slice, fb);
                    if (with_stats)
                        for (int i = 0; i < kStats; i++)  // the five arrays lie one after the other
                            bulk_load(smem_u32(stats + (st * kStats + i) * BT), a.nl2 + ((long long)i * a.slices + slice) * a.Rp + it.pos,
                                      BT * 4, fb);
                    n++;
                    if (++st == ns) {
                        st = 0;
                        parity ^= 1;
                    }
                }
                // copies still in flight must land before the block exits
                if (one) land(fx, 0);
                for (int x = max(0, n - ns); x < n; x++) land(smem_u32(&full[x % ns]), (x / ns) & 1);
            }
        } else if (warp == kWarps) {
            // ------------------------------------------------------ MMA issuer
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BT, BT, 0, 0);                         // S and dP
            constexpr uint32_t idA = idesc_bf16(BT, 64, 0, 1), idV = idesc_bf16(BT, 128, 0, 1);  // dq, dk; dv
            const uint64_t dX = desc_sw128(smem_u32(sX), 16, 1024);
            const uint64_t dY1 = desc_sw128(smem_u32(ring1), 16, 1024), dY2 = desc_sw128(smem_u32(ring2), 16, 1024);
            const uint64_t dM1 = desc_sw128(smem_u32(ring1), REGION, 1024);  // the tiles read along their rows
            const uint64_t dM2 = desc_sw128(smem_u32(ring2), REGION, 1024);
            // Rows of the streamed tiles whose P and dS are 0 by the mask of the lengths may
            // hold anything: they meet those zeros in the sums, so they are cleared.
            auto clear_rows = [&](unsigned char* tile, const Items<KEYS>& it) {
                if constexpr (KEYS) {
                    if (it.all || it.t0 + BT <= it.sp.lq) return;
                    int t = it.t0 + lane;
                    for (int x = lane; x < BT; x += 32, t += 32)
                        if (t % a.nq >= it.sp.lq)
                            for (int c = 0; c < 2; c++)
                                for (int e = 0; e < 8; e++)
                                    reinterpret_cast<uint4*>(tile + c * REGION + x * 128)[e] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const int live = it.sp.lk - it.pos;
                    if (live >= BT) return;
                    for (int c = 0; c < 2; c++)
                        for (int x = live * 8 + lane; x < BT * 8; x += 32)
                            reinterpret_cast<uint4*>(tile + c * REGION)[x] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
            };
            Stage<C::N1> s1, t1;  // stages of the next S and of the next sums
            Stage<C::N2> s2, t2;  // of the next dP and of the next sums
            auto issue_S = [&](int i) {  // of the tile in stage s1
                tc_fence_after();
                const uint64_t dA = dX + (i * REGION >> 4), dB = dY1 + ((s1.st * PAIR + i * REGION) >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ks++)
                    mma_ss(leader, tbase + (KEYS ? 0 : 128 * i), dA + (ks * 32 >> 4), dB + (ks * 32 >> 4), idS, ks > 0);
                commit(leader, smem_u32(&bar->s_full[i]));
            };
            auto take_1 = [&](const Items<KEYS>& it) {  // the tile in stage s1 is there
                if (!warp_wait(smem_u32(&bar->y1_full[s1.st]), s1.parity, abort_flag, a)) return false;
                clear_rows(ring1 + s1.st * PAIR, it);
                return true;
            };
            auto issue_dP = [&](const Items<KEYS>& it) {
                if (!warp_wait(smem_u32(&bar->y2_full[s2.st]), s2.parity, abort_flag, a)) return false;
                if (KEYS) clear_rows(ring2 + s2.st * PAIR, it);  // v only enters dP, which the mask covers
                tc_fence_after();
                const uint64_t dA = dX + (PAIR >> 4), dB = dY2 + (s2.st * PAIR >> 4);
#pragma unroll
                for (int ks = 0; ks < 8; ks++) {
                    const uint32_t off = (ks / 4) * REGION + (ks % 4) * 32;
                    mma_ss(leader, tbase + C::TM_DP, dA + (off >> 4), dB + (off >> 4), idS, ks > 0);
                }
                commit(leader, smem_u32(&bar->dp_full));
                if (!KEYS) commit(leader, smem_u32(&bar->y2_empty[s2.st]));
                s2.next();
                return true;
            };
            // acc += A B with A in tensor memory, 8 words per 16 rows of B, `step` columns apart
            auto issue_sum = [&](uint32_t acc, uint32_t op, uint32_t step, uint64_t dB, uint32_t id, bool fresh) {
#pragma unroll
                for (int ks = 0; ks < 8; ks++)
                    mma_ts(leader, tbase + acc, tbase + op + (step == 16 ? (ks / 2) * 32 + (ks % 2) * 8 : ks * 16), dB + (ks * 2048 >> 4), id,
                           !fresh || ks > 0);
            };
            bool ok = any && warp_wait(smem_u32(&bar->x_full), 0, abort_flag, a);
            if (ok) {
                Items<KEYS> it = first;
                uint32_t n = 0;  // tiles whose sums are issued
                ok = take_1(it);
                if (ok) issue_S(0);
                if (KEYS) ok = ok && warp_wait(smem_u32(&bar->s_read), 0, abort_flag, a);
                if (ok) issue_S(1);
                s1.next();
                ok = ok && issue_dP(it);
                it.next(a);
                for (bool fresh = true; ok; fresh = false, n++) {
                    const bool more = !it.done();
                    const uint64_t dT1 = dM1 + (t1.st * PAIR >> 4), dT2 = dM2 + (t2.st * PAIR >> 4);
                    ok = warp_wait(smem_u32(&bar->ready[0]), n & 1, abort_flag, a);
                    if (!ok) break;
                    tc_fence_after();
                    if constexpr (KEYS) {
                        issue_sum(C::TM_ACC, 0, 16, dT2, idV, fresh);  // dv
                        commit(leader, smem_u32(&bar->y2_empty[t2.st]));
                    } else {
                        issue_sum(C::TM_ACC, 0, 16, dT1, idA, fresh);  // dq_1
                    }
                    if (more) {
                        ok = take_1(it);
                        if (!ok) break;
                        issue_S(0);
                    }
                    ok = warp_wait(smem_u32(&bar->ready[1]), n & 1, abort_flag, a);
                    if (!ok) break;
                    tc_fence_after();
                    if constexpr (KEYS) {
                        issue_sum(C::TM_ACC + 128, C::TM_DP, 8, dT1, idA, fresh);                          // dk_1
                        if (more) {
                            ok = warp_wait(smem_u32(&bar->s_read), (n + 1) & 1, abort_flag, a);
                            if (!ok) break;
                            issue_S(1);
                        }
                        issue_sum(C::TM_ACC + 192, C::TM_DP + 8, 8, dT1 + (REGION >> 4), idA, fresh);      // dk_2
                        commit(leader, smem_u32(&bar->y1_empty[t1.st]));
                        if (more) ok = issue_dP(it);
                    } else {
                        if (more) ok = issue_dP(it);
                        issue_sum(C::TM_ACC + 64, 128, 16, dT1 + (REGION >> 4), idA, fresh);               // dq_2
                        commit(leader, smem_u32(&bar->y1_empty[t1.st]));
                        if (ok && more) issue_S(1);
                    }
                    t1.next();
                    t2.next();
                    if (!more) break;
                    s1.next();
                    it.next(a);
                }
                if (ok) commit(leader, smem_u32(&bar->acc_full));
            }
            // no MMA may be in flight when tensor memory is released
            commit(leader, smem_u32(&bar->drain));
            if (lane == 0) land(smem_u32(&bar->drain), 0);
            __syncwarp();
        }
    } else {
        // ---------------------------------------- elementwise, epilogue
        regs_inc<kRegsElementwise>();
        const int w = warp >> 2;  // quarter of the columns
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int lr = (warp & 3) * 32 + lane;  // row of the tile
        const float sl2 = a.scale * kDenseLog2e;
        const uint64_t sl2x2 = pack2(sl2, sl2);
        const int x = x0 + lr;  // stationary row
        const uint32_t tS = tbase + lanes + w * kCols, tG = tbase + C::TM_DP + lanes + w * kCols;
        uint32_t n = 0;
        float lam = 0.f, d2 = 0.f;  // rows: d2 the sum of P_2 dP
        int kend = 0;
        if constexpr (!KEYS) {
            float nl[2], nd[2];
            const long long row = (long long)slice * a.Rp + x, all = (long long)a.slices * a.Rp;  // Rp is a multiple of 128
#pragma unroll
            for (int i = 0; i < 2; i++) {
                nl[i] = a.nl2[i * all + row];
                nd[i] = a.nl2[(2 + i) * all + row];
            }
            lam = a.nl2[4 * all + row];
            kend = x < a.R ? dense_kend(a, sp, x < a.nq ? x : x % a.nq) : 0;
            uint64_t sum2 = 0ull;
            for (Items<KEYS> it = first; !it.done(); it.next(a), n++) {
                const int lim = kend - it.pos - w * kCols;
                const bool masked = __any_sync(0xffffffffu, kend - it.pos < BT);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint64_t nl2x2 = pack2(nl[i], nl[i]), ndx2 = pack2(nd[i], nd[i]);
                    bar_wait(smem_u32(&bar->s_full[i]), n & 1, abort_flag, a);
                    tc_fence_after();
                    uint32_t s[kCols], g[kCols];
                    tmem_ld32_nowait(tS + 128 * i, s);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) {
                        float e0, e1;
                        unpack2(fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2x2, nl2x2), e0, e1);
                        s[c] = __float_as_uint(ex2(e0));
                        s[c + 1] = __float_as_uint(ex2(e1));
                    }
                    if (i == 0) {
                        bar_wait(smem_u32(&bar->dp_full), n & 1, abort_flag, a);
                        tc_fence_after();
                    }
                    tmem_ld32_nowait(tG, g);
                    tmem_wait_ld();
                    if (masked) {  // S and dP of a key behind the lengths may be anything
#pragma unroll
                        for (int c = 0; c < kCols; c++) {
                            s[c] = c < lim ? s[c] : 0u;
                            g[c] = c < lim ? g[c] : 0u;
                        }
                    }
                    uint32_t o[kCols / 2];
#pragma unroll
                    for (int c = 0; c < kCols; c += 2) {
                        const uint64_t p2 = pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                        const uint64_t g2 = pack2(__uint_as_float(g[c]), __uint_as_float(g[c + 1]));
                        if (i == 1) sum2 = fma2(p2, g2, sum2);
                        float e0, e1;
                        unpack2(mul2(add2(g2, ndx2), p2), e0, e1);
                        o[c >> 1] = pack_bf16x2(e0, e1);
                    }
                    tmem_st16(tS + 128 * i, o);
                    tmem_wait_st();
                    tc_fence_before();
                    warp_arrive(smem_u32(&bar->ready[i]), lane);
                }
            }
            float u0, u1;
            unpack2(sum2, u0, u1);
            d2 = u0 + u1;
            // the sums of this part's keys, a quarter of the columns each
            if (x < a.Rp) f.d2[((long long)(part * 4 + w) * a.slices + slice) * a.Rp + x] = kend > 0 ? d2 : 0.f;
        } else {
            Stage<C::N1> s1;
            const int fr = (warp & 3) * 32 + (lane >> 2), fc = 2 * (lane & 3);  // first row and column of the fragments
            const uint32_t low = 16u << 16;                                    // the second 16 lanes
            for (Items<KEYS> it = first; !it.done(); it.next(a), n++) {
                // of these columns' rows; registers 16 h + 4 i + 2 e + k: column fc + 8 i + k, row fr + 16 h + 8 e
                const float* st = stats + s1.st * kStats * BT + w * kCols + fc;
                bar_wait(smem_u32(&bar->y1_full[s1.st]), s1.parity, abort_flag, a);
                uint32_t p[kCols], s[kCols];
                auto pair = [](const uint32_t* v) { return pack2(__uint_as_float(v[0]), __uint_as_float(v[1])); };
                auto put = [](uint32_t* v, uint64_t x) {
                    float e0, e1;
                    unpack2(x, e0, e1);
                    v[0] = __float_as_uint(e0);
                    v[1] = __float_as_uint(e1);
                };
                auto weights = [&](uint32_t* v, int i) {
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const uint64_t l = *reinterpret_cast<const uint64_t*>(st + i * BT + 2 * c);
#pragma unroll
                        for (int x = c; x < 32; x += (x & 2) ? 14 : 2) {
                            float e0, e1;
                            unpack2(fma2(pair(v + x), sl2x2, l), e0, e1);
                            v[x] = __float_as_uint(ex2(e0));
                            v[x + 1] = __float_as_uint(ex2(e1));
                        }
                    }
                };
                bar_wait(smem_u32(&bar->s_full[0]), n & 1, abort_flag, a);
                tc_fence_after();
                tmem_ld_frag(tS, p);
                tmem_ld_frag(tS + low, p + 16);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->s_read), lane);
                weights(p, 0);
                bar_wait(smem_u32(&bar->s_full[1]), n & 1, abort_flag, a);
                tc_fence_after();
                tmem_ld_frag(tS, s);
                tmem_ld_frag(tS + low, s + 16);
                tmem_wait_ld();
                weights(s, 1);
                // the lengths are in l2; causal order cuts where a row's keys end inside the block's keys
                if (a.causal && (it.t0 + BT > a.nq || dense_kend(a, sp, it.t0) < x0 + BT)) {
#pragma unroll
                    for (int c = 0; c < 16; c += 4)
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            const int last = (it.t0 + w * kCols + fc + 2 * c + k) % a.nq + sp.lk - sp.lq;  // key that this column's row sees last
#pragma unroll
                            for (int x = 0; x < 4; x++)
                                if (x0 + fr + 8 * x > last) p[16 * (x >> 1) + c + 2 * (x & 1) + k] = s[16 * (x >> 1) + c + 2 * (x & 1) + k] = 0u;
                        }
                }
                uint32_t o[kCols / 2];
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const uint64_t lam2 = *reinterpret_cast<const uint64_t*>(st + 4 * BT + 2 * c);
#pragma unroll
                    for (int x = c; x < 32; x += (x & 2) ? 14 : 2) {
                        put(s + x, mul2(pair(s + x), lam2));
                        o[x >> 1] = pack_bf16x2(__uint_as_float(p[x]) - __uint_as_float(s[x]), __uint_as_float(p[x + 1]) - __uint_as_float(s[x + 1]));
                    }
                }
                tmem_st_frag16(tS, o);
                tmem_st_frag16(tS + low, o + 8);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->ready[0]), lane);
                bar_wait(smem_u32(&bar->dp_full), n & 1, abort_flag, a);
                tc_fence_after();
                uint32_t o2[kCols / 2];
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    uint32_t g[16];
                    tmem_ld_frag(tG + h * low, g);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < 16; c += 4) {
                        const uint64_t d1 = *reinterpret_cast<const uint64_t*>(st + 2 * BT + 2 * c);
                        const uint64_t d2x = *reinterpret_cast<const uint64_t*>(st + 3 * BT + 2 * c);
#pragma unroll
                        for (int x = c; x < c + 4; x += 2) {
                            float e0, e1;
                            unpack2(mul2(add2(pair(g + x), d1), pair(p + 16 * h + x)), e0, e1);
                            o[8 * h + (x >> 1)] = pack_bf16x2(e0, e1);
                            unpack2(mul2(add2(pair(g + x), d2x), pair(s + 16 * h + x)), e0, e1);
                            o2[8 * h + (x >> 1)] = pack_bf16x2(e0, e1);
                        }
                    }
                    // 8 words of each dS where their 16 columns of dP were
                    tmem_st_frag8(tG + h * low, o + 8 * h);
                    tmem_st_frag8(tG + h * low + 8, o2 + 8 * h);
                    tmem_st_frag8(tG + h * low + 16, o + 8 * h + 4);
                    tmem_st_frag8(tG + h * low + 24, o2 + 8 * h + 4);
                }
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->ready[1]), lane);
                s1.next();
            }
        }
        // rows without a gradient hold whatever their padding made: zero
        const bool live = any && (KEYS ? x < sp.lk : kend > 0);
        if (any) {
            bar_wait(smem_u32(&bar->acc_full), 0, abort_flag, a);
            tc_fence_after();
        }
        const long long all2 = 2LL * a.slices * extent;  // rows of dq or dk
#pragma unroll
        for (int k = 0; k < (KEYS ? 4 : 2); k++) {
            // regions of 64 columns: dq_1, dq_2, or the two halves of dv, dk_1, dk_2
            const bool v = KEYS && k < 2;
            const int i = KEYS ? k - 2 : k;  // map
            const float scale = v ? 1.f : i == 0 ? a.scale : KEYS ? -a.scale : -lam * a.scale;
            const int c = w * 16;
            float o[16];
            if (any) tmem_ld16(tbase + C::TM_ACC + k * 64 + c + lanes, o);
#pragma unroll
            for (int e = 0; e < 16; e++) o[e] = live ? o[e] * scale : 0.f;
            const int cols = v ? 2 * a.d : a.d, col = v ? k * 64 + c : c;
            const long long row = (long long)(v ? slice : i == 0 ? m0 : m1) * extent + x;
            if (a.splits > 1) {
                // parts: dq; or dk of all parts, then dv of all parts
                float* dst = v ? a.part + a.splits * all2 * a.d + (part * (all2 / 2) + row) * cols
                               : a.part + (part * all2 + row) * cols;
                if (x < extent) diff_store16(dst + col, o, col, cols);
            } else if (any) {
                // the stationary tiles have been used up: their place takes the results
                unsigned char* out = sX + (v ? PAIR + k * REGION : i * REGION);
                put_chunk(out, lr, w * 2, o);
                put_chunk(out, lr, w * 2 + 1, o + 8);
            } else if (x < extent) {
                diff_store16(static_cast<__nv_bfloat16*>(v ? a.dv : KEYS ? a.dk : a.dq) + row * cols + col, o, col, cols);
            }
        }
        if (any && a.splits == 1) {
            fence_async_smem();
            named_barrier(1 + (warp & 3), 128);  // the four warps of these 32 rows
            if (w == 0 && lane == 0 && x < extent) {
                tma_store_3d(&zqk, smem_u32(sX + lr * 128), 0, x, m0);
                tma_store_3d(&zqk, smem_u32(sX + REGION + lr * 128), 0, x, m1);
                if (KEYS) {
                    tma_store_3d(&zv, smem_u32(sX + PAIR + lr * 128), 0, x, slice);
                    if (a.d > 32) tma_store_3d(&zv, smem_u32(sX + PAIR + REGION + lr * 128), 64, x, slice);
                }
                bulk_commit();
                bulk_wait_read();
            }
        }
        if constexpr (!KEYS) diff_lam_last(f, &bar->last);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarps) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
diff_bwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                   const __grid_constant__ CUtensorMap zq, const __grid_constant__ CUtensorMap zk,
                   const __grid_constant__ CUtensorMap zv, const __grid_constant__ DiffArgs aq,
                   const __grid_constant__ DiffArgs ak, int row_pieces, int key_pieces, int keys_first) {
    // longer pieces first
    const int piece = blockIdx.x < (keys_first ? 0 : row_pieces) ? blockIdx.x + key_pieces
                      : blockIdx.x - (keys_first ? 0 : row_pieces);
    if (piece < key_pieces)
        bwd_side<true>(mk, mv, mq, mg, zk, zv, ak, piece);
    else
        bwd_side<false>(mq, mg, mk, mv, zq, zq, aq, piece - key_pieces);
}

}  // namespace

// When the last of `first` pieces of `a` clocks and then `others` of `b` < a ends, one at a time on
// every SM.
static long long pieces_end(long long first, long long a, long long others, long long b) {
    const long long sms = kDenseSms, rounds = first / sms, left = first % sms;
    const long long even = (left * a + others * b + sms - 1) / sms;  // no sooner than this
    long long end = -1;
    for (int i = 0; i < 2; i++)
        for (const long long from : {0LL, a}) {
            const long long t = from + (std::max(0LL, even - from) + b - 1) / b * b + i * b;
            const bool all = (left == 0 || t >= a) && (sms - left) * (t / b) + left * (std::max(0LL, t - a) / b) >= others;
            if (all && (end < 0 || t < end)) end = t;
        }
    return rounds * a + std::max(end, even);
}

// Into how many parts the pieces of rows go along the keys and those of keys along the rows: what
// ends first by a count of clocks, in tenths of what a tile of a rows' piece takes. A tile of a
// keys' piece takes 13, a piece's beginning and end three tiles, joining parts 30 and what they
// write and read; a few long pieces beside many short ones, which copy more, take twice as long. Longer pieces go first. One query, 6 heads x 8,192 keys: 41 us, 53 with as many
// parts of either kind as SMs; 2 x 3 heads x 700 x 1,500, d = 96: 44 and 57.
void diff_tc_bwd_splits(const DiffShape& s, DenseSplit* rows, DenseSplit* keys) {
    constexpr int kParts[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
    const long long r = (s.R + BT - 1) / BT, k = (s.nk + BT - 1) / BT;
    // behind 64 columns a row or key block is several pieces of work
    const long long row_pieces = s.slices * r * (s.d > D ? 2 : 1), key_pieces = s.slices * k * (s.d > D ? 3 : 1);
    const long long row_join = (long long)s.slices * s.R * s.d / 65536, key_join = (long long)s.slices * s.nk * s.d / 32768;
    int best_r = 1, best_k = 1;
    long long best = 0;
    for (int nr : kParts) {
        if (nr > 1 && nr * 2 > k) break;
        for (int nk : kParts) {
            if (nk > 1 && nk * 2 > r) break;
            const long long lr = 10 * ((k + nr - 1) / nr + 3), lk = 13 * ((r + nk - 1) / nk + 3);
            const long long cr = row_pieces * nr, ck = key_pieces * nk, first = lr > lk ? cr : ck, b = std::min(lr, lk);
            long long a = std::max(lr, lk);
            if (first <= kDenseSms / 2 && b < a / 3) a *= 2;
            long long t = pieces_end(first, a, lr > lk ? ck : cr, b);
            if (nr > 1 || nk > 1) t += 30 + (nr > 1 ? nr * row_join : 0) + (nk > 1 ? nk * key_join : 0);
            if (best == 0 || t < best) {
                best = t;
                best_r = nr;
                best_k = nk;
            }
        }
    }
    rows->chunk = (int)((k + best_r - 1) / best_r) * BT;
    rows->splits = (s.nk + rows->chunk - 1) / rows->chunk;
    keys->chunk = (int)((r + best_k - 1) / best_k) * BT;
    keys->splits = (s.R + keys->chunk - 1) / keys->chunk;
}

int launch_diff_tc_bwd(const DiffShape& s, const DiffArgs& aq, const DiffArgs& ak, cudaStream_t st) {
    if (s.d > D) return launch_diff_tc_bwd_wide(s, aq, ak, st);
    constexpr int smem = Cfg<true>::SMEM > Cfg<false>::SMEM ? Cfg<true>::SMEM : Cfg<false>::SMEM;
    static_assert(smem <= 227 * 1024 && sizeof(Bars) <= 1024, "shared memory budget");
    const DenseArgs& a = aq.d;
    CUtensorMap mq, mk, mv, mg, zq, zk, zv;
    LLSA_TRY(make_tmap_rows(&mq, a.q, 2LL * s.slices, s.R, s.d, BT));
    LLSA_TRY(make_tmap_rows(&mg, a.dout, s.slices, s.R, 2 * s.d, BT));
    LLSA_TRY(make_tmap_rows(&mk, a.k, 2LL * s.slices, s.nk, s.d, BT));
    LLSA_TRY(make_tmap_rows(&mv, a.v, s.slices, s.nk, 2 * s.d, BT));
    LLSA_TRY(make_tmap_rows(&zq, a.dq, 2LL * s.slices, s.R, s.d, 32));
    LLSA_TRY(make_tmap_rows(&zk, a.dk, 2LL * s.slices, s.nk, s.d, 32));
    LLSA_TRY(make_tmap_rows(&zv, a.dv, s.slices, s.nk, 2 * s.d, 32));
    cudaFuncSetAttribute(diff_bwd_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const long long pq = (long long)((s.R + BT - 1) / BT) * s.slices * a.splits;
    const long long pk = (long long)((s.nk + BT - 1) / BT) * s.slices * ak.d.splits;
    if (pq + pk > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("diff_bwd_tc", st, launch_close(true, diff_bwd_tc_kernel, dim3((unsigned)(pq + pk)), kThreads, smem, st, mq, mg, mk, mv, zq,
                                                zk, zv, aq, ak, (int)pq, (int)pk, (int)(std::min(ak.d.chunk, s.R) >= std::min(a.chunk, s.nk))));
    return LLSA_OK;
}

}  // namespace llsa

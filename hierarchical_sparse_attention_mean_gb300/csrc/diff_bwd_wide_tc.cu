// diff_bwd_wide_tc.cu -- differential attention backward on the tcgen05 tensor cores for 64 <
// d <= 128 (bf16, 128 < 2 d <= 256 columns of v; TMA fills the rest of the tiles with zeros).
//
// Mathematics as in diff_bwd_tc.cu. The sums of dv, dk_1 and dk_2 together would be all of
// tensor memory, so a piece of work owns one of them:
//   dq_i: 128 query rows of a map, S = Q_i K_i^T, dP = dO V^T, dq_i += dS K_i,
//   dk_i: 128 keys of a map, S = K_i Q_i^T, dP = V dO^T, dk_i += dS Q_i,
//   dv:   128 keys, S of both maps, dv += (P_1 - lam P_2) dO.
// Scores are made three times per map and dP four times: 40 d operations per pair of a
// query and a key, where 20 d are needed and the four dense calls that this replaces took 56 d.
// P_1 - lam P_2 and dS are rounded to bf16, the type that these products have beside bf16
// inputs; statistics, D and sums stay in fp32, and dlam is summed from P_2 dP in fp32.
// Every sum has one owner and a fixed order.
//
// dq and dk are one code: 128 stationary rows (X1, X2) against a stream (Y1, Y2) of 128
// rows a tile, X2 and Y2 of 256 columns and Y2 fetched in halves. S is free as soon as it is
// read and dP has two buffers, so the tensor cores, 2,048 clocks per 128 x 128 pairs, run the
// next tile's S and dP while the threads make this one's dS, which is written over dP.
// dv: P_1 - lam P_2 is written over S_2, S_1 of the next tile is made meanwhile; 2,048
// clocks too.
//
// Bound by the chain of a tile, 2,700 clocks for dq, 3,200 for dk, 4,100 for dv, which copies 128
// KB a tile. 19 heads x 16,384 tokens of 128 columns: this kernel 16.6 ms (1,570 TFLOP/s of the
// 40 d), the call 17.0; 8 heads over 2, 4,095 tokens in causal order 285 us by itself, 306 in the
// call. Stream tiles of 64 rows took 1.2 times as long, as more, smaller copies and products do.
//
// Roles: warps 0-15 elementwise and epilogue (a thread per row and quarter of the columns),
// warps 16 and 17 issue the MMAs, warps 18 and 19 the copies of the two streams. Every piece
// gets a block of its own.
#include <algorithm>

#include "dense_tc.cuh"
#include "diff.h"

namespace llsa {
namespace {

using namespace tc;

constexpr int kWarps = 16, kCols = 32;
// 20 warps of 96 registers at launch = 61,440: the 512 elementwise threads take 104 of
// them, the 128 others keep 64.
constexpr int kThreads = (kWarps + 4) * 32, kRegsElementwise = 104, kRegsOther = 64;
constexpr int BT = kTileRows;
constexpr int REGION = BT * 128;  // bytes of 128 rows x 64 columns
constexpr int HALF = 2 * REGION;  // of 128 columns

enum Kind { kDq = 0, kDk = 1, kDv = 2 };

template <Kind KIND>
struct Cfg {
    static constexpr int NX = KIND == kDv ? 2 : 3;   // HALVES of stationary tiles: X1, X2 of two; or both maps' keys
    static constexpr int N1 = KIND == kDv ? 3 : 2, N2 = 2;
    static constexpr int NS = KIND == kDq ? 0 : 2;   // stages of the rows' numbers, two of 128 each
    static constexpr int SMEM = (NX + N1 + N2) * HALF + NS * 2 * BT * 4 + 1024;
    static constexpr int TM_DP = 128, TM_ACC = KIND == kDv ? 256 : 384;
};

struct Bars {
    uint64_t x_full, y1_full[3], y1_empty[3], y2_full[2], y2_empty[2], st_full[2], st_empty[2];
    uint64_t s_full[2], s_free, dp_full[2], ready[2], dp_free[2], acc_full, drain[2];
    uint32_t tmem_slot;
    int abort_flag, last;
};

struct Maps {
    const CUtensorMap &q, &g, &k, &v, &zq, &zk, &zv;
};

template <Kind KIND>
__device__ __forceinline__ void bwd_piece(const Maps& maps, const DiffArgs& f, int id) {
    using C = Cfg<KIND>;
    constexpr bool KEYS = KIND != kDq;
    const DenseArgs& a = f.d;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* sX = sm;
    unsigned char* ring1 = sm + C::NX * HALF;
    unsigned char* ring2 = ring1 + C::N1 * HALF;
    float* stats = reinterpret_cast<float*>(ring2 + C::N2 * HALF);
    Bars* bar = reinterpret_cast<Bars*>(ring2 + C::N2 * HALF + C::NS * 2 * BT * 4);
    volatile int* abort_flag = &bar->abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(sm) & 1023u) {  // the swizzled layouts need it; the whole block leaves
        if (threadIdx.x == 0) set_status(a.status, LLSA_ERR_TIMEOUT);
        return;
    }
    const int extent = KEYS ? a.nk : a.R;
    const int map = KIND == kDv ? 0 : id & 1;
    const DenseWork work = dense_work(a, KIND == kDv ? id : id >> 1, (extent + BT - 1) / BT);
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
    const int m0 = diff_matrix(a, slice, map);  // matrix of q and k (kDv: of the first map)

    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&bar->x_full), 1);
        for (int i = 0; i < 3; i++) {
            mbar_init(smem_u32(&bar->y1_full[i]), 1);
            mbar_init(smem_u32(&bar->y1_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->y2_full[i]), 1);
            mbar_init(smem_u32(&bar->y2_empty[i]), 1);
            mbar_init(smem_u32(&bar->st_full[i]), 1);
            mbar_init(smem_u32(&bar->st_empty[i]), kWarps);
            mbar_init(smem_u32(&bar->s_full[i]), 1);
            mbar_init(smem_u32(&bar->dp_full[i]), 1);
            mbar_init(smem_u32(&bar->ready[i]), kWarps);
            mbar_init(smem_u32(&bar->dp_free[i]), 1);
            mbar_init(smem_u32(&bar->drain[i]), 1);
        }
        mbar_init(smem_u32(&bar->s_free), kWarps);
        mbar_init(smem_u32(&bar->acc_full), 1);
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

    if (warp >= kWarps) {
        regs_dec<kRegsOther>();
        if (warp >= kWarps + 2) {
            // ----------------------------------------------------------- copies
            // Stream 1: tiles of q or k of 128 columns (kDv: both maps' in turn), and the
            // rows' numbers. Stream 2: halves of v or dout.
            if (lane == 0 && any && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const bool one = warp == kWarps + 2;
                const int ns = one ? C::N1 : C::N2;
                unsigned char* ring = one ? ring1 : ring2;
                uint64_t* full = one ? bar->y1_full : bar->y2_full;
                uint64_t* empty = one ? bar->y1_empty : bar->y2_empty;
                const CUtensorMap* map1 = KEYS ? &maps.q : &maps.k;
                const CUtensorMap* map2 = KEYS ? &maps.g : &maps.v;
                const CUtensorMap* own1 = KEYS ? &maps.k : &maps.q;
                const CUtensorMap* own2 = KEYS ? &maps.v : &maps.g;
                const uint32_t fx = smem_u32(&bar->x_full);
                if (one) {
                    mbar_arrive_expect_tx(fx, C::NX * HALF);
                    for (int c = 0; c < 2; c++) tma_load_3d(smem_u32(sX + c * REGION), own1, c * 64, x0, m0, fx);
                    if constexpr (KIND == kDv) {
                        for (int c = 0; c < 2; c++)
                            tma_load_3d(smem_u32(sX + HALF + c * REGION), own1, c * 64, x0, m0 + a.kv_heads, fx);
                    } else {
                        for (int c = 0; c < 4; c++) tma_load_3d(smem_u32(sX + HALF + c * REGION), own2, c * 64, x0, slice, fx);
                    }
                }
                int st = 0, n = 0, items = 0;
                uint32_t parity = 1;  // of the release that the stage's next use waits for
                bool ok = true;
                for (Items<KEYS> it = first; ok && !it.done(); it.next(a), items++) {
                    if (KEYS && one) {
                        const int k = items & 1;
                        if (items >= 2) ok = bar_wait(smem_u32(&bar->st_empty[k]), (items / 2 - 1) & 1, abort_flag, a);
                        if (!ok) break;
                        const uint32_t fs = smem_u32(&bar->st_full[k]);
                        mbar_arrive_expect_tx(fs, 2 * BT * 4);
                        const long long all = (long long)a.slices * a.Rp, row = (long long)slice * a.Rp + it.pos;
                        // -lse log2(e) of the map and its -D, or -lse log2(e) of both maps
                        bulk_load(smem_u32(stats + k * 2 * BT), a.nl2 + (KIND == kDv ? 0 : map) * all + row, BT * 4, fs);
                        bulk_load(smem_u32(stats + k * 2 * BT + BT), a.nl2 + (KIND == kDv ? 1 : 2 + map) * all + row, BT * 4, fs);
                    }
                    const int tiles = one ? (KIND == kDv ? 2 : 1) : 2;
                    for (int t = 0; t < tiles; t++) {
                        if (n >= ns) ok = bar_wait(smem_u32(&empty[st]), parity, abort_flag, a);
                        if (!ok) break;
                        const uint32_t fb = smem_u32(&full[st]);
                        mbar_arrive_expect_tx(fb, HALF);
                        for (int c = 0; c < 2; c++)
                            tma_load_3d(smem_u32(ring + st * HALF + c * REGION), one ? map1 : map2, (one ? 0 : t * 128) + c * 64, it.pos,
                                        one ? m0 + t * a.kv_heads : slice, fb);
                        n++;
                        if (++st == ns) {
                            st = 0;
                            parity ^= 1;
                        }
                    }
                }
                // copies still in flight must land before the block exits
                if (one) land(fx, 0);
                if (KEYS && one)
                    for (int x = max(0, items - 2); x < items; x++) land(smem_u32(&bar->st_full[x & 1]), (x / 2) & 1);
                for (int x = max(0, n - ns); x < n; x++) land(smem_u32(&full[x % ns]), (x / ns) & 1);
            }
        } else {
            // ----------------------------------------------------- MMA issuers
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BT, BT, 0, 0), idA = idesc_bf16(BT, 128, 0, 1);
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
            // acc (+)= A B^T over 128 columns
            auto mma_half = [&](uint32_t acc, uint64_t dA, uint64_t dB, bool fresh) {
#pragma unroll
                for (int ks = 0; ks < 8; ks++) {
                    const uint32_t off = (ks / 4) * REGION + (ks % 4) * 32;
                    mma_ss(leader, tbase + acc, dA + (off >> 4), dB + (off >> 4), idS, !fresh || ks > 0);
                }
            };
            // acc += A B with A in tensor memory, 16 words of every 32 columns
            auto issue_sum = [&](uint32_t acc, uint32_t op, uint64_t dB, bool fresh) {
#pragma unroll
                for (int ks = 0; ks < 8; ks++)
                    mma_ts(leader, tbase + acc, tbase + op + (ks / 2) * 32 + (ks % 2) * 8, dB + (ks * 2048 >> 4), idA, !fresh || ks > 0);
            };
            bool ok = any;
            if constexpr (KIND != kDv) {
                if (warp == kWarps) {  // S and dP
                    Stage<C::N1> s1;
                    Stage<C::N2> s2;
                    Stage<2> sb;
                    uint32_t n = 0;
                    ok = ok && warp_wait(smem_u32(&bar->x_full), 0, abort_flag, a);
                    for (Items<KEYS> it = first; ok && !it.done(); it.next(a), n++) {
                        ok = warp_wait(smem_u32(&bar->y1_full[s1.st]), s1.parity, abort_flag, a);
                        if (!ok) break;
                        clear_rows(ring1 + s1.st * HALF, it);
                        if (n > 0) ok = warp_wait(smem_u32(&bar->s_free), (n - 1) & 1, abort_flag, a);
                        if (!ok) break;
                        tc_fence_after();
                        mma_half(0, dX, dY1 + (s1.st * HALF >> 4), true);
                        commit(leader, smem_u32(&bar->s_full[0]));
                        s1.next();
                        if (n >= 2) ok = warp_wait(smem_u32(&bar->dp_free[sb.st]), sb.parity ^ 1, abort_flag, a);
                        for (int h = 0; ok && h < 2; h++) {
                            ok = warp_wait(smem_u32(&bar->y2_full[s2.st]), s2.parity, abort_flag, a);
                            if (!ok) break;
                            if (KEYS) clear_rows(ring2 + s2.st * HALF, it);  // v only enters dP, which the mask covers
                            tc_fence_after();
                            mma_half(C::TM_DP + sb.st * 128, dX + ((1 + h) * HALF >> 4), dY2 + (s2.st * HALF >> 4), h == 0);
                            commit(leader, smem_u32(&bar->y2_empty[s2.st]));
                            s2.next();
                        }
                        if (ok) commit(leader, smem_u32(&bar->dp_full[sb.st]));
                        sb.next();
                    }
                } else {  // the sums
                    Stage<C::N1> t1;
                    Stage<2> tb;
                    bool fresh = true;
                    for (Items<KEYS> it = first; ok && !it.done(); it.next(a)) {
                        ok = warp_wait(smem_u32(&bar->ready[tb.st]), tb.parity, abort_flag, a);
                        if (!ok) break;
                        tc_fence_after();
                        issue_sum(C::TM_ACC, C::TM_DP + tb.st * 128, dM1 + (t1.st * HALF >> 4), fresh);
                        commit(leader, smem_u32(&bar->dp_free[tb.st]));
                        commit(leader, smem_u32(&bar->y1_empty[t1.st]));
                        fresh = false;
                        t1.next();
                        tb.next();
                    }
                    if (ok) commit(leader, smem_u32(&bar->acc_full));
                }
            } else if (warp == kWarps) {
                // S of the first map is made as soon as the last one is read, S of the second behind
                // the product that uses up what lies over it.
                Stage<C::N1> s1;
                Stage<C::N2> s2;
                ok = ok && warp_wait(smem_u32(&bar->x_full), 0, abort_flag, a);
                auto issue_S = [&](int i, const Items<KEYS>& it) {
                    if (!warp_wait(smem_u32(&bar->y1_full[s1.st]), s1.parity, abort_flag, a)) return false;
                    clear_rows(ring1 + s1.st * HALF, it);
                    tc_fence_after();
                    mma_half(i * 128, dX + (i * HALF >> 4), dY1 + (s1.st * HALF >> 4), true);
                    commit(leader, smem_u32(&bar->s_full[i]));
                    commit(leader, smem_u32(&bar->y1_empty[s1.st]));
                    s1.next();
                    return true;
                };
                Items<KEYS> it = first, ahead = first;
                ok = ok && issue_S(0, it) && issue_S(1, it);
                uint32_t n = 0;
                for (bool fresh = true; ok; fresh = false, n++) {
                    ahead.next(a);
                    const bool more = !ahead.done();
                    if (more) ok = warp_wait(smem_u32(&bar->s_free), n & 1, abort_flag, a) && issue_S(0, ahead);
                    ok = ok && warp_wait(smem_u32(&bar->ready[0]), n & 1, abort_flag, a);
                    for (int h = 0; ok && h < 2; h++) {
                        ok = warp_wait(smem_u32(&bar->y2_full[s2.st]), s2.parity, abort_flag, a);
                        if (!ok) break;
                        clear_rows(ring2 + s2.st * HALF, it);
                        tc_fence_after();
                        issue_sum(C::TM_ACC + 128 * h, 128, dM2 + (s2.st * HALF >> 4), fresh);
                        commit(leader, smem_u32(&bar->y2_empty[s2.st]));
                        s2.next();
                    }
                    if (!ok || !more) break;
                    ok = issue_S(1, ahead);
                    it = ahead;
                }
                if (ok) commit(leader, smem_u32(&bar->acc_full));
            }
            // no MMA may be in flight when tensor memory is released
            commit(leader, smem_u32(&bar->drain[warp - kWarps]));
            if (lane == 0) land(smem_u32(&bar->drain[warp - kWarps]), 0);
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
        const uint32_t tS = tbase + lanes + w * kCols;
        const long long all = (long long)a.slices * a.Rp;  // of one of the rows' numbers
        const float* lams = a.nl2 + 4 * all + (long long)slice * a.Rp;
        const bool one_head = a.R == a.nq;  // one lam for all rows of the slice
        uint32_t n = 0;
        float lam = 0.f;
        int kend = 0;
        // Keys read tensor memory as fragments: registers 16 h + 4 i + 2 e + k of a tile are column
        // w kCols + fc + 8 i + k, row fr + 16 h + 8 e, so that a thread needs the numbers of 8
        // columns and not of 32: shared memory, where they are, is kept busy by the products.
        const int fr = (warp & 3) * 32 + (lane >> 2), fc = 2 * (lane & 3);
        const uint32_t low = 16u << 16;  // the second 16 lanes
        auto pair = [](const uint32_t* v) { return pack2(__uint_as_float(v[0]), __uint_as_float(v[1])); };
        auto put = [](uint32_t* v, uint64_t y) {
            float e0, e1;
            unpack2(y, e0, e1);
            v[0] = __float_as_uint(e0);
            v[1] = __float_as_uint(e1);
        };
        auto read = [&](uint32_t at, uint32_t* v) {
            tmem_ld_frag(at, v);
            tmem_ld_frag(at + low, v + 16);
            tmem_wait_ld();
        };
        auto write = [&](uint32_t at, const uint32_t* v) {
            tmem_st_frag16(at, v);
            tmem_st_frag16(at + low, v + 8);
            tmem_wait_st();
        };
        // 2^(scale log2(e) s + nl2) in place, nl2 of the tile's rows from `st` on
        auto weights = [&](uint32_t* v, const float* st) {
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
                const uint64_t l = *reinterpret_cast<const uint64_t*>(st + 2 * c);
#pragma unroll
                for (int x = c; x < 32; x += (x & 2) ? 14 : 2) {
                    float e0, e1;
                    unpack2(fma2(pair(v + x), sl2x2, l), e0, e1);
                    v[x] = __float_as_uint(ex2(e0));
                    v[x + 1] = __float_as_uint(ex2(e1));
                }
            }
        };
        // v times lam of the tile's rows, from row `pos` on
        auto times_lam = [&](uint32_t* v, int pos) {
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
                uint64_t l = pack2(lam, lam);
                if (!one_head) {
                    const float2 u = *reinterpret_cast<const float2*>(lams + pos + w * kCols + fc + 2 * c);
                    l = pack2(u.x, u.y);
                }
#pragma unroll
                for (int x = c; x < 32; x += (x & 2) ? 14 : 2) put(v + x, mul2(pair(v + x), l));
            }
        };
        // The lengths are in l2; causal order cuts where a row's keys end inside the block's keys.
        auto cut = [&](const Items<KEYS>& it, uint32_t* v, uint32_t* u) {
            if (!a.causal || !(it.t0 + BT > a.nq || dense_kend(a, sp, it.t0) < x0 + BT)) return;
#pragma unroll
            for (int c = 0; c < 16; c += 4)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const int last = (it.t0 + w * kCols + fc + 2 * c + k) % a.nq + sp.lk - sp.lq;  // key that this column's row sees last
#pragma unroll
                    for (int y = 0; y < 4; y++)
                        if (x0 + fr + 8 * y > last) v[16 * (y >> 1) + c + 2 * (y & 1) + k] = u[16 * (y >> 1) + c + 2 * (y & 1) + k] = 0u;
                }
        };
        if (KEYS && one_head) lam = diff_lam(f, diff_head(f, slice, 0));
        if constexpr (KIND == kDv) {
            for (Items<KEYS> it = first; !it.done(); it.next(a), n++) {
                const int k = n & 1;
                const float* st = stats + k * 2 * BT + w * kCols + fc;
                bar_wait(smem_u32(&bar->st_full[k]), (n / 2) & 1, abort_flag, a);
                uint32_t p[kCols], s[kCols], o[kCols / 2];
                bar_wait(smem_u32(&bar->s_full[0]), n & 1, abort_flag, a);
                tc_fence_after();
                read(tS, p);
                tc_fence_before();
                warp_arrive(smem_u32(&bar->s_free), lane);
                weights(p, st);
                bar_wait(smem_u32(&bar->s_full[1]), n & 1, abort_flag, a);
                tc_fence_after();
                read(tS + 128, s);
                weights(s, st + BT);
                times_lam(s, it.pos);
                cut(it, p, s);
#pragma unroll
                for (int c = 0; c < kCols; c += 2)
                    o[c >> 1] = pack_bf16x2(__uint_as_float(p[c]) - __uint_as_float(s[c]), __uint_as_float(p[c + 1]) - __uint_as_float(s[c + 1]));
                write(tS + 128, o);
                tc_fence_before();
                // only now: an arrival right behind the loads has overtaken the last of them, and
                // the next copy was there first
                warp_arrive(smem_u32(&bar->st_empty[k]), lane);
                warp_arrive(smem_u32(&bar->ready[0]), lane);
            }
        } else if constexpr (KIND == kDk) {
            Stage<2> sb;
            for (Items<KEYS> it = first; !it.done(); it.next(a), n++) {
                const int k = n & 1;
                const float* st = stats + k * 2 * BT + w * kCols + fc;  // -l2 of these columns' rows; -D BT further
                const uint32_t tG = tS + C::TM_DP + sb.st * 128;
                uint32_t s[kCols], g[kCols], o[kCols / 2];
                bar_wait(smem_u32(&bar->st_full[k]), (n / 2) & 1, abort_flag, a);
                bar_wait(smem_u32(&bar->s_full[0]), n & 1, abort_flag, a);
                tc_fence_after();
                read(tS, s);
                tc_fence_before();
                warp_arrive(smem_u32(&bar->s_free), lane);
                weights(s, st);
                if (map == 1 && !one_head) times_lam(s, it.pos);
                cut(it, s, s);
                bar_wait(smem_u32(&bar->dp_full[sb.st]), sb.parity, abort_flag, a);
                tc_fence_after();
                read(tG, g);
#pragma unroll
                for (int c = 0; c < 16; c += 4) {
                    const uint64_t nd = *reinterpret_cast<const uint64_t*>(st + BT + 2 * c);
#pragma unroll
                    for (int x = c; x < 32; x += (x & 2) ? 14 : 2) {
                        float e0, e1;
                        unpack2(mul2(add2(pair(g + x), nd), pair(s + x)), e0, e1);
                        o[x >> 1] = pack_bf16x2(e0, e1);
                    }
                }
                write(tG, o);
                tc_fence_before();
                warp_arrive(smem_u32(&bar->st_empty[k]), lane);
                warp_arrive(smem_u32(&bar->ready[sb.st]), lane);
                sb.next();
            }
        } else {
            const long long row = (long long)slice * a.Rp + x;  // Rp is a multiple of 128
            const float nl = a.nl2[map * all + row], nd = a.nl2[(2 + map) * all + row];
            const uint64_t nl2x2 = pack2(nl, nl), ndx2 = pack2(nd, nd);
            uint64_t sum2 = 0ull;
            lam = a.nl2[4 * all + row];
            kend = x < a.R ? dense_kend(a, sp, x < a.nq ? x : x % a.nq) : 0;
            Stage<2> sb;
            for (Items<KEYS> it = first; !it.done(); it.next(a), n++) {
                const uint32_t tG = tS + C::TM_DP + sb.st * 128;
                uint32_t s[kCols], g[kCols], o[kCols / 2];
                bar_wait(smem_u32(&bar->s_full[0]), n & 1, abort_flag, a);
                tc_fence_after();
                tmem_ld32_nowait(tS, s);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->s_free), lane);
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    float e0, e1;
                    unpack2(fma2(pair(s + c), sl2x2, nl2x2), e0, e1);
                    s[c] = __float_as_uint(ex2(e0));
                    s[c + 1] = __float_as_uint(ex2(e1));
                }
                bar_wait(smem_u32(&bar->dp_full[sb.st]), sb.parity, abort_flag, a);
                tc_fence_after();
                tmem_ld32_nowait(tG, g);
                tmem_wait_ld();
                if (__any_sync(0xffffffffu, kend - it.pos < BT)) {  // S and dP of a key behind the lengths may be anything
                    const int lim = kend - it.pos - w * kCols;
#pragma unroll
                    for (int c = 0; c < kCols; c++) {
                        s[c] = c < lim ? s[c] : 0u;
                        g[c] = c < lim ? g[c] : 0u;
                    }
                }
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    if (map == 1) sum2 = fma2(pair(s + c), pair(g + c), sum2);
                    float e0, e1;
                    unpack2(mul2(add2(pair(g + c), ndx2), pair(s + c)), e0, e1);
                    o[c >> 1] = pack_bf16x2(e0, e1);
                }
                tmem_st16(tG, o);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->ready[sb.st]), lane);
                sb.next();
            }
            if (map == 1) {
                // P_2 dP of this part's keys, a quarter of the columns each
                float u0, u1;
                unpack2(sum2, u0, u1);
                f.d2[((long long)(part * 4 + w) * a.slices + slice) * a.Rp + x] = kend > 0 ? u0 + u1 : 0.f;
            }
        }
        // rows without a gradient hold whatever their padding made: zero
        const bool live = any && (KEYS ? x < sp.lk : kend > 0);
        if (any) {
            bar_wait(smem_u32(&bar->acc_full), 0, abort_flag, a);
            tc_fence_after();
        }
        const long long all2 = 2LL * a.slices * extent;  // rows of dq or dk
        const float scale = KIND == kDv ? 1.f : map == 0 ? a.scale : KEYS ? (one_head ? -lam * a.scale : -a.scale) : -lam * a.scale;
        const int cols = KIND == kDv ? 2 * a.d : a.d;
        const long long row = (long long)(KIND == kDv ? slice : m0) * extent + x;
#pragma unroll
        for (int k = 0; k < (KIND == kDv ? 4 : 2); k++) {  // 64 columns
            const int c = k * 64 + w * 16;
            float o[16];
            if (any) tmem_ld16(tbase + C::TM_ACC + c + lanes, o);
#pragma unroll
            for (int e = 0; e < 16; e++) o[e] = live ? o[e] * scale : 0.f;
            if (a.splits > 1) {
                // parts: dq; or dk of all parts, then dv of all parts
                float* dst = KIND == kDv ? a.part + a.splits * all2 * a.d + (part * (all2 / 2) + row) * cols
                                         : a.part + (part * all2 + row) * cols;
                if (x < extent) diff_store16(dst + c, o, c, cols);
            } else if (any) {
                // the stationary tiles have been used up: their place takes the results
                put_chunk(sX + k * REGION, lr, w * 2, o);
                put_chunk(sX + k * REGION, lr, w * 2 + 1, o + 8);
            } else if (x < extent) {
                diff_store16(static_cast<__nv_bfloat16*>(KIND == kDv ? a.dv : KEYS ? a.dk : a.dq) + row * cols + c, o, c, cols);
            }
        }
        if (any && a.splits == 1) {
            fence_async_smem();
            named_barrier(1 + (warp & 3), 128);  // the four warps of these 32 rows
            if (w == 0 && lane == 0 && x < extent) {
                for (int c = 0; c * 64 < cols; c++)
                    tma_store_3d(KIND == kDv ? &maps.zv : KEYS ? &maps.zk : &maps.zq, smem_u32(sX + c * REGION + lr * 128), c * 64, x,
                                 KIND == kDv ? slice : m0);
                bulk_commit();
                bulk_wait_read();
            }
        }
        if (KIND == kDq && map == 1) diff_lam_last(f, &bar->last);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarps) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

// Longer pieces first, so that the last ones are short: those of keys have R / 128 tiles, those
// of rows nk / 128, and a tile costs most in dv (8 heads over 2, 4,095 tokens: dv first 500 us,
// dk first 571). In causal order every kind has short pieces at its end, and dk comes first (3 x 4
// heads over 2, 2,000 x 3,000 tokens: 254 us, dv first 262).
__global__ void __launch_bounds__(kThreads, 1)
diff_bwd_wide_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                        const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                        const __grid_constant__ CUtensorMap zq, const __grid_constant__ CUtensorMap zk,
                        const __grid_constant__ CUtensorMap zv, const __grid_constant__ DiffArgs aq,
                        const __grid_constant__ DiffArgs ak, int row_pieces, int key_pieces, int keys_first) {
    const Maps maps = {mq, mg, mk, mv, zq, zk, zv};
    int piece = blockIdx.x;
    if (keys_first) piece = piece < 3 * key_pieces ? piece + 2 * row_pieces : piece - 3 * key_pieces;
    if (piece < 2 * row_pieces) return bwd_piece<kDq>(maps, aq, piece);
    piece -= 2 * row_pieces;
    const int dk0 = ak.d.causal ? 0 : key_pieces, dv0 = ak.d.causal ? 2 * key_pieces : 0;
    if (piece >= dk0 && piece < dk0 + 2 * key_pieces) bwd_piece<kDk>(maps, ak, piece - dk0);
    else bwd_piece<kDv>(maps, ak, piece - dv0);
}

}  // namespace

int launch_diff_tc_bwd_wide(const DiffShape& s, const DiffArgs& aq, const DiffArgs& ak, cudaStream_t st) {
    constexpr int smem = std::max({Cfg<kDq>::SMEM, Cfg<kDk>::SMEM, Cfg<kDv>::SMEM});
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
    cudaFuncSetAttribute(diff_bwd_wide_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const long long pq = (long long)((s.R + BT - 1) / BT) * s.slices * a.splits;
    const long long pk = (long long)((s.nk + BT - 1) / BT) * s.slices * ak.d.splits;
    if (2 * pq + 3 * pk > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    // Closely behind the rows' numbers (8 heads, 4,096 tokens 513 -> 506 us), but not in causal
    // order: blocks then start where those leave first, which lays long pieces side by side (8
    // heads over 2, 4,095 tokens 313 -> 407 us).
    LLSA_LAUNCH("diff_bwd_wide_tc", st, launch_close(!s.causal, diff_bwd_wide_tc_kernel, dim3((unsigned)(2 * pq + 3 * pk)), kThreads, smem, st, mq,
                                                     mg, mk, mv, zq, zk, zv, aq, ak, (int)pq, (int)pk,
                                                     (int)(std::min(ak.d.chunk, s.R) >= std::min(a.chunk, s.nk))));
    return LLSA_OK;
}

}  // namespace llsa

// dense_bwd_tc.cu -- dense attention backward on the tcgen05 tensor cores (bf16,
// d <= 128; the tiles hold 64 or 128 columns, TMA fills the rest with zeros).
//
// Mathematics, with l2 = lse * log2(e) and D = dout . o of every query row from
// the pass before: P = 2^(scale log2(e) q.k - l2), dS = P (dout.v - D),
//   dq = scale dS K          by blocks that own 128 query rows,
//   dk = scale dS^T Q, dv = P^T dO   by blocks that own 128 keys.
// Every sum has one owner and a fixed order, so results repeat bit by bit. One
// pass for all three gradients would save two of seven matrix products per
// tile, at the price of adding dq up across blocks in memory in whatever order
// they run.
//
// Both kinds of blocks run in one launch, so that one kind fills the SMs that the
// other leaves (12 heads x 4,096 tokens 170 us in two launches, 154 in one; d = 128,
// 16 heads over 4 of 4,095 tokens, causal, 275 and 197). Their code is one: 128 stationary rows (X1, X2) against a stream of tiles of
// 128 rows (Y1, Y2), with (X1, X2, Y1, Y2) = (Q, dO, K, V) or (K, V, Q, dO). Per
// item: S = X1 Y1^T, dP = X2 Y2^T (128 x 128 fp32 in tensor memory), then P and
// dS as bf16 over dP's columns, then acc1 += dS Y1 and, for keys, acc2 += P Y2,
// with P and dS as tensor-memory operands. P and dS are rounded to bf16 there, the type
// that these products have beside bf16 inputs (2^-9 of each, independent from key to
// key; statistics, D and all sums stay in fp32). An M = 128 product of two
// shared-memory operands takes 64 clocks per 16 of K at N = 128 and 48 at N = 64
// (shared memory feeds it then), so tiles of 128 are worth their tensor memory.
//
// The next item's S, and dP where there is room for two of them (all but keys at
// 128 columns), are issued before this item's sums, so the tensor cores work
// while the threads turn S and dP into P and dS. All sixteen elementwise warps
// take one item together, a thread per row and quarter of the columns.
//
// At 64 columns one block per SM stays for the whole call and takes its share of
// the work: while the elementwise warps finish one piece, the others load and
// multiply for the next. At 128 columns shared memory holds one pair of
// stationary tiles, and every piece gets a block of its own (figures at the launch).
//
// Bound by the chain of an item at 64 columns (S, exp, dP, dS, stores; 0.72 us against
// 0.40 us of the tensor cores' time for an item of rows) and by the tensor cores at 128.
// 19 slices of 16,384 tokens: 3.2 ms at d = 64 (1,020 TFLOP/s of the 10 d
// operations per pair), 5.1 ms at d = 128 (1,270).
//
// Roles: warps 0-15 elementwise and epilogue, warps 16 and 17 issue the MMAs,
// warps 18 and 19 the copies of the two streams.
#include <algorithm>

#include "dense_tc.cuh"

namespace llsa {
namespace {

using namespace tc;

constexpr int kWarps = 16, kCols = 32;  // elementwise warps: a thread takes one row and kCols columns of an item
// 20 warps of 96 registers at launch = 61,440: the 512 elementwise threads take
// 104 of them, the 128 others keep 64.
constexpr int kThreads = (kWarps + 4) * 32, kRegsElementwise = 104, kRegsOther = 64;
constexpr int BT = kTileRows;

template <int D, bool KEYS>
struct Cfg {
    static constexpr int TILE = BT * D * 2;   // bytes of 128 rows
    static constexpr int REGION = BT * 128;   // bytes of 128 rows x 64 columns
    static constexpr int N1 = D == 64 ? 4 : 3, N2 = D == 64 ? 4 : 2;  // stages of the two streams
    static constexpr int NX = D == 64 ? 2 : 1;                        // pairs of stationary tiles
    static constexpr int NB = D == 128 && KEYS ? 1 : 2;               // dP buffers
    static constexpr int STATS = KEYS ? N2 * 2 * BT * 4 : 0;          // -l2 and -D of a row tile, with stream 2
    static constexpr int SMEM = (2 * NX + N1 + N2) * TILE + STATS + 1024;
    static constexpr int TM_DP = 128, TM_ACC = 128 + NB * 128;        // S at column 0
};

struct Bars {
    uint64_t x_full[2][2], x_free[2], y1_full[4], y1_empty[4], y2_full[4], y2_empty[4];
    uint64_t s_full, s_free, dp_full[2], ds_ready[2], dp_free[2], acc_full, acc_free, drain[2];
    PieceRing pieces;
    uint32_t tmem_slot;
    int abort_flag;
};

// One piece of work: 128 stationary rows of a slice against a part of the stream.
template <bool KEYS>
struct Piece {
    int slice, x0, part, pos, t0, stop;  // pos, t0: the first item
    DenseSpan sp;

    __device__ __forceinline__ void make(const DenseArgs& a, int id) {
        const DenseWork w = dense_work(a, id, ((KEYS ? a.nk : a.R) + BT - 1) / BT);
        slice = w.slice;
        part = w.part;
        // causal order: the last rows see the most keys, the first keys the most rows; those come first
        x0 = (a.causal && !KEYS ? w.blocks - 1 - w.block : w.block) * BT;
        sp = dense_span(a, slice);
        pos = a.splits > 1 ? part * a.chunk : 0;
        if constexpr (KEYS) {
            stop = x0 < sp.lk ? (a.splits > 1 ? min(a.R, pos + a.chunk) : a.R) : 0;
        } else {
            stop = dense_tile_kend(a, sp, x0 < a.nq ? x0 : x0 % a.nq, BT);
            if (a.splits > 1) stop = min(stop, pos + a.chunk);
        }
        t0 = 0;
        Items<KEYS> it = items(a);
        it.start(a);
        pos = it.pos;
        t0 = it.t0;
    }
    __device__ __forceinline__ Items<KEYS> items(const DenseArgs& a) const { return Items<KEYS>(a, sp, x0, pos, t0, stop); }
    __device__ __forceinline__ bool put(PieceRing* ring, int i, volatile int* abort_flag, const DenseArgs& a) const {
        return piece_put(ring, i, make_int4(slice, x0, part, pos), make_int4(t0, stop, sp.lq, sp.lk), abort_flag, a);
    }
    template <int LANES>
    __device__ __forceinline__ bool get(PieceRing* ring, int i, int lane, volatile int* abort_flag, const DenseArgs& a) {
        int4 x, y;
        if (!piece_get<LANES>(ring, i, x, y, lane, abort_flag, a)) return false;
        slice = x.x;
        x0 = x.y;
        part = x.z;
        pos = x.w;
        t0 = y.x;
        stop = y.y;
        sp.lq = y.z;
        sp.lk = y.w;
        return true;
    }
};

// Block `block` of the `blocks` that share the pieces of rows or of keys.
template <int D, bool KEYS>
__device__ __forceinline__ void bwd_side(const CUtensorMap& mx1, const CUtensorMap& mx2, const CUtensorMap& my1,
                                         const CUtensorMap& my2, const CUtensorMap& mz1, const CUtensorMap& mz2,
                                         const DenseArgs& a, int block, int blocks) {
    using C = Cfg<D, KEYS>;
    extern __shared__ __align__(1024) unsigned char sm[];
    unsigned char* sX = sm;  // [NX] X1, X2
    unsigned char* ring1 = sm + 2 * C::NX * C::TILE;
    unsigned char* ring2 = ring1 + C::N1 * C::TILE;
    float* stats = reinterpret_cast<float*>(ring2 + C::N2 * C::TILE);
    Bars* bar = reinterpret_cast<Bars*>(ring2 + C::N2 * C::TILE + C::STATS);
    volatile int* abort_flag = &bar->abort_flag;
    // broadcast, so that the compiler knows these as the same in a whole warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (smem_u32(sm) & 1023u) {  // the swizzled layouts need it; the whole block leaves
        if (threadIdx.x == 0) set_status(a.status, LLSA_ERR_TIMEOUT);
        return;
    }
    const int extent = KEYS ? a.nk : a.R;
    const int mine = dealt_pieces(a, block, blocks);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->x_full[0][i]), 1);
            mbar_init(smem_u32(&bar->x_full[1][i]), 1);
            mbar_init(smem_u32(&bar->x_free[i]), 4);
            mbar_init(smem_u32(&bar->dp_full[i]), 1);
            mbar_init(smem_u32(&bar->ds_ready[i]), kWarps);
            mbar_init(smem_u32(&bar->dp_free[i]), 1);
            mbar_init(smem_u32(&bar->drain[i]), 1);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(smem_u32(&bar->y1_full[i]), 1);
            mbar_init(smem_u32(&bar->y1_empty[i]), 1);
            mbar_init(smem_u32(&bar->y2_full[i]), 1);
            mbar_init(smem_u32(&bar->y2_empty[i]), 1);
        }
        mbar_init(smem_u32(&bar->s_full), 1);
        mbar_init(smem_u32(&bar->s_free), kWarps);
        mbar_init(smem_u32(&bar->acc_full), 1);
        mbar_init(smem_u32(&bar->acc_free), kWarps);
        piece_ring_init(&bar->pieces, kWarps + (C::NB > 1 ? 3 : 2));  // elementwise warps, issuers, the copies of stream 2
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kWarps) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    if (warp >= kWarps + 2 && lane == 0) {
        prefetch_map(warp == kWarps + 2 ? &mx1 : &mx2);
        prefetch_map(warp == kWarps + 2 ? &my1 : &my2);
        prefetch_map(warp == kWarps + 2 ? &mz1 : &mz2);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_slot, 0);

    // Every role walks the block's pieces. Counted on through them: the stages of
    // the rings and buffers, the items (n), and the pieces that have any (v).
    if (warp >= kWarps) {
        regs_dec<kRegsOther>();
        if (warp >= kWarps + 2) {
            // ----------------------------------------------------------- copies
            if (lane == 0 && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const int k = warp - kWarps - 2;  // stream
                const int ns = k == 0 ? C::N1 : C::N2;
                unsigned char* ring = k == 0 ? ring1 : ring2;
                uint64_t* full = k == 0 ? bar->y1_full : bar->y2_full;
                uint64_t* empty = k == 0 ? bar->y1_empty : bar->y2_empty;
                const CUtensorMap* mx = k == 0 ? &mx1 : &mx2;
                const CUtensorMap* my = k == 0 ? &my1 : &my2;
                int st = 0, n = 0, v = 0;
                uint32_t parity = 1;  // of the release that the stage's next use waits for
                bool ok = true;
                for (int i = 0; ok && i < mine; i++) {
                    Piece<KEYS> pc;
                    if (k == 0) {
                        pc.make(a, dealt(a, i, block, blocks));
                        ok = pc.put(&bar->pieces, i, abort_flag, a);
                    } else {
                        ok = pc.template get<1>(&bar->pieces, i, lane, abort_flag, a);
                    }
                    if (!ok) break;
                    Items<KEYS> it = pc.items(a);
                    if (it.done()) continue;
                    const int xb = v % C::NX;
                    if (v >= C::NX) ok = bar_wait(smem_u32(&bar->x_free[xb]), (v / C::NX - 1) & 1, abort_flag, a);
                    if (!ok) break;
                    const uint32_t fx = smem_u32(&bar->x_full[k][xb]);
                    mbar_arrive_expect_tx(fx, C::TILE);
                    for (int c = 0; c < D / 64; c++)
                        tma_load_3d(smem_u32(sX + (2 * xb + k) * C::TILE + c * C::REGION), mx, c * 64, pc.x0, pc.slice, fx);
                    v++;
                    for (; !it.done(); it.next(a)) {
                        if (n >= ns) ok = bar_wait(smem_u32(&empty[st]), parity, abort_flag, a);
                        if (!ok) break;
                        const uint32_t fb = smem_u32(&full[st]);
                        const bool with_stats = KEYS && k == 1;
                        mbar_arrive_expect_tx(fb, C::TILE + (with_stats ? 2 * BT * 4 : 0));
                        for (int c = 0; c < D / 64; c++)
                            tma_load_3d(smem_u32(ring + st * C::TILE + c * C::REGION), my, c * 64, it.pos, pc.slice, fb);
                        if (with_stats) {
                            const long long row = (long long)pc.slice * a.Rp + it.pos;
                            bulk_load(smem_u32(stats + st * 2 * BT), a.nl2 + row, BT * 4, fb);
                            bulk_load(smem_u32(stats + st * 2 * BT + BT), a.nd + row, BT * 4, fb);
                        }
                        n++;
                        if (++st == ns) {
                            st = 0;
                            parity ^= 1;
                        }
                    }
                }
                // copies still in flight must land before the block exits
                for (int x = max(0, v - C::NX); x < v; x++) land(smem_u32(&bar->x_full[k][x % C::NX]), (x / C::NX) & 1);
                for (int x = max(0, n - ns); x < n; x++) land(smem_u32(&full[x % ns]), (x / ns) & 1);
            }
        } else {
            // ----------------------------------------------------- MMA issuers
            // With two dP buffers warp kWarps issues S and dP, the next warp the
            // sums. With one, dP of the next item goes where this item's P and
            // dS are, so one warp issues all, dP right behind the sums that use
            // those up.
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BT, BT, 0, 0), idA = idesc_bf16(BT, D, 0, 1);
            const uint64_t dX = desc_sw128(smem_u32(sX), 16, 1024);
            const uint64_t dY1 = desc_sw128(smem_u32(ring1), 16, 1024), dY2 = desc_sw128(smem_u32(ring2), 16, 1024);
            const uint64_t dM1 = desc_sw128(smem_u32(ring1), C::REGION, 1024);  // the tiles read along their rows
            const uint64_t dM2 = desc_sw128(smem_u32(ring2), C::REGION, 1024);
            // Rows of the streamed tile whose P and dS are 0 by the mask of the
            // lengths may hold anything: they meet those zeros in the sums, so
            // they are cleared.
            auto clear_rows = [&](unsigned char* tile, const Items<KEYS>& it) {
                if constexpr (KEYS) {
                    if (it.all || it.t0 + BT <= it.sp.lq) return;
                    int t = it.t0 + lane;
                    for (int x = lane; x < BT; x += 32, t += 32)
                        if (t % a.nq >= it.sp.lq)
                            for (int c = 0; c < D / 64; c++)
                                for (int e = 0; e < 8; e++)
                                    reinterpret_cast<uint4*>(tile + c * C::REGION + x * 128)[e] = make_uint4(0u, 0u, 0u, 0u);
                } else {
                    const int live = it.sp.lk - it.pos;
                    if (live >= BT) return;
                    for (int c = 0; c < D / 64; c++)
                        for (int x = live * 8 + lane; x < BT * 8; x += 32)
                            reinterpret_cast<uint4*>(tile + c * C::REGION)[x] = make_uint4(0u, 0u, 0u, 0u);
                }
                fence_async_smem();
                __syncwarp();
            };
            // stages and buffers of the next S (s1), dP (s2, sb) and sums (t1, t2, tb)
            Stage<C::N1> s1, t1;
            Stage<C::N2> s2, t2;
            Stage<C::NB> sb, tb;
            Stage<C::NX> sx;
            uint32_t n = 0, nd = 0;  // S and dP issued
            int v = 0;
            uint64_t dX1 = 0, dX2 = 0;
            auto take_x = [&]() {
                dX1 = dX + (2 * sx.st * C::TILE >> 4);
                dX2 = dX1 + (C::TILE >> 4);
                return warp_wait(smem_u32(&bar->x_full[0][sx.st]), sx.parity, abort_flag, a) &&
                       warp_wait(smem_u32(&bar->x_full[1][sx.st]), sx.parity, abort_flag, a);
            };
            auto issue_S = [&](const Items<KEYS>& it) {
                if (!warp_wait(smem_u32(&bar->y1_full[s1.st]), s1.parity, abort_flag, a)) return false;
                clear_rows(ring1 + s1.st * C::TILE, it);
                if (n > 0 && !warp_wait(smem_u32(&bar->s_free), (n - 1) & 1, abort_flag, a)) return false;
                tc_fence_after();
                const uint64_t dT = dY1 + (s1.st * C::TILE >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++) {
                    const uint32_t off = (ks / 4) * C::REGION + (ks % 4) * 32;
                    mma_ss(leader, tbase, dX1 + (off >> 4), dT + (off >> 4), idS, ks > 0);
                }
                commit(leader, smem_u32(&bar->s_full));
                s1.next();
                n++;
                return true;
            };
            auto issue_dP = [&](const Items<KEYS>& it) {
                if (!warp_wait(smem_u32(&bar->y2_full[s2.st]), s2.parity, abort_flag, a)) return false;
                if (KEYS) clear_rows(ring2 + s2.st * C::TILE, it);  // V only enters dP, which the mask covers
                if (C::NB > 1 && nd >= C::NB && !warp_wait(smem_u32(&bar->dp_free[sb.st]), sb.parity ^ 1, abort_flag, a))
                    return false;
                tc_fence_after();
                const uint64_t dT = dY2 + (s2.st * C::TILE >> 4);
#pragma unroll
                for (int ks = 0; ks < D / 16; ks++) {
                    const uint32_t off = (ks / 4) * C::REGION + (ks % 4) * 32;
                    mma_ss(leader, tbase + C::TM_DP + sb.st * 128, dX2 + (off >> 4), dT + (off >> 4), idS, ks > 0);
                }
                commit(leader, smem_u32(&bar->dp_full[sb.st]));
                if (!KEYS) commit(leader, smem_u32(&bar->y2_empty[s2.st]));
                s2.next();
                sb.next();
                nd++;
                return true;
            };
            auto issue_sums = [&](bool fresh) {
                if (!warp_wait(smem_u32(&bar->ds_ready[tb.st]), tb.parity, abort_flag, a)) return false;
                tc_fence_after();
                const uint32_t p0 = tbase + C::TM_DP + tb.st * 128;
                const uint64_t dT1 = dM1 + (t1.st * C::TILE >> 4), dT2 = dM2 + (t2.st * C::TILE >> 4);
#pragma unroll
                for (int ks = 0; ks < BT / 16; ks++) {
                    const uint32_t op = p0 + (ks / 2) * 32 + (ks % 2) * 8;  // of every 32 columns: P, then dS, 16 words each
                    if constexpr (KEYS) {
                        mma_ts(leader, tbase + C::TM_ACC + D, op, dT2 + (ks * 2048 >> 4), idA, !fresh || ks > 0);
                        mma_ts(leader, tbase + C::TM_ACC, op + 16, dT1 + (ks * 2048 >> 4), idA, !fresh || ks > 0);
                    } else {
                        mma_ts(leader, tbase + C::TM_ACC, op, dT1 + (ks * 2048 >> 4), idA, !fresh || ks > 0);
                    }
                }
                if (C::NB > 1) commit(leader, smem_u32(&bar->dp_free[tb.st]));
                commit(leader, smem_u32(&bar->y1_empty[t1.st]));
                if (KEYS) commit(leader, smem_u32(&bar->y2_empty[t2.st]));
                t1.next();
                t2.next();
                tb.next();
                return true;
            };
            bool ok = C::NB > 1 || warp == kWarps;
            for (int i = 0; ok && i < mine; i++) {
                Piece<KEYS> pc;
                ok = pc.template get<32>(&bar->pieces, i, lane, abort_flag, a);
                if (!ok) break;
                Items<KEYS> it = pc.items(a);
                if (it.done()) continue;
                if (C::NB > 1 && warp == kWarps) {
                    ok = take_x();
                    for (; ok && !it.done(); it.next(a)) ok = issue_S(it) && issue_dP(it);
                } else if (C::NB > 1) {
                    if (v > 0) ok = warp_wait(smem_u32(&bar->acc_free), (v - 1) & 1, abort_flag, a);
                    for (bool fresh = true; ok && !it.done(); it.next(a), fresh = false) ok = issue_sums(fresh);
                    if (ok) commit(leader, smem_u32(&bar->acc_full));
                } else {
                    ok = take_x() && issue_S(it) && issue_dP(it);
                    if (ok && v > 0) ok = warp_wait(smem_u32(&bar->acc_free), (v - 1) & 1, abort_flag, a);
                    it.next(a);
                    for (bool fresh = true; ok; fresh = false) {
                        const bool more = !it.done();
                        if (more) ok = issue_S(it);
                        ok = ok && issue_sums(fresh);
                        if (!more) break;
                        ok = ok && issue_dP(it);
                        it.next(a);
                    }
                    if (ok) commit(leader, smem_u32(&bar->acc_full));
                }
                sx.next();
                v++;
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
        uint32_t n = 0;
        int v = 0;
        Stage<C::N2> s2;
        Stage<C::NB> sb;
        const bool storer = w == 0 && lane == 0;  // sends the results of this quarter of the rows
        bool storing = false;                     // and has some on their way, from stationary pair (v - 1) % NX
        auto stored = [&]() {
            if (storer && storing) {
                bulk_wait_read();
                mbar_arrive(smem_u32(&bar->x_free[(v - 1) % C::NX]));
            }
            storing = false;
        };
        for (int i = 0; i < mine; i++) {
            Piece<KEYS> pc;
            if (!pc.template get<32>(&bar->pieces, i, lane, abort_flag, a)) break;
            const DenseSpan sp = pc.sp;
            const int x = pc.x0 + lr;  // stationary row
            uint64_t nl2x2 = 0, ndx2 = 0;
            int kend = 0;
            if constexpr (!KEYS) {
                const long long row = (long long)pc.slice * a.Rp + x;  // Rp is a multiple of 128
                const float nl2 = a.nl2[row], nd = a.nd[row];
                nl2x2 = pack2(nl2, nl2);
                ndx2 = pack2(nd, nd);
                kend = x < a.R ? dense_kend(a, sp, x < a.nq ? x : x % a.nq) : 0;
            }
            Items<KEYS> it = pc.items(a);
            const bool any = !it.done();
            for (; !it.done(); it.next(a), n++) {
                const uint32_t tP = tbase + C::TM_DP + sb.st * 128 + w * kCols + lanes;
                const float* st = stats + s2.st * 2 * BT + w * kCols;  // KEYS: -l2 of these columns' rows; -D BT further
                bar_wait(smem_u32(&bar->s_full), n & 1, abort_flag, a);
                tc_fence_after();
                uint32_t s[kCols];
                tmem_ld32_nowait(tbase + lanes + w * kCols, s);
                if constexpr (KEYS) bar_wait(smem_u32(&bar->y2_full[s2.st]), s2.parity, abort_flag, a);
                tmem_wait_ld();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->s_free), lane);
                stored();
#pragma unroll
                for (int c = 0; c < kCols; c += 4) {
                    uint64_t l0 = nl2x2, l1 = nl2x2;
                    if constexpr (KEYS) {
                        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(st + c);
                        l0 = u.x;
                        l1 = u.y;
                    }
                    float e0, e1, e2, e3;
                    unpack2(fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2x2, l0), e0, e1);
                    unpack2(fma2(pack2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3])), sl2x2, l1), e2, e3);
                    s[c] = __float_as_uint(ex2(e0));
                    s[c + 1] = __float_as_uint(ex2(e1));
                    s[c + 2] = __float_as_uint(ex2(e2));
                    s[c + 3] = __float_as_uint(ex2(e3));
                }
                // which of this thread's columns the mask leaves
                bool masked;
                if constexpr (KEYS) {
                    // the lengths are in l2; causal order cuts where a row's keys end inside the block's keys
                    masked = a.causal && (it.t0 + BT > a.nq || dense_kend(a, sp, it.t0) < pc.x0 + BT);
                    if (masked) {
                        int t = (it.t0 + w * kCols) % a.nq;
#pragma unroll
                        for (int c = 0; c < kCols; c++) {
                            if (x > t + sp.lk - sp.lq) s[c] = 0u;
                            if (++t == a.nq) t = 0;
                        }
                    }
                } else {
                    masked = __any_sync(0xffffffffu, kend - it.pos < BT);
                    if (masked) {
#pragma unroll
                        for (int c = 0; c < kCols; c++)
                            if (w * kCols + c >= kend - it.pos) s[c] = 0u;
                    }
                }
                bar_wait(smem_u32(&bar->dp_full[sb.st]), sb.parity, abort_flag, a);
                tc_fence_after();
                uint32_t g[kCols];
                tmem_ld32_nowait(tP, g);
                tmem_wait_ld();
                uint32_t o[kCols / 2];
                if constexpr (KEYS) {
#pragma unroll
                    for (int c = 0; c < kCols; c += 2)
                        o[c >> 1] = pack_bf16x2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]));
                    tmem_st16(tP, o);
                }
#pragma unroll
                for (int c = 0; c < kCols; c += 4) {
                    uint64_t d0 = ndx2, d1 = ndx2;
                    if constexpr (KEYS) {
                        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(st + BT + c);
                        d0 = u.x;
                        d1 = u.y;
                    }
                    float e0, e1, e2, e3;
                    unpack2(mul2(add2(pack2(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), d0),
                                 pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1]))), e0, e1);
                    unpack2(mul2(add2(pack2(__uint_as_float(g[c + 2]), __uint_as_float(g[c + 3])), d1),
                                 pack2(__uint_as_float(s[c + 2]), __uint_as_float(s[c + 3]))), e2, e3);
                    if (!KEYS && masked) {  // dP of a key behind the lengths may be anything
                        const int lim = kend - it.pos - w * kCols;
                        e0 = c < lim ? e0 : 0.f;
                        e1 = c + 1 < lim ? e1 : 0.f;
                        e2 = c + 2 < lim ? e2 : 0.f;
                        e3 = c + 3 < lim ? e3 : 0.f;
                    }
                    o[c >> 1] = pack_bf16x2(e0, e1);
                    o[(c >> 1) + 1] = pack_bf16x2(e2, e3);
                }
                tmem_st16(KEYS ? tP + kCols / 2 : tP, o);
                tmem_wait_st();
                tc_fence_before();
                warp_arrive(smem_u32(&bar->ds_ready[sb.st]), lane);
                s2.next();
                sb.next();
            }
            const long long row = (long long)pc.slice * extent + x, all = (long long)a.slices * extent;
            // rows without a gradient hold whatever their padding made: zero
            const bool live = any && (KEYS ? x < sp.lk : kend > 0);
            unsigned char* out = sX + 2 * (v % C::NX) * C::TILE;  // the stationary tiles have been used up
            if (any) {
                bar_wait(smem_u32(&bar->acc_full), v & 1, abort_flag, a);
                tc_fence_after();
            }
#pragma unroll
            for (int k = 0; k < (KEYS ? 2 : 1); k++) {
                const float f = k == 0 ? a.scale : 1.f;
#pragma unroll
                for (int c = w * 16; c < D; c += 64) {
                    float o[16];
                    if (any) tmem_ld16(tbase + C::TM_ACC + k * D + c + lanes, o);
#pragma unroll
                    for (int i = 0; i < 16; i++) o[i] = live ? o[i] * f : 0.f;
                    if (a.splits > 1) {
                        float* dst = a.part + ((k * a.splits + pc.part) * all + row) * a.d + c;
                        if (x < extent)
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                if (c + i < a.d) store4(dst + i, o + i);
                    } else if (any) {
                        put_chunk(out + k * C::TILE + (c / 64) * C::REGION, lr, w * 2, o);
                        put_chunk(out + k * C::TILE + (c / 64) * C::REGION, lr, w * 2 + 1, o + 8);
                    } else if (x < extent) {  // nothing here: zeros, past the tiles that the next piece may be using
                        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(KEYS ? (k == 0 ? a.dk : a.dv) : a.dq) + row * a.d + c;
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            if (c + i < a.d) store4(dst + i, o + i);
                    }
                }
            }
            if (!any) continue;
            tc_fence_before();
            warp_arrive(smem_u32(&bar->acc_free), lane);
            if (a.splits == 1) {
                fence_async_smem();
                named_barrier(1 + (warp & 3), 128);  // the four warps of these 32 rows
                if (storer && x < extent) {
                    for (int k = 0; k < (KEYS ? 2 : 1); k++)
                        for (int c = 0; c < D / 64; c++)
                            tma_store_3d(k == 0 ? &mz1 : &mz2, smem_u32(out + k * C::TILE + c * C::REGION + lr * 128), c * 64, x,
                                         pc.slice);
                    bulk_commit();
                }
            }
            v++;
            storing = true;
            if (C::NX == 1) stored();
        }
        stored();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kWarps) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dense_bwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                    const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                    const __grid_constant__ CUtensorMap zq, const __grid_constant__ CUtensorMap zk,
                    const __grid_constant__ CUtensorMap zv, const __grid_constant__ DenseArgs aq,
                    const __grid_constant__ DenseArgs ak, int key_blocks) {
    const int block = blockIdx.x;
    if (block < key_blocks)
        bwd_side<D, true>(mk, mv, mq, mg, zk, zv, ak, block, key_blocks);
    else
        bwd_side<D, false>(mq, mg, mk, mv, zq, zq, aq, block - key_blocks, (int)gridDim.x - key_blocks);
}

// Resident blocks for the pieces of keys (pk, of ck each) beside those for the pieces
// of rows (pq, of cq): the share under which the last of both ends first. All of
// them, for two launches one after the other, where each side's pieces fill their
// rounds so well that this takes less than the share, `gap` included. In causal
// order pieces differ and even each other out over the rounds.
int share_blocks(long long pk, long long ck, long long pq, long long cq, long long gap, int blocks, bool causal) {
    if (pk + pq <= blocks) return (int)pk;
    auto time = [&](long long pieces, long long each, int b) {
        return causal ? (pieces * each + b - 1) / b : (pieces + b - 1) / b * each;
    };
    int best = blocks;
    long long least = time(pk, ck, blocks) + time(pq, cq, blocks) + gap;
    for (int b = 1; b < blocks; b++) {
        const long long t = std::max(time(pk, ck, b), time(pq, cq, blocks - b));
        if (t < least) {
            least = t;
            best = b;
        }
    }
    return best;
}

template <int D>
int launch(const DenseShape& s, DenseArgs aq, DenseArgs ak, cudaStream_t st) {
    using K = Cfg<D, true>;
    using Q = Cfg<D, false>;
    constexpr int smem = K::SMEM > Q::SMEM ? K::SMEM : Q::SMEM;
    static_assert(smem <= 227 * 1024 && sizeof(Bars) <= 1024, "shared memory budget");
    CUtensorMap mq, mk, mv, mg, zq, zk, zv;
    LLSA_TRY(make_tmap_rows(&mq, aq.q, s.slices, s.R, s.d, BT));
    LLSA_TRY(make_tmap_rows(&mg, aq.dout, s.slices, s.R, s.d, BT));
    LLSA_TRY(make_tmap_rows(&mk, aq.k, s.slices, s.nk, s.d, BT));
    LLSA_TRY(make_tmap_rows(&mv, aq.v, s.slices, s.nk, s.d, BT));
    LLSA_TRY(make_tmap_rows(&zq, aq.dq, s.slices, s.R, s.d, 32));
    LLSA_TRY(make_tmap_rows(&zk, aq.dk, s.slices, s.nk, s.d, 32));
    LLSA_TRY(make_tmap_rows(&zv, aq.dv, s.slices, s.nk, s.d, 32));
    cudaFuncSetAttribute(dense_bwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    const long long pq = (long long)((s.R + BT - 1) / BT) * s.slices * aq.splits;
    const long long pk = (long long)((s.nk + BT - 1) / BT) * s.slices * ak.splits;
    if (pq + pk > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    aq.pieces = (int)pq;
    ak.pieces = (int)pk;
    // A block per piece, dealt out by the hardware, where a resident one would wait for its
    // next stationary tiles: 16 heads over 4 of 4,095 tokens 312 us against 379, 19 slices of
    // 16,384 5,121 against 5,154 (4 x 12 heads x 4,096 queries x 333 keys 161 against 152).
    if constexpr (K::NX == 1) {
        LLSA_LAUNCH("dense_bwd_tc", st, dense_bwd_tc_kernel<D><<<(unsigned)(pq + pk), kThreads, smem, st>>>(
                                            mq, mg, mk, mv, zq, zk, zv, aq, ak, (int)pk));
        return LLSA_OK;
    }
    // An item of keys takes 0.77 us, one of rows 0.72 us (19 slices of 16,384 tokens), a
    // piece about three items' time more (152 slices with one item per piece), and
    // a second launch that of seven.
    const long long ck = 16 * ((std::min(ak.chunk, s.R) + BT - 1) / BT + 3), cq = 15 * ((std::min(aq.chunk, s.nk) + BT - 1) / BT + 3);
    const int grid = resident_blocks(pq + pk);
    const int share = share_blocks(pk, ck, pq, cq, 7 * 16, grid, s.causal);
    LLSA_LAUNCH("dense_bwd_tc", st,
                dense_bwd_tc_kernel<D><<<grid, kThreads, smem, st>>>(mq, mg, mk, mv, zq, zk, zv, aq, ak, share));
    if (share == grid)
        LLSA_LAUNCH("dense_bwd_tc", st,
                    dense_bwd_tc_kernel<D><<<grid, kThreads, smem, st>>>(mq, mg, mk, mv, zq, zk, zv, aq, ak, 0));
    return LLSA_OK;
}

}  // namespace

DenseSplit dense_tc_dq_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.R + BT - 1) / BT), s.nk, BT, 2);
}
DenseSplit dense_tc_dkv_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.nk + BT - 1) / BT), s.R, BT, 2);
}

int launch_dense_tc_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, cudaStream_t st) {
    return s.d <= 64 ? launch<64>(s, aq, ak, st) : launch<128>(s, aq, ak, st);
}

}  // namespace llsa

// dense_fwd_tc.cu -- dense attention forward on the tcgen05 tensor cores (bf16,
// d <= 128; the tiles hold 64 or 128 columns, TMA fills the rest with zeros).
//
// Mathematics: one pass over the keys. For a tile of 128 keys S = Q K^T; a row
// keeps a reference m (in units of log2, scaled), the sum l of 2^(s - m) and
// O = sum 2^(s - m) v. m follows the row's maximum lazily: it moves only when
// the maximum has passed it by more than 2^8, and l and O are rescaled then.
// Softmax does not depend on m, P = 2^(s - m) <= 2^8 has the same relative
// rounding in bf16 whatever its size, and sums are fp32, so this costs no
// precision; it saves reading O back for almost every tile. P is rounded to bf16,
// the type that P V has beside bf16 inputs; l sums it before that.
//
// A block takes 256 query rows as two tiles of 128 against a shared stream of
// key and value tiles, the two taking turns on the tensor cores. A thread holds
// its whole row of S in registers, so S may be overwritten as soon as it is read.
// At 64 columns of d tensor memory has room for P beside S (2 x (128 + 64) columns
// and 2 x 64 of O): the next S of a row tile is made while its softmax runs, and
// neither waits for the other. At 128 columns P lies over S, and goes to the
// tensor cores in two halves, so that P V begins while the second half is made.
//
// One block per SM stays for the whole call and takes its share of the work:
// while the softmax warps finish one piece (the last sums, the division, the
// stores), the others load and multiply for the next (figures at the launch).
//
// Bound by the tensor cores and the exponentials, which at 64 columns take the same
// time (an exponential is 4 clocks per warp and quarter of an SM: 512 clocks per 128 x
// 128 scores, as its two products do). 19 slices of 16,384 tokens: 988 us at d = 64
// (1,322 TFLOP/s of the 4 d operations per pair), 1,560 us at d = 128 (1,670).
//
// Roles: warps 0-3 and 4-7 softmax and epilogue (a thread per row of their
// tile), warps 8 and 9 issue the MMAs, warps 10 and 11 the copies of K and V.
#include <algorithm>
#include <type_traits>

#include "dense_tc.cuh"

namespace llsa {
namespace {

using namespace tc;

// 12 warps of 168 registers at launch = 64,512: 256 softmax threads take 216 of
// them, the 128 others keep 72.
constexpr int kThreads = 384, kRegsSoftmax = 216, kRegsOther = 72;
constexpr int BM = 128, BN = 128;

template <int D>
struct Cfg {
    static constexpr int TILE = 128 * D * 2;  // bytes of 128 rows
    static constexpr int REGION = 128 * 128;  // bytes of 128 rows x 64 columns
    static constexpr int STAGES = D == 64 ? 4 : 2;  // of K, and of V
    static constexpr int NQ = D == 64 ? 2 : 1;      // query tiles kept per row tile: the next piece's comes in early
    static constexpr bool APART = D == 64;          // P beside S
    static constexpr int HALVES = APART ? 1 : 2;    // parts in which P is handed over
    static constexpr int SMEM = 1024 + (2 * NQ + 2 * STAGES) * TILE + 1024;
    // tensor-memory columns: S of row tile w at 128 w
    static constexpr int TM_P = APART ? 256 : 0, P_STEP = APART ? 64 : 128, TM_O = APART ? 384 : 256;
};

struct Bars {
    uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], q_full[2][2], q_free[2][2];
    uint64_t s_full[2], s_free[2], p_full[2][2], o_done[2], o_free[2], drain[2];
    PieceRing pieces;
    uint32_t tmem_slot;
    int abort_flag;
};

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// One piece of work: 256 query rows of a slice against a part of its keys, or
// 128 of them where halves fill a round of blocks better.
struct Piece {
    int slice, r0, part, j_first, n[2], nt;  // n: key tiles of each row tile (-1: not there), nt: of both
    DenseSpan sp;

    __device__ __forceinline__ void make(const DenseArgs& a, int id) {
        const bool half = id >= a.whole;
        const DenseWork w = dense_work(a, half ? a.whole + (id - a.whole) / 2 : id, (a.R + 2 * BM - 1) / (2 * BM));
        slice = w.slice;
        part = w.part;
        // causal order gives the last rows the most keys: those come first
        r0 = (a.causal ? w.blocks - 1 - w.block : w.block) * 2 * BM + (half ? ((id - a.whole) & 1) * BM : 0);
        sp = dense_span(a, slice);
        j_first = part * a.chunk;
        const int j_stop = a.splits > 1 ? j_first + a.chunk : a.nk;
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const int row = r0 + w * BM;
            const int end = row < a.R ? min(dense_tile_kend(a, sp, row < a.nq ? row : row % a.nq, BM), j_stop) : 0;
            n[w] = end > j_first ? (end - j_first + BN - 1) / BN : 0;
        }
        if (half) n[1] = -1;
        nt = max(n[0], n[1]);
    }
    __device__ __forceinline__ bool put(PieceRing* ring, int i, volatile int* abort_flag, const DenseArgs& a) const {
        return piece_put(ring, i, make_int4(slice, r0, part, j_first), make_int4(n[0], n[1], sp.lq, sp.lk), abort_flag, a);
    }
    template <int LANES>
    __device__ __forceinline__ bool get(PieceRing* ring, int i, int lane, volatile int* abort_flag, const DenseArgs& a) {
        int4 x, y;
        if (!piece_get<LANES>(ring, i, x, y, lane, abort_flag, a)) return false;
        slice = x.x;
        r0 = x.y;
        part = x.z;
        j_first = x.w;
        n[0] = y.x;
        n[1] = y.y;
        nt = max(n[0], n[1]);
        sp.lq = y.z;
        sp.lk = y.w;
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dense_fwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                    const __grid_constant__ DenseArgs a) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sQ = sm;  // [NQ][2] tiles
    unsigned char* sK = sm + 2 * C::NQ * C::TILE;
    unsigned char* sV = sK + C::STAGES * C::TILE;
    Bars* bar = reinterpret_cast<Bars*>(sV + C::STAGES * C::TILE);
    volatile int* abort_flag = &bar->abort_flag;
    // broadcast, so that the compiler knows these as the same in a whole warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    const int mine = dealt_pieces(a, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; i++) {
            mbar_init(smem_u32(&bar->k_full[i]), 1);
            mbar_init(smem_u32(&bar->k_empty[i]), 1);
            mbar_init(smem_u32(&bar->v_full[i]), 1);
            mbar_init(smem_u32(&bar->v_empty[i]), 1);
        }
        for (int w = 0; w < 2; w++) {
            for (int q = 0; q < 2; q++) {
                mbar_init(smem_u32(&bar->q_full[w][q]), 1);
                mbar_init(smem_u32(&bar->q_free[w][q]), 4);
                mbar_init(smem_u32(&bar->p_full[w][q]), 4);
            }
            mbar_init(smem_u32(&bar->s_full[w]), 1);
            mbar_init(smem_u32(&bar->s_free[w]), 4);
            mbar_init(smem_u32(&bar->o_done[w]), 1);
            mbar_init(smem_u32(&bar->o_free[w]), 4);
            mbar_init(smem_u32(&bar->drain[w]), 1);
        }
        piece_ring_init(&bar->pieces, C::APART ? 11 : 10);  // softmax warps, issuers, the copies of V
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    if (warp == 11 && lane == 0) {
        prefetch_map(&mq);
        prefetch_map(&mk);
        prefetch_map(&mv);
        prefetch_map(&mo);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_slot, 0);

    // Every role walks the block's pieces. What is counted on through them: the
    // ring's stages, the items of a row tile (u), and the pieces in which a row
    // tile has work (v), which is when its query buffer and its O are used.
    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp >= 10) {
            // ------------------------------------------------------- copies
            if (lane == 0 && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const bool keys = warp == 10;
                unsigned char* ring = keys ? sK : sV;
                uint64_t* full = keys ? bar->k_full : bar->v_full;
                uint64_t* empty = keys ? bar->k_empty : bar->v_empty;
                const CUtensorMap* map = keys ? &mk : &mv;
                Stage<C::STAGES> s;
                int filled = 0, v[2] = {0, 0};
                bool ok = true;
                for (int i = 0; ok && i < mine; i++) {
                    Piece pc;
                    if (keys) {
                        pc.make(a, dealt(a, i, blockIdx.x, gridDim.x));
                        ok = pc.put(&bar->pieces, i, abort_flag, a);
                    } else {
                        ok = pc.get<1>(&bar->pieces, i, lane, abort_flag, a);
                    }
                    if (keys)
#pragma unroll
                        for (int w = 0; w < 2; w++) {
                            if (!ok || pc.n[w] <= 0) continue;  // no keys, or half a piece: no query tile
                            const int q = v[w] % C::NQ, use = v[w] / C::NQ;
                            if (use > 0) ok = bar_wait(smem_u32(&bar->q_free[w][q]), (use - 1) & 1, abort_flag, a);
                            if (!ok) continue;
                            const uint32_t qb = smem_u32(&bar->q_full[w][q]);
                            mbar_arrive_expect_tx(qb, C::TILE);
                            for (int c = 0; c < D / 64; c++)
                                tma_load_3d(smem_u32(sQ + (2 * q + w) * C::TILE + c * C::REGION), &mq, c * 64, pc.r0 + w * BM,
                                            pc.slice, qb);
                            v[w]++;
                        }
                    for (int t = 0; ok && t < pc.nt; t++, s.next()) {
                        if (filled >= C::STAGES) ok = bar_wait(smem_u32(&empty[s.st]), s.parity ^ 1, abort_flag, a);
                        if (!ok) break;
                        const uint32_t fb = smem_u32(&full[s.st]);
                        mbar_arrive_expect_tx(fb, C::TILE);
                        for (int c = 0; c < D / 64; c++)
                            tma_load_3d(smem_u32(ring + s.st * C::TILE + c * C::REGION), map, c * 64, pc.j_first + t * BN,
                                        pc.slice, fb);
                        filled++;
                    }
                }
                // copies still in flight must land before the block exits
                for (int x = max(0, filled - C::STAGES); x < filled; x++)
                    land(smem_u32(&full[x % C::STAGES]), (x / C::STAGES) & 1);
                if (keys)
                    for (int w = 0; w < 2; w++)
                        for (int x = max(0, v[w] - C::NQ); x < v[w]; x++)
                            land(smem_u32(&bar->q_full[w][x % C::NQ]), (x / C::NQ) & 1);
            }
        } else {
            // ---------------------------------------------- S and O issuers
            // With P beside S the two products of a row tile do not meet in
            // tensor memory, and warp 8 issues S, warp 9 O += P V. With P over S,
            // warp 8 issues both, a row tile's next S right behind the product that
            // uses up its P: the tensor cores run them in that order, with no wait
            // in between.
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BM, BN, 0, 0), idO = idesc_bf16(BM, D, 0, 1);
            const uint64_t dQ = desc_sw128(smem_u32(sQ), 16, 1024), dK = desc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t dV = desc_sw128(smem_u32(sV), C::REGION, 1024);
            auto issue = [&](auto with_s, auto with_o) {
                constexpr bool does_s = decltype(with_s)::value, does_o = decltype(with_o)::value;
                bool ok = true;
                Stage<C::STAGES> sk, sv;
                int u[2] = {0, 0}, v[2] = {0, 0};  // u: of the products that this warp issues last (S, or O)
                auto issue_s = [&](int w, int q) {
                    tc_fence_after();
                    const uint64_t dA = dQ + ((2 * q + w) * C::TILE >> 4), dT = dK + (sk.st * C::TILE >> 4);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ks++) {
                        const uint32_t off = (ks / 4) * C::REGION + (ks % 4) * 32;
                        mma_ss(leader, tbase + w * 128, dA + (off >> 4), dT + (off >> 4), idS, ks > 0);
                    }
                    commit(leader, smem_u32(&bar->s_full[w]));
                };
                for (int i = 0; ok && i < mine; i++) {
                    Piece pc;
                    ok = pc.get<32>(&bar->pieces, i, lane, abort_flag, a);
                    if (!ok) break;
                    // key tile t: its S (APART), or its O and the S of tile t + 1
                    for (int t = C::APART ? 0 : -1; ok && t < pc.nt; t++) {
                        const int ts = C::APART ? t : t + 1;  // tile of S
                        const bool s_here = does_s && ts < pc.nt, o_here = does_o && t >= 0;
                        if (s_here) ok = warp_wait(smem_u32(&bar->k_full[sk.st]), sk.parity, abort_flag, a);
                        if (ok && o_here) {
                            ok = warp_wait(smem_u32(&bar->v_full[sv.st]), sv.parity, abort_flag, a);
                            // values behind the last valid key may be anything: their weights are 0, so they must be finite
                            const int live = pc.sp.lk - (pc.j_first + t * BN);
                            if (ok && live < BN) {
                                unsigned char* v0 = sV + sv.st * C::TILE;
                                for (int c = 0; c < D / 64; c++)
                                    for (int x = live * 8 + lane; x < BN * 8; x += 32)
                                        *reinterpret_cast<uint4*>(v0 + c * C::REGION + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                                fence_async_smem();
                                __syncwarp();
                            }
                        }
#pragma unroll
                        for (int w = 0; w < 2; w++) {
                            if (o_here && t < pc.n[w]) {
                                if (ok && t == 0 && v[w] > 0) ok = warp_wait(smem_u32(&bar->o_free[w]), (v[w] - 1) & 1, abort_flag, a);
                                const uint64_t dT = dV + (sv.st * C::TILE >> 4);
#pragma unroll
                                for (int h = 0; h < C::HALVES; h++) {
                                    ok = ok && warp_wait(smem_u32(&bar->p_full[w][h]), u[w] & 1, abort_flag, a);
                                    if (!ok) continue;
                                    tc_fence_after();
#pragma unroll
                                    for (int ks = h * 8 / C::HALVES; ks < (h + 1) * 8 / C::HALVES; ks++)
                                        mma_ts(leader, tbase + C::TM_O + w * D, tbase + C::TM_P + w * C::P_STEP + 8 * ks,
                                               dT + (ks * 2048 >> 4), idO, t > 0 || ks > 0);
                                }
                                if (ok) commit(leader, smem_u32(&bar->o_done[w]));
                                u[w]++;
                            }
                            if (s_here && ts < pc.n[w]) {
                                const int q = v[w] % C::NQ;
                                if (ok && ts == 0) ok = warp_wait(smem_u32(&bar->q_full[w][q]), (v[w] / C::NQ) & 1, abort_flag, a);
                                if (C::APART) {  // the last S is read
                                    if (ok && u[w] > 0) ok = warp_wait(smem_u32(&bar->s_free[w]), (u[w] - 1) & 1, abort_flag, a);
                                    u[w]++;
                                }
                                if (ok) issue_s(w, q);
                            }
                        }
                        if (s_here) {
                            if (ok) commit(leader, smem_u32(&bar->k_empty[sk.st]));
                            sk.next();
                        }
                        if (o_here) {
                            if (ok) commit(leader, smem_u32(&bar->v_empty[sv.st]));
                            sv.next();
                        }
                    }
#pragma unroll
                    for (int w = 0; w < 2; w++) v[w] += pc.n[w] > 0;
                }
            };
            if constexpr (C::APART) {
                if (warp == 8) issue(std::true_type{}, std::false_type{});
                else issue(std::false_type{}, std::true_type{});
            } else if (warp == 8) {
                issue(std::true_type{}, std::true_type{});
            }
            // no MMA may be in flight when tensor memory is released
            commit(leader, smem_u32(&bar->drain[warp - 8]));
            if (lane == 0) land(smem_u32(&bar->drain[warp - 8]), 0);
            __syncwarp();
        }
    } else {
        // ----------------------------------------------- softmax, epilogue
        regs_inc<kRegsSoftmax>();
        const int w = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tbase + w * 128 + lanes, tP = tbase + C::TM_P + w * C::P_STEP + lanes;
        const uint32_t tO = tbase + C::TM_O + w * D + lanes;
        const int lr = (warp & 3) * 32 + lane;  // row of the tile
        const float sl2 = a.scale * kDenseLog2e;
        const uint64_t sl2x2 = pack2(sl2, sl2);
        int u = 0, v = 0;
        auto stored = [&]() {  // the last results have left query buffer (v - 1) % NQ
            if (lane == 0) {
                bulk_wait_read();
                mbar_arrive(smem_u32(&bar->q_free[w][(v - 1) % C::NQ]));
            }
        };
        for (int i = 0; i < mine; i++) {
            // what only the epilogue needs is read again there: the registers hold a row of S
            const int slot = i % kPieceSlots;
            if (!warp_wait(smem_u32(&bar->pieces.full[slot]), (i / kPieceSlots) & 1, abort_flag, a)) break;
            const int4 head = bar->pieces.slot[slot][0], tail = bar->pieces.slot[slot][1];
            const int n = w == 0 ? tail.x : tail.y;
            int lim;  // keys that this row sees from the current tile on
            {
                const int r = head.y + w * BM + lr;
                DenseSpan sp;
                sp.lq = tail.z;
                sp.lk = tail.w;
                lim = (r < a.R ? dense_kend(a, sp, r < a.nq ? r : r % a.nq) : 0) - head.w;
            }
            float m = -INFINITY;
            uint64_t l4[2] = {0ull, 0ull};  // the row's sum in four parts
            for (int t = 0; t < n; t++, u++, lim -= BN) {
                bar_wait(smem_u32(&bar->s_full[w]), u & 1, abort_flag, a);
                tc_fence_after();
                uint32_t s[128];
#pragma unroll
                for (int c = 0; c < 4; c++) tmem_ld32_nowait(tS + 32 * c, s + 32 * c);
                tmem_wait_ld();
                if (C::APART) {
                    tc_fence_before();
                    warp_arrive(smem_u32(&bar->s_free[w]), lane);
                }
                if (C::NQ > 1 && t == 0 && v > 0) stored();
                if (__any_sync(0xffffffffu, lim < BN)) {
#pragma unroll
                    for (int q = 0; q < 128; q += 32)
                        if (__any_sync(0xffffffffu, lim < q + 32))
#pragma unroll
                            for (int c = q; c < q + 32; c++) s[c] = c < lim ? s[c] : 0xff800000u;
                }
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < 128; c += 8)
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        x[i] = max3(x[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * sl2;
                const bool grow = top > m + 8.f;
                if (__any_sync(0xffffffffu, grow)) {
                    const float f = grow ? ex2(m - top) : 1.f;  // 2^-inf = 0 at a row's first keys
                    if (grow) m = top;
                    const uint64_t f2 = pack2(f, f);
                    l4[0] = mul2(l4[0], f2);
                    l4[1] = mul2(l4[1], f2);
                    if (t > 0) {
                        bar_wait(smem_u32(&bar->o_done[w]), (u - 1) & 1, abort_flag, a);  // O is at rest
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < D; c += 32) {
                            uint32_t o[32];
                            tmem_ld32_nowait(tO + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tO + c, o);
                        }
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                const uint64_t shift2 = pack2(shift, shift);
                if (C::APART && u > 0) {  // the last P is used up
                    bar_wait(smem_u32(&bar->o_done[w]), (u - 1) & 1, abort_flag, a);
                    tc_fence_after();
                }
                uint32_t p[64];
#pragma unroll
                for (int c = 0; c < 64; c++) {
                    float e0, e1;
                    unpack2(fma2(pack2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, shift2), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    l4[c & 1] = add2(l4[c & 1], pack2(e0, e1));
                    p[c] = pack_bf16x2(e0, e1);
                    if (c % 16 == 15) tmem_st16(tP + c - 15, p + c - 15);
                    if ((c + 1) % (64 / C::HALVES) == 0) {
                        tmem_wait_st();
                        tc_fence_before();
                        warp_arrive(smem_u32(&bar->p_full[w][c / (64 / C::HALVES)]), lane);
                    }
                }
            }
            float l0, l1, l2, l3;
            unpack2(l4[0], l0, l1);
            unpack2(l4[1], l2, l3);
            const float l = (l0 + l1) + (l2 + l3);
            const float inv = l == 0.f ? 0.f : a.splits > 1 ? 1.f : 1.f / l;
            const int4 piece = bar->pieces.slot[slot][0];  // slice, first row, part
            const int r = piece.y + w * BM + lr;
            const long long row = (long long)piece.x * a.R + r, prow = (long long)piece.z * a.slices * a.R + row;
            warp_arrive(smem_u32(&bar->pieces.free[slot]), lane);
            if (n < 0) continue;  // half a piece: the other half's rows
            if (r < a.R) {
                if (a.splits > 1)
                    reinterpret_cast<float2*>(a.part + (long long)a.splits * a.slices * a.R * a.d)[prow] = make_float2(m, l);
                else
                    a.lse_out[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            }
            if (n == 0) {  // no key for these rows
                if (r < a.R)
                    for (int c = 0; c < a.d; c += 8) {
                        const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                        if (a.splits > 1) {
                            store4(a.part + prow * a.d + c, zero);
                            store4(a.part + prow * a.d + c + 4, zero);
                        } else {
                            __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.o_out) + row * a.d + c;
                            store4(dst, zero);
                            store4(dst + 4, zero);
                        }
                    }
                continue;
            }
            bar_wait(smem_u32(&bar->o_done[w]), (u - 1) & 1, abort_flag, a);
            tc_fence_after();
            // the query tile has been used up: its place takes the output rows, 32 of them per warp
            unsigned char* out = sQ + (2 * (v % C::NQ) + w) * C::TILE;
#pragma unroll
            for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32_nowait(tO + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) f[e] = __uint_as_float(o[i + e]) * inv;
                    if (a.splits == 1) {
                        put_chunk(out + (c / 64) * C::REGION, lr, (c % 64 + i) / 8, f);
                    } else if (r < a.R && c + i < a.d) {
                        float* dst = a.part + prow * a.d + c + i;
                        store4(dst, f);
                        store4(dst + 4, f + 4);
                    }
                }
            }
            tc_fence_before();
            warp_arrive(smem_u32(&bar->o_free[w]), lane);
            if (a.splits == 1) {
                fence_async_smem();
                __syncwarp();
                if (lane == 0 && r < a.R) {
                    for (int c = 0; c < D / 64; c++)
                        tma_store_3d(&mo, smem_u32(out + c * C::REGION + lr * 128), c * 64, r, piece.x);
                    bulk_commit();
                }
            }
            v++;
            if (C::NQ == 1) stored();  // the next query tile waits for the place
        }
        if (C::NQ > 1 && v > 0) stored();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <int D>
int launch(const DenseShape& s, DenseArgs a, cudaStream_t st) {
    using C = Cfg<D>;
    static_assert(C::SMEM <= 227 * 1024 && sizeof(Bars) <= 1024, "shared memory budget");
    CUtensorMap mq, mk, mv, mo;
    LLSA_TRY(make_tmap_rows(&mq, a.q, s.slices, s.R, s.d, BM));
    LLSA_TRY(make_tmap_rows(&mk, a.k, s.slices, s.nk, s.d, BN));
    LLSA_TRY(make_tmap_rows(&mv, a.v, s.slices, s.nk, s.d, BN));
    LLSA_TRY(make_tmap_rows(&mo, a.o_out, s.slices, s.R, s.d, 32));
    cudaFuncSetAttribute(dense_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    long long pieces = (long long)((s.R + 2 * BM - 1) / (2 * BM)) * s.slices * a.splits;
    if (pieces > kDenseMaxPieces / 2) return LLSA_ERR_UNSUPPORTED;
    // A last round that leaves half of the SMs idle is dealt out in halves: a row
    // tile alone takes about 3/4 of the time of two.
    const int sms = sm_count();
    const long long rest = pieces % sms;
    a.whole = (int)(2 * rest <= sms && a.splits == 1 ? pieces - rest : pieces);
    pieces += pieces - a.whole;
    a.pieces = (int)pieces;
    // resident blocks against one per piece: 12 heads x 4,096 tokens 61.0 us and 63.3, 4 x 12 heads x 4,096
    // queries x 333 keys 33.7 and 43.1; at 128 columns 88.0 and 88.7, 50.6 and 58.0
    const int grid = resident_blocks(pieces);
    LLSA_LAUNCH("dense_fwd_tc", st, dense_fwd_tc_kernel<D><<<grid, kThreads, C::SMEM, st>>>(mq, mk, mv, mo, a));
    return LLSA_OK;
}

}  // namespace

bool dense_tc_supported(const DenseShape& s) {
    return s.dtype == LLSA_DTYPE_BF16 && s.d <= 128 && s.R > 0 && s.nk > 0;
}

DenseSplit dense_tc_fwd_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.R + 2 * BM - 1) / (2 * BM)), s.nk, BN, 8);
}

int launch_dense_tc_fwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    return s.d <= 64 ? launch<64>(s, a, st) : launch<128>(s, a, st);
}

}  // namespace llsa

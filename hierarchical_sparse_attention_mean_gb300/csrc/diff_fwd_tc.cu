// diff_fwd_tc.cu -- differential attention forward on the tcgen05 tensor cores (bf16; the
// tiles hold 64 or 128 columns of q and k, TMA fills the rest with zeros).
//
// Mathematics: one pass over the keys for both maps. For a tile of 128 keys
// S_i = Q_i K_i^T; each map's row keeps a reference m_i, the sum l_i of 2^(s - m_i) and
// O_i = sum 2^(s - m_i) v, with the lazy m of dense attention (dense_fwd_tc.cu). At the
// end o = O_1 / l_1 - lam O_2 / l_2, formed in fp32 and rounded once: rounded apart, two
// maps that attend alike would leave the roundings of what cancels. P is rounded to bf16,
// the type that P V has beside bf16 inputs; l sums it before that.
//
// The two maps take the places that dense attention gives to two row tiles: a block
// takes 128 query rows, the maps take turns on the tensor cores, each with its own stream
// of key tiles and both with the same value tiles, which are loaded once. Tensor memory
// is full: S of both maps (2 x 128 columns, P over S, handed over in two halves) and 128
// columns of both O. Values of more than 128 columns (d > 64) go in halves of 128, a
// piece of work each, whose scores are made twice: 16 d operations per pair of a query
// and a key instead of 12 d.
//
// Bound by the tensor cores: 1,536 clocks per 128 x 128 pairs at 64 columns, where the
// exponentials of both maps take 1,024. 19 heads x 16,384 tokens of 64 columns: 2,359 us, 1,660
// TFLOP/s, 85 % of what a large matrix product was measured at; of 128 columns 6,340 us, 1,648
// TFLOP/s of the 16 d. 2 x 6 x 4,096 tokens, d = 64: 121 us, 384 pieces in three rounds of 152.
// S and P of 64 keys in two places per map, so that a map's products run beside its own
// exponentials, took 138 against 126 with cold caches: S of 64 keys reads shared memory 1.5 times as much as S of 128.
// A piece's end behind the first tile of the next, with a place for the output rows taken from
// the stages of K, took 134 against 128.
//
// One block per SM stays for the whole call and takes its share of the pieces: while
// the softmax warps finish one, the others load for the next.
//
// Roles: warps 0-3 and 4-7 softmax of the first and second map and epilogue (a thread
// per row), warp 8 issues the MMAs, warp 10 copies Q and K, warp 11 V.
#include <algorithm>

#include "dense_tc.cuh"
#include "diff.h"

namespace llsa {
namespace {

using namespace tc;

// 12 warps of 168 registers at launch = 64,512: 256 softmax threads take 232 of
// them, the 128 others keep 40. Of a row of S 12 bytes still spill at 64 columns, 52 at 128; with 216
// registers so much does that 2 x 6 x 4,096 tokens take 212 us.
constexpr int kThreads = 384, kRegsSoftmax = 232, kRegsOther = 40;
constexpr int BM = 128, BN = 128, VC = 128;  // rows, keys, columns of V of a piece

template <int D>
struct Cfg {
    static constexpr int REGION = 128 * 128;      // bytes of 128 rows x 64 columns
    static constexpr int TILE = D / 64 * REGION;  // of a tile of Q or K
    static constexpr int VTILE = 2 * REGION;
    static constexpr int NQ = D == 64 ? 2 : 1;    // pairs of query tiles: the next piece's come in early
    static constexpr int NK = D == 64 ? 6 : 3, NV = 2;  // stages of K (a map's tile each), of V
    static constexpr int SMEM = 1024 + 2 * NQ * TILE + NK * TILE + NV * VTILE + 2048;
    static constexpr int TM_O = 256;  // tensor-memory columns: S of map w at 128 w, O at 256 + 128 w
};

struct Bars {
    float l[2][BM];  // the sums of both maps' rows, at the end of a piece
    uint64_t k_full[6], k_empty[6], v_full[2], v_empty[2], q_full[2], q_free[2];
    uint64_t s_full[2], p_full[2][2], o_done[2], o_free[2], l_ready, drain;
    PieceRing pieces;
    uint32_t tmem_slot;
    int abort_flag;
};

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// One piece of work: 128 query rows of a slice against a part of its keys, for 128
// columns of its values.
struct Piece {
    int slice, r0, part, col, j_first, n;
    DenseSpan sp;

    __device__ __forceinline__ void make(const DenseArgs& a, int id, int cols) {
        col = id % cols * VC;
        const DenseWork w = dense_work(a, id / cols, (a.R + BM - 1) / BM);
        slice = w.slice;
        part = w.part;
        // causal order gives the last rows the most keys: those come first
        r0 = (a.causal ? w.blocks - 1 - w.block : w.block) * BM;
        sp = dense_span(a, slice);
        j_first = part * a.chunk;
        const int j_stop = a.splits > 1 ? j_first + a.chunk : a.nk;
        const int end = min(dense_tile_kend(a, sp, r0 < a.nq ? r0 : r0 % a.nq, BM), j_stop);
        n = end > j_first ? (end - j_first + BN - 1) / BN : 0;
    }
    __device__ __forceinline__ bool put(PieceRing* ring, int i, volatile int* abort_flag, const DenseArgs& a) const {
        return piece_put(ring, i, make_int4(slice, r0, part, j_first), make_int4(n, col, sp.lq, sp.lk), abort_flag, a);
    }
    __device__ __forceinline__ void take(int4 x, int4 y) {
        slice = x.x;
        r0 = x.y;
        part = x.z;
        j_first = x.w;
        n = y.x;
        col = y.y;
        sp.lq = y.z;
        sp.lk = y.w;
    }
    template <int LANES>
    __device__ __forceinline__ bool get(PieceRing* ring, int i, int lane, volatile int* abort_flag, const DenseArgs& a) {
        int4 x, y;
        if (!piece_get<LANES>(ring, i, x, y, lane, abort_flag, a)) return false;
        take(x, y);
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
diff_fwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                   const __grid_constant__ CUtensorMap mo2, const __grid_constant__ DiffArgs f) {
    using C = Cfg<D>;
    const DenseArgs& a = f.d;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sQ = sm;  // [NQ][2] tiles
    unsigned char* sK = sm + 2 * C::NQ * C::TILE;
    unsigned char* sV = sK + C::NK * C::TILE;
    Bars* bar = reinterpret_cast<Bars*>(sV + C::NV * C::VTILE);
    volatile int* abort_flag = &bar->abort_flag;
    // broadcast, so that the compiler knows these as the same in a whole warp
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int cols = (2 * a.d + VC - 1) / VC;

    const int mine = dealt_pieces(a, blockIdx.x, gridDim.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < 6; i++) {
            mbar_init(smem_u32(&bar->k_full[i]), 1);
            mbar_init(smem_u32(&bar->k_empty[i]), 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(smem_u32(&bar->v_full[i]), 1);
            mbar_init(smem_u32(&bar->v_empty[i]), 1);
            mbar_init(smem_u32(&bar->q_full[i]), 1);
            mbar_init(smem_u32(&bar->q_free[i]), 8);
            mbar_init(smem_u32(&bar->s_full[i]), 1);
            mbar_init(smem_u32(&bar->p_full[i][0]), 4);
            mbar_init(smem_u32(&bar->p_full[i][1]), 4);
            mbar_init(smem_u32(&bar->o_done[i]), 1);
            mbar_init(smem_u32(&bar->o_free[i]), 8);
        }
        mbar_init(smem_u32(&bar->l_ready), 8);
        mbar_init(smem_u32(&bar->drain), 1);
        piece_ring_init(&bar->pieces, 10);  // softmax warps, the issuer, the copies of V
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    if (warp == 11 && lane == 0) {
        prefetch_map(&mq);
        prefetch_map(&mk);
        prefetch_map(&mv);
        prefetch_map(&mo);
        prefetch_map(&mo2);
    }
    tc_fence_before();
    close_wait();
    __syncthreads();
    tc_fence_after();
    close_ahead();  // the block has its tensor memory
    const uint32_t tbase = __shfl_sync(0xffffffffu, bar->tmem_slot, 0);

    // Every role walks the block's pieces. What is counted on through them: the rings'
    // stages, the key tiles (u), and the pieces that have any (v), which is when query
    // buffers and O are used.
    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp >= 10) {
            // ------------------------------------------------------- copies
            if (lane == 0 && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                const bool keys = warp == 10;
                Stage<C::NK> sk;
                Stage<C::NV> sv;
                int filled = 0, v = 0;
                bool ok = true;
                for (int i = 0; ok && i < mine; i++) {
                    Piece pc;
                    if (keys) {
                        pc.make(a, dealt(a, i, blockIdx.x, gridDim.x), cols);
                        ok = pc.put(&bar->pieces, i, abort_flag, a);
                    } else {
                        ok = pc.get<1>(&bar->pieces, i, lane, abort_flag, a);
                    }
                    if (!ok || pc.n == 0) continue;
                    const int m0 = diff_matrix(a, pc.slice, 0), m1 = m0 + a.kv_heads;
                    if (keys) {
                        const int q = v % C::NQ, use = v / C::NQ;
                        if (use > 0) ok = bar_wait(smem_u32(&bar->q_free[q]), (use - 1) & 1, abort_flag, a);
                        if (!ok) continue;
                        const uint32_t qb = smem_u32(&bar->q_full[q]);
                        mbar_arrive_expect_tx(qb, 2 * C::TILE);
                        for (int w = 0; w < 2; w++)
                            for (int c = 0; c < D / 64; c++)
                                tma_load_3d(smem_u32(sQ + (2 * q + w) * C::TILE + c * C::REGION), &mq, c * 64, pc.r0,
                                            w ? m1 : m0, qb);
                        v++;
                        for (int t = 0; ok && t < 2 * pc.n; t++, sk.next()) {
                            if (filled >= C::NK) ok = bar_wait(smem_u32(&bar->k_empty[sk.st]), sk.parity ^ 1, abort_flag, a);
                            if (!ok) break;
                            const uint32_t fb = smem_u32(&bar->k_full[sk.st]);
                            mbar_arrive_expect_tx(fb, C::TILE);
                            for (int c = 0; c < D / 64; c++)
                                tma_load_3d(smem_u32(sK + sk.st * C::TILE + c * C::REGION), &mk, c * 64,
                                            pc.j_first + (t >> 1) * BN, t & 1 ? m1 : m0, fb);
                            filled++;
                        }
                    } else {
                        for (int t = 0; ok && t < pc.n; t++, sv.next()) {
                            if (filled >= C::NV) ok = bar_wait(smem_u32(&bar->v_empty[sv.st]), sv.parity ^ 1, abort_flag, a);
                            if (!ok) break;
                            const uint32_t fb = smem_u32(&bar->v_full[sv.st]);
                            mbar_arrive_expect_tx(fb, C::VTILE);
                            for (int c = 0; c < 2; c++)
                                tma_load_3d(smem_u32(sV + sv.st * C::VTILE + c * C::REGION), &mv, pc.col + c * 64,
                                            pc.j_first + t * BN, pc.slice, fb);
                            filled++;
                        }
                    }
                }
                // copies still in flight must land before the block exits
                const int ns = keys ? C::NK : C::NV;
                uint64_t* full = keys ? bar->k_full : bar->v_full;
                for (int x = max(0, filled - ns); x < filled; x++) land(smem_u32(&full[x % ns]), (x / ns) & 1);
                if (keys)
                    for (int x = max(0, v - C::NQ); x < v; x++) land(smem_u32(&bar->q_full[x % C::NQ]), (x / C::NQ) & 1);
            }
        } else if (warp == 8) {
            // --------------------------------------------------- MMA issuer
            // A map's next S right behind the product that uses up its P: the tensor
            // cores run them in that order, with no wait in between.
            const uint32_t leader = elect_lane();
            constexpr uint32_t idS = idesc_bf16(BM, BN, 0, 0), idO = idesc_bf16(BM, VC, 0, 1);
            const uint64_t dQ = desc_sw128(smem_u32(sQ), 16, 1024), dK = desc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t dV = desc_sw128(smem_u32(sV), C::REGION, 1024);
            bool ok = true;
            Stage<C::NK> sk;
            Stage<C::NV> sv;
            int u = 0, v = 0;  // u: of the tiles whose O is issued
            for (int i = 0; ok && i < mine; i++) {
                Piece pc;
                ok = pc.get<32>(&bar->pieces, i, lane, abort_flag, a);
                if (!ok || pc.n == 0) continue;
                const int q = v % C::NQ;
                ok = warp_wait(smem_u32(&bar->q_full[q]), (v / C::NQ) & 1, abort_flag, a);
                // key tile t: its O and the S of tile t + 1
                for (int t = -1; ok && t < pc.n; t++) {
                    if (t >= 0) {
                        ok = warp_wait(smem_u32(&bar->v_full[sv.st]), sv.parity, abort_flag, a);
                        // values behind the last valid key may be anything: their weights are 0, so they must be finite
                        const int live = pc.sp.lk - (pc.j_first + t * BN);
                        if (ok && live < BN) {
                            unsigned char* v0 = sV + sv.st * C::VTILE;
                            for (int c = 0; c < 2; c++)
                                for (int x = live * 8 + lane; x < BN * 8; x += 32)
                                    *reinterpret_cast<uint4*>(v0 + c * C::REGION + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                            fence_async_smem();
                            __syncwarp();
                        }
                    }
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        if (t >= 0) {
                            if (ok && t == 0 && v > 0) ok = warp_wait(smem_u32(&bar->o_free[w]), (v - 1) & 1, abort_flag, a);
                            const uint64_t dT = dV + (sv.st * C::VTILE >> 4);
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                ok = ok && warp_wait(smem_u32(&bar->p_full[w][h]), u & 1, abort_flag, a);
                                if (!ok) continue;
                                tc_fence_after();
#pragma unroll
                                for (int ks = 4 * h; ks < 4 * h + 4; ks++)
                                    mma_ts(leader, tbase + C::TM_O + w * VC, tbase + w * 128 + 8 * ks, dT + (ks * 2048 >> 4), idO,
                                           t > 0 || ks > 0);
                            }
                            if (ok) commit(leader, smem_u32(&bar->o_done[w]));
                        }
                        if (ok && t + 1 < pc.n) {
                            ok = warp_wait(smem_u32(&bar->k_full[sk.st]), sk.parity, abort_flag, a);
                            if (!ok) continue;
                            tc_fence_after();
                            const uint64_t dA = dQ + ((2 * q + w) * C::TILE >> 4), dT = dK + (sk.st * C::TILE >> 4);
#pragma unroll
                            for (int ks = 0; ks < D / 16; ks++) {
                                const uint32_t off = (ks / 4) * C::REGION + (ks % 4) * 32;
                                mma_ss(leader, tbase + w * 128, dA + (off >> 4), dT + (off >> 4), idS, ks > 0);
                            }
                            commit(leader, smem_u32(&bar->s_full[w]));
                            commit(leader, smem_u32(&bar->k_empty[sk.st]));
                            sk.next();
                        }
                    }
                    if (t >= 0) {
                        if (ok) commit(leader, smem_u32(&bar->v_empty[sv.st]));
                        sv.next();
                        u++;
                    }
                }
                v++;
            }
            // no MMA may be in flight when tensor memory is released
            commit(leader, smem_u32(&bar->drain));
            if (lane == 0) land(smem_u32(&bar->drain), 0);
            __syncwarp();
        }
    } else {
        // ----------------------------------------------- softmax, epilogue
        regs_inc<kRegsSoftmax>();
        const int w = warp >> 2;  // map; in the epilogue, half of the columns
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tbase + w * 128 + lanes, tO = tbase + C::TM_O + lanes;
        const int lr = (warp & 3) * 32 + lane;  // row of the tile
        const float sl2 = a.scale * kDenseLog2e;
        const uint64_t sl2x2 = pack2(sl2, sl2);
        int u = 0, v = 0;
        auto stored = [&]() {  // this warp's last results have left query buffer (v - 1) % NQ
            if (lane == 0) {
                bulk_wait_read();
                mbar_arrive(smem_u32(&bar->q_free[(v - 1) % C::NQ]));
            }
        };
        for (int i = 0; i < mine; i++) {
            // what only the epilogue needs is read again there: the registers hold a row of S
            const int slot = i % kPieceSlots;
            if (!warp_wait(smem_u32(&bar->pieces.full[slot]), (i / kPieceSlots) & 1, abort_flag, a)) break;
            const int4 head = bar->pieces.slot[slot][0], tail = bar->pieces.slot[slot][1];
            const int n = tail.x;
            int lim;  // keys that this row sees from the current tile on
            {
                const int r = head.y + lr;
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
                    const float g = grow ? ex2(m - top) : 1.f;  // 2^-inf = 0 at a row's first keys
                    if (grow) m = top;
                    const uint64_t g2 = pack2(g, g);
                    l4[0] = mul2(l4[0], g2);
                    l4[1] = mul2(l4[1], g2);
                    if (t > 0) {
                        bar_wait(smem_u32(&bar->o_done[w]), (u - 1) & 1, abort_flag, a);  // O is at rest
                        tc_fence_after();
#pragma unroll
                        for (int c = 0; c < VC; c += 32) {
                            uint32_t o[32];
                            tmem_ld32_nowait(tO + w * VC + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; i++) o[i] = __float_as_uint(__uint_as_float(o[i]) * g);
                            tmem_st32(tO + w * VC + c, o);
                        }
                    }
                }
                const float shift = m == -INFINITY ? 0.f : -m;
                const uint64_t shift2 = pack2(shift, shift);
                uint32_t p[64];
#pragma unroll
                for (int c = 0; c < 64; c++) {
                    float e0, e1;
                    unpack2(fma2(pack2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2x2, shift2), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    l4[c & 1] = add2(l4[c & 1], pack2(e0, e1));
                    p[c] = pack_bf16x2(e0, e1);
                    if (c % 16 == 15) tmem_st16(tS + c - 15, p + c - 15);
                    if ((c + 1) % 32 == 0) {
                        tmem_wait_st();
                        tc_fence_before();
                        warp_arrive(smem_u32(&bar->p_full[w][c / 32]), lane);
                    }
                }
            }
            float l0, l1, l2, l3;
            unpack2(l4[0], l0, l1);
            unpack2(l4[1], l2, l3);
            const float l = (l0 + l1) + (l2 + l3);
            Piece pc;
            pc.take(bar->pieces.slot[slot][0], bar->pieces.slot[slot][1]);
            // the slot is free when its numbers have come: an arrival could overtake loads that nothing waits for
            if (__all_sync(0xffffffffu, (pc.col | pc.slice) >= 0)) warp_arrive(smem_u32(&bar->pieces.free[slot]), lane);
            const int r = pc.r0 + lr, dv = 2 * a.d;
            const bool here = r < a.R;
            const long long row = (long long)pc.slice * a.R + r, prow = diff_part(a, pc.part, w, row);
            if (here && pc.col == 0) {
                if (a.splits > 1) diff_part_ml(a)[prow] = make_float2(m, l);
                else a.lse_out[diff_row(f, pc.slice, w, r)] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
            }
            if (n == 0) {  // no key for these rows
                const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                const int stop = min(dv, pc.col + VC);
                if (here) {
                    if (a.splits > 1) {
                        for (int c = pc.col; c < stop; c += 4) store4(a.part + prow * dv + c, zero);
                    } else {
                        for (int c = pc.col + 64 * w; c < min(stop, pc.col + 64 * w + 64); c += 8) {
                            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o_out) + row * dv + c) = make_uint4(0u, 0u, 0u, 0u);
                            if (f.o2_out)
                                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(f.o2_out) + row * dv + c) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                continue;
            }
            float lam = here ? diff_lam(f, diff_head(f, pc.slice, r)) : 0.f;  // comes while O is being finished
            if (a.splits == 1) {
                // l has one place: all warps have read the last piece's sums before they left its O. With one
                // key tile nothing else holds this back, as S waits for no O.
                if (v > 0) bar_wait(smem_u32(&bar->o_free[w]), (v - 1) & 1, abort_flag, a);
                bar->l[w][lr] = l;
                warp_arrive(smem_u32(&bar->l_ready), lane);
            }
            bar_wait(smem_u32(&bar->o_done[w]), (u - 1) & 1, abort_flag, a);
            if (a.splits > 1) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < VC; c += 32) {
                    uint32_t o[32];
                    tmem_ld32_nowait(tO + w * VC + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float y[4] = {__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                            __uint_as_float(o[i + 3])};
                        if (here && pc.col + c + i < dv) store4(a.part + prow * dv + pc.col + c + i, y);
                    }
                }
                tc_fence_before();
                warp_arrive(smem_u32(&bar->o_free[0]), lane);
                warp_arrive(smem_u32(&bar->o_free[1]), lane);
                v++;
                if (C::NQ == 1) stored();
                continue;
            }
            // the sums of both maps, and both O; the query tiles have been used up: their place
            // takes the output rows, 32 rows and 64 columns per warp
            bar_wait(smem_u32(&bar->o_done[w ^ 1]), (u - 1) & 1, abort_flag, a);
            tc_fence_after();
            bar_wait(smem_u32(&bar->l_ready), v & 1, abort_flag, a);
            const float la = bar->l[0][lr], lb = bar->l[1][lr];
            const float inv1 = la == 0.f ? 0.f : 1.f / la, inv2 = lb == 0.f ? 0.f : 1.f / lb;
            if (lb == 0.f) lam = 0.f;  // no key: o is 0 whatever lam is
            unsigned char* out = sQ + 2 * (v % C::NQ) * C::TILE + w * C::REGION;
            unsigned char* out2 = D == 64 ? out : out + C::TILE;
            uint32_t kept[32];  // o2's row, packed
#pragma unroll
            for (int c = 0; c < 64; c += 16) {
                uint32_t x[16], y[16];
                tmem_ld16_nowait(tO + w * 64 + c, x);
                tmem_ld16_nowait(tO + VC + w * 64 + c, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; i += 8) {
                    float p[8], q[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        q[e] = __uint_as_float(y[i + e]) * inv2;
                        p[e] = fmaf(-lam, q[e], __uint_as_float(x[i + e]) * inv1);
                    }
                    put_chunk(out, lr, (c + i) / 8, p);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) kept[(c + i + e) / 2] = pack_bf16x2(q[e], q[e + 1]);
                }
            }
            tc_fence_before();
            warp_arrive(smem_u32(&bar->o_free[0]), lane);
            warp_arrive(smem_u32(&bar->o_free[1]), lane);
            const int col = pc.col + 64 * w;
            const bool sends = lane == 0 && here && col < dv;  // rows behind the slice are dropped
            auto send = [&](const CUtensorMap* map, const unsigned char* from) {
                fence_async_smem();
                __syncwarp();
                if (sends) {
                    tma_store_3d(map, smem_u32(from + lr * 128), col, r, pc.slice);
                    bulk_commit();
                }
            };
            send(&mo, out);
            if (f.o2_out) {
                if (out2 == out) {
                    if (lane == 0) bulk_wait_read();
                    __syncwarp();
                }
#pragma unroll
                for (int c = 0; c < 8; c++)
                    *reinterpret_cast<uint4*>(out2 + lr * 128 + ((c ^ (lr & 7)) << 4)) =
                        make_uint4(kept[4 * c], kept[4 * c + 1], kept[4 * c + 2], kept[4 * c + 3]);
                send(&mo2, out2);
            }
            v++;
            if (C::NQ == 1) stored();  // the next query tiles wait for the place
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
int launch(const DiffShape& s, DiffArgs f, cudaStream_t st) {
    using C = Cfg<D>;
    static_assert(C::SMEM <= 227 * 1024 && sizeof(Bars) <= 2048, "shared memory budget");
    DenseArgs& a = f.d;
    CUtensorMap mq, mk, mv, mo, mo2;
    LLSA_TRY(make_tmap_rows(&mq, a.q, 2LL * s.slices, s.R, s.d, BM));
    LLSA_TRY(make_tmap_rows(&mk, a.k, 2LL * s.slices, s.nk, s.d, BN));
    LLSA_TRY(make_tmap_rows(&mv, a.v, s.slices, s.nk, 2 * s.d, BN));
    LLSA_TRY(make_tmap_rows(&mo, a.o_out, s.slices, s.R, 2 * s.d, 32));
    LLSA_TRY(make_tmap_rows(&mo2, f.o2_out ? f.o2_out : a.o_out, s.slices, s.R, 2 * s.d, 32));
    cudaFuncSetAttribute(diff_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    const long long pieces = (long long)((s.R + BM - 1) / BM) * s.slices * a.splits * ((2 * s.d + VC - 1) / VC);
    if (pieces > kDenseMaxPieces) return LLSA_ERR_UNSUPPORTED;
    a.pieces = (int)pieces;
    const int grid = resident_blocks(pieces);
    LLSA_LAUNCH("diff_fwd_tc", st, launch_close(close_first(st), diff_fwd_tc_kernel<D>, dim3(grid), kThreads, C::SMEM, st, mq, mk, mv, mo, mo2, f));
    return LLSA_OK;
}

}  // namespace

bool diff_tc_supported(const DiffShape& s) { return s.dtype == LLSA_DTYPE_BF16 && s.R > 0 && s.nk > 0; }

DenseSplit diff_tc_fwd_split(const DiffShape& s) {
    return dense_make_split((long long)s.slices * ((s.R + BM - 1) / BM) * ((2 * s.d + VC - 1) / VC), s.nk, BN, 8);
}

int launch_diff_tc_fwd(const DiffShape& s, const DiffArgs& a, cudaStream_t st) {
    return s.d <= 64 ? launch<64>(s, a, st) : launch<128>(s, a, st);
}

}  // namespace llsa

// dense_fwd_tc.cu -- dense attention forward on the tcgen05 tensor cores (bf16,
// d <= 128; the tiles hold 64 or 128 columns, TMA fills the rest with zeros).
//
// Mathematics: one pass over the keys. For a tile of 128 keys S = Q K^T; a row
// keeps a reference m (in units of log2, scaled), the sum l of 2^(s - m) and
// O = sum 2^(s - m) v. m follows the row's maximum lazily: it moves only when
// the maximum has passed it by more than 2^8, and l and O are rescaled then.
// Softmax does not depend on m, P = 2^(s - m) <= 2^8 has the same relative
// rounding in bf16 whatever its size, and sums are fp32, so this costs no
// precision; it saves reading O back for almost every tile.
//
// A block takes 256 query rows as two tiles of 128 against a shared stream of
// key and value tiles. While the softmax of one tile runs, the tensor cores
// work for the other: per tile, in one in-order stream, O += P V, then the next
// S. S and P share tensor memory (a thread holds its whole row of S in
// registers before it writes P); 2 x 128 columns S / P and 2 x D columns O.
//
// Roles: warps 0-3 and 4-7 softmax and epilogue (a thread per row of their
// tile), warp 8 issues the MMAs, warp 9 the copies; warps 10 and 11 only fill
// the warpgroup whose registers the softmax takes over.
#include <algorithm>

#include "dense.h"
#include "tc.cuh"

namespace llsa {
namespace {

using namespace tc;

// 12 warps of 168 registers at launch = 64,512: 256 softmax threads take 208 of
// them, the 128 others keep 88.
constexpr int kThreads = 384, kRegsSoftmax = 208, kRegsOther = 88;
constexpr int BM = 128, BN = 128;

template <int D>
struct Cfg {
    static constexpr int TILE = 128 * D * 2;  // bytes of 128 rows
    static constexpr int REGION = 128 * 128;  // bytes of 128 rows x 64 columns
    static constexpr int STAGES = D == 64 ? 8 : 4;
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE + 1024;
    static constexpr int TM_O = 256;          // tensor-memory columns: S / P at 0 and 128, O behind them
};

struct Bars {
    uint64_t full[8], empty[8], q_full[2], s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem_slot;
    int abort_flag;
};

// A whole warp waits; false as soon as any wait of the block gave up.
__device__ __forceinline__ bool warp_wait(uint32_t mbar, uint32_t parity, volatile int* abort_flag, const DenseArgs& a) {
    return __all_sync(0xffffffffu, mbar_wait(mbar, parity, abort_flag, a.status, a.spin));
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dense_fwd_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ DenseArgs a) {
    using C = Cfg<D>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* sQ = sm;
    unsigned char* ring = sm + 2 * C::TILE;
    Bars* bar = reinterpret_cast<Bars*>(ring + C::STAGES * C::TILE);
    volatile int* abort_flag = &bar->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // blocks of a slice from its last rows to its first: causal order gives those the most keys
    const int blocks = (a.R + 2 * BM - 1) / (2 * BM);
    const int slice = blockIdx.x / blocks;
    const int r0 = (blocks - 1 - (int)(blockIdx.x - slice * blocks)) * 2 * BM;
    const int part = blockIdx.y;
    const DenseSpan sp = dense_span(a, slice);
    const int j_first = part * a.chunk;
    const int j_stop = a.splits > 1 ? j_first + a.chunk : a.nk;
    int n[2];  // key tiles of each row tile
#pragma unroll
    for (int w = 0; w < 2; w++) {
        const int row = r0 + w * BM;
        const int end = row < a.R ? min(dense_tile_kend(a, sp, row % a.nq, BM), j_stop) : 0;
        n[w] = end > j_first ? (end - j_first + BN - 1) / BN : 0;
    }
    const int nt = max(n[0], n[1]);

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; s++) {
            mbar_init(smem_u32(&bar->full[s]), 1);
            mbar_init(smem_u32(&bar->empty[s]), 1);
        }
        for (int w = 0; w < 2; w++) {
            mbar_init(smem_u32(&bar->q_full[w]), 1);
            mbar_init(smem_u32(&bar->s_full[w]), 1);
            mbar_init(smem_u32(&bar->p_full[w]), 128);
            mbar_init(smem_u32(&bar->o_full[w]), 1);
        }
        mbar_init(smem_u32(&bar->drain), 1);
        bar->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) tmem_alloc(smem_u32(&bar->tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = bar->tmem_slot;

    if (warp >= 8) {
        regs_dec<kRegsOther>();
        if (warp == 9) {
            // ----------------------------------------------------------- copies
            // tile sequence K(0), V(0), K(1), V(1), ... through one ring
            if (lane == 0 && !(a.test_flags & LLSA_TEST_NO_COPIES)) {
                for (int w = 0; w < 2; w++)
                    if (n[w] > 0) {
                        mbar_arrive_expect_tx(smem_u32(&bar->q_full[w]), C::TILE);
                        for (int c = 0; c < D / 64; c++)
                            tma_load_3d(smem_u32(sQ + w * C::TILE + c * C::REGION), &mq, c * 64, r0 + w * BM, slice,
                                        smem_u32(&bar->q_full[w]));
                    }
                int s = 0;
                for (; s < 2 * nt; s++) {
                    const int st = s % C::STAGES, use = s / C::STAGES;
                    if (use > 0 && !mbar_wait(smem_u32(&bar->empty[st]), (use - 1) & 1, abort_flag, a.status, a.spin)) break;
                    const uint32_t fb = smem_u32(&bar->full[st]);
                    mbar_arrive_expect_tx(fb, C::TILE);
                    for (int c = 0; c < D / 64; c++)
                        tma_load_3d(smem_u32(ring + st * C::TILE + c * C::REGION), (s & 1) ? &mv : &mk, c * 64,
                                    j_first + (s >> 1) * BN, slice, fb);
                }
                // copies still in flight must land before the block exits
                for (int w = 0; w < 2; w++)
                    if (n[w] > 0)
                        for (int it = 0; it < kSpinLimit && !mbar_try(smem_u32(&bar->q_full[w]), 0); it++) {
                        }
                for (int x = max(0, s - C::STAGES); x < s; x++)
                    for (int it = 0; it < kSpinLimit && !mbar_try(smem_u32(&bar->full[x % C::STAGES]), (x / C::STAGES) & 1);
                         it++) {
                    }
            }
        } else if (warp == 8) {
            // ------------------------------------------------------- MMA issuer
            constexpr uint32_t idS = idesc_bf16(BM, BN, 0, 0), idO = idesc_bf16(BM, D, 0, 1);
            const uint64_t dQ = desc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t dK = desc_sw128(smem_u32(ring), 16, 1024);
            const uint64_t dV = desc_sw128(smem_u32(ring), C::REGION, 1024);
            auto ring_wait = [&](int s) {
                return warp_wait(smem_u32(&bar->full[s % C::STAGES]), (s / C::STAGES) & 1, abort_flag, a);
            };
            auto issue_S = [&](int w, int t) {
                const uint32_t k0 = (uint32_t)((2 * t) % C::STAGES * C::TILE);
    #pragma unroll
                for (int ks = 0; ks < D / 16; ks++) {
                    const uint32_t off = (ks / 4) * C::REGION + (ks % 4) * 32;
                    mma_bf16_warp(tbase + w * 128, dQ + ((w * C::TILE + off) >> 4), dK + ((k0 + off) >> 4), idS, ks > 0);
                }
                mma_commit_warp(smem_u32(&bar->s_full[w]));
            };
            auto issue_O = [&](int w, int t) {
                const uint32_t v0 = (uint32_t)((2 * t + 1) % C::STAGES * C::TILE);
    #pragma unroll
                for (int ks = 0; ks < BN / 16; ks++)
                    mma_bf16_ts_warp(tbase + C::TM_O + w * D, tbase + w * 128 + 8 * ks, dV + ((v0 + ks * 2048) >> 4), idO,
                                     t > 0 || ks > 0);
            };
            bool ok = true;
            if (nt > 0) {
                for (int w = 0; w < 2 && ok; w++)
                    if (n[w] > 0) ok = warp_wait(smem_u32(&bar->q_full[w]), 0, abort_flag, a);
                ok = ok && ring_wait(0);
                if (ok) {
                    tc_fence_after();
                    for (int w = 0; w < 2; w++)
                        if (n[w] > 0) issue_S(w, 0);
                    mma_commit_warp(smem_u32(&bar->empty[0]));
                }
            }
            for (int t = 0; t < nt && ok; t++) {
                bool have_v = false, have_k = false;
                for (int w = 0; w < 2 && ok; w++) {
                    if (t >= n[w]) continue;
                    ok = warp_wait(smem_u32(&bar->p_full[w]), t & 1, abort_flag, a);
                    if (!ok) break;
                    if (!have_v) {
                        ok = ring_wait(2 * t + 1);
                        if (!ok) break;
                        // values behind the last valid key may be anything: their weights are 0, so they must be finite
                        const int live = sp.lk - (j_first + t * BN);
                        if (live < BN) {
                            unsigned char* v0 = ring + (2 * t + 1) % C::STAGES * C::TILE;
                            for (int c = 0; c < D / 64; c++)
                                for (int x = live * 8 + lane; x < BN * 8; x += 32)
                                    *reinterpret_cast<uint4*>(v0 + c * C::REGION + x * 16) = make_uint4(0u, 0u, 0u, 0u);
                            fence_async_smem();
                            __syncwarp();
                        }
                        have_v = true;
                    }
                    tc_fence_after();
                    issue_O(w, t);
                    if (t + 1 == n[w]) {
                        mma_commit_warp(smem_u32(&bar->o_full[w]));
                    } else {
                        if (!have_k) {
                            ok = ring_wait(2 * t + 2);
                            if (!ok) break;
                            tc_fence_after();
                            have_k = true;
                        }
                        issue_S(w, t + 1);
                    }
                }
                if (!ok) break;
                mma_commit_warp(smem_u32(&bar->empty[(2 * t + 1) % C::STAGES]));
                if (t + 1 < nt) mma_commit_warp(smem_u32(&bar->empty[(2 * t + 2) % C::STAGES]));
            }
            // no MMA may be in flight when tensor memory is released
            mma_commit_warp(smem_u32(&bar->drain));
            if (lane == 0)
                for (int it = 0; it < kSpinLimit && !mbar_try(smem_u32(&bar->drain), 0); it++) {
                }
            __syncwarp();
    }
    } else {
        // ----------------------------------------------- softmax, epilogue
        regs_inc<kRegsSoftmax>();
        const int w = warp >> 2;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tbase + w * 128 + lanes, tO = tbase + C::TM_O + w * D + lanes;
        const int r = r0 + w * BM + (warp & 3) * 32 + lane;
        const int kend = r < a.R ? dense_kend(a, sp, r % a.nq) : 0;
        const float sl2 = a.scale * kDenseLog2e;
        const uint64_t sl2x2 = pack2(sl2, sl2);
        float m = -INFINITY;
        uint64_t l4[2] = {0ull, 0ull};  // the row's sum in four parts
        for (int t = 0; t < n[w]; t++) {
            mbar_wait(smem_u32(&bar->s_full[w]), t & 1, abort_flag, a.status, a.spin);
            tc_fence_after();
            uint32_t s[128];
#pragma unroll
            for (int c = 0; c < 4; c++) tmem_ld32_nowait(tS + 32 * c, s + 32 * c);
            tmem_wait_ld();
            const int lim = kend - (j_first + t * BN);
            if (__any_sync(0xffffffffu, lim < BN)) {
#pragma unroll
                for (int c = 0; c < 128; c++) s[c] = c < lim ? s[c] : 0xff800000u;
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
                    // S(t) is there, and with it everything issued before it: O is at rest
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
#pragma unroll
            for (int c = 0; c < 128; c += 32) {
                uint32_t p[16];
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float e0, e1;
                    unpack2(fma2(pack2(__uint_as_float(s[c + i]), __uint_as_float(s[c + i + 1])), sl2x2, shift2), e0, e1);
                    e0 = ex2(e0);
                    e1 = ex2(e1);
                    l4[(i >> 1) & 1] = add2(l4[(i >> 1) & 1], pack2(e0, e1));
                    p[i >> 1] = pack_bf16x2(e0, e1);
                }
                tmem_st16(tS + (c >> 1), p);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(smem_u32(&bar->p_full[w]));
        }
        float l0, l1, l2, l3;
        unpack2(l4[0], l0, l1);
        unpack2(l4[1], l2, l3);
        const float l = (l0 + l1) + (l2 + l3);
        if (n[w] > 0) {
            mbar_wait(smem_u32(&bar->o_full[w]), 0, abort_flag, a.status, a.spin);
            tc_fence_after();
        }
        const long long row = (long long)slice * a.R + r, prow = (long long)part * a.slices * a.R + row;
        const float inv = l > 0.f ? (a.splits > 1 ? 1.f : 1.f / l) : 0.f;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            if (n[w] > 0) {
                tmem_ld32_nowait(tO + c, o);
                tmem_wait_ld();
            }
            if (r < a.R) {
#pragma unroll
                for (int i = 0; i < 32; i += 8) {
                    if (c + i >= a.d) break;
                    float f[8];
#pragma unroll
                    for (int e = 0; e < 8; e++) f[e] = n[w] > 0 ? __uint_as_float(o[i + e]) * inv : 0.f;
                    if (a.splits > 1) {
                        float* dst = a.part + prow * a.d + c + i;
                        store4(dst, f);
                        store4(dst + 4, f + 4);
                    } else {
                        uint4 u;
                        u.x = pack_bf16x2(f[0], f[1]);
                        u.y = pack_bf16x2(f[2], f[3]);
                        u.z = pack_bf16x2(f[4], f[5]);
                        u.w = pack_bf16x2(f[6], f[7]);
                        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.o_out) + row * a.d + c + i) = u;
                    }
                }
            }
        }
        if (r < a.R) {
            if (a.splits > 1)
                reinterpret_cast<float2*>(a.part + (long long)a.splits * a.slices * a.R * a.d)[prow] = make_float2(m, l);
            else
                a.lse_out[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tbase, 512);
    }
}

template <int D>
int launch(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    using C = Cfg<D>;
    static_assert(C::SMEM <= 227 * 1024 && sizeof(Bars) <= 1024, "shared memory budget");
    CUtensorMap mq, mk, mv;
    LLSA_TRY(make_tmap_rows(&mq, a.q, s.slices, s.R, s.d, BM));
    LLSA_TRY(make_tmap_rows(&mk, a.k, s.slices, s.nk, s.d, BN));
    LLSA_TRY(make_tmap_rows(&mv, a.v, s.slices, s.nk, s.d, BN));
    cudaFuncSetAttribute(dense_fwd_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    const long long blocks = (long long)((s.R + 2 * BM - 1) / (2 * BM)) * s.slices;
    if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
    LLSA_LAUNCH("dense_fwd_tc", st,
                dense_fwd_tc_kernel<D><<<dim3((unsigned)blocks, a.splits), kThreads, C::SMEM, st>>>(mq, mk, mv, a));
    return LLSA_OK;
}

}  // namespace

bool dense_tc_supported(const DenseShape& s) {
    return s.dtype == LLSA_DTYPE_BF16 && s.d <= 128 && s.R > 0 && s.nk > 0;
}

DenseSplit dense_tc_fwd_split(const DenseShape& s) {
    return dense_make_split((long long)s.slices * ((s.R + 2 * BM - 1) / (2 * BM)), s.nk, BN, 2);
}

int launch_dense_tc_fwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    return s.d <= 64 ? launch<64>(s, a, st) : launch<128>(s, a, st);
}

}  // namespace llsa

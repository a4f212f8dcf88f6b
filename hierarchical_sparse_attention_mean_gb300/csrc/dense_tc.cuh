// dense_tc.cuh -- waits and arrivals of the dense tensor-core kernels.
#pragma once

#include "dense.h"
#include "tc.cuh"

namespace llsa {
namespace tc {

// A bounded wait that first looks: a phase that has completed costs one test
// (about 24 clocks) instead of a try_wait.
__device__ __forceinline__ bool bar_wait(uint32_t mbar, uint32_t parity, volatile int* abort_flag, const DenseArgs& a) {
    if (mbar_test(mbar, parity)) return true;
    return mbar_wait(mbar, parity, abort_flag, a.status, a.spin);
}

// A whole warp waits; false as soon as any wait of the block gave up.
__device__ __forceinline__ bool warp_wait(uint32_t mbar, uint32_t parity, volatile int* abort_flag, const DenseArgs& a) {
    return __all_sync(0xffffffffu, bar_wait(mbar, parity, abort_flag, a));
}

// The lane of a warp that issues, chosen once per role: 1 in that lane, 0 elsewhere.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}\n" : "=r"(r));
    return r;
}

// MMAs and commits of a converged warp, issued by the chosen lane.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 e, %5, 0;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                 :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 e, %5, 0;\n"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
                 :: "r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(leader));
}
__device__ __forceinline__ void commit(uint32_t leader, uint32_t mbar) {
    asm volatile("{\n.reg .pred e;\nsetp.ne.b32 e, %1, 0;\n"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n"
                 :: "r"(mbar), "r"(leader) : "memory");
}

// One arrival for the whole warp, after what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint32_t mbar, int lane) {
    __syncwarp();
    if (lane == 0) mbar_arrive(mbar);
}

// Copies in flight must land before a block exits.
__device__ __forceinline__ void land(uint32_t mbar, uint32_t parity) {
    for (int i = 0; i < kSpinLimit && !mbar_try(mbar, parity); i++) {
    }
}

// Eight fp32 values as bf16 into chunk `chunk` (16 bytes) of row `row` of a tile
// region of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ void put_chunk(unsigned char* region, int row, int chunk, const float* v) {
    uint4 u;
    u.x = pack_bf16x2(v[0], v[1]);
    u.y = pack_bf16x2(v[2], v[3]);
    u.z = pack_bf16x2(v[4], v[5]);
    u.w = pack_bf16x2(v[6], v[7]);
    *reinterpret_cast<uint4*>(region + row * 128 + ((chunk ^ (row & 7)) << 4)) = u;
}

// A stage of a ring and the parity of its current use.
template <int N>
struct Stage {
    int st = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++st == N) {
            st = 0;
            parity ^= 1;
        }
    }
};

constexpr int kTileRows = 128;  // rows of every tile of the backward kernels

// The items of a block: tiles of ROWS rows of the streamed side, those that the
// mask leaves nothing of skipped. Every role walks the same list.
template <bool KEYS, int ROWS = kTileRows>
struct Items {
    int pos, t0, stop;  // first row of the tile; its token in its head (KEYS); end of the axis
    int x0;             // the block's first stationary row
    bool all;           // no tile to skip, no row to clear
    DenseSpan sp;

    __device__ __forceinline__ Items(const DenseArgs& a, DenseSpan s, int x0_, int pos_, int t0_, int end)
        : pos(pos_), t0(t0_), stop(end), x0(x0_), all(!KEYS || (!a.causal && s.lq == a.nq)), sp(s) {}
    __device__ __forceinline__ void start(const DenseArgs& a) {
        if (all) return;
        t0 = pos % a.nq;
        settle(a);
    }
    __device__ __forceinline__ bool done() const { return pos >= stop; }
    __device__ __forceinline__ void next(const DenseArgs& a) {
        pos += ROWS;
        if (all) return;
        turn(a);
        settle(a);
    }

private:
    __device__ __forceinline__ void turn(const DenseArgs& a) {
        t0 += ROWS;
        if (t0 >= a.nq) t0 = t0 - a.nq < a.nq ? t0 - a.nq : t0 % a.nq;
    }
    __device__ __forceinline__ void settle(const DenseArgs& a) {
        while (pos < stop && dense_tile_kend(a, sp, t0, ROWS) <= x0) {
            pos += ROWS;
            turn(a);
        }
    }
};

// Pieces are dealt to the resident blocks in rounds. In causal order they get
// lighter and lighter, so every other round goes backwards there: forwards alone
// the first block would get the heaviest of every round (12 heads x 4,096 tokens
// at d = 64, forward 42.6 us so and 35.8 in turns).
__device__ __forceinline__ int dealt(const DenseArgs& a, int i, int block, int blocks) {
    return i * blocks + (a.causal && (i & 1) ? blocks - 1 - block : block);
}
__device__ __forceinline__ int dealt_pieces(const DenseArgs& a, int block, int blocks) {
    const int full = a.pieces / blocks;
    return full + (dealt(a, full, block, blocks) < a.pieces ? 1 : 0);
}

// Host: resident blocks of a call, one per SM.
inline int resident_blocks(long long pieces) {
    const int most = test_flags() & LLSA_TEST_FEW_BLOCKS ? 3 : sm_count();
    return (int)(pieces < most ? pieces : most);
}

// The pieces of a resident block, worked out by one copying thread (divisions and
// loads of the lengths: some 1,500 clocks) ahead of the roles that read them.
constexpr int kPieceSlots = 4;

struct PieceRing {
    int4 slot[kPieceSlots][2];
    uint64_t full[kPieceSlots], free[kPieceSlots];
};

// One thread.
__device__ __forceinline__ void piece_ring_init(PieceRing* r, int readers) {
    for (int i = 0; i < kPieceSlots; i++) {
        mbar_init(smem_u32(&r->full[i]), 1);
        mbar_init(smem_u32(&r->free[i]), readers);
    }
}

// The writing thread: piece number i.
__device__ __forceinline__ bool piece_put(PieceRing* r, int i, int4 x, int4 y, volatile int* abort_flag, const DenseArgs& a) {
    const int s = i % kPieceSlots, use = i / kPieceSlots;
    if (use > 0 && !bar_wait(smem_u32(&r->free[s]), (use - 1) & 1, abort_flag, a)) return false;
    r->slot[s][0] = x;
    r->slot[s][1] = y;
    mbar_arrive(smem_u32(&r->full[s]));
    return true;
}

// A reading warp (`lanes` 32) or thread (1): piece number i; one arrival per reader.
template <int LANES>
__device__ __forceinline__ bool piece_get(PieceRing* r, int i, int4& x, int4& y, int lane, volatile int* abort_flag,
                                          const DenseArgs& a) {
    const int s = i % kPieceSlots;
    const bool ok = LANES == 32 ? warp_wait(smem_u32(&r->full[s]), (i / kPieceSlots) & 1, abort_flag, a)
                                : bar_wait(smem_u32(&r->full[s]), (i / kPieceSlots) & 1, abort_flag, a);
    if (!ok) return false;
    x = r->slot[s][0];
    y = r->slot[s][1];
    if (LANES == 32) warp_arrive(smem_u32(&r->free[s]), lane);
    else mbar_arrive(smem_u32(&r->free[s]));
    return true;
}

}  // namespace tc
}  // namespace llsa

// dense_split.cuh -- operands as bf16 planes, three for fp32 and one for bf16: what the
// kernels on them share.
#pragma once

#include "dense_tc.cuh"

namespace llsa {
namespace tc {

// The terms of a product of three planes each: six. Of one plane: one.
template <int PL>
constexpr int kTerms = PL == 3 ? 6 : 1;

// Of the six, small ones first: plane of the first operand, of the second.
template <int PL>
__device__ __forceinline__ constexpr int term_a(int i) { return PL == 1 ? 0 : i == 0 ? 2 : i == 1 ? 0 : i == 2 ? 1 : i == 3 ? 1 : 0; }
template <int PL>
__device__ __forceinline__ constexpr int term_b(int i) { return PL == 1 ? 0 : i == 0 ? 0 : i == 1 ? 2 : i == 2 ? 1 : i == 3 ? 0 : i == 4 ? 1 : 0; }

// Two fp32 values as three packed bf16 pairs.
__device__ __forceinline__ void split2(float x, float y, uint32_t& p1, uint32_t& p2, uint32_t& p3) {
    p1 = pack_bf16x2(x, y);
    x -= __uint_as_float(p1 << 16);
    y -= __uint_as_float(p1 & 0xffff0000u);
    p2 = pack_bf16x2(x, y);
    x -= __uint_as_float(p2 << 16);
    y -= __uint_as_float(p2 & 0xffff0000u);
    p3 = pack_bf16x2(x, y);
}

// One thread: the planes of ROWS rows from `row` on, 64 columns after 64 columns,
// in one copy each. `more` bytes come with them on the same barrier.
template <int ROWS, int D, int PL>
__device__ __forceinline__ void load_planes(unsigned char* dst, const CUtensorMap* map, int row, int slice, uint32_t mbar,
                                            int more = 0) {
    mbar_arrive_expect_tx(mbar, PL * ROWS * D * 2 + more);
    for (int c = 0; c < D / 64; c++) tma_load_4d(smem_u32(dst + c * PL * ROWS * 128), map, c * 64, row, slice, 0, mbar);
}

template <int COLS, typename T>
__device__ __forceinline__ void store_rowpart(T* dst, const float* o, float f, int c0, int d) {
#pragma unroll
    for (int c = 0; c < COLS; c += 4)
        if (c0 + c < d) {
            const float v[4] = {o[c] * f, o[c + 1] * f, o[c + 2] * f, o[c + 3] * f};
            store4(dst + c0 + c, v);
        }
}

}  // namespace tc
}  // namespace llsa

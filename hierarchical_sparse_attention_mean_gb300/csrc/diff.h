// diff.h -- what the differential attention kernels share.
//
// o = P1 V - lam P2 V with P_i = softmax(scale Q_i K_i^T): two maps with query and key
// heads of d columns over one value head of 2 d. Rows, slices and the mask are those of
// dense attention (dense.h): a slice is a batch entry and value head, its R = G nq rows
// are the tokens of the G heads that share it, and map i of slice (b, g) is matrix
// (2 b + i) kv_heads + g of q and of k. Both maps see the same mask.
#pragma once

#include "dense.h"

namespace llsa {

constexpr int kDiffStats = 5;  // numbers per query row in the backward pass: -lse log2(e) and -D of both maps, lam

struct DiffShape {
    int batch, heads, kv_heads, G, nq, nk, d, dtype, lam_dtype, causal;
    int wide;    // q, k, dq, dk and o2 are fp32, whatever dtype
    int slices;  // batch * kv_heads
    int R, Rp;   // rows per slice, and padded to kDenseRowPad
    float scale;
    DenseShape four;  // the same call as four dense ones (diff_api.cu)
};

struct DiffArgs {
    DenseArgs d;  // slices, rows, lengths, mask, status; q, k, v, dout, and o of the call
    const void* lam;
    int lam_bf16, heads;
    const void* o2;  // the second map's output (backward)
    void* o2_out;    // or NULL (forward)
    // Backward: nl2 of DenseArgs holds kDiffStats arrays [slices][Rp], -lse log2(e) and -D of
    // both maps and lam; d2 takes sums of P_2 dP of every row, [parts of dq][4][slices][Rp].
    float* d2;
    // Of a small call, the last block of dq sums d2 to dlam: *lam_ticket counts the lam_pieces
    // of them. NULL: a kernel after it does.
    int* lam_ticket;
    void* dlam;
    int lam_pieces, lam_sets;
};

// Eight values as fp32, from memory that a kernel before this one may have written while this one
// was set up (load8 reads through the cache for what stays as it is).
__device__ __forceinline__ void diff_load8(const __nv_bfloat16* p, float* f) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void diff_load8(const float* p, float* f) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float4 x = *reinterpret_cast<const float4*>(p + i);
        f[i] = x.x;
        f[i + 1] = x.y;
        f[i + 2] = x.z;
        f[i + 3] = x.w;
    }
}

// Weight of the second map in the rows of head h.
__device__ __forceinline__ float diff_lam(const DiffArgs& a, int h) {
    return a.lam_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.lam)[h]) : static_cast<const float*>(a.lam)[h];
}

// Head of row r of a slice.
__device__ __forceinline__ int diff_head(const DiffArgs& a, int slice, int r) {
    return slice % a.d.kv_heads * (a.heads / a.d.kv_heads) + r / a.d.nq;
}

// The same for row r of a slice, and 0 where the row sees no key: it has o = 0 and no gradient
// whatever lam is, infinite or no number.
__device__ __forceinline__ float diff_lam_row(const DiffArgs& a, int slice, int r) {
    const float lam = diff_lam(a, diff_head(a, slice, r));
    return isfinite(lam) || dense_kend(a.d, dense_span(a.d, slice), r % a.d.nq) > 0 ? lam : 0.f;
}

// Row r of map i of a slice in an array over [batch][2 heads][nq].
__device__ __forceinline__ long long diff_row(const DiffArgs& a, int slice, int i, int r) {
    const int b = slice / a.d.kv_heads, g = slice - b * a.d.kv_heads;
    return ((long long)(2 * b + i) * a.d.kv_heads + g) * a.d.R + r;
}

// Matrix of map i of a slice in q, k, dq and dk.
__device__ __forceinline__ int diff_matrix(const DenseArgs& a, int slice, int i) {
    return slice + (slice / a.kv_heads + i) * a.kv_heads;  // (2 b + i) kv_heads + g
}

// 16 results of a row from column c on, of an output of `cols` columns.
template <typename T>
__device__ __forceinline__ void diff_store16(T* dst, const float* o, int c, int cols) {
#pragma unroll
    for (int i = 0; i < 16; i += 4)
        if (c + i < cols) store4(dst + i, o + i);
}

// A split of the keys leaves, per part, O unnormalised [splits][2][slices R][2 d] and then
// (maximum in units of log2, sum) pairs [splits][2][slices R], in DenseArgs::part.
__device__ __forceinline__ long long diff_part(const DenseArgs& a, int part, int i, long long row) {
    return ((long long)part * 2 + i) * a.slices * a.R + row;
}
__device__ __forceinline__ float2* diff_part_ml(const DenseArgs& a) {
    return reinterpret_cast<float2*>(a.part + (long long)a.splits * 2 * a.slices * a.R * 2 * a.d);
}
// Writes dlam where lam_ticket asks for it, by 512 threads of a block that has written its part of
// d2. A warp per head, so every sum has a fixed order whichever block is the last. `last`:
// shared memory of the block.
__device__ __forceinline__ void diff_lam_last(const DiffArgs& f, int* last) {
    if (!f.lam_ticket) return;
    const DenseArgs& a = f.d;
    __threadfence();
    asm volatile("bar.sync 5, 512;" ::: "memory");
    if (threadIdx.x == 0) *last = atomicAdd(f.lam_ticket, 1) == f.lam_pieces - 1;
    asm volatile("bar.sync 5, 512;" ::: "memory");
    if (!*last) return;
    __threadfence();
    const int lane = threadIdx.x & 31, G = f.heads / a.kv_heads, rows = a.slices / a.kv_heads * a.nq;
    const long long all = (long long)a.slices * a.Rp;
    for (int h = threadIdx.x >> 5; h < f.heads; h += 16) {
        const int g = h / G;
        float sum = 0.f;
        for (int row = lane; row < rows; row += 32) {
            const int b = row / a.nq, t = row - b * a.nq;
            const float* from = f.d2 + ((long long)b * a.kv_heads + g) * a.Rp + (h - g * G) * a.nq + t;
#pragma unroll 4
            for (int i = 0; i < f.lam_sets; i++) sum += __ldcg(from + i * all);
        }
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane != 0) continue;
        if (f.lam_bf16) static_cast<__nv_bfloat16*>(f.dlam)[h] = __float2bfloat16_rn(-sum);
        else static_cast<float*>(f.dlam)[h] = -sum;
    }
}

inline size_t diff_part_bytes(const DiffShape& s, int splits) {
    return splits > 1 ? (size_t)splits * 2 * s.slices * s.R * (2 * s.d + 2) * sizeof(float) : 0;
}

// diff_few.cu: forward of a few rows per value head.
bool diff_few_supported(const DiffShape& s);
DenseSplit diff_few_split(const DiffShape& s);
int launch_diff_few(const DiffShape& s, const DiffArgs& a, cudaStream_t st);

// diff_fwd_tc.cu: forward on the tensor cores (bf16).
bool diff_tc_supported(const DiffShape& s);
DenseSplit diff_tc_fwd_split(const DiffShape& s);
int launch_diff_tc_fwd(const DiffShape& s, const DiffArgs& a, cudaStream_t st);

// diff_bwd_tc.cu: backward on the tensor cores (bf16); diff_bwd_wide_tc.cu: behind 64 columns.
void diff_tc_bwd_splits(const DiffShape& s, DenseSplit* rows, DenseSplit* keys);
int launch_diff_tc_bwd(const DiffShape& s, const DiffArgs& aq, const DiffArgs& ak, cudaStream_t st);
int launch_diff_tc_bwd_wide(const DiffShape& s, const DiffArgs& aq, const DiffArgs& ak, cudaStream_t st);

}  // namespace llsa

// dense.h -- what the dense attention kernels share: their arguments, the
// mask's arithmetic and the launchers.
//
// Rows. The query heads that share a key head lie next to each other in
// [batch, heads, nq, d], so the kernels see batch * kv_heads slices of
// G * nq query rows (G = heads / kv_heads) over nk keys: row r of a slice is
// token r % nq of the slice's head r / nq. One pass over K and V then serves
// all heads that share them, a single token's G heads included, and dk, dv sum
// over those heads in one place.
//
// Mask. Every rule of the call (lengths, padding, causal order) leaves row r
// the keys 0 .. kend(r) - 1, so one number per row is the mask. A row without keys is
// known by its sum of weights, 0 (o = 0, lse = -infinity); the sum of a row with a NaN
// among its scores is NaN, and so are its o and lse.
#pragma once

#include "internal.h"

namespace llsa {

constexpr float kDenseLog2e = 1.4426950408889634f;
constexpr int kDenseRowPad = 128;  // rows of a slice in the per-row arrays: a multiple of this
constexpr int kDenseMaxExtent = 1 << 30;  // rows of a slice, keys of a slice
constexpr int kDenseSms = 152;  // splits, and so the workspace, go by the GB300's SMs

struct DenseShape {
    int batch, heads, kv_heads, G, nq, nk, d, dtype, causal;
    int slices;   // batch * kv_heads
    int R, Rp;    // rows per slice, and padded to kDenseRowPad
    float scale;
};

struct DenseArgs {
    const void *q, *k, *v, *o, *dout;
    const float* lse;
    const int *q_len, *k_len;
    void *o_out, *dq, *dk, *dv;
    float* lse_out;
    float* nl2;   // [slices][Rp]: -lse * log2(e); -infinity for rows without keys
    float* nd;    // [slices][Rp]: -D = -dout . o; 0 for those rows
    float* part;  // partial sums of a split axis (layout: see the kernels)
    int splits, chunk;  // parts of the split axis, and how many of its elements each takes
    int pieces;         // pieces of work that the resident blocks share (tensor-core kernels)
    int whole;          // of them, those before the halved ones (forward)
    int four;           // slices share planes of q, k and v, as diff_api.cu lays them out
    int slices, kv_heads, nq, nk, R, Rp, d, causal;
    float scale;
    int* status;
    int spin, test_flags;
};

struct DenseSpan {
    int lq, lk;
};

// Where the planes of a slice's q and k, and of its v, lie among those of all slices. Four calls
// as one (diff_api.cu): slice ((2 b + i) 2 + j) kv + g has the q and k of (2 b + i) kv + g and the v of
// (2 b + j) kv + g.
__device__ __forceinline__ int dense_qk_slice(const DenseArgs& a, int slice) {
    if (!a.four) return slice;
    const int kv = a.kv_heads / 4, x = slice / kv;
    return (x >> 1) * kv + slice - x * kv;
}
__device__ __forceinline__ int dense_v_slice(const DenseArgs& a, int slice) {
    if (!a.four) return slice;
    const int kv = a.kv_heads / 4, x = slice / kv;
    return ((x >> 2) * 2 + (x & 1)) * kv + slice - x * kv;
}
// Slices of those planes.
inline long long dense_plane_slices(const DenseArgs& a) { return a.four ? a.slices / 2 : a.slices; }

// Valid query and key tokens of a slice's batch entry.
__device__ __forceinline__ DenseSpan dense_span(const DenseArgs& a, int slice) {
    const int b = slice / a.kv_heads;
    DenseSpan s;
    s.lq = a.nq;
    s.lk = a.nk;
    if (a.q_len) {
        const int v = a.q_len[b];
        s.lq = min(max(v, 0), a.nq);
        if (s.lq != v) set_status(a.status, LLSA_ERR_BAD_INDEX);
    }
    if (a.k_len) {
        const int v = a.k_len[b];
        s.lk = min(max(v, 0), a.nk);
        if (s.lk != v) set_status(a.status, LLSA_ERR_BAD_INDEX);
    }
    return s;
}

// Keys that token t of a head sees: 0 .. kend - 1.
__device__ __forceinline__ int dense_kend(const DenseArgs& a, DenseSpan s, int t) {
    if (t >= s.lq) return 0;
    return a.causal ? min(max(t + s.lk - s.lq + 1, 0), s.lk) : s.lk;
}

// A bound on kend over `rows` consecutive rows whose first is token t0 of its
// head (they may run into the next heads); 0 when none of them sees a key.
__device__ __forceinline__ int dense_tile_kend(const DenseArgs& a, DenseSpan s, int t0, int rows) {
    const bool wraps = t0 + rows > a.nq;
    if (!wraps && t0 >= s.lq) return 0;
    const int last = wraps ? s.lq - 1 : min(t0 + rows, s.lq) - 1;
    return last < 0 ? 0 : dense_kend(a, s, last);
}

// Piece `id` of a call's work: block `block` of `blocks` along the owned axis of
// a slice, part `part` of the split one. In causal order blocks differ in
// work: all slices' first blocks come first, so the heaviest ones are dealt out
// evenly before the light ones. Otherwise the blocks of a slice stay together
// and share its keys in L2.
struct DenseWork {
    int slice, part, block, blocks;
};

constexpr long long kDenseMaxPieces = 0x7fffffffLL - 1024;

__device__ __forceinline__ DenseWork dense_work(const DenseArgs& a, int id, int blocks) {
    DenseWork w;
    w.blocks = blocks;
    const int sets = a.slices * a.splits;
    int set;
    if (a.causal) {
        w.block = id / sets;
        set = id - w.block * sets;
    } else {
        set = id / blocks;
        w.block = id - set * blocks;
    }
    w.slice = a.splits > 1 ? set / a.splits : set;
    w.part = set - w.slice * a.splits;
    return w;
}

int derive_dense(const llsa_dense_params* p, DenseShape* s);  // checks the parameters
DenseArgs dense_args(const DenseShape& s);                     // what a launch needs besides its pointers
inline int dense_check_lens(const int32_t* q_len, const int32_t* k_len) {
    return (reinterpret_cast<uintptr_t>(q_len) | reinterpret_cast<uintptr_t>(k_len)) & 3u ? LLSA_ERR_ALIGN : LLSA_OK;
}
size_t dense_fwd_workspace(const DenseShape& s);
size_t dense_bwd_workspace(const DenseShape& s);
int launch_dense_fwd(const DenseShape& s, DenseArgs a, void* ws, cudaStream_t st);
int launch_dense_bwd(const DenseShape& s, DenseArgs a, void* ws, cudaStream_t st);
// Whether a call in fp32 runs on planes, and its passes behind those that make them: forward with
// `part` for a split's parts; backward also behind the rows' numbers (nl2, nd of `a`).
bool dense_fwd_on_planes(const DenseShape& s);
bool dense_bwd_on_planes(const DenseShape& s);
size_t dense_fwd_parts(const DenseShape& s);
size_t dense_bwd_parts(const DenseShape& s);
int launch_dense_fwd_planes(const DenseShape& s, DenseArgs a, const void* const* planes, void* part, cudaStream_t st);
int launch_dense_bwd_planes(const DenseShape& s, DenseArgs a, void* const* planes, void* part, cudaStream_t st);

// Sums of the parts of up to three outputs, in ascending order: out = sum_p part[p n ..], rounded to `dtype`.
struct DenseSums {
    const float* part[3];
    void* out[3];
    long long n[3];
    int parts[3];
    int outs = 0;
    void add(const float* p, void* o, long long count, int splits) {
        part[outs] = p;
        out[outs] = o;
        n[outs] = count;
        parts[outs++] = splits;
    }
};
int launch_dense_sums(int dtype, const DenseSums& sums, cudaStream_t st);

struct DenseSplit {
    int splits, chunk;  // parts, and elements of the split axis per part (a multiple of `tile`)
};

// How a long axis of `extent` elements in tiles is split where the other axis
// gives too few blocks: as many parts as still fit one wave of blocks, each of
// `least` tiles at least.
inline DenseSplit dense_make_split(long long blocks, int extent, int tile, int least) {
    const long long units = (extent + tile - 1) / tile;
    long long n = blocks > 0 ? kDenseSms / blocks : 1;
    n = n > units / least ? units / least : n;
    n = n < 1 ? 1 : n;
    DenseSplit p;
    p.chunk = (int)((units + n - 1) / n) * tile;
    p.splits = extent > 0 ? (extent + p.chunk - 1) / p.chunk : 1;
    return p;
}

// dense_simt.cu: fp32 behind 128 columns on the CUDA cores.
DenseSplit dense_simt_fwd_split(const DenseShape& s);  // dq: the same
DenseSplit dense_simt_dkv_split(const DenseShape& s);
int launch_dense_simt_fwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st);
int launch_dense_simt_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, cudaStream_t st);

// dense_few.cu: a handful of rows per key head.
bool dense_few_supported(const DenseShape& s);
bool dense_few_bwd_supported(const DenseShape& s);
DenseSplit dense_few_split(const DenseShape& s);  // of the keys, in both directions
int launch_dense_few(const DenseShape& s, const DenseArgs& a, cudaStream_t st);
int launch_dense_few_bwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st);

// dense_keys.cu: forward of fp32 against a handful of keys.
bool dense_keys_supported(const DenseShape& s);
int launch_dense_keys(const DenseShape& s, const DenseArgs& a, cudaStream_t st);

// dense_fwd_tc.cu, dense_bwd_tc.cu: tensor-core kernels (bf16, d <= 128).
bool dense_tc_supported(const DenseShape& s);
DenseSplit dense_tc_fwd_split(const DenseShape& s);
DenseSplit dense_tc_dq_split(const DenseShape& s);
DenseSplit dense_tc_dkv_split(const DenseShape& s);
int launch_dense_tc_fwd(const DenseShape& s, const DenseArgs& a, cudaStream_t st);
int launch_dense_tc_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, cudaStream_t st);

// dense_split_tc.cu: fp32 up to 128 columns and bf16 behind 128 on the tensor cores (planes: fp32, three bf16 planes
// of q, k, v, or of q, dout, k, v, at the start of the workspace).
bool dense_split_supported(const DenseShape& s);
DenseSplit dense_split_fwd_split(const DenseShape& s);  // dq: the same
DenseSplit dense_split_dkv_split(const DenseShape& s);
size_t dense_split_planes(const DenseShape& s, bool backward);  // bytes
int launch_dense_split_fwd(const DenseShape& s, const DenseArgs& a, void* ws, cudaStream_t st);
// fp32, from planes that are there already ([3][slices][R or nk][d] each of q, k, v).
int launch_dense_split_fwd_planes(const DenseShape& s, const DenseArgs& a, const void* const* planes, cudaStream_t st);
int make_dense_split_planes(const DenseShape& s, const DenseArgs& a, void* ws, void** planes, cudaStream_t st);
// dense_split_wide_tc.cu: the backward pass of fp32 behind 64 columns and of bf16.
int launch_dense_split_wide_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, void* const* planes,
                                cudaStream_t st);
int launch_dense_split_bwd(const DenseShape& s, const DenseArgs& aq, const DenseArgs& ak, void* const* planes,
                           cudaStream_t st);

}  // namespace llsa

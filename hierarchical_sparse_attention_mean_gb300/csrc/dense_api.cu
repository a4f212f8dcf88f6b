// dense_api.cu -- the C entries of dense attention: validation, workspace,
// choice of kernels, and the passes around the attention kernels (the per-row
// numbers of the backward pass, the joins of a split axis).
#include <math.h>
#include <string.h>

#include <algorithm>

#include "dense.h"
#include "entry.h"

namespace llsa {
namespace {

constexpr int kThreads = 256;

size_t align_up(size_t x) { return (x + 255) & ~(size_t)255; }

// ------------------------------------------------------ per-row numbers --

// -lse * log2(e) and -D = -dout . o of every query row; rows that see no key
// (and the padding to Rp) get -infinity, so that their probabilities are
// 2^(s - inf) = 0, and D = 0. A block per 128 rows, eight lanes per row, four
// rows each at a time. Bound by HBM: dout and o are read once (152 slices of
// 4,096 rows at d = 64 28 us of 24; one row per eight lanes took 42).
constexpr int kRowsEach = kDenseRowPad / (kThreads / 8);

__device__ __forceinline__ float dot16(const uint4& x, const uint4& y, const __nv_bfloat16*) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sum = fmaf(__uint_as_float(u[i] << 16), __uint_as_float(v[i] << 16), sum);
        sum = fmaf(__uint_as_float(u[i] & 0xffff0000u), __uint_as_float(v[i] & 0xffff0000u), sum);
    }
    return sum;
}
__device__ __forceinline__ float dot16(const uint4& x, const uint4& y, const float*) {
    float sum = __uint_as_float(x.x) * __uint_as_float(y.x);
    sum = fmaf(__uint_as_float(x.y), __uint_as_float(y.y), sum);
    sum = fmaf(__uint_as_float(x.z), __uint_as_float(y.z), sum);
    return fmaf(__uint_as_float(x.w), __uint_as_float(y.w), sum);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) dense_rows_kernel(const __grid_constant__ DenseArgs a) {
    constexpr int E = 16 / sizeof(T);
    const unsigned per = (unsigned)a.Rp / kDenseRowPad, slice = blockIdx.x / per;
    const int r0 = (int)(blockIdx.x - slice * per) * kDenseRowPad + (threadIdx.x >> 3), part = threadIdx.x & 7;
    const DenseSpan sp = dense_span(a, (int)slice);
    float lse[kRowsEach], sum[kRowsEach];
    bool on[kRowsEach];
#pragma unroll
    for (int u = 0; u < kRowsEach; u++) {
        const int r = r0 + u * (kThreads / 8);
        on[u] = r < a.R && dense_kend(a, sp, r < a.nq ? r : r % a.nq) > 0;
        lse[u] = on[u] ? __ldg(a.lse + (long long)slice * a.R + r) : -INFINITY;
        sum[u] = 0.f;
    }
    for (int c = part * E; c < a.d; c += 8 * E) {
        uint4 x[kRowsEach], y[kRowsEach];
        const long long at = ((long long)slice * a.R + r0) * a.d + c;
#pragma unroll
        for (int u = 0; u < kRowsEach; u++) {
            x[u] = y[u] = make_uint4(0u, 0u, 0u, 0u);
            if (on[u]) {
                x[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.dout) + at + (long long)u * (kThreads / 8) * a.d));
                y[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.o) + at + (long long)u * (kThreads / 8) * a.d));
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsEach; u++) sum[u] += dot16(x[u], y[u], static_cast<const T*>(nullptr));
    }
#pragma unroll
    for (int u = 0; u < kRowsEach; u++) {
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
        if (part == 0) {
            const long long idx = (long long)slice * a.Rp + r0 + u * (kThreads / 8);
            a.nl2[idx] = lse[u] == -INFINITY ? -INFINITY : -lse[u] * kDenseLog2e;
            a.nd[idx] = lse[u] == -INFINITY ? 0.f : -sum[u];
        }
    }
}

// ------------------------------------------------------- joins of a split --

// o and lse of every query row from the parts of a split over the keys: a warp per
// row. The weights of 32 parts are worked out at once, a lane each; then each half of
// the warp (d <= 64) or all of it takes every second or every part, many loads at a
// time: with few rows the latency of the parts is what this costs (12 rows of 25 parts
// 3 us; part after part, 6).
template <typename T>
__global__ void __launch_bounds__(kThreads) dense_join_fwd_kernel(const __grid_constant__ DenseArgs a) {
    const long long rows = (long long)a.slices * a.R;
    const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    const int lane = threadIdx.x & 31;
    if (row >= rows) return;
    const float2* ml = reinterpret_cast<const float2*>(a.part + (long long)a.splits * rows * a.d);
    float m = -INFINITY, l = 0.f;
    for (int p = lane; p < a.splits; p += 32) m = fmaxf(m, ml[p * rows + row].x);
    m = warp_max(m);
    const float shift = m == -INFINITY ? 0.f : m;
    for (int p = lane; p < a.splits; p += 32) {
        const float2 x = ml[p * rows + row];
        l = fmaf(x.y, exp2f(x.x - shift), l);
    }
    l = warp_sum(l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int at_once = a.d <= 64 ? 2 : 1, sub = at_once == 2 ? lane >> 4 : 0;
    const int c = (at_once == 2 ? lane & 15 : lane) * 4;  // and c + 128 behind 128 columns
    float acc[2][4] = {};
    for (int p0 = 0; p0 < a.splits; p0 += 32) {
        const float w = p0 + lane < a.splits ? exp2f(ml[(p0 + lane) * rows + row].x - shift) : 0.f;
        const int n = min(32, a.splits - p0);
#pragma unroll 8
        for (int i = 0; i < n; i += at_once) {
            const float wi = __shfl_sync(0xffffffffu, w, (i + sub) & 31);
            const float* from = a.part + ((p0 + i + sub) * rows + row) * a.d + c;
#pragma unroll
            for (int k = 0; k < 2; k++)
                if (c + 128 * k < a.d && i + sub < n) {
                    const float4 x = *reinterpret_cast<const float4*>(from + 128 * k);
                    acc[k][0] = fmaf(wi, x.x, acc[k][0]);
                    acc[k][1] = fmaf(wi, x.y, acc[k][1]);
                    acc[k][2] = fmaf(wi, x.z, acc[k][2]);
                    acc[k][3] = fmaf(wi, x.w, acc[k][3]);
                }
        }
    }
#pragma unroll
    for (int k = 0; k < 2; k++) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            if (at_once == 2) acc[k][i] += __shfl_xor_sync(0xffffffffu, acc[k][i], 16);
            acc[k][i] *= inv;
        }
        if (sub == 0 && c + 128 * k < a.d) store4(static_cast<T*>(a.o_out) + row * a.d + c + 128 * k, acc[k]);
    }
    if (lane == 0) a.lse_out[row] = l == 0.f ? -INFINITY : m * 0.6931471805599453f + logf(l);
}

// Sums of the parts of up to three outputs (blockIdx.y).
template <typename T>
__global__ void __launch_bounds__(kThreads) dense_join_sum_kernel(const __grid_constant__ DenseSums a) {
    const int t = blockIdx.y;
    const long long n = a.n[t], i = ((long long)blockIdx.x * kThreads + threadIdx.x) * 4;
    if (i >= n) return;
    const float* part = a.part[t];
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = 0; p < a.parts[t]; p++) {
        const float4 x = *reinterpret_cast<const float4*>(part + p * n + i);
        acc[0] += x.x;
        acc[1] += x.y;
        acc[2] += x.z;
        acc[3] += x.w;
    }
    store4(static_cast<T*>(a.out[t]) + i, acc);
}

// What is left of a call without rows or without keys: `n` 16-byte units of zeros in
// one or two outputs, lse of `rows` rows that see nothing, and the report of lengths
// outside their range.
__global__ void __launch_bounds__(kThreads)
dense_nothing_kernel(const __grid_constant__ DenseArgs a, uint4* x, uint4* y, long long n, float* lse, long long rows) {
    const long long first = (long long)blockIdx.x * kThreads + threadIdx.x, step = (long long)gridDim.x * kThreads;
    for (long long s = first * a.kv_heads; s < a.slices; s += step * a.kv_heads) dense_span(a, (int)s);
    for (long long i = first; i < n; i += step) {
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (y) y[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    for (long long i = first; i < rows; i += step) lse[i] = -INFINITY;
}

// Which kernels take a call.
enum class Path { kNone, kFew, kKeys, kTc, kSplit, kSimt };

Path fwd_path(const DenseShape& s) {
    return s.R == 0 || s.nk == 0      ? Path::kNone
           : dense_few_supported(s)   ? Path::kFew
           : dense_keys_supported(s)  ? Path::kKeys
           : dense_tc_supported(s)    ? Path::kTc
           : dense_split_supported(s) ? Path::kSplit
                                      : Path::kSimt;
}
Path bwd_path(const DenseShape& s) {
    return s.R == 0 || s.nk == 0        ? Path::kNone
           : dense_few_bwd_supported(s) ? Path::kFew
           : dense_tc_supported(s)      ? Path::kTc
           : dense_split_supported(s)   ? Path::kSplit
                                        : Path::kSimt;
}

DenseSplit fwd_split(const DenseShape& s) {
    switch (fwd_path(s)) {
        case Path::kNone:
        case Path::kKeys: return {1, s.nk};
        case Path::kFew: return dense_few_split(s);
        case Path::kTc: return dense_tc_fwd_split(s);
        case Path::kSplit: return dense_split_fwd_split(s);
        default: return dense_simt_fwd_split(s);
    }
}
DenseSplit dq_split(const DenseShape& s) {
    switch (bwd_path(s)) {
        case Path::kNone: return {1, s.nk};
        case Path::kFew: return dense_few_split(s);
        case Path::kTc: return dense_tc_dq_split(s);
        case Path::kSplit: return dense_split_fwd_split(s);
        default: return dense_simt_fwd_split(s);
    }
}
DenseSplit dkv_split(const DenseShape& s) {
    switch (bwd_path(s)) {
        case Path::kNone:
        case Path::kFew: return {1, s.nk};  // dk, dv: of the blocks that own the keys
        case Path::kTc: return dense_tc_dkv_split(s);
        case Path::kSplit: return dense_split_dkv_split(s);
        default: return dense_simt_dkv_split(s);
    }
}

}  // namespace

int derive_dense(const llsa_dense_params* p, DenseShape* s) {
    if (!p) return LLSA_ERR_INVALID_ARG;
    if (p->batch < 0 || p->heads < 0 || p->kv_heads < 0 || p->nq < 0 || p->nk < 0) return LLSA_ERR_INVALID_ARG;
    if (p->dtype != LLSA_DTYPE_BF16 && p->dtype != LLSA_DTYPE_F32) return LLSA_ERR_DTYPE;
    if (p->causal != 0 && p->causal != 1) return LLSA_ERR_INVALID_ARG;
    if (!(p->scale >= 0.0f) || isinf(p->scale)) return LLSA_ERR_INVALID_ARG;
    if (p->d < 8 || p->d > 256 || p->d % 8 != 0) return LLSA_ERR_SHAPE;
    memset(s, 0, sizeof(*s));
    s->batch = p->batch;
    s->heads = p->heads;
    s->kv_heads = p->kv_heads ? p->kv_heads : p->heads;
    if (s->heads == 0) {
        if (s->kv_heads != 0) return LLSA_ERR_SHAPE;
    } else if (s->heads % s->kv_heads != 0) {
        return LLSA_ERR_SHAPE;
    }
    s->G = s->heads ? s->heads / s->kv_heads : 0;
    s->nq = p->nq;
    s->nk = p->nk;
    s->d = p->d;
    s->dtype = p->dtype;
    s->causal = p->causal;
    s->scale = p->scale > 0.0f ? p->scale : 1.0f / sqrtf((float)p->d);
    const long long slices = (long long)s->batch * s->kv_heads, R = (long long)s->G * s->nq;
    if (slices > kDenseMaxExtent || R > kDenseMaxExtent || s->nk > kDenseMaxExtent) return LLSA_ERR_UNSUPPORTED;
    s->slices = (int)slices;
    s->R = (int)R;
    s->Rp = (s->R + kDenseRowPad - 1) / kDenseRowPad * kDenseRowPad;
    // up to 2^68: more than 64 bits hold
    if ((double)slices * std::max(s->Rp, s->nk) * s->d > (double)(1LL << 40)) return LLSA_ERR_UNSUPPORTED;
    return LLSA_OK;
}

DenseArgs dense_args(const DenseShape& s) {
    DenseArgs a;
    memset(&a, 0, sizeof(a));
    a.splits = 1;
    a.slices = s.slices;
    a.kv_heads = s.kv_heads;
    a.nq = s.nq;
    a.nk = s.nk;
    a.R = s.R;
    a.Rp = s.Rp;
    a.d = s.d;
    a.causal = s.causal;
    a.scale = s.scale;
    a.status = status_ptr();
    a.spin = wait_limit();
    a.test_flags = test_flags();
    return a;
}

bool dense_fwd_on_planes(const DenseShape& s) { return s.dtype == LLSA_DTYPE_F32 && fwd_path(s) == Path::kSplit; }
bool dense_bwd_on_planes(const DenseShape& s) { return s.dtype == LLSA_DTYPE_F32 && bwd_path(s) == Path::kSplit; }

size_t dense_fwd_parts(const DenseShape& s) {
    const DenseSplit p = fwd_split(s);
    return p.splits > 1 ? (size_t)p.splits * s.slices * s.R * (s.d + 2) * sizeof(float) : 0;
}

size_t dense_fwd_workspace(const DenseShape& s) {
    return (fwd_path(s) == Path::kSplit ? dense_split_planes(s, false) : 0) + dense_fwd_parts(s);
}

// The per-row numbers of the backward pass, one array of the two (the kernels for
// a handful of rows work them out).
static size_t dense_rows_bytes(const DenseShape& s) {
    const Path path = bwd_path(s);
    return path == Path::kNone || path == Path::kFew ? 0 : align_up((size_t)s.slices * s.Rp * sizeof(float));
}

// A call without rows or without keys: zeros in x and y (or NULL) of `elems` elements, and
// lse (or NULL).
static int launch_dense_nothing(const DenseShape& s, const DenseArgs& a, void* x, void* y, long long elems, float* lse,
                                cudaStream_t st) {
    const long long n = elems / (s.dtype == LLSA_DTYPE_BF16 ? 8 : 4), rows = lse ? (long long)s.slices * s.R : 0;
    const int blocks = (int)std::min<long long>((n + kThreads - 1) / kThreads, 8LL * kDenseSms);
    LLSA_LAUNCH("dense_nothing", st,
                dense_nothing_kernel<<<blocks, kThreads, 0, st>>>(a, static_cast<uint4*>(x), static_cast<uint4*>(y), n, lse, rows));
    return LLSA_OK;
}

size_t dense_bwd_parts(const DenseShape& s) {
    const DenseSplit pq = dq_split(s), pk = dkv_split(s);
    const size_t dq = pq.splits > 1 ? (size_t)pq.splits * s.slices * s.R * s.d * sizeof(float) : 0;
    const size_t dkv = pk.splits > 1 ? (size_t)pk.splits * 2 * s.slices * s.nk * s.d * sizeof(float) : 0;
    return align_up(dq) + dkv;
}

size_t dense_bwd_workspace(const DenseShape& s) {
    return (bwd_path(s) == Path::kSplit ? dense_split_planes(s, true) : 0) + 2 * dense_rows_bytes(s) + dense_bwd_parts(s);
}

static int launch_dense_join(const DenseShape& s, const DenseArgs& a, cudaStream_t st) {
    if (a.splits == 1) return LLSA_OK;
    const long long rows = (long long)s.slices * s.R;
    const unsigned blocks = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
    if (s.dtype == LLSA_DTYPE_BF16)
        LLSA_LAUNCH("dense_join_fwd", st, dense_join_fwd_kernel<__nv_bfloat16><<<blocks, kThreads, 0, st>>>(a));
    else
        LLSA_LAUNCH("dense_join_fwd", st, dense_join_fwd_kernel<float><<<blocks, kThreads, 0, st>>>(a));
    return LLSA_OK;
}

int launch_dense_fwd(const DenseShape& s, DenseArgs a, void* ws, cudaStream_t st) {
    if (s.R == 0) return LLSA_OK;
    const DenseSplit p = fwd_split(s);
    a.splits = p.splits;
    a.chunk = p.chunk;
    const Path path = fwd_path(s);
    if (path == Path::kNone) return launch_dense_nothing(s, a, a.o_out, nullptr, (long long)s.slices * s.R * s.d, a.lse_out, st);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + (path == Path::kSplit ? dense_split_planes(s, false) : 0));
    switch (path) {
        case Path::kFew: LLSA_TRY(launch_dense_few(s, a, st)); break;
        case Path::kKeys: LLSA_TRY(launch_dense_keys(s, a, st)); break;
        case Path::kTc: LLSA_TRY(launch_dense_tc_fwd(s, a, st)); break;
        case Path::kSplit: LLSA_TRY(launch_dense_split_fwd(s, a, ws, st)); break;
        default: LLSA_TRY(launch_dense_simt_fwd(s, a, st));
    }
    return launch_dense_join(s, a, st);
}

int launch_dense_fwd_planes(const DenseShape& s, DenseArgs a, const void* const* planes, void* part, cudaStream_t st) {
    const DenseSplit p = fwd_split(s);
    a.splits = p.splits;
    a.chunk = p.chunk;
    a.part = static_cast<float*>(part);
    LLSA_TRY(launch_dense_split_fwd_planes(s, a, planes, st));
    return launch_dense_join(s, a, st);
}

static int launch_dense_bwd_sides(const DenseShape& s, DenseArgs a, void* const* planes, void* part, cudaStream_t st);

int launch_dense_bwd(const DenseShape& s, DenseArgs a, void* ws, cudaStream_t st) {
    const bool bf16 = s.dtype == LLSA_DTYPE_BF16;
    const Path path = bwd_path(s);
    if (path == Path::kNone)
        return s.R > 0 ? launch_dense_nothing(s, a, a.dq, nullptr, (long long)s.slices * s.R * s.d, nullptr, st)
                       : launch_dense_nothing(s, a, a.dk, a.dv, (long long)s.slices * s.nk * s.d, nullptr, st);
    const size_t rows = dense_rows_bytes(s);
    void* planes[4];
    if (path == Path::kSplit) {
        LLSA_TRY(make_dense_split_planes(s, a, ws, planes, st));
        ws = static_cast<char*>(ws) + dense_split_planes(s, true);
    }
    a.nl2 = static_cast<float*>(ws);
    a.nd = reinterpret_cast<float*>(static_cast<char*>(ws) + rows);
    if (path != Path::kFew) {
        const long long blocks = (long long)s.slices * (s.Rp / kDenseRowPad);
        if (blocks > 0x7fffffffLL) return LLSA_ERR_UNSUPPORTED;
        if (bf16)
            LLSA_LAUNCH("dense_rows", st, dense_rows_kernel<__nv_bfloat16><<<(unsigned)blocks, kThreads, 0, st>>>(a));
        else
            LLSA_LAUNCH("dense_rows", st, dense_rows_kernel<float><<<(unsigned)blocks, kThreads, 0, st>>>(a));
    }
    return launch_dense_bwd_sides(s, a, path == Path::kSplit ? planes : nullptr, static_cast<char*>(ws) + 2 * rows, st);
}

int launch_dense_bwd_planes(const DenseShape& s, DenseArgs a, void* const* planes, void* part, cudaStream_t st) {
    return launch_dense_bwd_sides(s, a, planes, part, st);
}

static int launch_dense_bwd_sides(const DenseShape& s, DenseArgs a, void* const* planes, void* part, cudaStream_t st) {
    const Path path = bwd_path(s);
    // dq by blocks of query rows (aq), dk and dv by blocks of keys (ak)
    const DenseSplit pq = dq_split(s), pk = dkv_split(s);
    const long long nq = (long long)s.slices * s.R * s.d, nk = (long long)s.slices * s.nk * s.d;
    DenseArgs aq = a, ak = a;
    aq.splits = pq.splits;
    aq.chunk = pq.chunk;
    ak.splits = pk.splits;
    ak.chunk = pk.chunk;
    aq.part = static_cast<float*>(part);
    ak.part = aq.part + (pq.splits > 1 ? align_up((size_t)pq.splits * nq * sizeof(float)) / sizeof(float) : 0);
    switch (path) {
        case Path::kFew: LLSA_TRY(launch_dense_few_bwd(s, aq, st)); break;
        case Path::kTc: LLSA_TRY(launch_dense_tc_bwd(s, aq, ak, st)); break;
        case Path::kSplit: LLSA_TRY(launch_dense_split_bwd(s, aq, ak, planes, st)); break;
        default: LLSA_TRY(launch_dense_simt_bwd(s, aq, ak, st));
    }
    DenseSums sums;
    if (pq.splits > 1) sums.add(aq.part, a.dq, nq, pq.splits);
    if (pk.splits > 1) {
        sums.add(ak.part, a.dk, nk, pk.splits);
        sums.add(ak.part + pk.splits * nk, a.dv, nk, pk.splits);
    }
    return launch_dense_sums(s.dtype, sums, st);
}

int launch_dense_sums(int dtype, const DenseSums& sums, cudaStream_t st) {
    if (sums.outs == 0) return LLSA_OK;
    long long most = 0;
    for (int i = 0; i < sums.outs; i++) most = std::max(most, sums.n[i]);
    const dim3 grid((unsigned)((most / 4 + kThreads - 1) / kThreads), (unsigned)sums.outs);
    if (dtype == LLSA_DTYPE_BF16)
        LLSA_LAUNCH("dense_join_sum", st, dense_join_sum_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(sums));
    else
        LLSA_LAUNCH("dense_join_sum", st, dense_join_sum_kernel<float><<<grid, kThreads, 0, st>>>(sums));
    return LLSA_OK;
}

}  // namespace llsa

using namespace llsa;

extern "C" {

size_t llsa_dense_workspace_bytes(const llsa_dense_params* p, int op) {
    DenseShape s;
    if (derive_dense(p, &s) != LLSA_OK || s.slices == 0) return 0;
    switch (op) {
        case LLSA_OP_DENSE_FWD: return dense_fwd_workspace(s);
        case LLSA_OP_DENSE_BWD: return dense_bwd_workspace(s);
        default: return 0;
    }
}

int llsa_dense_fwd(const llsa_dense_params* p, const void* q, const void* k, const void* v, const int32_t* q_len,
                   const int32_t* k_len, void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
    CallRange range("llsa_dense_fwd");
    DenseShape s;
    LLSA_TRY(derive_dense(p, &s));
    if (s.slices == 0 || s.R == 0) return LLSA_OK;
    LLSA_TRY(check_ptrs({q, o, lse}));
    if (s.nk > 0) LLSA_TRY(check_ptrs({k, v}));
    LLSA_TRY(dense_check_lens(q_len, k_len));
    const size_t need = dense_fwd_workspace(s);
    if (need > 0 && (!ws || ws_bytes < need)) return LLSA_ERR_WORKSPACE;
    if (need > 0) LLSA_TRY(check_ptrs({ws}));
    LLSA_TRY(device_ready());
    DenseArgs a = dense_args(s);
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_len = q_len;
    a.k_len = k_len;
    a.o_out = o;
    a.lse_out = lse;
    return launch_dense_fwd(s, a, ws, static_cast<cudaStream_t>(stream));
}

int llsa_dense_bwd(const llsa_dense_params* p, const void* q, const void* k, const void* v, const void* o,
                   const float* lse, const void* dout, const int32_t* q_len, const int32_t* k_len, void* dq,
                   void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    CallRange range("llsa_dense_bwd");
    DenseShape s;
    LLSA_TRY(derive_dense(p, &s));
    if (s.slices == 0 || (s.R == 0 && s.nk == 0)) return LLSA_OK;
    if (s.R > 0) LLSA_TRY(check_ptrs({q, o, lse, dout, dq}));
    if (s.nk > 0) LLSA_TRY(check_ptrs({k, v, dk, dv}));
    LLSA_TRY(dense_check_lens(q_len, k_len));
    const size_t need = dense_bwd_workspace(s);
    if (need > 0 && (!ws || ws_bytes < need)) return LLSA_ERR_WORKSPACE;
    if (need > 0) LLSA_TRY(check_ptrs({ws}));
    LLSA_TRY(device_ready());
    DenseArgs a = dense_args(s);
    a.q = q;
    a.k = k;
    a.v = v;
    a.o = o;
    a.lse = lse;
    a.dout = dout;
    a.q_len = q_len;
    a.k_len = k_len;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    return launch_dense_bwd(s, a, ws, static_cast<cudaStream_t>(stream));
}

}  // extern "C"

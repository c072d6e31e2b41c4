// gdn_norm.cu -- normalisation of the rule's outputs (gdn_norm_fwd) and the entry points of both
// passes; the backward's kernels are in gdn_norm_bwd.cu.
//
// A row x of N values (a head's output, or a hidden state): m its mean (0 for the root-mean-square
// norm), s = 1 / sqrt(mean((x - m)^2) + eps), y = ((x - m) s w + b) z sigmoid(z). One pass over memory:
// a row sits in its group's registers while its sums are formed (the squares after the mean, so
// nothing cancels), and the next row is on its way meanwhile.
#include <algorithm>
#include <cmath>

#include "gdn_norm.cuh"

namespace gdn {
namespace norm {
namespace {

constexpr int kFwdThreadsPerSm = 2048;

template <bool BLOCK, bool VEC, bool XB, bool YB, bool GATED>
__global__ void __launch_bounds__(BLOCK ? kMaxThreads : 256) fwd_kernel(Params p) {
    __shared__ float part[2][3][32];
    int half = 0;
    const int G = BLOCK ? blockDim.x : p.g;
    const int t = threadIdx.x % G;
    const int per_warp = BLOCK ? 1 : 32 / G;              // rows a warp holds at once
    const int sub = BLOCK ? 0 : (threadIdx.x & 31) / G;   // which of them is this thread's
    const int c = first_col<VEC>(0, t, G), step = col_step<VEC>(G);
    const long long stride = (long long)gridDim.x * (blockDim.x / G);
    // (the trip count is the same for all threads of a warp, and of a block where that holds one row)
    long long row0 = (long long)blockIdx.x * (blockDim.x / G) + (BLOCK ? 0 : (threadIdx.x >> 5) * per_warp);

    float w[8], b[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int col = c + e * step;
        w[e] = p.w && col < p.N ? __ldg(p.w + col) : 1.f;
        b[e] = p.b && col < p.N ? __ldg(p.b + col) : 0.f;
    }
    Eight<XB, VEC> nx;
    Eight<YB, VEC> nz;
    auto fetch = [&](long long row) {
        const int n = row < p.rows ? p.N : 0;
        nx.load(p.x, row * p.N, c, step, n);
        if constexpr (GATED) nz.load(p.z, row * p.N, c, step, n);
    };
    fetch(row0 + sub);
    for (; row0 < p.rows; row0 += stride) {
        const long long row = row0 + sub;
        float x[8], z[8];
        nx.values(x);
        if constexpr (GATED) nz.values(z);
        fetch(row + stride);
        if (!p.rms) {
            float s[1] = {0.f};
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += x[e];
            group_sum<BLOCK>(s, G, part, half);
            const float mean = s[0] * p.inv_n;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = c + e * step < p.N ? x[e] - mean : 0.f;
        }
        float q[1] = {0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) q[0] = fmaf(x[e], x[e], q[0]);
        group_sum<BLOCK>(q, G, part, half);
        const float rstd = rsqrtf(fmaf(q[0], p.inv_n, p.eps));
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = fmaf(x[e] * rstd, w[e], b[e]);
            if constexpr (GATED) x[e] *= z[e] * sigmoid(z[e]);
        }
        Eight<YB, VEC>::store(p.y, row * p.N, c, step, row < p.rows ? p.N : 0, x);
    }
}

// Rows of more than 4096 values, one a block: the weights come from the cache, as holding them as well would
// take the registers of the row.
template <int R, bool VEC, bool XB, bool YB, bool GATED>
__global__ void __launch_bounds__(kMaxThreads) wide_fwd_kernel(Params p) {
    __shared__ float part[2][3][32];
    int half = 0;
    const int G = kMaxThreads, t = threadIdx.x, step = col_step<VEC>(G);
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        Eight<XB, VEC> rx[R];
        Eight<YB, VEC> rz[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rx[i].load(p.x, row * p.N, first_col<VEC>(i, t, G), step, p.N);
            if constexpr (GATED) rz[i].load(p.z, row * p.N, first_col<VEC>(i, t, G), step, p.N);
        }
        float mean = 0.f;
        if (!p.rms) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float x[8];
                rx[i].values(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[0] += x[e];
            }
            group_sum<true>(s, G, part, half);
            mean = s[0] * p.inv_n;
        }
        float q[1] = {0.f};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float x[8];
            rx[i].values(x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xm = first_col<VEC>(i, t, G) + e * step < p.N ? x[e] - mean : 0.f;
                q[0] = fmaf(xm, xm, q[0]);
            }
        }
        group_sum<true>(q, G, part, half);
        const float rstd = rsqrtf(fmaf(q[0], p.inv_n, p.eps));
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = first_col<VEC>(i, t, G);
            float x[8], z[8];
            rx[i].values(x);
            if constexpr (GATED) rz[i].values(z);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int col = c + e * step;
                const float w = p.w && col < p.N ? __ldg(p.w + col) : 1.f;
                const float b = p.b && col < p.N ? __ldg(p.b + col) : 0.f;
                x[e] = fmaf((x[e] - mean) * rstd, w, b);
                if constexpr (GATED) x[e] *= z[e] * sigmoid(z[e]);
            }
            Eight<YB, VEC>::store(p.y, row * p.N, c, step, p.N, x);
        }
    }
}

template <int R, bool BLOCK, bool VEC, bool XB, bool YB, bool GATED>
void fwd(const Params& p, const Shape& s, int blocks, cudaStream_t st) {
    if constexpr (R == 1)
        fwd_kernel<BLOCK, VEC, XB, YB, GATED><<<blocks, s.threads, 0, st>>>(p);
    else
        wide_fwd_kernel<R, VEC, XB, YB, GATED><<<blocks, s.threads, 0, st>>>(p);
}
template <int R, bool BLOCK, bool VEC, bool XB, bool YB>
void fwd_gated(const Params& p, const Shape& s, int blocks, cudaStream_t st) {
    p.z ? fwd<R, BLOCK, VEC, XB, YB, true>(p, s, blocks, st) : fwd<R, BLOCK, VEC, XB, YB, false>(p, s, blocks, st);
}
template <int R, bool BLOCK, bool VEC>
void fwd_types(const Params& p, const Shape& s, bool xb, bool yb, int blocks, cudaStream_t st) {
    if (xb)
        yb ? fwd_gated<R, BLOCK, VEC, true, true>(p, s, blocks, st) : fwd_gated<R, BLOCK, VEC, true, false>(p, s, blocks, st);
    else
        yb ? fwd_gated<R, BLOCK, VEC, false, true>(p, s, blocks, st) : fwd_gated<R, BLOCK, VEC, false, false>(p, s, blocks, st);
}
template <int R, bool BLOCK>
void fwd_vec(const Params& p, const Shape& s, bool xb, bool yb, int blocks, cudaStream_t st) {
    s.vec ? fwd_types<R, BLOCK, true>(p, s, xb, yb, blocks, st) : fwd_types<R, BLOCK, false>(p, s, xb, yb, blocks, st);
}

gdn_status check(long long rows, int N, int x_dtype, int y_dtype, int rms, float eps, const void* x,
                 const void* y) {
    if (rows < 0 || N < 1 || (rms != 0 && rms != 1)) return GDN_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || std::isinf(eps)) return GDN_ERR_INVALID_ARG;
    if (N > kMaxN || rows >= (1LL << 40) / N) return GDN_ERR_UNSUPPORTED_SHAPE;
    for (int t : {x_dtype, y_dtype})
        if (t != GDN_DTYPE_F32 && t != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED_DTYPE;
    if (rows > 0 && (!x || !y)) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

bool misaligned(const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) & 15u; }

}  // namespace

cudaError_t launch_fwd(const Params& p, const Shape& s, bool xb, bool yb, int sms, cudaStream_t st) {
    const long long per = s.threads / s.g;
    const int blocks = (int)std::min((p.rows + per - 1) / per, (long long)sms * (kFwdThreadsPerSm / s.threads));
    if (!s.block)
        fwd_vec<1, false>(p, s, xb, yb, blocks, st);
    else if (s.r == 1)
        fwd_vec<1, true>(p, s, xb, yb, blocks, st);
    else
        fwd_vec<2, true>(p, s, xb, yb, blocks, st);
    return cudaGetLastError();
}

}  // namespace norm
}  // namespace gdn

using namespace gdn;
using namespace gdn::norm;

extern "C" {

gdn_status gdn_norm_fwd(long long rows, int N, int x_dtype, int y_dtype, int rms, float eps,
                        const void* x, const float* w, const float* b, const void* z, void* y,
                        void* stream) {
    gdn_status st = check(rows, N, x_dtype, y_dtype, rms, eps, x, y);
    if (st != GDN_OK) return st;
    for (const void* ptr : {x, (const void*)w, (const void*)b, z, (const void*)y})
        if (misaligned(ptr)) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    if (rows == 0) return GDN_OK;
    Params p{};
    p.x = x;
    p.w = w;
    p.b = b;
    p.z = z;
    p.y = y;
    p.rows = rows;
    const Shape s = shape_of(N);
    p.N = N;
    p.g = s.g;
    p.rms = rms;
    p.eps = eps;
    p.inv_n = 1.f / N;
    const cudaError_t e = launch_fwd(p, s, x_dtype == GDN_DTYPE_BF16, y_dtype == GDN_DTYPE_BF16,
                                     std::max(1, current_sm_count()), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_norm_bwd_workspace_bytes(long long rows, int N) {
    if (rows < 0 || N < 1 || N > kMaxN || rows >= (1LL << 40) / N) return 0;
    return kWsHeader + ws_round(sizeof(float) * 2 * (size_t)N * (size_t)bwd_blocks(rows, shape_of(N), kSmBound));
}

gdn_status gdn_norm_bwd(long long rows, int N, int x_dtype, int y_dtype, int rms, float eps,
                        const void* x, const float* w, const float* b, const void* z, const void* dy,
                        void* dx, void* dz, float* dw, float* db, void* workspace,
                        size_t workspace_bytes, void* stream) {
    gdn_status st = check(rows, N, x_dtype, y_dtype, rms, eps, x, dx);
    if (st != GDN_OK) return st;
    if ((rows > 0 && !dy) || (dz && !z)) return GDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdn_norm_bwd_workspace_bytes(rows, N)) return GDN_ERR_WORKSPACE;
    for (const void* ptr : {x, (const void*)w, (const void*)b, z, dy, (const void*)dx, (const void*)dz,
                            (const void*)dw, (const void*)db, (const void*)workspace})
        if (misaligned(ptr)) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    const Shape s = shape_of(N);
    Params p{};
    p.x = x;
    p.w = w;
    p.b = b;
    p.z = z;
    p.dy = dy;
    p.y = dx;
    p.dz = dz;
    p.partial = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kWsHeader);
    p.rows = rows;
    p.N = N;
    p.g = s.g;
    p.rms = rms;
    p.eps = eps;
    p.inv_n = 1.f / N;
    const int sms = std::min(std::max(1, current_sm_count()), kSmBound);
    const cudaError_t e = launch_bwd(p, s, x_dtype == GDN_DTYPE_BF16, y_dtype == GDN_DTYPE_BF16,
                                     bwd_blocks(rows, s, sms), dw, db, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

// gdn_norm.cu -- normalisation of the rule's outputs (gdn_norm_fwd) and the entry points of both
// passes; the backward's kernels are in gdn_norm_bwd.cu.
//
// A row x of N values (a head's output, or a hidden state): m its mean (0 for the root-mean-square
// norm), s = 1 / sqrt(mean((x - m)^2) + eps), y = ((x - m) s w + b) z sigmoid(z). One pass over memory:
// a row sits in its group's registers while its sums are formed, and the next row is on its way meanwhile.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "gdn_norm.cuh"

namespace gdn {
namespace norm {
namespace {

// GB: threads of a row's block; 0: rows of at most 512 values, several to a block of 256 threads
template <int GB, int R, int L, bool XB, bool YB, bool GATED>
struct Fwd {
    // More blocks with shallow rings, rather than few with deep ones: 12 -> 4 takes 29200 rows of 2000 from 87.8 to
    // 77.7 us in fp32 and from 39.0 to 37.9 in bf16, 4096 rows of 8192 from 31.4 to 23.4 in bf16. Rows of pairs with fp32
    // meet at a barrier for each row and want the depth: 73.2 against 84.3 us for 29200 rows of 1999.
    static constexpr int kAhead = L == 2 && !(XB && YB) ? 12 : 4;
    using Rows = std::conditional_t<GATED, Ring<L, R, kAhead, XB, YB>, Ring<L, R, kAhead, XB>>;
};

// (Two blocks of 512 an SM where that spills at most four registers: with one, 4096 rows of 8192 in
// bf16 take 31.4 us, not 27.5, from cold caches.)
template <int GB, int R, int L, bool XB, bool YB, bool GATED>
__global__ void __launch_bounds__(GB ? GB : 256, GB == 512 && L != 2 && XB && !GATED ? 2 : 0) fwd_kernel(Params p) {
    using Rows = typename Fwd<GB, R, L, XB, YB, GATED>::Rows;
    extern __shared__ __align__(16) char stages[];
    __shared__ float part[2][64];
    int half = 0;
    const int G = GB ? GB : p.g;
    const int t = threadIdx.x % G;
    const int rows_block = GB ? 1 : 256 / G;              // rows a block holds at once, and a warp
    const int rows_warp = GB ? 1 : 32 / G;
    const int sub = GB ? 0 : (threadIdx.x & 31) / G;      // which of the warp's is this thread's
    const long long stride = (long long)gridDim.x * rows_block;
    // (the trip count is the same for all threads of a warp, and of a block where that holds one row)
    long long row0 = (long long)blockIdx.x * rows_block + (GB ? 0 : (threadIdx.x >> 5) * rows_warp);

    const int odd = L == 2 ? (int)((row0 + sub) * p.N & 1) : 0;
    const Rows ring{(unsigned)__cvta_generic_to_shared(stages), G, t, (int)threadIdx.x, GB ? GB : 256, p.N, odd, p.rows};
    auto fetch = [&](int stage, long long row) {
        ring.template fetch<0>(stage, p.x, row);
        if constexpr (GATED) ring.template fetch<1>(stage, p.z, row);
        Rows::commit();
    };
#pragma unroll 1
    for (int k = 0; k < Rows::kAhead; ++k) fetch(k, row0 + sub + k * stride);
    pair_t w[R][4], b[R][4];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        parameter<L>(w[i], p.w, first_col<L>(i, t, G, odd), G, p.N, 1.f);
        parameter<L>(b[i], p.b, first_col<L>(i, t, G, odd), G, p.N, 0.f);
    }
    for (int stage = 0; row0 < p.rows; row0 += stride, stage = stage == Rows::kAhead ? 0 : stage + 1) {
        const long long row = row0 + sub;
        Rows::template wait<GB, GB>();
        fetch(stage == 0 ? Rows::kAhead : stage - 1, row + Rows::kAhead * stride);
        pair_t x[R][4], sq = 0, sx = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (GB && !warp_has<L>(i, t, G, p.N)) continue;
            ring.template read<0>(stage, i, row, x[i]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sq = fma2(x[i][k], x[i][k], sq);
                sx = add2(sx, x[i][k]);
            }
        }
        float mean = 0.f, var;   // mean: of what x holds
        if (p.rms) {
            float q[1] = {total(sq)};
            group_sum<GB, GB>(q, G, part, half);
            var = q[0] * p.inv_n;
        } else {
            float s[2] = {total(sq), total(sx)};
            group_sum<GB, GB>(s, G, part, half);
            mean = s[1] * p.inv_n;
            var = fmaf(-mean, mean, s[0] * p.inv_n);
            const bool again = large_mean(mean, var);
            if (GB ? again : __any_sync(0xffffffffu, again)) {   // (a warp's other rows stay as they are)
                const float off = GB || again ? mean : 0.f;
                sq = sx = 0;
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    if (GB && !warp_has<L>(i, t, G, p.N)) continue;
                    centre<L>(x[i], first_col<L>(i, t, G, odd), G, p.N, off);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sq = fma2(x[i][k], x[i][k], sq);
                        sx = add2(sx, x[i][k]);
                    }
                }
                float q[2] = {total(sq), total(sx)};
                group_sum<GB, GB>(q, G, part, half);
                if (GB || again) {
                    mean = q[1] * p.inv_n;
                    var = centred_var(q[0] * p.inv_n, mean);
                }
            }
        }
        const float rstd = rsqrtf(var + p.eps);
        const pair_t scale = both(rstd), level = both(-mean * rstd);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            if (GB && !warp_has<L>(i, t, G, p.N)) continue;
            const int c = first_col<L>(i, t, G, odd);
            float y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) x[i][k] = fma2(fma2(x[i][k], scale, level), w[i][k], b[i][k]);
            single(x[i], y);
            if constexpr (GATED) {
                float z[8];
                ring.template read<1>(stage, i, row, z);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= z[e] * sigmoid(z[e]);
            }
            store8<YB, L>(p.y, row * p.N, c, G, row < p.rows ? p.N : 0, y);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int GB, int R, int L, bool XB, bool YB, bool GATED>
cudaError_t fwd(const Params& p, const Shape& s, int sms, cudaStream_t st) {
    using Rows = typename Fwd<GB, R, L, XB, YB, GATED>::Rows;
    static std::atomic<int> known[kDevices];
    const auto kernel = fwd_kernel<GB, R, L, XB, YB, GATED>;
    constexpr int threads = GB ? GB : 256;
    const int smem = Rows::bytes(threads, s.g);
    const int resident = resident_blocks(kernel, threads, smem, known);
    if (resident < 1) return cudaErrorLaunchOutOfResources;
    const long long per = threads / s.g;
    long long blocks = (p.rows + per - 1) / per;
    if (blocks > (long long)resident * sms) {
        blocks = (long long)resident * sms;
        if (per == 1) blocks &= ~1LL;   // an even number of rows at once: a group's rows start alike
    }
    kernel<<<(int)blocks, threads, smem, st>>>(p);
    return cudaGetLastError();
}
template <int GB, int R, int L>
cudaError_t fwd_types(const Params& p, const Shape& s, bool xb, bool yb, int sms, cudaStream_t st) {
    if (xb && yb) return p.z ? fwd<GB, R, L, true, true, true>(p, s, sms, st) : fwd<GB, R, L, true, true, false>(p, s, sms, st);
    if constexpr (L < 8) {
        if (xb) return p.z ? fwd<GB, R, L, true, false, true>(p, s, sms, st) : fwd<GB, R, L, true, false, false>(p, s, sms, st);
        if (yb) return p.z ? fwd<GB, R, L, false, true, true>(p, s, sms, st) : fwd<GB, R, L, false, true, false>(p, s, sms, st);
        return p.z ? fwd<GB, R, L, false, false, true>(p, s, sms, st) : fwd<GB, R, L, false, false, false>(p, s, sms, st);
    }
    return cudaErrorInvalidValue;
}
template <int GB, int R>
cudaError_t fwd_layout(const Params& p, const Shape& s, bool xb, bool yb, int sms, cudaStream_t st) {
    if (p.N % 8 == 0 && xb && yb) return fwd_types<GB, R, 8>(p, s, xb, yb, sms, st);
    return p.N % 4 == 0 ? fwd_types<GB, R, 4>(p, s, xb, yb, sms, st) : fwd_types<GB, R, 2>(p, s, xb, yb, sms, st);
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
    if (s.g <= 32) return s.r == 1 ? fwd_layout<0, 1>(p, s, xb, yb, sms, st) : fwd_layout<0, 2>(p, s, xb, yb, sms, st);
    if (s.g == 64) return fwd_layout<64, 2>(p, s, xb, yb, sms, st);
    if (s.g == 128) return fwd_layout<128, 2>(p, s, xb, yb, sms, st);
    if (s.g == 256) return fwd_layout<256, 2>(p, s, xb, yb, sms, st);
    return fwd_layout<512, 2>(p, s, xb, yb, sms, st);
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
                                     std::max(2, current_sm_count()), reinterpret_cast<cudaStream_t>(stream));
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
    const int sms = std::min(std::max(2, current_sm_count()), kSmBound);
    const cudaError_t e = launch_bwd(p, s, x_dtype == GDN_DTYPE_BF16, y_dtype == GDN_DTYPE_BF16,
                                     sms, dw, db, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

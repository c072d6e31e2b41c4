// gdn_qk_norm.cu -- the root-mean-square norm of every query and key head with the rotation by the token's position, in one pass
// (gdn_qk_norm_fwd), and its gradients (gdn_qk_norm_bwd).
//
// A head's K channels x of one token at position n, with s = 1 / sqrt(mean(x^2) + eps):
//   u = x s w,   (y_a, y_b) = (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = n freq_i
// for the R / 2 pairs (a, b) of rotated channels, y = u for the others. Backward, with e the gradient on y turned back
// by -t:   dw = sum over rows of e x s,   d = e w,   dx = s (d - x s mean(d x s)).
//
// Bound by memory: x (and dy) read once, y (dx) written once. A row is a few hundred bytes, so a group of
// up to 32 lanes takes one token and walks over its heads: the angles' sines and cosines are formed once for them all and stay
// in registers with the weights. A lane holds both members of its pairs, so that the rotation crosses no lanes.
//
// Angles. n freq is wanted modulo a turn; in fp32 it would be off by n 2^-24. freq / 2 pi is turned into a
// 64-bit fraction of a turn (one fp64 product per pair of a group); n times that, wrapping as integers do, is the angle
// modulo a turn to n 2^-53 of it.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda_bf16.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kMaxK = 256;
constexpr int kThreads = 256;
constexpr int kDevices = 64;
constexpr int kMaxBlocks = 1024;   // of the backward: rows of partial sums in the workspace

struct QkParams {
    const void* x[2];        // q, k
    const void* dy[2];
    void* y[2];              // forward: y; backward: dx
    const float* w[2];       // null: ones
    const float* freq;
    const int* pos;          // null: the token's place in its sequence
    float* partial;          // backward: [blocks][2][K]
    long long tokens, x_stride[2], y_stride[2], dy_stride[2];   // values from one token to the next
    long long groups;        // groups of lanes with work: tokens x parts
    int T, H[2], K, R, interleaved, G, parts, per;              // a token's heads in `parts` of `per` each
    float eps, inv_k;
};

template <int VEC, bool BF>
struct Raw {   // VEC values as stored
    static constexpr int kBytes = VEC * (BF ? 2 : 4);
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    unsigned u[kWords];
    __device__ __forceinline__ void load(const void* base, long long at) {
        const char* p = (const char*)base + at * (BF ? 2 : 4);
        if constexpr (kBytes == 2) {
            u[0] = *reinterpret_cast<const unsigned short*>(p);
        } else if constexpr (kBytes == 4) {
            u[0] = __ldg(reinterpret_cast<const unsigned*>(p));
        } else if constexpr (kBytes == 8) {
            const uint2 t = __ldg(reinterpret_cast<const uint2*>(p));
            u[0] = t.x, u[1] = t.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 t = __ldg(reinterpret_cast<const uint4*>(p) + i);
                u[4 * i] = t.x, u[4 * i + 1] = t.y, u[4 * i + 2] = t.z, u[4 * i + 3] = t.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (unsigned& t : u) t = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (BF) return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
        return __uint_as_float(u[BF ? 0 : i]);
    }
};

template <int VEC, bool BF>
__device__ __forceinline__ void store(void* base, long long at, const float (&f)[VEC]) {
    char* p = (char*)base + at * (BF ? 2 : 4);
    if constexpr (BF) {
        if constexpr (VEC == 1) {
            *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(f[0]);
        } else {
            unsigned u[VEC / 2 > 0 ? VEC / 2 : 1];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                const __nv_bfloat162 t = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                u[i] = *reinterpret_cast<const unsigned*>(&t);
            }
            if constexpr (VEC == 2) *reinterpret_cast<unsigned*>(p) = u[0];
            if constexpr (VEC == 4) *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
            if constexpr (VEC == 8) *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    } else {
        if constexpr (VEC == 1) *reinterpret_cast<float*>(p) = f[0];
        if constexpr (VEC == 2) *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i)
            reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    }
}

// Which channels a lane holds: units of VEC pairs; unit u's first and second members start at channel first(u) and
// second(u) (rotated pairs apart by R / 2 or side by side; the unrotated rest in two runs the same way).
template <int VEC, int UPL>
struct Units {
    int n, nr, lane, G, K, R, il;
    __device__ __forceinline__ Units(const QkParams& p, int l)
        : n(p.K / (2 * VEC)), nr(p.R / (2 * VEC)), lane(l), G(p.G), K(p.K), R(p.R), il(p.interleaved) {}
    __device__ __forceinline__ int unit(int i) const { return lane + i * G; }
    __device__ __forceinline__ bool has(int i) const { return unit(i) < n; }
    __device__ __forceinline__ bool turned(int i) const { return unit(i) < nr; }
    __device__ __forceinline__ int first(int i) const {
        const int u = unit(i);
        if (u < nr) return il ? 2 * VEC * u : VEC * u;
        return R + VEC * (u - nr);
    }
    __device__ __forceinline__ int second(int i) const {
        const int u = unit(i);
        if (u < nr) return il ? 2 * VEC * u + VEC : R / 2 + VEC * u;
        return R + (K - R) / 2 + VEC * (u - nr);
    }
    // the number of the unit's first pair among the rotated ones
    __device__ __forceinline__ int pair0(int i) const { return VEC * unit(i); }
};

// In an interleaved unit the 2 VEC values lie in order: pair e is (2 e, 2 e + 1). f: the values in the order of the
// two loads; e-th pair's members:
template <int VEC>
__device__ __forceinline__ void members(const float (&a)[VEC], const float (&b)[VEC], int e, bool il, float& x, float& y) {
    x = a[e];
    y = b[e];
    if (VEC == 1 || !il) return;
    const int i = 2 * e;
    x = i < VEC ? a[i % VEC] : b[i % VEC];
    y = i + 1 < VEC ? a[(i + 1) % VEC] : b[(i + 1) % VEC];
}
template <int VEC>
__device__ __forceinline__ void put(float (&a)[VEC], float (&b)[VEC], int e, bool il, float x, float y) {
    if (VEC == 1 || !il) {
        a[e] = x;
        b[e] = y;
        return;
    }
    const int i = 2 * e;
    (i < VEC ? a[i % VEC] : b[i % VEC]) = x;
    (i + 1 < VEC ? a[(i + 1) % VEC] : b[(i + 1) % VEC]) = y;
}

// cosines and sines of a lane's pairs at position n (1 and 0 for channels that are not rotated)
template <int VEC, int UPL, bool IL>
__device__ __forceinline__ void turns(const QkParams& p, const Units<VEC, UPL>& un, const unsigned long long (&step)[UPL][VEC],
                                      int n, float (&c)[UPL][VEC], float (&s)[UPL][VEC]) {
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const unsigned long long a = (unsigned long long)(long long)n * step[i][e];
            sincospif((float)(int)(a >> 32) * 0x1p-31f, &s[i][e], &c[i][e]);
        }
}
template <int VEC, int UPL>
__device__ __forceinline__ void steps(const QkParams& p, const Units<VEC, UPL>& un, unsigned long long (&step)[UPL][VEC]) {
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            step[i][e] = 0;
            if (un.has(i) && un.turned(i)) {
                const double f = (double)__ldg(p.freq + un.pair0(i) + e) * 0.15915494309189533577;   // 1 / 2 pi
                step[i][e] = __double2ull_rd((f - floor(f)) * 0x1p64);
            }
        }
}

__device__ __forceinline__ float group_sum(float x, int G) {
    for (int off = G / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

template <int VEC, int UPL, bool XB, bool YB, bool IL>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const QkParams p) {
    const int G = p.G, lane = threadIdx.x % G;
    const Units<VEC, UPL> un(p, lane);
    const long long group = ((long long)blockIdx.x * kThreads + threadIdx.x) / G;
    // (a whole warp leaves together or stays: groups without work take part in the exchanges)
    const bool live = group < p.groups;
    const long long token = live ? group / p.parts : 0;
    const int part = live ? (int)(group - token * p.parts) : 0;
    const int h_end = live ? min(p.H[0] + p.H[1], (part + 1) * p.per) : 0;
    unsigned long long step[UPL][VEC];
    float c[UPL][VEC], s[UPL][VEC];
    steps(p, un, step);
    turns<VEC, UPL, IL>(p, un, step, p.pos ? (live ? __ldg(p.pos + token) : 0) : (int)(token % p.T), c, s);
    int h = part * p.per;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
        const int h0 = side ? p.H[0] : 0, hn = min(h_end, h0 + p.H[side]);
        if (!__any_sync(0xffffffffu, h < hn)) continue;
        const long long xb = token * p.x_stride[side], yb = token * p.y_stride[side];
        float wa[UPL][VEC], wb[UPL][VEC];
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                wa[i][e] = wb[i][e] = 1.f;
                if (un.has(i) && p.w[side]) {
                    wa[i][e] = __ldg(p.w[side] + un.first(i) + e);
                    wb[i][e] = __ldg(p.w[side] + un.second(i) + e);
                }
            }
        // two heads at a time: the second one's loads are under way while the first is worked on
        Raw<VEC, XB> a[2][UPL], b[2][UPL];
        auto fetch = [&](int k, int hh) {
#pragma unroll
            for (int i = 0; i < UPL; ++i) {
                a[k][i].zero();
                b[k][i].zero();
                if (un.has(i) && hh < hn) {
                    a[k][i].load(p.x[side], xb + (long long)(hh - h0) * p.K + un.first(i));
                    b[k][i].load(p.x[side], xb + (long long)(hh - h0) * p.K + un.second(i));
                }
            }
        };
        fetch(0, h);
        while (__any_sync(0xffffffffu, h < hn)) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                fetch(k ^ 1, h + 1);
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < UPL; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        sq = fmaf(a[k][i].at(e), a[k][i].at(e), sq);
                        sq = fmaf(b[k][i].at(e), b[k][i].at(e), sq);
                    }
                const float rstd = rsqrtf(fmaf(group_sum(sq, G), p.inv_k, p.eps));
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    float ya[VEC], yb_[VEC], va[VEC], vb[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        va[e] = a[k][i].at(e) * rstd * wa[i][e];
                        vb[e] = b[k][i].at(e) * rstd * wb[i][e];
                    }
                    const bool on = un.turned(i);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        float x, y;
                        members(va, vb, e, IL, x, y);
                        put(ya, yb_, e, IL, x * c[i][e] - y * s[i][e], y * c[i][e] + x * s[i][e]);
                    }
                    if (un.has(i) && h < hn) {
                        const long long at = yb + (long long)(h - h0) * p.K;
                        store<VEC, YB>(p.y[side], at + un.first(i), on ? ya : va);
                        store<VEC, YB>(p.y[side], at + un.second(i), on ? yb_ : vb);
                    }
                }
                h = h < hn ? h + 1 : h;
            }
        }
    }
}

// The gradients. Groups walk over (token, part) items in a fixed order; dw of their rows stays in registers, is joined in
// shared memory at the end and goes to the workspace, one row of sums a block; qk_sum_kernel adds those up in order.
template <int VEC, int UPL, bool XB, bool YB, bool IL>
__global__ void __launch_bounds__(kThreads) qk_bwd_kernel(const QkParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ float sums[2][kMaxK];
    const int G = p.G, lane = threadIdx.x % G;
    const Units<VEC, UPL> un(p, lane);
    const int mine = threadIdx.x / G, rows = kThreads / G;
    unsigned long long step[UPL][VEC];
    steps(p, un, step);
    float w[2][2][UPL][VEC], dw[2][2][UPL][VEC];
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
        for (int i = 0; i < UPL; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                w[side][0][i][e] = w[side][1][i][e] = 1.f;
                dw[side][0][i][e] = dw[side][1][i][e] = 0.f;
                if (un.has(i) && p.w[side]) {
                    w[side][0][i][e] = __ldg(p.w[side] + un.first(i) + e);
                    w[side][1][i][e] = __ldg(p.w[side] + un.second(i) + e);
                }
            }
    const long long stride = (long long)gridDim.x * rows;
    for (long long g0 = (long long)blockIdx.x * rows; g0 < p.groups; g0 += stride) {
        const long long group = g0 + mine;
        const bool live = group < p.groups;
        const long long token = live ? group / p.parts : 0;
        const int part = live ? (int)(group - token * p.parts) : 0;
        const int h_end = live ? min(p.H[0] + p.H[1], (part + 1) * p.per) : 0;
        float c[UPL][VEC], s[UPL][VEC];
        turns<VEC, UPL, IL>(p, un, step, p.pos ? (live ? __ldg(p.pos + token) : 0) : (int)(token % p.T), c, s);
        int h = part * p.per;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const int h0 = side ? p.H[0] : 0, hn = min(h_end, h0 + p.H[side]);
            const long long xb = token * p.x_stride[side], db = token * p.dy_stride[side], yb = token * p.y_stride[side];
#pragma unroll 1
            while (__any_sync(0xffffffffu, h < hn)) {
                Raw<VEC, XB> a[UPL], b[UPL];
                Raw<VEC, YB> da[UPL], db_[UPL];
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    a[i].zero();
                    b[i].zero();
                    da[i].zero();
                    db_[i].zero();
                    if (un.has(i) && h < hn) {
                        const long long at = xb + (long long)(h - h0) * p.K, dat = db + (long long)(h - h0) * p.K;
                        a[i].load(p.x[side], at + un.first(i));
                        b[i].load(p.x[side], at + un.second(i));
                        da[i].load(p.dy[side], dat + un.first(i));
                        db_[i].load(p.dy[side], dat + un.second(i));
                    }
                }
                float ea[UPL][VEC], eb[UPL][VEC];
                float sq = 0.f, dot = 0.f;
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    float va[VEC], vb[VEC];
                    const bool on = un.turned(i);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        va[e] = ea[i][e] = da[i].at(e);
                        vb[e] = eb[i][e] = db_[i].at(e);
                    }
                    if (on) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            float x, y;
                            members(va, vb, e, IL, x, y);
                            put(ea[i], eb[i], e, IL, x * c[i][e] + y * s[i][e], y * c[i][e] - x * s[i][e]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        sq = fmaf(a[i].at(e), a[i].at(e), sq);
                        sq = fmaf(b[i].at(e), b[i].at(e), sq);
                        dot = fmaf(ea[i][e] * w[side][0][i][e], a[i].at(e), dot);
                        dot = fmaf(eb[i][e] * w[side][1][i][e], b[i].at(e), dot);
                    }
                }
                const float rstd = rsqrtf(fmaf(group_sum(sq, G), p.inv_k, p.eps));
                const float mean = group_sum(dot, G) * p.inv_k * rstd;   // of d u
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    float xa[VEC], xb_[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float ua = a[i].at(e) * rstd, ub = b[i].at(e) * rstd;
                        dw[side][0][i][e] = fmaf(ea[i][e], ua, dw[side][0][i][e]);
                        dw[side][1][i][e] = fmaf(eb[i][e], ub, dw[side][1][i][e]);
                        xa[e] = rstd * fmaf(-ua, mean, ea[i][e] * w[side][0][i][e]);
                        xb_[e] = rstd * fmaf(-ub, mean, eb[i][e] * w[side][1][i][e]);
                    }
                    if (un.has(i) && h < hn) {
                        const long long at = yb + (long long)(h - h0) * p.K;
                        store<VEC, XB>(p.y[side], at + un.first(i), xa);
                        store<VEC, XB>(p.y[side], at + un.second(i), xb_);
                    }
                }
                h = h < hn ? h + 1 : h;
            }
        }
    }
    if (!p.partial) return;
    // the groups of a warp first (their lanes hold the same channels), then the warps in turn
    for (int w0 = 0; w0 < kThreads / 32; ++w0) {
        if (threadIdx.x / 32 == w0) {
#pragma unroll
            for (int side = 0; side < 2; ++side)
#pragma unroll
                for (int half = 0; half < 2; ++half)
#pragma unroll
                    for (int i = 0; i < UPL; ++i)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            float t = dw[side][half][i][e];
                            for (int off = 16; off >= G; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
                            if ((threadIdx.x & 31) < G && un.has(i)) {
                                float* to = &sums[side][(half ? un.second(i) : un.first(i)) + e];
                                *to = w0 ? *to + t : t;
                            }
                        }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < 2 * p.K; i += kThreads)
        p.partial[(long long)blockIdx.x * 2 * p.K + i] = sums[i / p.K][i % p.K];
}

// dw[side][i] = the sum over the blocks' rows: a block of 256 threads for 8 columns, 32 partial sums each
__global__ void __launch_bounds__(kThreads) qk_sum_kernel(const float* partial, int blocks, int K, float* dwq, float* dwk) {
    __shared__ float part[32][9];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int col = threadIdx.x % 8, row = threadIdx.x / 8, i = blockIdx.x * 8 + col;
    float t = 0.f;
    if (i < 2 * K)
        for (int b = row; b < blocks; b += 32) t += __ldcg(partial + (long long)b * 2 * K + i);
    part[row][col] = t;
    __syncthreads();
    if (threadIdx.x < 8 && i < 2 * K) {
        float total = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) total += part[r][threadIdx.x];
        float* to = i < K ? dwq : dwk;
        if (to) to[i % K] = total;
    }
}

// ------------------------------------------------------------------------------------ host

gdn_status check(const gdn_qk_problem* p) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B < 1 || p->T < 0 || p->Hq < 1 || p->Hk < 1 || p->K < 2 || p->R < 0) return GDN_ERR_INVALID_ARG;
    if (p->interleaved != 0 && p->interleaved != 1) return GDN_ERR_INVALID_ARG;
    if (!(p->eps >= 0.f) || std::isinf(p->eps)) return GDN_ERR_INVALID_ARG;
    if (p->K > kMaxK || p->K % 2 || p->R > p->K || p->R % 2) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (p->Hq > 4096 || p->Hk > 4096 || (long long)p->B * p->T >= (1LL << 31)) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (p->q_stride < (long long)p->Hq * p->K || p->k_stride < (long long)p->Hk * p->K) return GDN_ERR_INVALID_ARG;
    if (p->q_stride >= (1LL << 31) || p->k_stride >= (1LL << 31)) return GDN_ERR_UNSUPPORTED_SHAPE;
    for (int t : {p->x_dtype, p->y_dtype})
        if (t != GDN_DTYPE_F32 && t != GDN_DTYPE_BF16) return GDN_ERR_UNSUPPORTED_DTYPE;
    return GDN_OK;
}

// The most pairs a lane may hold at once: 16 bytes of the wider type, and as many as alignment and the channels' runs allow.
int widest(const gdn_qk_problem& p, std::initializer_list<const void*> xs, std::initializer_list<const void*> ys) {
    int vec = p.x_dtype == GDN_DTYPE_F32 || p.y_dtype == GDN_DTYPE_F32 ? 4 : 8;
    const int run = p.interleaved ? p.R : p.R / 2, rest = (p.K - p.R) / 2;
    const int xe = p.x_dtype == GDN_DTYPE_BF16 ? 2 : 4, ye = p.y_dtype == GDN_DTYPE_BF16 ? 2 : 4;
    for (; vec > 1; vec /= 2) {
        bool ok = run % (p.interleaved ? 2 * vec : vec) == 0 && rest % vec == 0 && p.K % (2 * vec) == 0 &&
                  p.q_stride % vec == 0 && p.k_stride % vec == 0;
        for (const void* x : xs) ok &= reinterpret_cast<uintptr_t>(x) % (vec * xe) == 0;
        for (const void* y : ys) ok &= reinterpret_cast<uintptr_t>(y) % (vec * ye) == 0;
        if (ok) break;
    }
    return vec;
}

bool off_type(const void* ptr, int dtype) {
    return reinterpret_cast<uintptr_t>(ptr) % (dtype == GDN_DTYPE_BF16 ? 2 : 4) != 0;
}

void fill(QkParams& c, const gdn_qk_problem& p, int vec) {
    c.tokens = (long long)p.B * p.T;
    c.T = p.T;
    c.H[0] = p.Hq;
    c.H[1] = p.Hk;
    c.K = p.K;
    c.R = p.R;
    c.interleaved = p.interleaved;
    c.eps = p.eps;
    c.inv_k = 1.f / p.K;
    c.G = 1;
    while (c.G < 32 && c.G < p.K / (2 * vec)) c.G *= 2;
}

// A token's heads in parts: whole where the tokens alone give every SM its warps; else so many that they do (each
// part forms the angles again).
void split(QkParams& c, long long lanes_wanted) {
    const int heads = c.H[0] + c.H[1];
    const long long want = std::max(1LL, lanes_wanted / std::max(1LL, c.tokens * c.G));
    c.parts = (int)std::min<long long>(heads, want);
    c.per = (heads + c.parts - 1) / c.parts;
    c.parts = (heads + c.per - 1) / c.per;
    c.groups = c.tokens * c.parts;
}

template <int VEC, int UPL, bool XB, bool YB>
cudaError_t fwd(const QkParams& c, cudaStream_t s) {
    const long long blocks = (c.groups * c.G + kThreads - 1) / kThreads;
    if (c.interleaved)
        qk_fwd_kernel<VEC, UPL, XB, YB, true><<<(unsigned)blocks, kThreads, 0, s>>>(c);
    else
        qk_fwd_kernel<VEC, UPL, XB, YB, false><<<(unsigned)blocks, kThreads, 0, s>>>(c);
    return cudaGetLastError();
}
template <int VEC, int UPL, bool XB, bool YB>
cudaError_t bwd(const QkParams& c, int blocks, cudaStream_t s) {
    if (c.interleaved)
        qk_bwd_kernel<VEC, UPL, XB, YB, true><<<blocks, kThreads, 0, s>>>(c);
    else
        qk_bwd_kernel<VEC, UPL, XB, YB, false><<<blocks, kThreads, 0, s>>>(c);
    return cudaGetLastError();
}
// (UPL: units of VEC pairs a lane, 32 lanes holding a row of up to 256 channels)
template <bool XB, bool YB, class F>
cudaError_t by_vec(int vec, F f) {
    if constexpr (XB && YB)
        if (vec == 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    if (vec == 4) return f(std::integral_constant<int, 4>(), std::integral_constant<int, 1>());
    if (vec == 2) return f(std::integral_constant<int, 2>(), std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 1>(), std::integral_constant<int, 4>());
}
template <class F>
cudaError_t by_type(const gdn_qk_problem& p, F f) {
    const bool xb = p.x_dtype == GDN_DTYPE_BF16, yb = p.y_dtype == GDN_DTYPE_BF16;
    if (xb) return yb ? f(std::true_type(), std::true_type()) : f(std::true_type(), std::false_type());
    return yb ? f(std::false_type(), std::true_type()) : f(std::false_type(), std::false_type());
}

int bwd_blocks(const QkParams& c, int sms) {
    const long long rows = kThreads / c.G;
    return (int)std::max(1LL, std::min<long long>({(c.groups + rows - 1) / rows, 3LL * sms, (long long)kMaxBlocks}));
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_qk_norm_fwd(const gdn_qk_problem* p, const void* q, const void* k, const float* wq, const float* wk,
                           const float* freq, const int* positions, void* yq, void* yk, void* stream) {
    gdn_status st = check(p);
    if (st != GDN_OK) return st;
    const bool any = p->T > 0;
    if (any && (!q || !k || !yq || !yk || (p->R > 0 && !freq))) return GDN_ERR_INVALID_ARG;
    for (const void* x : {q, k})
        if (off_type(x, p->x_dtype)) return GDN_ERR_MISALIGNED;
    for (const void* y : {(const void*)yq, (const void*)yk})
        if (off_type(y, p->y_dtype)) return GDN_ERR_MISALIGNED;
    for (const void* f : {(const void*)wq, (const void*)wk, (const void*)freq, (const void*)positions})
        if (off_type(f, GDN_DTYPE_F32)) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    if (!any) return GDN_OK;
    const int vec = widest(*p, {q, k}, {yq, yk});
    QkParams c{};
    fill(c, *p, vec);
    c.x[0] = q, c.x[1] = k;
    c.y[0] = yq, c.y[1] = yk;
    c.w[0] = wq, c.w[1] = wk;
    c.freq = freq;
    c.pos = positions;
    c.x_stride[0] = p->q_stride, c.x_stride[1] = p->k_stride;
    c.y_stride[0] = (long long)p->Hq * p->K, c.y_stride[1] = (long long)p->Hk * p->K;
    split(c, 1024LL * std::max(1, current_sm_count()));
    if ((c.groups * c.G + kThreads - 1) / kThreads >= (1LL << 31)) return GDN_ERR_UNSUPPORTED_SHAPE;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(*p, [&](auto xb, auto yb) {
        return by_vec<xb.value, yb.value>(vec, [&](auto v, auto u) { return fwd<v.value, u.value, xb.value, yb.value>(c, s); });
    });
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_bwd_workspace_bytes(int K) {
    if (K < 2 || K > kMaxK || K % 2) return 0;
    return kWsHeader + ws_round(sizeof(float) * 2 * (size_t)K * kMaxBlocks);
}

gdn_status gdn_qk_norm_bwd(const gdn_qk_problem* p, const void* q, const void* k, const float* wq, const float* wk,
                           const float* freq, const int* positions, const void* dyq, const void* dyk, void* dq,
                           void* dk, float* dwq, float* dwk, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = check(p);
    if (st != GDN_OK) return st;
    const bool any = p->T > 0;
    if (any && (!q || !k || !dyq || !dyk || !dq || !dk || (p->R > 0 && !freq))) return GDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdn_qk_norm_bwd_workspace_bytes(p->K)) return GDN_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return GDN_ERR_MISALIGNED;
    for (const void* x : {q, k, (const void*)dq, (const void*)dk})
        if (off_type(x, p->x_dtype)) return GDN_ERR_MISALIGNED;
    for (const void* y : {dyq, dyk})
        if (off_type(y, p->y_dtype)) return GDN_ERR_MISALIGNED;
    for (const void* f : {(const void*)wq, (const void*)wk, (const void*)freq, (const void*)positions, (const void*)dwq, (const void*)dwk})
        if (off_type(f, GDN_DTYPE_F32)) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    if (!any && !dwq && !dwk) return GDN_OK;
    const int vec = widest(*p, {q, k, dq, dk}, {dyq, dyk});
    QkParams c{};
    fill(c, *p, vec);
    c.x[0] = q, c.x[1] = k;
    c.dy[0] = dyq, c.dy[1] = dyk;
    c.y[0] = dq, c.y[1] = dk;
    c.w[0] = wq, c.w[1] = wk;
    c.freq = freq;
    c.pos = positions;
    c.x_stride[0] = c.y_stride[0] = p->q_stride, c.x_stride[1] = c.y_stride[1] = p->k_stride;
    c.dy_stride[0] = (long long)p->Hq * p->K, c.dy_stride[1] = (long long)p->Hk * p->K;
    if (dwq || dwk) c.partial = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kWsHeader);
    const int sms = std::max(1, current_sm_count());
    if (p->T == 0) c.T = 1;   // no tokens: the sums are zeros
    split(c, 3LL * kThreads * sms);
    const int blocks = bwd_blocks(c, sms);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = by_type(*p, [&](auto xb, auto yb) {
        return by_vec<xb.value, yb.value>(vec, [&](auto v, auto u) { return bwd<v.value, u.value, xb.value, yb.value>(c, blocks, s); });
    });
    if (e != cudaSuccess || !c.partial) return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((2 * p->K + 7) / 8);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, qk_sum_kernel, (const float*)c.partial, blocks, p->K, dwq, dwk);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

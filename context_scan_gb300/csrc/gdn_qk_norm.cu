// gdn_qk_norm.cu -- the root-mean-square norm of every query and key head with the rotation by the token's position, in one pass
// (gdn_qk_norm_fwd), and its gradients (gdn_qk_norm_bwd).
//
// A head's K channels x of one token at position n, with s = 1 / sqrt(mean(x^2) + eps):
//   u = x s w,   (y_a, y_b) = (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = n freq_i
// for the R / 2 pairs (a, b) of rotated channels, y = u for the others. Backward, with e the gradient on y turned back
// by -t:   dw = sum over rows of e x s,   d = e w,   dx = s (d - x s mean(d x s)).
//
// Bound by memory: x (and dy) read once, y (dx) written once. A row is a few hundred bytes, so a group of
// up to 32 lanes takes one token and walks over some of its heads: the angles' sines and cosines are formed once for them all
// and stay in registers with the weights. A lane holds both members of its pairs, so that the rotation crosses no lanes. A
// block works on the queries or on the keys (so that it holds one set of weights and, backward, one of their sums), and
// a group reads its next head's row while it works on one.
//
// Angles. n freq is wanted modulo a turn; in fp32 it would be off by n 2^-24. freq / 2 pi is turned into a
// 64-bit fraction of a turn (one fp64 product per pair and block); n times that, wrapping as integers do, is the angle
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

struct Side {                // the queries, or the keys
    const void* x;
    const void* dy;
    void* y;                 // forward: y; backward: dx
    const float* w;          // null: ones
    long long x_stride, y_stride, dy_stride;   // values from one token to the next
    long long groups;        // groups of lanes with work: tokens x parts
    int H, parts, per;       // a token's heads in `parts` of `per` each
};
struct QkParams {
    Side side[2];
    const float* freq;
    const int* pos;          // null: the token's place in its sequence
    float* partial;          // backward: [blocks][K] sums
    int blocks0;             // the first blocks are the queries'
    int T, K, R, interleaved, G;
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

// Every rotated pair's turn from one position to the next, as a 64-bit fraction, in shared memory (zeros for pairs
// that are not rotated).
__device__ __forceinline__ void make_steps(const QkParams& p, unsigned long long* step) {
    for (int i = threadIdx.x; i < kMaxK / 2; i += kThreads) {
        step[i] = 0;
        if (i < p.R / 2) {
            const double f = (double)__ldg(p.freq + i) * 0.15915494309189533577;   // 1 / 2 pi
            step[i] = __double2ull_rd((f - floor(f)) * 0x1p64);
        }
    }
    __syncthreads();
}
// cosines and sines of a lane's pairs at position n (1 and 0 for channels that are not rotated)
template <int VEC, int UPL>
__device__ __forceinline__ void turns(const Units<VEC, UPL>& un, const unsigned long long* step, int n, float (&c)[UPL][VEC],
                                      float (&s)[UPL][VEC]) {
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const unsigned long long a = un.has(i) ? (unsigned long long)(long long)n * step[un.pair0(i) + e] : 0;
            sincospif((float)(int)(a >> 32) * 0x1p-31f, &s[i][e], &c[i][e]);
        }
}

__device__ __forceinline__ float group_sum(float x, int G) {
    for (int off = G / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// The work of a group in one round: a token's heads h0 .. h1 - 1 (none: h0 == h1).
struct Work {
    long long token;
    int h0, h1;
    __device__ __forceinline__ Work(const Side& s, long long group) {
        token = 0;
        h0 = h1 = 0;
        if (group < s.groups) {
            token = s.parts == 1 ? group : group / s.parts;
            h0 = (int)(group - token * s.parts) * s.per;
            h1 = min(s.H, h0 + s.per);
        }
    }
};

template <int VEC, int UPL, bool BF>
struct Row {   // a head's values that a lane holds
    Raw<VEC, BF> a[UPL], b[UPL];
    __device__ __forceinline__ void load(const Units<VEC, UPL>& un, const void* base, long long at, bool on) {
#pragma unroll
        for (int i = 0; i < UPL; ++i)
            if (on && un.has(i)) {
                a[i].load(base, at + un.first(i));
                b[i].load(base, at + un.second(i));
            }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < UPL; ++i) {
            a[i].zero();
            b[i].zero();
        }
    }
};

template <int VEC, int UPL, bool XB, bool YB, bool IL>
__global__ void __launch_bounds__(kThreads) qk_fwd_kernel(const __grid_constant__ QkParams p) {
    __shared__ unsigned long long step[kMaxK / 2];
    make_steps(p, step);
    const bool keys = (int)blockIdx.x >= p.blocks0;
    const Side& s = p.side[keys];
    const int block = keys ? blockIdx.x - p.blocks0 : blockIdx.x, blocks = keys ? gridDim.x - p.blocks0 : p.blocks0;
    const int G = p.G;
    const Units<VEC, UPL> un(p, threadIdx.x % G);
    const int rows = kThreads / G, mine = threadIdx.x / G;
    float wa[UPL][VEC], wb[UPL][VEC];
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            wa[i][e] = wb[i][e] = 1.f;
            if (un.has(i) && s.w) {
                wa[i][e] = __ldg(s.w + un.first(i) + e);
                wb[i][e] = __ldg(s.w + un.second(i) + e);
            }
        }
    // (a warp's groups take part in its exchanges whether or not they have work)
    for (long long g0 = (long long)block * rows; g0 < s.groups; g0 += (long long)blocks * rows) {
        const Work wk(s, g0 + mine);
        Row<VEC, UPL, XB> row[2];
        row[0].zero();
        row[1].zero();
        long long xat = wk.token * s.x_stride + (long long)wk.h0 * p.K, yat = wk.token * s.y_stride + (long long)wk.h0 * p.K;
        row[0].load(un, s.x, xat, wk.h0 < wk.h1);
        float c[UPL][VEC], sn[UPL][VEC];
        turns<VEC, UPL>(un, step, p.pos ? (wk.h0 < wk.h1 ? __ldg(p.pos + wk.token) : 0) : (int)(wk.token % p.T), c, sn);
        for (int h = wk.h0; __any_sync(0xffffffffu, h < wk.h1); h += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                row[k ^ 1].load(un, s.x, xat + p.K, h + k + 1 < wk.h1);
                float sq = 0.f;
#pragma unroll
                for (int i = 0; i < UPL; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        sq = fmaf(row[k].a[i].at(e), row[k].a[i].at(e), sq);
                        sq = fmaf(row[k].b[i].at(e), row[k].b[i].at(e), sq);
                    }
                const float rstd = rsqrtf(fmaf(group_sum(sq, G), p.inv_k, p.eps));
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    float va[VEC], vb[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        va[e] = row[k].a[i].at(e) * rstd * wa[i][e];
                        vb[e] = row[k].b[i].at(e) * rstd * wb[i][e];
                    }
                    if (un.turned(i)) {
                        float ya[VEC], yb[VEC];
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            float x, y;
                            members(va, vb, e, IL, x, y);
                            put(ya, yb, e, IL, x * c[i][e] - y * sn[i][e], y * c[i][e] + x * sn[i][e]);
                        }
#pragma unroll
                        for (int e = 0; e < VEC; ++e) va[e] = ya[e], vb[e] = yb[e];
                    }
                    if (un.has(i) && h + k < wk.h1) {
                        store<VEC, YB>(s.y, yat + un.first(i), va);
                        store<VEC, YB>(s.y, yat + un.second(i), vb);
                    }
                }
                xat += p.K;
                yat += p.K;
            }
        }
    }
}

// The gradients. Groups walk over their work in a fixed order; dw of their rows stays in registers, is joined in
// shared memory at the end and goes to the workspace, one row of sums a block; qk_sum_kernel adds those up in order.
// (Two blocks an SM: at one, with two rows on their way in each group, memory waits for the lanes.)
template <int VEC, int UPL, bool XB, bool YB, bool IL>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_kernel(const __grid_constant__ QkParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ unsigned long long step[kMaxK / 2];
    __shared__ float sums[kMaxK];
    make_steps(p, step);
    const bool keys = (int)blockIdx.x >= p.blocks0;
    const Side& s = p.side[keys];
    const int block = keys ? blockIdx.x - p.blocks0 : blockIdx.x, blocks = keys ? gridDim.x - p.blocks0 : p.blocks0;
    const int G = p.G;
    const Units<VEC, UPL> un(p, threadIdx.x % G);
    const int rows = kThreads / G, mine = threadIdx.x / G;
    float w[2][UPL][VEC], dw[2][UPL][VEC];
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[0][i][e] = w[1][i][e] = 1.f;
            dw[0][i][e] = dw[1][i][e] = 0.f;
            if (un.has(i) && s.w) {
                w[0][i][e] = __ldg(s.w + un.first(i) + e);
                w[1][i][e] = __ldg(s.w + un.second(i) + e);
            }
        }
    for (long long g0 = (long long)block * rows; g0 < s.groups; g0 += (long long)blocks * rows) {
        const Work wk(s, g0 + mine);
        Row<VEC, UPL, XB> row[2];
        Row<VEC, UPL, YB> grad[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            row[k].zero();
            grad[k].zero();
        }
        const long long first = (long long)wk.h0 * p.K;
        long long xat = wk.token * s.x_stride + first, dat = wk.token * s.dy_stride + first, yat = wk.token * s.y_stride + first;
        row[0].load(un, s.x, xat, wk.h0 < wk.h1);
        grad[0].load(un, s.dy, dat, wk.h0 < wk.h1);
        float c[UPL][VEC], sn[UPL][VEC];
        turns<VEC, UPL>(un, step, p.pos ? (wk.h0 < wk.h1 ? __ldg(p.pos + wk.token) : 0) : (int)(wk.token % p.T), c, sn);
        for (int h = wk.h0; __any_sync(0xffffffffu, h < wk.h1); h += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                row[k ^ 1].load(un, s.x, xat + p.K, h + k + 1 < wk.h1);
                grad[k ^ 1].load(un, s.dy, dat + p.K, h + k + 1 < wk.h1);
                const bool on = h + k < wk.h1;
                float sq = 0.f, dot = 0.f, ea[UPL][VEC], eb[UPL][VEC];   // e: dy turned back
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    float va[VEC], vb[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        va[e] = ea[i][e] = grad[k].a[i].at(e);
                        vb[e] = eb[i][e] = grad[k].b[i].at(e);
                    }
                    if (un.turned(i)) {
#pragma unroll
                        for (int e = 0; e < VEC; ++e) {
                            float x, y;
                            members(va, vb, e, IL, x, y);
                            put(ea[i], eb[i], e, IL, x * c[i][e] + y * sn[i][e], y * c[i][e] - x * sn[i][e]);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xa = row[k].a[i].at(e), xb = row[k].b[i].at(e);
                        sq = fmaf(xa, xa, sq);
                        sq = fmaf(xb, xb, sq);
                        dot = fmaf(ea[i][e] * w[0][i][e], xa, dot);
                        dot = fmaf(eb[i][e] * w[1][i][e], xb, dot);
                    }
                }
                const float rstd = rsqrtf(fmaf(group_sum(sq, G), p.inv_k, p.eps));
                // (a row that there is none of any more was this group's last but one: its sums stay out)
                const float scale = on ? rstd : 0.f;
                const float mean = group_sum(dot, G) * p.inv_k * rstd * rstd;   // of d u, times another s for u
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    float da[VEC], db[VEC];
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        const float xa = row[k].a[i].at(e), xb = row[k].b[i].at(e);
                        dw[0][i][e] = fmaf(ea[i][e], on ? xa * scale : 0.f, dw[0][i][e]);
                        dw[1][i][e] = fmaf(eb[i][e], on ? xb * scale : 0.f, dw[1][i][e]);
                        da[e] = rstd * fmaf(-xa, mean, ea[i][e] * w[0][i][e]);
                        db[e] = rstd * fmaf(-xb, mean, eb[i][e] * w[1][i][e]);
                    }
                    if (un.has(i) && on) {
                        store<VEC, XB>(s.y, yat + un.first(i), da);
                        store<VEC, XB>(s.y, yat + un.second(i), db);
                    }
                }
                xat += p.K;
                dat += p.K;
                yat += p.K;
            }
        }
    }
    if (!p.partial) return;
    // the groups of a warp first (their lanes hold the same channels), then the warps in turn
    for (int w0 = 0; w0 < kThreads / 32; ++w0) {
        if (threadIdx.x / 32 == w0) {
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int i = 0; i < UPL; ++i)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        float t = dw[half][i][e];
                        for (int off = 16; off >= G; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
                        if ((threadIdx.x & 31) < G && un.has(i)) {
                            float* to = &sums[(half ? un.second(i) : un.first(i)) + e];
                            *to = w0 ? *to + t : t;
                        }
                    }
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < p.K; i += kThreads) p.partial[(long long)blockIdx.x * p.K + i] = sums[i];
}

// dw[i] = the sum over the blocks' rows, of the queries' (blockIdx.y 0) or the keys' blocks: a block of 256 threads for 8
// columns, 32 partial sums each
__global__ void __launch_bounds__(kThreads) qk_sum_kernel(const float* partial, int blocks0, int blocks, int K, float* dwq, float* dwk) {
    __shared__ float part[32][9];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float* to = blockIdx.y ? dwk : dwq;
    if (!to) return;
    const int col = threadIdx.x % 8, row = threadIdx.x / 8, i = blockIdx.x * 8 + col;
    float t = 0.f;
    if (i < K)
        for (int b = (blockIdx.y ? blocks0 : 0) + row; b < (blockIdx.y ? blocks : blocks0); b += 32) t += __ldcg(partial + (long long)b * K + i);
    part[row][col] = t;
    __syncthreads();
    if (threadIdx.x < 8 && i < K) {
        float total = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) total += part[r][threadIdx.x];
        to[i] = total;
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

// The sizes, and how tokens' heads are dealt to groups and blocks: `resident` blocks in all, to queries and keys by their heads,
// that go round their work four times or more (so that the last round weighs little) where there is that much; a token's heads
// whole where its tokens alone give that, else in parts of four heads at least, down to single ones where lanes would
// have no work at all (each part forms the angles again).
int fill(QkParams& c, const gdn_qk_problem& p, int vec, int resident) {
    c.T = std::max(p.T, 1);
    c.K = p.K;
    c.R = p.R;
    c.interleaved = p.interleaved;
    c.eps = p.eps;
    c.inv_k = 1.f / p.K;
    c.G = 1;
    while (c.G < 32 && c.G < p.K / (2 * vec)) c.G *= 2;
    const long long tokens = (long long)p.B * p.T, rows = kThreads / c.G;
    int blocks[2];
    for (int i = 0; i < 2; ++i) {
        Side& s = c.side[i];
        s.H = i ? p.Hk : p.Hq;
        const long long share = std::max(1LL, (long long)resident * s.H / (p.Hq + p.Hk));   // blocks
        const long long round = share * rows, want = tokens > 0 ? (4 * round + tokens - 1) / tokens : 1;
        long long parts = std::min<long long>(want, (s.H + 3) / 4);
        if (tokens * parts < round) parts = std::min<long long>(s.H, (round + tokens - 1) / std::max(1LL, tokens));
        parts = std::max(1LL, parts);
        s.per = (int)((s.H + parts - 1) / parts);
        s.parts = (s.H + s.per - 1) / s.per;
        s.groups = tokens * s.parts;
        blocks[i] = (int)std::max(1LL, std::min(share, (s.groups + rows - 1) / rows));
    }
    c.blocks0 = blocks[0];
    return blocks[0] + blocks[1];
}

template <class F>
int resident_of(F kernel, std::atomic<int> (&known)[kDevices]) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    std::atomic<int>* k = dev < kDevices ? &known[dev] : nullptr;
    int n = k ? k->load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kThreads, 0) != cudaSuccess || n < 1) n = 1;
        if (k) k->store(n, std::memory_order_relaxed);
    }
    return n;
}

template <int VEC, int UPL, bool XB, bool YB, bool IL>
cudaError_t fwd(QkParams& c, const gdn_qk_problem& p, int sms, cudaStream_t s) {
    static std::atomic<int> known[kDevices];
    const auto kernel = qk_fwd_kernel<VEC, UPL, XB, YB, IL>;
    const int blocks = fill(c, p, VEC, resident_of(kernel, known) * sms);
    kernel<<<blocks, kThreads, 0, s>>>(c);
    return cudaGetLastError();
}
template <int VEC, int UPL, bool XB, bool YB, bool IL>
cudaError_t bwd(QkParams& c, const gdn_qk_problem& p, int sms, float* dwq, float* dwk, cudaStream_t s) {
    static std::atomic<int> known[kDevices];
    const auto kernel = qk_bwd_kernel<VEC, UPL, XB, YB, IL>;
    const int blocks = fill(c, p, VEC, std::min(resident_of(kernel, known) * sms, kMaxBlocks - 2));
    kernel<<<blocks, kThreads, 0, s>>>(c);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !c.partial) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((c.K + 7) / 8, 2);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_sum_kernel, (const float*)c.partial, c.blocks0, blocks, c.K, dwq, dwk);
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
    const int vec = widest(*p, {q, k}, {yq, yk}), sms = std::max(1, current_sm_count());
    QkParams c{};
    c.side[0].x = q, c.side[1].x = k;
    c.side[0].y = yq, c.side[1].y = yk;
    c.side[0].w = wq, c.side[1].w = wk;
    c.freq = freq;
    c.pos = positions;
    c.side[0].x_stride = p->q_stride, c.side[1].x_stride = p->k_stride;
    c.side[0].y_stride = (long long)p->Hq * p->K, c.side[1].y_stride = (long long)p->Hk * p->K;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(*p, [&](auto xb, auto yb) {
        return by_vec<xb.value, yb.value>(vec, [&](auto v, auto u) {
            return p->interleaved ? fwd<v.value, u.value, xb.value, yb.value, true>(c, *p, sms, s)
                                  : fwd<v.value, u.value, xb.value, yb.value, false>(c, *p, sms, s);
        });
    });
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_qk_norm_bwd_workspace_bytes(int K) {
    if (K < 2 || K > kMaxK || K % 2) return 0;
    return kWsHeader + ws_round(sizeof(float) * (size_t)K * kMaxBlocks);
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
    const int vec = widest(*p, {q, k, dq, dk}, {dyq, dyk}), sms = std::max(1, current_sm_count());
    QkParams c{};
    c.side[0].x = q, c.side[1].x = k;
    c.side[0].dy = dyq, c.side[1].dy = dyk;
    c.side[0].y = dq, c.side[1].y = dk;
    c.side[0].w = wq, c.side[1].w = wk;
    c.freq = freq;
    c.pos = positions;
    c.side[0].x_stride = c.side[0].y_stride = p->q_stride, c.side[1].x_stride = c.side[1].y_stride = p->k_stride;
    c.side[0].dy_stride = (long long)p->Hq * p->K, c.side[1].dy_stride = (long long)p->Hk * p->K;
    if (dwq || dwk) c.partial = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kWsHeader);
    gdn_qk_problem sizes = *p;
    if (!any) sizes.R = 0;   // (no tokens: the sums are zeros, and no frequency is read)
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(sizes, [&](auto xb, auto yb) {
        return by_vec<xb.value, yb.value>(vec, [&](auto v, auto u) {
            return p->interleaved ? bwd<v.value, u.value, xb.value, yb.value, true>(c, sizes, sms, dwq, dwk, s)
                                  : bwd<v.value, u.value, xb.value, yb.value, false>(c, sizes, sms, dwq, dwk, s);
        });
    });
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

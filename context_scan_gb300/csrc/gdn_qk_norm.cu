// gdn_qk_norm.cu -- the root-mean-square norm of every query and key head with the rotation by the token's position, in one pass
// (gdn_qk_norm_fwd), and its gradients (gdn_qk_norm_bwd).
//
// A head's K channels x of one token at position n, with s = 1 / sqrt(mean(x^2) + eps):
//   u = x s w,   (y_a, y_b) = (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = n freq_i
// for the R / 2 pairs (a, b) of rotated channels, y = u for the others. Backward, with e the gradient on y turned back
// by -t:   dw = sum over rows of e x s,   d = e w,   dx = s (d - x s mean(d x s)).
//
// Memory's work: x (and dy) read once, y (dx) written once. A row is a few hundred bytes, so a group of
// up to 32 lanes takes one token and walks over some of its heads: the angles' sines and cosines are formed once for them all
// and stay in registers. A lane holds both members of its pairs, so that the rotation crosses no lanes. A
// block works on the queries or on the keys (so that it holds one set of weights, in shared memory, and, backward, one of their
// sums), and a group reads its next head's row while it works on one (two rows ahead: 129 us instead of 126 and 98
// instead of 93). Measured: 32768 tokens of 32 + 8 heads of 128 in bf16 125 us, 5.4 TB/s of 6.8; gradients of 8192 tokens of 32 + 32
// heads, 64 channels rotated, 91 us, 4.4 TB/s. What bounds them: forward 78 % of memory's
// throughput, and its latency with 22 warps an SM (half of a warp's time between two instructions); backward 66 % and 69 % of
// the issue slots.
//
// Angles. n freq is wanted modulo a turn; in fp32 it would be off by n 2^-24. freq / 2 pi is turned into a
// 64-bit fraction of a turn, rounded once (integer products with the digits of 1 / 2 pi that count for freq's exponent, as in
// Payne and Hanek's argument reduction, once per pair and block); n times that, wrapping as integers do, is the angle modulo a
// turn to n 2^-65 of it, 2^-34 for the farthest position, whatever freq.
#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda_bf16.h>

#include "gdn_internal.h"
#include "gdn_pair.cuh"

namespace gdn {
namespace {

constexpr int kMaxK = 256;
constexpr int kThreads = 256;
constexpr int kDevices = 64;
// pairs a lane holds at most, backward: with 4, three blocks of 80 registers a thread an SM and 92 us for 524288 rows of
// 128 in bf16; with 8 two blocks and 110 us. (Forward 8: three blocks and 125 us for 1310720 rows; with 4 131.)
constexpr int kBwdVec = 4;
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

__device__ __forceinline__ float total(pair_t x) {
    float lo, hi;
    unpack(x, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ pair_t both(float x) { return pack(x, x); }

// A unit's values in fp32, by pairs of channels that turn together: x the first members, y the second ones, two
// channels to a register pair for the two-wide instructions (of a single channel the second place is 0). In an
// interleaved unit the 2 VEC values of the two loads lie in order, pair e being (2 e, 2 e + 1).
template <int VEC>
struct Members {
    static constexpr int N = (VEC + 1) / 2;
    pair_t x[N], y[N];
    template <bool IL, class A, class B>   // a(i), b(i): the i-th values of the two loads
    __device__ __forceinline__ void take(A a, B b) {
        float mx[2 * N], my[2 * N];
        mx[2 * N - 1] = my[2 * N - 1] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = 2 * e, j = 2 * e + 1;
            mx[e] = !IL || VEC == 1 ? a(e) : i < VEC ? a(i % VEC) : b(i % VEC);
            my[e] = !IL || VEC == 1 ? b(e) : j < VEC ? a(j % VEC) : b(j % VEC);
        }
#pragma unroll
        for (int n = 0; n < N; ++n) {
            x[n] = pack(mx[2 * n], mx[2 * n + 1]);
            y[n] = pack(my[2 * n], my[2 * n + 1]);
        }
    }
    template <bool IL>
    __device__ __forceinline__ void give(float (&a)[VEC], float (&b)[VEC]) const {
        float mx[2 * N], my[2 * N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            unpack(x[n], mx[2 * n], mx[2 * n + 1]);
            unpack(y[n], my[2 * n], my[2 * n + 1]);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int i = 2 * e, j = 2 * e + 1;
            (!IL || VEC == 1 ? a[e] : i < VEC ? a[i % VEC] : b[i % VEC]) = mx[e];
            (!IL || VEC == 1 ? b[e] : j < VEC ? a[j % VEC] : b[j % VEC]) = my[e];
        }
    }
    // turned by the angles of cosines c and sines s (BACK: the other way round)
    template <bool BACK>
    __device__ __forceinline__ void turn(const pair_t (&c)[N], const pair_t (&s)[N]) {
        const pair_t less = both(-1.f);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const pair_t u = x[n], v = y[n];
            if constexpr (BACK) {
                x[n] = fma2(v, s[n], mul2(u, c[n]));
                y[n] = fma2(mul2(u, s[n]), less, mul2(v, c[n]));
            } else {
                x[n] = fma2(mul2(v, s[n]), less, mul2(u, c[n]));
                y[n] = fma2(u, s[n], mul2(v, c[n]));
            }
        }
    }
    // in shared memory, 2 N pairs a unit
    __device__ __forceinline__ void put(pair_t* to) const {
#pragma unroll
        for (int n = 0; n < N; ++n) to[n] = x[n], to[N + n] = y[n];
    }
    __device__ __forceinline__ void get(const pair_t* from) {   // (volatile: not kept in registers over the rows)
        const unsigned at = (unsigned)__cvta_generic_to_shared(from);
        if constexpr (N % 2 == 0) {
#pragma unroll
            for (int n = 0; n < N; n += 2) {
                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(x[n]), "=l"(x[n + 1]) : "r"(at + 8 * n));
                asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(y[n]), "=l"(y[n + 1]) : "r"(at + 8 * (N + n)));
            }
        } else {
#pragma unroll
            for (int n = 0; n < N; ++n) {
                asm volatile("ld.shared.b64 %0, [%1];" : "=l"(x[n]) : "r"(at + 8 * n));
                asm volatile("ld.shared.b64 %0, [%1];" : "=l"(y[n]) : "r"(at + 8 * (N + n)));
            }
        }
    }
};
// A side's weights in shared memory, by units (in registers they would cost a block an SM).
template <int VEC>
struct Weights {
    static constexpr int N = Members<VEC>::N;
    pair_t w[kMaxK / (2 * VEC) * 2 * N];
};
template <int VEC, int UPL, bool IL>
__device__ __forceinline__ void make_weights(const Units<VEC, UPL>& un, const float* w, Weights<VEC>& to) {
#pragma unroll
    for (int i = 0; i < UPL; ++i)
        if ((int)threadIdx.x < un.G && un.has(i)) {
            Members<VEC> m;
            m.template take<IL>([&](int e) { return w ? __ldg(w + un.first(i) + e) : 1.f; },
                                [&](int e) { return w ? __ldg(w + un.second(i) + e) : 1.f; });
            m.put(to.w + 2 * Members<VEC>::N * un.unit(i));
        }
    __syncthreads();
}

// 64 binary digits of 1 / 2 pi from place p behind the point on (zeros before it), p from -149 to 169
__device__ __forceinline__ unsigned long long turn_digits(int p) {
    constexpr unsigned long long d[4] = {0x28be60db9391054a, 0x7f09d5f47d4d3770, 0x36d8a5664f10e410, 0x7f9458eaf7aef158};
    if (p < 0) return p <= -64 ? 0 : d[0] >> -p;
    const unsigned long long hi = p < 64 ? d[0] : p < 128 ? d[1] : d[2], lo = p < 64 ? d[1] : p < 128 ? d[2] : d[3];
    return p % 64 ? hi << p % 64 | lo >> (64 - p % 64) : hi;
}
// f / 2 pi modulo 1, times 2^64, rounded: f = +-m 2^e, m of 24 bits, times 128 digits of 1 / 2 pi from place e on (those before
// give whole turns)
__device__ __forceinline__ unsigned long long turn_of(float f) {
    const unsigned bits = __float_as_uint(f), field = bits >> 23 & 255u;
    const unsigned long long m = (bits & 0x7fffffu) | (field ? 0x800000u : 0u);
    const int e = (int)max(field, 1u) - 150;
    const unsigned long long hi = turn_digits(e), lo = turn_digits(e + 64);
    const unsigned long long turn = m * hi + __umul64hi(m, lo) + (m * lo >> 63);
    return bits >> 31 ? 0 - turn : turn;
}
// Every rotated pair's turn from one position to the next, as a 64-bit fraction, in shared memory (zeros for pairs
// that are not rotated).
__device__ __forceinline__ void make_steps(const QkParams& p, unsigned long long* step) {
    for (int i = threadIdx.x; i < kMaxK / 2; i += kThreads) step[i] = i < p.R / 2 ? turn_of(__ldg(p.freq + i)) : 0;
    __syncthreads();
}
// cosines and sines of a lane's pairs at position n
template <int VEC, int UPL>
struct Turns {
    static constexpr int N = (VEC + 1) / 2;
    pair_t c[UPL][N], s[UPL][N];
    __device__ __forceinline__ Turns(const Units<VEC, UPL>& un, const unsigned long long* step, int n) {
#pragma unroll
        for (int i = 0; i < UPL; ++i) {
            float co[2 * N], si[2 * N];
            co[2 * N - 1] = si[2 * N - 1] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const unsigned long long a = un.has(i) && un.turned(i) ? (unsigned long long)(long long)n * step[un.pair0(i) + e] : 0;
                sincospif((float)(int)(a >> 32) * 0x1p-31f, &si[e], &co[e]);
            }
#pragma unroll
            for (int k = 0; k < N; ++k) {
                c[i][k] = pack(co[2 * k], co[2 * k + 1]);
                s[i][k] = pack(si[2 * k], si[2 * k + 1]);
            }
        }
    }
};

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
__global__ void __launch_bounds__(kThreads, VEC == 8 ? 3 : VEC == 1 ? 2 : 4) qk_fwd_kernel(const __grid_constant__ QkParams p) {
    __shared__ unsigned long long step[kMaxK / 2];
    __shared__ __align__(16) Weights<VEC> weights;
    make_steps(p, step);
    const bool keys = (int)blockIdx.x >= p.blocks0;
    const Side& s = p.side[keys];
    const int block = keys ? blockIdx.x - p.blocks0 : blockIdx.x, blocks = keys ? gridDim.x - p.blocks0 : p.blocks0;
    const int G = p.G;
    const Units<VEC, UPL> un(p, threadIdx.x % G);
    const int rows = kThreads / G, mine = threadIdx.x / G;
    constexpr int N = Members<VEC>::N;
    make_weights<VEC, UPL, IL>(un, s.w, weights);
    // (a warp's groups take part in its exchanges whether or not they have work)
    for (long long g0 = (long long)block * rows; g0 < s.groups; g0 += (long long)blocks * rows) {
        const Work wk(s, g0 + mine);
        Row<VEC, UPL, XB> row[2];
        row[0].zero();
        row[1].zero();
        long long xat = wk.token * s.x_stride + (long long)wk.h0 * p.K, yat = wk.token * s.y_stride + (long long)wk.h0 * p.K;
        row[0].load(un, s.x, xat, wk.h0 < wk.h1);
        const Turns<VEC, UPL> t(un, step, p.pos ? (wk.h0 < wk.h1 ? __ldg(p.pos + wk.token) : 0) : (int)(wk.token % p.T));
        for (int h = wk.h0; __any_sync(0xffffffffu, h < wk.h1); h += 2) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                row[k ^ 1].load(un, s.x, xat + p.K, h + k + 1 < wk.h1);
                Members<VEC> m[UPL];
                pair_t sq = 0;
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    m[i].template take<IL>([&](int e) { return row[k].a[i].at(e); }, [&](int e) { return row[k].b[i].at(e); });
#pragma unroll
                    for (int n = 0; n < N; ++n) sq = fma2(m[i].y[n], m[i].y[n], fma2(m[i].x[n], m[i].x[n], sq));
                }
                const pair_t rstd = both(rsqrtf(fmaf(group_sum(total(sq), G), p.inv_k, p.eps)));
#pragma unroll
                for (int i = 0; i < UPL; ++i) {
                    Members<VEC> w;
                    w.get(weights.w + 2 * N * min(un.unit(i), un.n - 1));
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        m[i].x[n] = mul2(mul2(m[i].x[n], rstd), w.x[n]);
                        m[i].y[n] = mul2(mul2(m[i].y[n], rstd), w.y[n]);
                    }
                    if (un.turned(i)) m[i].template turn<false>(t.c[i], t.s[i]);
                    float a[VEC], b[VEC];
                    m[i].template give<IL>(a, b);
                    if (un.has(i) && h + k < wk.h1) {
                        store<VEC, YB>(s.y, yat + un.first(i), a);
                        store<VEC, YB>(s.y, yat + un.second(i), b);
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
template <int VEC, int UPL, bool XB, bool YB, bool IL>
__global__ void __launch_bounds__(kThreads, VEC == 1 ? 2 : 3) qk_bwd_kernel(const __grid_constant__ QkParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ unsigned long long step[kMaxK / 2];
    __shared__ __align__(16) Weights<VEC> weights;
    __shared__ float sums[kThreads / 32][kMaxK];
    make_steps(p, step);
    const bool keys = (int)blockIdx.x >= p.blocks0;
    const Side& s = p.side[keys];
    const int block = keys ? blockIdx.x - p.blocks0 : blockIdx.x, blocks = keys ? gridDim.x - p.blocks0 : p.blocks0;
    const int G = p.G;
    const Units<VEC, UPL> un(p, threadIdx.x % G);
    const int rows = kThreads / G, mine = threadIdx.x / G;
    constexpr int N = Members<VEC>::N;
    Members<VEC> dw[UPL];
    make_weights<VEC, UPL, IL>(un, s.w, weights);
#pragma unroll
    for (int i = 0; i < UPL; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) dw[i].x[n] = dw[i].y[n] = 0;
    for (long long g0 = (long long)block * rows; g0 < s.groups; g0 += (long long)blocks * rows) {
        const Work wk(s, g0 + mine);
        Row<VEC, UPL, XB> next_row;
        Row<VEC, UPL, YB> next_grad;
        next_row.zero();
        next_grad.zero();
        const long long first = (long long)wk.h0 * p.K;
        long long xat = wk.token * s.x_stride + first, dat = wk.token * s.dy_stride + first, yat = wk.token * s.y_stride + first;
        next_row.load(un, s.x, xat, wk.h0 < wk.h1);
        next_grad.load(un, s.dy, dat, wk.h0 < wk.h1);
        const Turns<VEC, UPL> t(un, step, p.pos ? (wk.h0 < wk.h1 ? __ldg(p.pos + wk.token) : 0) : (int)(wk.token % p.T));
#pragma unroll 1
        for (int h = wk.h0; __any_sync(0xffffffffu, h < wk.h1); ++h) {
            const Row<VEC, UPL, XB> row = next_row;
            const Row<VEC, UPL, YB> grad = next_grad;
            next_row.load(un, s.x, xat + p.K, h + 1 < wk.h1);
            next_grad.load(un, s.dy, dat + p.K, h + 1 < wk.h1);
            const bool on = h < wk.h1;
            Members<VEC> x[UPL], g[UPL];   // g: dy turned back
            pair_t sq = 0, dot = 0;
#pragma unroll
            for (int i = 0; i < UPL; ++i) {
                x[i].template take<IL>([&](int e) { return row.a[i].at(e); }, [&](int e) { return row.b[i].at(e); });
                g[i].template take<IL>([&](int e) { return grad.a[i].at(e); }, [&](int e) { return grad.b[i].at(e); });
                if (un.turned(i)) g[i].template turn<true>(t.c[i], t.s[i]);
                Members<VEC> w;
                w.get(weights.w + 2 * N * min(un.unit(i), un.n - 1));
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    sq = fma2(x[i].y[n], x[i].y[n], fma2(x[i].x[n], x[i].x[n], sq));
                    dot = fma2(mul2(g[i].x[n], w.x[n]), x[i].x[n], dot);
                    dot = fma2(mul2(g[i].y[n], w.y[n]), x[i].y[n], dot);
                }
            }
            const float s1 = rsqrtf(fmaf(group_sum(total(sq), G), p.inv_k, p.eps));
            const float m1 = group_sum(total(dot), G) * p.inv_k * s1 * s1 * s1;   // mean(d u), times s^2 for -u s
            // (behind the group's last row its values are still there: out of the sums by a factor of 0)
            const pair_t rstd = both(s1), kept = both(on ? s1 : 0.f), minus = both(-m1);
#pragma unroll
            for (int i = 0; i < UPL; ++i) {
                Members<VEC> w;
                w.get(weights.w + 2 * N * min(un.unit(i), un.n - 1));
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    dw[i].x[n] = fma2(g[i].x[n], mul2(x[i].x[n], kept), dw[i].x[n]);
                    dw[i].y[n] = fma2(g[i].y[n], mul2(x[i].y[n], kept), dw[i].y[n]);
                    x[i].x[n] = fma2(x[i].x[n], minus, mul2(rstd, mul2(g[i].x[n], w.x[n])));
                    x[i].y[n] = fma2(x[i].y[n], minus, mul2(rstd, mul2(g[i].y[n], w.y[n])));
                }
                float a[VEC], b[VEC];
                x[i].template give<IL>(a, b);
                if (un.has(i) && on) {
                    store<VEC, XB>(s.y, yat + un.first(i), a);
                    store<VEC, XB>(s.y, yat + un.second(i), b);
                }
            }
            xat += p.K;
            dat += p.K;
            yat += p.K;
        }
    }
    if (!p.partial) return;
    // the groups of a warp first (their lanes hold the same channels), then the warps, side by side in shared memory
    float* mine_ = sums[threadIdx.x / 32];
#pragma unroll
    for (int i = 0; i < UPL; ++i) {
        float v[2][VEC];
        dw[i].template give<IL>(v[0], v[1]);
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float t = v[half][e];
                for (int off = 16; off >= G; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
                if ((threadIdx.x & 31) < G && un.has(i)) mine_[(half ? un.second(i) : un.first(i)) + e] = t;
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < p.K; i += kThreads) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < kThreads / 32; ++k) t += sums[k][i];
        p.partial[(long long)blockIdx.x * p.K + i] = t;
    }
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
template <int MOST, bool XB, bool YB, class F>
cudaError_t by_vec(int vec, F f) {
    if constexpr (XB && YB && MOST == 8)
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
        return by_vec<8, xb.value, yb.value>(vec, [&](auto v, auto u) {
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
    const int vec = std::min(kBwdVec, widest(*p, {q, k, dq, dk}, {dyq, dyk})), sms = std::max(1, current_sm_count());
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
        return by_vec<kBwdVec, xb.value, yb.value>(vec, [&](auto v, auto u) {
            return p->interleaved ? bwd<v.value, u.value, xb.value, yb.value, true>(c, sizes, sms, dwq, dwk, s)
                                  : bwd<v.value, u.value, xb.value, yb.value, false>(c, sizes, sms, dwq, dwk, s);
        });
    });
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

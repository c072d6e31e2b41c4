// gdn_norm.cuh -- what the normalisation's two passes share: rows dealt to groups of threads, loads and
// stores of eight values in any of the storage types, sums over a group.
#pragma once

#include <cuda_bf16.h>

#include "gdn_internal.h"

namespace gdn {
namespace norm {

// A row of N values belongs to a group of G threads: a part of a warp (G <= 32, a power of two) or a whole
// block; every thread holds R times eight of its values (one up to N = 4096, two beyond, at G = 512). Where N % 8 == 0 the eight are consecutive and
// move as vectors (16-byte aligned rows); else they are G apart, so that a warp's single loads and
// stores still cover consecutive values.
struct Params {
    const void* x;
    const float* w;      // null: ones
    const float* b;      // null: zeros
    const void* z;       // null: no gate
    const void* dy;
    void* y;             // forward: y; backward: dx
    void* dz;            // null: not wanted
    float* partial;      // backward: [blocks][2][N] sums of dw and db
    long long rows;
    int N, g;            // g: threads of a row where it is less than a block
    int rms;
    float eps, inv_n;
};

template <bool BF, bool VEC>
struct Eight;

template <bool BF>
struct Eight<BF, true> {
    uint4 u[BF ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, long long row0, int c, int step, int n) {
        (void)step;
        if (c < n) {
            const uint4* p = reinterpret_cast<const uint4*>((const char*)base + (row0 + c) * (BF ? 2 : 4));
            u[0] = __ldcs(p);
            if constexpr (!BF) u[1] = __ldcs(p + 1);
        } else {
            u[0] = make_uint4(0, 0, 0, 0);
            if constexpr (!BF) u[1] = make_uint4(0, 0, 0, 0);
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        const unsigned a[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(a[i] << 16);
                f[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
            }
        } else {
            const unsigned d[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = __uint_as_float(a[i]);
                f[4 + i] = __uint_as_float(d[i]);
            }
        }
    }
    static __device__ __forceinline__ void store(void* base, long long row0, int c, int step, int n,
                                                 const float (&f)[8]) {
        (void)step;
        if (c >= n) return;
        uint4* p = reinterpret_cast<uint4*>((char*)base + (row0 + c) * (BF ? 2 : 4));
        if constexpr (BF) {
            unsigned a[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                a[i] = *reinterpret_cast<const unsigned*>(&h);
            }
            __stcs(p, make_uint4(a[0], a[1], a[2], a[3]));
        } else {
            __stcs(p, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                 __float_as_uint(f[3])));
            __stcs(p + 1, make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                                     __float_as_uint(f[7])));
        }
    }
};

template <bool BF>
struct Eight<BF, false> {
    float v[8];
    __device__ __forceinline__ void load(const void* base, long long row0, int c, int step, int n) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = c + e * step;
            v[e] = 0.f;
            if (at < n) {
                if constexpr (BF)
                    v[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[row0 + at]);
                else
                    v[e] = reinterpret_cast<const float*>(base)[row0 + at];
            }
        }
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[e];
    }
    static __device__ __forceinline__ void store(void* base, long long row0, int c, int step, int n,
                                                 const float (&f)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = c + e * step;
            if (at < n) {
                if constexpr (BF)
                    reinterpret_cast<__nv_bfloat16*>(base)[row0 + at] = __float2bfloat16_rn(f[e]);
                else
                    reinterpret_cast<float*>(base)[row0 + at] = f[e];
            }
        }
    }
};

// The first column of thread t's i-th eight values, and the distance between them.
template <bool VEC>
__device__ __forceinline__ int first_col(int i, int t, int G) {
    return VEC ? (i * G + t) * 8 : i * 8 * G + t;
}
template <bool VEC>
__device__ __forceinline__ int col_step(int G) {
    return VEC ? 1 : G;
}

// Sums of M values over the group, the same in each of its threads. Blocks: every call uses the other half of
// `part`, whose readers are behind the barrier of the call in between.
template <bool BLOCK, int M>
__device__ __forceinline__ void group_sum(float (&x)[M], int G, float (*part)[3][32], int& half) {
    const int first = BLOCK ? 16 : G / 2;
#pragma unroll
    for (int m = 0; m < M; ++m)
        for (int off = first; off > 0; off >>= 1) x[m] += __shfl_xor_sync(0xffffffffu, x[m], off);
    if constexpr (BLOCK) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
        for (int m = 0; m < M; ++m)
            if (lane == 0) part[half][m][warp] = x[m];
        __syncthreads();
#pragma unroll
        for (int m = 0; m < M; ++m) {
            x[m] = lane < warps ? part[half][m][lane] : 0.f;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) x[m] += __shfl_xor_sync(0xffffffffu, x[m], off);
        }
        half ^= 1;
    }
}

// (exp may overflow to infinity: the quotient is then 0)
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + expf(-z)); }

// How a call is laid out: threads of a row and of a block, eights of a thread, blocks at most.
struct Shape {
    bool block, vec;
    int g, threads, r;
};
inline Shape shape_of(int N) {
    Shape s{};
    s.vec = N % 8 == 0;
    const int eights = (N + 7) / 8;
    s.r = eights > 512 ? 2 : 1;
    int g = 8;
    while (g * s.r < eights) g *= 2;
    s.block = g > 32;
    s.g = g;
    s.threads = s.block ? g : 256;
    return s;
}
constexpr int kMaxN = 8192;
constexpr int kMaxThreads = 512;
constexpr int kSmBound = 256;           // SMs of any device that sizes a workspace
constexpr int kThreadsPerSm = 1024;     // of the backward's grid

// blocks of the backward on `sms` SMs
inline long long bwd_blocks(long long rows, const Shape& s, int sms) {
    const long long per = s.threads / s.g;
    const long long need = (rows + per - 1) / per;
    const long long most = (long long)sms * (kThreadsPerSm / s.threads);
    return need < most ? need : most;
}

cudaError_t launch_fwd(const Params& p, const Shape& s, bool xb, bool yb, int sms, cudaStream_t st);
// ... with dw and db (null: not wanted) summed over the rows; rows == 0 gives zeros
cudaError_t launch_bwd(const Params& p, const Shape& s, bool xb, bool yb, long long blocks, float* dw, float* db,
                       cudaStream_t st);

}  // namespace norm
}  // namespace gdn

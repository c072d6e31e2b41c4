// gdn_norm.cuh -- what the normalisation's two passes share: rows dealt to groups of threads, rows staged in
// shared memory ahead of their use, stores, sums over a group.
#pragma once

#include <algorithm>
#include <atomic>

#include <cuda_bf16.h>

#include "gdn_internal.h"
#include "gdn_pair.cuh"

namespace gdn {
namespace norm {

// A row of N values belongs to a group of G threads: a part of a warp (G <= 32, a power of two) or a whole
// block; every thread holds R times eight of its values: one up to N = 256, two beyond (what a row costs besides its
// values -- the exchange, the addresses -- is then shared by twice as many). How the eight lie, L:
//  8  side by side, 16 bytes of bf16 an access; N % 8 == 0, all types bf16
//  4  two fours, 4 G apart: 16 bytes of fp32 or 8 of bf16 an access, a warp's side by side (with eight side by
//     side fp32 leaves every other 16 bytes to the next access: 87 against 73 us for 29200 rows of 2000);
//     N % 4 == 0
//  2  four pairs, 2 G apart, for any N. With N odd every other row starts between two pairs' places; a group takes
//     rows of one kind only, and on the odd ones its pairs start one column earlier (the first one's first
//     value is none).
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

constexpr int kMaxN = 8192;
constexpr int kMaxThreads = 512;
constexpr int kSmBound = 256;           // SMs of any device that sizes a workspace

// The first column of thread t's i-th eight values (-1: none), and the column of its e-th value; odd: the row starts at
// an odd value.
template <int L>
__device__ __forceinline__ int first_col(int i, int t, int G, int odd) {
    return L * (i * (8 / L) * G + t) - (L == 2 ? odd : 0);
}
template <int L>
__device__ __forceinline__ int col_of(int c, int G, int e) { return c + (e / L) * L * G + e % L; }
__device__ __forceinline__ bool has(int col, int n) { return (unsigned)col < (unsigned)n; }

// Whether any lane of this thread's warp has columns among the i-th eights. (The forward leaves out those that
// have none: 45 -> 40 us for 29200 rows of 2000 in bf16; the backward, whose registers are full, took longer with
// such branches, 63 -> 78 us.)
template <int L>
__device__ __forceinline__ bool warp_has(int i, int t, int G, int n) {
    return i == 0 || first_col<L>(i, t & ~31, G, 0) < n + 1;
}

__device__ __forceinline__ pair_t both(float x) { return pack(x, x); }
__device__ __forceinline__ float total(pair_t x) {
    float lo, hi;
    unpack(x, lo, hi);
    return lo + hi;
}
__device__ __forceinline__ void single(const pair_t (&p)[4], float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack(p[i], f[2 * i], f[2 * i + 1]);
}
// a parameter's eight values of this thread's columns
template <int L>
__device__ __forceinline__ void parameter(pair_t (&f)[4], const float* from, int c, int G, int n, float none) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = both(none);
    if (!from) return;
    if constexpr (L == 8) {
        if (c >= n) return;
        const float4 a = __ldg(reinterpret_cast<const float4*>(from + c));
        const float4 b = __ldg(reinterpret_cast<const float4*>(from + c + 4));
        f[0] = pack(a.x, a.y);
        f[1] = pack(a.z, a.w);
        f[2] = pack(b.x, b.y);
        f[3] = pack(b.z, b.w);
    } else if constexpr (L == 4) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c0 = col_of<L>(c, G, 4 * k);
            if (c0 >= n) continue;
            const float4 a = __ldg(reinterpret_cast<const float4*>(from + c0));
            f[2 * k] = pack(a.x, a.y);
            f[2 * k + 1] = pack(a.z, a.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c0 = col_of<L>(c, G, 2 * i);
            f[i] = pack(has(c0, n) ? __ldg(from + c0) : none, has(c0 + 1, n) ? __ldg(from + c0 + 1) : none);
        }
    }
}

__device__ __forceinline__ unsigned bf16_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&h);
}

template <bool BF, int L>
__device__ __forceinline__ void store8(void* base, long long row0, int c, int G, int n, const float (&f)[8]) {
    if constexpr (L == 8) {
        static_assert(BF, "eight side by side are bf16");
        if (c < n)
            *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(base) + row0 + c) =
                make_uint4(bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3]), bf16_pair(f[4], f[5]), bf16_pair(f[6], f[7]));
    } else if constexpr (L == 4) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c0 = col_of<4>(c, G, 4 * k);
            if (c0 >= n) continue;
            if constexpr (BF)
                *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(base) + row0 + c0) =
                    make_uint2(bf16_pair(f[4 * k], f[4 * k + 1]), bf16_pair(f[4 * k + 2], f[4 * k + 3]));
            else
                *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + row0 + c0) =
                    make_float4(f[4 * k], f[4 * k + 1], f[4 * k + 2], f[4 * k + 3]);
        }
    } else {
        // (bf16 rows of more than 512: 53 -> 46 us for 29200 rows of 1999; the other ones lose by the branch)
        if (BF && G > 32 && c >= 0 && c + 6 * G + 1 < n) {   // all but the row's ends, without a look at each
#pragma unroll
            for (int k = 0; k < 4; ++k)
                *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(base) + row0 + c + 2 * k * G) =
                    __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            return;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c0 = c + 2 * k * G;
            const long long at = row0 + c0;   // even
            if constexpr (BF) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
                __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(base) + at;
                if (has(c0, n) && c0 + 1 < n)
                    *reinterpret_cast<__nv_bfloat162*>(to) = h;
                else if (has(c0, n))
                    to[0] = h.x;
                else if (has(c0 + 1, n))
                    to[1] = h.y;
            } else {
                float* to = reinterpret_cast<float*>(base) + at;
                if (has(c0, n) && c0 + 1 < n)
                    *reinterpret_cast<float2*>(to) = make_float2(f[2 * k], f[2 * k + 1]);
                else if (has(c0, n))
                    to[0] = f[2 * k];
                else if (has(c0 + 1, n))
                    to[1] = f[2 * k + 1];
            }
        }
    }
}

// The threads of a row meet: GB of the block's BLOCK threads, or (GB == 0) a part of a warp. (Numbered barriers only
// where a block has several groups: with numbers known at run time a block reserves 16 of the SM's 64.)
template <int GB, int BLOCK>
__device__ __forceinline__ void group_barrier() {
    if constexpr (GB == 0)
        __syncwarp();
    else if constexpr (GB == BLOCK)
        __syncthreads();
    else
        asm volatile("barrier.sync %0, %1;" ::"r"(1 + threadIdx.x / GB), "n"(GB) : "memory");
}

// Rows on their way: a ring of kDepth stages in shared memory, filled by asynchronous 16-byte copies kDepth - 1
// rows ahead, so that an SM has enough under way whatever the registers allow: about AHEAD pieces of 16 bytes a
// thread. L = 8 and 4: every thread copies and reads its own pieces, and needs no one else. L = 2: a row starts
// anywhere within 16 bytes, so the group copies the aligned pieces that cover it (the last one of the tensor cut short
// at its end) and reads pairs at the row's offset, after a barrier.
template <int L, int R, int AHEAD, bool... BF>
struct Ring {
    static constexpr bool kOwn = L != 2;   // a thread reads what it copied
    static constexpr bool kBf[] = {BF...};
    static constexpr int kTensors = sizeof...(BF);
    static constexpr int es(int t) { return kBf[t] ? 2 : 4; }
    static constexpr int pieces(int t) { return R * es(t) / 2; }   // of a thread
    static constexpr int first_piece(int t) { return t == 0 ? 0 : first_piece(t - 1) + pieces(t - 1); }
    static constexpr int kPieces = first_piece(kTensors - 1) + pieces(kTensors - 1);
    static constexpr int kAhead = AHEAD / kPieces < 1 ? 1 : AHEAD / kPieces > 6 ? 6 : AHEAD / kPieces;   // rows
    static constexpr int kDepth = kAhead + 1;
    static constexpr int kSlack = 2;   // L = 2: pieces more than the values take, a group and tensor
    static constexpr int bytes(int threads, int G) {
        return kOwn ? kDepth * kPieces * threads * 16
                   : kDepth * (kPieces * threads + kSlack * kTensors * (threads / G)) * 16;
    }

    unsigned base;   // shared memory
    int G, t, tid, threads, N, odd;
    long long rows;

    template <int T>
    __device__ __forceinline__ unsigned region(int stage) const {   // L = 2: of this group
        constexpr int kFirst = first_piece(T), kMine = pieces(T);
        const int groups = threads / G;
        return base + 16u * (stage * (kPieces * threads + kSlack * kTensors * groups) +
                             (kFirst * threads + kSlack * T * groups) + (tid / G) * (kMine * G + kSlack));
    }
    template <int T>
    __device__ __forceinline__ unsigned piece(int stage, int k) const {   // of this thread
        constexpr int kFirst = first_piece(T);
        return base + 16u * ((stage * kPieces + kFirst + k) * threads + tid);
    }
    template <int BYTES>
    static __device__ __forceinline__ void copy(unsigned to, const void* from, int n) {
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(n) : "memory");
    }
    template <int T>
    __device__ __forceinline__ void fetch(int stage, const void* from, long long row) const {
        constexpr int E = es(T);
        const char* src = reinterpret_cast<const char*>(from);
        if constexpr (kOwn) {
            constexpr int B = L * E < 16 ? L * E : 16;   // of a copy: 16, or 8 for four of bf16
            const int c = first_col<L>(0, t, G, 0);
            const char* at = src + (row * N + c) * E;
#pragma unroll
            for (int j = 0; j < R * 8 / L; ++j) {   // L columns each, L G apart
                const bool in = c + j * L * G < N && row < rows;
                static_assert(L * E <= 16, "one copy");
                copy<B>(piece<T>(stage, j * B / 16) + j * B % 16, in ? at + j * L * G * E : src, in ? B : 0);
            }
        } else if (row < rows) {
            const long long lo = row * N * E, a = lo & ~15LL;
            const int n = ((int)(lo - a) + N * E + 15) / 16;                          // pieces
            const int left = (int)min(rows * N * E - a, (long long)(1 << 20));        // bytes to the tensor's end
            const char* at = src + a + 16 * t;
            const unsigned to = region<T>(stage) + 16u * t;
#pragma unroll
            for (int j = 0; j <= pieces(T); ++j)
                if (t + j * G < n) copy<16>(to + 16u * j * G, at + 16 * j * G, min(16, left - 16 * (t + j * G)));
        }
    }
    static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // the oldest row's copies are complete (and, L = 2, everyone's; also, everyone has read the row before)
    template <int GB, int BLOCK>
    static __device__ __forceinline__ void wait() {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        if constexpr (!kOwn) group_barrier<GB, BLOCK>();
    }
    // this thread's i-th eight of a staged row
    template <int T>
    __device__ __forceinline__ void read(int stage, int i, long long row, float (&f)[8]) const {
        constexpr int E = es(T);
        if constexpr (kOwn) {
            unsigned u[E * 2];
#pragma unroll
            for (int k = 0; k < E / 2; ++k)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(u[4 * k]), "=r"(u[4 * k + 1]), "=r"(u[4 * k + 2]), "=r"(u[4 * k + 3])
                             : "r"(piece<T>(stage, i * (E / 2) + k)));
#pragma unroll
            for (int e = 0; e < 8; ++e)
                f[e] = E == 4 ? __uint_as_float(u[E == 4 ? e : 0])
                              : __uint_as_float(e & 1 ? u[e / 2] & 0xffff0000u : u[e / 2] << 16);
        } else {
            const int c = first_col<2>(i, t, G, odd), step = 2 * G, n = G > 32 || row < rows ? N : 0;   // (a block's rows are there)
            const unsigned at = region<T>(stage) + (unsigned)((row * N * E) & 15) + E * c;
            if constexpr (E == 2) {
                if (step > 64 && c >= 0 && c + 3 * step + 1 < n) {   // (as they are written)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        unsigned u;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(at + 2u * k * step));
                        f[2 * k] = __uint_as_float(u << 16);
                        f[2 * k + 1] = __uint_as_float(u & 0xffff0000u);
                    }
                    return;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {   // (an end pair's other value is another row's)
                const int c0 = c + k * step;
                float lo = 0.f, hi = 0.f;
                if (c0 < n) {
                    if constexpr (E == 2) {
                        unsigned u;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(at + 2u * k * step));
                        lo = __uint_as_float(u << 16);
                        hi = __uint_as_float(u & 0xffff0000u);
                    } else {
                        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(lo), "=f"(hi) : "r"(at + 4u * k * step));
                    }
                }
                f[2 * k] = has(c0, n) ? lo : 0.f;
                f[2 * k + 1] = c0 + 1 < n ? hi : 0.f;
            }
        }
    }
    template <int T>
    __device__ __forceinline__ void read(int stage, int i, long long row, pair_t (&p)[4]) const {
        float f[8];
        read<T>(stage, i, row, f);
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = pack(f[2 * k], f[2 * k + 1]);
    }
};

// Sums of M (1, 2 or 4) values over the group, the same in each of its threads. G threads (a
// multiple of 32), or (G == 0) g of a warp. Where there are several values the lanes first halve them among themselves, so that
// four values take not much more than one. Several warps: every call uses the other half of `part` (this
// group's), whose readers are behind the barrier of the call in between.
template <int G, int BLOCK, int M>
__device__ __forceinline__ void group_sum(float (&x)[M], int g, float (*part)[64], int& half) {
    const int lane = threadIdx.x & 31;
    int off = G ? 16 : g / 2;
#pragma unroll
    for (int n = M / 2; n >= 1; n /= 2, off /= 2) {
        const bool up = lane & off;
#pragma unroll
        for (int m = 0; m < n; ++m) {
            const float keep = up ? x[m + n] : x[m], send = up ? x[m] : x[m + n];
            x[m] = keep + __shfl_xor_sync(0xffffffffu, send, off);
        }
    }
    float one = x[0];
    if constexpr (G == 0) {
        for (; off > 0; off /= 2) one += __shfl_xor_sync(0xffffffffu, one, off);
        // value m is with the lanes whose upper bits say m
        const int base = lane & ~(g - 1);
#pragma unroll
        for (int m = 0; m < M; ++m) x[m] = M == 1 ? one : __shfl_sync(0xffffffffu, one, base + m * (g / M));
    } else {
        constexpr int WARPS = G / 32, ALL = M * WARPS;
#pragma unroll
        for (int o = 16 / M; o > 0; o /= 2) one += __shfl_xor_sync(0xffffffffu, one, o);
        if (lane % (32 / M) == 0) part[half][lane / (32 / M) * WARPS + (threadIdx.x >> 5) % WARPS] = one;
        group_barrier<G, BLOCK>();
        if constexpr (ALL <= 32) {
            one = part[half][lane % ALL];
#pragma unroll
            for (int o = WARPS / 2; o > 0; o /= 2) one += __shfl_xor_sync(0xffffffffu, one, o);
#pragma unroll
            for (int m = 0; m < M; ++m) x[m] = __shfl_sync(0xffffffffu, one, m * WARPS);
        } else {   // 16 warps, four values: two to a lane
            float two = part[half][lane + 32];
            one = part[half][lane];
#pragma unroll
            for (int o = WARPS / 2; o > 0; o /= 2) {
                one += __shfl_xor_sync(0xffffffffu, one, o);
                two += __shfl_xor_sync(0xffffffffu, two, o);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) x[m] = __shfl_sync(0xffffffffu, m < 2 ? one : two, (m & 1) * WARPS);
        }
        half ^= 1;
    }
}

// The layer norm's mean and variance come from one exchange, as sums of x and x^2. The variance is then a
// difference: while the mean is within two standard deviations of zero its rounding errors are up to five times a
// two-pass sum's (E[x^2] <= 5 var). fp32 rows of 2000, y against 64 bits, RMS (largest): as good as two passes at a mean of 0.2
// deviations, 1.1e-7 against 0.9e-7 at one, 2.3e-7 (3.3e-6) against 1.3e-7 (1.3e-6) at 1.9. A row with a larger mean goes
// round once more: that mean, which may be off by a few of its own last bits (the sum's, and 1 / N is rounded), is
// taken off the values, which leaves them exact where the mean is large, and the rest's mean and square give what it
// missed: 0.6e-7 at 5 and at 100 deviations, where two passes give 3.6e-7 and 62e-7. (Without the rest's mean rows of
// one value 100 came out as -0.005, N = 1000, eps = 1e-6.)
__device__ __forceinline__ bool large_mean(float mean, float var) { return mean * mean > 4.f * var; }
// mean taken off a thread's eight values (there is none in columns past the row)
template <int L>
__device__ __forceinline__ void centre(pair_t (&x)[4], int c, int G, int n, float mean) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int c0 = col_of<L>(c, G, 2 * k);
        const float lo = has(c0, n) ? -mean : 0.f, hi = L != 2 ? lo : has(c0 + 1, n) ? -mean : 0.f;
        x[k] = add2(x[k], pack(lo, hi));
    }
}
// from E[x^2] of values with a small mean (NaN stays)
__device__ __forceinline__ float centred_var(float square, float mean) {
    const float var = fmaf(-mean, mean, square);
    return var < 0.f ? 0.f : var;
}

// 1 / (1 + exp(-z)) from the hardware's approximations of 2^x and 1 / x (2 and 1 ulp, subnormals as zero): the
// roundings of z log2(e) and of that constant add 0.6 |z| ulp of the exponential, which shows for negative z: 60 times half an ulp
// of sigmoid(-80) = 2e-35, never more than half an ulp of 1. With expf, good to 2 ulp whatever z, gated rows take up to
// 10 % longer forward and 17 % backward (29200 rows of 1999 in bf16 75 -> 83 and 136 -> 156 us). 2^x may overflow to
// infinity: the quotient is then 0.
__device__ __forceinline__ float sigmoid(float z) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// How a call is laid out: threads of a row (8 to 512), eights of a thread.
struct Shape {
    int g, r;
};
inline Shape shape_of(int N) {
    Shape s{};
    const int eights = (N + 7) / 8;
    s.r = eights > 32 ? 2 : 1;
    s.g = 8;
    while (s.g * s.r < eights) s.g *= 2;
    return s;
}

// blocks (of kMaxThreads threads, one an SM) of the backward on `sms` >= 2 SMs
inline long long bwd_blocks(long long rows, const Shape& s, int sms) {
    const long long per = kMaxThreads / s.g, need = (rows + per - 1) / per;
    if (need <= sms) return need;
    return per == 1 ? sms & ~1 : sms;   // (an even number of rows at once: a group's rows start alike)
}

// Blocks of a kernel that are on an SM at once with `smem` bytes each, asked (and the shared memory allowed) once for
// each kernel and device, and again when smem changes: `known` holds the last answer and its smem in KiB. 0: an
// error.
constexpr int kDevices = 64;
constexpr int kMost = 200 * 1024;   // shared memory, above any call's
template <class Kernel>
int resident_blocks(Kernel* kernel, int threads, int smem, std::atomic<int> (&known)[kDevices]) {
    int dev = 0, per_sm = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    std::atomic<int>& last = known[dev % kDevices];
    const int kib = (smem + 1023) / 1024, have = last.load(std::memory_order_relaxed);
    if (have != 0 && have / 256 == kib) return have % 256;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, kib * 1024) != cudaSuccess)
        return 0;
    last.store(kib * 256 + per_sm, std::memory_order_relaxed);
    return per_sm;
}

cudaError_t launch_fwd(const Params& p, const Shape& s, bool xb, bool yb, int sms, cudaStream_t st);
// ... with dw and db (null: not wanted) summed over the rows; rows == 0 gives zeros
cudaError_t launch_bwd(const Params& p, const Shape& s, bool xb, bool yb, int sms, float* dw, float* db,
                       cudaStream_t st);

}  // namespace norm
}  // namespace gdn

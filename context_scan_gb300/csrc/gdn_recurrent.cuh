// gdn_recurrent.cuh -- what the recurrent forms over a state cache share (the gated delta rule in
// gdn_recurrent.cu, linear attention in gdn_linear_recurrent.cu): a warp's columns of a state in registers,
// the checks of lengths and slots, the order of the sequences. Internal linkage.
#pragma once

#include <climits>

#include <cuda_bf16.h>

#include "gdn_internal.h"
#include "gdn_pair.cuh"

namespace gdn {
namespace {

constexpr int kTokens = 8;   // tokens of a block
constexpr int kWarps = 4;    // of every thread block
// detail words of GDN_ERR_INVALID_ARG
constexpr unsigned kTagLengths = 0x41, kTagSlotRange = 0x42, kTagSlotShared = 0x43;
constexpr int kNobody = -1, kShared = -2;

struct RecurrentParams {
    const void* q;
    const void* k;
    const void* v;
    const void* g;
    const void* beta;
    void* o;
    float* state;
    const int* slots_in;
    const int* slots_out;
    const int* cu;
    const int* owner;      // per slot: the one sequence that writes it (claim_kernel), or null
    const int* cu_bad;     // claim_kernel's verdict on cu
    DeviceError* err;
    int nseq, T, H, Hqk, V, num_slots;
    int out_bf16, decay_first, per_token;
    int padded;            // the last entry of cu may lie before T: the tokens behind it are nobody's
    int ordered;           // the longest sequences first (ordered_sequence), by lengths in steps of
    int order_shift;       // 2^order_shift tokens
};

__device__ __forceinline__ float total(pair_t x) {
    float lo, hi;
    unpack(x, lo, hi);
    return lo + hi;
}

// eight consecutive values as stored
template <bool BF>
struct Raw8 {
    uint4 w[BF ? 1 : 2];
    __device__ __forceinline__ void load(const void* base, long long at) {
        const uint4* p = reinterpret_cast<const uint4*>(
            BF ? (const char*)base + 2 * at : (const char*)base + 4 * at);
        w[0] = __ldg(p);
        if constexpr (!BF) w[1] = __ldg(p + 1);
    }
    __device__ __forceinline__ void zero() {
        w[0] = make_uint4(0, 0, 0, 0);
        if constexpr (!BF) w[1] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void values(float (&f)[8]) const {
        const unsigned u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        if constexpr (BF) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            }
        } else {
            const unsigned t[4] = {w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[i] = __uint_as_float(u[i]);
                f[4 + i] = __uint_as_float(t[i]);
            }
        }
    }
};

// four consecutive values as stored
template <bool BF>
struct Raw4 {
    unsigned u[BF ? 2 : 4];
    __device__ __forceinline__ void load(const void* base, long long at) {
        if constexpr (BF) {
            const uint2 x = __ldg(reinterpret_cast<const uint2*>((const char*)base + 2 * at));
            u[0] = x.x, u[1] = x.y;
        } else {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>((const char*)base + 4 * at));
            u[0] = x.x, u[1] = x.y, u[2] = x.z, u[3] = x.w;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (unsigned& x : u) x = 0;
    }
    __device__ __forceinline__ void values(float (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = !BF ? __uint_as_float(u[BF ? 0 : i])
                       : __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
    }
    __device__ __forceinline__ void pairs(pair_t (&d)[2]) const {
        float f[4];
        values(f);
        d[0] = pack(f[0], f[1]);
        d[1] = pack(f[2], f[3]);
    }
};

template <bool BF>
__device__ __forceinline__ float load1(const void* base, long long at) {
    if constexpr (BF) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[at]);
    return reinterpret_cast<const float*>(base)[at];
}

__device__ __forceinline__ void put8(float* to, const float (&f)[8]) {
    *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void put4(float* to, const float (&f)[4]) {
    *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
}

__device__ __forceinline__ void report(DeviceError* e, unsigned detail) {
    if (atomicCAS(&e->code, 0u, (unsigned)GDN_ERR_INVALID_ARG) == 0u) atomicExch(&e->detail, detail);
}

// Tokens of sequence s; an entry that points outside the T tokens gives an empty sequence (the
// check of the whole array refuses the call before anything is written).
__device__ __forceinline__ void token_range(const RecurrentParams& p, int s, int& lo, int& n) {
    lo = s * p.T;   // (B * T < 2^31)
    n = p.T;
    if (p.cu) {
        lo = __ldg(p.cu + s);
        const int hi = __ldg(p.cu + s + 1);
        if (lo < 0 || hi < lo || hi > p.T)
            lo = n = 0;
        else
            n = hi - lo;
    }
}

__device__ __forceinline__ bool bad_ends(const RecurrentParams& p) {
    const int last = __ldg(p.cu + p.nseq);
    return __ldg(p.cu) != 0 || (p.padded ? last < 0 || last > p.T : last != p.T);
}

// Which sequence writes each slot, for batches whose pairs of sequences are too many to be
// compared by every block of the rule (see launch_recurrent): claims in the `owner` table, of which
// only the entries that the call names are touched. A slot that a sequence writes and another one
// reads or writes is kShared and is not written at all. One CTA.
constexpr int kClaimThreads = 1024;
__global__ void __launch_bounds__(kClaimThreads)
    claim_kernel(RecurrentParams p, int* owner, int* cu_bad, int nout) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int t = threadIdx.x;
    bool bad = false;
    if (p.cu) {
        for (int s = t; s < p.nseq; s += kClaimThreads) bad |= p.cu[s] < 0 || p.cu[s + 1] < p.cu[s];
        if (t == 0) bad |= bad_ends(p);
    }
    bad = __syncthreads_or(bad);
    if (t == 0) {
        *cu_bad = bad;
        if (bad) report(p.err, kTagLengths);
    }
    if (bad || !p.slots_out) return;
    if (p.padded && p.per_token && p.cu) nout = p.cu[p.nseq];
    auto named = [&](const int* slots, int i) {
        const int d = slots ? slots[i] : -1;
        return d >= 0 && d < p.num_slots ? d : -1;
    };
    for (int i = t; i < nout; i += kClaimThreads) {
        const int d = named(p.slots_out, i);
        if (d >= 0) owner[d] = kNobody;
    }
    for (int i = t; i < p.nseq; i += kClaimThreads) {
        const int d = named(p.slots_in, i);
        if (d >= 0) owner[d] = kNobody;
    }
    __syncthreads();
    for (int i = t; i < nout; i += kClaimThreads) {
        const int d = named(p.slots_out, i);
        if (d < 0) continue;
        int s = i;
        if (p.per_token) {
            if (p.cu) {   // the sequence of token i: the last one that starts at or before it
                int a = 0, b = p.nseq;
                while (b - a > 1) {
                    const int m = (a + b) / 2;
                    (p.cu[m] <= i ? a : b) = m;
                }
                s = a;
            } else {
                s = i / p.T;
            }
        }
        const int was = atomicCAS(owner + d, kNobody, s);
        if (was != kNobody && was != s) atomicExch(owner + d, kShared);
    }
    __syncthreads();
    for (int i = t; i < p.nseq; i += kClaimThreads) {
        const int d = named(p.slots_in, i);
        if (d < 0) continue;
        const int was = atomicAdd(owner + d, 0);
        if (was != kNobody && was != i) atomicExch(owner + d, kShared);
    }
}

// CW columns of one head's state in a warp: lane (rg, cl) holds CPL adjacent columns of every RG-th quad
// of rows, the rows in pairs for the two-wide fp32 instructions.
template <int K, int CW, int CPL>
struct Tile {
    static constexpr int CL = CW / CPL;        // lanes along the columns
    static constexpr int RG = 32 / CL;         // lanes along the rows
    static constexpr int NQ = K / 4 / RG;      // row quads of a lane
    static_assert(NQ >= 1 && RG >= 1 && (CPL == 1 || CPL == 2 || CPL == 4), "a tile's shape");
    pair_t S[NQ][2][CPL];
    int lane, cl, rg;

    __device__ __forceinline__ explicit Tile(int l) : lane(l), cl(l % CL), rg(l / CL) {}
    __device__ __forceinline__ int row(int i) const { return 4 * (i * RG + rg); }   // first of quad i
    __device__ __forceinline__ int col(int c) const { return CPL * cl + c; }        // this lane's c-th

    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < CPL; ++c) S[i][j][c] = 0;
    }
    // base: row 0, this warp's column 0
    __device__ __forceinline__ void load(const float* base, int V) {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float a[CPL], b[CPL];
                const float* at = base + (row(i) + 2 * j) * V + col(0);
                if constexpr (CPL == 4) {
                    const float4 x = __ldcs(reinterpret_cast<const float4*>(at));
                    const float4 y = __ldcs(reinterpret_cast<const float4*>(at + V));
                    a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
                    b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
                } else if constexpr (CPL == 2) {
                    const float2 x = __ldcs(reinterpret_cast<const float2*>(at));
                    const float2 y = __ldcs(reinterpret_cast<const float2*>(at + V));
                    a[0] = x.x, a[1] = x.y;
                    b[0] = y.x, b[1] = y.y;
                } else {
                    a[0] = __ldcs(at);
                    b[0] = __ldcs(at + V);
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) S[i][j][c] = pack(a[c], b[c]);
            }
    }
    __device__ __forceinline__ void store(float* base, int V) const {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float a[CPL], b[CPL];
#pragma unroll
                for (int c = 0; c < CPL; ++c) unpack(S[i][j][c], a[c], b[c]);
                float* at = base + (row(i) + 2 * j) * V + col(0);
                if constexpr (CPL == 4) {
                    __stcs(reinterpret_cast<float4*>(at), make_float4(a[0], a[1], a[2], a[3]));
                    __stcs(reinterpret_cast<float4*>(at + V), make_float4(b[0], b[1], b[2], b[3]));
                } else if constexpr (CPL == 2) {
                    __stcs(reinterpret_cast<float2*>(at), make_float2(a[0], a[1]));
                    __stcs(reinterpret_cast<float2*>(at + V), make_float2(b[0], b[1]));
                } else {
                    __stcs(at, a[0]);
                    __stcs(at + V, b[0]);
                }
            }
    }
    // Sums over the lanes that hold the same columns: lane l ends with the whole sum of its column own().
    __device__ __forceinline__ float join(const pair_t (&acc)[CPL]) const {
        float d[CPL];
#pragma unroll
        for (int c = 0; c < CPL; ++c) d[c] = total(acc[c]);
        int off = 16;
#pragma unroll
        for (int n = CPL / 2; n >= 1; n /= 2) {   // each half of the lanes takes half of the columns
            const bool up = lane & off;
#pragma unroll
            for (int c = 0; c < n; ++c) {
                const float keep = up ? d[c + n] : d[c], send = up ? d[c] : d[c + n];
                d[c] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
            off /= 2;
        }
        return rows_sum(d[0], off);
    }
    // (the lanes that hold the same own() column, from distance off on)
    __device__ __forceinline__ float rows_sum(float x, int off) const {
#pragma unroll
        for (; off >= CL; off /= 2) x += __shfl_xor_sync(0xffffffffu, x, off);
        return x;
    }
    __device__ __forceinline__ int own() const {
        int c = 0, off = 16;
#pragma unroll
        for (int n = CPL / 2; n >= 1; n /= 2, off /= 2) c += lane & off ? n : 0;
        return c;
    }
    // one lane for each column
    __device__ __forceinline__ bool first() const { return (lane & (32 / CPL - 1) & ~(CL - 1)) == 0; }
    // The other way: from each lane's value of its own() column to the values of all its columns, twice over.
    __device__ __forceinline__ void spread(float mine, pair_t (&r)[CPL]) const {
        float d[CPL];
        d[0] = mine;
        int off = 32 / CPL;
#pragma unroll
        for (int n = 1; n < CPL; n *= 2, off *= 2) {
            const bool up = lane & off;
#pragma unroll
            for (int c = 0; c < n; ++c) {
                const float other = __shfl_xor_sync(0xffffffffu, d[c], off);
                d[c + n] = up ? d[c] : other;
                d[c] = up ? other : d[c];
            }
        }
#pragma unroll
        for (int c = 0; c < CPL; ++c) r[c] = pack(d[c], d[c]);
    }
};

struct Place {   // of a warp: sequence, head, first column, and where its states start
    int s, h, col0, hk;
    long long page, off;
    __device__ __forceinline__ Place(const RecurrentParams& p, int K, int CW, int warp) {
        const int COLS = CW * kWarps, tiles = p.V / COLS;
        const int hs = blockIdx.x / tiles;
        s = hs / p.H;
        h = hs - s * p.H;
        col0 = (blockIdx.x - hs * tiles) * COLS + warp * CW;
        hk = h / (p.H / p.Hqk);
        page = (long long)p.H * K * p.V;
        off = (long long)h * K * p.V + col0;
    }
};

__device__ __forceinline__ void store_o(const RecurrentParams& p, long long at, float o) {
    if (p.out_bf16)
        reinterpret_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(o);
    else
        reinterpret_cast<float*>(p.o)[at] = o;
}

// Whether another sequence names the slot that sequence s writes (every lane looks at some; the answer is the
// warp's). Only where no claims were made.
__device__ __forceinline__ bool named_by_others(const RecurrentParams& p, int s, int slot, int lane) {
    bool shared = false;
    for (int j = lane; j < p.nseq; j += 32)
        shared |= j != s && (__ldg(p.slots_out + j) == slot || (p.slots_in && __ldg(p.slots_in + j) == slot));
    return __any_sync(0xffffffffu, shared);
}

// What the checks say before anything is written: false when the call or the sequence is refused; `write`:
// whether the final state may go to slot_out.
__device__ __forceinline__ bool admitted(const RecurrentParams& p, const Place& at, int slot_in, int slot_out,
                                         int lane, bool& write) {
    const bool tell = lane == 0 && at.col0 == 0;   // one warp a head
    write = slot_out >= 0 && slot_out < p.num_slots;
    if (p.owner) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (__ldcg(p.cu_bad)) return false;
        if (write && __ldcg(p.owner + slot_out) != at.s) {
            write = false;
            if (tell) report(p.err, kTagSlotShared);
        }
    } else {
        if (p.cu) {
            bool bad = lane == 0 && bad_ends(p);
            for (int j = lane; j < p.nseq; j += 32) bad |= __ldg(p.cu + j + 1) < __ldg(p.cu + j);
            if (__any_sync(0xffffffffu, bad)) {
                if (tell) report(p.err, kTagLengths);
                return false;
            }
        }
        if (write && p.nseq > 1 && named_by_others(p, at.s, slot_out, lane)) {
            write = false;
            if (tell) report(p.err, kTagSlotShared);
        }
    }
    if (tell && (slot_in >= p.num_slots || slot_out >= p.num_slots)) report(p.err, kTagSlotRange);
    return slot_in < p.num_slots;
}

// Which sequence the thread blocks with number `mine` among the sequences take: the mine-th in the order of falling
// length (in steps of 2^shift tokens; equal ones by number), so that the long ones start first and the
// short ones fill the gaps at the end. Every block sorts for itself, by counting.
constexpr int kBuckets = 128;
__device__ __forceinline__ int ordered_sequence(const RecurrentParams& p, int mine) {
    __shared__ __align__(16) int count[kBuckets];
    __shared__ int found;
    const int t = threadIdx.x, lane = t & 31;
    auto bucket = [&](int i) {   // the longest in bucket 0
        const int l = (int)((unsigned)__ldg(p.cu + i + 1) - (unsigned)__ldg(p.cu + i)) >> p.order_shift;
        return kBuckets - 1 - min(max(l, 0), kBuckets - 1);
    };
    count[t] = 0;
    __syncthreads();
    for (int i = t; i < p.nseq; i += 32 * kWarps) atomicAdd(&count[bucket(i)], 1);
    __syncthreads();
    if (t < 32) {
        // the bucket that holds number `mine`, and which of it that is
        const int4 c = *reinterpret_cast<const int4*>(&count[4 * lane]);
        const int sum = c.x + c.y + c.z + c.w;
        int before = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, before, off);
            if (lane >= off) before += y;
        }
        before -= sum;
        const int at = 31 - __clz(__ballot_sync(0xffffffffu, before <= mine));   // the last lane that starts at or before
        int left = mine - before, b = 4 * lane;
        const int n[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (b == 4 * lane + j && left >= n[j]) {
                left -= n[j];
                ++b;
            }
        b = __shfl_sync(0xffffffffu, b, at);
        left = __shfl_sync(0xffffffffu, left, at);
        // the left-th of the bucket's sequences
        for (int i0 = 0; i0 < p.nseq; i0 += 32) {
            const unsigned in = __ballot_sync(0xffffffffu, i0 + lane < p.nseq && bucket(min(i0 + lane, p.nseq - 1)) == b);
            if (left < __popc(in)) {
                const bool me = (in >> lane & 1u) && __popc(in & ((1u << lane) - 1u)) == left;
                if (me) found = i0 + lane;
                break;
            }
            left -= __popc(in);
        }
    }
    __syncthreads();
    return found;
}
static_assert(kBuckets == 32 * kWarps, "a thread for each bucket");

// Each block of the rule looks for other sequences that name its slot when there are at most this many
// sequences; above it, and where states are kept after every token, claim_kernel does so once.
constexpr int kInlineSeqs = 512;
constexpr int kOrderSeqs = 1024;
constexpr int kMostTokens = INT_MAX - 4096;   // of all sequences: token numbers and the steps beyond the last one in an int

gdn_status check(const gdn_problem* p, int Hqk, int nseq, const int* cu, int num_slots, int per_token) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B < 1 || p->H < 1 || p->T < 0 || nseq < 1 || Hqk < 1 || num_slots < 0) return GDN_ERR_INVALID_ARG;
    if (cu ? p->B != 1 : p->B != nseq) return GDN_ERR_INVALID_ARG;
    if (p->decay_first != 0 && p->decay_first != 1) return GDN_ERR_INVALID_ARG;
    if (p->gate_k != 0 && p->gate_k != 1) return GDN_ERR_INVALID_ARG;
    if (per_token != 0 && per_token != 1) return GDN_ERR_INVALID_ARG;
    if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (p->H % Hqk != 0) return GDN_ERR_UNSUPPORTED_SHAPE;
    if ((p->in_dtype != GDN_DTYPE_F32 && p->in_dtype != GDN_DTYPE_BF16) ||
        (p->out_dtype != GDN_DTYPE_F32 && p->out_dtype != GDN_DTYPE_BF16))
        return GDN_ERR_UNSUPPORTED_DTYPE;
    // (the grid at its finest split in 31 bits)
    if ((long long)p->B * p->T > kMostTokens || (long long)nseq * p->H * 4 >= (1LL << 31))
        return GDN_ERR_UNSUPPORTED_SHAPE;
    return GDN_OK;
}

// What precedes the rule's kernel: the steps of the order, and the claims where they are wanted.
gdn_status claim(RecurrentParams& c, const gdn_problem& p, int average, char* ws, cudaStream_t s) {
    for (; (4LL * average) >> c.order_shift >= kBuckets; ++c.order_shift) {
    }
    if (c.nseq > kInlineSeqs || (c.per_token && c.nseq > 1)) {
        int* owner = reinterpret_cast<int*>(ws + kWsHeader);
        int* cu_bad = reinterpret_cast<int*>(ws + kWsVerdict);
        const long long nout = c.per_token ? (long long)p.B * p.T : c.nseq;
        claim_kernel<<<1, kClaimThreads, 0, s>>>(c, owner, cu_bad, (int)nout);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
        c.owner = owner;
        c.cu_bad = cu_bad;
    }
    return GDN_OK;
}

}  // namespace
}  // namespace gdn

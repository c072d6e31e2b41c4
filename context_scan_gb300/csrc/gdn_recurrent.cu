// gdn_recurrent.cu -- the recurrent gated delta rule over a state cache (gdn_recurrent_fwd):
// every sequence's tokens in order from the state in one cache page, fp32 throughout.
//
// Per sequence, head and token ("RFC: HyperParallel Linear Attention Context Parallel", section
// 2.1; the decayed read as in "Context Parallelism in ART", section 08), with E = exp(g) or, per
// key channel, diag(exp(g)), and H_read = H or E H:
//   r = beta (v - k^T H_read),   H' = E H + k r^T,   o = q^T H' = (E q)^T H + (q . k) r.
//
// The last form lets both products read the state before the update, so a token takes one pass
// of sums, one exchange between lanes and one pass of updates.
//
// Every column of the state is independent given k, q and the gates. A warp owns CW columns of one
// head, all K rows of them in registers (Tile below), so the state is read from memory once, when the
// sequence starts, and written once, when it ends (or after every token when the caller keeps
// them all). Three kernels, whose measurements stand beside the rule that picks one (launch_k):
//  - decode_kernel, one token a sequence: bound by the memory traffic of the states. A warp needs
//    nothing of another one, so it waits for nothing but its own loads; four blocks of 128 registers a
//    thread keep 128 KB of states on their way per SM. 256 sequences, H = 32, K = V = 128:
//    172 us, 6.3 TB/s (93 % of a copy); tokens_kernel took 214 us there.
//  - tokens_kernel, token by token: for a few tokens a sequence, where the traffic is still the bound (48 sequences of 1 to
//    8 tokens, every state kept: 94 us, 6.0 TB/s).
//  - pairs_kernel, two tokens at a time: for many tokens, bound by the fp32 pipe, which the two-wide
//    multiply-adds hold for two cycles each, and by the passes' other instructions (37 sequences of up to 63
//    tokens, H = 16, per-channel gates: 66 us, the pipe busy for 31 of them; 71 token by token, 95 without the
//    order of ordered_sequence), and for few warps, bound by a token's chain of dependent instructions (5
//    sequences of 130 tokens: 22.7 us, 28.5 token by token). Blocks of eight tokens (all products with the state
//    first, then a triangular solve in each lane) and the next token's sums formed beside the update both took longer:
//    what they save in waiting they spend in instructions.
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
        if (t == 0) bad |= p.cu[0] != 0 || p.cu[p.nseq] != p.T;
    }
    bad = __syncthreads_or(bad);
    if (t == 0) {
        *cu_bad = bad;
        if (bad) report(p.err, kTagLengths);
    }
    if (bad || !p.slots_out) return;
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
            bool bad = lane == 0 && (__ldg(p.cu) != 0 || __ldg(p.cu + p.nseq) != p.T);
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

// One token a sequence (p.T == 1, no cu_seqlens, states at the end).
template <int K, int CW, int CPL, bool GATEK, bool BF>
__global__ void __launch_bounds__(32 * kWarps, CW == 16 ? 4 : 1) decode_kernel(RecurrentParams p) {
    using Cols = Tile<K, CW, CPL>;
    constexpr int NQ = Cols::NQ;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place at(p, K, CW, warp);
    Cols tile(lane);

    const int slot_in = p.slots_in ? __ldg(p.slots_in + at.s) : -1;
    const int slot_out = p.slots_out ? __ldg(p.slots_out + at.s) : -1;
    // the token's values that this lane needs, of its rows and of its own column
    Raw4<BF> rk[NQ], rq[NQ], rg[NQ];
    const long long kq = ((long long)at.s * p.Hqk + at.hk) * K, sh = (long long)at.s * p.H + at.h;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        rk[i].load(p.k, kq + tile.row(i));
        rq[i].load(p.q, kq + tile.row(i));
        if constexpr (GATEK) rg[i].load(p.g, sh * K + tile.row(i));
    }
    const long long oat = sh * p.V + at.col0 + tile.col(tile.own());
    const float v = load1<BF>(p.v, oat), beta = load1<BF>(p.beta, sh);
    const float g = GATEK ? 0.f : load1<BF>(p.g, sh);
    if (slot_in >= 0 && slot_in < p.num_slots)
        tile.load(p.state + slot_in * at.page + at.off, p.V);
    else
        tile.zero();
    bool write;
    if (!admitted(p, at, slot_in, slot_out, lane, write)) return;

    const float e = expf(g);
    pair_t k2[NQ][2], e2[NQ][2], ak[CPL] = {}, aq[CPL] = {}, qk2 = 0;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        pair_t q2[2];
        rk[i].pairs(k2[i]);
        rq[i].pairs(q2);
        if constexpr (GATEK) {
            pair_t g2[2];
            rg[i].pairs(g2);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float x, y;
                unpack(g2[j], x, y);
                e2[i][j] = pack(expf(x), expf(y));
            }
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            qk2 = fma2(q2[j], k2[i][j], qk2);
            pair_t kr = k2[i][j], qr = q2[j];
            if constexpr (GATEK) {
                if (p.decay_first) kr = mul2(kr, e2[i][j]);
                qr = mul2(qr, e2[i][j]);
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                ak[c] = fma2(tile.S[i][j][c], kr, ak[c]);
                aq[c] = fma2(tile.S[i][j][c], qr, aq[c]);
            }
        }
    }
    const float qk = tile.rows_sum(total(qk2), 16);
    const float sk = tile.join(ak), sq = tile.join(aq);
    const float r = beta * (v - (!GATEK && p.decay_first ? e * sk : sk));
    if (tile.first()) store_o(p, oat, fmaf(qk, r, e * sq));
    if (!write) return;
    pair_t r2[CPL];
    tile.spread(r, r2);
#pragma unroll
    for (int i = 0; i < NQ; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < CPL; ++c)
                tile.S[i][j][c] = fma2(k2[i][j], r2[c], mul2(tile.S[i][j][c], GATEK ? e2[i][j] : pack(e, e)));
    tile.store(p.state + slot_out * at.page + at.off, p.V);
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

// Token by token: kTokens of them staged in shared memory at a time while the next ones load.
template <int K, int CW, int CPL, bool GATEK, bool BF>
__global__ void __launch_bounds__(32 * kWarps, CW == 16 ? 4 : 1) tokens_kernel(RecurrentParams p) {
    using Cols = Tile<K, CW, CPL>;
    constexpr int NQ = Cols::NQ, C = kTokens;
    constexpr int KV8 = K / 8;            // threads that stage one token's k and q, eight channels each
    constexpr int COLS = CW * kWarps;
    static_assert(C * KV8 <= 32 * kWarps && C * COLS / 8 <= 32 * kWarps, "one piece a thread");

    __shared__ __align__(16) float ks[2][C][K], qs[2][C][K];               // qs: E q for gates per channel
    __shared__ __align__(16) float es[2][GATEK ? C : 1][GATEK ? K : 4];    // exp(g), per channel
    __shared__ __align__(16) float kr[2][GATEK ? C : 1][GATEK ? K : 4];    // k as the read sees it
    __shared__ __align__(16) float vs[2][C][COLS];
    __shared__ float4 sc[2][C];   // exp(g), beta, q . k

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Place at(p, K, CW, warp);
    if (p.ordered) at.s = ordered_sequence(p, at.s);
    Cols tile(lane);

    const int slot_in = p.slots_in ? __ldg(p.slots_in + at.s) : -1;
    int lo, n;
    token_range(p, at.s, lo, n);
    const int slot_out = p.slots_out && !p.per_token ? __ldg(p.slots_out + at.s) : -1;
    if (slot_in >= 0 && slot_in < p.num_slots)
        tile.load(p.state + slot_in * at.page + at.off, p.V);
    else
        tile.zero();

    // staging: thread tid brings eight key channels of token st's k, q (and gates) and eight columns of
    // token vt's v
    const int st = tid / KV8, sk = 8 * (tid % KV8);
    const int vt = tid / (COLS / 8), vc = 8 * (tid % (COLS / 8));
    Raw8<BF> rk, rq, rv, rg;
    float raw_g = 0.f, raw_b = 0.f;
    auto load_tokens = [&](int t0) {
        if (st < C && t0 + st < n) {
            const long long tok = lo + t0 + st;
            const long long a = (tok * p.Hqk + at.hk) * K + sk;
            rk.load(p.k, a);
            rq.load(p.q, a);
            if constexpr (GATEK) rg.load(p.g, (tok * p.H + at.h) * K + sk);
        }
        if (vt < C && t0 + vt < n)
            rv.load(p.v, ((long long)(lo + t0 + vt) * p.H + at.h) * p.V + (at.col0 - warp * CW) + vc);
        if (tid < C && t0 + tid < n) {
            const long long a = (long long)(lo + t0 + tid) * p.H + at.h;
            raw_b = load1<BF>(p.beta, a);
            if constexpr (!GATEK) raw_g = load1<BF>(p.g, a);
        }
    };
    auto store_tokens = [&](int b) {
        float fk[8], fq[8];
        rk.values(fk);
        rq.values(fq);
        float qk = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) qk = fmaf(fq[i], fk[i], qk);
#pragma unroll
        for (int off = KV8 / 2; off > 0; off >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, off);
        if (st < C) {
            put8(&ks[b][st][sk], fk);
            if constexpr (GATEK) {
                float e[8];
                rg.values(e);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    e[i] = expf(e[i]);
                    fq[i] *= e[i];
                    if (p.decay_first) fk[i] *= e[i];
                }
                put8(&es[b][st][sk], e);
                put8(&kr[b][st][sk], fk);
            }
            put8(&qs[b][st][sk], fq);
            if (sk == 0) sc[b][st].z = qk;
        }
        if (vt < C) {
            float f[8];
            rv.values(f);
            put8(&vs[b][vt][vc], f);
        }
        if (tid < C) {
            sc[b][tid].x = expf(raw_g);
            sc[b][tid].y = raw_b;
        }
    };
    rk.zero();
    rq.zero();
    rv.zero();
    rg.zero();
    if (n > 0) load_tokens(0);

    bool write;
    // (every warp of the block comes to the same verdict on the call and the sequence)
    if (!admitted(p, at, slot_in, slot_out, lane, write)) return;

    const int oc = tile.col(tile.own());   // this lane's column once sums are joined
    const bool first = tile.first();
    const long long ostep = (long long)p.H * p.V;
    long long oat = ((long long)lo * p.H + at.h) * p.V + at.col0 + oc;
    for (int t0 = 0, b = 0; t0 < n; t0 += C, b ^= 1) {
        // (buffer b was last read before the barrier of the block in between)
        store_tokens(b);
        __syncthreads();
        if (t0 + C < n) load_tokens(t0 + C);
        const int m = min(C, n - t0);
#pragma unroll 1
        for (int t = 0; t < m; ++t) {
            const float4 g4 = sc[b][t];   // exp(g), beta, q . k
            const float vt_ = vs[b][t][warp * CW + oc];
            pair_t ak[CPL] = {}, aq[CPL] = {};
            const float* kread = GATEK ? kr[b][t] : ks[b][t];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(kread + tile.row(i));
                const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(&qs[b][t][tile.row(i)]);
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    ak[c] = fma2(tile.S[i][0][c], k2.x, ak[c]);
                    aq[c] = fma2(tile.S[i][0][c], q2.x, aq[c]);
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    ak[c] = fma2(tile.S[i][1][c], k2.y, ak[c]);
                    aq[c] = fma2(tile.S[i][1][c], q2.y, aq[c]);
                }
            }
            const float sk_ = tile.join(ak), sq_ = tile.join(aq);
            const float e = GATEK ? 1.f : g4.x;
            const float r = g4.y * (vt_ - (!GATEK && p.decay_first ? e * sk_ : sk_));
            if (first) store_o(p, oat, fmaf(g4.z, r, e * sq_));
            oat += ostep;
            pair_t r2[CPL];
            tile.spread(r, r2);
            const pair_t e2 = pack(e, e);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&ks[b][t][tile.row(i)]);
                pair_t ex = e2, ey = e2;
                if constexpr (GATEK) {
                    const ulonglong2 ek = *reinterpret_cast<const ulonglong2*>(&es[b][t][tile.row(i)]);
                    ex = ek.x;
                    ey = ek.y;
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    tile.S[i][0][c] = fma2(k2.x, r2[c], mul2(tile.S[i][0][c], ex));
                    tile.S[i][1][c] = fma2(k2.y, r2[c], mul2(tile.S[i][1][c], ey));
                }
            }
            if (p.per_token && p.slots_out) {
                const int slot = __ldg(p.slots_out + lo + t0 + t);
                if (slot >= p.num_slots) {
                    if (lane == 0) report(p.err, kTagSlotRange);
                } else if (slot >= 0) {
                    if (!p.owner || __ldcg(p.owner + slot) == at.s)
                        tile.store(p.state + slot * at.page + at.off, p.V);
                    else if (lane == 0)
                        report(p.err, kTagSlotShared);
                }
            }
        }
    }
    if (write) tile.store(p.state + slot_out * at.page + at.off, p.V);
}

// Any number of tokens a sequence, by twos: with S0 the state before tokens 1 and 2, c21 = k2read . k1 and so on,
//   r1 = beta1 (v1 - k1read^T S0),        o1 = (E1 q1)^T S0 + (q1 . k1) r1,
//   r2 = beta2 (v2 - (E1 k2read)^T S0 - (k2read . k1) r1),
//   o2 = (E1 E2 q2)^T S0 + (E2 q2 . k1) r1 + (q2 . k2) r2,
//   S2 = E1 E2 S0 + (E2 k1) r1^T + k2 r2^T
// (kread = k, or E k for the decayed read): seven multiply-adds a state value where two single tokens take eight,
// and half as many waits for a sum across lanes. kTokens tokens are staged in shared memory at a time while the next
// ones load; a token that the last pair lacks is staged as zeros.
template <int K, int CW, int CPL, bool GATEK, bool BF>
__global__ void __launch_bounds__(32 * kWarps, CW == 16 ? 3 : 1) pairs_kernel(RecurrentParams p) {
    using Cols = Tile<K, CW, CPL>;
    constexpr int NQ = Cols::NQ, C = kTokens, P = C / 2;
    constexpr int KV4 = K / 4;            // threads that stage one pair's k and q, four channels each
    constexpr int COLS = CW * kWarps;
    static_assert(P * KV4 <= 32 * kWarps && C * COLS / 8 <= 32 * kWarps, "one piece a thread");

    // as the update (per channel: E2 k1, k2), the outputs (E1 q1, E1 E2 q2) and the reads (k1read, E1 k2read) take them
    __shared__ __align__(16) float ks[2][C][K], qs[2][C][K];
    __shared__ __align__(16) float kr[2][GATEK ? C : 1][GATEK ? K : 4];
    __shared__ __align__(16) float es[2][GATEK ? P : 1][GATEK ? K : 4];    // E1 E2
    __shared__ __align__(16) float vs[2][C][COLS];
    __shared__ float2 gb[2][C];           // exp(g) (scalar gates), beta
    __shared__ __align__(16) float dots[2][P][4];   // q1 . k1, q2 . k2, k2read . k1, E2 q2 . k1 (scalar gates: without the gates)

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Place at(p, K, CW, warp);
    if (p.ordered) at.s = ordered_sequence(p, at.s);
    Cols tile(lane);

    const int slot_in = p.slots_in ? __ldg(p.slots_in + at.s) : -1;
    int lo, n;
    token_range(p, at.s, lo, n);
    const int slot_out = p.slots_out ? __ldg(p.slots_out + at.s) : -1;
    if (slot_in >= 0 && slot_in < p.num_slots)
        tile.load(p.state + slot_in * at.page + at.off, p.V);
    else
        tile.zero();

    // staging: thread tid brings four key channels of pair sp's k, q (and gates) and eight columns of
    // token vt's v
    const int sp = tid / KV4, sk = 4 * (tid % KV4);
    const int vt = tid / (COLS / 8), vc = 8 * (tid % (COLS / 8));
    Raw4<BF> rk[2], rq[2], rg[2];
    Raw8<BF> rv;
    float raw_g, raw_b;
    auto load_tokens = [&](int t0) {
        rv.zero();
        raw_g = raw_b = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            rk[j].zero();
            rq[j].zero();
            rg[j].zero();
            const int t = t0 + 2 * sp + j;
            if (sp < P && t < n) {
                const long long tok = lo + t;
                const long long a = (tok * p.Hqk + at.hk) * K + sk;
                rk[j].load(p.k, a);
                rq[j].load(p.q, a);
                if constexpr (GATEK) rg[j].load(p.g, (tok * p.H + at.h) * K + sk);
            }
        }
        if (vt < C && t0 + vt < n)
            rv.load(p.v, ((long long)(lo + t0 + vt) * p.H + at.h) * p.V + (at.col0 - warp * CW) + vc);
        if (tid < C && t0 + tid < n) {
            const long long a = (long long)(lo + t0 + tid) * p.H + at.h;
            raw_b = load1<BF>(p.beta, a);
            if constexpr (!GATEK) raw_g = load1<BF>(p.g, a);
        }
    };
    auto store_tokens = [&](int b) {
        float k1[4], k2[4], q1[4], q2[4];
        rk[0].values(k1);
        rk[1].values(k2);
        rq[0].values(q1);
        rq[1].values(q2);
        float d[4] = {};   // q1 . k1, q2 . k2, k2read . k1, E2 q2 . k1
        float x1[4], x2[4], e1[4], e2[4];   // k1read, k2read
        if constexpr (GATEK) {
            rg[0].values(e1);
            rg[1].values(e2);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[0] = fmaf(q1[i], k1[i], d[0]);
            d[1] = fmaf(q2[i], k2[i], d[1]);
            x1[i] = k1[i];
            x2[i] = k2[i];
            if constexpr (GATEK) {
                e1[i] = expf(e1[i]);
                e2[i] = expf(e2[i]);
                q1[i] *= e1[i];
                q2[i] *= e2[i];
                if (p.decay_first) {
                    x1[i] *= e1[i];
                    x2[i] *= e2[i];
                }
            }
            d[2] = fmaf(x2[i], k1[i], d[2]);
            d[3] = fmaf(q2[i], k1[i], d[3]);
            if constexpr (GATEK) {
                q2[i] *= e1[i];
                x2[i] *= e1[i];
                k1[i] *= e2[i];
                e1[i] *= e2[i];
            }
        }
        // the four sums over the pair's lanes, which first halve them among themselves
        int off = KV4 / 2;
#pragma unroll
        for (int h = 2; h >= 1; h /= 2, off /= 2) {
            const bool up = lane & off;
#pragma unroll
            for (int i = 0; i < h; ++i) {
                const float keep = up ? d[i + h] : d[i], send = up ? d[i] : d[i + h];
                d[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
        }
#pragma unroll
        for (; off > 0; off /= 2) d[0] += __shfl_xor_sync(0xffffffffu, d[0], off);
        if (sp < P) {
            put4(&ks[b][2 * sp][sk], k1);
            put4(&ks[b][2 * sp + 1][sk], k2);
            put4(&qs[b][2 * sp][sk], q1);
            put4(&qs[b][2 * sp + 1][sk], q2);
            if constexpr (GATEK) {
                put4(&kr[b][2 * sp][sk], x1);
                put4(&kr[b][2 * sp + 1][sk], x2);
                put4(&es[b][sp][sk], e1);
            }
            if (sk % KV4 == 0) dots[b][sp][sk / KV4] = d[0];   // (lanes 0, KV4 / 4, KV4 / 2, 3 KV4 / 4 of the pair)
        }
        if (vt < C) {
            float f[8];
            rv.values(f);
            put8(&vs[b][vt][vc], f);
        }
        if (tid < C) gb[b][tid] = make_float2(GATEK ? 1.f : expf(raw_g), raw_b);
    };
    load_tokens(0);

    bool write;
    // (every warp of the block comes to the same verdict on the call and the sequence)
    if (!admitted(p, at, slot_in, slot_out, lane, write)) return;

    const int oc = tile.col(tile.own());   // this lane's column once sums are joined
    const bool first = tile.first();
    const long long ostep = (long long)p.H * p.V;
    long long oat = ((long long)lo * p.H + at.h) * p.V + at.col0 + oc;
    for (int t0 = 0, b = 0; t0 < n; t0 += C, b ^= 1) {
        // (buffer b was last read before the barrier of the block in between)
        store_tokens(b);
        __syncthreads();
        if (t0 + C < n) load_tokens(t0 + C);
        const int m = min(C, n - t0);
#pragma unroll 1
        for (int t = 0; t < m; t += 2) {
            pair_t a1[CPL], a2[CPL], q1[CPL], q2[CPL];
            const float* r1_ = GATEK ? kr[b][t] : ks[b][t];
            const float* r2_ = GATEK ? kr[b][t + 1] : ks[b][t + 1];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 x1 = *reinterpret_cast<const ulonglong2*>(r1_ + tile.row(i));
                const ulonglong2 y1 = *reinterpret_cast<const ulonglong2*>(&qs[b][t][tile.row(i)]);
                const ulonglong2 x2 = *reinterpret_cast<const ulonglong2*>(r2_ + tile.row(i));
                const ulonglong2 y2 = *reinterpret_cast<const ulonglong2*>(&qs[b][t + 1][tile.row(i)]);
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    a1[c] = i ? fma2(tile.S[i][0][c], x1.x, a1[c]) : mul2(tile.S[i][0][c], x1.x);
                    a2[c] = i ? fma2(tile.S[i][0][c], x2.x, a2[c]) : mul2(tile.S[i][0][c], x2.x);
                    q1[c] = i ? fma2(tile.S[i][0][c], y1.x, q1[c]) : mul2(tile.S[i][0][c], y1.x);
                    q2[c] = i ? fma2(tile.S[i][0][c], y2.x, q2[c]) : mul2(tile.S[i][0][c], y2.x);
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    a1[c] = fma2(tile.S[i][1][c], x1.y, a1[c]);
                    a2[c] = fma2(tile.S[i][1][c], x2.y, a2[c]);
                    q1[c] = fma2(tile.S[i][1][c], y1.y, q1[c]);
                    q2[c] = fma2(tile.S[i][1][c], y2.y, q2[c]);
                }
            }
            // (k is read again for the update: kept in registers until then it would push the state out of them)
            if constexpr (CPL == 4) asm volatile("" ::: "memory");
            const float2 g1 = gb[b][t], g2 = gb[b][t + 1];   // exp(g), beta
            const float4 d = *reinterpret_cast<const float4*>(dots[b][t / 2]);
            const float v1 = vs[b][t][warp * CW + oc], v2 = vs[b][t + 1][warp * CW + oc];
            float s1 = tile.join(a1), s2 = tile.join(a2), o1 = tile.join(q1), o2 = tile.join(q2);
            float kk = d.z, q21 = d.w;
            if constexpr (!GATEK) {
                const float e12 = g1.x * g2.x;
                o1 *= g1.x;
                o2 *= e12;
                s1 *= p.decay_first ? g1.x : 1.f;
                s2 *= p.decay_first ? e12 : g1.x;
                kk *= p.decay_first ? g2.x : 1.f;
                q21 *= g2.x;
            }
            const bool both = t + 1 < m;
            const float r1 = g1.y * (v1 - s1);
            const float r2 = both ? g2.y * (v2 - fmaf(kk, r1, s2)) : 0.f;
            if (first) {
                store_o(p, oat, fmaf(d.x, r1, o1));
                if (both) store_o(p, oat + ostep, fmaf(d.y, r2, fmaf(q21, r1, o2)));
            }
            oat += 2 * ostep;
            pair_t u1[CPL], u2[CPL];
            tile.spread(GATEK ? r1 : g2.x * r1, u1);
            tile.spread(r2, u2);
            const float e12 = g1.x * g2.x;
            const pair_t e2 = pack(e12, e12);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 k1 = *reinterpret_cast<const ulonglong2*>(&ks[b][t][tile.row(i)]);
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&ks[b][t + 1][tile.row(i)]);
                pair_t ex = e2, ey = e2;
                if constexpr (GATEK) {
                    const ulonglong2 ek = *reinterpret_cast<const ulonglong2*>(&es[b][t / 2][tile.row(i)]);
                    ex = ek.x;
                    ey = ek.y;
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    tile.S[i][0][c] = fma2(k2.x, u2[c], fma2(k1.x, u1[c], mul2(tile.S[i][0][c], ex)));
                    tile.S[i][1][c] = fma2(k2.y, u2[c], fma2(k1.y, u1[c], mul2(tile.S[i][1][c], ey)));
                }
            }
        }
    }
    if (write) tile.store(p.state + slot_out * at.page + at.off, p.V);
}

enum class Kernel { kDecode, kTokens, kPairs };
template <Kernel WHICH, int K, int CW, int CPL, bool GATEK, bool BF>
constexpr auto kernel_of() {
    if constexpr (WHICH == Kernel::kDecode)
        return decode_kernel<K, CW, CPL, GATEK, BF>;
    else if constexpr (WHICH == Kernel::kTokens)
        return tokens_kernel<K, CW, CPL, GATEK, BF>;
    else
        return pairs_kernel<K, CW, CPL, GATEK, BF>;
}
template <Kernel WHICH, int K, int CW, int CPL>
cudaError_t launch(const RecurrentParams& p, bool gate_k, bool bf16, cudaStream_t s) {
    const auto fn = gate_k ? (bf16 ? kernel_of<WHICH, K, CW, CPL, true, true>() : kernel_of<WHICH, K, CW, CPL, true, false>())
                           : (bf16 ? kernel_of<WHICH, K, CW, CPL, false, true>() : kernel_of<WHICH, K, CW, CPL, false, false>());
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.nseq * p.H * (p.V / (CW * kWarps))));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.owner ? 1 : 0;   // the dependent of claim_kernel
    RecurrentParams copy = p;
    void* args[] = {&copy};
    return cudaLaunchKernelExC(&cfg, (const void*)fn, args);
}

// The split. One token a sequence: decode_kernel, 16 columns a warp always (half a warp's 64 B of a row; at 8 columns
// the same time up to four sequences of 32 heads, more beyond: 49.7 against 59.9 us at 64 of them).
// More tokens, enough columns to fill the SMs with twelve warps of 16 each:
//  - few tokens a sequence on average: bound by the states' traffic. tokens_kernel, 16 columns a warp, four blocks an SM:
//    240 us for 256 sequences of up to two tokens, 32 heads, against 250 by pairs;
//  - many: pairs_kernel, and 32 columns a warp where K = V = 128, two blocks an SM, whose exchanges and addresses serve
//    twice the columns: 310 us for 64 sequences of 40 to 63 tokens, 32 heads, per-channel gates, against 344 by
//    single tokens and 344 by pairs at 16 columns.
// Fewer columns: pairs_kernel with 8, 4 or 2 of them a warp, one a lane. A token's time is then a warp's chain of
// instructions, which is shorter with fewer rows a lane although the sums cross more lanes. 8, 4 and 2 columns (by
// single tokens), K = V = 128, 63 tokens, cold: 29.2, 27.1 and 25.1 us for one sequence of 8 heads, 27.1, 25.1
// and 25.1 for two, 33.3, 33.3 and 41.5 for eight (of up to 63), 45.6, 47.6 and 64.0 for eight of 16 heads; 39.4, 37.3
// and 31.2 us for five of 130 tokens, 2 heads, K = V = 64, where pairs take 25.1.
// A state after every token: single tokens.
constexpr int kWideWarpsPerSm = 12, kManyTokens = 12;
constexpr int kQuarterWarpsPerSm = 8, kEighthWarpsPerSm = 4;   // of 4 and 2 columns, at most
template <int K>
cudaError_t launch_k(const RecurrentParams& p, int average, bool gate_k, bool bf16, int sms, cudaStream_t s) {
    if (p.T == 1 && !p.cu) return launch<Kernel::kDecode, K, 16, 4>(p, gate_k, bf16, s);
    const long long warps = (long long)p.nseq * p.H * (p.V / 16);
    if (warps >= (long long)kWideWarpsPerSm * sms) {
        if (p.per_token || average < kManyTokens) return launch<Kernel::kTokens, K, 16, 4>(p, gate_k, bf16, s);
        if constexpr (K == 128)
            if (p.V == 128) return launch<Kernel::kPairs, K, 32, 4>(p, gate_k, bf16, s);
        return launch<Kernel::kPairs, K, 16, 4>(p, gate_k, bf16, s);
    }
    if (p.per_token) return launch<Kernel::kTokens, K, 8, 1>(p, gate_k, bf16, s);
    if (8 * warps <= (long long)kEighthWarpsPerSm * sms) return launch<Kernel::kPairs, K, 2, 1>(p, gate_k, bf16, s);
    if (4 * warps <= (long long)kQuarterWarpsPerSm * sms) return launch<Kernel::kPairs, K, 4, 1>(p, gate_k, bf16, s);
    return launch<Kernel::kPairs, K, 8, 1>(p, gate_k, bf16, s);
}

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

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

size_t gdn_recurrent_workspace_bytes(int num_slots) {
    if (num_slots < 0) return 0;
    return kWsHeader + ws_round(sizeof(int) * (size_t)num_slots);
}

gdn_status gdn_recurrent_fwd(const gdn_problem* p, int Hqk, int nseq, const int* cu_seqlens,
                             const void* q, const void* k, const void* v, const void* g,
                             const void* beta, float* state, int num_slots, const int* slots_in,
                             const int* slots_out, int per_token, void* o, void* workspace,
                             size_t workspace_bytes, void* stream) {
    gdn_status st = check(p, Hqk, nseq, cu_seqlens, num_slots, per_token);
    if (st != GDN_OK) return st;
    if (p->T > 0 && (!q || !k || !v || !g || !beta || !o)) return GDN_ERR_INVALID_ARG;
    if ((slots_in || slots_out) && !state && num_slots > 0) return GDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdn_recurrent_workspace_bytes(num_slots)) return GDN_ERR_WORKSPACE;
    for (const void* ptr : {q, k, v, g, beta, (const void*)state, (const void*)o, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(ptr) & 15u) return GDN_ERR_MISALIGNED;
    for (const int* ptr : {cu_seqlens, slots_in, slots_out})
        if (reinterpret_cast<uintptr_t>(ptr) & 3u) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(workspace);
    RecurrentParams c{};
    c.q = q;
    c.k = k;
    c.v = v;
    c.g = g;
    c.beta = beta;
    c.o = o;
    c.state = state;
    c.slots_in = slots_in;
    c.slots_out = slots_out;
    c.cu = cu_seqlens;
    c.err = reinterpret_cast<DeviceError*>(ws);
    c.nseq = nseq;
    c.T = p->T;
    c.H = p->H;
    c.Hqk = Hqk;
    c.V = p->V;
    c.num_slots = num_slots;
    c.out_bf16 = p->out_dtype == GDN_DTYPE_BF16;
    c.decay_first = p->decay_first;
    if (!slots_out || (p->T == 1 && !cu_seqlens)) per_token = 0;   // no states to keep, or the final ones
    c.per_token = per_token;
    // The longest sequences first, where there is something to gain: several tokens a sequence on average, and more
    // blocks than the SMs hold at once. 37 sequences of up to 63 tokens, H = 16: 95 us without, 72 with;
    // a few tokens each leave less to gain than the sorting costs.
    const int average = cu_seqlens ? p->T / nseq : p->T;
    c.ordered = cu_seqlens && nseq > 1 && nseq <= kOrderSeqs && average >= kManyTokens &&
                (long long)nseq * p->H * (p->V / 64) > 4LL * current_sm_count();
    for (; (4LL * average) >> c.order_shift >= kBuckets; ++c.order_shift) {
    }
    if (nseq > kInlineSeqs || (per_token && nseq > 1)) {
        int* owner = reinterpret_cast<int*>(ws + kWsHeader);
        int* cu_bad = reinterpret_cast<int*>(ws + kWsVerdict);
        const long long nout = per_token ? (long long)p->B * p->T : nseq;
        claim_kernel<<<1, kClaimThreads, 0, s>>>(c, owner, cu_bad, (int)nout);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
        c.owner = owner;
        c.cu_bad = cu_bad;
    }
    const bool bf16 = p->in_dtype == GDN_DTYPE_BF16;
    const int sms = current_sm_count();
    if ((p->K == 64 ? launch_k<64>(c, average, p->gate_k, bf16, sms, s)
                    : launch_k<128>(c, average, p->gate_k, bf16, sms, s)) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

}  // extern "C"

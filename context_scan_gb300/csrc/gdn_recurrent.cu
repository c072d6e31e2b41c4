// gdn_recurrent.cu -- the recurrent gated delta rule over a state cache (gdn_recurrent_fwd):
// every sequence's tokens one after another from the state in one cache page, fp32 throughout.
//
// Per sequence, head and token ("RFC: HyperParallel Linear Attention Context Parallel", section
// 2.1; the decayed read as in "Context Parallelism in ART", section 08), with E = exp(g) or, per
// key channel, diag(exp(g)), and H_read = H or E H:
//   r = beta (v - k^T H_read),   H' = E H + k r^T,   o = q^T H' = (E q)^T H + (q . k) r.
// The last form lets both products read the state before the update, so a token takes one pass
// of sums, one exchange between lanes and one pass of updates.
//
// Split: every column of the state is independent given k, q and the gates. A warp owns CW
// columns of one head, all K rows of them in registers (each lane four columns of every
// 128 / CW -th quad of rows, the rows in pairs for the two-wide fp32 instructions), so the state is
// read from memory once, when the sequence starts, and written once, when it ends (or after every
// token when the caller keeps them all). The tokens' k, q, v and gates are staged in shared memory
// eight at a time, the next eight loading while these are worked on.
#include <cuda_bf16.h>

#include "gdn_internal.h"

namespace gdn {
namespace {

constexpr int kTokens = 8;   // tokens staged at once
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
};

using pair_t = unsigned long long;   // two fp32 values of one column, rows 2 i and 2 i + 1

__device__ __forceinline__ pair_t pack(float lo, float hi) {
    pair_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack(pair_t x, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ pair_t fma2(pair_t a, pair_t b, pair_t c) {
    pair_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ pair_t mul2(pair_t a, pair_t b) {
    pair_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
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

template <bool BF>
__device__ __forceinline__ float load1(const void* base, long long at) {
    if constexpr (BF) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[at]);
    return reinterpret_cast<const float*>(base)[at];
}

__device__ __forceinline__ void put8(float* to, const float (&f)[8]) {
    *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
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

template <int K, int CW, int WARPS, bool GATEK, bool BF>
__global__ void __launch_bounds__(32 * WARPS) recurrent_kernel(RecurrentParams p) {
    constexpr int THREADS = 32 * WARPS;
    constexpr int CL = CW / 4;            // lanes along the columns, four columns each
    constexpr int RG = 32 / CL;           // lanes along the rows
    constexpr int NQ = K / 4 / RG;        // row quads of a lane: quads i * RG + rg
    constexpr int COLS = CW * WARPS;      // columns of the CTA
    constexpr int KV8 = K / 8;            // threads that stage one token's k and q
    constexpr int TB = THREADS / KV8 < kTokens ? THREADS / KV8 : kTokens;
    constexpr int NV = (TB * COLS / 8 + THREADS - 1) / THREADS;
    static_assert(NQ >= 1 && NV == 1, "one vector of v a thread");

    __shared__ __align__(16) float ks[2][TB][K], qs[2][TB][K];
    __shared__ __align__(16) float es[2][GATEK ? TB : 1][GATEK ? K : 4];   // exp(g), per channel
    __shared__ __align__(16) float kr[2][GATEK ? TB : 1][GATEK ? K : 4];   // k as the read sees it
    __shared__ __align__(16) float vs[2][TB][COLS];
    __shared__ float4 sc[2][TB];   // exp(g), beta, q . k

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cl = lane % CL, rg = lane / CL;
    const int tiles = p.V / COLS;
    const int tile = blockIdx.x % tiles;
    const int h = (blockIdx.x / tiles) % p.H;
    const int s = blockIdx.x / (tiles * p.H);
    const int c0 = tile * COLS + warp * CW + 4 * cl;   // this lane's columns c0 .. c0 + 3
    const int hk = h / (p.H / p.Hqk);

    const int slot_in = p.slots_in ? __ldg(p.slots_in + s) : -1;
    int lo, n;
    token_range(p, s, lo, n);
    const int slot_out = p.slots_out && !p.per_token ? __ldg(p.slots_out + s) : -1;

    // the state, on its way while the tokens and the checks are looked at
    pair_t S[NQ][2][4];
    const long long page = (long long)p.H * K * p.V;
    const long long lane_off = (long long)h * K * p.V + c0;
    const bool in_ok = slot_in < p.num_slots;
    if (slot_in >= 0 && in_ok) {
        const float* src = p.state + slot_in * page + lane_off;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float* row = src + (long long)(4 * (i * RG + rg) + 2 * j) * p.V;
                const float4 a = __ldcg(reinterpret_cast<const float4*>(row));
                const float4 b = __ldcg(reinterpret_cast<const float4*>(row + p.V));
                S[i][j][0] = pack(a.x, b.x);
                S[i][j][1] = pack(a.y, b.y);
                S[i][j][2] = pack(a.z, b.z);
                S[i][j][3] = pack(a.w, b.w);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) S[i][j][c] = 0;
    }

    // staging: thread tid holds eight key channels of token tid / KV8's k and q, and eight
    // columns of token tid / (COLS / 8)'s v
    const int st = tid / KV8, sk = 8 * (tid % KV8);
    const int vt = tid / (COLS / 8), vc = 8 * (tid % (COLS / 8));
    Raw8<BF> rk, rq, rv, rgk;
    float raw_g = 0.f, raw_b = 0.f;
    auto load_tokens = [&](int t0) {
        rk.zero();
        rq.zero();
        if (st < TB && t0 + st < n) {
            const long long tok = lo + t0 + st;
            const long long at = (tok * p.Hqk + hk) * K + sk;
            rk.load(p.k, at);
            rq.load(p.q, at);
            if constexpr (GATEK) rgk.load(p.g, (tok * p.H + h) * K + sk);
        } else if constexpr (GATEK) {
            rgk.zero();
        }
        if (vt < TB && t0 + vt < n) rv.load(p.v, ((long long)(lo + t0 + vt) * p.H + h) * p.V + tile * COLS + vc);
        if (tid < TB && t0 + tid < n) {
            const long long at = (long long)(lo + t0 + tid) * p.H + h;
            raw_b = load1<BF>(p.beta, at);
            if constexpr (!GATEK) raw_g = load1<BF>(p.g, at);
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
        if (st < TB) {
            put8(&ks[b][st][sk], fk);
            if constexpr (GATEK) {
                float e[8];
                rgk.values(e);
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
        if (vt < TB) {
            float f[8];
            rv.values(f);
            put8(&vs[b][vt][vc], f);
        }
        if (tid < TB) {
            sc[b][tid].x = expf(raw_g);
            sc[b][tid].y = raw_b;
        }
    };
    if (n > 0) load_tokens(0);

    // nothing is written before the lengths and the slots are known to be good
    bool write_state = slot_out >= 0 && slot_out < p.num_slots;
    if (p.owner) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (__ldcg(p.cu_bad)) return;
        if (write_state && __ldcg(p.owner + slot_out) != s) {
            write_state = false;
            if (tid == 0) report(p.err, kTagSlotShared);
        }
    } else {
        if (p.cu) {
            bool bad = tid == 0 && (__ldg(p.cu) != 0 || __ldg(p.cu + p.nseq) != p.T);
            for (int j = tid; j < p.nseq; j += THREADS) bad |= __ldg(p.cu + j + 1) < __ldg(p.cu + j);
            if (__syncthreads_or(bad)) {
                if (tid == 0) report(p.err, kTagLengths);
                return;
            }
        }
        if (write_state && p.nseq > 1) {
            bool shared = false;
            for (int j = tid; j < p.nseq; j += THREADS)
                shared |= j != s && (__ldg(p.slots_out + j) == slot_out ||
                                     (p.slots_in && __ldg(p.slots_in + j) == slot_out));
            if (__syncthreads_or(shared)) {
                write_state = false;
                if (tid == 0) report(p.err, kTagSlotShared);
            }
        }
    }
    if (tid == 0 && (!in_ok || slot_out >= p.num_slots)) report(p.err, kTagSlotRange);
    if (!in_ok) return;

    auto store_state = [&](int slot) {
        float* dst = p.state + slot * page + lane_off;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float* row = dst + (long long)(4 * (i * RG + rg) + 2 * j) * p.V;
                float4 a, b;
                unpack(S[i][j][0], a.x, b.x);
                unpack(S[i][j][1], a.y, b.y);
                unpack(S[i][j][2], a.z, b.z);
                unpack(S[i][j][3], a.w, b.w);
                *reinterpret_cast<float4*>(row) = a;
                *reinterpret_cast<float4*>(row + p.V) = b;
            }
        }
    };

    const bool up16 = lane & 16, up8 = lane & 8;
    const int oc = (up16 ? 2 : 0) + (up8 ? 1 : 0);   // this lane's column once the sums are joined
    const bool writes_o = (lane & 7 & ~(CL - 1)) == 0;
    for (int t0 = 0, b = 0; t0 < n; t0 += TB, b ^= 1) {
        // (buffer b was last read before the barrier of the block in between)
        store_tokens(b);
        __syncthreads();
        if (t0 + TB < n) load_tokens(t0 + TB);
        const int m = min(TB, n - t0);
        for (int t = 0; t < m; ++t) {
            // the sums over the rows: of this lane's, then of the lanes that hold the same columns
            pair_t ak[4] = {0, 0, 0, 0}, aq[4] = {0, 0, 0, 0};
            const float* kread = GATEK ? kr[b][t] : ks[b][t];
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(kread + 4 * (i * RG + rg));
                const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(&qs[b][t][4 * (i * RG + rg)]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    ak[c] = fma2(S[i][0][c], k2.x, ak[c]);
                    aq[c] = fma2(S[i][0][c], q2.x, aq[c]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    ak[c] = fma2(S[i][1][c], k2.y, ak[c]);
                    aq[c] = fma2(S[i][1][c], q2.y, aq[c]);
                }
            }
            float dk[4], dq[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                dk[c] = total(ak[c]);
                dq[c] = total(aq[c]);
            }
            auto join = [&](const float (&d)[4]) {   // lane l ends with its column oc's whole sum
                float x = up16 ? d[2] : d[0], y = up16 ? d[3] : d[1];
                x += __shfl_xor_sync(0xffffffffu, up16 ? d[0] : d[2], 16);
                y += __shfl_xor_sync(0xffffffffu, up16 ? d[1] : d[3], 16);
                float z = up8 ? y : x;
                z += __shfl_xor_sync(0xffffffffu, up8 ? x : y, 8);
#pragma unroll
                for (int off = 4; off >= CL; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
                return z;
            };
            const float sk_ = join(dk), sq_ = join(dq);
            const float4 g4 = sc[b][t];   // exp(g), beta, q . k
            const float e = GATEK ? 1.f : g4.x;
            const float read = !GATEK && p.decay_first ? e * sk_ : sk_;
            const float r = g4.y * (vs[b][t][warp * CW + 4 * cl + oc] - read);
            if (writes_o) {
                const long long at = ((long long)(lo + t0 + t) * p.H + h) * p.V + c0 + oc;
                const float o = fmaf(g4.z, r, e * sq_);
                if (p.out_bf16)
                    reinterpret_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(o);
                else
                    reinterpret_cast<float*>(p.o)[at] = o;
            }
            // r of all four columns, then the update
            const float ro = __shfl_xor_sync(0xffffffffu, r, 8);
            const float x = up8 ? ro : r, y = up8 ? r : ro;
            const float xo = __shfl_xor_sync(0xffffffffu, x, 16), yo = __shfl_xor_sync(0xffffffffu, y, 16);
            const float rc[4] = {up16 ? xo : x, up16 ? yo : y, up16 ? x : xo, up16 ? y : yo};
            pair_t r2[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) r2[c] = pack(rc[c], rc[c]);
            const pair_t e2 = pack(e, e);
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&ks[b][t][4 * (i * RG + rg)]);
                pair_t ex = e2, ey = e2;
                if constexpr (GATEK) {
                    const ulonglong2 ek = *reinterpret_cast<const ulonglong2*>(&es[b][t][4 * (i * RG + rg)]);
                    ex = ek.x;
                    ey = ek.y;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    S[i][0][c] = fma2(k2.x, r2[c], mul2(S[i][0][c], ex));
                    S[i][1][c] = fma2(k2.y, r2[c], mul2(S[i][1][c], ey));
                }
            }
            if (p.per_token && p.slots_out) {
                const int slot = __ldg(p.slots_out + lo + t0 + t);
                if (slot >= p.num_slots) {
                    if (tid == 0) report(p.err, kTagSlotRange);
                } else if (slot >= 0) {
                    if (!p.owner || __ldcg(p.owner + slot) == s)
                        store_state(slot);
                    else if (tid == 0)
                        report(p.err, kTagSlotShared);
                }
            }
        }
    }
    if (write_state) store_state(slot_out);
}

template <int K, int CW, int WARPS>
cudaError_t launch(const RecurrentParams& p, bool gate_k, bool bf16, cudaStream_t s) {
    const void* fn = gate_k ? (bf16 ? (const void*)recurrent_kernel<K, CW, WARPS, true, true>
                                    : (const void*)recurrent_kernel<K, CW, WARPS, true, false>)
                            : (bf16 ? (const void*)recurrent_kernel<K, CW, WARPS, false, true>
                                    : (const void*)recurrent_kernel<K, CW, WARPS, false, false>);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.nseq * p.H * (p.V / (CW * WARPS))));
    cfg.blockDim = dim3(32 * WARPS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.owner ? 1 : 0;   // the dependent of claim_kernel
    RecurrentParams copy = p;
    void* args[] = {&copy};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int K>
cudaError_t launch_k(const RecurrentParams& p, bool gate_k, bool bf16, int sms, cudaStream_t s) {
    const long long warps = (long long)p.nseq * p.H * (p.V / 32);
    if (warps >= 8LL * sms)
        return p.V == 64 ? launch<K, 32, 2>(p, gate_k, bf16, s) : launch<K, 32, 4>(p, gate_k, bf16, s);
    if (warps >= 4LL * sms) return launch<K, 16, 4>(p, gate_k, bf16, s);
    return launch<K, 8, 4>(p, gate_k, bf16, s);
}

// Each block of the rule looks for other sequences that name its slot when there are at most this many
// sequences; above it, and where states are kept after every token, claim_kernel does so once.
constexpr int kInlineSeqs = 512;

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
    // token numbers, and the grid at its finest split, in 31 bits
    if ((long long)p->B * p->T >= (1LL << 31) || (long long)nseq * p->H * 4 >= (1LL << 31))
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
    c.per_token = per_token;
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
    if ((p->K == 64 ? launch_k<64>(c, p->gate_k, bf16, sms, s)
                    : launch_k<128>(c, p->gate_k, bf16, sms, s)) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

}  // extern "C"

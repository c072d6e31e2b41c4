// gdn_linear.cu -- entry points of the chunked linear attention with a decay for each head (gdn_linear_fwd,
// gdn_linear_bwd): checks, how sequences are cut into pieces, the plan of a packed batch, gradients of shared heads.
#include <algorithm>
#include <climits>

#include "gdn_linear.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kPlanThreads = 1024;
constexpr unsigned kTagLengths = 0x51;
// words of the workspace's header, from kWsVerdict on: entries of the two phases, tokens of all sequences
enum { kCount1 = 0, kCount2, kTokens };

struct Cut {
    int first = 0, rest = 0;     // chunks of piece 0 and of the others; rest 0: no sequence is cut
    int pieces = 1;              // of every sequence, where all have T tokens
    long long entries2 = 0;      // bound on the entries of phase 2, which bounds the middle pieces' sums too
};

// How sequences are cut. `room`: kernel blocks that the GPU holds at once, `per`: blocks that one piece takes. A sequence cut
// into piece 0 of `first` chunks and others of `rest` takes first + rest chunks' time instead of all of them (a sum over a
// piece takes about half of a forward's time, so first = rest / 2 ends with the sums), and a second launch, which is
// worth kSaved chunks.
constexpr int kSaved = 4;
Cut cut(long long T, int nseq, bool packed, long long room, long long per) {
    Cut c;
    const long long at_once = room / per;
    if (at_once < 2) return c;
    if (!packed) {
        const long long n = (T + kChunk - 1) / kChunk;
        const long long more = std::min(at_once / nseq, n);   // pieces behind the first one
        if (more < 2) return c;
        const long long rest = (2 * n + 2 * more) / (2 * more + 1);   // n / (more + 1/2), rounded up
        long long first = n - more * rest;
        if (first < 1) first = std::max(1LL, rest / 2);
        if (first + rest + kSaved > n) return c;
        c.first = (int)first;
        c.rest = (int)rest;
        c.pieces = 1 + (int)((n - first + rest - 1) / rest);
        c.entries2 = (long long)nseq * (c.pieces - 1);
        return c;
    }
    const long long most = T / kChunk + nseq;   // chunks of any lengths
    const long long n = T / kChunk + nseq / 2;  // and as a rule
    const long long rest = std::max(1LL, (n + at_once - 1) / at_once), first = (rest + 1) / 2;
    if (first + rest + kSaved > T / kChunk + 1) return c;
    c.first = (int)first;
    c.rest = (int)rest;
    c.entries2 = most / rest + std::min<long long>(nseq, most / (first + rest + kSaved));
    return c;
}

// whether a sequence of n chunks is cut, and into how many pieces (packed batches)
__host__ __device__ inline int pieces_of(int n, int first, int rest) {
    return rest > 0 && n >= first + rest + kSaved ? 1 + (n - first + rest - 1) / rest : 1;
}

// Checks the lengths of a packed batch and makes the phases' entries: every sequence's piece 0, then the middle pieces;
// the pieces from 1 on. Bad lengths are recorded and leave no entries, so that nothing is written.
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int* cu, int nseq, int T, int first, int rest, int bound2, int* words, int4* table1, int4* table2,
                DeviceError* err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int warp_sum[32];
    const int t = threadIdx.x;
    bool bad = t == 0 && (cu[0] != 0 || cu[nseq] > T);
    for (int s = t; s < nseq; s += kPlanThreads) bad |= cu[s + 1] < cu[s];
    if (__syncthreads_or(bad)) {
        if (t == 0) {
            if (atomicCAS(&err->code, 0u, (unsigned)GDN_ERR_INVALID_ARG) == 0u) atomicExch(&err->detail, kTagLengths);
            words[kCount1] = words[kCount2] = words[kTokens] = 0;
        }
        return;
    }
    int before = 0;   // pieces behind the first ones of all sequences before this round's
    for (int s0 = 0; s0 < nseq; s0 += kPlanThreads) {
        const int s = s0 + t;
        const int n = s < nseq ? (int)(((long long)cu[s + 1] - cu[s] + kChunk - 1) / kChunk) : 0;
        const int pieces = s < nseq ? pieces_of(n, first, rest) : 1;
        int sum = pieces - 1;   // inclusive sums over the warp, then over the warps
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, sum, off);
            if ((t & 31) >= off) sum += y;
        }
        if ((t & 31) == 31) warp_sum[t >> 5] = sum;
        __syncthreads();
        if (t < 32) {
            int x = warp_sum[t];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (t >= off) x += y;
            }
            warp_sum[t] = x;
        }
        __syncthreads();
        const int slot0 = before + sum - (pieces - 1) + (t >= 32 ? warp_sum[(t >> 5) - 1] : 0);
        if (s < nseq && slot0 + pieces - 1 <= bound2) {
            table1[s] = make_int4(s, 0, pieces, slot0);
            for (int q = 1; q < pieces; ++q) {
                table2[slot0 + q - 1] = make_int4(s, q, pieces, slot0);
                // (the last piece's place among the sums stays empty: seq -1)
                table1[nseq + slot0 + q - 1] = make_int4(q < pieces - 1 ? s : -1, q, pieces, slot0);
            }
        } else if (s < nseq) {
            table1[s] = make_int4(s, 0, 1, 0);   // (the bound holds: not reached)
        }
        before += warp_sum[31];
        __syncthreads();
    }
    if (t == 0) {
        words[kCount1] = nseq + before;
        words[kCount2] = before;
        words[kTokens] = cu[nseq];
    }
}

// out[t][g][k] = the sum over the heads h of group g, in order, of part[t][h][k], four values a thread
__global__ void __launch_bounds__(256) group_kernel(const float* part, void* out, int out_bf16, long long fours, int H, int groups,
                                                    int D, const int* tokens) {
    const int rep = H / groups, d4 = D / 4;
    if (tokens) fours = min(fours, (long long)__ldcg(tokens) * groups * d4);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < fours; i += (long long)gridDim.x * 256) {
        const int k = (int)(i % d4);
        const long long tg = i / d4;   // token * groups + group: its first head is tg * rep
        const float4* from = reinterpret_cast<const float4*>(part) + (tg * rep) * d4 + k;
        float4 s = __ldcs(from);
        for (int r = 1; r < rep; ++r) {
            const float4 x = __ldcs(from + (long long)r * d4);
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        if (out_bf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            uint2 u;
            u.x = *reinterpret_cast<const unsigned*>(&lo);
            u.y = *reinterpret_cast<const unsigned*>(&hi);
            reinterpret_cast<uint2*>(out)[i] = u;
        } else {
            reinterpret_cast<float4*>(out)[i] = s;
        }
    }
}

gdn_status check(const gdn_problem* p, int Hqk, int nseq, bool packed) {
    if (!p) return GDN_ERR_INVALID_ARG;
    if (p->B < 1 || p->H < 1 || p->T < 0 || nseq < 1 || Hqk < 1) return GDN_ERR_INVALID_ARG;
    if (packed ? p->B != 1 : p->B != nseq) return GDN_ERR_INVALID_ARG;
    if (p->decay_first || p->gate_k) return GDN_ERR_INVALID_ARG;
    if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128)) return GDN_ERR_UNSUPPORTED_SHAPE;
    if (p->H % Hqk != 0) return GDN_ERR_UNSUPPORTED_SHAPE;
    if ((p->in_dtype != GDN_DTYPE_F32 && p->in_dtype != GDN_DTYPE_BF16) ||
        (p->out_dtype != GDN_DTYPE_F32 && p->out_dtype != GDN_DTYPE_BF16))
        return GDN_ERR_UNSUPPORTED_DTYPE;
    // (token numbers and the steps behind the last one in an int; the grid in 31 bits)
    if ((long long)p->B * p->T > INT_MAX - 4096 || (long long)nseq * p->H >= (1LL << 28) || p->H > (1 << 20))
        return GDN_ERR_UNSUPPORTED_SHAPE;
    return GDN_OK;
}

// blocks that one piece takes, and that the GPU holds at once
long long blocks_of(const gdn_problem& p, bool tc, int roles) {
    if (tc) return (long long)p.H * roles;
    return (long long)p.H * (roles == 3 ? 2 * p.K / 64 + p.V / 64 : p.V / 64);
}
long long room_of(bool tc, int sms) { return (tc ? 1LL : 2LL) * sms; }

struct Layout {
    size_t table1, table2, slots, part[2], total;
    size_t slot_bytes;   // of one role
};
Layout layout(const gdn_problem& p, int Hqk, int nseq, bool packed, const Cut& c, bool backward) {
    Layout l{};
    size_t at = kWsHeader;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += ws_round(bytes);
        return here;
    };
    if (packed) {
        l.table1 = take(sizeof(int4) * (size_t)(nseq + c.entries2));
        l.table2 = take(sizeof(int4) * (size_t)c.entries2);
    }
    l.slot_bytes = ws_round(sizeof(float) * (size_t)c.entries2 * p.H * p.K * p.V);
    l.slots = take(l.slot_bytes * (backward ? 3 : 1));
    if (backward && Hqk != p.H)
        for (size_t& x : l.part) x = take(sizeof(float) * (size_t)p.B * p.T * p.H * p.K);
    l.total = at;
    return l;
}

bool misaligned(const void* ptr, unsigned bytes) { return reinterpret_cast<uintptr_t>(ptr) & (bytes - 1); }

// Both directions: the roles' pieces in one or two launches, behind the plan of a packed batch.
gdn_status run(Params& c, const gdn_problem& p, int Hqk, bool backward, void* workspace, cudaStream_t s) {
    const bool packed = c.cu != nullptr;
    const bool tc = tc_supported(c);
    const int sms = current_sm_count();
    const Cut k = cut(p.T, c.nseq, packed, room_of(tc, sms), blocks_of(p, tc, c.nroles));
    const Layout l = layout(p, Hqk, c.nseq, packed, k, backward);
    char* ws = reinterpret_cast<char*>(workspace);
    c.err = reinterpret_cast<DeviceError*>(ws);
    c.first = k.first;
    c.rest = k.rest;
    c.pieces = k.pieces;
    for (int i = 0; i < c.nroles; ++i) c.role[i].slots = reinterpret_cast<float*>(ws + l.slots + i * l.slot_bytes);
    int* words = reinterpret_cast<int*>(ws + kWsVerdict);
    int4* table1 = reinterpret_cast<int4*>(ws + l.table1);
    int4* table2 = reinterpret_cast<int4*>(ws + l.table2);
    if (packed) {
        plan_kernel<<<1, kPlanThreads, 0, s>>>(c.cu, c.nseq, p.T, k.first, k.rest, (int)k.entries2, words, table1, table2, c.err);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    }
    auto phase = [&](int number, long long entries) {
        c.phase = number;
        c.entries = (int)entries;
        c.table = reinterpret_cast<const int*>(number == 1 ? table1 : table2);
        c.count = words + (number == 1 ? kCount1 : kCount2);
        c.dependent = packed || number == 2;
        return tc ? launch_tc(c, s) : launch_simt(c, s);
    };
    const long long middle = packed ? k.entries2 : k.rest ? (long long)c.nseq * (k.pieces - 2) : 0;
    if (phase(1, c.nseq + middle) != cudaSuccess) return GDN_ERR_CUDA;
    if (k.entries2 > 0 && phase(2, k.entries2) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
}

}  // namespace
}  // namespace linear
}  // namespace gdn

using namespace gdn;
using namespace gdn::linear;

extern "C" {

size_t gdn_linear_workspace_bytes(const gdn_problem* p, int Hqk, int nseq, int backward) {
    size_t most = 0;
    for (int packed = 0; packed < 2; ++packed) {
        if (check(p, Hqk, nseq, packed) != GDN_OK) continue;
        for (int tc = 0; tc < 2; ++tc) {   // (which kernels run depends on the output's type too)
            const Cut c = cut(p->T, nseq, packed, room_of(tc, current_sm_count()), blocks_of(*p, tc, backward ? 3 : 1));
            most = std::max(most, layout(*p, Hqk, nseq, packed, c, backward != 0).total);
        }
    }
    return most;
}

gdn_status gdn_linear_fwd(const gdn_problem* p, int Hqk, int nseq, const int* cu_seqlens, const void* q, const void* k,
                          const void* v, const float* decay, const float* h0, void* o, float* h_final, void* workspace,
                          size_t workspace_bytes, void* stream) {
    gdn_status st = check(p, Hqk, nseq, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!decay || (p->T > 0 && (!q || !k || !v || !o))) return GDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdn_linear_workspace_bytes(p, Hqk, nseq, 0)) return GDN_ERR_WORKSPACE;
    for (const void* ptr : {q, k, v, (const void*)h0, (const void*)o, (const void*)h_final, (const void*)workspace})
        if (misaligned(ptr, 16)) return GDN_ERR_MISALIGNED;
    for (const void* ptr : {(const void*)cu_seqlens, (const void*)decay})
        if (misaligned(ptr, 4)) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    Params c{};
    Role& r = c.role[0];
    r.a = q, r.b = k, r.c = v;
    r.out = o;
    r.start = h0;
    r.last = h_final;
    r.a_heads = r.b_heads = Hqk;
    r.c_heads = p->H;
    r.a_bf16 = r.b_bf16 = r.c_bf16 = p->in_dtype == GDN_DTYPE_BF16;
    r.out_bf16 = p->out_dtype == GDN_DTYPE_BF16;
    r.dA = p->K;
    r.dC = p->V;
    c.nroles = 1;
    c.decay = decay;
    c.cu = cu_seqlens;
    c.nseq = nseq;
    c.T = p->T;
    c.H = p->H;
    return run(c, *p, Hqk, false, workspace, reinterpret_cast<cudaStream_t>(stream));
}

gdn_status gdn_linear_bwd(const gdn_problem* p, int Hqk, int nseq, const int* cu_seqlens, const void* q, const void* k,
                          const void* v, const float* decay, const float* h0, const void* dO, const float* dht, void* dq,
                          void* dk, void* dv, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    gdn_status st = check(p, Hqk, nseq, cu_seqlens != nullptr);
    if (st != GDN_OK) return st;
    if (!decay || (p->T > 0 && (!q || !k || !v || !dO || !dq || !dk || !dv))) return GDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdn_linear_workspace_bytes(p, Hqk, nseq, 1)) return GDN_ERR_WORKSPACE;
    for (const void* ptr : {q, k, v, (const void*)h0, dO, (const void*)dht, (const void*)dq, (const void*)dk, (const void*)dv,
                            (const void*)dh0, (const void*)workspace})
        if (misaligned(ptr, 16)) return GDN_ERR_MISALIGNED;
    for (const void* ptr : {(const void*)cu_seqlens, (const void*)decay})
        if (misaligned(ptr, 4)) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int in = p->in_dtype == GDN_DTYPE_BF16, out = p->out_dtype == GDN_DTYPE_BF16;
    const bool grouped = Hqk != p->H;
    Params c{};
    c.nroles = 3;
    c.decay = decay;
    c.cu = cu_seqlens;
    c.nseq = nseq;
    c.T = p->T;
    c.H = p->H;
    for (int i = 0; i < 3; ++i) {
        Role& r = c.role[i];
        const bool is_dq = i == 0, is_dv = i == 2;
        r.a = is_dq ? dO : is_dv ? k : v;
        r.b = is_dq ? v : is_dv ? q : dO;
        r.c = is_dq ? k : is_dv ? dO : q;
        r.a_heads = is_dv ? Hqk : p->H;
        r.b_heads = is_dv ? Hqk : p->H;
        r.c_heads = is_dv ? p->H : Hqk;
        r.a_bf16 = is_dq ? out : in;
        r.b_bf16 = is_dq || is_dv ? in : out;
        r.c_bf16 = is_dv ? out : in;
        r.out = is_dq ? dq : is_dv ? dv : dk;
        r.out_bf16 = in;
        r.dA = is_dv ? p->K : p->V;
        r.dC = is_dv ? p->V : p->K;
        r.rev = !is_dq;
        r.state_t = !is_dv;
        r.start = is_dq ? h0 : dht;
        r.last = is_dv ? dh0 : nullptr;
    }
    // the gradients of shared heads: each head's own in the workspace, then their sums
    char* ws = reinterpret_cast<char*>(workspace);
    const bool tc = tc_supported(c);
    const Layout l = layout(*p, Hqk, nseq, cu_seqlens != nullptr,
                            cut(p->T, nseq, cu_seqlens != nullptr, room_of(tc, current_sm_count()), blocks_of(*p, tc, 3)), true);
    if (grouped)
        for (int i = 0; i < 2; ++i) {
            c.role[i].out = ws + l.part[i];
            c.role[i].out_bf16 = 0;
        }
    st = run(c, *p, Hqk, true, workspace, s);
    if (st != GDN_OK || !grouped || p->T == 0) return st;
    for (int i = 0; i < 2; ++i) {
        const long long fours = (long long)p->B * p->T * Hqk * p->K / 4;
        const unsigned blocks = (unsigned)std::min<long long>((fours + 255) / 256, 16LL * std::max(1, current_sm_count()));
        group_kernel<<<blocks, 256, 0, s>>>(reinterpret_cast<const float*>(ws + l.part[i]), i ? dk : dq, in, fours, p->H, Hqk,
                                            p->K, cu_seqlens ? reinterpret_cast<const int*>(ws + kWsVerdict) + kTokens : nullptr);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
    }
    return GDN_OK;
}

}  // extern "C"

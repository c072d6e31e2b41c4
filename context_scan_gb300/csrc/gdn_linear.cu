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
// How chains are cut into pieces. `room`: pieces that the GPU runs at once. A chain of n chunks cut into piece 0 of `first` and
// others of `rest` takes first + rest chunks' time instead of n (a sum over a piece takes about half of a forward's time,
// so that first = rest / 2 ends with the sums), and a second launch, which is worth kSaved chunks.
constexpr int kSaved = 3;
struct Cut {
    int whole = INT_MAX;         // chains that are not cut come first
    int first = 0, rest = 0, pieces = 1;
    long long blocks2 = 0;       // of phase 2, which has as many pieces as phase 1 has piece 0s and sums of cut chains
};
__host__ __device__ inline int first_of(int rest) { return (rest + 1) / 2; }

// Chains of n chunks each: as many as fill the GPU whole rounds run in one piece, the others are cut so that they fill it too.
Cut cut_even(long long T, long long chains, long long room) {
    Cut c;
    const long long n = (T + kChunk - 1) / kChunk, left = room > 0 ? chains % room : 0;
    if (left == 0) return c;
    const long long more = std::min(room / left, n);       // pieces behind the first one
    if (more < 2) return c;
    const long long rest = (2 * n + 2 * more) / (2 * more + 1);   // n / (more + 1/2), rounded up
    long long first = n - more * rest;
    if (first < 1) first = first_of((int)rest);
    if (first + rest + kSaved > n) return c;
    c.whole = (int)(chains - left);
    c.first = (int)first;
    c.rest = (int)rest;
    c.pieces = 1 + (int)((n - first + rest - 1) / rest);
    c.blocks2 = left * (c.pieces - 1);
    return c;
}

// Packed sequences: whether the plan may cut any, with room for `room` pieces behind first ones.
bool cut_possible(long long T, long long room) { return room >= 2 && T / kChunk + 1 >= 2 + kSaved; }

// a sequence of n chunks, in a batch that is cut
__device__ __forceinline__ int more_pieces(int n, int first, int rest) { return n > first + 1 ? (n - first + rest - 1) / rest : 0; }

// Checks the lengths of a packed batch and makes the phases' entries: every sequence's piece 0, then the middle pieces;
// the pieces from 1 on. Bad lengths are recorded and leave no entries, so that nothing is written. The cut: the
// shortest `rest` with which at most `room` pieces lie behind first ones (every warp tries one), where that takes less time
// than no cut. Times in chunks: the longest piece, or, where there are more pieces than room, an even share of all and half of
// the longest. Longer sequences come first, any number of them, sorted by counting chunks (in steps of a power of two where a
// length exceeds 1023 chunks). Whole calls on sequences of up to three tokens, one head, K = V = 64: 300 sequences 18.5 us, 1000 45 us
// (25.6 and 107 when every thread counted the longer ones).
__device__ __forceinline__ long long warp_total(long long x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}
// exclusive sum of x over the block's threads; `scratch` has a place for each warp
__device__ __forceinline__ int block_scan(int x, int* scratch, int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += y;
    }
    __syncthreads();   // (the scratch of the call before)
    if (lane == 31) scratch[warp] = sum;
    __syncthreads();
    int before = scratch[lane];   // every warp sums all of them up
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, before, off);
        if (lane >= off) before += y;
    }
    all = __shfl_sync(0xffffffffu, before, 31);
    const int mine = __shfl_sync(0xffffffffu, before, warp > 0 ? warp - 1 : 0);
    return sum - x + (warp > 0 ? mine : 0);
}
// counter[b] += 1 for every lane that is `on` (all lanes take part), one addition for those of a warp with the same b; the lane's
// place among all that have counted there
__device__ __forceinline__ int count_up(int* counter, int b, bool on) {
    const int lane = threadIdx.x & 31;
    const unsigned same = __match_any_sync(0xffffffffu, on ? b : -1);
    const int first = __ffs(same) - 1;
    int from = 0;
    if (on && lane == first) from = atomicAdd(counter + b, __popc(same));
    return __shfl_sync(0xffffffffu, from, first) + __popc(same & ((1u << lane) - 1u));
}
__global__ void __launch_bounds__(kPlanThreads)
    plan_kernel(const int* cu, int nseq, int T, int room, int* words, int4* table1, int4* table2, DeviceError* err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __shared__ int warp_sum[32], warp_max[32];
    __shared__ long long warp_time[32];
    __shared__ int place[kPlanThreads];   // of the next sequence of a length, the longest first
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
    bool bad = t == 0 && (cu[0] != 0 || cu[nseq] > T);
    int longest = 0;
    long long all = 0;
    for (int s = t; s < nseq; s += kPlanThreads) {
        const int a = cu[s], b = cu[s + 1];
        bad |= b < a;
        const int n = (int)(((long long)b - a + kChunk - 1) / kChunk);
        longest = max(longest, n);
        all += n;
    }
    if (__syncthreads_or(bad)) {
        if (t == 0) {
            if (atomicCAS(&err->code, 0u, (unsigned)GDN_ERR_INVALID_ARG) == 0u) atomicExch(&err->detail, kTagLengths);
            words[kCount1] = words[kCount2] = words[kTokens] = 0;
        }
        return;
    }
    auto chunks = [&](int s) { return (cu[s + 1] - cu[s] + kChunk - 1) / kChunk; };
    int first = 0, rest = 0;
    longest = __reduce_max_sync(0xffffffffu, longest);
    all = warp_total(all);
    if (lane == 0) {
        warp_max[warp] = longest;
        warp_time[warp] = all;
    }
    place[t] = 0;
    __syncthreads();
    longest = __reduce_max_sync(0xffffffffu, warp_max[lane]);
    all = warp_total(warp_time[lane]);
    if (room > 0) {
        const long long uncut = nseq > room ? max((long long)longest, all / room + longest / 2) : longest;
        // lengths worth trying: from what an even cut of all chunks would give on, in steps of a sixteenth, three times as far
        // a round
        const int even = max(1, (int)(((long long)cu[nseq] / kChunk) / (room + nseq)));
        for (int r0 = even; r0 + first_of(r0) + kSaved <= longest; r0 *= 3) {
            const int step = (r0 + 15) / 16, r = r0 + warp * step, f = first_of(r);
            long long count = 0, work = 0;   // pieces behind first ones; chunks of phase 1 (sums by half)
            for (int s = lane; s < nseq; s += 32) {
                const int n = chunks(s), more = more_pieces(n, f, r);
                count += more;
                work += more ? f + (more - 1) * r / 2 : n;
            }
            count = warp_total(count);
            work = warp_total(work);
            const long long phase1 = nseq + count > room + room / 4 ? max((long long)f, work / room + f / 2) : f + 1;
            __syncthreads();
            if (lane == 0) {
                warp_sum[warp] = count <= room;
                warp_time[warp] = phase1 + r + kSaved;
            }
            __syncthreads();
            const unsigned fit = __ballot_sync(0xffffffffu, warp_sum[lane]);
            if (fit) {
                if (warp_time[__ffs(fit) - 1] <= uncut) rest = r0 + (__ffs(fit) - 1) * step;
                first = first_of(rest);
                break;
            }
        }
    }
    int step = 0, sum;
    while (longest >> step >= kPlanThreads) ++step;
    auto bucket = [&](int s) { return kPlanThreads - 1 - (chunks(s) >> step); };
    for (int s0 = 0; s0 < nseq; s0 += kPlanThreads) count_up(place, s0 + t < nseq ? bucket(s0 + t) : 0, s0 + t < nseq);
    __syncthreads();
    const int ahead = block_scan(place[t], warp_sum, sum);
    place[t] = ahead;
    __syncthreads();
    int before = 0;   // pieces behind the first ones of all sequences before this round's
    for (int s0 = 0; s0 < nseq; s0 += kPlanThreads) {
        const int s = s0 + t;
        const bool on = s < nseq;
        const int pieces = on && rest > 0 ? 1 + more_pieces(chunks(s), first, rest) : 1;
        const int slot0 = before + block_scan(pieces - 1, warp_sum, sum);
        before += sum;
        const int at = count_up(place, on ? bucket(s) : 0, on);
        if (!on) continue;
        table1[at] = make_int4(s, 0, pieces, slot0);
        for (int q = 1; q < pieces; ++q) {
            table2[slot0 + q - 1] = make_int4(s, q, pieces, slot0);
            // (the last piece's place among the sums stays empty: sequence -1)
            table1[nseq + slot0 + q - 1] = make_int4(q < pieces - 1 ? s : -1, q, pieces, slot0);
        }
    }
    if (t == 0) {
        words[kCount1] = nseq + before;
        words[kCount2] = before;
        words[kTokens] = cu[nseq];
        words[kFirst] = first;
        words[kRest] = rest;
    }
}

// out[t][g][k] = the sum over the heads h of group g, in order, of part[t][h][k], four values a thread; dq (blockIdx.y 0), dk
struct Groups {
    const float* part[2];
    void* out[2];
    const int* tokens;   // of packed sequences, on the device; or null
    long long fours;
    int out_bf16, H, groups, D;
};
__global__ void __launch_bounds__(256) group_kernel(const Groups g) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int rep = g.H / g.groups, d4 = g.D / 4;
    long long fours = g.fours;
    if (g.tokens) fours = min(fours, (long long)__ldcg(g.tokens) * g.groups * d4);
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < fours; i += (long long)gridDim.x * 256) {
        const int k = (int)(i % d4);
        const long long tg = i / d4;   // token * groups + group: its first head is tg * rep
        const float4* from = reinterpret_cast<const float4*>(g.part[blockIdx.y]) + (tg * rep) * d4 + k;
        float4 s = __ldcs(from);
        for (int r = 1; r < rep; ++r) {
            const float4 x = __ldcs(from + (long long)r * d4);
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        if (g.out_bf16) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(s.x, s.y), hi = __floats2bfloat162_rn(s.z, s.w);
            uint2 u;
            u.x = *reinterpret_cast<const unsigned*>(&lo);
            u.y = *reinterpret_cast<const unsigned*>(&hi);
            reinterpret_cast<uint2*>(g.out[blockIdx.y])[i] = u;
        } else {
            reinterpret_cast<float4*>(g.out[blockIdx.y])[i] = s;
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

// Blocks that the GPU runs at once, in pieces of one chain; and of one sequence with all its heads and roles (packed)
long long room_of(const gdn_problem& p, bool tc, int sms, bool backward) {
    return tc ? sms : 2LL * sms / (std::max(backward ? p.K : 0, p.V) / 64);
}
long long packed_room(const gdn_problem& p, bool tc, int sms, bool backward) {
    const long long room = room_of(p, tc, sms, backward) / ((long long)p.H * (backward ? 3 : 1));
    return cut_possible(p.T, room) ? room : 0;
}

struct Layout {
    size_t table1, table2, slots, part[2], total;
};
Layout layout(const gdn_problem& p, int Hqk, int nseq, bool packed, bool tc, int sms, bool backward, Cut* even = nullptr) {
    Layout l{};
    size_t at = kWsHeader;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += ws_round(bytes);
        return here;
    };
    const long long width = (long long)p.H * (backward ? 3 : 1);
    long long states;
    if (packed) {
        const long long room = packed_room(p, tc, sms, backward);
        l.table1 = take(sizeof(int4) * (size_t)(nseq + room));
        l.table2 = take(sizeof(int4) * (size_t)room);
        states = room * width;
    } else {
        const Cut c = cut_even(p.T, nseq * width, room_of(p, tc, sms, backward));
        if (even) *even = c;
        states = c.blocks2;
    }
    l.slots = take(sizeof(float) * (size_t)states * p.K * p.V);
    if (backward && Hqk != p.H)
        for (size_t& x : l.part) x = take(sizeof(float) * (size_t)p.B * p.T * p.H * p.K);
    l.total = at;
    return l;
}

bool misaligned(const void* ptr, unsigned bytes) { return reinterpret_cast<uintptr_t>(ptr) & (bytes - 1); }

// Both directions: the chains' pieces in one or two launches, behind the plan of a packed batch.
gdn_status run(Params& c, const gdn_problem& p, int Hqk, bool backward, void* workspace, cudaStream_t s) {
    const bool packed = c.cu != nullptr;
    const bool tc = tc_supported(c);
    const int sms = current_sm_count();
    Cut k;
    const Layout l = layout(p, Hqk, c.nseq, packed, tc, sms, backward, &k);
    char* ws = reinterpret_cast<char*>(workspace);
    c.err = reinterpret_cast<DeviceError*>(ws);
    c.slots = reinterpret_cast<float*>(ws + l.slots);
    c.whole = k.whole;
    c.first = k.first;
    c.rest = k.rest;
    c.pieces = k.pieces;
    int* words = reinterpret_cast<int*>(ws + kWsVerdict);
    int4* table1 = reinterpret_cast<int4*>(ws + l.table1);
    int4* table2 = reinterpret_cast<int4*>(ws + l.table2);
    const long long width = (long long)c.H * c.nroles, chains = c.nseq * width;
    long long blocks1 = chains, blocks2 = 0;
    if (packed) {
        const int room = (int)packed_room(p, tc, sms, backward);
        plan_kernel<<<1, kPlanThreads, 0, s>>>(c.cu, c.nseq, p.T, room, words, table1, table2, c.err);
        if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
        blocks2 = room * width;
        blocks1 += blocks2;
    } else if (k.blocks2 > 0) {
        blocks2 = k.blocks2;
        blocks1 += blocks2 / (k.pieces - 1) * (k.pieces - 2);
    }
    c.words = words;
    // Roles of different sizes or outputs run different code, and the two SMs of a pair share what holds it: with a head's roles
    // side by side their CTAs keep displacing each other's. So blocks of one role lie side by side there (gradients of 1 x
    // 32768 tokens of 64 heads, K = 64, V = 128: 930 us instead of 1360; with a quarter of the heads for q and k, K = V = 128: 1507
    // instead of 1526). Else a head's roles do, which read the same tensors (K = V = 128: 1036 us, by role 1059).
    c.by_role = tc && c.nroles > 1 && (p.K != p.V || Hqk != p.H);
    c.phase = 1;
    c.blocks = (int)blocks1;
    c.table = reinterpret_cast<const int*>(table1);
    c.dependent = packed;
    Params phases[2] = {c, c};
    phases[1].phase = 2;
    phases[1].blocks = (int)blocks2;
    phases[1].table = reinterpret_cast<const int*>(table2);
    phases[1].dependent = 1;
    const int n = blocks2 > 0 ? 2 : 1;
    return (tc ? launch_tc(phases, n, s) : launch_simt(phases, n, s)) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
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
        for (int tc = 0; tc < 2; ++tc)   // (which kernels run depends on the output's type too)
            most = std::max(most, layout(*p, Hqk, nseq, packed, tc, current_sm_count(), backward != 0).total);
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
    const Layout l = layout(*p, Hqk, nseq, cu_seqlens != nullptr, tc_supported(c), current_sm_count(), true);
    if (grouped)
        for (int i = 0; i < 2; ++i) {
            c.role[i].out = ws + l.part[i];
            c.role[i].out_bf16 = 0;
        }
    st = run(c, *p, Hqk, true, workspace, s);
    if (st != GDN_OK || !grouped || p->T == 0) return st;
    Groups g{};
    for (int i = 0; i < 2; ++i) g.part[i] = reinterpret_cast<const float*>(ws + l.part[i]);
    g.out[0] = dq;
    g.out[1] = dk;
    g.tokens = cu_seqlens ? reinterpret_cast<const int*>(ws + kWsVerdict) + kTokens : nullptr;
    g.fours = (long long)p->B * p->T * Hqk * p->K / 4;
    g.out_bf16 = in;
    g.H = p->H;
    g.groups = Hqk;
    g.D = p->K;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min<long long>((g.fours + 255) / 256, 8LL * std::max(1, current_sm_count())), 2);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, group_kernel, g) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

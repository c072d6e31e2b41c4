// gdn_linear_recurrent.cu -- the recurrent form of linear attention with a decay for each head over a
// state cache (gdn_linear_recurrent_fwd): every sequence's tokens in order from the state in one cache
// page, fp32 throughout.
//
// Per sequence, head and token, with w = exp(decay[h]):
//   H' = w H + k v^T,   o = q^T H'.
//
// As in gdn_recurrent.cu a warp holds some columns of one head's state, all K rows of them, in registers, and
// every column is independent of the others; here the update needs nothing that the lanes have to exchange, so
// a token is one pass over the state: decayed, updated, and read for the output. Bound by memory: each state is read and
// written once.
#include "gdn_recurrent.cuh"

namespace gdn {
namespace {

// the factor of a head's state; -inf, and what is as good as that, gives 0
__device__ __forceinline__ float head_weight(const RecurrentParams& p, int h) {
    return expf(__ldg(reinterpret_cast<const float*>(p.g) + h));
}

template <int CPL, bool BF>
__device__ __forceinline__ void load_cols(const void* base, long long at, pair_t (&v2)[CPL]) {
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const float v = load1<BF>(base, at + c);
        v2[c] = pack(v, v);
    }
}

// One token a sequence (p.T == 1, no cu_seqlens, states at the end).
template <int K, int CW, int CPL, bool BF>
__global__ void __launch_bounds__(32 * kWarps, 4) linear_decode_kernel(RecurrentParams p) {
    using Cols = Tile<K, CW, CPL>;
    constexpr int NQ = Cols::NQ;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Place at(p, K, CW, warp);
    Cols tile(lane);

    const int slot_in = p.slots_in ? __ldg(p.slots_in + at.s) : -1;
    const int slot_out = p.slots_out ? __ldg(p.slots_out + at.s) : -1;
    Raw4<BF> rk[NQ], rq[NQ];
    const long long kq = ((long long)at.s * p.Hqk + at.hk) * K, sh = (long long)at.s * p.H + at.h;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        rk[i].load(p.k, kq + tile.row(i));
        rq[i].load(p.q, kq + tile.row(i));
    }
    pair_t v2[CPL];
    load_cols<CPL, BF>(p.v, sh * p.V + at.col0 + tile.col(0), v2);
    const float w = head_weight(p, at.h);
    if (slot_in >= 0 && slot_in < p.num_slots)
        tile.load(p.state + slot_in * at.page + at.off, p.V);
    else
        tile.zero();
    bool write;
    if (!admitted(p, at, slot_in, slot_out, lane, write)) return;

    const pair_t w2 = pack(w, w);
    pair_t acc[CPL] = {};
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
        pair_t k2[2], q2[2];
        rk[i].pairs(k2);
        rq[i].pairs(q2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                tile.S[i][j][c] = fma2(k2[j], v2[c], mul2(tile.S[i][j][c], w2));
                acc[c] = fma2(tile.S[i][j][c], q2[j], acc[c]);
            }
    }
    if (write) tile.store(p.state + slot_out * at.page + at.off, p.V);
    const float o = tile.join(acc);
    if (tile.first()) store_o(p, sh * p.V + at.col0 + tile.col(tile.own()), o);
}

// Token by token: kTokens of them staged in shared memory at a time while the next ones load.
template <int K, int CW, int CPL, bool BF>
__global__ void __launch_bounds__(32 * kWarps, CW == 16 ? 4 : 1) linear_tokens_kernel(RecurrentParams p) {
    using Cols = Tile<K, CW, CPL>;
    constexpr int NQ = Cols::NQ, C = kTokens;
    constexpr int KV8 = K / 8;            // threads that stage one token's k and q, eight channels each
    constexpr int COLS = CW * kWarps;
    static_assert(C * KV8 <= 32 * kWarps && C * COLS / 8 <= 32 * kWarps, "one piece a thread");

    __shared__ __align__(16) float ks[2][C][K], qs[2][C][K];
    __shared__ __align__(16) float vs[2][C][COLS];

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
    const float w = head_weight(p, at.h);
    const pair_t w2 = pack(w, w);

    // staging: thread tid brings eight key channels of token st's k and q and eight columns of token vt's v
    const int st = tid / KV8, sk = 8 * (tid % KV8);
    const int vt = tid / (COLS / 8), vc = 8 * (tid % (COLS / 8));
    Raw8<BF> rk, rq, rv;
    auto load_tokens = [&](int t0) {
        if (st < C && t0 + st < n) {
            const long long a = ((long long)(lo + t0 + st) * p.Hqk + at.hk) * K + sk;
            rk.load(p.k, a);
            rq.load(p.q, a);
        }
        if (vt < C && t0 + vt < n)
            rv.load(p.v, ((long long)(lo + t0 + vt) * p.H + at.h) * p.V + (at.col0 - warp * CW) + vc);
    };
    auto store_tokens = [&](int b) {
        float f[8];
        if (st < C) {
            rk.values(f);
            put8(&ks[b][st][sk], f);
            rq.values(f);
            put8(&qs[b][st][sk], f);
        }
        if (vt < C) {
            rv.values(f);
            put8(&vs[b][vt][vc], f);
        }
    };
    rk.zero();
    rq.zero();
    rv.zero();
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
            pair_t v2[CPL], acc[CPL] = {};
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                const float v = vs[b][t][warp * CW + tile.col(c)];
                v2[c] = pack(v, v);
            }
#pragma unroll
            for (int i = 0; i < NQ; ++i) {
                const ulonglong2 k2 = *reinterpret_cast<const ulonglong2*>(&ks[b][t][tile.row(i)]);
                const ulonglong2 q2 = *reinterpret_cast<const ulonglong2*>(&qs[b][t][tile.row(i)]);
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    tile.S[i][0][c] = fma2(k2.x, v2[c], mul2(tile.S[i][0][c], w2));
                    tile.S[i][1][c] = fma2(k2.y, v2[c], mul2(tile.S[i][1][c], w2));
                }
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    acc[c] = fma2(tile.S[i][0][c], q2.x, acc[c]);
                    acc[c] = fma2(tile.S[i][1][c], q2.y, acc[c]);
                }
            }
            const float o = tile.join(acc);
            if (first) store_o(p, oat, o);
            oat += ostep;
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

cudaError_t launch_fn(const void* fn, const RecurrentParams& p, int cols, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)p.nseq * p.H * (p.V / cols)));
    cfg.blockDim = dim3(32 * kWarps);
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

// 16 columns a warp read every token's k and q least often; 8 columns make twice as many warps. us (16 / 8 columns; K = V = 128,
// bf16, by the number of 16-column warps and the tokens a sequence, cold caches):
//   warps     128          512          1024         2048         8192
//   8 tokens  10.2 / 8.2   10.2 / 10.2  12.3 / 14.5  16.4 / 20.5  41.0 / 55.3
//   64        26.6 / 23.6  26.6 / 28.5  36.9 / 47.1  57.3 / 71.7  164 / 236
// (K = V = 64, 256 warps: 10.2 / 8.2 and 20.5 / 22.5.) So 8 only while 16 leave half of the schedulers without a warp. One
// token of each of 256 sequences of 32 heads takes linear_decode_kernel 171 us, 6.3 TB/s; 1 to 8 draft tokens of 48 with the
// state kept after each linear_tokens_kernel 93 us, 6.0 TB/s.
template <int K, bool BF>
cudaError_t launch_k(const RecurrentParams& p, int sms, cudaStream_t s) {
    if (p.T == 1 && !p.cu) return launch_fn((const void*)linear_decode_kernel<K, 16, 4, BF>, p, 16 * kWarps, s);
    const long long warps = (long long)p.nseq * p.H * (p.V / 16);
    if (warps >= 2LL * sms) return launch_fn((const void*)linear_tokens_kernel<K, 16, 4, BF>, p, 16 * kWarps, s);
    return launch_fn((const void*)linear_tokens_kernel<K, 8, 1, BF>, p, 8 * kWarps, s);
}

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" {

gdn_status gdn_linear_recurrent_fwd(const gdn_problem* p, int Hqk, int nseq, const int* cu_seqlens, const void* q,
                                    const void* k, const void* v, const float* decay, float* state,
                                    int num_slots, const int* slots_in, const int* slots_out,
                                    int per_token, void* o, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    gdn_status st = check(p, Hqk, nseq, cu_seqlens, num_slots, per_token);
    if (st != GDN_OK) return st;
    if (p->decay_first || p->gate_k) return GDN_ERR_INVALID_ARG;
    if (!decay || (p->T > 0 && (!q || !k || !v || !o))) return GDN_ERR_INVALID_ARG;
    if ((slots_in || slots_out) && !state && num_slots > 0) return GDN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < gdn_recurrent_workspace_bytes(num_slots)) return GDN_ERR_WORKSPACE;
    for (const void* ptr : {q, k, v, (const void*)state, (const void*)o, (const void*)workspace})
        if (reinterpret_cast<uintptr_t>(ptr) & 15u) return GDN_ERR_MISALIGNED;
    for (const void* ptr : {(const void*)cu_seqlens, (const void*)slots_in, (const void*)slots_out, (const void*)decay})
        if (reinterpret_cast<uintptr_t>(ptr) & 3u) return GDN_ERR_MISALIGNED;
    if ((st = current_device_status()) != GDN_OK) return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    char* ws = reinterpret_cast<char*>(workspace);
    RecurrentParams c{};
    c.q = q;
    c.k = k;
    c.v = v;
    c.g = decay;
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
    c.padded = 1;
    c.per_token = slots_out && (p->T != 1 || cu_seqlens) ? per_token : 0;   // no states to keep, or the final ones
    const int average = cu_seqlens ? p->T / nseq : p->T;
    c.ordered = cu_seqlens && nseq > 1 && nseq <= kOrderSeqs && average >= 12 &&
                (long long)nseq * p->H * (p->V / 64) > 4LL * current_sm_count();
    if ((st = claim(c, *p, average, ws, s)) != GDN_OK) return st;
    const int sms = current_sm_count();
    const bool bf16 = p->in_dtype == GDN_DTYPE_BF16;
    const cudaError_t e = p->K == 64 ? (bf16 ? launch_k<64, true>(c, sms, s) : launch_k<64, false>(c, sms, s))
                                     : (bf16 ? launch_k<128, true>(c, sms, s) : launch_k<128, false>(c, sms, s));
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"

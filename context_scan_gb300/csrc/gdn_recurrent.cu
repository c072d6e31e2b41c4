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
#include "gdn_recurrent.cuh"

namespace gdn {
namespace {

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
    if ((st = claim(c, *p, average, ws, s)) != GDN_OK) return st;
    const bool bf16 = p->in_dtype == GDN_DTYPE_BF16;
    const int sms = current_sm_count();
    if ((p->K == 64 ? launch_k<64>(c, average, p->gate_k, bf16, sms, s)
                    : launch_k<128>(c, average, p->gate_k, bf16, sms, s)) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
}

}  // extern "C"

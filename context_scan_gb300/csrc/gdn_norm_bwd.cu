// gdn_norm_bwd.cu -- gradients of the normalisation (gdn_norm_bwd, entered in gdn_norm.cu).
//
// With xm = x - m (m = 0 for the root-mean-square norm), s = 1 / sqrt(mean(xm^2) + eps) and
// d = dy z sigmoid(z) (dy without a gate), all means over the row:
//   dz = dy (xm s w + b) sigmoid(z) (1 + z (1 - sigmoid(z)))
//   dx = s (d w - mean(d w) - xm s^2 mean(d w xm))   (without mean(d w) for the root-mean-square norm)
//   dw = sum over rows of d xm s,   db = sum over rows of d.
// The statistics are formed again from x, which has to be read anyway, so nothing is kept from the
// forward. A row is read once and stays in registers. The rows' sums dw, db go over a thread's own rows in
// registers, then over the block's groups and the blocks in a fixed order: no atomics, the same
// result every time.
#include <type_traits>

#include "gdn_norm.cuh"

namespace gdn {
namespace norm {
namespace {

// from d = dy: d = dy z sigmoid(z), dyg = dy sigmoid(z) (1 + z (1 - sigmoid(z)))
__device__ __forceinline__ void gate(pair_t& d, pair_t& dyg, pair_t z) {
    float z0, z1;
    unpack(z, z0, z1);
    const pair_t sg = pack(sigmoid(z0), sigmoid(z1)), one = both(1.f);
    const pair_t dsg = mul2(d, sg);
    dyg = mul2(dsg, fma2(z, fma2(sg, both(-1.f), one), one));
    d = mul2(dsg, z);
}

// Eight columns' sums to shared memory, 16 bytes a store where the columns allow. (One by one, eight side by side
// would meet in the same banks: 2 us at 2048 columns. So do the lanes t and t + 4 that put their first fours at the
// same time, so one of them begins with its second.)
template <int L>
__device__ __forceinline__ void put_sums(float* to, int c, int G, int n, const float (&f)[8], int t) {
    if constexpr (L == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = col_of<L>(c, G, e);
            if (has(col, n)) to[col] = f[e];
        }
    } else {
        const int turn = L == 8 ? (t >> 2) & 1 : 0;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const bool second = k != turn;
            const int col = second ? col_of<L>(c, G, 4) : c;
            if (col < n)
                *reinterpret_cast<float4*>(to + col) = second ? make_float4(f[4], f[5], f[6], f[7])
                                                              : make_float4(f[0], f[1], f[2], f[3]);
        }
    }
}

// A block of kMaxThreads threads; GB of them to a row, 0: a part of a warp (rows of at most 512 values)
template <int GB, int R, int L, bool XB, bool YB, bool GATED>
struct Bwd {
    // (With 4, 6, 8, 12 and 20: 29200 rows of 2000 in bf16 68.0, 67.9, 62.4, 63.9 and 67.0 us; 262144 rows of 128 with a gate, x in
    // fp32, 79.6, 79.6, 82.7, 82.7 and 80.5; 467200 rows of 128 in bf16 67.2, 66.2, 66.6, 67.3 and 67.3.)
    static constexpr int kAhead = R == 1 ? 6 : 8;
    using Rows = std::conditional_t<GATED, Ring<L, R, kAhead, XB, YB, YB>, Ring<L, R, kAhead, XB, YB>>;
    // Rows of pairs read w and b from shared memory, where their pairs can be aligned: one copy for each way that rows
    // start (a block of one row at a time meets only one of them): 29200 rows of 1999 103 -> 86 us in bf16, 131 -> 110 in fp32.
    static constexpr int kCopies = GB == kMaxThreads ? 1 : 2;
    static constexpr int kWidth = 8 * R * GB;
    static constexpr int kParams = kCopies * kWidth * (GATED ? 2 : 1) * (int)sizeof(float);
    static constexpr bool kShared = L == 2 && R > 1 && GB > 0 && Rows::bytes(kMaxThreads, GB ? GB : 32) + kParams <= kMost;
    static int smem(int g) {   // (the sums over the groups, at the end, take the place of the stages)
        return std::max(Rows::bytes(kMaxThreads, g) + (kShared ? kParams : 0), kMaxThreads * 8 * R * 2 * (int)sizeof(float));
    }
};

template <int GB, int R, int L, bool XB, bool YB, bool GATED>
__global__ void __launch_bounds__(kMaxThreads) bwd_kernel(Params p) {
    using Plan = Bwd<GB, R, L, XB, YB, GATED>;
    using Rows = typename Plan::Rows;
    extern __shared__ __align__(16) char stages[];
    __shared__ float parts[GB ? kMaxThreads / GB : 1][2][64];
    float(*part)[64] = parts[GB ? threadIdx.x / GB : 0];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int half = 0;
    const int G = GB ? GB : p.g;
    const int t = threadIdx.x % G;
    const int rows_block = kMaxThreads / G;               // rows a block holds at once, and a warp
    const int rows_warp = GB ? 1 : 32 / G;
    const int sub = GB ? 0 : (threadIdx.x & 31) / G;      // which of the warp's is this thread's
    const long long stride = (long long)gridDim.x * rows_block;
    // (the trip count is the same for all threads of a warp, and of a group)
    long long row0 = (long long)blockIdx.x * rows_block + (GB ? threadIdx.x / G : (threadIdx.x >> 5) * rows_warp);

    const int odd = L == 2 ? (int)((row0 + sub) * p.N & 1) : 0;
    const Rows ring{(unsigned)__cvta_generic_to_shared(stages), G, t, (int)threadIdx.x, kMaxThreads, p.N, odd, p.rows};
    auto fetch = [&](int stage, long long row) {
        ring.template fetch<0>(stage, p.x, row);
        ring.template fetch<1>(stage, p.dy, row);
        if constexpr (GATED) ring.template fetch<2>(stage, p.z, row);
        Rows::commit();
    };
#pragma unroll 1
    for (int k = 0; k < Rows::kAhead; ++k) fetch(k, row0 + sub + k * stride);
    pair_t w[4], b[4], dw2[R][4] = {}, db2[R][4] = {};
    if constexpr (R == 1) {
        parameter<L>(w, p.w, first_col<L>(0, t, G, odd), G, p.N, 1.f);
        if constexpr (GATED) parameter<L>(b, p.b, first_col<L>(0, t, G, odd), G, p.N, 0.f);
    }
    float* shared_w = nullptr;   // as this group's rows start
    if constexpr (Plan::kShared) {
        constexpr int W = Plan::kWidth, COPIES = Plan::kCopies;
        float* all = reinterpret_cast<float*>(stages + Rows::bytes(kMaxThreads, GB));
#pragma unroll
        for (int q = 0; q < COPIES; ++q)
            for (int j = threadIdx.x; j < W; j += kMaxThreads) {
                const int col = j - (COPIES == 1 ? odd : q);
                all[q * W + j] = !has(col, p.N) ? 0.f : p.w ? __ldg(p.w + col) : 1.f;
                if constexpr (GATED) all[(COPIES + q) * W + j] = has(col, p.N) && p.b ? __ldg(p.b + col) : 0.f;
            }
        shared_w = all + (COPIES == 1 ? 0 : odd * W);
        __syncthreads();
    }
    // the i-th eight columns' w (which = 0) or b
    auto parameters = [&](pair_t (&f)[4], int which, int i) {
        const int c = first_col<L>(i, t, G, odd);
        if constexpr (Plan::kShared) {
            const float* from = shared_w + which * Plan::kCopies * Plan::kWidth + c + odd;
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = *reinterpret_cast<const pair_t*>(from + 2 * k * G);
        } else {
            parameter<L>(f, which ? p.b : p.w, c, G, p.N, which ? 0.f : 1.f);
        }
    };
    for (int stage = 0; row0 < p.rows; row0 += stride, stage = stage == Rows::kAhead ? 0 : stage + 1) {
        const long long row = row0 + sub;
        Rows::template wait<GB, kMaxThreads>();
        fetch(stage == 0 ? Rows::kAhead : stage - 1, row + Rows::kAhead * stride);
        // d w is formed twice rather than kept where w is at hand for the second time, and registers are short: 29200 gated
        // rows in bf16, 1999 values 160 -> 130 us, 2000 138 -> 114; 1999 of x in fp32 193 -> 156.
        constexpr bool kAgain = Plan::kShared || (R > 1 && GATED);
        pair_t x[R][4], d[R][4], dxh[R][4], dyg[R][4];
        pair_t xx = 0, dx_ = 0, ds = 0, xs = 0;   // sums of x^2, d w x, d w, x
#pragma unroll
        for (int i = 0; i < R; ++i) {
            ring.template read<0>(stage, i, row, x[i]);
            ring.template read<1>(stage, i, row, d[i]);
            if constexpr (GATED) {
                pair_t z[4];
                ring.template read<2>(stage, i, row, z);
#pragma unroll
                for (int k = 0; k < 4; ++k) gate(d[i][k], dyg[i][k], z[k]);
            }
            if constexpr (R > 1) parameters(w, 0, i);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                dxh[i][k] = mul2(d[i][k], w[k]);
                xx = fma2(x[i][k], x[i][k], xx);
                dx_ = fma2(dxh[i][k], x[i][k], dx_);
                ds = add2(ds, dxh[i][k]);
                xs = add2(xs, x[i][k]);
            }
        }
        float mean = 0.f, mean_d = 0.f, var, cross;   // mean: of what x holds; cross: mean(d w xm)
        if (p.rms) {
            float q[2] = {total(xx), total(dx_)};
            group_sum<GB, kMaxThreads>(q, G, part, half);
            var = q[0] * p.inv_n;
            cross = q[1] * p.inv_n;
        } else {
            float s[4] = {total(xx), total(dx_), total(ds), total(xs)};
            group_sum<GB, kMaxThreads>(s, G, part, half);
            mean = s[3] * p.inv_n;
            mean_d = s[2] * p.inv_n;
            var = fmaf(-mean, mean, s[0] * p.inv_n);
            cross = fmaf(-mean, mean_d, s[1] * p.inv_n);
            const bool again = large_mean(mean, var);
            if (GB ? again : __any_sync(0xffffffffu, again)) {   // (a warp's other rows stay as they are)
                const float off = GB || again ? mean : 0.f;
                float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    float v[8], f[8];
                    single(x[i], v);
                    if constexpr (kAgain) {
                        parameters(w, 0, i);
#pragma unroll
                        for (int k = 0; k < 4; ++k) dxh[i][k] = mul2(d[i][k], w[k]);
                    }
                    single(dxh[i], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        v[e] = has(col_of<L>(first_col<L>(i, t, G, odd), G, e), p.N) ? v[e] - off : 0.f;
                        q[0] = fmaf(v[e], v[e], q[0]);
                        q[1] = fmaf(f[e], v[e], q[1]);
                        q[2] += v[e];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[i][k] = pack(v[2 * k], v[2 * k + 1]);
                }
                group_sum<GB, kMaxThreads>(q, G, part, half);
                if (GB || again) {
                    mean = q[2] * p.inv_n;
                    var = centred_var(q[0] * p.inv_n, mean);
                    cross = fmaf(-mean, mean_d, q[1] * p.inv_n);
                }
            }
        }
        // (0 for rows behind the last one, whose sums then add nothing even with eps = 0)
        const float rstd = row < p.rows ? rsqrtf(var + p.eps) : 0.f;
        // with xh = xm s: dx = s d w - s mean(d w) - xh s^2 mean(d w xm)
        const pair_t scale = both(rstd), level = both(-mean * rstd), along = both(-rstd * rstd * cross),
                     level_d = both(-rstd * mean_d);
        const int n = GB || row < p.rows ? p.N : 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = first_col<L>(i, t, G, odd);
            if constexpr (kAgain) parameters(w, 0, i);
            if constexpr (R > 1 && GATED) parameters(b, 1, i);
            float out[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const pair_t xh = fma2(x[i][k], scale, level);
                const pair_t dw_ = kAgain ? mul2(d[i][k], w[k]) : dxh[i][k];
                if constexpr (GATED) dyg[i][k] = mul2(dyg[i][k], fma2(xh, w[k], b[k]));
                dw2[i][k] = fma2(d[i][k], xh, dw2[i][k]);
                db2[i][k] = add2(db2[i][k], d[i][k]);
                x[i][k] = fma2(xh, along, fma2(dw_, scale, level_d));
            }
            single(x[i], out);
            store8<XB, L>(p.y, row * p.N, c, G, n, out);
            if constexpr (GATED)
                if (p.dz) {
                    single(dyg[i], out);
                    store8<YB, L>(p.dz, row * p.N, c, G, n, out);
                }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!p.partial) return;
    // dw, db over the rows of the block's groups, through shared memory (the stages, which are not needed any more)
    const int width = 8 * R * G, set = threadIdx.x / G;
    float* sum = reinterpret_cast<float*>(stages);   // [groups][2][width]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int c = first_col<L>(i, t, G, odd);
        float dw[8], db[8];
        single(dw2[i], dw);
        single(db2[i], db);
        put_sums<L>(sum + 2 * set * width, c, G, p.N, dw, t);
        put_sums<L>(sum + (2 * set + 1) * width, c, G, p.N, db, t);
    }
    __syncthreads();
    float* out = p.partial + (long long)blockIdx.x * 2 * p.N;
    for (int i = threadIdx.x; i < 2 * p.N; i += kMaxThreads) {
        const int which = i >= p.N, col = which ? i - p.N : i;
        float a = 0.f;
#pragma unroll 4
        for (int k = 0; k < rows_block; ++k) a += sum[(2 * k + which) * width + col];
        out[i] = a;
    }
}

// dw and db from the blocks' sums: 32 columns a block, 32 threads to a column.
__global__ void __launch_bounds__(1024) columns_kernel(const float* partial, int blocks, int N, float* dw, float* db) {
    __shared__ float sum[32][33];
    const int lane = threadIdx.x & 31, k = threadIdx.x >> 5;
    float* out = blockIdx.y ? db : dw;
    const int c = blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!out) return;
    float a = 0.f;
    if (c < N) {
        const float* from = partial + (long long)blockIdx.y * N + c;
        int i = k;
        for (; i + 7 * 32 < blocks; i += 8 * 32) {   // eight loads on their way
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __ldcg(from + (long long)(i + 32 * j) * 2 * N);
#pragma unroll
            for (int j = 0; j < 8; ++j) a += v[j];
        }
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = i + 32 * j < blocks ? __ldcg(from + (long long)(i + 32 * j) * 2 * N) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) a += v[j];
    }
    sum[k][lane] = a;
    __syncthreads();
    a = sum[lane][k];   // thread (lane, k): the lane-th part of column k
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    const int col = blockIdx.x * 32 + k;
    if (lane == 0 && col < N) out[col] = a;
}

template <int GB, int R, int L, bool XB, bool YB, bool GATED>
cudaError_t bwd(const Params& p, const Shape& s, int blocks, cudaStream_t st) {
    using Rows = typename Bwd<GB, R, L, XB, YB, GATED>::Rows;
    static std::atomic<int> known[kDevices];
    const auto kernel = bwd_kernel<GB, R, L, XB, YB, GATED>;
    const int smem = Bwd<GB, R, L, XB, YB, GATED>::smem(s.g);
    if (resident_blocks(kernel, kMaxThreads, smem, known) < 1) return cudaErrorLaunchOutOfResources;
    kernel<<<blocks, kMaxThreads, smem, st>>>(p);
    return cudaGetLastError();
}
template <int GB, int R, int L>
cudaError_t bwd_types(const Params& p, const Shape& s, bool xb, bool yb, int blocks, cudaStream_t st) {
    if (xb && yb)
        return p.z ? bwd<GB, R, L, true, true, true>(p, s, blocks, st) : bwd<GB, R, L, true, true, false>(p, s, blocks, st);
    if constexpr (L < 8) {
        if (xb)
            return p.z ? bwd<GB, R, L, true, false, true>(p, s, blocks, st)
                       : bwd<GB, R, L, true, false, false>(p, s, blocks, st);
        if (yb)
            return p.z ? bwd<GB, R, L, false, true, true>(p, s, blocks, st)
                       : bwd<GB, R, L, false, true, false>(p, s, blocks, st);
        return p.z ? bwd<GB, R, L, false, false, true>(p, s, blocks, st)
                   : bwd<GB, R, L, false, false, false>(p, s, blocks, st);
    }
    return cudaErrorInvalidValue;
}
template <int GB, int R>
cudaError_t bwd_layout(const Params& p, const Shape& s, bool xb, bool yb, int blocks, cudaStream_t st) {
    if (p.N % 8 == 0 && xb && yb) return bwd_types<GB, R, 8>(p, s, xb, yb, blocks, st);
    return p.N % 4 == 0 ? bwd_types<GB, R, 4>(p, s, xb, yb, blocks, st) : bwd_types<GB, R, 2>(p, s, xb, yb, blocks, st);
}

}  // namespace

cudaError_t launch_bwd(const Params& p_in, const Shape& s, bool xb, bool yb, int sms, float* dw, float* db,
                       cudaStream_t st) {
    Params p = p_in;
    if (!dw && !db) p.partial = nullptr;
    const int blocks = (int)bwd_blocks(p.rows, s, sms);
    if (blocks > 0) {
        const cudaError_t e = s.g <= 32    ? (s.r == 1 ? bwd_layout<0, 1>(p, s, xb, yb, blocks, st)
                                                       : bwd_layout<0, 2>(p, s, xb, yb, blocks, st))
                              : s.g == 64  ? bwd_layout<64, 2>(p, s, xb, yb, blocks, st)
                              : s.g == 128 ? bwd_layout<128, 2>(p, s, xb, yb, blocks, st)
                              : s.g == 256 ? bwd_layout<256, 2>(p, s, xb, yb, blocks, st)
                                           : bwd_layout<512, 2>(p, s, xb, yb, blocks, st);
        if (e != cudaSuccess) return e;
    }
    if (!p.partial) return cudaSuccess;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.N + 31) / 32), 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 0 ? 1 : 0;   // the dependent of the rows' launch
    return cudaLaunchKernelEx(&cfg, columns_kernel, (const float*)p.partial, blocks, p.N, dw, db);
}

}  // namespace norm
}  // namespace gdn

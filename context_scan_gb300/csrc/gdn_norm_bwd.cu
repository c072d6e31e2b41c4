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
#include "gdn_norm.cuh"

namespace gdn {
namespace norm {
namespace {

// d, and for the gate dyg = dy sigmoid(z) (1 + z (1 - sigmoid(z))), from dy (in d) and z
__device__ __forceinline__ void gate(float (&d)[8], float (&dyg)[8], const float (&z)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float sg = sigmoid(z[e]);
        dyg[e] = d[e] * sg * fmaf(z[e], 1.f - sg, 1.f);
        d[e] *= z[e] * sg;
    }
}

template <bool BLOCK, bool VEC, bool XB, bool YB, bool GATED>
__global__ void __launch_bounds__(BLOCK ? kMaxThreads : 256) bwd_kernel(Params p) {
    __shared__ float part[2][3][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int half = 0;
    const int G = BLOCK ? blockDim.x : p.g;
    const int t = threadIdx.x % G;
    const int per_warp = BLOCK ? 1 : 32 / G;              // rows a warp holds at once
    const int sub = BLOCK ? 0 : (threadIdx.x & 31) / G;   // which of them is this thread's
    const int c = first_col<VEC>(0, t, G), step = col_step<VEC>(G);
    const long long stride = (long long)gridDim.x * (blockDim.x / G);
    long long row0 = (long long)blockIdx.x * (blockDim.x / G) + (BLOCK ? 0 : (threadIdx.x >> 5) * per_warp);

    float w[8], b[8], dw[8], db[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int col = c + e * step;
        w[e] = p.w && col < p.N ? __ldg(p.w + col) : 1.f;
        if constexpr (GATED) b[e] = p.b && col < p.N ? __ldg(p.b + col) : 0.f;
        dw[e] = db[e] = 0.f;
    }
    Eight<XB, VEC> nx;
    Eight<YB, VEC> nz, nd;
    auto fetch = [&](long long row) {
        const int n = row < p.rows ? p.N : 0;
        nx.load(p.x, row * p.N, c, step, n);
        nd.load(p.dy, row * p.N, c, step, n);
        if constexpr (GATED) nz.load(p.z, row * p.N, c, step, n);
    };
    fetch(row0 + sub);
    for (; row0 < p.rows; row0 += stride) {
        const long long row = row0 + sub;
        float x[8], d[8], dyg[8];
        nx.values(x);
        nd.values(d);
        if constexpr (GATED) {
            float z[8];
            nz.values(z);
            gate(d, dyg, z);
        }
        fetch(row + stride);
        if (!p.rms) {
            float s[1] = {0.f};
#pragma unroll
            for (int e = 0; e < 8; ++e) s[0] += x[e];
            group_sum<BLOCK>(s, G, part, half);
            const float mean = s[0] * p.inv_n;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = c + e * step < p.N ? x[e] - mean : 0.f;
        }
        float s[3] = {0.f, 0.f, 0.f};   // of xm^2, d w xm, d w
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float dxh = d[e] * w[e];
            s[0] = fmaf(x[e], x[e], s[0]);
            s[1] = fmaf(dxh, x[e], s[1]);
            s[2] += dxh;
        }
        group_sum<BLOCK>(s, G, part, half);
        const float rstd = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
        const float along = rstd * rstd * s[1] * p.inv_n;
        const float mean_d = p.rms ? 0.f : s[2] * p.inv_n;
        const int n = row < p.rows ? p.N : 0;
        float dx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float xh = x[e] * rstd;
            dx[e] = rstd * (fmaf(d[e], w[e], -mean_d) - x[e] * along);
            if constexpr (GATED) dyg[e] *= fmaf(xh, w[e], b[e]);
            if (row < p.rows) {   // (with eps = 0 the rows behind the last one are not finite)
                dw[e] = fmaf(d[e], xh, dw[e]);
                db[e] += d[e];
            }
        }
        Eight<XB, VEC>::store(p.y, row * p.N, c, step, n, dx);
        if constexpr (GATED)
            if (p.dz) Eight<YB, VEC>::store(p.dz, row * p.N, c, step, n, dyg);
    }
    if (!p.partial) return;
    float* out = p.partial + (long long)blockIdx.x * 2 * p.N;
    if constexpr (BLOCK) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = c + e * step;
            if (col < p.N) {
                out[col] = dw[e];
                out[p.N + col] = db[e];
            }
        }
    } else {
        // over a warp's rows by exchange, over the block's eight warps through shared memory
        __shared__ float sum[8][2][256];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            for (int off = 16; off >= G; off >>= 1) {
                dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], off);
                db[e] += __shfl_xor_sync(0xffffffffu, db[e], off);
            }
            if (sub == 0) {
                sum[threadIdx.x >> 5][0][c + e * step] = dw[e];
                sum[threadIdx.x >> 5][1][c + e * step] = db[e];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * p.N; i += blockDim.x) {
            const int which = i >= p.N, col = which ? i - p.N : i;
            float a = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) a += sum[k][which][col];
            out[i] = a;
        }
    }
}

// Rows of more than 4096 values, one a block: what is loaded stays in registers as stored and is worked out
// again after the sums; the weights come from the cache, and a thread's sums of dw and db stand in
// shared memory, each column with the one thread that has it in every row.
template <int R, bool VEC, bool XB, bool YB, bool GATED>
__global__ void __launch_bounds__(kMaxThreads) wide_bwd_kernel(Params p) {
    extern __shared__ float acc[];   // dw [N], db [N]
    __shared__ float part[2][3][32];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int half = 0;
    const int G = kMaxThreads, t = threadIdx.x, step = col_step<VEC>(G);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = first_col<VEC>(i, t, G) + e * step;
            if (p.partial && col < p.N) acc[col] = acc[p.N + col] = 0.f;
        }
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        Eight<XB, VEC> rx[R];
        Eight<YB, VEC> rz[R], rd[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = first_col<VEC>(i, t, G);
            rx[i].load(p.x, row * p.N, c, step, p.N);
            rd[i].load(p.dy, row * p.N, c, step, p.N);
            if constexpr (GATED) rz[i].load(p.z, row * p.N, c, step, p.N);
        }
        float mean = 0.f;
        if (!p.rms) {
            float s[1] = {0.f};
#pragma unroll
            for (int i = 0; i < R; ++i) {
                float x[8];
                rx[i].values(x);
#pragma unroll
                for (int e = 0; e < 8; ++e) s[0] += x[e];
            }
            group_sum<true>(s, G, part, half);
            mean = s[0] * p.inv_n;
        }
        auto terms = [&](int i, float (&x)[8], float (&d)[8], float (&dyg)[8]) {
            rx[i].values(x);
            rd[i].values(d);
            if constexpr (GATED) {
                float z[8];
                rz[i].values(z);
                gate(d, dyg, z);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = first_col<VEC>(i, t, G) + e * step < p.N ? x[e] - mean : 0.f;
        };
        auto weight = [&](const float* a, int col, float none) {
            return a && col < p.N ? __ldg(a + col) : none;
        };
        float s[3] = {0.f, 0.f, 0.f};   // of xm^2, d w xm, d w
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float x[8], d[8], dyg[8];
            terms(i, x, d, dyg);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float dxh = d[e] * weight(p.w, first_col<VEC>(i, t, G) + e * step, 1.f);
                s[0] = fmaf(x[e], x[e], s[0]);
                s[1] = fmaf(dxh, x[e], s[1]);
                s[2] += dxh;
            }
        }
        group_sum<true>(s, G, part, half);
        const float rstd = rsqrtf(fmaf(s[0], p.inv_n, p.eps));
        const float along = rstd * rstd * s[1] * p.inv_n;
        const float mean_d = p.rms ? 0.f : s[2] * p.inv_n;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int c = first_col<VEC>(i, t, G);
            float x[8], d[8], dyg[8];
            terms(i, x, d, dyg);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int col = c + e * step;
                const float w = weight(p.w, col, 1.f), xh = x[e] * rstd;
                if (p.partial && col < p.N) {
                    acc[col] = fmaf(d[e], xh, acc[col]);
                    acc[p.N + col] += d[e];
                }
                if constexpr (GATED) dyg[e] *= fmaf(xh, w, weight(p.b, col, 0.f));
                x[e] = rstd * (fmaf(d[e], w, -mean_d) - x[e] * along);
            }
            Eight<XB, VEC>::store(p.y, row * p.N, c, step, p.N, x);
            if constexpr (GATED)
                if (p.dz) Eight<YB, VEC>::store(p.dz, row * p.N, c, step, p.N, dyg);
        }
    }
    if (!p.partial) return;
    float* out = p.partial + (long long)blockIdx.x * 2 * p.N;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int col = first_col<VEC>(i, t, G) + e * step;
            if (col < p.N) {
                out[col] = acc[col];
                out[p.N + col] = acc[p.N + col];
            }
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
    if (c < N)
        for (int i = k; i < blocks; i += 32) a += __ldcg(partial + ((long long)i * 2 + blockIdx.y) * N + c);
    sum[k][lane] = a;
    __syncthreads();
    a = sum[lane][k];   // thread (lane, k): the lane-th part of column k
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a += __shfl_xor_sync(0xffffffffu, a, off);
    const int col = blockIdx.x * 32 + k;
    if (lane == 0 && col < N) out[col] = a;
}

template <int R, bool BLOCK, bool VEC, bool XB, bool YB, bool GATED>
cudaError_t bwd(const Params& p, const Shape& s, int blocks, cudaStream_t st) {
    if constexpr (R == 1) {
        bwd_kernel<BLOCK, VEC, XB, YB, GATED><<<blocks, s.threads, 0, st>>>(p);
    } else {
        const int smem = p.partial ? 2 * p.N * (int)sizeof(float) : 0;
        const cudaError_t e = cudaFuncSetAttribute(wide_bwd_kernel<R, VEC, XB, YB, GATED>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        wide_bwd_kernel<R, VEC, XB, YB, GATED><<<blocks, s.threads, smem, st>>>(p);
    }
    return cudaGetLastError();
}
template <int R, bool BLOCK, bool VEC, bool XB, bool YB>
cudaError_t bwd_gated(const Params& p, const Shape& s, int blocks, cudaStream_t st) {
    return p.z ? bwd<R, BLOCK, VEC, XB, YB, true>(p, s, blocks, st)
               : bwd<R, BLOCK, VEC, XB, YB, false>(p, s, blocks, st);
}
template <int R, bool BLOCK, bool VEC>
cudaError_t bwd_types(const Params& p, const Shape& s, bool xb, bool yb, int blocks, cudaStream_t st) {
    if (xb)
        return yb ? bwd_gated<R, BLOCK, VEC, true, true>(p, s, blocks, st)
                  : bwd_gated<R, BLOCK, VEC, true, false>(p, s, blocks, st);
    return yb ? bwd_gated<R, BLOCK, VEC, false, true>(p, s, blocks, st)
              : bwd_gated<R, BLOCK, VEC, false, false>(p, s, blocks, st);
}
template <int R, bool BLOCK>
cudaError_t bwd_vec(const Params& p, const Shape& s, bool xb, bool yb, int blocks, cudaStream_t st) {
    return s.vec ? bwd_types<R, BLOCK, true>(p, s, xb, yb, blocks, st)
                 : bwd_types<R, BLOCK, false>(p, s, xb, yb, blocks, st);
}

}  // namespace

cudaError_t launch_bwd(const Params& p_in, const Shape& s, bool xb, bool yb, long long nblocks, float* dw,
                       float* db, cudaStream_t st) {
    Params p = p_in;
    if (!dw && !db) p.partial = nullptr;
    const int blocks = (int)nblocks;
    if (blocks > 0) {
        const cudaError_t e = !s.block ? bwd_vec<1, false>(p, s, xb, yb, blocks, st)
                              : s.r == 1 ? bwd_vec<1, true>(p, s, xb, yb, blocks, st)
                                         : bwd_vec<2, true>(p, s, xb, yb, blocks, st);
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

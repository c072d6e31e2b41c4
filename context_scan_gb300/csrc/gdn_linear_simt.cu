// gdn_linear_simt.cu -- linear attention with a decay for each head on the fp32 CUDA cores: any of the types, fp32
// arithmetic throughout. For fp32 tensors (which the tensor cores would have to take in several parts each) and for
// batches whose inputs and outputs differ in type.
//
// A block of 256 threads owns one piece of one sequence, one head and 64 columns of the state, and walks over steps of 32
// tokens: A, B, C tiles and the state X in shared memory as fp32; P = (A B^T) with the weights; out = P C + w^.. A X;
// X' = w^n X + B^T C. A thread keeps 8 x 4 (dA = 128) values of the state in registers and the next step's tokens
// on their way. C lies there once more with the weights of the update (8.2 -> 7.8 ms for the case below). Full of blocks it is bound
// by the fp32 pipe and shared memory's reads beside it (1.4 of 4.5 cycles an instruction waits for them): 2 x 32768 fp32 tokens of 32
// heads, K = V = 128, take 7.8 ms, bf16 ones with fp32 outputs 9.3, 20 times what the tensor cores do. With few
// blocks the steps are a chain: 5 sequences of 130 fp32 tokens, 2 heads, K = V = 64: 28.6 us, five steps of 5 us.
#include "gdn_linear.cuh"
#include "gdn_pair.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kS = 32;        // tokens of a step
constexpr int kTile = 64;     // columns of a block
constexpr int kThreads = 256;

__device__ __forceinline__ void load4(const void* base, bool bf16, long long at, float (&f)[4]) {
    if (bf16) {
        const uint2 t = __ldg(reinterpret_cast<const uint2*>((const char*)base + 2 * at));
        f[0] = __uint_as_float(t.x << 16);
        f[1] = __uint_as_float(t.x & 0xffff0000u);
        f[2] = __uint_as_float(t.y << 16);
        f[3] = __uint_as_float(t.y & 0xffff0000u);
    } else {
        const float4 t = __ldg(reinterpret_cast<const float4*>((const char*)base + 4 * at));
        f[0] = t.x, f[1] = t.y, f[2] = t.z, f[3] = t.w;
    }
}

__device__ __forceinline__ float total(pair_t x) {
    float lo, hi;
    unpack(x, lo, hi);
    return lo + hi;
}

template <int DA>
struct Smem {
    float A[kS][DA + 4];
    float B[kS][DA + 4];
    float C[kS][kTile], W[kS][kTile];   // W: C with the weights of the update
    float P[kS][kS + 4];
    // rows in pairs, for the two-wide fp32 instructions; of every four columns the first two lie in the first half (16 bytes
    // a lane, a warp's side by side)
    pair_t X[DA / 2][kTile];
    float weight[kS + 2];   // w^0 .. w^32 and beyond
};

template <int DA>
__device__ __forceinline__ void walk(const Params& p, const Role& r, const Item& it, int first, int rest, int tile, Smem<DA>& sm) {
    const int tid = threadIdx.x, h = it.h;
    const bool sums = p.phase == 1 && it.piece > 0;
    const float lg = log2_weight(p.decay, h);
    const int col0 = tile * kTile;
    if (tid <= kS + 1) sm.weight[tid] = exp2f(lg * tid);

    // the state: rows 8 tr .. (DA / 16 of them), columns 4 tc .. of this tile
    constexpr int RT = DA / 16;
    const int tc = tid % 16, tr = tid / 16;
    pair_t X[RT / 2][4];   // rows in pairs
#pragma unroll
    for (int i = 0; i < RT / 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) X[i][c] = 0;
    const long long state = (long long)DA * r.dC;
    auto place = [&](int i, int c) {   // in a state as the caller stores it
        const long long row = RT * tr + i, col = col0 + 4 * tc + c;
        return r.state_t ? col * DA + row : row * r.dC + col;
    };
    auto slot = [&](int q) { return p.slots + (it.slot + (long long)(q - 1) * it.slot_step) * state; };
    auto slot_at = [&](int i) { return (long long)(RT * tr + i) * r.dC + col0 + 4 * tc; };
    if (it.piece == 0) {
        if (r.start) {
            const float* from = r.start + ((long long)it.seq * p.H + h) * state;
#pragma unroll
            for (int i = 0; i < RT; i += 2)
#pragma unroll
                for (int c = 0; c < 4; ++c) X[i / 2][c] = pack(__ldg(from + place(i, c)), __ldg(from + place(i + 1, c)));
        }
    } else if (!sums) {
        for (int q = 1; q <= it.piece; ++q) {
            // entering piece q: from the state entering piece q - 1 and that piece's sum
            const float keep = q == 1 ? 0.f
                : exp2f(lg * tokens_of(first + (q - 2) * rest, first + (q - 1) * rest, it.len, r.rev));
            const float* from = slot(q);
            const pair_t keep2 = pack(keep, keep);
#pragma unroll
            for (int i = 0; i < RT; i += 2) {
                const float4 u = __ldcg(reinterpret_cast<const float4*>(from + slot_at(i)));
                const float4 v = __ldcg(reinterpret_cast<const float4*>(from + slot_at(i + 1)));
                const pair_t t[4] = {pack(u.x, v.x), pack(u.y, v.y), pack(u.z, v.z), pack(u.w, v.w)};
#pragma unroll
                for (int c = 0; c < 4; ++c) X[i / 2][c] = q == 1 ? t[c] : fma2(keep2, X[i / 2][c], t[c]);
            }
        }
    }
    const int ah = h / (p.H / r.a_heads), bh = h / (p.H / r.b_heads), ch = h / (p.H / r.c_heads);
    const int n = (it.len + kChunk - 1) / kChunk;
    const int t0 = kChunk * (r.rev ? n - it.m1 : it.m0);               // the piece's tokens, in memory order
    const int t1 = min(it.len, kChunk * (r.rev ? n - it.m0 : it.m1));
    const int steps = (t1 - t0 + kS - 1) / kS;

    // staging: the step's tokens as fours of values
    constexpr int AF = kS * DA / 4 / kThreads, CF = kS * kTile / 4 / kThreads;
    float fa[AF][4], fb[AF][4], fc[CF][4];
    auto fetch = [&](int st) {
        const int base = t0 + kS * st, m = min(kS, t1 - base);
#pragma unroll
        for (int i = 0; i < AF; ++i) {
            const int at = tid + i * kThreads, row = at / (DA / 4), c = 4 * (at % (DA / 4));
#pragma unroll
            for (int x = 0; x < 4; ++x) fa[i][x] = fb[i][x] = 0.f;
            if (row < m) {
                const long long tok = it.lo + base + row;
                load4(r.b, r.b_bf16, (tok * r.b_heads + bh) * DA + c, fb[i]);
                if (!sums) load4(r.a, r.a_bf16, (tok * r.a_heads + ah) * DA + c, fa[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < CF; ++i) {
            const int at = tid + i * kThreads, row = at / (kTile / 4), c = 4 * (at % (kTile / 4));
#pragma unroll
            for (int x = 0; x < 4; ++x) fc[i][x] = 0.f;
            if (row < m) load4(r.c, r.c_bf16, ((long long)(it.lo + base + row) * r.c_heads + ch) * r.dC + col0 + c, fc[i]);
        }
    };
    if (steps > 0) fetch(r.rev ? steps - 1 : 0);
    for (int i = 0; i < steps; ++i) {
        const int st = r.rev ? steps - 1 - i : i;
        const int base = t0 + kS * st, L = min(kS, t1 - base);
        __syncthreads();   // (the step before has read its tiles)
#pragma unroll
        for (int j = 0; j < AF; ++j) {
            const int at = tid + j * kThreads, row = at / (DA / 4), c = 4 * (at % (DA / 4));
            *reinterpret_cast<float4*>(&sm.A[row][c]) = make_float4(fa[j][0], fa[j][1], fa[j][2], fa[j][3]);
            *reinterpret_cast<float4*>(&sm.B[row][c]) = make_float4(fb[j][0], fb[j][1], fb[j][2], fb[j][3]);
        }
#pragma unroll
        for (int j = 0; j < CF; ++j) {
            const int at = tid + j * kThreads, row = at / (kTile / 4), c = 4 * (at % (kTile / 4));
            *reinterpret_cast<float4*>(&sm.C[row][c]) = make_float4(fc[j][0], fc[j][1], fc[j][2], fc[j][3]);
            const float wj = row < L ? sm.weight[r.rev ? row + 1 : L - 1 - row] : 0.f;
            *reinterpret_cast<float4*>(&sm.W[row][c]) = make_float4(fc[j][0] * wj, fc[j][1] * wj, fc[j][2] * wj, fc[j][3] * wj);
        }
#pragma unroll
        for (int j = 0; j < RT / 2; ++j)
#pragma unroll
            for (int c = 0; c < 4; c += 2)
                *reinterpret_cast<ulonglong2*>(&sm.X[RT / 2 * tr + j][kTile / 4 * c + 2 * tc]) = make_ulonglong2(X[j][c], X[j][c + 1]);
        __syncthreads();
        if (i + 1 < steps) fetch(r.rev ? steps - 2 - i : i + 1);
        if (!sums) {
            // P: rows pr, pr + 16, columns pc, pc + 16
            const int pr = tid / 16, pc = tid % 16;
            pair_t d2[2][2] = {};
#pragma unroll 4
            for (int k = 0; k < DA; k += 4) {
                ulonglong2 x[2], y[2];
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    x[z] = *reinterpret_cast<const ulonglong2*>(&sm.A[pr + 16 * z][k]);
                    y[z] = *reinterpret_cast<const ulonglong2*>(&sm.B[pc + 16 * z][k]);
                }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int v = 0; v < 2; ++v) d2[u][v] = fma2(x[u].y, y[v].y, fma2(x[u].x, y[v].x, d2[u][v]));
            }
            float d[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int v = 0; v < 2; ++v) d[u][v] = total(d2[u][v]);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int row = pr + 16 * u, col = pc + 16 * v, gap = r.rev ? col - row : row - col;
                    sm.P[row][col] = gap >= 0 ? d[u][v] * sm.weight[gap] : 0.f;
                }
            __syncthreads();
            // out: rows orow, orow + 16, columns 4 tc ..
            const int orow = tid / 16;
            float intra[2][4] = {}, inter[2][4];
            pair_t sums2[2][4] = {};
#pragma unroll 2
            for (int k = 0; k < DA; k += 4) {
                const ulonglong2 x0 = *reinterpret_cast<const ulonglong2*>(&sm.A[orow][k]);
                const ulonglong2 x1 = *reinterpret_cast<const ulonglong2*>(&sm.A[orow + 16][k]);
#pragma unroll
                for (int z = 0; z < 2; ++z)
#pragma unroll
                    for (int c = 0; c < 4; c += 2) {
                        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&sm.X[k / 2 + z][kTile / 4 * c + 2 * tc]);
                        sums2[0][c] = fma2(z ? x0.y : x0.x, y.x, sums2[0][c]);
                        sums2[1][c] = fma2(z ? x1.y : x1.x, y.x, sums2[1][c]);
                        sums2[0][c + 1] = fma2(z ? x0.y : x0.x, y.y, sums2[0][c + 1]);
                        sums2[1][c + 1] = fma2(z ? x1.y : x1.x, y.y, sums2[1][c + 1]);
                    }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < 4; ++c) inter[u][c] = total(sums2[u][c]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int row = orow + 16 * u;
                // (the tokens that this row sees: a later one's infinity must not reach it as 0 times infinity)
                const int j0 = r.rev ? row : 0, j1 = r.rev ? L : min(row + 1, L);
#pragma unroll 4
                for (int j = j0; j < j1; ++j) {
                    const float x = sm.P[row][j];
                    const float4 y = *reinterpret_cast<const float4*>(&sm.C[j][4 * tc]);
                    intra[u][0] = fmaf(x, y.x, intra[u][0]);
                    intra[u][1] = fmaf(x, y.y, intra[u][1]);
                    intra[u][2] = fmaf(x, y.z, intra[u][2]);
                    intra[u][3] = fmaf(x, y.w, intra[u][3]);
                }
                if (row < L) {
                    const float keep = sm.weight[r.rev ? L - 1 - row : row + 1];
                    float f[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) f[c] = fmaf(keep, inter[u][c], intra[u][c]);
                    const long long at = ((long long)(it.lo + base + row) * p.H + h) * r.dC + col0 + 4 * tc;
                    if (r.out_bf16) {
                        const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
                        uint2 t;
                        t.x = *reinterpret_cast<const unsigned*>(&lo);
                        t.y = *reinterpret_cast<const unsigned*>(&hi);
                        *reinterpret_cast<uint2*>((char*)r.out + 2 * at) = t;
                    } else {
                        *reinterpret_cast<float4*>((char*)r.out + 4 * at) = make_float4(f[0], f[1], f[2], f[3]);
                    }
                }
            }
        }
        // X' = w^L X + sum_j w^(L - 1 - j + s) b_j c_j^T (j in the role's direction)
        const pair_t keep = pack(sm.weight[L], sm.weight[L]);
#pragma unroll
        for (int j = 0; j < RT / 2; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) X[j][c] = mul2(X[j][c], keep);
#pragma unroll 4
        for (int j = 0; j < L; ++j) {
            const float4 y = *reinterpret_cast<const float4*>(&sm.W[j][4 * tc]);
            const pair_t v[4] = {pack(y.x, y.x), pack(y.y, y.y), pack(y.z, y.z), pack(y.w, y.w)};
#pragma unroll
            for (int x = 0; x < RT; x += 4) {
                const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(&sm.B[j][RT * tr + x]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    X[x / 2][c] = fma2(b.x, v[c], X[x / 2][c]);
                    X[x / 2 + 1][c] = fma2(b.y, v[c], X[x / 2 + 1][c]);
                }
            }
        }
    }
    // where the state goes: behind the last piece to the caller, behind the others' first phase to the next piece's slot
    if (it.piece == it.pieces - 1) {
        if (r.last) {
            float* to = r.last + ((long long)it.seq * p.H + h) * state;
#pragma unroll
            for (int i = 0; i < RT; i += 2)
#pragma unroll
                for (int c = 0; c < 4; ++c) unpack(X[i / 2][c], to[place(i, c)], to[place(i + 1, c)]);
        }
    } else if (p.phase == 1) {
        float* to = slot(it.piece + 1);
#pragma unroll
        for (int i = 0; i < RT; i += 2) {
            float4 a, b;
            unpack(X[i / 2][0], a.x, b.x);
            unpack(X[i / 2][1], a.y, b.y);
            unpack(X[i / 2][2], a.z, b.z);
            unpack(X[i / 2][3], a.w, b.w);
            *reinterpret_cast<float4*>(to + slot_at(i)) = a;
            *reinterpret_cast<float4*>(to + slot_at(i + 1)) = b;
        }
    }
}

__global__ void __launch_bounds__(kThreads, 2) simt_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) char raw[];
    if (p.dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tile = blockIdx.x % p.tiles;
    Item it;
    int first, rest;
    if (!item_of(p, blockIdx.x / p.tiles, it, first, rest)) return;
    const Role& r = p.role[it.role];
    if (tile * kTile >= r.dC) return;
    if (r.dA == 64)
        walk<64>(p, r, it, first, rest, tile, *reinterpret_cast<Smem<64>*>(raw));
    else
        walk<128>(p, r, it, first, rest, tile, *reinterpret_cast<Smem<128>*>(raw));
}

}  // namespace

cudaError_t launch_simt(const Params* phases, int n, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<128>));
    for (int i = 0; i < n && e == cudaSuccess; ++i) {
        Params p = phases[i];
        int dA = 0, dC = 0;
        for (int k = 0; k < p.nroles; ++k) dA = max(dA, p.role[k].dA), dC = max(dC, p.role[k].dC);
        p.tiles = dC / kTile;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)((long long)p.blocks * p.tiles));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = dA == 64 ? sizeof(Smem<64>) : sizeof(Smem<128>);
        cfg.stream = s;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = p.dependent ? 1 : 0;
        e = cudaLaunchKernelEx(&cfg, simt_kernel, p);
    }
    return e;
}

}  // namespace linear
}  // namespace gdn

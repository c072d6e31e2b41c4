// gdn_linear_tc.cu -- linear attention with a decay for each head on the 5th-generation tensor cores: bf16 inputs and outputs
// (the forward and, with the roles changed, the three gradients: gdn_linear.cuh).
//
// A CTA owns one piece of one sequence and one head, and walks over its chunks of 128 tokens. Per chunk, with weights w^..
// of the head's constant decay:
//   S = A B^T                              128 x 128 x dA
//   P = S with the weights of the gaps, masked, rounded to bf16 (tensor memory, over S)
//   O = A X                                128 x dC x dA, X the state entering the chunk, rounded to bf16 (shared memory)
//   O = w^(i + 1 - s) O, row by row        (through registers: the row's weight is not rounded)
//   O += P C                               128 x dC x 128
//   U^T = Cw^T B                           dC x dA x 128, Cw = C with the weights of the update, as an unevaluated sum of
//                                          two bf16 values (tensor memory), so that the state gets products good to 2^-17
//   X' = w^L X + U                         fp32, in registers
// The state never passes through bf16 on its own way. U is formed transposed, with the scaled operand in tensor memory:
// its 128 rows (channels of C) are then the lanes, each of which scales its own channel; the chunk's tiles fill shared
// memory (two stages of A, B, C: 192 KB, and 32 KB of X), which would not hold scaled copies as well.
// P and X are rounded to bf16 because the products' other operand is bf16 (fp32 ones would take two or three parts each): outputs
// off by 2.3e-3 of their RMS instead of a bf16 result's 1.7e-3. Cw has two parts because a third one takes 24 instead of 16
// MMAs a chunk and room that only slices of 32 tokens leave: 25 % of the forward's time, 19 % of the gradients', for states off by
// 4 to 6e-7 of their RMS instead of 2.4e-6.
//
// Warps: 0-7 P and the outputs; 8-15 the state: Cw (each half of them 64 tokens), X (each half 64 rows) and the scaling of O;
// 16 loads (TMA, 128-byte swizzle), 17 issues S and O += P C, 19 O = A X and U, 18 stores bf16 outputs (TMA). P takes S's place in
// tensor memory, outputs leave through A's tile. Every wait on an mbarrier is bounded: on expiry it sets a flag that ends the
// other waits too; the CTA then lets what it issued retire, records GDN_ERR_TIMEOUT, frees tensor memory and returns.
//
// Measured (dA = dC = 128), from pieces of 64 and of 128 chunks, calls back to back: with half of the SMs at work a chunk takes 1.91 us
// (3800 cycles at 1.99 GHz), with all of them 2.94 us in the gradients (5350 cycles at the 1.82 GHz that the power limit leaves) and 3.1 us
// in the forward, which then moves 6.4 TB/s. By arithmetic: shared memory's traffic 450 KB, 3500 cycles (tiles written
// once and read by two or three products, X, Cw and the outputs), the MMAs 40 of 64 cycles, one chain of S, P, O += P C from one
// chunk to the next. Sums alone take 1.7 us a chunk at most (103 of them in 172 us). 2 x 32768 tokens of 32 heads: 462 us, 4.67
// TB/s of 6.80; their gradients at 2 x 8192: 283 us.
//
// Code. The two SMs of a pair share what holds their instructions, and 20 warps are at as many places of the code: what the
// compiler unrolls counts. With every wait's loop unrolled (118 KB instead of 79, without the copies for a second pass) the first case took 472 us.
//
// A sequence's last chunk may hold fewer than 128 tokens: the rows of B and C behind it (the next sequence's) are
// overwritten by zeros in shared memory, so that nothing of another sequence enters a sum, not as 0 times NaN either. Nor
// does an infinity or a NaN of a token reach tokens that do not see it: see run_again.
#include <atomic>
#include <cstring>

#include "gdn_linear.cuh"
#include "gdn_pair.cuh"
#include "gdn_tc_common.cuh"

namespace gdn {
namespace linear {
namespace {

constexpr int kThreads = 640;   // five warpgroups
constexpr int kOutThreads = 256, kStateThreads = 256;
constexpr int kStateWarp0 = 8;
constexpr int kRegsOut = 72, kRegsState = 144, kRegsRest = 48, kRegsLaunch = 96;
static_assert(256 * kRegsOut + 256 * kRegsState + 128 * kRegsRest == kRegsLaunch * kThreads, "the registers of the launch");
constexpr int kLoadWarp = 16, kMmaWarp = 17, kStoreWarp = 18, kStateMmaWarp = 19;
constexpr long long kWaitLimit = 4000000000LL;   // SM cycles, some two seconds (for the waits while shutting down)
constexpr int kWaitTries = 1 << 20;              // of a wait: a second or so at least, 20 at most

constexpr uint32_t kHalf = 16384;                // 128 tokens x 64 features
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr uint32_t kStage = 3 * kTileBytes;      // A, B, C
constexpr uint32_t kX = 2 * kStage;              // [dA / 64][dC rows of 128 bytes]
constexpr uint32_t kTab = kX + kTileBytes;       // w^0 .. w^128
constexpr uint32_t kKey = kTab + 132 * 4;        // weights of the update (see below): 256
constexpr uint32_t kBar = kKey + 256 * 4;
// a second pass is wanted (see run_again); in it, for each half of the tokens and column of C, the first token, in the role's
// direction, whose value is infinite or NaN, or kNone
constexpr uint32_t kOdd = kBar + 200, kOddToken = kBar + 208;
constexpr int kNone = 255;
constexpr uint32_t kSmem = kOddToken + 256 + 1024;   // (with the slack of a 1024-byte alignment)
static_assert(kSmem <= 232448, "shared memory");
static_assert(kTab % 16 == 0 && kKey % 16 == 0 && kBar % 16 == 0, "alignment");

// tensor memory, columns
constexpr uint32_t kTmS = 0, kTmU = 128, kTmHi = 256, kTmLo = 320, kTmO = 384;

// mbarriers, 8 bytes each from kBar on. A wait names a phase by its parity, so no barrier may get two phases ahead of any warp that
// waits on it, however long that warp is held up: between two phases of each lies something that every one of its
// waiters does only once it has seen the first.
enum {
    B_FULL0 = 0, B_FULL1,    // a stage: B and C have come
    B_EMPTY0, B_EMPTY1,      //          B and C are done with
    B_AFULL0, B_AFULL1,      //          A has come
    B_AFREE0, B_AFREE1,      //          the outputs have left A's tile
    B_OUT0, B_OUT1,          //          bf16 outputs lie in A's tile
    B_S, B_P,                // S, P are in tensor memory
    B_OI, B_OSCALED, B_O,    // O = A X; with the rows' weights; with P C
    B_OFREE,                 // O has been read
    B_VD, B_U,               // Cw, U are in tensor memory
    B_X,                     // X is in shared memory
    B_ZERO,                  // the rows behind the sequence's end are zeros
    B_TAKEN,                 // second pass: C is finite
    B_DRAIN0, B_DRAIN1,      // shutting down: what the two MMA warps issued has retired
    B_N
};
constexpr unsigned kTag = 0x60;   // + the barrier's number
static_assert(kBar + 8 * B_N + 12 <= kOdd, "the barriers, the flag and tensor memory's address");

struct TcParams {
    Params p;
    CUtensorMap a[kMaxRoles], b[kMaxRoles], c[kMaxRoles], out[kMaxRoles];
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]),
        "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]),
        "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]),
        "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
        : "memory");
}

// one MMA by the lane with `first`; and the arrival of the barrier once that lane's MMAs have retired
template <uint32_t ID>
__device__ __forceinline__ void mma_one_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate, uint32_t first) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "n"(ID), "r"(accumulate), "r"(first)
        : "memory");
}
template <uint32_t ID>
__device__ __forceinline__ void mma_one_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate, uint32_t first) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "n"(ID), "r"(accumulate), "r"(first)
        : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t bar, uint32_t first) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(bar), "r"(first)
        : "memory");
}

// a box from shared memory to global, in the thread's open group; its commit; the wait until the groups' boxes have been read
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, uint32_t from, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(from), "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ void ldmatrix_trans(uint32_t at, uint32_t (&v)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
}
// 16 lanes x 8 columns: register 2 g + h holds lane 8 h + T / 4, column 4 g + T % 4
__device__ __forceinline__ void tmem_st_16x128b_x2(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ float lds(uint32_t at) {
    float x;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(x) : "r"(at));
    return x;
}
__device__ __forceinline__ int lds_int(uint32_t at) {   // (volatile, these: what other threads write)
    int x;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ int lds_u8(uint32_t at) {
    int x;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ int lds_u16(uint32_t at) {
    int x;
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
    return x;
}
__device__ __forceinline__ void sts_int(uint32_t at, int x) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(x) : "memory"); }
__device__ __forceinline__ void sts_u8(uint32_t at, int x) { asm volatile("st.shared.u8 [%0], %1;" ::"r"(at), "r"(x) : "memory"); }
__device__ __forceinline__ void sts_zero16(uint32_t at) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((unsigned short)0) : "memory");
}
__device__ __forceinline__ float4 lds4(uint32_t at) {
    float4 x;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at));
    return x;
}
__device__ __forceinline__ void sts4(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// while shutting down after a wait that ran out: lets what the CTA issued retire
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, long long limit) {
    const long long t0 = clock64();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > limit) return;
}

// What every warp of the CTA knows of its work. Its waits are those of gdn_tc_common.cuh with the loop in place and
// the limit counted in tries (each of at most 20 us): a call would put the caller's registers on the stack, which, with
// all of the SM's memory shared, is in L2; and every warp walks through its waits once a chunk, so their code is short.
struct Work {
    const Params* p;
    const Role* r;
    Item it;
    int h, chunks, n;      // chunks of the piece, of the sequence
    int first, rest;
    bool sums;             // phase 1's middle pieces: U alone
    uint32_t base, tmem;
    volatile int* abort_flag;
    float lg;
    __device__ __forceinline__ int phys(int m) const { return r->rev ? n - 1 - (it.m0 + m) : it.m0 + m; }
    __device__ __forceinline__ int length(int m) const { return min(kChunk, it.len - kChunk * phys(m)); }
    __device__ __forceinline__ uint32_t bar(int i) const { return base + kBar + 8 * i; }
    // tensor memory of Cw; sums alone have two, the other in the place of S, and form a chunk's Cw during the last one's U
    __device__ __forceinline__ uint32_t cw(int m) const { return sums && (m & 1) ? kTmS : kTmHi; }
    // the whole warp waits; every lane gets the same verdict
    __device__ __forceinline__ bool wait(int i, int parity) const {
#pragma unroll 1
        for (int left = kWaitTries; !__all_sync(0xffffffffu, mbar_try_wait_suspend(bar(i), parity & 1, 20000u)); --left) {
            if (__any_sync(0xffffffffu, *abort_flag)) return false;
            if (left == 0) {
                *abort_flag = kTag + i;   // (the CTA's end records it)
                return false;
            }
        }
        return true;
    }
    __device__ __forceinline__ bool wait1(int i, int parity) const {   // one lane
#pragma unroll 1
        for (int left = kWaitTries; !mbar_try_wait_suspend(bar(i), parity & 1, 20000u); --left) {
            if (*abort_flag) return false;
            if (left == 0) {
                *abort_flag = kTag + i;   // (the CTA's end records it)
                return false;
            }
        }
        return true;
    }
};

// The loads of a piece's chunks (one lane): the first two of them, for which there is nothing to wait for, before the CTA is
// set up; the others (in a second pass, where `from` is 0, all) as the stages become free.
template <int DA, int DC, bool FIRST>
__device__ __forceinline__ void load_warp(const Work& w, const CUtensorMap* ma, const CUtensorMap* mb, const CUtensorMap* mc, int from = 0) {
    const int heads = w.p->H;
    const int ah = w.h / (heads / w.r->a_heads), bh = w.h / (heads / w.r->b_heads), ch = w.h / (heads / w.r->c_heads);
    int issued = min(from, w.chunks), issued_a = w.sums ? 0 : issued;
#pragma unroll 1
    for (int m = from; m < (FIRST ? min(2, w.chunks) : w.chunks); ++m) {
        const int s = m & 1;
        if (!FIRST && m >= 2 && !w.wait1(B_EMPTY0 + s, (m >> 1) - 1)) break;
        const uint32_t to = w.base + s * kStage;
        const int row = w.it.lo + kChunk * w.phys(m);
        mbar_arrive_expect_tx(w.bar(B_FULL0 + s), (DA / 64 + DC / 64) * kHalf);
#pragma unroll
        for (int f = 0; f < DC / 64; ++f) tma_load_3d(to + 2 * kTileBytes + f * kHalf, mc, w.bar(B_FULL0 + s), 64 * f, ch, row);
#pragma unroll
        for (int f = 0; f < DA / 64; ++f) tma_load_3d(to + kTileBytes + f * kHalf, mb, w.bar(B_FULL0 + s), 64 * f, bh, row);
        issued = max(issued, m + 1);
        if (w.sums) continue;
        // (A's tile holds the outputs of chunk m - 2 until they have left)
        if (!FIRST && m >= 2 && !w.wait1(B_AFREE0 + s, (m >> 1) - 1)) break;
        mbar_arrive_expect_tx(w.bar(B_AFULL0 + s), (DA / 64) * kHalf);
#pragma unroll
        for (int f = 0; f < DA / 64; ++f) tma_load_3d(to + f * kHalf, ma, w.bar(B_AFULL0 + s), 64 * f, ah, row);
        issued_a = max(issued_a, m + 1);
    }
    if (!FIRST && *w.abort_flag) {   // (what is in flight lands before shared memory is given back)
        for (int m = max(0, issued - 2); m < issued; ++m) drain(w.bar(B_FULL0 + (m & 1)), (m >> 1) & 1, kWaitLimit);
        for (int m = max(0, issued_a - 2); m < issued_a; ++m) drain(w.bar(B_AFULL0 + (m & 1)), (m >> 1) & 1, kWaitLimit);
    }
}

// The MMAs: one warp issues S and O += P C, another one O = A X and U, so that what a step costs besides its MMAs (some
// hundred cycles of waits and commits) passes while the other's are at work. The whole warp walks through the code, with
// values that are the same in every lane, and the first lane issues: descriptors then stay in uniform registers (under a
// branch on the lane each MMA took some 140 cycles to issue). Operands whose rows hold the contraction advance by 32 bytes a
// step within a half, the others by 16 rows of 128 bytes; in descriptors, in units of 16 bytes.
template <uint32_t ID, int STEPS>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b, uint32_t b_half, uint32_t first) {
    uint64_t da = desc_k(a), db = desc_k(b);
#pragma unroll 1
    for (int f = 0; f < STEPS / 4; ++f, da += kHalf / 16, db += b_half / 16)
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_one_ss<ID>(d, da + 2 * k, db + 2 * k, f + k > 0, first);
}
template <uint32_t ID, int PARTS, int APART>
__device__ __forceinline__ void mma_tokens(uint32_t d, uint32_t a, uint32_t b, uint32_t accumulate, uint32_t first) {
    const uint64_t db = desc_mn(b, kHalf);
#pragma unroll 1
    for (int k = 0; k < 8 * PARTS; k += 4, accumulate = 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) mma_one_ts<ID>(d, a + APART * (k + i), db + 128 * (k % 8 + i), i ? 1u : accumulate, first);
}

template <int DA, int DC>
__device__ __forceinline__ void intra_warp(const Work& w, int lane) {
    constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false), ID_OP = idesc_bf16(128, DC, false, true);
    const uint32_t first = lane == 0;
    int m = 0;
    for (; m < w.chunks; ++m) {
        const int st = m & 1;
        const uint32_t A = w.base + st * kStage, B = A + kTileBytes, C = B + kTileBytes;
        if (!w.wait(B_FULL0 + st, m >> 1) || !w.wait(B_AFULL0 + st, m >> 1)) break;
        if (w.length(m) < kChunk && !w.wait(B_ZERO, 0)) break;
        if (m > 0 && !w.wait(B_O, m - 1)) break;   // (P has been read)
        tc_fence_after();
        mma_rows<ID_S, DA / 16>(w.tmem + kTmS, A, B, kHalf, first);
        commit_one(w.bar(B_S), first);
        if (!w.wait(B_P, m) || !w.wait(B_OSCALED, m)) break;
        tc_fence_after();
        mma_tokens<ID_OP, 1, 16>(w.tmem + kTmO, w.tmem + kTmS, C, 1, first);
        commit_one(w.bar(B_O), first);
        commit_one(w.bar(B_EMPTY0 + st), first);
    }
    if (m < w.chunks) {
        commit_one(w.bar(B_DRAIN0), first);
        drain(w.bar(B_DRAIN0), 0, kWaitLimit);
    }
}

template <int DA, int DC>
__device__ __forceinline__ void state_mma_warp(const Work& w, int lane) {
    constexpr uint32_t ID_OI = idesc_bf16(128, DC, false, false), ID_U = idesc_bf16(128, DA, false, true);
    static_assert(kTmLo == kTmHi + 64, "one part behind the other");
    const uint32_t first = lane == 0;
    int m = 0;
    for (; m < w.chunks; ++m) {
        const int st = m & 1;
        const uint32_t A = w.base + st * kStage, B = A + kTileBytes;
        if (!w.wait(B_FULL0 + st, m >> 1)) break;
        if (w.length(m) < kChunk && !w.wait(B_ZERO, 0)) break;
        if (!w.sums) {
            if (!w.wait(B_AFULL0 + st, m >> 1) || !w.wait(B_X, m) || (m > 0 && !w.wait(B_OFREE, m - 1))) break;
            tc_fence_after();
            mma_rows<ID_OI, DA / 16>(w.tmem + kTmO, A, w.base + kX, DC * 128, first);
            commit_one(w.bar(B_OI), first);
        }
        if (!w.wait(B_VD, m)) break;
        tc_fence_after();
        mma_tokens<ID_U, 2, 8>(w.tmem + kTmU, w.tmem + w.cw(m), B, 0, first);
        commit_one(w.bar(B_U), first);
        commit_one(w.bar(B_EMPTY0 + st), first);
    }
    if (m < w.chunks) {
        commit_one(w.bar(B_DRAIN1), first);
        drain(w.bar(B_DRAIN1), 0, kWaitLimit);
    }
}

// P and the outputs: thread = row (token) of the chunk = lane of tensor memory; of every 32 columns of P one half of the warps
// takes the first 16 and the other the last, of the outputs' columns each takes a half. P's 16 columns (8 of tensor
// memory, packed) replace the first 8 of the 16 of S that they come from, so that no thread writes where another one still reads.
template <int DA, int DC, bool OUT_BF16>
__device__ __forceinline__ void out_warps(const Work& w, const CUtensorMap* map, int warp, int lane) {
    const Role& r = *w.r;
    const int half = warp >> 2, quarter = warp & 3;
    const int row = 32 * quarter + lane;
    const uint32_t lanes = w.tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t tab = w.base + kTab;
    // The weight of row i and column j is w^|i - j|. Columns in blocks of 32: w^(31 - c) (or, backward in time, w^c) for the column
    // of a block, times what is left of the gap, one value a row and block. In the diagonal block that is w^(lane - 31) (or
    // w^-lane), which fp32 holds for heads that lose fewer than 2^100 over a block; `steep` ones take 2^(log2 w gap) as it is.
    // (Of the diagonal block only the bits of columns that the row sees stay: what lies behind it, infinities too, becomes
    // zero.)
    pair_t col[8];
    uint32_t seen[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = 16 * half + 2 * i;
        col[i] = pack(lds(tab + 4 * (r.rev ? c : 31 - c)), lds(tab + 4 * (r.rev ? c + 1 : 30 - c)));
        seen[i] = ((r.rev ? c >= lane : c <= lane) ? 0xffffu : 0u) | ((r.rev ? c + 1 >= lane : c + 1 <= lane) ? 0xffff0000u : 0u);
    }
    const bool steep = !(w.lg * 31.f > -100.f);
    const float diag = exp2f(r.rev ? -w.lg * lane : w.lg * (lane - 31));
    const int b0 = r.rev ? quarter : 0, b1 = r.rev ? 4 : quarter + 1;   // the blocks that the row sees anything of
    for (int m = 0; m < w.chunks; ++m) {
        const int L = w.length(m);
        if (!w.wait(B_S, m)) return store_wait();
        tc_fence_after();
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            const uint32_t at = lanes + kTmS + 32 * b + 16 * half;
            uint32_t q[8];
            if (b < b0 || b >= b1) {
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] = 0;
            } else {
                float x[16];
                tmem_ld16(at, x);
                const float f = b == quarter ? diag : lds(tab + 4 * (r.rev ? 32 * (b - quarter) - lane : 32 * (quarter - b) + lane - 31));
                const uint32_t all = b == quarter ? 0u : 0xffffffffu;
                const pair_t f2 = pack(f, f);
                tmem_wait_ld();
                if (!steep) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float lo, hi;
                        unpack(mul2(pack(x[2 * i], x[2 * i + 1]), mul2(f2, col[i])), lo, hi);
                        q[i] = pack_bf16(lo, hi) & (seen[i] | all);
                    }
                } else {
                    const int gap0 = r.rev ? 32 * b + 16 * half - row : row - 32 * b - 16 * half;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int gap = r.rev ? gap0 + 2 * i : gap0 - 2 * i, gap1 = r.rev ? gap + 1 : gap - 1;
                        q[i] = pack_bf16(gap >= 0 ? x[2 * i] * ex2(w.lg * gap) : 0.f, gap1 >= 0 ? x[2 * i + 1] * ex2(w.lg * gap1) : 0.f);
                    }
                }
            }
            tmem_st8(at, q);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(w.bar(B_P));
        if (!w.wait(B_O, m)) return store_wait();
        tc_fence_after();
        // out through A's tile, which is done with: 128 rows of 128 bytes in each half of it
        const int row0 = w.it.lo + kChunk * w.phys(m) + 32 * quarter, rows = min(32, L - 32 * quarter);
        constexpr int kSize = OUT_BF16 ? 2 : 4, kPer = 128 / kSize;   // features of 128 bytes
        constexpr int kMine = DC / 2;                                 // this half's columns
        constexpr int kBoxes = kMine > kPer ? kMine / kPer : 1;       // fp32 with DC = 128: two, one after the other
        constexpr int kSteps = kMine / kBoxes / 16;
#pragma unroll 1
        for (int b = 0; b < kBoxes; ++b) {
            const int first = kMine * half + kMine / kBoxes * b;      // column
            // (bf16 outputs of 64 columns: both halves' in one row of 128 bytes)
            constexpr bool kShare = OUT_BF16 && DC == 64;
            const uint32_t box = w.base + (m & 1) * kStage + (kShare ? 0 : half * kHalf) + quarter * 4096;
            const int piece0 = kShare ? 4 * half : 0;                 // 16-byte pieces of a row
            if (b > 0) {   // (the first has to leave before the next)
                store_wait();
                __syncwarp();
            }
#pragma unroll 1
            for (int z = 0; z < kSteps; ++z) {
                float f[16];
                tmem_ld16(lanes + kTmO + first + 16 * z, f);
                tmem_wait_ld();
                if (b == kBoxes - 1 && z == kSteps - 1) {
                    tc_fence_before();
                    mbar_arrive(w.bar(B_OFREE));
                }
                if constexpr (OUT_BF16) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        sts4(box + sw128(lane, piece0 + 2 * z + k), pack_bf16(f[8 * k], f[8 * k + 1]), pack_bf16(f[8 * k + 2], f[8 * k + 3]),
                             pack_bf16(f[8 * k + 4], f[8 * k + 5]), pack_bf16(f[8 * k + 6], f[8 * k + 7]));
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        sts4(box + sw128(lane, 4 * z + k), __float_as_uint(f[4 * k]), __float_as_uint(f[4 * k + 1]),
                             __float_as_uint(f[4 * k + 2]), __float_as_uint(f[4 * k + 3]));
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (!OUT_BF16 && rows == 32) {
                if (lane == 0) tma_store_3d(map, box, first, w.h, row0);
            } else if (OUT_BF16 ? L < kChunk : rows < 32) {   // the sequence ends in this chunk: row by row
                constexpr int kPieces = kMine / kBoxes * kSize / 16;   // of 16 bytes in a row: 4 or 8 lanes each
#pragma unroll 1
                for (int i = lane / kPieces; i < rows; i += 32 / kPieces) {
                    const int k = lane % kPieces;
                    const float4 v = lds4(box + sw128(i, piece0 + k));
                    char* to = (char*)r.out + (((long long)(row0 + i) * w.p->H + w.h) * DC + first) * kSize + 16 * k;
                    *reinterpret_cast<float4*>(to) = v;
                }
                __syncwarp();
            }
        }
        if constexpr (OUT_BF16) {
            mbar_arrive(w.bar(B_OUT0 + (m & 1)));   // (to store_warp)
        } else {
            store_wait();
            __syncwarp();
            if (lane == 0) mbar_arrive(w.bar(B_AFREE0 + (m & 1)));
        }
    }
    store_wait();
}

// Sends the bf16 outputs from A's tile and gives it back to the loads (one lane).
template <int DC>
__device__ __forceinline__ void store_warp(const Work& w, const CUtensorMap* map) {
    for (int m = 0; m < w.chunks; ++m) {
        if (!w.wait1(B_OUT0 + (m & 1), m >> 1)) break;
        if (w.length(m) == kChunk) {   // (a sequence's last rows have gone by other ways)
#pragma unroll
            for (int b = 0; b < DC / 64; ++b)
                tma_store_3d(map, w.base + (m & 1) * kStage + b * kHalf, 64 * b, w.h, w.it.lo + kChunk * w.phys(m));
            store_wait();
        }
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 8;" ::"r"(w.bar(B_AFREE0 + (m & 1))) : "memory");
    }
    store_wait();
}

// Cw and the state: thread = channel of C = lane of tensor memory; the two halves of the warps take 64 tokens of Cw and 64
// rows of the state each
template <int DA, int DC, bool CAREFUL>
__device__ __forceinline__ void state_warps(const Work& w, int warp, int lane) {
    const Role& r = *w.r;
    const int half = warp >> 2, quarter = warp & 3;
    const int chan = 32 * quarter + lane, c = chan & (DC - 1);   // (with DC = 64, lanes 64 .. repeat channels 0 ..)
    const bool mine = chan < DC && 64 * half < DA;               // holds rows of the state
    const uint32_t lanes = w.tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t key = w.base + kKey;
    constexpr long long kState = (long long)DA * DC;
    float X[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) X[i] = 0.f;
    auto slot = [&](int q) {
        return w.p->slots + (w.it.slot + (long long)(q - 1) * w.it.slot_step) * kState + (long long)64 * half * DC + c;
    };
    auto given = [&](auto base) {   // of a state as the caller stores it: this thread's row 0
        const auto at = base + ((long long)w.it.seq * w.p->H + w.h) * kState;
        return r.state_t ? at + (long long)c * DA + 64 * half : at + (long long)64 * half * DC + c;
    };
    if (w.p->phase == 2) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (mine) {
        if (w.it.piece == 0) {
            if (r.start) {
                const float* from = given(r.start);
                if (r.state_t) {
#pragma unroll
                    for (int i = 0; i < 64; i += 4) {
                        const float4 t = __ldg(reinterpret_cast<const float4*>(from + i));
                        X[i] = t.x, X[i + 1] = t.y, X[i + 2] = t.z, X[i + 3] = t.w;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) X[i] = __ldg(from + i * DC);
                }
            }
        } else if (!w.sums) {
#pragma unroll 1
            for (int q = 1; q <= w.it.piece; ++q) {
                // entering piece q: from the state entering piece q - 1 and that piece's sum (q = 1: what piece 0 left)
                const float keep = q == 1 ? 0.f
                    : exp2f(w.lg * tokens_of(w.first + (q - 2) * w.rest, w.first + (q - 1) * w.rest, w.it.len, r.rev));
                const float* from = slot(q);
#pragma unroll
                for (int i = 0; i < 64; ++i) X[i] = fmaf(keep, X[i], __ldcg(from + i * DC));
            }
        }
    }
    auto put_x = [&]() {   // the state as the next chunk's outputs read it
        if (mine) {
            const uint32_t to = w.base + kX + half * (DC * 128);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                sts4(to + sw128(c, k), pack_bf16(X[8 * k], X[8 * k + 1]), pack_bf16(X[8 * k + 2], X[8 * k + 3]),
                     pack_bf16(X[8 * k + 4], X[8 * k + 5]), pack_bf16(X[8 * k + 6], X[8 * k + 7]));
        }
        fence_proxy_async();
        mbar_arrive(w.bar(B_X));
    };
    if (!w.sums && w.chunks > 0) put_x();
    // Cw's fragments: an 8 x 8 matrix of tokens x channels, loaded with transposition, leaves a lane channel lane / 4 of
    // tokens 2 (lane % 4) and the next one; two of them (channels 0 .. 7 and 8 .. 15) are what a 16 x 128-bit store to
    // tensor memory takes for 16 channels (its lanes) and four token pairs (its columns). A lane's row address:
    const int chan0 = (32 * quarter) & (DC - 1);
    // (lanes 0 .. 15: tokens of group g, 16 .. 31: of group g + 1; 16 channels further on, bit 5 of the address flips)
    const uint32_t ldm = (chan0 >> 6) * kHalf + half * 8192 + (lane >> 4) * 1024 + (lane & 7) * 128 +
                         (((((chan0 & 63) >> 3) + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
    const int tok = 64 * half + 2 * (lane & 3);   // of its pairs in 8-token group 0
    auto take_u = [&](int m) {   // X' = w^L X + U
        if (!w.wait(B_U, m)) return false;
        tc_fence_after();
        const float keep = exp2f(w.lg * w.length(m));
        if (64 * half < DA) {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float u[32];
                tmem_ld32(lanes + kTmU + 64 * half + 32 * b, u);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 2)
                    unpack(fma2(pack(keep, keep), pack(X[32 * b + i], X[32 * b + i + 1]), pack(u[i], u[i + 1])), X[32 * b + i],
                           X[32 * b + i + 1]);
            }
        }
        return true;
    };
    // Second pass: this thread's 64 values of C that are infinite or NaN leave the tile (Cw has them); where the first one was
    auto take_out = [&](int m) {
        if (chan < DC) {   // (what its warp made Cw from)
            const uint32_t column = w.base + (m & 1) * kStage + 2 * kTileBytes + (c >> 6) * kHalf + half * 8192 + 2 * (c & 7);
            int token = kNone;
#pragma unroll 1
            for (int i = 0; i < 64; ++i) {   // (the last one to be met stays)
                const int t = r.rev ? i : 63 - i;
                const uint32_t at = column + t * 128 + ((((c & 63) >> 3) ^ (t & 7)) << 4);
                if ((lds_u16(at) & 0x7f80) != 0x7f80) continue;
                sts_zero16(at);
                token = 64 * half + t;
            }
            sts_u8(w.base + kOddToken + 128 * half + c, token);
            fence_proxy_async();
        }
        mbar_arrive(w.bar(B_TAKEN));
    };
    // ... and O's rows that see one get NaN in its column, for P C to be added to: this thread's row, half of the columns
    auto put_nan = [&]() {
#pragma unroll 1
        for (int k = DC / 2 * half; k < DC / 2 * (half + 1); ++k) {
            const int a = lds_u8(w.base + kOddToken + k), b = lds_u8(w.base + kOddToken + 128 + k);
            if (a == kNone && b == kNone) continue;
            uint32_t x;
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(x) : "r"(lanes + kTmO + k) : "memory");
            tmem_wait_ld();
            if (r.rev ? (a != kNone && chan <= a) || (b != kNone && chan <= b) : chan >= a || chan >= b) x = 0x7fffffffu;
            asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(lanes + kTmO + k), "r"(x) : "memory");
        }
        tmem_wait_st();
    };
    bool zeroed = false;
    for (int m = 0; m < w.chunks; ++m) {
        const int L = w.length(m);
        const uint32_t B = w.base + (m & 1) * kStage + kTileBytes, C = B + kTileBytes;
        if (!w.wait(B_FULL0 + (m & 1), m >> 1)) return;
        if (L < kChunk && !zeroed) {
            zeroed = true;
            const int t = 128 * half + chan;   // two threads a row, one a tile
            const int row = t >> 1;
            if (row >= L) {
                const uint32_t tile = t & 1 ? C : B;
                const int halves = t & 1 ? DC / 64 : DA / 64;
#pragma unroll 1
                for (int f = 0; f < halves; ++f)
#pragma unroll
                    for (int k = 0; k < 8; ++k) sts4(tile + f * kHalf + row * 128 + 16 * k, 0, 0, 0, 0);
            }
            fence_proxy_async();
            mbar_arrive(w.bar(B_ZERO));
            if (!w.wait(B_ZERO, 0)) return;
        }
        // Cw = hi + lo of 64 tokens' values of 32 channels, 16 tokens and 16 channels at a time: the value rounded to bf16,
        // and the rest of it, rounded
        const uint32_t weights = key + 4 * (tok + (r.rev ? 0 : kChunk - L));
        const uint32_t cw_at = w.cw(m);
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
            const uint32_t to = lanes + cw_at + ((uint32_t)(16 * x) << 16) + 32 * half;
            const uint32_t from = C + (ldm ^ 32 * x);
#pragma unroll
            for (int g = 0; g < 8; g += 2) {
                uint32_t v[4], hi[4], lo[4];   // two 8-token groups x 16 channels
                ldmatrix_trans(from + g * 1024, v);
                const pair_t weight[2] = {pack(lds(weights + 32 * g), lds(weights + 32 * g + 4)),
                                          pack(lds(weights + 32 * g + 32), lds(weights + 32 * g + 36))};
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // (group g + i / 2, channels 8 (i % 2) ..)
                    const pair_t y = mul2(pack(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xffff0000u)), weight[i / 2]);
                    float a, b;
                    unpack(y, a, b);
                    hi[i] = pack_bf16(a, b);
                    unpack(fma2(pack(__uint_as_float(hi[i] << 16), __uint_as_float(hi[i] & 0xffff0000u)), pack(-1.f, -1.f), y), a, b);
                    lo[i] = pack_bf16(a, b);
                }
                tmem_st_16x128b_x2(to + 4 * g, hi);
                tmem_st_16x128b_x2(to + (kTmLo - kTmHi) + 4 * g, lo);
            }
        }
        tmem_wait_st();
        // (sums alone: U of the chunk before, while this chunk's Cw waits. Not behind the arrival: a warp held up there for as long
        // as the next U takes would find B_U a phase too far, and wait for ever)
        if (w.sums && m > 0 && !take_u(m - 1)) return;
        tc_fence_before();
        mbar_arrive(w.bar(B_VD));
        if (!w.sums) {   // the rows' weights on O = A X, while U is formed: half of the columns each; here lane = row
            if (!w.wait(B_OI, m)) return;
            tc_fence_after();
            if constexpr (CAREFUL) {   // (behind B_X the tokens of the chunk before have been read)
                if (!w.wait(B_X, m)) return;
                take_out(m);
            }
            const int row = chan;
            const float keep = exp2f(w.lg * (r.rev ? max(L - 1 - row, 0) : row + 1));
            const pair_t keep2 = pack(keep, keep);
#pragma unroll 1
            for (int b = 0; b < DC / 64; ++b) {
                float x[32];
                tmem_ld32(lanes + kTmO + DC / 2 * half + 32 * b, x);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; i += 2) unpack(mul2(pack(x[i], x[i + 1]), keep2), x[i], x[i + 1]);
                tmem_st32(lanes + kTmO + DC / 2 * half + 32 * b, x);
            }
            tmem_wait_st();
            if constexpr (CAREFUL) {
                if (!w.wait(B_TAKEN, m)) return;
                put_nan();
            }
            tc_fence_before();
            mbar_arrive(w.bar(B_OSCALED));
        }
        if (!w.sums && !take_u(m)) return;
        if (!w.sums && m + 1 < w.chunks) {
            tc_fence_before();
            put_x();
        }
    }
    if (w.sums && !take_u(w.chunks - 1)) return;
    // (row 0 tells: a value of C that is not finite makes U's whole column NaN)
    if (mine && !w.sums && !(fabsf(X[0]) <= 3.4028235e38f)) sts_int(w.base + kOdd, 1);
    // where the state goes: behind the last piece to the caller, behind the others' first phase to the next piece's slot
    if (!mine) return;
    if (w.it.piece == w.it.pieces - 1) {
        if (r.last) {
            float* to = given(r.last);
            const int step = r.state_t ? 1 : DC;
#pragma unroll
            for (int i = 0; i < 64; ++i) to[i * step] = X[i];
        }
    } else if (w.p->phase == 1) {
        float* to = slot(w.it.piece + 1);
#pragma unroll
        for (int i = 0; i < 64; ++i) to[i * DC] = X[i];
    }
}

// how many arrivals end a phase of barrier i
__device__ __forceinline__ int arrivals(int i, bool sums) {
    switch (i) {
        case B_EMPTY0: case B_EMPTY1:                                  // commits: of O += P C and U, of sums alone U
            return sums ? 1 : 2;
        case B_AFREE0: case B_AFREE1:                                  // fp32: a lane of each output warp; bf16: store_warp, at once
            return kOutThreads / 32;
        case B_P: case B_OUT0: case B_OUT1: case B_OFREE:              // every output thread
            return kOutThreads;
        case B_OSCALED: case B_VD: case B_X: case B_ZERO: case B_TAKEN:   // every state thread
            return kStateThreads;
        default:                                                       // B_FULL, B_AFULL: the loading lane, beside its bytes;
            return 1;                                                  // B_S, B_OI, B_O, B_U, B_DRAIN: a commit
    }
}
__device__ __forceinline__ void init_barriers(const Work& w) {
    for (int i = 0; i < B_N; ++i) mbar_init(w.bar(i), arrivals(i, w.sums));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_proxy_async();
}

// Where all warps end a pass over the piece; whether another one follows.
//
// O += P C spreads an infinity or a NaN of C over all rows of its chunk, 0 times NaN being NaN. Whether there was one is
// seen by the state at the piece's end, which is then NaN in that column; the piece is then walked through a second time, in
// which the state's warps take what is not finite out of C's tile and give NaN to the rows that see it. So the pieces that
// have none pay for one look at the end. (Looking through C as it comes cost the training gradients 3 to 4 %, by the state's warps or
// an idle one; the second pass costs them 1 %, as long as the warps with much code have it behind the first one instead of in a
// loop around it: 285 us instead of 293, 283 without it.)
__device__ __forceinline__ bool run_again(const Work& w, int pass) {
    __syncwarp();
    tc_fence_before();
    asm volatile("barrier.sync 0;" ::: "memory");
    tc_fence_after();
    if (pass > 0 || *w.abort_flag || !lds_int(w.base + kOdd)) return false;
    // the outputs have to be there before they are written again; nothing may arrive at a barrier that is made anew
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (threadIdx.x == 32 * kLoadWarp) {
        bool ended = true;
        for (int m = max(0, w.chunks - 2); m < w.chunks; ++m) ended = ended && w.wait1(B_EMPTY0 + (m & 1), m >> 1);
        if (ended) {
            for (int i = 0; i < B_N; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(w.bar(i)) : "memory");
            init_barriers(w);
        }
    }
    asm volatile("barrier.sync 0;" ::: "memory");
    return !*w.abort_flag;
}

template <int K, int V>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const __grid_constant__ TcParams q) {
    extern __shared__ uint8_t smem_raw[];
    const Params& p = q.p;
    // Phase 1 waits for the plan that names its pieces, and then lets phase 2's blocks start on the SMs that it leaves: these
    // set up and load, and wait only before they read phase 1's states.
    if (p.phase == 1) {
        if (p.dependent) asm volatile("griddepcontrol.wait;" ::: "memory");
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    }
    Work w;
    w.p = &p;
    if (!item_of(p, blockIdx.x, w.it, w.first, w.rest)) {
        // Every block of phase 2 waits for phase 1, those without work too (of a packed batch that is not cut, all): what comes behind
        // this grid in the stream waits for this grid alone, and reads what phase 1 wrote.
        if (p.phase == 2) asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    const int role = w.it.role;
    w.r = &p.role[role];
    w.h = w.it.h;
    w.sums = p.phase == 1 && w.it.piece > 0;
    w.chunks = w.it.m1 - w.it.m0;
    w.n = (w.it.len + kChunk - 1) / kChunk;
    w.lg = log2_weight(p.decay, w.h);
    w.base = (smem_u32(smem_raw) + 1023) & ~1023u;
    uint8_t* sm = smem_raw + (w.base - smem_u32(smem_raw));
    w.abort_flag = reinterpret_cast<volatile int*>(sm + kBar + 8 * B_N);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kBar + 8 * B_N + 8);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const bool turned = K != V && w.r->state_t;   // dA = V, dC = K
    if (warp == kLoadWarp && lane == 0) {
        init_barriers(w);
        *w.abort_flag = 0;
        sts_int(w.base + kOdd, 0);
        turned ? load_warp<V, K, true>(w, &q.a[role], &q.b[role], &q.c[role])
               : load_warp<K, V, true>(w, &q.a[role], &q.b[role], &q.c[role]);
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    float* tab = reinterpret_cast<float*>(sm + kTab);
    float* key = reinterpret_cast<float*>(sm + kKey);
    if (tid <= 128) tab[tid] = exp2f(w.lg * tid);
    // the update's weights: forward w^(127 - j), read from place 128 - L on in a shorter chunk; backward w^(j + 1)
    if (tid < 256) key[tid] = tid < 128 ? exp2f(w.lg * (w.r->rev ? tid + 1 : 127 - tid)) : 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    w.tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    // The launch's 96 registers a thread, dealt anew: 256 x 72 + 256 x 144 + 128 x 48 = 640 x 96. (At 96 the state's warps
    // spill, and the stack is in L2.)
    if (warp < kStateWarp0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
        const bool bf16 = w.r->out_bf16;
        const CUtensorMap* map = &q.out[role];
        if (w.sums) {
        } else if (turned) {
            bf16 ? out_warps<V, K, true>(w, map, warp, lane) : out_warps<V, K, false>(w, map, warp, lane);
        } else {
            bf16 ? out_warps<K, V, true>(w, map, warp, lane) : out_warps<K, V, false>(w, map, warp, lane);
        }
        if (run_again(w, 0)) {
            if (w.sums) {
            } else if (turned) {
                bf16 ? out_warps<V, K, true>(w, map, warp, lane) : out_warps<V, K, false>(w, map, warp, lane);
            } else {
                bf16 ? out_warps<K, V, true>(w, map, warp, lane) : out_warps<K, V, false>(w, map, warp, lane);
            }
            run_again(w, 1);
        }
    } else if (warp < kLoadWarp) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
        turned ? state_warps<V, K, false>(w, warp - kStateWarp0, lane) : state_warps<K, V, false>(w, warp - kStateWarp0, lane);
        if (run_again(w, 0)) {
            turned ? state_warps<V, K, true>(w, warp - kStateWarp0, lane) : state_warps<K, V, true>(w, warp - kStateWarp0, lane);
            run_again(w, 1);
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        int pass = 0;
        do {
            if (lane == 0 && warp == kLoadWarp)
                turned ? load_warp<V, K, false>(w, &q.a[role], &q.b[role], &q.c[role], pass > 0 ? 0 : 2)
                       : load_warp<K, V, false>(w, &q.a[role], &q.b[role], &q.c[role], pass > 0 ? 0 : 2);
            if (lane == 0 && warp == kStoreWarp && !w.sums && w.r->out_bf16) {
                const CUtensorMap* map = &q.out[role];
                turned ? store_warp<K>(w, map) : store_warp<V>(w, map);
            }
            if (warp == kMmaWarp && !w.sums) turned ? intra_warp<V, K>(w, lane) : intra_warp<K, V>(w, lane);
            if (warp == kStateMmaWarp) turned ? state_mma_warp<V, K>(w, lane) : state_mma_warp<K, V>(w, lane);
        } while (run_again(w, pass++));
    }
    if (tid == 0 && *w.abort_flag) record_error(p.err, GDN_ERR_TIMEOUT, *w.abort_flag);
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(w.tmem), "r"(512u) : "memory");
}

// [tokens, heads, D]; box = 128 bytes of features x 1 head x `rows` tokens
bool tile_map(CUtensorMap* m, const void* ptr, bool bf16, int D, int heads, long long tokens, int rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t size = bf16 ? 2 : 4;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)D * size, (cuuint64_t)heads * D * size};
    cuuint32_t box[3] = {(cuuint32_t)(128 / size), 1, (cuuint32_t)rows};
    cuuint32_t es[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void*>(ptr), dims,
              strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int K, int V>
cudaError_t launch(const TcParams& q, cudaStream_t s) {
    static std::atomic<unsigned long long> set{0};   // devices on which the shared memory has been asked for
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(set.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(tc_kernel<K, V>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        if (dev < 64) set.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)q.p.blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = q.p.dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, tc_kernel<K, V>, q);
}

}  // namespace

bool tc_supported(const Params& p) {
    if (p.T == 0 || !encode_fn()) return false;
    for (int i = 0; i < p.nroles; ++i)
        if (!p.role[i].a_bf16 || !p.role[i].b_bf16 || !p.role[i].c_bf16) return false;
    return p.nroles == kMaxRoles || p.role[0].out_bf16;   // (gradients of shared heads leave as fp32, to be summed)
}

cudaError_t launch_tc(const Params* phases, int n, cudaStream_t s) {
    TcParams q;
    memset(&q, 0, sizeof q);
    const Params& p = phases[0];
    const long long tokens = p.cu ? p.T : (long long)p.nseq * p.T;
    // a tensor in several roles has one map
    struct Known {
        const void* ptr;
        int D, heads;
        const CUtensorMap* map;
    } known[4];
    int count = 0;
    auto load_map = [&](CUtensorMap* m, const void* ptr, int D, int heads) {
        for (int i = 0; i < count; ++i)
            if (known[i].ptr == ptr && known[i].D == D && known[i].heads == heads) {
                *m = *known[i].map;
                return true;
            }
        if (!tile_map(m, ptr, true, D, heads, tokens, kChunk)) return false;
        if (count < 4) known[count++] = Known{ptr, D, heads, m};
        return true;
    };
    for (int i = 0; i < p.nroles; ++i) {
        const Role& r = p.role[i];
        if (!load_map(&q.a[i], r.a, r.dA, r.a_heads) || !load_map(&q.b[i], r.b, r.dA, r.b_heads) ||
            !load_map(&q.c[i], r.c, r.dC, r.c_heads) ||
            !tile_map(&q.out[i], r.out, r.out_bf16, r.dC, p.H, tokens, r.out_bf16 ? kChunk : 32))
            return cudaErrorInvalidValue;
    }
    // (K, V: of the roles whose state is stored as it is)
    const bool t = p.role[0].state_t;
    const int K = t ? p.role[0].dC : p.role[0].dA, V = t ? p.role[0].dA : p.role[0].dC;
    cudaError_t e = cudaSuccess;
    for (int i = 0; i < n && e == cudaSuccess; ++i) {
        q.p = phases[i];
        if (K == 64)
            e = V == 64 ? launch<64, 64>(q, s) : launch<64, 128>(q, s);
        else
            e = V == 64 ? launch<128, 64>(q, s) : launch<128, 128>(q, s);
    }
    return e;
}

}  // namespace linear
}  // namespace gdn

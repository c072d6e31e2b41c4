// gdn_linear.cuh -- what the chunked kernels of linear attention with a decay for each head share: roles, pieces.
//
// One kernel serves the forward and the three gradients. With w = exp(decay[h]) it computes, along a sequence's tokens,
//   out_i = sum_{j <= i} w^(i - j) (a_i . b_j) c_j + w^(i + 1 - s) a_i X,   X' = w^n X + sum_j w^(n - 1 - j + s) b_j c_j^T
// from a start state X [dA, dC]. The forward is (a, b, c) = (q, k, v), s = 0, X the state. With D_t the gradient on the
// state after token t, D_t = w D_{t+1} + q_t dO_t^T, the gradients are dq_t = H_t dO_t, dk_t = D_t v_t, dv_t = k_t D_t,
// dh0 = w D_0, so that
//   dq is (dO, v, k), s = 0, from h0^T;
//   dk is (v, dO, q) and dv is (k, q, dO), s = 1, along the tokens from last to first, from dht^T and dht.
//
// Chunks of 128 tokens, counted from each sequence's first token, so that the last one may be shorter ("first" and
// "next" below follow the role's direction). A sequence's chunks are cut into pieces where its heads alone would leave SMs
// idle: piece 0 (`first` chunks) runs from the start state beside the sums U_p = sum_j w^.. b_j c_j^T of pieces 1 .. P-2;
// then pieces 1 .. P-1 run at once, each from the state that it joins from piece 0's last one and the sums before it.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "gdn_internal.h"

namespace gdn {
namespace linear {

constexpr int kChunk = 128;      // tokens
constexpr int kMaxRoles = 3;
constexpr float kLog2e = 1.4426950408889634f;

struct Role {
    const void *a, *b, *c;
    void* out;             // [tokens][H][dC]
    const float* start;    // [nseq][H] states, or null: zero
    float* last;           // receives the states behind the last token, or null
    int a_heads, b_heads, c_heads;   // head h of the rule reads head h / (H / heads)
    int a_bf16, b_bf16, c_bf16, out_bf16;
    int dA, dC;
    int rev;               // from the last token to the first; s = 1
    int state_t;           // start and last are stored [dC][dA]
};

// What a kernel block does: one piece of a chain, which is one sequence, head and role.
struct Item {
    int seq, h, role;
    int lo, len;           // the sequence's first token and length
    int piece, pieces;
    int m0, m1;            // its chunks, by number in the role's direction
    long long slot;        // state-sized places in the workspace: of piece p >= 1 at slot + (p - 1) slot_step, the state entering
    int slot_step;         // it (p = 1, written by piece 0), or the sum over piece p - 1
};

struct Params {
    Role role[kMaxRoles];
    int nroles;
    const float* decay;    // [H], natural log
    float* slots;
    const int* cu;         // packed batches; null: nseq sequences of T tokens
    const int* table;      // packed: the phase's entries, four ints each (sequence or -1, piece, pieces, slot of piece 1), all of
    const int* words;      // whose heads and roles are cut alike; and the words of the plan
    int nseq, T, H;
    int whole;             // not packed: chains before this number run in one piece, the others in `pieces`
    int first, rest, pieces;   // chunks of piece 0 and of the others (not packed)
    int phase;             // 1: piece 0 of every chain, sums of the middle pieces; 2: the other pieces
    int blocks;            // of the phase, by tiles
    int tiles;             // of the columns, of the role with the most of them
    int by_role;           // a sequence's chains in the order of their roles, not of their heads
    int dependent;         // launched while the grid before it still runs
    DeviceError* err;
};
// words of a packed batch's plan, in the workspace's header from kWsVerdict on: entries of the phases, tokens of all
// sequences, chunks of piece 0 and of the others
enum { kCount1 = 0, kCount2, kTokens, kFirst, kRest };

// What block number e of the phase does; false: nothing. It wants sums alone where 1 <= piece in phase 1.
__device__ __forceinline__ bool item_of(const Params& p, int e, Item& it, int& first, int& rest) {
    const int width = p.H * p.nroles;   // chains of a sequence
    int chain;
    if (p.cu) {
        const int entry = e / width;
        chain = e - entry * width;
        if (entry >= __ldcg(p.words + (p.phase == 1 ? kCount1 : kCount2))) return false;
        const int4 f = __ldcg(reinterpret_cast<const int4*>(p.table) + entry);
        if (f.x < 0) return false;
        it.seq = f.x;
        it.piece = f.y;
        it.pieces = f.z;
        it.slot = (long long)f.w * width + chain;
        it.slot_step = width;
        it.lo = __ldg(p.cu + it.seq);
        it.len = __ldg(p.cu + it.seq + 1) - it.lo;
        first = __ldcg(p.words + kFirst);
        rest = __ldcg(p.words + kRest);
    } else {
        const int chains = p.nseq * width;
        if (p.phase == 2) {
            chain = p.whole + e / (p.pieces - 1);
            it.piece = 1 + e % (p.pieces - 1);
        } else if (e < chains) {
            chain = e;
            it.piece = 0;
        } else {
            chain = p.whole + (e - chains) / (p.pieces - 2);
            it.piece = 1 + (e - chains) % (p.pieces - 2);
        }
        it.pieces = chain < p.whole ? 1 : p.pieces;
        it.slot = (long long)(chain - p.whole) * (p.pieces - 1);
        it.slot_step = 1;
        it.seq = chain / width;
        chain -= it.seq * width;
        it.lo = it.seq * p.T;
        it.len = p.T;
        first = p.first;
        rest = p.rest;
    }
    if (p.by_role) {
        it.role = chain / p.H;
        it.h = chain - it.role * p.H;
    } else {
        it.h = chain / p.nroles;
        it.role = chain - it.h * p.nroles;
    }
    const int n = (it.len + kChunk - 1) / kChunk;
    it.m0 = it.piece == 0 ? 0 : first + (it.piece - 1) * rest;
    it.m1 = it.piece == it.pieces - 1 ? n : first + it.piece * rest;
    return true;
}

// tokens of chunks m0 .. m1 - 1 (in the role's direction) of a sequence of len tokens
__device__ __forceinline__ int tokens_of(int m0, int m1, int len, int rev) {
    const int n = (len + kChunk - 1) / kChunk;
    const int a = rev ? n - m1 : m0, b = rev ? n - m0 : m1;
    return min(b * kChunk, len) - a * kChunk;
}

// log2 of a head's weight; decays beyond any that leaves a trace in fp32 (and -inf) are as good as -200
__device__ __forceinline__ float log2_weight(const float* decay, int h) {
    const float g = __ldg(decay + h);
    return (g < -200.f ? -200.f : g) * kLog2e;
}

// One launch for each of n phases.
cudaError_t launch_simt(const Params* phases, int n, cudaStream_t s);
bool tc_supported(const Params& p);
cudaError_t launch_tc(const Params* phases, int n, cudaStream_t s);

}  // namespace linear
}  // namespace gdn

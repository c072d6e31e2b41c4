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
    float* slots;          // workspace: [slot][H][dA][dC]; slot of piece p >= 1: the state entering it (p = 1, written by
                           // piece 0), or the sum over piece p - 1
    int a_heads, b_heads, c_heads;   // head h of the rule reads head h / (H / heads)
    int a_bf16, b_bf16, c_bf16, out_bf16;
    int dA, dC;
    int rev;               // from the last token to the first; s = 1
    int state_t;           // start and last are stored [dC][dA]
};

// One piece of one sequence, for a kernel block.
struct Item {
    int seq, lo, len;      // the sequence's first token and length
    int piece, pieces;
    int m0, m1;            // its chunks, by number in the role's direction
    int slot0;             // slot of piece 1
};

// A packed batch's pieces, made on the device: entries of kFields ints.
constexpr int kFields = 4;   // sequence, piece, pieces, slot0
struct Params {
    Role role[kMaxRoles];
    int nroles;
    const float* decay;    // [H], natural log
    const int* cu;         // packed batches; null: nseq sequences of T tokens
    const int* table;      // this phase's entries, and how many of them there are
    const int* count;
    int nseq, T, H;
    int first, rest;       // chunks of piece 0 and of the others
    int pieces;            // of every sequence, where the batch is not packed
    int phase;             // 1: piece 0 of every sequence, sums of the middle ones; 2: the other pieces
    int entries;           // grid: entries x H x tiles, by roles
    int tiles;             // of the columns, of the role with the most of them
    int dependent;         // launched while the grid before it still runs
    DeviceError* err;
};

// What entry e of the phase is; false: nothing. Whether it wants sums alone: 1 <= piece in phase 1.
__device__ __forceinline__ bool item_of(const Params& p, int e, Item& it) {
    if (p.cu) {
        if (e >= __ldcg(p.count)) return false;
        const int4 f = __ldcg(reinterpret_cast<const int4*>(p.table) + e);
        if (f.x < 0) return false;
        it.seq = f.x;
        it.piece = f.y;
        it.pieces = f.z;
        it.slot0 = f.w;
        it.lo = __ldg(p.cu + it.seq);
        it.len = __ldg(p.cu + it.seq + 1) - it.lo;
    } else {
        it.pieces = p.pieces;
        if (p.phase == 1) {
            it.seq = e;
            it.piece = 0;
            if (e >= p.nseq) {
                it.seq = (e - p.nseq) / (p.pieces - 2);
                it.piece = 1 + (e - p.nseq) % (p.pieces - 2);
            }
        } else {
            it.seq = e / (p.pieces - 1);
            it.piece = 1 + e % (p.pieces - 1);
        }
        it.slot0 = it.seq * (p.pieces - 1);
        it.lo = it.seq * p.T;
        it.len = p.T;
    }
    const int n = (it.len + kChunk - 1) / kChunk;
    it.m0 = it.piece == 0 ? 0 : p.first + (it.piece - 1) * p.rest;
    it.m1 = it.piece == it.pieces - 1 ? n : p.first + it.piece * p.rest;
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

// One launch of a phase.
cudaError_t launch_simt(const Params& p, cudaStream_t s);
bool tc_supported(const Params& p);
cudaError_t launch_tc(const Params& p, cudaStream_t s);

}  // namespace linear
}  // namespace gdn

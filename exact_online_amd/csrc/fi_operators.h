// fi_operators.h -- declarations shared by the host side of the operators
// around the mixers (fi_operators.cpp) and their kernels (fi_lattn.hip,
// fi_dense.hip, fi_scores.hip, fi_delta.hip, fi_rotary.hip, fi_verify.hip).  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fi {

// ------------------------------------------------------------ linear attention
struct View {
    void *p;
    int64_t row, pos, head;
};

// most B Hkv of a call: a launch has at most 2^32 threads, and 8 workgroups of 256 for each
constexpr int64_t kLattnMaxRows = (int64_t)1 << 20;

struct LattnCall {
    int64_t B, n_slots;
    int L, H, Hkv, G, dk, dv;   // G = H / Hkv
    float scale;
    int io_bf16, fresh;
    int vec;                    // every view loads whole 16-byte units
    const float *ld;            // [Hkv] log decay
    View q, k, v, o;
    const int32_t *lens, *slots;
    float *state;
    // the chunked form: segments of seg_chunks chunks, and (`entries`) their entry
    // states ws[B Hkv][nseg][dk][dv]
    int nseg, seg_chunks, entries;
    float *ws;
    int hsplit;                 // workgroups that share out a group's query heads
};

// One position (L = 1), recurrent form.
hipError_t launch_lattn_step(const LattnCall &c, hipStream_t st);
// Chunked form; ws holds lattn_ws_bytes, which is the most that plan_lattn makes any
// call of these sizes and smaller ones use.
hipError_t launch_lattn_chunk(LattnCall c, hipStream_t st);
void plan_lattn(LattnCall &c);   // segments, entry states, shares of query heads
size_t lattn_ws_used(const LattnCall &c);
size_t lattn_ws_bytes(int64_t B, int64_t L, int H, int Hkv, int dk, int dv, int io_bf16);

// ------------------------------------------------------------ dense product
// most M and N: a launch has at most 2^32 threads
constexpr int64_t kDenseMaxRows = (int64_t)1 << 27;

struct DenseCall {
    int64_t M, N, K;
    int io_bf16, out_bf16, act;
    const void *x, *w, *bias, *res;
    void *y;
    int64_t ldx, ldw, ldr, ldy;
    // a product split over K: parts of k_split, part[splits][M][ldp]
    float *part;
    int64_t k_split, ldp;
    int splits;
};

// Chooses the kernel; c.part holds dense_ws_bytes of the handle's M, N, K, the most
// that plan_dense makes a call of M rows or fewer use.
hipError_t launch_dense(DenseCall c, hipStream_t st);
void plan_dense(DenseCall &c);   // parts of K
size_t dense_ws_used(const DenseCall &c);
size_t dense_ws_bytes(int64_t M, int64_t N, int64_t K, int io_bf16);

// ------------------------------------------------------------ token scores
constexpr int kScoresMaxK = 32;

struct ScoresCall {
    int64_t rows, V, ld;
    int k, io_bf16;
    float scale;
    const void *logits;
    const int64_t *targets;
    float *logprob, *entropy, *lse, *top;
    int64_t *top_id;
    // a row's parts of `per` logits; of several: pst[rows][parts][3] and pkey[rows][parts][k]
    int parts;
    int64_t per;
    float *pst;
    unsigned long long *pkey;
};

hipError_t launch_scores(ScoresCall c, hipStream_t st);
void plan_scores(ScoresCall &c);   // a row's parts
size_t scores_ws_used(const ScoresCall &c);                      // rows x parts of a call
size_t scores_ws_parts(int64_t rows, int64_t V, int io_bf16);   // the most of any call of so many rows or fewer

// ------------------------------------------------------------ gated delta rule
struct DeltaCall {
    int64_t B, n_slots;
    int L, Hk, Hv, G, dk, dv;   // G = Hv / Hk
    float scale;
    int io_bf16, fresh, hold;
    int vec;                    // every view loads whole 16-byte units
    View q, k, v, o, ld, beta;
    const int32_t *lens, *slots;
    float *state;
    // the chunked form: chunks chunk0 .. chunk0 + chunks - 1 of every row at a time, in nseg segments of seg_chunks
    int chunk0, chunks, nseg, seg_chunks;
    int narrow;                 // slices of 64 columns where others have 128
    float *tri;                 // [B Hv][chunks] systems and gates (dl_floats each)
    float *ent, *move;          // of several segments: [B Hv][nseg][dk][dv] states before them, [B Hv][nseg][w][w] what they do to a
                                // state, w the keys of the kernel (dk, up to 64, 128 or 256)
    float *carry;               // [B Hv][dk][dv] states between two runs of chunks
};

// Recurrent form, position by position.
hipError_t launch_delta_step(const DeltaCall &c, hipStream_t st);
// Any number of positions; ws holds delta_ws_bytes, the most that plan_delta makes any call of these sizes and smaller ones use.
hipError_t launch_delta_prompt(DeltaCall c, float *ws, hipStream_t st);
enum class DeltaRoute { steps, few, chunks };
DeltaRoute delta_route(const DeltaCall &c);
void plan_delta(DeltaCall &c);   // chunks at a time, segments
void place_delta(DeltaCall &c, float *ws);   // a planned call's tri, ent, move and carry
size_t delta_ws_used(const DeltaCall &c);
size_t delta_ws_bytes(int64_t B, int64_t L, int Hv, int dk, int dv, int io_bf16);

// ------------------------------------------------------------ normed and turned heads
struct RotaryCall {
    int64_t B;
    int L, Hq, Hk, d, rot, norm, pairs, io_bf16;
    float eps;
    const double *turns;        // [rot / 2] turns of a position: inv_freq / 2 pi
    View q, k, qo, ko;
    const void *wq, *wk;
    const int32_t *first, *positions;
    int unit;                   // elements that every head and its halves load and store at once
    int shares;                 // waves that share out a position's heads
};

hipError_t launch_rotary(RotaryCall c, hipStream_t st);

// ------------------------------------------------------------ drafted tokens
constexpr int kVerifyMaxRows = 1 << 22;   // rows of logits of a call
constexpr double kVerifyOctave = 256 * 1.4426950408889634074;   // 256 log2 e

struct VerifyCall {
    int64_t B, V;
    int N, io_bf16;
    double scale, draft_scale;  // with kVerifyOctave
    const void *target, *draft;
    int64_t target_row, target_ld, draft_row, draft_ld;
    const int64_t *tokens;
    const int32_t *lens;
    const float *u, *r;
    int64_t *out;
    int32_t *kept;
    float *logprob;
    // a row's parts of `per` logits: sums[B (2 N + 1)][parts] of the probabilities against ref; its blocks of
    // `block` logits, shared out among `keepers` workgroups: rest[B][blocks] of what the token is drawn from
    int parts, blocks, keepers;
    int64_t per, block;
    double *sums, *ref, *rest;
};

hipError_t launch_verify(VerifyCall c, hipStream_t st);
void plan_verify(VerifyCall &c);   // a row's parts and blocks
size_t verify_ws_used(const VerifyCall &c);                            // doubles of a call
size_t verify_ws_doubles(int64_t B, int N, int64_t V);   // the most of any call of so many rows and drafts or fewer

}  // namespace fi

// fi_operators.h -- declarations shared by the host side of the operators
// around the mixers (fi_operators.cpp) and their kernels (fi_lattn.hip,
// fi_dense.hip, fi_scores.hip).  Not part of the public C ABI.
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

}  // namespace fi

// fi_dense.hip -- dense product with bias, activation and residual (fi_dense_*):
//     y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + res[m][n].
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

using V16 = float __attribute__((ext_vector_type(16)));

// act(v + bias) + res of W neighbouring outputs from (m, n), stored; `bias`
// holds theirs.
template <bool IO, int W>
__device__ __forceinline__ void dense_out(const DenseCall& a, int64_t m, int64_t n, const float* bias, float* v) {
    if (m >= a.M || n >= a.N) return;
    const int64_t left = a.N - n;
#pragma unroll
    for (int r = 0; r < W; ++r) v[r] += bias[r];
    if (a.act != 2)
#pragma unroll
        for (int r = 0; r < W; ++r) v[r] = activate(v[r], a.act);
    const auto store = [&](auto* y, const auto* q) {
        using T = std::remove_reference_t<decltype(*y)>;
        using Run = T __attribute__((ext_vector_type(W), aligned(sizeof(T))));
        if (left >= W) {
            Run t = {};
            if (a.res) t = *gmem(reinterpret_cast<const Run*>(q));
            if (a.res)
#pragma unroll
                for (int r = 0; r < W; ++r) v[r] += (float)t[r];
#pragma unroll
            for (int r = 0; r < W; ++r) t[r] = (T)v[r];
            *gmem(reinterpret_cast<Run*>(y)) = t;
        } else {
#pragma unroll
            for (int r = 0; r < W; ++r)
                if (r < left) gmem(y)[r] = (T)(v[r] + (a.res ? (float)gmem(q)[r] : 0.f));
        }
    };
    if (a.out_bf16) store(static_cast<BF*>(a.y) + m * a.ldy + n, static_cast<const BF*>(a.res) + m * a.ldr + n);
    else store(static_cast<float*>(a.y) + m * a.ldy + n, static_cast<const float*>(a.res) + m * a.ldr + n);
}

// bias[n .. n + W), zero beyond its end
template <bool IO, int W>
__device__ __forceinline__ void load_bias(const DenseCall& a, int64_t n, float* b) {
#pragma unroll
    for (int r = 0; r < W; ++r) b[r] = a.bias && n + r < a.N ? get_io<IO>(a.bias, n + r) : 0.f;
}

// ------------------------------------------------------------ tiles of many rows
// A workgroup of WM x WN waves has one BM x BN tile of y, a wave TM x TN
// products of 32 x 32; the products are taken as w x^T, so that a lane's
// results are neighbours in a row of y.

// Workgroups go round the 8 XCDs: each XCD gets one run of tiles, in which
// four rows of tiles go together along N (they share w in its L2).
template <int BM, int BN>
struct Tile {
    int64_t m0, n0, k0, k1;
    uint32_t split;
    __device__ __forceinline__ Tile(const DenseCall& a, uint32_t job) {
        const uint32_t tm = (uint32_t)((a.M + BM - 1) / BM), tn = (uint32_t)((a.N + BN - 1) / BN), tiles = tm * tn;
        const uint32_t at = job % tiles, per = tiles / 8, over = tiles % 8, xcd = at % 8;
        split = job / tiles;
        const uint32_t id = xcd * per + (xcd < over ? xcd : over) + at / 8;
        const uint32_t gm = id / (4 * tn) * 4, rows = tm - gm < 4 ? tm - gm : 4, in = id - gm * tn;
        m0 = (int64_t)(gm + in % rows) * BM;
        n0 = (int64_t)(in / rows) * BN;
        k0 = split * a.k_split;
        k1 = k0 + a.k_split < a.K ? k0 + a.k_split : a.K;
    }
};

// A wave's results, 32 rows at a time through its part of LDS (`out`, 32 rows
// of TN * 32), so that whole lines are stored.
template <bool IO, int TM, int TN>
__device__ __forceinline__ void dense_results(const DenseCall& a, int64_t m, int64_t n, uint32_t split, V16 (&acc)[TN][TM],
                                              float* out, uint32_t lane) {
    constexpr int UR = TN * 8, LANES = UR / 2, STEP = kWave / LANES;   // 16-byte units of a row; lanes, 8 results each; rows at once
    const auto unit_of = [](uint32_t row, uint32_t u) { return (row * UR + (u ^ (UR == 8 ? row / 2 % 8 : row % 16))) * 4; };
    const uint32_t l32 = lane % 32, half = lane / 32, row_ = lane / LANES, col = lane % LANES;
    float bias[8];
    load_bias<IO, 8>(a, n + col * 8, bias);
#pragma unroll
    for (int j = 0; j < TM; ++j) {
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
                *smem_ptr(reinterpret_cast<V4*>(out + unit_of(l32, 8 * i + 2 * q + half))) =
                    V4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        wave_order();
#pragma unroll 2
        for (int r = 0; r < 32; r += STEP) {
            const uint32_t row = r + row_;
            const V4 v0 = *smem_ptr(reinterpret_cast<const V4*>(out + unit_of(row, 2 * col)));
            const V4 v1 = *smem_ptr(reinterpret_cast<const V4*>(out + unit_of(row, 2 * col + 1)));
            float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
            const int64_t mm = m + 32 * j + row, nn = n + col * 8;
            if (a.splits == 1) dense_out<IO, 8>(a, mm, nn, bias, v);
            else if (mm < a.M && nn < a.ldp) {   // rows of `part` are a multiple of eight long
                V4* to = reinterpret_cast<V4*>(a.part + (split * a.M + mm) * a.ldp + nn);
                gmem(to)[0] = v0;
                gmem(to)[1] = v1;
            }
        }
        wave_order();
    }
}

// The products of a wave's TN x TM, `between(p)` after the p-th.
template <bool BF16, int TM, int TN, class F>
__device__ __forceinline__ void dense_mma(V16 (&acc)[TN][TM], const typename Mm<BF16>::Frag (&fw)[TN],
                                          const typename Mm<BF16>::Frag (&fx)[TM], F between) {
#pragma unroll
    for (int p = 0; p < TM * TN; ++p) {
        const int i = p / TM, j = p % TM;
        if constexpr (BF16) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[i], fx[j], acc[i][j], 0, 0, 0);
        else
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fw[i][e], fx[j][e], acc[i][j], 0, 0, 0);
        between(p);
    }
}

// Rows in whole 16-byte units.  K goes by in steps of 128 bytes of a row (half
// lines cost the L2 as much as whole ones), loaded straight into one of STAGES
// LDS buffers, STAGES - 1 steps ahead; a step has four parts, and the operands of each
// are read during the products of the one before.  A row's eight units are
// stored at u ^ (row / 2 % 8): the lanes that read one unit of 16 rows then
// meet every bank once.
//
// bf16, 256 x 256: 8192^3 888 us (1240 TFLOP/s, the library's 1411), 16384 x 4096
// x 1024 157 us, and 181 to 186 with bias and GELU.  The product itself keeps the
// matrix cores as busy as the power limit leaves them (clock 1.5 to 1.9 GHz);
// then a tile's end, which the next tile of the CU waits for: stores (128 KB of
// every CU at once: 7 us), GELU (17 operations and two transcendental ones for each
// output: 10 us a tile).  256 x 128 with steps of 64 bytes in three stages: 990
// TFLOP/s at 8192^3; 128 x 128, two on a CU: 1065, and 207 us (216 with GELU, which
// it hides) at 16384 x 4096 x 1024.  64 x 64 takes three stages, as its steps are
// short against the loads' way (1000^3: 9.2 us with two, 8.3 with three).
template <bool BF16, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM* WN * kWave, 2) void k_dense(DenseCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int E = M::E, U = 8, BK = U * E, NTH = WM * WN * kWave, ROWS = BM + BN;
    constexpr int UX = BM * U / NTH, UN = ROWS * U / NTH;      // units per thread: of x, of both
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    static_assert(UX * NTH == BM * U && UN * NTH == ROWS * U, "every thread loads the same");
    static_assert(WM * WN * 32 * TN * 32 * 4 <= STAGES * ROWS * U * 16, "the waves' results fit");
    __shared__ __align__(16) T lds[STAGES][ROWS * BK];

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t l32 = lane % 32, half = lane / 32;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    const Tile<BM, BN> t(a, blockIdx.x);
    // a unit's place: a wave's own base and the lane's offset in bytes (the
    // rows of a tile span less than 2^32)
    const char* const xb = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + t.m0 * a.ldx + t.k0);
    const char* const wb = reinterpret_cast<const char*>(static_cast<const T*>(a.w) + t.n0 * a.ldw + t.k0);
    uint32_t off[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        const int u = i * NTH + tid, unit = u % U ^ (u / U / 2 % U);
        const int64_t last = (i < UX ? a.M - t.m0 : a.N - t.n0) - 1;   // rows beyond the end are not stored
        int row = u / U - (i < UX ? 0 : BM);
        row = row < last ? row : (int)last;
        off[i] = ((uint32_t)row * (uint32_t)(i < UX ? a.ldx : a.ldw) + unit * E) * (uint32_t)sizeof(T);
    }
    // (the empty asm: the places stay a scalar base and a 32-bit offset, and are
    // not turned into 64-bit ones that are carried through the loop)
    const auto fetch_one = [&](int i, int k, int stage) {
        uint32_t o = off[i];
        asm volatile("" : "+v"(o));
        __builtin_amdgcn_global_load_lds((const FI_GLOBAL void*)((i < UX ? xb : wb) + (int64_t)k * (U * 16) + o),
                                         (FI_SHARED void*)(&lds[stage][(i * NTH + wave * kWave) * E]), 16, 0, 0);
    };
    V16 acc[TN][TM] = {};
    uint32_t lane_at = (l32 * U + (half ^ (l32 / 2 % U))) * 16;   // of part 0's unit in the lane's row
    // operand r of a part: w's first tile, x's tiles, w's other tiles (the order of their use)
    const auto read_one = [&](Frag (&fw)[TN], Frag (&fx)[TM], int r, int stage, int s) {
        const uint32_t at = (lane_at ^ (2 * s * 16)) + stage * (ROWS * U * 16);   // bytes
        const FI_SHARED char* p = smem_ptr(reinterpret_cast<const char*>(&lds[0][0])) + at;
        if (r == 0 || r > TM) {
            const int i = r == 0 ? 0 : r - TM;
            fw[i] = *reinterpret_cast<const FI_SHARED Frag*>(p + (BM + wn + 32 * i) * U * 16);
        } else fx[r - 1] = *reinterpret_cast<const FI_SHARED Frag*>(p + (wm + 32 * (r - 1)) * U * 16);
    };
    // The products of one part; behind each goes one read of the next part's
    // operands, in the first half of them, and (LOAD) a share of the loads of step
    // `load`: a product takes 32 cycles of the matrix pipe, which the wave's other
    // instructions fill.
    const auto part = [&](Frag (&cw)[TN], Frag (&cx)[TM], Frag (&nw)[TN], Frag (&nx)[TM], int stage, int s, auto LOAD, int load, int into) {
        asm volatile("" : "+v"(lane_at));   // one address a part, not all of them throughout
        constexpr int P = TM * TN, R = TM + TN, RP = (2 * R + P - 1) / P, FP = (UN + P - 1) / P;
        dense_mma<BF16, TM, TN>(acc, cw, cx, [&](int p) {
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int r = p * RP; r < (p + 1) * RP && r < R; ++r) read_one(nw, nx, r, stage, s);
            if constexpr (LOAD)
#pragma unroll
                for (int i = p * FP; i < (p + 1) * FP && i < UN; ++i) fetch_one(i, load, into);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // The wave's loads but the newest `left` steps' have arrived in LDS and its
    // reads of LDS are done, in every wave.  (Loads into LDS count as vector
    // memory operations and complete in order; a fence would wait for all.)
    const auto arrive = [](auto left) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(left * UN) : "memory");
    };
    using Some = std::integral_constant<int, STAGES - 2>;
    const int steps = (int)((t.k1 - t.k0) / BK), tail = (int)((t.k1 - t.k0) % BK);
    Frag w0[TN], x0[TM], w1[TN] = {}, x1[TM] = {};
    if (steps > 0) {
        // (beyond the end the last step's loads again: no branch, one count of loads)
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k)
#pragma unroll
            for (int i = 0; i < UN; ++i) fetch_one(i, k < steps ? k : steps - 1, k);
        arrive(Some{});
        using std::false_type;
        using std::true_type;
        int stage = 0, into = STAGES - 1;   // buffers of step k and of the step that is loaded during it
        for (int k = 0; k < steps; ++k) {
            // the last part of step k - 1, and loads into that step's buffer
            part(w1, x1, w0, x0, stage, 0, true_type{}, k + STAGES - 1 < steps ? k + STAGES - 1 : steps - 1, into);
            part(w0, x0, w1, x1, stage, 1, false_type{}, 0, 0);
            part(w1, x1, w0, x0, stage, 2, false_type{}, 0, 0);
            part(w0, x0, w1, x1, stage, 3, false_type{}, 0, 0);
            arrive(Some{});
            into = stage;
            stage = stage == STAGES - 1 ? 0 : stage + 1;
        }
        arrive(std::integral_constant<int, 0>{});
    }
    const auto nothing = [](int) {};
    dense_mma<BF16, TM, TN>(acc, w1, x1, nothing);
    if (tail) {   // the last, shorter step
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int u = i * NTH + tid, unit = u % U ^ (u / U / 2 % U);
            const Frag f = load_loose<BF16>(reinterpret_cast<const T*>((i < UX ? xb : wb) + (int64_t)steps * (U * 16) + off[i]), 0, tail - unit * E);
            *smem_ptr(reinterpret_cast<Frag*>(&lds[0][u * E])) = f;
        }
        team_sync();
#pragma unroll 1
        for (int s = 0; s < U / 2; ++s) {
#pragma unroll
            for (int r = 0; r < TM + TN; ++r) read_one(w0, x0, r, 0, s);
            dense_mma<BF16, TM, TN>(acc, w0, x0, nothing);
        }
        team_sync();
    }
    dense_results<BF16, TM, TN>(a, t.m0 + wm, t.n0 + wn, t.split, acc,
                                reinterpret_cast<float*>(&lds[0][0]) + wave * 32 * TN * 32, lane);
}

// Rows at any alignment: K in steps of 128 bytes through registers into two
// LDS buffers (a row's eight units at u ^ (row / 2 % 8)).  Two steps are in flight
// in registers (one: 53 us where this takes 41 to 47, 1777 x 1025 x 999, fp32, with bias and
// residual; 88 of fp32's 154 TFLOP/s: with 476 tiles a CU has one or two, and
// their start and end show).
template <bool BF16, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * kWave) void k_dense_loose(DenseCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int E = M::E, U = 8, BK = U * E, NTH = WM * WN * kWave, ROWS = BM + BN;
    constexpr int UX = BM * U / NTH, UN = ROWS * U / NTH;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    __shared__ __align__(16) T lds[2][ROWS * BK];

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t l32 = lane % 32, half = lane / 32;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    const Tile<BM, BN> t(a, blockIdx.x);
    const T* row[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        const int u = i * NTH + tid;
        const int64_t r = i < UX ? t.m0 + u / U : t.n0 + u / U - BM, last = (i < UX ? a.M : a.N) - 1;   // rows beyond the end are not stored
        row[i] = static_cast<const T*>(i < UX ? a.x : a.w) + (r < last ? r : last) * (i < UX ? a.ldx : a.ldw) + t.k0 +
                 (u % U ^ (u / U / 2 % U)) * E;
    }
    using Loose = T __attribute__((ext_vector_type(E), aligned(sizeof(T))));
    Frag hold[2][UN];   // two steps in flight
    const auto fetch = [&](Frag (&h)[UN], int k) {   // a whole step: no branch, so that nothing waits for the loads before their use
#pragma unroll
        for (int i = 0; i < UN; ++i) h[i] = *gmem(reinterpret_cast<const Loose*>(row[i] + (int64_t)k * BK));
    };
    const auto settle = [&](const Frag (&h)[UN], int buf) {
#pragma unroll
        for (int i = 0; i < UN; ++i) *smem_ptr(reinterpret_cast<Frag*>(&lds[buf][(i * NTH + tid) * E])) = h[i];
    };
    V16 acc[TN][TM] = {};
    const auto products = [&](int buf) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            Frag fw[TN], fx[TM];
            const uint32_t unit = (2 * s + half) ^ (l32 / 2 % U);
#pragma unroll
            for (int i = 0; i < TN; ++i)
                fw[i] = *smem_ptr(reinterpret_cast<const Frag*>(&lds[buf][((BM + wn + 32 * i + l32) * U + unit) * E]));
#pragma unroll
            for (int i = 0; i < TM; ++i)
                fx[i] = *smem_ptr(reinterpret_cast<const Frag*>(&lds[buf][((wm + 32 * i + l32) * U + unit) * E]));
            dense_mma<BF16, TM, TN>(acc, fw, fx, [](int) {});
        }
    };
    const int steps = (int)((t.k1 - t.k0) / BK), tail = (int)((t.k1 - t.k0) % BK);
    const auto some = [&](int k) { return k < steps ? k : steps - 1; };
    if (steps > 0) {
        fetch(hold[0], 0);
        fetch(hold[1], some(1));
        settle(hold[0], 0);
        fetch(hold[0], some(2));
        for (int k = 0; k < steps; k += 2) {
            team_sync();
            products(0);
            settle(hold[1], 1);
            fetch(hold[1], some(k + 3));
            team_sync();
            if (k + 1 < steps) products(1);
            settle(hold[0], 0);
            fetch(hold[0], some(k + 4));
        }
        team_sync();
    }
    if (tail) {   // the last, shorter step
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int u = i * NTH + tid;
            hold[0][i] = load_loose<BF16>(row[i] + (int64_t)steps * BK, 0, tail - (u % U ^ (u / U / 2 % U)) * E);
        }
        settle(hold[0], 0);
        team_sync();
        products(0);
    }
    team_sync();
    dense_results<BF16, TM, TN>(a, t.m0 + wm, t.n0 + wn, t.split, acc,
                                reinterpret_cast<float*>(&lds[0][0]) + wave * 32 * TN * 32, lane);
}

// The parts of a product split over K, summed in their order.
template <bool IO>
__global__ __launch_bounds__(256) void k_dense_join(DenseCall a) {
    const int64_t per = a.ldp / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.M * per) return;
    const int64_t m = i / per, n = i % per * 8;
    V4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = s0;
    for (int s = 0; s < a.splits; ++s) {
        const V4* p = reinterpret_cast<const V4*>(a.part + (s * a.M + m) * a.ldp + n);
        s0 += gmem(p)[0];
        s1 += gmem(p)[1];
    }
    float v[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w}, bias[8];
    load_bias<IO, 8>(a, n, bias);
    dense_out<IO, 8>(a, m, n, bias, v);
}

// ------------------------------------------------------------ few rows
// Up to 16 MT rows of x: w goes by once, from memory to the matrix cores'
// operands; KW waves of a workgroup split K of 16 outputs between them.  Bound
// by w: one row, 32768 x 1024, bf16: 11.9 us (5.6 TB/s: some of w is still in the
// last-level cache), 131072 x 1024: 40 us (6.7 TB/s).  Eight steps' loads (four with
// sixteen waves) are in flight at once.  (For 17 to 32 rows that is more than the 128
// registers of a lane of sixteen waves: 22 of them go to scratch, and the figures at
// few_rows are measured so.)
template <bool BF16, int MT, int KW, bool ALIGNED>
__global__ __launch_bounds__((KW > 4 ? KW : 4) * kWave) void k_dense_few(DenseCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int WAVES = KW > 4 ? KW : 4, TILES = WAVES / KW, UNROLL = KW > 4 ? 4 : 8;
    __shared__ V4 red[WAVES][MT][kWave];
    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, l16 = lane % 16, g = lane / 16;
    const int part = wave % KW;
    const int64_t n0 = ((int64_t)blockIdx.x * TILES + wave / KW) * 16;
    const int64_t n = n0 + l16 < a.N ? n0 + l16 : a.N - 1;   // outputs beyond the end are not stored
    const T* w = static_cast<const T*>(a.w) + n * a.ldw;
    const T* x[MT];
    bool xin[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        xin[i] = 16 * i + l16 < a.M;
        x[i] = static_cast<const T*>(a.x) + (xin[i] ? 16 * i + l16 : 0) * a.ldx;
    }
    V4 acc[MT] = {};
    const int64_t steps = (a.K + M::KB - 1) / M::KB, s0 = steps * part / KW, s1 = steps * (part + 1) / KW;
    const auto sweep = [&](auto load) {
        for (int64_t s = s0; s < s1; s += UNROLL) {
            Frag fw[UNROLL], fx[UNROLL][MT];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int64_t k = (s + u) * M::KB + g * M::E;
                fw[u] = load(w, k, s + u < s1);
#pragma unroll
                for (int i = 0; i < MT; ++i) fx[u][i] = load(x[i], k, s + u < s1 && xin[i]);
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u)
#pragma unroll
                for (int i = 0; i < MT; ++i) acc[i] = M::mma(fw[u], fx[u][i], acc[i]);
        }
    };
    if (n0 < a.N) {
        using Words = T __attribute__((ext_vector_type(M::E), aligned(4)));
        uintptr_t low = reinterpret_cast<uintptr_t>(w);
#pragma unroll
        for (int i = 0; i < MT; ++i) low |= reinterpret_cast<uintptr_t>(x[i]);
        if constexpr (ALIGNED)   // K is whole units
            sweep([&](const T* p, int64_t k, bool in) { return in && k < a.K ? *gmem(reinterpret_cast<const Frag*>(p + k)) : Frag{}; });
        // otherwise the last unit comes after the loop
        else if (!BF16 || !__any(low % 4 != 0))
            sweep([&](const T* p, int64_t k, bool in) -> Frag { return in && k + M::E < a.K ? Frag(*gmem(reinterpret_cast<const Words*>(p + k))) : Frag{}; });
        else sweep([&](const T* p, int64_t k, bool in) { return in && k + M::E < a.K ? load_by_words<BF16>(p + k) : Frag{}; });
    }
    if (!ALIGNED && part == KW - 1 && n0 < a.N) {
        const int64_t k = (a.K - 1) / M::E * M::E;
        const bool here = k % M::KB / M::E == g;   // the lanes whose unit it is
        Frag fw = {};
        if (here) fw = load_loose<BF16>(w, k, a.K);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            Frag fx = {};
            if (here && xin[i]) fx = load_loose<BF16>(x[i], k, a.K);
            acc[i] = M::mma(fw, fx, acc[i]);
        }
    }
    if constexpr (KW > 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[i];
        __syncthreads();
        if (part) return;
        for (int p = 1; p < KW; ++p)
#pragma unroll
            for (int i = 0; i < MT; ++i) acc[i] += red[wave + p][i][lane];
    }
    if (n0 < a.N)
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            float v[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w}, bias[4];
            load_bias<BF16, 4>(a, n0 + 4 * g, bias);
            dense_out<BF16, 4>(a, 16 * i + l16, n0 + 4 * g, bias, v);
        }
}

namespace {

constexpr int64_t kCus = 256;

int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

template <bool BF16, int MT, int KW>
void few(const DenseCall& c, bool direct, hipStream_t st) {
    constexpr int WAVES = KW > 4 ? KW : 4;
    const int64_t tiles = (c.N + 15) / 16;
    const unsigned grid = (unsigned)((tiles + WAVES / KW - 1) / (WAVES / KW));
    if (direct) k_dense_few<BF16, MT, KW, true><<<grid, WAVES * kWave, 0, st>>>(c);
    else k_dense_few<BF16, MT, KW, false><<<grid, WAVES * kWave, 0, st>>>(c);
}

template <bool BF16, int BM, int BN, int WM, int WN, int STAGES>
void tile(const DenseCall& c, bool direct, hipStream_t st) {
    const unsigned grid = (unsigned)(tiles_of(c.M, c.N, BM, BN) * c.splits);
    if (direct) k_dense<BF16, BM, BN, WM, WN, STAGES><<<grid, WM * WN * kWave, 0, st>>>(c);
    else k_dense_loose<BF16, BM, BN, WM, WN><<<grid, WM * WN * kWave, 0, st>>>(c);
    if (c.splits > 1)
        k_dense_join<BF16><<<(unsigned)((c.M * (c.ldp / 8) + 255) / 256), 256, 0, st>>>(c);
}

// Rows that k_dense_few takes: 16 at any size, and 32 where w is small (32
// rows, us here / in tiles: 4096 x 1024 6.4 / 7.1, but 2048 x 4096 14.5 / 10.6
// and 32768 x 1024 24.1 / 16.6: x is read again by every 16 outputs).
bool few_rows(int64_t M, int64_t N, int64_t K) { return M <= 16 || (M <= 32 && N < 8192 && K <= 2048); }

// Parts that K is split into, where tiles of 64 x 64 are fewer than half the
// CUs: at least 1024 long each (fp32, whose products take eight times as long,
// 256), as the join costs as much as some 600 of bf16's K.  us, 64 rows by
// 4096, bf16, whole / in parts: K = 1024 7.5 / 12.5, 2048 11.1 / 11.1, 8192 34 /
// 19.6; 256 rows by 1024, bf16, K = 4096, parts of 512 / 1024 / 2048: 14.8 / 12.8 /
// 14.6; 200 rows by 1000, fp32, K = 1000, parts of 128 / 256 / whole: 16.5 / 15.1 /
// 25.2; 41 rows by 256, fp32, K = 3904, parts of 256 / 512 / 1024: 15.2 / 19.1 / 32.6.
int64_t splits_of(int64_t M, int64_t N, int64_t K, bool io_bf16) {
    const int64_t t = tiles_of(M, N, 64, 64);
    if (few_rows(M, N, K) || 2 * t > kCus) return 1;
    int64_t n = 2 * kCus / t;
    const int64_t most = K / (io_bf16 ? 1024 : 256);
    if (n > most) n = most;
    return n < 1 ? 1 : n;
}

// The time of a launch in rounds over the CUs, which hold at most `at_once`
// workgroups each: a round with i on a CU costs cost[i], measured with K =
// 1024, in hundredths of bf16's round of 256 x 256 tiles (36 us) and of fp32's
// two 128 x 128 tiles on a CU (150 us; fp32 keeps the matrix cores busy with
// fewer).  us by 256 x 256 / 128 x 128 / 128 x 64 / 64 x 64: bf16 4096 x 4096 37.6 / 41.7 /
// - / 61.0, 2048 x 4096 35.0 / 22.5 / 32.0 / 37.4, 2048 x 2048 27.7 / 15.1 / 13.6 / 19.0, 1024 x
// 1024 25.7 / 12.7 / 12.1 / 8.8, 3000 x 3000 36.6 / 46.4 / 42.1 / 50.3; fp32 2048 x 2048 240 / 74.5 /
// 77.8 / 92.8, 2500 x 1500 245 / 75.6 / 71.7 / 88.3, 1777 x 1025 241 / 71.3 / 44.8 / 44.2.
// (Unaligned rows go by 128 x 128 and 64 x 64 only: bf16's 2048 x 2048 x 1023 28.0 /
// 33.1 / 43.9 from 128 x 128 on.)
struct TileSize {
    int m, n, at_once, cost[2][4];   // of fp32, of bf16
};
constexpr TileSize kTiles[] = {{64, 64, 3, {{0, 17, 28, 40}, {0, 22, 27, 38}}},
                               {128, 128, 2, {{0, 50, 93}, {0, 42, 58}}},
                               {128, 64, 3, {{0, 29, 52, 70}, {0, 30, 38, 62}}},
                               {256, 256, 1, {{0, 156}, {0, 100}}}};
int best_tile(int64_t M, int64_t N, bool io_bf16, bool direct) {   // the largest of the cheapest
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < (direct ? 4 : 2); ++i) {
        const TileSize& t = kTiles[i];
        const int* cost = t.cost[io_bf16];
        const int64_t tiles = tiles_of(M, N, t.m, t.n), round = t.at_once * kCus;
        const int64_t all = tiles / round * cost[t.at_once] + cost[(tiles % round + kCus - 1) / kCus];
        if (all <= least) {
            least = all;
            best = i;
        }
    }
    return best;
}

template <bool BF16>
hipError_t run(const DenseCall& c, hipStream_t st) {
    constexpr int E = BF16 ? 8 : 4;
    const auto whole = [](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % E == 0 && ld < (1 << 21); };
    const bool direct = whole(c.x, c.ldx) && whole(c.w, c.ldw);
    if (few_rows(c.M, c.N, c.K)) {
        const bool al = direct && c.K % E == 0;
        // 16 outputs for one wave, or for four or sixteen where there are fewer than
        // some eight waves for each CU (one row, us by 1 / 4 / 16: 131072 x 100
        // 9.2 / 18.0 / -, 32768 x 1024 12.2 / 12.1 / 17.8, 16384 x 1024 7.9 / 6.9 /
        // 8.9, 4096 x 4096 24.5 / 7.7 / 7.1)
        const int64_t t = (c.N + 15) / 16;
        if (c.M > 16) few<BF16, 2, 16>(c, al, st);
        else if (t >= 8 * kCus) few<BF16, 1, 1>(c, al, st);
        else if (t >= 2 * kCus) few<BF16, 1, 4>(c, al, st);
        else few<BF16, 1, 16>(c, al, st);
        return hipGetLastError();
    }
    switch (c.splits > 1 ? 0 : best_tile(c.M, c.N, BF16, direct)) {
        case 0: tile<BF16, 64, 64, 2, 2, 3>(c, direct, st); break;
        case 1: tile<BF16, 128, 128, 2, 2, 2>(c, direct, st); break;
        case 2: k_dense<BF16, 128, 64, 2, 2, 2><<<(unsigned)tiles_of(c.M, c.N, 128, 64), 4 * kWave, 0, st>>>(c); break;
        default: k_dense<BF16, 256, 256, 2, 4, 2><<<(unsigned)tiles_of(c.M, c.N, 256, 256), 8 * kWave, 0, st>>>(c);
    }
    return hipGetLastError();
}

}  // namespace

void plan_dense(DenseCall& c) {
    const int64_t n = splits_of(c.M, c.N, c.K, c.io_bf16), step = c.io_bf16 ? 64 : 32;   // K in whole steps of 128 bytes
    c.ldp = (c.N + 7) / 8 * 8;
    c.k_split = n > 1 ? ((c.K + n - 1) / n + step - 1) / step * step : c.K;
    c.splits = (int)((c.K + c.k_split - 1) / c.k_split);
    if (c.splits == 1) c.part = nullptr;
}

size_t dense_ws_used(const DenseCall& c) { return c.splits > 1 ? (size_t)c.splits * c.M * c.ldp * sizeof(float) : 0; }

size_t dense_ws_bytes(int64_t M, int64_t N, int64_t K, int io_bf16) {
    int64_t most = 0;
    for (int64_t m = 64; m - 63 <= M; m += 64) {   // the parts depend on the number of tile rows
        const int64_t rows = m < M ? m : M, n = splits_of(rows, N, K, io_bf16);
        if (tiles_of(m, N, 64, 64) * 2 > kCus) break;
        if (n > 1 && n * rows > most) most = n * rows;
    }
    return (size_t)(most * ((N + 7) / 8 * 8)) * sizeof(float);
}

hipError_t launch_dense(DenseCall c, hipStream_t st) {
    plan_dense(c);
    return c.io_bf16 ? run<true>(c, st) : run<false>(c, st);
}

}  // namespace fi

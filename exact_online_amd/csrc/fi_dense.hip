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
// A workgroup of WM x WN waves has a BM x BN tile of y at a time; K goes by in
// steps of 128 bytes of a row, two LDS buffers, the next step's loads in
// flight during a step's products (the next tile's first step during a tile's
// last results).  A row's eight 16-byte units are stored at u ^ (row / 2 % 8):
// the 16 lanes that read one unit of 16 rows then meet every bank once.  The
// products are taken as w x^T, so that a lane's results are neighbours in a
// row of y; they go through LDS once more, so that whole lines are stored.
template <bool BF16, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM* WN * kWave) void k_dense(DenseCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int E = M::E, BK = 8 * E, NTH = WM * WN * kWave, ROWS = BM + BN;
    constexpr int UX = BM * 8 / NTH, UN = ROWS * 8 / NTH;      // units per thread: of x, of both
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;        // 32 x 32 products of a wave
    constexpr int UR = TN * 8;                                 // 16-byte units of a wave's row of results
    static_assert(WM * WN * 32 * UR * 16 <= ROWS * BK * (int)sizeof(T), "the waves' results fit one buffer");
    __shared__ __align__(16) T lds[2][ROWS * BK];

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t l32 = lane % 32, half = lane / 32;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN, tiles = tm * tn, all = tiles * a.splits;
    int64_t m0, n0, k0, k1, split;
    // a unit's place: a wave's own base and the lane's offset in bytes (DIRECT:
    // the rows of a tile span less than 2^32)
    using Off = std::conditional_t<DIRECT, uint32_t, int64_t>;
    const char *xb, *wb;
    Off off[UN];
    // workgroups go round the 8 XCDs: each XCD gets one run of tiles, in which
    // four rows of tiles go together along N (they share w in its L2)
    const auto place = [&](int64_t job) {
        const int64_t at = job % tiles, per = tiles / 8, over = tiles % 8, xcd = at % 8;
        split = job / tiles;
        const int64_t id = xcd * per + (xcd < over ? xcd : over) + at / 8;
        const int64_t gm = id / (4 * tn) * 4, rows = tm - gm < 4 ? tm - gm : 4, in = id - gm * tn;
        m0 = (gm + in % rows) * BM;
        n0 = in / rows * BN;
        k0 = split * a.k_split;
        k1 = k0 + a.k_split < a.K ? k0 + a.k_split : a.K;
        xb = reinterpret_cast<const char*>(static_cast<const T*>(a.x) + m0 * a.ldx);
        wb = reinterpret_cast<const char*>(static_cast<const T*>(a.w) + n0 * a.ldw);
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int u = i * NTH + tid, unit = u % 8 ^ (u / 16 % 8);
            int row = u / 8 - (i < UX ? 0 : BM);
            const int64_t last = (i < UX ? a.M - m0 : a.N - n0) - 1;   // rows beyond the end are not stored
            row = row < last ? row : (int)last;
            off[i] = ((Off)row * (Off)(i < UX ? a.ldx : a.ldw) + unit * E) * (Off)sizeof(T);
        }
    };
    Frag hold[UN];
    const auto whole = [&](int64_t k) { return DIRECT && k + BK <= k1; };
    const auto fetch = [&](int64_t k, int buf) {
        if (whole(k)) {
#pragma unroll
            for (int i = 0; i < UN; ++i)
                __builtin_amdgcn_global_load_lds((const FI_GLOBAL void*)((i < UX ? xb : wb) + k * (int)sizeof(T) + off[i]),
                                                 (FI_SHARED void*)(&lds[buf][(i * NTH + wave * kWave) * E]), 16, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int u = i * NTH + tid, unit = u % 8 ^ (u / 8 / 2 % 8);
                hold[i] = load_loose<BF16>(reinterpret_cast<const T*>((i < UX ? xb : wb) + off[i]) + k, 0, k1 - k - unit * E);
            }
        }
    };
    const auto settle = [&](int64_t k, int buf) {
        if (whole(k)) return;
#pragma unroll
        for (int i = 0; i < UN; ++i) *smem_ptr(reinterpret_cast<Frag*>(&lds[buf][(i * NTH + tid) * E])) = hold[i];
    };
    int buf = 0;
    int64_t job = blockIdx.x;
    place(job);
    fetch(k0, 0);
    while (true) {
        settle(k0, buf);
        V16 acc[TN][TM] = {};
        for (int64_t k = k0; k < k1; k += BK, buf ^= 1) {
            __syncthreads();
            const bool more = k + BK < k1;
            if (more) fetch(k + BK, buf ^ 1);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                Frag fw[TN], fx[TM];
#pragma unroll
                for (int i = 0; i < TN; ++i) {
                    const uint32_t row = BM + wn + 32 * i + l32;
                    fw[i] = *smem_ptr(reinterpret_cast<const Frag*>(&lds[buf][(row * 8 + ((2 * s + half) ^ (l32 / 2 % 8))) * E]));
                }
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    const uint32_t row = wm + 32 * i + l32;
                    fx[i] = *smem_ptr(reinterpret_cast<const Frag*>(&lds[buf][(row * 8 + ((2 * s + half) ^ (l32 / 2 % 8))) * E]));
                }
#pragma unroll
                for (int i = 0; i < TN; ++i)
#pragma unroll
                    for (int j = 0; j < TM; ++j) {
                        if constexpr (BF16) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fw[i], fx[j], acc[i][j], 0, 0, 0);
                        else
#pragma unroll
                            for (int e = 0; e < 4; ++e) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fw[i][e], fx[j][e], acc[i][j], 0, 0, 0);
                    }
            }
            if (more) settle(k + BK, buf ^ 1);
        }
        // buf is the buffer of the step before the last one, free for the next
        // tile since the last step's barrier; the last step's takes the results
        const int64_t m = m0 + wm, n = n0 + wn, part = split;
        job += gridDim.x;
        const bool next = job < all;
        if (next) {
            place(job);
            if (whole(k0)) fetch(k0, buf);
        }
        __syncthreads();
        float* const out = reinterpret_cast<float*>(lds[buf ^ 1]) + wave * 32 * UR * 4;
        const auto unit_of = [](uint32_t row, uint32_t u) { return (row * UR + (u ^ (UR == 8 ? row / 2 % 8 : row % 16))) * 4; };
        constexpr int LANES = UR / 2, STEP = kWave / LANES;   // lanes of a row, 8 results each; rows of an instruction
        const uint32_t row_ = lane / LANES, col = lane % LANES;
        float bias[8];
        load_bias<BF16, 8>(a, n + col * 8, bias);
#pragma unroll
        for (int j = 0; j < TM; ++j) {
#pragma unroll
            for (int i = 0; i < TN; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *smem_ptr(reinterpret_cast<V4*>(out + unit_of(l32, 8 * i + 2 * q + half))) =
                        V4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
            // a wave's LDS operations are performed in order
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll 1
            for (int r = 0; r < 32; r += STEP) {
                const uint32_t row = r + row_;
                const V4 v0 = *smem_ptr(reinterpret_cast<const V4*>(out + unit_of(row, 2 * col)));
                const V4 v1 = *smem_ptr(reinterpret_cast<const V4*>(out + unit_of(row, 2 * col + 1)));
                float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
                const int64_t mm = m + 32 * j + row, nn = n + col * 8;
                if (a.splits == 1) dense_out<BF16, 8>(a, mm, nn, bias, v);
                else if (mm < a.M) {   // rows of `part` are a multiple of eight long
                    V4* to = reinterpret_cast<V4*>(a.part + (part * a.M + mm) * a.ldp + nn);
                    if (nn < a.ldp) {
                        gmem(to)[0] = v0;
                        gmem(to)[1] = v1;
                    }
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
        if (!next) return;
        if (!whole(k0)) fetch(k0, buf);
    }
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
// operands; KW waves of a workgroup split K of 16 outputs between them.
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
    const auto load = [&](const T* p, int64_t k, bool in) -> Frag {
        if (!in) return Frag{};
        if constexpr (ALIGNED) return k < a.K ? *gmem(reinterpret_cast<const Frag*>(p + k)) : Frag{};   // K is whole units
        else return load_loose<BF16>(p, k, a.K);
    };
    V4 acc[MT] = {};
    const int64_t steps = (a.K + M::KB - 1) / M::KB, s0 = steps * part / KW, s1 = steps * (part + 1) / KW;
    if (n0 < a.N)
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

template <bool BF16, int MT, int KW>
void few(const DenseCall& c, bool direct, hipStream_t st) {
    constexpr int WAVES = KW > 4 ? KW : 4;
    const int64_t tiles = (c.N + 15) / 16;
    const unsigned grid = (unsigned)((tiles + WAVES / KW - 1) / (WAVES / KW));
    if (direct) k_dense_few<BF16, MT, KW, true><<<grid, WAVES * kWave, 0, st>>>(c);
    else k_dense_few<BF16, MT, KW, false><<<grid, WAVES * kWave, 0, st>>>(c);
}

constexpr int64_t kCus = 256;

template <bool BF16, int BM, int BN, int WM, int WN>
void tile(const DenseCall& c, bool direct, hipStream_t st) {
    const int64_t jobs = ((c.M + BM - 1) / BM) * ((c.N + BN - 1) / BN) * c.splits;
    constexpr int64_t kRoom = kCus * (BM == 256 ? 1 : BM == 128 ? 2 : 4);   // workgroups that are resident together
    const unsigned grid = (unsigned)(jobs < kRoom ? jobs : kRoom);
    if (direct) k_dense<BF16, BM, BN, WM, WN, true><<<grid, WM * WN * kWave, 0, st>>>(c);
    else k_dense<BF16, BM, BN, WM, WN, false><<<grid, WM * WN * kWave, 0, st>>>(c);
    if (c.splits > 1)
        k_dense_join<BF16><<<(unsigned)((c.M * (c.ldp / 8) + 255) / 256), 256, 0, st>>>(c);
}

constexpr int64_t kFewRows = 32;
constexpr int64_t kMinSplitK = 256;    // of K, for one part

int64_t tiles_of(int64_t M, int64_t N, int bm, int bn) { return ((M + bm - 1) / bm) * ((N + bn - 1) / bn); }

// parts that K of a product of M rows is split into (tiles of 64 x 64)
int64_t splits_of(int64_t M, int64_t N, int64_t K) {
    const int64_t t = tiles_of(M, N, 64, 64);
    if (M <= kFewRows || 2 * t > kCus) return 1;
    int64_t n = 2 * kCus / t;
    if (n > K / kMinSplitK) n = K / kMinSplitK;
    return n < 1 ? 1 : n;
}

template <bool BF16>
hipError_t run(DenseCall& c, hipStream_t st) {
    constexpr int es = BF16 ? 2 : 4, E = 16 / es, BK = 8 * E;
    const auto whole = [](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % E == 0 && ld < (1 << 21); };
    const bool direct = whole(c.x, c.ldx) && whole(c.w, c.ldw);
    c.splits = 1;
    c.k_split = c.K;
    if (c.M <= kFewRows) {
        c.part = nullptr;
        const bool al = direct && c.K % E == 0;
        const int64_t t = (c.N + 15) / 16;   // 16 outputs each: one wave, or four or sixteen, for some eight waves per CU
        if (c.M <= 16) {
            if (t >= 8 * kCus) few<BF16, 1, 1>(c, al, st);
            else if (t >= 2 * kCus) few<BF16, 1, 4>(c, al, st);
            else few<BF16, 1, 16>(c, al, st);
        } else {
            if (t >= 8 * kCus) few<BF16, 2, 1>(c, al, st);
            else if (t >= 2 * kCus) few<BF16, 2, 4>(c, al, st);
            else few<BF16, 2, 16>(c, al, st);
        }
        return hipGetLastError();
    }
    const int64_t n = splits_of(c.M, c.N, c.K);
    if (n > 1) {
        c.k_split = ((c.K + n - 1) / n + BK - 1) / BK * BK;
        c.splits = (int)((c.K + c.k_split - 1) / c.k_split);
    }
    if (c.splits == 1) c.part = nullptr;
    if (c.splits > 1 || tiles_of(c.M, c.N, 128, 128) < kCus) tile<BF16, 64, 64, 2, 2>(c, direct, st);
    else if (tiles_of(c.M, c.N, 256, 256) < kCus) tile<BF16, 128, 128, 2, 2>(c, direct, st);
    else tile<BF16, 256, 256, 2, 4>(c, direct, st);
    return hipGetLastError();
}

}  // namespace

size_t dense_ws_bytes(int64_t M, int64_t N, int64_t K) {
    int64_t most = 0;
    for (int64_t m = 64; m - 63 <= M; m += 64) {   // the parts depend on the number of tile rows
        const int64_t rows = m < M ? m : M, n = splits_of(rows, N, K);
        if (tiles_of(m, N, 64, 64) * 2 > kCus) break;
        if (n > 1 && n * rows > most) most = n * rows;
    }
    return (size_t)(most * ((N + 7) / 8 * 8)) * sizeof(float);
}

hipError_t launch_dense(DenseCall c, hipStream_t st) {
    c.ldp = (c.N + 7) / 8 * 8;
    return c.io_bf16 ? run<true>(c, st) : run<false>(c, st);
}

}  // namespace fi

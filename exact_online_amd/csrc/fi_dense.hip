// fi_dense.hip -- dense product with bias, activation and residual (fi_dense_*):
//     y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + res[m][n].
#include "fi_opdev.hpp"

namespace fi {

using V16 = float __attribute__((ext_vector_type(16)));

// act(v + bias) + res of four neighbouring outputs, stored
template <bool IO>
__device__ __forceinline__ void dense_out(const DenseCall& a, int64_t m, int64_t n, V4 v) {
    if (m >= a.M || n >= a.N) return;
    const int cnt = a.N - n < 4 ? (int)(a.N - n) : 4;
    if (a.bias)
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (r < cnt) v[r] += get_io<IO>(a.bias, n + r);
    if (a.act == 0) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = activate<0>(v[r]);
    } else if (a.act == 1) {
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = activate<1>(v[r]);
    }
    if (a.out_bf16) {
        using Four = BF __attribute__((ext_vector_type(4), aligned(2)));
        BF* y = static_cast<BF*>(a.y) + m * a.ldy + n;
        const BF* q = static_cast<const BF*>(a.res) + m * a.ldr + n;
        if (cnt == 4) {
            if (a.res) {
                const Four t = *gmem(reinterpret_cast<const Four*>(q));
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] += (float)t[r];
            }
            Four t;
#pragma unroll
            for (int r = 0; r < 4; ++r) t[r] = (BF)v[r];
            *gmem(reinterpret_cast<Four*>(y)) = t;
        } else
            for (int r = 0; r < cnt; ++r) gmem(y)[r] = (BF)(v[r] + (a.res ? (float)gmem(q)[r] : 0.f));
    } else {
        using Four = float __attribute__((ext_vector_type(4), aligned(4)));
        float* y = static_cast<float*>(a.y) + m * a.ldy + n;
        const float* q = static_cast<const float*>(a.res) + m * a.ldr + n;
        if (cnt == 4) {
            if (a.res) v += *gmem(reinterpret_cast<const Four*>(q));
            *gmem(reinterpret_cast<Four*>(y)) = v;
        } else
            for (int r = 0; r < cnt; ++r) gmem(y)[r] = v[r] + (a.res ? gmem(q)[r] : 0.f);
    }
}

// ------------------------------------------------------------ tiles of many rows
// A workgroup of WM x WN waves has a BM x BN tile of y; K goes by in steps of
// 128 bytes of a row, two LDS buffers, the next step's loads in flight during
// a step's products.  A row's eight 16-byte units are stored at u ^ (row / 2 %
// 8): the 16 lanes that read one unit of 16 rows then meet every bank once.
// The products are taken as w x^T, so that a lane's results are neighbours in
// a row of y.
template <bool BF16, int BM, int BN, int WM, int WN, bool DIRECT>
__global__ __launch_bounds__(WM* WN * kWave) void k_dense(DenseCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int E = M::E, BK = 8 * E, NTH = WM * WN * kWave, ROWS = BM + BN;
    constexpr int UX = BM * 8 / NTH, UN = ROWS * 8 / NTH;      // units per thread: of x, of both
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;        // 32 x 32 products of a wave
    __shared__ __align__(16) T lds[2][ROWS * BK];

    const int tid = threadIdx.x, wave = tid / kWave, lane = tid % kWave, l32 = lane % 32, half = lane / 32;
    const int wm = wave / WN * (BM / WM), wn = wave % WN * (BN / WN);
    const int64_t tm = (a.M + BM - 1) / BM, tn = (a.N + BN - 1) / BN, tiles = tm * tn;
    // workgroups go round the 8 XCDs: each XCD gets one run of tiles, in which
    // four rows of tiles go together along N (they share w in its L2)
    const int64_t at = blockIdx.x % tiles, split = blockIdx.x / tiles;
    const int64_t per = tiles / 8, over = tiles % 8, xcd = at % 8;
    const int64_t id = xcd * per + (xcd < over ? xcd : over) + at / 8;
    const int64_t gm = id / (4 * tn) * 4, rows = tm - gm < 4 ? tm - gm : 4, in = id - gm * tn;
    const int64_t m0 = (gm + in % rows) * BM, n0 = in / rows * BN;
    const int64_t k0 = split * a.k_split, k1 = k0 + a.k_split < a.K ? k0 + a.k_split : a.K;

    const T* src[UN];
#pragma unroll
    for (int i = 0; i < UN; ++i) {
        const int u = i * NTH + tid, row = u / 8, unit = u % 8 ^ (row / 2 % 8);
        if (i < UX) {
            const int64_t m = m0 + row < a.M ? m0 + row : a.M - 1;   // rows beyond the end are not stored
            src[i] = static_cast<const T*>(a.x) + m * a.ldx + unit * E;
        } else {
            const int64_t n = n0 + row - BM < a.N ? n0 + row - BM : a.N - 1;
            src[i] = static_cast<const T*>(a.w) + n * a.ldw + unit * E;
        }
    }
    V16 acc[TN][TM] = {};
    Frag hold[UN];
    const auto whole = [&](int64_t k) { return DIRECT && k + BK <= k1; };
    const auto fetch = [&](int64_t k, int buf) {
        if (whole(k)) {
#pragma unroll
            for (int i = 0; i < UN; ++i)
                __builtin_amdgcn_global_load_lds((const FI_GLOBAL void*)(src[i] + k),
                                                 (FI_SHARED void*)(&lds[buf][(i * NTH + wave * kWave) * E]), 16, 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < UN; ++i) {
                const int u = i * NTH + tid, unit = u % 8 ^ (u / 8 / 2 % 8);
                hold[i] = load_loose<BF16>(src[i] + k, 0, k1 - k - unit * E);
            }
        }
    };
    const auto settle = [&](int64_t k, int buf) {
        if (whole(k)) return;
#pragma unroll
        for (int i = 0; i < UN; ++i) *smem_ptr(reinterpret_cast<Frag*>(&lds[buf][(i * NTH + tid) * E])) = hold[i];
    };
    fetch(k0, 0);
    settle(k0, 0);
    int buf = 0;
    for (int64_t k = k0; k < k1; k += BK, buf ^= 1) {
        __syncthreads();
        const bool more = k + BK < k1;
        if (more) fetch(k + BK, buf ^ 1);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            Frag fw[TN], fx[TM];
#pragma unroll
            for (int i = 0; i < TN; ++i) {
                const int row = BM + wn + 32 * i + l32;
                fw[i] = *smem_ptr(reinterpret_cast<const Frag*>(&lds[buf][(row * 8 + ((2 * s + half) ^ (row / 2 % 8))) * E]));
            }
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int row = wm + 32 * i + l32;
                fx[i] = *smem_ptr(reinterpret_cast<const Frag*>(&lds[buf][(row * 8 + ((2 * s + half) ^ (row / 2 % 8))) * E]));
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
#pragma unroll
    for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int i = 0; i < TN; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t m = m0 + wm + 32 * j + l32, n = n0 + wn + 32 * i + 8 * q + 4 * half;
                const V4 v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
                if (!a.part) dense_out<BF16>(a, m, n, v);
                else if (m < a.M) {
                    // rows of `part` are a multiple of four long
                    if (n < a.N) *gmem(reinterpret_cast<V4*>(a.part + (split * a.M + m) * a.ldp + n)) = v;
                }
            }
}

// The parts of a product split over K, summed in their order.
template <bool IO>
__global__ __launch_bounds__(256) void k_dense_join(DenseCall a) {
    const int64_t per = a.ldp / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= a.M * per) return;
    const int64_t m = i / per, n = i % per * 4;
    V4 v = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < a.splits; ++s) v += *gmem(reinterpret_cast<const V4*>(a.part + (s * a.M + m) * a.ldp + n));
    dense_out<IO>(a, m, n, v);
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
        for (int i = 0; i < MT; ++i) dense_out<BF16>(a, 16 * i + l16, n0 + 4 * g, acc[i]);
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

template <bool BF16, int BM, int BN, int WM, int WN>
void tile(const DenseCall& c, bool direct, hipStream_t st) {
    const unsigned grid = (unsigned)(((c.M + BM - 1) / BM) * ((c.N + BN - 1) / BN) * c.splits);
    if (direct) k_dense<BF16, BM, BN, WM, WN, true><<<grid, WM * WN * kWave, 0, st>>>(c);
    else k_dense<BF16, BM, BN, WM, WN, false><<<grid, WM * WN * kWave, 0, st>>>(c);
    if (c.splits > 1)
        k_dense_join<BF16><<<(unsigned)((c.M * (c.ldp / 4) + 255) / 256), 256, 0, st>>>(c);
}

constexpr int64_t kCus = 256;
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
    const auto whole = [](const void* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % E == 0; };
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
    return (size_t)(most * ((N + 3) / 4 * 4)) * sizeof(float);
}

hipError_t launch_dense(DenseCall c, hipStream_t st) {
    c.ldp = (c.N + 3) / 4 * 4;
    return c.io_bf16 ? run<true>(c, st) : run<false>(c, st);
}

}  // namespace fi

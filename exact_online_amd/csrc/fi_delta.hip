// fi_delta.hip -- the gated delta rule (fi_delta_*).
//
// Per row b, value head n and position t, a = exp(log_decay[t]):
//     u[t] = beta[t] (v[t] - a S[t-1]^T k[t]),   S[t] = a S[t-1] + k[t] u[t]^T,   o[t] = scale S[t]^T q[t].
#include <algorithm>
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

// A state's decay by a = e^g, the same for all of the wave: near one as S + (a - 1) S, as the rounding of a (up to
// 2^-25 of S, always to one side) would add up over long memories; from a half down as a S, as a - 1 near -1 holds
// a to no more than 2^-25 of the whole S, which may be all that is left.  FLAT: two operations for one, and no branch.
template <bool FLAT, class Each>
__device__ __forceinline__ void decayed(float em1, float a, Each each) {
    if constexpr (FLAT) {
        const bool near = em1 > -0.5f;
        const float f = near ? em1 : a, c = near ? 1.f : 0.f;
        each([f, c](float s) { return fmaf(f, s, c * s); });
    } else if (__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(em1))) > -0.5f) {
        each([em1](float s) { return fmaf(em1, s, s); });
    } else {
        each([a](float s) { return a * s; });
    }
}

// ------------------------------------------------------------ recurrent form
// Position by position: a workgroup has dk x 32 of one (row, head)'s state in its
// registers, thread (r, c) = (tid / 8, tid % 8) the columns 4c .. 4c+3 of the
// slice and the rows r, r + 32, ...: columns of S never meet, so slices need no
// exchange, and rows of the slice are whole lines of memory.  Both products
// with the state before the position are formed at once, S^T k and S^T q; then
// o = a S^T q + (k . q) u needs no second pass over S.
// Bound by the state, read and written once: 200 rows x 32 heads of 128 x 128 (845 MB
// with q, k, v and o) take 164 to 168 us, 5.0 to 5.2 TB/s, what a large copy reaches
// (5.0).  One row: 4.9 us, a launch and two trips to memory.  Further positions of a call
// cost 12 us each (64 rows of these), vector operations on the state in its registers.
constexpr int kDsThreads = 256, kDsWaves = kDsThreads / kWave;
constexpr int kDsCols = 32;
constexpr int kDsRows = kDsThreads / (kDsCols / 4);   // rows in one sweep

template <bool BF16, int RPT, bool VEC>
__global__ __launch_bounds__(kDsThreads) void k_delta_step(DeltaCall a) {
    constexpr int ROWS = kDsRows * RPT;
    __shared__ float ks[2][ROWS], qs[2][ROWS];
    __shared__ __align__(16) float vs[2][kDsCols], red[2][kDsWaves][2][kDsCols];   // read in 16-byte units
    __shared__ float kqs[2][kDsWaves];
    const int tid = threadIdx.x, c = tid % (kDsCols / 4), r = tid / (kDsCols / 4), wave = tid / kWave;
    const int slices = (a.dv + kDsCols - 1) / kDsCols;
    const int64_t b = blockIdx.x / slices / a.Hv;
    const int n = blockIdx.x / slices % a.Hv, col0 = blockIdx.x % slices * kDsCols;
    const int dk = a.dk, dv = a.dv;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;
    const int col = col0 + 4 * c, left = dv - col;   // columns of the state from the thread's first on

    float* const sp = in && a.state ? a.state + (slot * a.Hv + n) * dk * (int64_t)dv + r * dv + col : nullptr;
    V4 S[RPT] = {};
    if (sp && !a.fresh) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (r + i * kDsRows < dk) {
                const FI_GLOBAL float* p = gmem(sp + i * kDsRows * dv);
                if constexpr (VEC) {
                    if (left > 0) S[i] = *reinterpret_cast<const FI_GLOBAL V4*>(p);
                } else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) S[i][j] = p[j];
            }
    }
    const int64_t kb = b * a.k.row + n / a.G * a.k.head, qb = b * a.q.row + n / a.G * a.q.head, vb = b * a.v.row + n * a.v.head + col0;
    const float* const ldp = static_cast<const float*>(a.ld.p) + b * a.ld.row + n * a.ld.head;
    const float* const bp = static_cast<const float*>(a.beta.p) + b * a.beta.row + n * a.beta.head;
    const int64_t ob = b * a.o.row + n * a.o.head + col;
    // the next position's: asked for a position ahead
    float nk = 0.f, nq = 0.f, nv = 0.f, nld = 0.f, nbeta = 0.f;
    const auto ask = [&](int64_t t) {
        if (tid < dk) {
            nk = get_io<BF16>(a.k.p, kb + t * a.k.pos + tid);
            nq = get_io<BF16>(a.q.p, qb + t * a.q.pos + tid);
        }
        if (tid < kDsCols && col0 + tid < dv) nv = get_io<BF16>(a.v.p, vb + t * a.v.pos + tid);
        nld = gmem(ldp)[t * a.ld.pos];
        nbeta = gmem(bp)[t * a.beta.pos];
    };
    if (len > 0) ask(0);
    for (int t = 0; t < len; ++t) {
        const int at = t % 2;
        if (tid < ROWS) ks[at][tid] = nk, qs[at][tid] = nq;
        if (tid < kDsCols) vs[at][tid] = nv;
        const float em1 = expm1f(nld), decay = expf(nld), beta = nbeta;
        __syncthreads();
        if (t + 1 < len) ask(t + 1);
        decayed<false>(em1, decay, [&](auto f) {
#pragma unroll
            for (int i = 0; i < 4 * RPT; ++i) S[i / 4][i % 4] = f(S[i / 4][i % 4]);
        });
        V4 sk = {0.f, 0.f, 0.f, 0.f}, sq = sk;
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float k = ks[at][r + i * kDsRows], q = qs[at][r + i * kDsRows];
            kq = fmaf(k, q, kq);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sk[j] = fmaf(k, S[i][j], sk[j]);
                sq[j] = fmaf(q, S[i][j], sq[j]);
            }
        }
#pragma unroll
        for (int d = 8; d < kWave; d <<= 1) {
            kq += __shfl_xor(kq, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sk[j] += __shfl_xor(sk[j], d);
                sq[j] += __shfl_xor(sq[j], d);
            }
        }
        if (tid % kWave < 8) {
            *smem_ptr(reinterpret_cast<V4*>(&red[at][wave][0][4 * c])) = sk;
            *smem_ptr(reinterpret_cast<V4*>(&red[at][wave][1][4 * c])) = sq;
            if (c == 0) kqs[at][wave] = kq;
        }
        __syncthreads();
        sk = sq = {0.f, 0.f, 0.f, 0.f};
        kq = 0.f;
#pragma unroll
        for (int w = 0; w < kDsWaves; ++w) {
            sk += *smem_ptr(reinterpret_cast<const V4*>(&red[at][w][0][4 * c]));
            sq += *smem_ptr(reinterpret_cast<const V4*>(&red[at][w][1][4 * c]));
            kq += kqs[at][w];
        }
        const V4 u = beta * (*smem_ptr(reinterpret_cast<const V4*>(&vs[at][4 * c])) - sk);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float k = ks[at][r + i * kDsRows];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = fmaf(k, u[j], S[i][j]);
        }
        if (r == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) put_io<BF16>(a.o.p, ob + t * a.o.pos + j, a.scale * fmaf(kq, u[j], sq[j]));
    }
    if (sp && !a.hold && (len > 0 || a.fresh)) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (r + i * kDsRows < dk) {
                FI_GLOBAL float* p = gmem(sp + i * kDsRows * dv);
                if constexpr (VEC) {
                    if (left > 0) *reinterpret_cast<FI_GLOBAL V4*>(p) = S[i];
                } else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) p[j] = S[i][j];
            }
    }
    for (int t = len + r; t < a.L; t += kDsRows)   // o is zero past the row's end
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) put_io<BF16>(a.o.p, ob + t * a.o.pos + j, 0.f);
}

hipError_t launch_delta_step(const DeltaCall& c, hipStream_t st) {
    const bool small = c.dk <= 4 * kDsRows, vec = c.dv % 4 == 0;   // the state's rows are whole 16-byte units
    const dim3 grid((unsigned)((c.dv + kDsCols - 1) / kDsCols * c.Hv * c.B));   // B Hv <= kLattnMaxRows
    const auto go = [&](auto bf, auto rpt) {
        constexpr bool BF16 = decltype(bf)::value;
        constexpr int RPT = decltype(rpt)::value;
        if (vec) k_delta_step<BF16, RPT, true><<<grid, kDsThreads, 0, st>>>(c);
        else k_delta_step<BF16, RPT, false><<<grid, kDsThreads, 0, st>>>(c);
    };
    using std::integral_constant;
    if (c.io_bf16 && small) go(std::true_type{}, integral_constant<int, 4>{});
    else if (c.io_bf16) go(std::true_type{}, integral_constant<int, 8>{});
    else if (small) go(std::false_type{}, integral_constant<int, 4>{});
    else go(std::false_type{}, integral_constant<int, 8>{});
    return hipGetLastError();
}

// ------------------------------------------------------------ chunked form
// With Q, K, V a chunk's C positions, E the state before it, G_i the sum of the
// log decays to position i (it included) and i, j < C:
//     A[i][j] = beta_i e^{G_i - G_j} k_i . k_j  (j < i),   T = (I + A)^{-1} diag(beta)
//     U = T (V - diag(e^{G_i}) K E)
//     O = scale (diag(e^{G_i}) Q E + P U),   P[i][j] = e^{G_i - G_j} q_i . k_j  (j <= i)
//     S = e^{G_C} E + K^T diag(e^{G_C - G_j}) U
// T does not depend on the state: k_delta_tri forms it for all chunks at once.
// k_delta_chunk then follows a row's chunks, a workgroup to a head and a slice of
// columns of S, 16 or 32 columns to a wave.
//
// Long rows of few heads are split into segments.  What a segment does to the
// state before it is linear: S = M E + N; OUT = false forms N (the state from
// zero) and M (the same, without values, from the identity: dk more columns),
// k_delta_join the states before the segments, and OUT = true starts from those.
//
// Numbers (bf16): the operands of the matrix cores are bf16.  q, k and v are that as they
// are; S, T, R = V - .. and U, held in fp32, enter the state's recurrence in three parts
// each, which hold all of their 24 bits (products of parts below 2^-24 are left out): the state is as far from
// 64 bits as fp32 sums are, 2e-7 of its norm (with two parts 2e-6, for 15% less time).  Outputs are rounded to
// bf16, and take S, P and U in two parts, 2^-18 of them.  fp32: fp32 products throughout.
//
// Measured: one row of 65536, 16 heads of 128 x 128, bf16 (1.07 GB once: 218 us): 1092 to 1205 us on different cards (under
// the profiler systems 161, segments' states 609, join 53, outputs 536).  8 ragged rows of up to 2048, 32
// heads: 269 to 288, systems 79 of them.  fp32, two rows of 4001, 16 heads of 64 x 64: 131 to 134.  Two thirds
// of the time are the instructions of a wave: a product of 16 cycles and the four vector operations that go with
// it (splits most of all) take 26 to 27 together even side by side; the rest is waits, with 1.4 to 1.8
// waves on a SIMD.  LDS is 20 to 43% busy, memory a fifth.  Wide heads (no more than one wave on a SIMD, some of its
// registers in scratch), two rows of 4000, 8 heads of 192 x 192 and 256 x 256: bf16 389 and 402, fp32 861 and 909;
// 16 rows of 1000, which are not split: 352 and 353, 865 and 916 (without the branch of a state's decay 317 and 339, 855 and 900).
template <bool BF16>
struct Dl {
    static constexpr int C = BF16 ? 64 : 32, CT = C / 16;               // positions of a chunk, tiles of them
    static constexpr int KB = Mm<BF16>::KB, E = Mm<BF16>::E, PER = KB / 16;   // tiles of an operand
    static constexpr int NF = BF16 ? 6 : 3;                            // operands of a lower triangle of C x C
    static constexpr int PARTS = BF16 ? 3 : 1, HALF = BF16 ? 2 : 1;     // parts of an fp32 factor, of one for an output
    static constexpr int TRI = NF * kWave * E, GATES = 4 * C;           // floats of a chunk: T, then the gates
    // operand (it, kb) of the triangle
    static __device__ __forceinline__ int frag(int it, int kb) { return BF16 ? (it / 2 * (it / 2 + 1) + it % 2 * (it / 2 + 1)) + kb : it * (it + 1) / 2 + kb; }
};
constexpr float kLog2E = 1.44269504088896341f;

// Sums of C log decays, to each position (its own included), as two floats, in lanes % C.
// Below -150 a decay is 0 in fp32: clamped, so that differences stay finite.
struct Gate {
    float hi, lo;
};
template <int C>
__device__ __forceinline__ Gate gate_sum(float g) {
    const double s = scan64<C>(g < -150.f ? -150.0 : (double)g);
    const float hi = (float)s;
    return {hi, (float)(s - hi)};
}
__device__ __forceinline__ float exp_of(Gate a, Gate b) {   // e^{a - b}, a <= b
    return __builtin_amdgcn_exp2f(((a.hi - b.hi) + (a.lo - b.lo)) * kLog2E);
}

// One chunk's T and gates (reading k and writing them, 13 KB for 64 positions of bf16, bounds 64K x 16 heads to
// 100 us; 148 are taken, half of a wave's time in the substitution and its waits).  A wave has 16 rows of A: it forms the block on the diagonal, inverts
// it by substitution to D_i (stable, where powers of A would not be: equal keys make them as
// large as binomials), and the blocks before it; then the waves meet, and
//     T_ij = -(sum_{j < k <= i} T_ik A_kj) D_j,   j = i - 1, i - 2, ..,
// is formed transposed, so that a result is the next product's operand as it lies in
// the registers, and what is stored is the operand that k_delta_chunk loads.
template <bool BF16, int DK, bool VEC>
__global__ __launch_bounds__(Dl<BF16>::CT * kWave, DK <= 128 ? 4 : 2) void k_delta_tri(DeltaCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    using D = Dl<BF16>;
    constexpr int C = D::C, CT = D::CT, E = D::E, KB = D::KB, NK = DK / KB, PA = C + 4;
    __shared__ __align__(16) float as[C * PA], ds[CT][16][20], gs[CT][3][C];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int l16 = lane % 16, g = lane / 16;
    const int64_t unit = blockIdx.x, task = unit / a.chunks;
    const int c = a.chunk0 + (int)(unit - task * a.chunks);
    const int64_t b = task / a.Hv;
    const int n = (int)(task - b * a.Hv), dk = a.dk;
    const int64_t slot = a.slots ? a.slots[b] : b;
    int len = a.lens ? a.lens[b] : a.L;
    len = slot >= 0 && slot < a.n_slots ? (len > a.L ? a.L : len) : 0;
    const int t0 = c * C, left = len - t0;   // positions from the chunk's first on
    if (left <= 0) return;

    // everything that the wave reads is asked for at once
    const int at = t0 + lane % C;
    float ld = 0.f, beta = 0.f;
    if (lane % C < left) {
        ld = gmem(static_cast<const float*>(a.ld.p))[b * a.ld.row + at * a.ld.pos + n * a.ld.head];
        beta = gmem(static_cast<const float*>(a.beta.p))[b * a.beta.row + at * a.beta.pos + n * a.beta.head];
    }
    const T* const kp = static_cast<const T*>(a.k.p) + b * a.k.row + n / a.G * a.k.head;
    const auto rows = [&](int tile, Frag* f) {
        const int r = 16 * tile + l16;
        const T* p = kp + (int64_t)(t0 + (r < left ? r : left - 1)) * a.k.pos;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            const int col = kb * KB + g * E;
            f[kb] = Frag{};
            if (r < left && col < dk) {
                if constexpr (VEC) f[kb] = *gmem(reinterpret_cast<const Frag*>(p + col));
                else f[kb] = load_loose<BF16>(p, col, dk);
            }
        }
    };
    Frag own[NK], before[CT - 1][NK];
    rows(wave, own);
#pragma unroll
    for (int j = 0; j < CT - 1; ++j)
        if (j < wave) rows(j, before[j]);

    const Gate mine = gate_sum<C>(ld);
    const auto last = [](float x) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), C - 1)); };
    if (lane < C) {
        gs[wave][0][lane] = mine.hi;   // a copy of its own: the waves need not wait for one another here
        gs[wave][1][lane] = mine.lo;
        gs[wave][2][lane] = beta;
        if (wave == 0) {
            float* const to = a.tri + unit * (D::TRI + D::GATES) + D::TRI;
            const Gate zero = {0.f, 0.f}, end = {last(mine.hi), last(mine.lo)};
            to[lane] = exp_of(mine, zero);
            to[C + lane] = exp_of(end, mine);
            to[2 * C + lane] = mine.hi;
            to[3 * C + lane] = mine.lo;
        }
    }
    wave_order();
    const V4 ghi = *smem_ptr(reinterpret_cast<const V4*>(&gs[wave][0][16 * wave + 4 * g])),
             glo = *smem_ptr(reinterpret_cast<const V4*>(&gs[wave][1][16 * wave + 4 * g])),
             gb = *smem_ptr(reinterpret_cast<const V4*>(&gs[wave][2][16 * wave + 4 * g]));
    const auto block = [&](int jt, const Frag* f) {   // A's tile (wave, jt)
        V4 p[2] = {};
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) p[kb % 2] = M::mma(own[kb], f[kb], p[kb % 2]);
        p[0] += p[1];
        const int j = 16 * jt + l16;
        const Gate gj = {gs[wave][0][j], gs[wave][1][j]};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 16 * wave + 4 * g + r;
            const float x = gb[r] * exp_of(Gate{ghi[r], glo[r]}, gj) * p[0][r];
            as[i * PA + j] = j < i ? x : 0.f;
        }
    };
    block(wave, own);
    wave_order();
    // row l16 of D_wave: x (I + A) = e, from the last column on
    float x[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = j == l16 ? 1.f : 0.f;
#pragma unroll
    for (int k = 15; k > 0; --k)
#pragma unroll
        for (int j0 = 0; j0 < k; j0 += 4) {
            const V4 y = *smem_ptr(reinterpret_cast<const V4*>(&as[(16 * wave + k) * PA + 16 * wave + j0]));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j0 + j < k) x[j0 + j] = fmaf(-x[k], y[j], x[j0 + j]);
        }
    if (g == 0)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
            *smem_ptr(reinterpret_cast<V4*>(&ds[wave][l16][j])) = V4{x[j], x[j + 1], x[j + 2], x[j + 3]};
#pragma unroll
    for (int j = 0; j < CT - 1; ++j)
        if (j < wave) block(j, before[j]);
    __syncthreads();
    // t: block (wave, j), transposed: its columns 4 g .. 4 g + 3 of row l16; the block on the diagonal last in t,
    // those before it towards the front: indexes are constants
    V4 t[CT];
#pragma unroll
    for (int r = 0; r < 4; ++r) t[CT - 1][r] = g == 0 ? x[r] : g == 1 ? x[4 + r] : g == 2 ? x[8 + r] : x[12 + r];
    const auto column = [&](const float* p, int pitch) {
        const FI_SHARED float* q = smem_ptr(p) + 4 * g * pitch + l16;
        return V4{q[0], q[pitch], q[2 * pitch], q[3 * pitch]};
    };
    float* const to = a.tri + unit * (D::TRI + D::GATES);
    // with beta, as operands: tile j of row `wave` is the part j % PER of operand j / PER
    const auto put = [&](int j, V4 v) {
        *gmem(reinterpret_cast<V4*>(to + (D::frag(wave, j / D::PER) * kWave + lane) * E + j % D::PER * 4)) = v;
    };
    const auto with_beta = [&](int j, V4 v) { put(j, v * *smem_ptr(reinterpret_cast<const V4*>(&gs[wave][2][16 * j + 4 * g]))); };
    with_beta(wave, t[CT - 1]);
    if (D::PER == 2 && wave % 2 == 0) put(wave + 1, V4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
    for (int back = 1; back < CT; ++back) {
        const int j = wave - back;
        if (j < 0) break;
        V4 s[2] = {};
#pragma unroll
        for (int near = 0; near < back; ++near)   // block (wave, wave - near)
            s[near % 2] = Mm<false>::mma(column(as + 16 * (wave - near) * PA + 16 * j, PA), t[CT - 1 - near], s[near % 2]);
        t[CT - 1 - back] = -Mm<false>::mma(column(&ds[j][0][0], 20), s[0] + s[1], V4{0.f, 0.f, 0.f, 0.f});
        with_beta(j, t[CT - 1 - back]);
    }
}

// Values of a block's tiles as the sum of N parts, each the nearest to what is
// left: two hold an fp32 value to 2^-18, three hold it whole.
template <bool BF16, int N>
__device__ __forceinline__ void split(const V4* x, typename Mm<BF16>::Frag* f) {
    if constexpr (BF16) {
        using BF2 = BF __attribute__((ext_vector_type(2)));
        uint32_t part[N][4];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            V2 y = {x[e / 4][e % 4], x[e / 4][e % 4 + 1]};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t u = part[i][e / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(y, BF2));
                if (i + 1 < N) {
                    y.x -= __uint_as_float(u << 16);
                    y.y -= __uint_as_float(u & 0xFFFF0000u);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __builtin_bit_cast(BF8, part[i]);
    } else f[0] = x[0];
}
// The same of four values, to LDS: part i at to + i * pitch
template <bool BF16, int N>
__device__ __forceinline__ void split_to(V4 x, typename Mm<BF16>::T* to, int pitch) {
    if constexpr (BF16) {
        using U2 = uint32_t __attribute__((ext_vector_type(2)));
        using BF2 = BF __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            U2 u;
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                u[e / 2] = __builtin_bit_cast(uint32_t, __builtin_convertvector(V2{x[e], x[e + 1]}, BF2));
                x[e] -= __uint_as_float(u[e / 2] << 16);
                x[e + 1] -= __uint_as_float(u[e / 2] & 0xFFFF0000u);
            }
            *smem_ptr(reinterpret_cast<U2*>(to + i * pitch)) = u;
        }
    } else *smem_ptr(reinterpret_cast<V4*>(to)) = x;
}

// A slice is DVS = 16 NC WAVES columns.  A wave has NC tiles of 16 columns of S in its registers, which are the
// operand of its products as they lie there: lane (g, l16) of tile kt has column l16 and the rows row_of(kt) + r,
// so that the tiles of one operand hold rows that follow one another for each lane.
// The waves meet only in P and in what is staged.  Outputs of 128-wide heads take eight waves of one tile (one workgroup
// on a CU: four waves of two tiles, 256 registers each, leave a SIMD one wave: ragged rows 316 and 503 us), the
// segments' states four of two (two workgroups on a CU; 64K positions 530 and 606 us).
template <bool BF16, int DK, int WAVES, int NC, bool OUT, bool VEC>
__global__ __launch_bounds__(WAVES * kWave, DK <= 128 || WAVES == 8 ? 2 : 1) void k_delta_chunk(DeltaCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    using Four = T __attribute__((ext_vector_type(4)));
    using D = Dl<BF16>;
    constexpr int C = D::C, CT = D::CT, E = D::E, KB = D::KB, PER = D::PER, NF = D::NF, PARTS = D::PARTS, HALF = D::HALF;
    constexpr int NTH = WAVES * kWave, KT = DK / 16, DVS = 16 * NC * WAVES;
    constexpr int PV = DVS + E;                                  // V's LDS rows
    constexpr int UK = C * DK / E / NTH, UV = C * DVS / E / NTH; // 16-byte units of a thread
    constexpr int UT = (D::TRI / 4 + NTH - 1) / NTH;             // fours of T of a thread
    __shared__ __align__(16) T ks[C * DK], vs[C * PV], qs[OUT ? C * DK : 1], ps[OUT ? HALF * D::TRI : 1], ts[PARTS * D::TRI];
    __shared__ __align__(16) float gs[D::GATES];                 // e^{G_i}, e^{G_C - G_i}, G_i in two floats

    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t l16 = (uint32_t)lane % 16, g = (uint32_t)lane / 16;
    const int dk = a.dk, dv = a.dv;
    const int values = (dv + DVS - 1) / DVS, slices = OUT ? values : values + (dk + DVS - 1) / DVS;
    // the slices of one segment read the same Q and K: eight workgroups apart, on one XCD and its L2
    const int tasks = (int)a.B * a.Hv, unit = blockIdx.x / (8 * slices) * 8 + blockIdx.x % 8, slice = blockIdx.x / 8 % slices;
    if (unit >= tasks * a.nseg) return;
    const int seg = unit / tasks, task = unit % tasks, b = task / a.Hv, n = task % a.Hv;
    const bool moves = !OUT && slice >= values;                  // columns of what the segment does to a state
    const int col0 = (moves ? slice - values : slice) * DVS;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;
    const int chunks = (len + C - 1) / C, stop = a.chunk0 + a.chunks < chunks ? a.chunk0 + a.chunks : chunks;
    const int c0 = a.chunk0 + seg * a.seg_chunks;
    int c1 = c0 + a.seg_chunks;
    if (c1 > stop) c1 = stop;
    if (!OUT && c1 >= stop) return;      // a row's last segment hands nothing on
    if (moves && seg == 0 && a.chunk0 == 0 && a.fresh) return;   // (there is nothing before it to move)

    if constexpr (OUT) {                 // o is zero past the row's end
        const bool last = seg == a.nseg - 1 && a.chunk0 + a.chunks >= (a.L + C - 1) / C;
        const int64_t end = (int64_t)(seg == a.nseg - 1 ? a.chunk0 + a.chunks : c0 + a.seg_chunks) * C, z1 = last || end > a.L ? a.L : end;
        const int64_t z0 = len > c0 * C ? len : c0 * C;
        constexpr int Z = VEC ? E : 1, UNITS = DVS / Z;   // elements of a store, stores of a row
        const int col = col0 + tid % UNITS * Z;
        if (col < dv)
            for (int64_t t = z0 + tid / UNITS; t < z1; t += NTH / UNITS) {
                T* const p = static_cast<T*>(a.o.p) + b * a.o.row + t * a.o.pos + n * a.o.head + col;
                if constexpr (VEC) *gmem(reinterpret_cast<Frag*>(p)) = Frag{};
                else *gmem(p) = (T)0.f;
            }
        if (c0 >= stop && !(c0 == 0 && in && a.fresh)) return;   // (a fresh row without positions leaves zeros)
    }

    // the lane's part of S: rows row_of(kt) + r of the columns scol + 16 nc
    const auto row_of = [&](int kt) { return BF16 ? kt / 2 * 32 + (int)g * 8 + kt % 2 * 4 : 16 * kt + 4 * (int)g; };
    float* const sp = a.state && in ? a.state + (slot * a.Hv + n) * dk * (int64_t)dv : nullptr;
    float* const ep = a.nseg > 1 ? a.ent + ((int64_t)task * a.nseg + seg) * dk * dv : nullptr;
    float* const cp = a.carry ? a.carry + (int64_t)task * dk * dv : nullptr;
    const float* const from = !OUT ? nullptr : ep ? ep : a.chunk0 ? cp : a.fresh ? nullptr : sp;
    const int wcol = 16 * NC * wave, scol = col0 + wcol + (int)l16;
    V4 S[NC][KT] = {};
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
        const int col = scol + 16 * nc;
        if (from && col < dv)
#pragma unroll
            for (int i = 0; i < 4 * KT; ++i) {
                const int row = row_of(i / 4) + i % 4;
                if (row < dk) S[nc][i / 4][i % 4] = gmem(from)[row * dv + col];
            }
        if (moves)
#pragma unroll
            for (int i = 0; i < 4 * KT; ++i)
                if (row_of(i / 4) + i % 4 == col && col < dk) S[nc][i / 4][i % 4] = 1.f;
    }

    // Staging: a thread has the same columns of rows RK (RV) apart.  Loads are of
    // valid places always: columns past the head's end are blanked on their way to
    // LDS, rows past the row's repeat its last, and weigh nothing (beta is 0 there).
    constexpr int RK = NTH * E / DK, RV = NTH * E / DVS;
    const int kcol = tid % (DK / E) * E, krow = tid / (DK / E), vcol = tid % (DVS / E) * E, vrow = tid / (DVS / E);
    const bool kin = kcol < dk, vin = !moves && col0 + vcol < dv;
    const int kleft = kin ? dk - kcol : 0, vleft = vin ? dv - col0 - vcol : 0;   // elements from there on
    const int klcol = kin ? kcol : 0, vlcol = vin ? vcol : 0;
    const T* const kp = static_cast<const T*>(a.k.p) + b * a.k.row + n / a.G * a.k.head;
    const T* const qp = static_cast<const T*>(a.q.p) + b * a.q.row + n / a.G * a.q.head;
    const T* const vp = static_cast<const T*>(a.v.p) + b * a.v.row + n * a.v.head + (moves ? 0 : col0);
    const float* const tp = a.tri + (int64_t)task * a.chunks * (D::TRI + D::GATES);
    Frag fk[UK], fv[UV], fq[UK];
    V4 ft[UT];
    float fg;
    const auto fetch = [&](auto& f, const T* p, int64_t pos, int c, int row, int step, int col, int left) {
        constexpr int count = sizeof(f) / sizeof(f[0]);
        const int t0 = c * C, most = len - 1 - t0;
        p += t0 * pos;
#pragma unroll
        for (int i = 0; i < count; ++i) {
            const int r = row + i * step < most ? row + i * step : most;
            if constexpr (VEC) {
                const uint32_t off = (uint32_t)(r * (int)pos + col) * sizeof(T);
                f[i] = *gmem(reinterpret_cast<const Frag*>(reinterpret_cast<const char*>(p) + off));
            } else f[i] = load_loose<BF16>(p + r * pos + col, 0, left);
        }
    };
    const auto fetch_t = [&](int c) {
        const float* p = tp + (int64_t)(c - a.chunk0) * (D::TRI + D::GATES);
#pragma unroll
        for (int i = 0; i < UT; ++i)
            if ((i + 1) * NTH <= D::TRI / 4 || tid + i * NTH < D::TRI / 4) ft[i] = *gmem(reinterpret_cast<const V4*>(p + 4 * (tid + i * NTH)));
        if (tid < D::GATES) fg = gmem(p)[D::TRI + tid];
    };
    // Q and K in LDS: unit (16 bytes) u of row r at u ^ mix(r): 16 lanes with 16 rows meet every bank once
    const auto place = [](uint32_t row, uint32_t u) -> uint32_t {
        constexpr int UNITS = DK / E;
        const uint32_t m = !BF16 ? row % 16 : UNITS == 8 ? 4 * (row / 2 % 2) + row / 4 % 4 : 4 * (row % 4) + row / 4 % 4;
        return (row * UNITS + (u ^ m)) * E;
    };
    const auto put_rows = [&](T* to, auto& f) {
#pragma unroll
        for (int i = 0; i < UK; ++i) {
            if (!kin) f[i] = Frag{};
            *smem_ptr(reinterpret_cast<Frag*>(to + place(krow + i * RK, kcol / E))) = f[i];
        }
    };
    const auto row_frag = [&](const T* from, int tile, int kb) {
        return *smem_ptr(reinterpret_cast<const Frag*>(from + place(16 * tile + l16, kb * 4 + g)));
    };
    // tile kt of K's columns, as an operand over the positions of block kb
    const auto transposed = [&](int kt, int kb) {
        Frag f;
        if constexpr (BF16) {
            // a 16-lane group reads 4 positions x 16 columns and gets them transposed
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const T* p = ks + place(KB * kb + 16 * h + 4 * g + l16 / 4, kt / 2 * 4 + l16 % 4) + kt % 2 * 4;
                const BF4 y = __builtin_bit_cast(BF4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((FI_SHARED S4*)(p)));
#pragma unroll
                for (int e = 0; e < 4; ++e) f[4 * h + e] = y[e];
            }
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = smem_ptr(ks)[place(KB * kb + 4 * g + e, 4 * kt + l16 / 4) + l16 % 4];
        }
        return f;
    };
    const auto tri_frag = [&](const T* from, int part, int f) {
        return *smem_ptr(reinterpret_cast<const Frag*>(from + (part * NF + f) * kWave * E + lane * E));
    };
    const auto fetch_all = [&](int c) {
        fetch(fk, kp, a.k.pos, c, krow, RK, klcol, kleft);
        if (!moves) fetch(fv, vp, a.v.pos, c, vrow, RV, vlcol, vleft);
        if constexpr (OUT) fetch(fq, qp, a.q.pos, c, krow, RK, klcol, kleft);
        fetch_t(c);
    };

    // the halves of P's operands that lie above the diagonal
    if constexpr (OUT && PER == 2)
        if (wave < CT / 2) split_to<BF16, HALF>(V4{0.f, 0.f, 0.f, 0.f}, ps + (D::frag(2 * wave, wave) * kWave + lane) * E + 4, D::TRI);
    if (c0 < c1) fetch_all(c0);
    for (int c = c0; c < c1; ++c) {
        const int rows = len - c * C;   // positions from the chunk's first on
        put_rows(ks, fk);
        if constexpr (OUT) put_rows(qs, fq);
        if (!moves) {
#pragma unroll
            for (int i = 0; i < UV; ++i) {
                if (!vin) fv[i] = Frag{};
                *smem_ptr(reinterpret_cast<Frag*>(vs + (vrow + i * RV) * PV + vcol)) = fv[i];
            }
        }
#pragma unroll
        for (int i = 0; i < UT; ++i)
            if ((i + 1) * NTH <= D::TRI / 4 || tid + i * NTH < D::TRI / 4) split_to<BF16, PARTS>(ft[i], ts + 4 * (tid + i * NTH), D::TRI);
        if (tid < D::GATES) gs[tid] = fg;
        __syncthreads();
        // the next chunk's (the last one's again at the end: no branch, so that nothing waits for them before
        // their use); where registers are short behind the outputs
        constexpr bool EARLY = NC == 1;
        if constexpr (EARLY) fetch_all(c + 1 < c1 ? c + 1 : c);

        if constexpr (OUT) {
            // P^T, tiles of 16 keys x 16 queries, jt <= it, shared out among the waves (the last
            // ones form the last tile again: without branches the products below run beside it)
            constexpr int TILES = CT * (CT + 1) / 2;
#pragma unroll
            for (int at = 0; at < TILES; at += WAVES) {
                const int tile = at + WAVES <= TILES || at + wave < TILES ? at + wave : TILES - 1;
                const int it = tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3, jt = tile - it * (it + 1) / 2;
                V4 p[2] = {};
#pragma unroll
                for (int kb = 0; kb < DK / KB; ++kb) p[kb % 2] = M::mma(row_frag(ks, jt, kb), row_frag(qs, it, kb), p[kb % 2]);
                p[0] += p[1];
                const int i = 16 * it + l16;
                const Gate gi = {gs[2 * C + i], gs[3 * C + i]};
                const V4 hi = *smem_ptr(reinterpret_cast<const V4*>(&gs[2 * C + 16 * jt + 4 * g])),
                         lo = *smem_ptr(reinterpret_cast<const V4*>(&gs[3 * C + 16 * jt + 4 * g]));
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * jt + 4 * g + r;
                    const float x = p[0][r] * exp_of(gi, Gate{hi[r], lo[r]});
                    p[0][r] = j <= i ? x : 0.f;
                }
                split_to<BF16, HALF>(p[0], ps + (D::frag(it, jt / PER) * kWave + lane) * E + jt % PER * 4, D::TRI);
            }
        }
        // K E (rows are positions), and O^T = E^T Q^T (columns are positions).  The longest run of products goes
        // first where another wave of the SIMD splits or stages (ragged rows 284 -> 278 us, 64K positions 1163 -> 1129).
        __builtin_amdgcn_s_setprio(1);
        V4 R[NC][CT] = {}, O[OUT ? NC : 1][OUT ? CT : 1] = {};
#pragma unroll
        for (int kb = 0; kb < DK / KB; ++kb) {
            Frag f[NC][PARTS];
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) split<BF16, PARTS>(&S[nc][kb * PER], f[nc]);
            Frag k[CT], q[OUT ? CT : 1];
#pragma unroll
            for (int it = 0; it < CT; ++it) {
                k[it] = row_frag(ks, it, kb);
                if constexpr (OUT) q[it] = row_frag(qs, it, kb);
            }
#pragma unroll
            for (int i = PARTS - 1; i >= 0; --i)
#pragma unroll
                for (int it = 0; it < CT; ++it)
#pragma unroll
                    for (int nc = 0; nc < NC; ++nc) {
                        R[nc][it] = M::mma(k[it], f[nc][i], R[nc][it]);
                        if constexpr (OUT) {
                            if (i < HALF) O[nc][it] = M::mma(f[nc][i], q[it], O[nc][it]);
                        }
                    }
        }
        __builtin_amdgcn_s_setprio(0);
        // S: its decay, as E is not read again.  bf16 by a branch (64K positions 1105 us here, 1118 before S's products, 1120
        // without one), fp32 without (two rows of 4001 133; by a branch 137, before S's products 134.5)
        decayed<!BF16>(expm1f(gs[3 * C - 1]) + gs[C - 1] * gs[4 * C - 1], gs[C - 1], [&](auto f) {
#pragma unroll
            for (int i = 0; i < NC * KT * 4; ++i) S[i / (4 * KT)][i / 4 % KT][i % 4] = f(S[i / (4 * KT)][i / 4 % KT][i % 4]);
        });
        // R = V - diag(e^G) K E
#pragma unroll
        for (int it = 0; it < CT; ++it) {
            const V4 e = *smem_ptr(reinterpret_cast<const V4*>(&gs[16 * it + 4 * g]));
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) {
                V4 v = {0.f, 0.f, 0.f, 0.f};
                if (!moves) {
                    if constexpr (BF16) {
                        const T* p = vs + (16 * it + 4 * g + l16 / 4) * PV + wcol + 16 * nc + l16 % 4 * 4;
                        const BF4 y = __builtin_bit_cast(BF4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((FI_SHARED S4*)(p)));
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = (float)y[r];
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) v[r] = smem_ptr(vs)[(16 * it + 4 * g + r) * PV + wcol + 16 * nc + l16];
                    }
                }
#pragma unroll
                for (int r = 0; r < 4; ++r) R[nc][it][r] = fmaf(-e[r], R[nc][it][r], v[r]);
            }
        }
        // U = T R
        V4 U[NC][CT] = {};
#pragma unroll
        for (int kb = 0; kb < C / KB; ++kb) {
            Frag f[NC][PARTS];
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) split<BF16, PARTS>(&R[nc][kb * PER], f[nc]);
#pragma unroll
            for (int p = PARTS - 1; p >= 0; --p) {
                Frag t[CT];
#pragma unroll
                for (int it = kb * PER; it < CT; ++it) t[it] = tri_frag(ts, p, D::frag(it, kb));
#pragma unroll
                for (int i = PARTS - 1 - p; i >= 0; --i)
#pragma unroll
                    for (int it = kb * PER; it < CT; ++it)
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc) U[nc][it] = M::mma(t[it], f[nc][i], U[nc][it]);
            }
        }
        if constexpr (OUT) {
            // O = e^G Q E + P U
#pragma unroll
            for (int it = 0; it < CT; ++it) {
                const float e = gs[16 * it + l16];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) O[nc][it] *= e;
            }
            __syncthreads();
#pragma unroll
            for (int kb = 0; kb < C / KB; ++kb) {
                Frag f[NC][HALF];
#pragma unroll
                for (int nc = 0; nc < NC; ++nc) split<BF16, HALF>(&U[nc][kb * PER], f[nc]);
#pragma unroll
                for (int p = HALF - 1; p >= 0; --p) {
                    Frag t[CT];
#pragma unroll
                    for (int it = kb * PER; it < CT; ++it) t[it] = tri_frag(ps, p, D::frag(it, kb));
#pragma unroll
                    for (int i = HALF - 1 - p; i >= 0; --i)
#pragma unroll
                        for (int it = kb * PER; it < CT; ++it)
#pragma unroll
                            for (int nc = 0; nc < NC; ++nc) O[nc][it] = M::mma(f[nc][i], t[it], O[nc][it]);
                }
            }
            const bool whole = rows >= C;
            T* const op = static_cast<T*>(a.o.p) + b * a.o.row + n * a.o.head + (int64_t)c * C * a.o.pos + col0 + wcol;
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) {
                const int left = dv - (col0 + wcol + 16 * nc + 4 * (int)g);
#pragma unroll
                for (int it = 0; it < CT; ++it) {
                    Four y;
#pragma unroll
                    for (int r = 0; r < 4; ++r) y[r] = (T)(a.scale * O[nc][it][r]);
                    if (whole || 16 * it + (int)l16 < rows) {
                        T* to = op + (16 * it + l16) * a.o.pos + 16 * nc + 4 * g;
                        if constexpr (VEC) {
                            if (left > 0) *gmem(reinterpret_cast<Four*>(to)) = y;
                        } else
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (r < left) gmem(to)[r] = y[r];
                    }
                }
            }
        }
        if constexpr (!EARLY) fetch_all(c + 1 < c1 ? c + 1 : c);
        // S takes the chunk's own products
#pragma unroll
        for (int kb = 0; kb < C / KB; ++kb) {
            Frag f[NC][PARTS];
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) {
#pragma unroll
                for (int it = kb * PER; it < (kb + 1) * PER; ++it)
                    U[nc][it] *= *smem_ptr(reinterpret_cast<const V4*>(&gs[C + 16 * it + 4 * g]));
                split<BF16, PARTS>(&U[nc][kb * PER], f[nc]);
            }
#pragma unroll
            for (int k0 = 0; k0 < KT; k0 += 4) {   // a few at a time: a product does not wait for the one before
                Frag k[4];
#pragma unroll
                for (int kt = 0; kt < 4; ++kt) k[kt] = transposed(k0 + kt, kb);
#pragma unroll
                for (int i = PARTS - 1; i >= 0; --i)
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt)
#pragma unroll
                        for (int nc = 0; nc < NC; ++nc) S[nc][k0 + kt] = M::mma(k[kt], f[nc][i], S[nc][k0 + kt]);
            }
        }
        __syncthreads();
    }
    float* to;
    if constexpr (OUT) to = c1 < chunks ? (c1 == a.chunk0 + a.chunks ? cp : nullptr) : a.hold ? nullptr : sp;
    else to = moves ? a.move + ((int64_t)task * a.nseg + seg) * DK * DK : ep + (int64_t)dk * dv;
    if (!to) return;
    // (M is kept whole, DK x DK: its rows and columns beyond dk are zero)
    const int width = moves ? DK : dv, height = moves ? DK : dk;
#pragma unroll
    for (int nc = 0; nc < NC; ++nc) {
        const int col = scol + 16 * nc;
        if (col < width)
#pragma unroll
            for (int i = 0; i < 4 * KT; ++i) {
                const int row = row_of(i / 4) + i % 4;
                if (row < height) gmem(to)[row * width + col] = S[nc][i / 4][i % 4];
            }
    }
}

// ------------------------------------------------------------ few positions
// The chunked form with chunks of 16 positions, all of it in one wave: a wave follows a
// row and head with 16 columns of S, forms T and P for itself and meets no other.  For
// calls of a few chunks of 16, where one launch and no workspace are worth more than
// forming T once for all columns.  Bound by the state's way from memory: five held positions of 64 rows, 32 heads of 128 x
// 128 (147 MB) 38.6 us, 3.8 TB/s; where the state is written too 68 (4.1 TB/s).
constexpr int kDfWaves = 4, kDfC = 16;

template <bool BF16, int DK, bool VEC>
__global__ __launch_bounds__(kDfWaves * kWave, BF16 && DK <= 128 ? 3 : DK <= 128 ? 2 : 1) void k_delta_few(DeltaCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    using Four = T __attribute__((ext_vector_type(4)));
    using D = Dl<BF16>;
    constexpr int E = D::E, KB = D::KB, NK = DK / KB, KT = DK / 16, PER = D::PER, PARTS = D::PARTS, HALF = D::HALF, C = kDfC;
    __shared__ __align__(16) T ks_[kDfWaves][C * DK];
    __shared__ __align__(16) float as_[kDfWaves][C][20], gs_[kDfWaves][4][C];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t l16 = (uint32_t)lane % 16, g = (uint32_t)lane / 16;
    T* const ks = ks_[wave];
    float (* const as)[20] = as_[wave];
    float (* const gs)[C] = gs_[wave];
    const int dk = a.dk, dv = a.dv, slices = (dv + 16 * kDfWaves - 1) / (16 * kDfWaves);
    const int64_t task = blockIdx.x / slices, b = task / a.Hv;
    const int n = (int)(task - b * a.Hv), col0 = (blockIdx.x % slices * kDfWaves + wave) * 16, col = col0 + (int)l16;
    if (col0 >= dv) return;   // (nothing waits for this wave)
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;

    const auto row_of = [&](int kt) { return BF16 ? kt / 2 * 32 + (int)g * 8 + kt % 2 * 4 : 16 * kt + 4 * (int)g; };
    float* const sp = a.state && in ? a.state + (slot * a.Hv + n) * dk * (int64_t)dv : nullptr;
    V4 S[KT] = {};
    if (sp && !a.fresh && col < dv && len > 0)
#pragma unroll
        for (int i = 0; i < 4 * KT; ++i) {
            const int row = row_of(i / 4) + i % 4;
            if (row < dk) S[i / 4][i % 4] = gmem(sp)[row * dv + col];
        }
    const T* const kp = static_cast<const T*>(a.k.p) + b * a.k.row + n / a.G * a.k.head;
    const T* const qp = static_cast<const T*>(a.q.p) + b * a.q.row + n / a.G * a.q.head;
    const T* const vp = static_cast<const T*>(a.v.p) + b * a.v.row + n * a.v.head + (col < dv ? col : col0);
    const float* const ldp = static_cast<const float*>(a.ld.p) + b * a.ld.row + n * a.ld.head;
    const float* const bp = static_cast<const float*>(a.beta.p) + b * a.beta.row + n * a.beta.head;
    Frag fk[NK], fq[NK];
    float fv[4], fld, fbeta;
    // a chunk's: rows past the row's end repeat its last, and weigh nothing (beta is 0 there)
    const auto fetch = [&](int t0) {
        const int most = len - 1 - t0, r = (int)l16 < most ? (int)l16 : most;
        const T *k = kp + (int64_t)(t0 + r) * a.k.pos, *q = qp + (int64_t)(t0 + r) * a.q.pos;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            const int c = kb * KB + (int)g * E;
            fk[kb] = fq[kb] = Frag{};
            if (c < dk) {
                if constexpr (VEC) {
                    fk[kb] = *gmem(reinterpret_cast<const Frag*>(k + c));
                    fq[kb] = *gmem(reinterpret_cast<const Frag*>(q + c));
                } else {
                    fk[kb] = load_loose<BF16>(k, c, dk);
                    fq[kb] = load_loose<BF16>(q, c, dk);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int p = 4 * (int)g + i < most ? 4 * (int)g + i : most;
            fv[i] = (float)gmem(vp)[(int64_t)(t0 + p) * a.v.pos];
        }
        fld = fbeta = 0.f;
        if ((int)l16 <= most) {
            fld = gmem(ldp)[(int64_t)(t0 + (int)l16) * a.ld.pos];
            fbeta = gmem(bp)[(int64_t)(t0 + (int)l16) * a.beta.pos];
        }
    };
    const auto place = [](uint32_t row, uint32_t u) -> uint32_t {   // as in k_delta_chunk
        constexpr int UNITS = DK / E;
        const uint32_t m = !BF16 ? row % 16 : UNITS == 8 ? 4 * (row / 2 % 2) + row / 4 % 4 : 4 * (row % 4) + row / 4 % 4;
        return (row * UNITS + (u ^ m)) * E;
    };
    // four values as the first half of an operand over KB positions, the rest of which are none
    const auto operand = [](V4 x, auto& f) {
        constexpr int N = sizeof(f) / sizeof(f[0]);
        const V4 both[2] = {x, {0.f, 0.f, 0.f, 0.f}};
        split<BF16, N>(both, f);
    };
    if (len > 0) fetch(0);
    for (int t0 = 0; t0 < len; t0 += C) {
        const int left = len - t0;
        const bool moves = !a.hold || t0 + C < len;   // the state is needed again
        const Gate mine = gate_sum<C>(fld);
        if (g == 0) {
            gs[0][l16] = mine.hi;
            gs[1][l16] = mine.lo;
            gs[2][l16] = fbeta;
        }
        if (moves)
#pragma unroll
            for (int kb = 0; kb < NK; ++kb) *smem_ptr(reinterpret_cast<Frag*>(ks + place(l16, kb * 4 + g))) = fk[kb];
        wave_order();
        const V4 hi = *smem_ptr(reinterpret_cast<const V4*>(&gs[0][4 * g])), lo = *smem_ptr(reinterpret_cast<const V4*>(&gs[1][4 * g])),
                 beta = *smem_ptr(reinterpret_cast<const V4*>(&gs[2][4 * g]));
        const Gate zero = {0.f, 0.f}, end = {gs[0][C - 1], gs[1][C - 1]};
        // K K^T (rows i = 4 g + r, column j = l16) and its mirror for P (rows j, column i)
        V4 p = {0.f, 0.f, 0.f, 0.f}, w = p;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            p = M::mma(fk[kb], fk[kb], p);
            w = M::mma(fk[kb], fq[kb], w);
        }
        V4 from_start, to_end;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int i = 4 * (int)g + r;
            const Gate at = {hi[r], lo[r]};
            const float x = beta[r] * exp_of(at, mine) * p[r], y = w[r] * exp_of(mine, at);
            as[i][l16] = (int)l16 < i ? x : 0.f;
            w[r] = i <= (int)l16 ? y : 0.f;
            from_start[r] = exp_of(at, zero);
            to_end[r] = exp_of(end, at);
        }
        __builtin_amdgcn_sched_barrier(0);   // (here and below: operands are not all read, and kept, before their use)
        // K E, and O^T = E^T Q^T
        V4 R = {0.f, 0.f, 0.f, 0.f}, O = R;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
            Frag f[PARTS];
            split<BF16, PARTS>(&S[kb * PER], f);
#pragma unroll
            for (int i = PARTS - 1; i >= 0; --i) {
                R = M::mma(fk[kb], f[i], R);
                if (i < HALF) O = M::mma(f[i], fq[kb], O);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        wave_order();
        // row l16 of (I + A)^{-1}: x (I + A) = e, from the last column on
        float x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = j == (int)l16 ? 1.f : 0.f;
#pragma unroll
        for (int k = 15; k > 0; --k) {
            if (k >= left) continue;   // (rows of no positions are the identity's)
#pragma unroll
            for (int j0 = 0; j0 < k; j0 += 4) {
                const V4 y = *smem_ptr(reinterpret_cast<const V4*>(&as[k][j0]));
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j0 + j < k) x[j0 + j] = fmaf(-x[k], y[j], x[j0 + j]);
            }
        }
        V4 tt, v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            tt[r] = (g == 0 ? x[r] : g == 1 ? x[4 + r] : g == 2 ? x[8 + r] : x[12 + r]) * beta[r];
            v[r] = fmaf(-from_start[r], R[r], fv[r]);
        }
        const float mine_start = exp_of(mine, zero);
        if (t0 + C < len) fetch(t0 + C);
        // U = T R, O = e^G Q E + P U
        V4 U = {0.f, 0.f, 0.f, 0.f};
        {
            Frag f[PARTS], h[PARTS];
            operand(tt, f);
            operand(v, h);
#pragma unroll
            for (int i = PARTS - 1; i >= 0; --i)
#pragma unroll
                for (int j = PARTS - 1 - i; j >= 0; --j) U = M::mma(f[i], h[j], U);
        }
        {
            Frag f[HALF], h[HALF];
            operand(U, f);
            operand(w, h);
            O *= mine_start;
#pragma unroll
            for (int i = HALF - 1; i >= 0; --i)
#pragma unroll
                for (int j = HALF - 1 - i; j >= 0; --j) O = M::mma(f[i], h[j], O);
        }
        if ((int)l16 < left) {
            Four y;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = (T)(a.scale * O[r]);
            T* const to = static_cast<T*>(a.o.p) + b * a.o.row + n * a.o.head + (int64_t)(t0 + (int)l16) * a.o.pos + col0 + 4 * (int)g;
            const int room = dv - (col0 + 4 * (int)g);
            if constexpr (VEC) {
                if (room > 0) *gmem(reinterpret_cast<Four*>(to)) = y;
            } else
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r < room) gmem(to)[r] = y[r];
        }
        __builtin_amdgcn_sched_barrier(0);
        if (moves) {
            const float whole = exp_of(end, zero);
            decayed<!BF16>(expm1f(end.hi) + whole * end.lo, whole, [&](auto to) {
#pragma unroll
                for (int i = 0; i < 4 * KT; ++i) S[i / 4][i % 4] = to(S[i / 4][i % 4]);
            });
            Frag f[PARTS];
            operand(U * to_end, f);
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                Frag k = {};
                if constexpr (BF16) {
                    const T* q = ks + place(4 * g + l16 / 4, kt / 2 * 4 + l16 % 4) + kt % 2 * 4;
                    const BF4 y = __builtin_bit_cast(BF4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((FI_SHARED S4*)(q)));
#pragma unroll
                    for (int e = 0; e < 4; ++e) k[e] = y[e];
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) k[e] = smem_ptr(ks)[place(4 * g + e, 4 * kt + l16 / 4) + l16 % 4];
                }
#pragma unroll
                for (int i = PARTS - 1; i >= 0; --i) S[kt] = M::mma(k, f[i], S[kt]);
                if (kt % 4 == 3) __builtin_amdgcn_sched_barrier(0);
            }
        }
        wave_order();
    }
    if (sp && !a.hold && (len > 0 || a.fresh) && col < dv)
#pragma unroll
        for (int i = 0; i < 4 * KT; ++i) {
            const int row = row_of(i / 4) + i % 4;
            if (row < dk) gmem(sp)[row * dv + col] = S[i / 4][i % 4];
        }
    for (int t = len + (int)g; t < a.L; t += 4)   // o is zero past the row's end
        if (col < dv) gmem(static_cast<T*>(a.o.p))[b * a.o.row + n * a.o.head + (int64_t)t * a.o.pos + col] = (T)0.f;
}

template <bool BF16>
static void delta_few(const DeltaCall& c, hipStream_t st) {
    const unsigned grid = (unsigned)(c.B * c.Hv * ((c.dv + 16 * kDfWaves - 1) / (16 * kDfWaves)));   // B Hv <= kLattnMaxRows
    const auto go = [&](auto dk) {
        constexpr int DK = decltype(dk)::value;
        if (c.vec) k_delta_few<BF16, DK, true><<<grid, kDfWaves * kWave, 0, st>>>(c);
        else k_delta_few<BF16, DK, false><<<grid, kDfWaves * kWave, 0, st>>>(c);
    };
    if (c.dk <= 64) go(std::integral_constant<int, 64>{});
    else if (c.dk <= 128) go(std::integral_constant<int, 128>{});
    else go(std::integral_constant<int, 256>{});
}

static hipError_t launch_delta_few(const DeltaCall& c, hipStream_t st) {
    if (c.io_bf16) delta_few<true>(c, st);
    else delta_few<false>(c, st);
    return hipGetLastError();
}

// States before a split row's segments, in place: ent[s + 1] holds what segment s
// makes of zero and becomes M_s ent[s] + that; ent[0] is the row's state.
// A workgroup has a slice of 16 columns, a wave 16 rows of it; they meet in LDS.  What
// the next segment needs is asked for a segment ahead.
constexpr int dj_threads(int dk) { return dk / 16 * kWave; }
template <int DK>
__global__ __launch_bounds__(dj_threads(DK)) void k_delta_join(DeltaCall a, int C) {
    constexpr int KT = DK / 16, NTH = dj_threads(DK), PE = DK + 4;   // LDS columns
    constexpr bool AHEAD = DK <= 128;                                 // (registers for one segment's M only)
    __shared__ __align__(16) float es[2][16 * PE];                    // the state, transposed
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave), l16 = lane % 16, g = lane / 16;
    const int dk = a.dk, dv = a.dv, slices = (dv + 15) / 16;
    const int64_t task = blockIdx.x / slices, b = task / a.Hv;
    const int n = (int)(task - b * a.Hv), col0 = blockIdx.x % slices * 16, col = col0 + l16;
    const int64_t slot = a.slots ? a.slots[b] : b;
    if (slot < 0 || slot >= a.n_slots) return;
    int len = a.lens ? a.lens[b] : a.L;
    len = len < 0 ? 0 : len > a.L ? a.L : len;
    const int chunks = (len + C - 1) / C, stop = a.chunk0 + a.chunks < chunks ? a.chunk0 + a.chunks : chunks;
    const int segs = stop <= a.chunk0 ? 1 : (stop - a.chunk0 + a.seg_chunks - 1) / a.seg_chunks;
    float* const ent = a.ent + task * a.nseg * dk * dv;
    const float* const mine = a.move + task * a.nseg * DK * DK + (16 * wave + l16) * DK + 4 * g;
    const int row0 = 16 * wave + 4 * g;
    V4 m[KT], ahead[AHEAD ? KT : 1], add, next = {0.f, 0.f, 0.f, 0.f};
    const auto ask = [&](int s, auto& x, V4& y) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) x[kt] = *gmem(reinterpret_cast<const V4*>(mine + (int64_t)s * DK * DK + 16 * kt));
        const float* const p = ent + (int64_t)(s + 1) * dk * dv;
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = row0 + r < dk && col < dv ? gmem(p)[(row0 + r) * dv + col] : 0.f;
    };
    if (segs > 1) ask(0, m, add);
    const float* const from = a.chunk0 ? a.carry + task * dk * dv : a.fresh || !a.state ? nullptr : a.state + (slot * a.Hv + n) * dk * (int64_t)dv;
    for (int i = tid; i < 16 * DK; i += NTH) {
        const int row = i / 16, c = col0 + i % 16;
        const float x = from && row < dk && c < dv ? gmem(from)[row * dv + c] : 0.f;
        es[0][i % 16 * PE + row] = x;
        if (row < dk && c < dv) gmem(ent)[row * dv + c] = x;
    }
    __syncthreads();
    for (int s = 0; s + 1 < segs; ++s) {
        if constexpr (AHEAD) {
            if (s + 2 < segs) ask(s + 1, ahead, next);
        }
        V4 acc[2] = {add, {0.f, 0.f, 0.f, 0.f}};   // two, as a product waits for the one before
        if (s || from)   // (before a fresh row's first segment there is nothing, and M_0 is not formed)
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
                acc[kt % 2] = Mm<false>::mma(m[kt], *smem_ptr(reinterpret_cast<const V4*>(&es[s % 2][l16 * PE + 16 * kt + 4 * g])), acc[kt % 2]);
        acc[0] += acc[1];
        *smem_ptr(reinterpret_cast<V4*>(&es[(s + 1) % 2][l16 * PE + row0])) = acc[0];
        float* const to = ent + (int64_t)(s + 1) * dk * dv;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (row0 + r < dk && col < dv) gmem(to)[(row0 + r) * dv + col] = acc[0][r];
        if constexpr (AHEAD) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) m[kt] = ahead[kt];
            add = next;
        } else if (s + 2 < segs) ask(s + 1, m, add);
        __syncthreads();
    }
}

namespace {

// Chunks of all heads whose systems are held at a time (bf16: 436 MB), and of each head at least (53 KB; each
// further run of chunks reads and writes the state, 64 KB of 128 x 128, once more).
constexpr int64_t kDlTri = 32768, kDlTriEach = 4;
int64_t dl_held(int64_t tasks) { return std::max(kDlTri / tasks, kDlTriEach); }
constexpr int64_t kDlWorkgroups = 256;  // wanted of a launch

int dl_chunk(int io_bf16) { return io_bf16 ? Dl<true>::C : Dl<false>::C; }
int64_t dl_floats(int io_bf16) { return io_bf16 ? Dl<true>::TRI + Dl<true>::GATES : Dl<false>::TRI + Dl<false>::GATES; }
int64_t dl_wide(int dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }   // keys of the kernels
int dl_cols(int dk) { return dk <= 64 ? 64 : 128; }
// Each chunk of a segment takes its time twice, and some 40 us go into segments' states and
// their join: rows are split into kDlFewest segments of kDlLeast chunks at least (us, 16 heads of 128 x 128, bf16, one row
// of 512: unsplit 51, in 2 75; of 1024: 87, in 2 116, in 4 83; 8 rows of 1000: 106, in 2 162; 4 rows of 2048:
// 223, in 4 186).
constexpr int64_t kDlLeast = 4, kDlFewest = 4;
// Rows that are not split, and leave CUs empty: slices of 64 columns for 128 (the same heads, one row of
// 512: 61 -> 51 us, 8 of 512 73 -> 63).
constexpr int64_t kDlNarrow = 128;      // slices of such a launch


// (WAVES x NC columns of 16 to a slice; the segments' pass may share them out otherwise)
template <bool BF16, int DK, int WAVES, int NC, int SWAVES, int SNC, bool VEC>
void delta_launches(const DeltaCall& c, hipStream_t st) {
    constexpr int DVS = 16 * NC * WAVES;
    static_assert(WAVES * NC == SWAVES * SNC, "the same slices");
    const int64_t tasks = c.B * c.Hv, units = tasks * c.nseg;
    const int values = (c.dv + DVS - 1) / DVS, all = values + (c.dk + DVS - 1) / DVS;
    k_delta_tri<BF16, DK, VEC><<<(unsigned)(tasks * c.chunks), Dl<BF16>::CT * kWave, 0, st>>>(c);
    if (c.nseg > 1) {
        k_delta_chunk<BF16, DK, SWAVES, SNC, false, VEC><<<(unsigned)((units + 7) / 8 * 8 * all), SWAVES * kWave, 0, st>>>(c);
        k_delta_join<DK><<<(unsigned)(tasks * ((c.dv + 15) / 16)), dj_threads(DK), 0, st>>>(c, Dl<BF16>::C);
    }
    k_delta_chunk<BF16, DK, WAVES, NC, true, VEC><<<(unsigned)((units + 7) / 8 * 8 * values), WAVES * kWave, 0, st>>>(c);
}

template <bool BF16>
void delta_dims(const DeltaCall& c, hipStream_t st) {
    if (c.dk <= 64) c.vec ? delta_launches<BF16, 64, 4, 1, 4, 1, true>(c, st) : delta_launches<BF16, 64, 4, 1, 4, 1, false>(c, st);
    else if (c.dk <= 128 && c.narrow) c.vec ? delta_launches<BF16, 128, 4, 1, 4, 1, true>(c, st) : delta_launches<BF16, 128, 4, 1, 4, 1, false>(c, st);
    else if (c.dk <= 128) c.vec ? delta_launches<BF16, 128, 8, 1, 4, 2, true>(c, st) : delta_launches<BF16, 128, 8, 1, 4, 2, false>(c, st);
    else c.vec ? delta_launches<BF16, 256, 4, 2, 4, 2, true>(c, st) : delta_launches<BF16, 256, 4, 2, 4, 2, false>(c, st);
}

}  // namespace

// By steps up to a few positions, then chunks of 16 in one launch, then systems of whole
// chunks (us, heads of 128 x 128, 32 on 16, with states, steps / 16 / whole.  bf16, one row of 3: 9 / 10
// / 20, of 5: 10 / 10 / 20, of 48: - / 19 / 21, of 64: - / 23 / 21; 64 rows of 2: 50 / 66 / 129, of 5: 88 / 68 / 130,
// of 48: - / 133 / 140, of 64: - / 158 / 146.  fp32, whose products take longer, 64 rows of 5: 91 / 122 / 148, of 8:
// 125 / - / 148, of 16: 238 / 143 / 151, of 32: - / 215 / 160; one row of 32: 38 / 20 / 24, of 48: - / 25 / 32).
// Other head sizes go by the same borders, which were not measured for them.
DeltaRoute delta_route(const DeltaCall& c) {
    if (c.L <= (c.io_bf16 ? 3 : 6)) return DeltaRoute::steps;
    const bool busy = c.B * c.Hv > 512;   // the CUs are full
    return c.L <= (c.io_bf16 || !busy ? 48 : 16) ? DeltaRoute::few : DeltaRoute::chunks;
}

void plan_delta(DeltaCall& c) {
    const int C = dl_chunk(c.io_bf16);
    const int64_t tasks = c.B * c.Hv, all = (c.L + C - 1) / C, most = dl_held(tasks);
    c.chunk0 = 0;
    c.chunks = (int)(all < most ? all : most);
    const int slices = (c.dv + dl_cols(c.dk) - 1) / dl_cols(c.dk);
    int64_t n = kDlWorkgroups / (tasks * slices);
    if (n > c.chunks / kDlLeast) n = c.chunks / kDlLeast;
    if (n < kDlFewest) n = 1;
    c.narrow = n == 1 && c.dk > 64 && c.dk <= 128 && tasks * slices <= kDlNarrow;
    c.seg_chunks = c.chunks ? (int)((c.chunks + n - 1) / n) : 1;
    c.nseg = c.chunks ? (c.chunks + c.seg_chunks - 1) / c.seg_chunks : 1;
}

namespace {

// the workspace's parts, in floats; whole 16-byte units, in which systems and moves are read
struct DeltaParts {
    size_t tri, ent, move, carry;
    size_t all() const { return tri + ent + move + carry; }
};
DeltaParts delta_parts(const DeltaCall& c) {
    const size_t tasks = (size_t)c.B * c.Hv, states = (size_t)c.dk * c.dv, segs = c.nseg > 1 ? tasks * c.nseg : 0;
    const int C = dl_chunk(c.io_bf16);
    return {tasks * c.chunks * dl_floats(c.io_bf16), (segs * states + 3) / 4 * 4, segs * dl_wide(c.dk) * dl_wide(c.dk),
            (c.L + C - 1) / C > c.chunks ? tasks * states : 0};
}

}  // namespace

size_t delta_ws_used(const DeltaCall& c) { return delta_route(c) != DeltaRoute::chunks ? 0 : delta_parts(c).all() * sizeof(float); }

size_t delta_ws_bytes(int64_t B, int64_t L, int Hv, int dk, int dv, int io_bf16) {
    DeltaCall c = {};
    c.L = (int)L;
    c.B = B, c.Hv = Hv, c.io_bf16 = io_bf16;
    if (delta_route(c) != DeltaRoute::chunks) return 0;   // nor do smaller calls
    const int64_t C = dl_chunk(io_bf16), tasks = B * Hv, chunks = (L + C - 1) / C;
    // systems: of all chunks, or of as many as are held at a time of any call
    const int64_t tri = std::min(tasks * chunks, std::max(kDlTri, tasks * kDlTriEach));
    // segments: at most kDlWorkgroups over all heads and slices of any call
    const int slices = (dv + dl_cols(dk) - 1) / dl_cols(dk);
    const int64_t segs = chunks >= kDlFewest * kDlLeast ? kDlWorkgroups / slices : 0;
    const int64_t carry = chunks > dl_held(tasks) ? tasks * dk * dv : 0;
    return (size_t)(tri * dl_floats(io_bf16) + (segs * dk * dv + 3) / 4 * 4 + segs * dl_wide(dk) * dl_wide(dk) + carry) * sizeof(float);
}

void place_delta(DeltaCall& c, float* ws) {
    const DeltaParts p = delta_parts(c);
    c.tri = ws;
    c.ent = c.tri + p.tri;
    c.move = c.ent + p.ent;
    c.carry = p.carry ? c.move + p.move : nullptr;
}

hipError_t launch_delta_prompt(DeltaCall c, float* ws, hipStream_t st) {
    const DeltaRoute route = delta_route(c);
    if (route == DeltaRoute::steps) return launch_delta_step(c, st);
    if (route == DeltaRoute::few) return launch_delta_few(c, st);
    plan_delta(c);
    place_delta(c, ws);
    const int C = dl_chunk(c.io_bf16), all = (c.L + C - 1) / C, held = c.chunks;
    do {
        if (all - c.chunk0 < held) c.chunks = all - c.chunk0;
        if (c.io_bf16) delta_dims<true>(c, st);
        else delta_dims<false>(c, st);
        c.chunk0 += held;
    } while (c.chunk0 < all);
    return hipGetLastError();
}

}  // namespace fi

// fi_rotary.hip -- queries and keys normed for each head and turned by their
// position, in one pass (fi_rotary_*).
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

constexpr int kRoThreads = 256, kRoWaves = kRoThreads / kWave;

// cos and sin of 2 pi x, x in turns: reduced in 64 bits to at most an eighth of
// a turn, where the series to the 9th and 10th power are off by less than 3e-9.
__device__ __forceinline__ void turn(double x, float& cos_, float& sin_) {
    x -= rint(x);
    const double q = rint(4.0 * x);
    const float t = (float)(fma(q, -0.25, x)) * 6.28318530717958648f, s = t * t;
    float a = fmaf(s, 1.f / 362880.f, -1.f / 5040.f);
    a = fmaf(s, a, 1.f / 120.f);
    a = fmaf(s, a, -1.f / 6.f);
    a = fmaf(t * s, a, t);
    float c = fmaf(s, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(s, c, -1.f / 720.f);
    c = fmaf(s, c, 1.f / 24.f);
    c = fmaf(s, c, -0.5f);
    c = fmaf(s, c, 1.f);
    const int quarter = (int)q & 3;
    const float sn = quarter & 1 ? c : a, cs = quarter & 1 ? a : c;
    sin_ = quarter & 2 ? -sn : sn;
    cos_ = (quarter + 1) & 2 ? -cs : cs;
}

// A wave takes a position, and passes over its heads (or a share of them)
// with 2^log lanes to a head.  A lane has P pairs of units of E elements, of
// which both halves of every pair to be turned are its own: nothing is
// exchanged but the sum of squares.  The position's angles are formed once.
// Bound by memory: 16384 positions of 32 + 8 heads of 128, bf16 (336 MB), 74 us, 4.5 TB/s (a
// copy 5.0), the vector units 65% busy (without the next pass's loads ahead 80 us).  A few tokens: 4.4 us, a launch
// and a trip to memory.
// PART: some elements are not turned, and are chosen as they are (as a turn by 0 an infinity or a NaN
// would reach its neighbour): two choices a pair, 16384 positions of 40 heads of 80, 48 of them
// turned, 49 us for 46; heads that are turned whole go without.
template <bool BF16, int E, int P, bool ADJACENT, bool PART>
__global__ __launch_bounds__(kRoThreads) void k_rotary(RotaryCall a, int log, int64_t positions) {
    using T = typename Mm<BF16>::T;
    using Unit = T __attribute__((ext_vector_type(E)));
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int lanes = 1 << log, l = lane & (lanes - 1), mine = lane >> log, each = kWave >> log;   // heads of a pass
    const int d = a.d, heads = a.Hq + a.Hk, passes = (heads + each - 1) / each, half = a.rot / 2;
    // the lane's units, and the index of its first pair (turned where below half)
    int c0[P], c1[P], pair[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
        const int j = l + p * lanes;
        if (ADJACENT) c0[p] = 2 * E * j, c1[p] = c0[p] + E, pair[p] = E * j;
        else if (E * j < half) c0[p] = E * j, c1[p] = c0[p] + half, pair[p] = E * j;
        else c0[p] = a.rot + 2 * (E * j - half), c1[p] = c0[p] + E, pair[p] = half;
    }
    const int64_t total = positions * a.shares;
    for (int64_t id = (int64_t)blockIdx.x * kRoWaves + wave; id < total; id += (int64_t)gridDim.x * kRoWaves) {
        const int64_t at = id / a.shares, b = at / a.L;
        const int share = (int)(id - at * a.shares), t = (int)(at - b * a.L);
        const int64_t where = a.positions ? a.positions[at] : a.first ? (int64_t)a.first[b] + t : t;
        // a pass's units are asked for a pass ahead, the first before the angles are formed
        Unit next[P][2] = {};
        const auto load = [&](int pass) {
            const int h = pass * each + mine;
            const bool key = h >= a.Hq, some = h < heads;
            const View& from = key ? a.k : a.q;
            const T* const x = static_cast<const T*>(from.p) + b * from.row + t * from.pos + (key ? h - a.Hq : h) * from.head;
#pragma unroll
            for (int p = 0; p < P; ++p) {
                if (some && c0[p] < d) next[p][0] = *gmem(reinterpret_cast<const Unit*>(x + c0[p]));
                if (some && c1[p] < d) next[p][1] = *gmem(reinterpret_cast<const Unit*>(x + c1[p]));
            }
        };
        load(share);
        float cs[P][E], sn[P][E];
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                cs[p][e] = 1.f, sn[p][e] = 0.f;
                if (pair[p] + e < half) turn((double)where * gmem(a.turns)[pair[p] + e], cs[p][e], sn[p][e]);
            }
        for (int pass = share; pass < passes; pass += a.shares) {
            const int h = pass * each + mine;
            const bool key = h >= a.Hq, some = h < heads;
            const View& to = key ? a.ko : a.qo;
            T* const y = static_cast<T*>(to.p) + b * to.row + t * to.pos + (key ? h - a.Hq : h) * to.head;
            const T* const w = static_cast<const T*>(key ? a.wk : a.wq);
            Unit u[P][2];
#pragma unroll
            for (int p = 0; p < P; ++p) u[p][0] = next[p][0], u[p][1] = next[p][1];
            if (pass + a.shares < passes) load(pass + a.shares);
            float v[P][2 * E], sum = 0.f;
#pragma unroll
            for (int p = 0; p < P; ++p)
#pragma unroll
                for (int e = 0; e < 2 * E; ++e) {
                    v[p][e] = (float)u[p][e / E][e % E];
                    sum = fmaf(v[p][e], v[p][e], sum);
                }
            if (a.norm) {
                for (int i = 1; i < lanes; i <<= 1) sum += __shfl_xor(sum, i);
                const float f = 1.f / sqrtf((a.norm == 1 ? sum / (float)d : sum) + a.eps);
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int e = 0; e < 2 * E; ++e) v[p][e] *= f;
            }
            if (w) {
                Unit f[P][2] = {};
#pragma unroll
                for (int p = 0; p < P; ++p) {
                    if (some && c0[p] < d) f[p][0] = *gmem(reinterpret_cast<const Unit*>(w + c0[p]));
                    if (some && c1[p] < d) f[p][1] = *gmem(reinterpret_cast<const Unit*>(w + c1[p]));
#pragma unroll
                    for (int e = 0; e < 2 * E; ++e) v[p][e] *= (float)f[p][e / E][e % E];
                }
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                Unit r[2];
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const int i = ADJACENT ? 2 * e : e, j = ADJACENT ? 2 * e + 1 : E + e;
                    // (what is not turned is no pair: an infinity or a NaN stays by itself)
                    const bool turned = !PART || pair[p] + e < half;
                    r[i / E][i % E] = (T)(turned ? fmaf(v[p][i], cs[p][e], -v[p][j] * sn[p][e]) : v[p][i]);
                    r[j / E][j % E] = (T)(turned ? fmaf(v[p][j], cs[p][e], v[p][i] * sn[p][e]) : v[p][j]);
                }
                if (some && c0[p] < d) *gmem(reinterpret_cast<Unit*>(y + c0[p])) = r[0];
                if (some && c1[p] < d) *gmem(reinterpret_cast<Unit*>(y + c1[p])) = r[1];
            }
        }
    }
}

namespace {

constexpr int64_t kRoWanted = 4096;        // waves wanted of a launch
constexpr int64_t kRoBlocks = 1 << 16;     // workgroups of a launch at most

template <bool BF16, int E, int P, bool ADJACENT, bool PART>
void rotary_launch(const RotaryCall& c, int log, int64_t positions, unsigned grid, hipStream_t st) {
    k_rotary<BF16, E, P, ADJACENT, PART><<<grid, kRoThreads, 0, st>>>(c, log, positions);
}
template <bool BF16, int E, int P>
void rotary_go(RotaryCall c, hipStream_t st) {
    const int pairs = (c.d + 2 * E - 1) / (2 * E);   // of units, of a head
    int log = 0;
    while (P << log < pairs) ++log;
    const int64_t positions = c.B * c.L;
    const int each = kWave >> log, passes = (c.Hq + c.Hk + each - 1) / each;
    int64_t shares = kRoWanted / positions;
    c.shares = (int)(shares < 1 ? 1 : shares > passes ? passes : shares);
    const int64_t blocks = (positions * c.shares + kRoWaves - 1) / kRoWaves;
    const unsigned grid = (unsigned)(blocks < kRoBlocks ? blocks : kRoBlocks);
    const bool part = c.rot < c.d;
    if (c.pairs) part ? rotary_launch<BF16, E, P, true, true>(c, log, positions, grid, st) : rotary_launch<BF16, E, P, true, false>(c, log, positions, grid, st);
    else part ? rotary_launch<BF16, E, P, false, true>(c, log, positions, grid, st) : rotary_launch<BF16, E, P, false, false>(c, log, positions, grid, st);
}

template <bool BF16>
void rotary_unit(const RotaryCall& c, hipStream_t st) {
    // (a head of 256 elements has 128 pairs: two for each lane where a unit is one element)
    if (c.unit == 1) rotary_go<BF16, 1, 2>(c, st);
    else if (c.unit == 2) rotary_go<BF16, 2, 1>(c, st);
    else if (c.unit == 4) rotary_go<BF16, 4, 1>(c, st);
    else if constexpr (BF16) rotary_go<BF16, 8, 1>(c, st);
}

}  // namespace

hipError_t launch_rotary(RotaryCall c, hipStream_t st) {
    if (c.io_bf16) rotary_unit<true>(c, st);
    else rotary_unit<false>(c, st);
    return hipGetLastError();
}

}  // namespace fi

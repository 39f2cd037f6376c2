// fi_verify.hip -- drafted tokens against the target's probabilities (fi_verify_*).
//
// Everything is held in 64 bits, powers to 2^-48 of themselves: which token a random number falls on depends
// on running sums of up to 2^31 probabilities, whose borders lie closer than
// fp32 tells apart.
//
// Three launches: sums of all rows of logits; what is kept, and the weights that the token
// is drawn from; the token.  64 rows of up to 5 drafts x 100003, bf16 (77 MB: 16 us): 35 + 18 + 6.4 us;
// 96 of 8 x 32768 without drafts' logits (57 MB) 24 + 10.4 + 5; one row of 4 x 131072, fp32, 4.8 + 6.7 + 5.0.
// The sums are 11 operations of 64 bits and 5 around them for each logit, which keep the vector units 50 to 59% busy, with 3
// waves of a SIMD on average (parts of places without drafts have none); the rest is waits.  With the series alone (23 operations of 64 bits, some of them slow
// ones) the sums took 69 us.  More waves at a time (64 registers) change nothing.
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

constexpr int kVeThreads = 256, kVeWaves = kVeThreads / kWave;
constexpr int kVeRun = 8;                          // logits of a thread that follow one another
constexpr int kVeBlock = kVeThreads * kVeRun;      // logits of a workgroup at a time
constexpr int kVeMaxParts = 2 * kWave, kVeMaxBlocks = 2 * kWave;
constexpr int kVeMaxDrafts = 63, kVeMaxRows = 2 * kVeMaxDrafts + 1;
constexpr int kVeTable = 256;                      // powers of an octave
constexpr double kVeLow = -1020.0 * kVeTable;      // the least power that is formed
constexpr double kVeNone = -1e300;                 // the reference of a part without a token

// 2^{x / 256} for kVeLow <= x <= 256000 to 2^-48 of itself: n = rint(x), 2^{n / 256} from a
// table in LDS and an exponent, and the series of e^{r ln 2 / 256}, r = x - n, to the 4th power (the
// next term is 4e-17).  The table's entry i is less i << 12 in its high word, so that n << 12 is added whole.
// Scales come with the 256, so that an operation has one constant at most.  (With 32 entries and the 5th
// power, and the exponent put into the product, the sums took 42 us for 35, 27 for 24.)
struct Powers {
    const FI_SHARED double* table;
    double first;   // (ln 2 / 256)^4 / 4!, kept in a register
};
__device__ __forceinline__ Powers make_powers(double* t, int tid) {
    if (tid < kVeTable)
        t[tid] = __longlong_as_double(__double_as_longlong(exp2((double)tid / kVeTable)) - ((long long)tid << 44));
    double first = 2.239395190875157e-12;
    asm("" : "+v"(first));
    return {smem_ptr(t), first};
}
struct Factors {
    double scale, series;
};
constexpr double kVeShift = 6755399441055744.0;   // 1.5 2^52: a sum's lowest bits are the nearest whole number
__device__ __forceinline__ Factors raised(double k, double r, const Powers& to) {   // k = n + kVeShift
    using Words = uint32_t __attribute__((ext_vector_type(2)));
    const uint32_t n = (uint32_t)(uint64_t)__double_as_longlong(k);
    double p = __builtin_fma(r, to.first, 3.308302680541371e-09);   // the 3rd power's, and so on
    p = __builtin_fma(r, p, 3.665565596910106e-06);
    p = __builtin_fma(r, p, 0.0027076061740622863);
    p = __builtin_fma(r, p, 1.0);
    Words t = __builtin_bit_cast(Words, (double)to.table[n & (kVeTable - 1)]);
    t.y += n << 12;
    return {__builtin_bit_cast(double, t), p};
}
__device__ __forceinline__ Factors power(double x, const Powers& to) {
    const double k = x + kVeShift;
    return raised(k, x - (k - kVeShift), to);
}
constexpr double kVeLeast = 0x1p-1020;   // 2^{kVeLow / 256}
// What a sum against `ref` is times against the larger reference `now`.
__device__ __forceinline__ double share(double ref, double now, double c, const Powers& to) {
    const Factors f = power(fmax((ref - now) * c, kVeLow), to);
    return f.scale * f.series;
}
// A logit's weight against the reference; what is far below it or -inf weighs nothing: the clamped
// power is kVeLeast, without a rounding.
__device__ __forceinline__ double weight(float z, double ref, double c, const Powers& to) {
    const Factors f = power(fmax(((double)z - ref) * c, kVeLow), to);
    return __builtin_fma(f.scale, f.series, -kVeLeast);
}

__device__ __forceinline__ int drafts_of(const VerifyCall& a, int64_t b) {
    const int n = a.lens ? a.lens[b] : a.N;
    return n < 0 ? 0 : n > a.N ? a.N : n;
}
__device__ __forceinline__ int rows_of(const VerifyCall& a) { return a.draft ? 2 * a.N + 1 : a.N + 1; }   // of logits, for a row

// Row i of logits of row b: the target's at place i <= N, then the drafts'.
template <bool BF16>
__device__ __forceinline__ const typename Mm<BF16>::T* logits_of(const VerifyCall& a, int64_t b, int i) {
    using T = typename Mm<BF16>::T;
    return i <= a.N ? static_cast<const T*>(a.target) + b * a.target_row + i * a.target_ld
                    : static_cast<const T*>(a.draft) + b * a.draft_row + (i - a.N - 1) * a.draft_ld;
}

// A wave takes one part of one row of logits: the sum of 2^((z - R) c / 256) with a reference R near the
// largest z (differences first: they are exact, however large the logits are).  A row
// that is no distribution has a sum that is NaN or 0.
template <bool BF16>
__global__ __launch_bounds__(kVeThreads) void k_verify_sums(VerifyCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    using Loose = T __attribute__((ext_vector_type(M::E), aligned(sizeof(T))));
    constexpr int E = M::E, UN = 16 / E, STEP = kWave * E;
    __shared__ double table_[kVeTable];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), rows = rows_of(a);
    const int64_t unit = (int64_t)blockIdx.x * kVeWaves + wave, row = unit / a.parts, b = row / rows;
    const int i = (int)(row - b * rows);
    bool here = b < a.B;
    if (here) {
        const int n = drafts_of(a, b);
        here = i <= a.N ? i <= n : i - a.N - 1 < n;   // a draft there
    }
    const T* const z = here ? logits_of<BF16>(a, b, i) : nullptr;
    const double c = i <= a.N ? a.scale : a.draft_scale;
    const int64_t v0 = (unit - row * a.parts) * a.per, v1 = !here ? v0 : v0 + a.per < a.V ? v0 + a.per : a.V;
    const float inf = __builtin_inff();
    const auto load = [&](Frag* f, int64_t v) {
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t at = v + u * STEP + lane * E;
            if (at + E <= v1) f[u] = *gmem(reinterpret_cast<const Loose*>(z + at));
            else
#pragma unroll
                for (int e = 0; e < E; ++e) f[u][e] = at + e < v1 ? gmem(z)[at + e] : (T)-inf;
        }
    };
    Frag f[UN], next[UN];
    load(f, v0);
    const Powers to = make_powers(table_, threadIdx.x);
    __syncthreads();
    if (!here) return;
    const double low = kVeLow / c;
    double R = kVeNone, sum = 0.0;
    bool good = true;
    for (int64_t v = v0; v < v1; v += UN * STEP) {
        if (v + UN * STEP < v1) load(next, v + UN * STEP);
        float most = -inf;
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                most = fmaxf(most, (float)f[u][e]);
                good = good && (float)f[u][e] < inf;   // false for NaN
            }
        if (__ballot(most > -inf && ((double)most - R) * c > 64.0 * kVeTable)) {
            const double now = (double)wave_max(most);
            sum *= share(R, now, c, to);
            R = now;
        }
        double s[4] = {};
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {   // (what is clamped adds some 2^-1020)
                const double x = fmax((double)(float)f[u][e] - R, low), k = __builtin_fma(x, c, kVeShift);
                const Factors w = raised(k, __builtin_fma(x, c, kVeShift - k), to);
                s[(u * E + e) % 4] = __builtin_fma(w.scale, w.series, s[(u * E + e) % 4]);
            }
        sum += (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
        for (int u = 0; u < UN; ++u) f[u] = next[u];
    }
    sum = R == kVeNone ? 0.0 : sum64(sum);
    if (__ballot(!good)) sum = __builtin_nan("");
    if (lane == 0) {
        a.sums[unit] = sum;
        a.ref[unit] = R;
    }
}

// A row's whole sum against 2^ref, in every lane of the wave.
struct Sum {
    double ref, sum;
};
struct Parts {
    double sum[2], ref[2];
};
__device__ __forceinline__ Parts parts_of(const VerifyCall& a, int64_t row, int lane) {
    const double *s = a.sums + row * a.parts, *f = a.ref + row * a.parts;
    Parts p = {{0.0, 0.0}, {kVeNone, kVeNone}};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + i * kWave < a.parts) p.sum[i] = s[lane + i * kWave], p.ref[i] = f[lane + i * kWave];
    return p;
}
__device__ __forceinline__ Sum whole(Parts p, double c, const Powers& to) {
    // (references are logits, or kVeNone: their order is that of fp32)
    const float most = wave_max(fmaxf(p.ref[0] > kVeNone ? (float)p.ref[0] : -__FLT_MAX__, p.ref[1] > kVeNone ? (float)p.ref[1] : -__FLT_MAX__));
    const double R = (double)most;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 2; ++i) s += p.sum[i] * share(p.ref[i], R, c, to);
    return {R, sum64(s)};
}
__device__ __forceinline__ bool is_some(Sum s) { return s.sum > 0.0 && s.sum < __builtin_inf(); }   // false for NaN

// What a row's token is drawn from: w = p, less q or without the certain draft.
struct Weights {
    Sum p, q;
    double cp, cq, ip, iq;   // scales, and 1 / sums
    int64_t without;         // a token left out, or -1
    bool less;               // q is taken off

    // (each product rounded by itself: equal logits leave nothing)
    __device__ __forceinline__ double of(float zp, float zq, int64_t at, const Powers& to) const {
#pragma clang fp contract(off)
        double w = weight(zp, p.ref, cp, to) * ip;
        if (less) w = fmax(w - weight(zq, q.ref, cq, to) * iq, 0.0);
        return at == without ? 0.0 : w;
    }
};

// A thread's kVeRun logits from v; -inf from v1 on
template <bool BF16>
__device__ __forceinline__ void load_run(float* to, const typename Mm<BF16>::T* z, int64_t v, int64_t v1) {
    using M = Mm<BF16>;
    using Loose = typename M::T __attribute__((ext_vector_type(M::E), aligned(sizeof(typename M::T))));
#pragma unroll
    for (int u = 0; u < kVeRun; u += M::E) {
        if (v + u + M::E <= v1) {
            const typename M::Frag f = *gmem(reinterpret_cast<const Loose*>(z + v + u));
#pragma unroll
            for (int e = 0; e < M::E; ++e) to[u + e] = (float)f[e];
        } else
#pragma unroll
            for (int e = 0; e < M::E; ++e) to[u + e] = v + u + e < v1 ? (float)gmem(z)[v + u + e] : -__builtin_inff();
    }
}

// The weights of row b at the place `kept`, from the sums of its rows of logits.
__device__ __forceinline__ Weights weights_of(const VerifyCall& a, int64_t b, int kept, int n, Sum p, Sum q) {
    Weights w = {p, q, a.scale, a.draft_scale, 1.0 / p.sum, 0.0, -1, false};
    if (kept < n) {
        if (!a.draft) w.without = a.tokens[b * a.N + kept];
        else if (is_some(q)) w.less = true, w.iq = 1.0 / q.sum;
    }
    return w;
}

// The weights of one block of row b, a thread's own sum of them
template <bool BF16>
__device__ __forceinline__ double block_sum(const VerifyCall& a, const Weights& w, const typename Mm<BF16>::T* zp, const typename Mm<BF16>::T* zq,
                                            int64_t v0, int tid, const Powers& to) {
    const int64_t v1 = v0 + a.block < a.V ? v0 + a.block : a.V;
    double sum = 0.0;
    for (int64_t v = v0 + tid * kVeRun; v < v1; v += kVeBlock) {
        float p[kVeRun], q[kVeRun];
        load_run<BF16>(p, zp, v, v1);
        if (w.less) load_run<BF16>(q, zq, v, v1);
#pragma unroll
        for (int e = 0; e < kVeRun; ++e) sum += w.of(p[e], w.less ? q[e] : 0.f, v + e, to);
    }
    return sum;
}

// Every workgroup of a row finds how many drafts are kept (the first writes that, the tokens
// and their log probabilities) and adds up the weights of its blocks, which the token is drawn from.
template <bool BF16>
__global__ __launch_bounds__(kVeThreads) void k_verify_keep(VerifyCall a) {
    __shared__ Sum got[kVeMaxRows];
    __shared__ double part[2][kVeWaves], table_[kVeTable];
    __shared__ int kept_;
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave), rows = rows_of(a);
    const int64_t b = blockIdx.x / a.keepers;
    const int me = blockIdx.x % a.keepers, n = drafts_of(a, b);
    // everything that does not wait for the sums
    int64_t x = -1;
    float zp = 0.f, zq = 0.f, u = 0.f;
    bool known = false;
    if (wave == 0 && lane < n) {
        x = a.tokens[b * a.N + lane];
        u = a.u[b * a.N + lane];
        known = x >= 0 && x < a.V;
        if (known) {
            zp = get_io<BF16>(logits_of<BF16>(a, b, lane), x);
            if (a.draft) zq = get_io<BF16>(logits_of<BF16>(a, b, a.N + 1 + lane), x);
        }
    }
    const auto used = [&](int i) { return i < rows && (i <= a.N ? i <= n : i - a.N - 1 < n); };
    Parts next = {};
    if (used(wave)) next = parts_of(a, b * rows + wave, lane);
    const Powers to = make_powers(table_, tid);
    __syncthreads();
    for (int i = wave; i < rows; i += kVeWaves) {
        const Parts p = next;
        if (used(i + kVeWaves)) next = parts_of(a, b * rows + i + kVeWaves, lane);
        if (used(i)) {
            const Sum s = whole(p, i <= a.N ? a.scale : a.draft_scale, to);
            if (lane == 0) got[i] = s;
        }
    }
    __syncthreads();
    if (wave == 0) {
        bool keep = false;
        Sum p = {0.0, 0.0};
        if (known) p = got[lane];
        if (is_some(p)) {
            // u q < p, times both sums
            Sum s = {0.0, 1.0};
            double q = 1.0;
            if (a.draft) {
                s = got[a.N + 1 + lane];
                q = is_some(s) ? weight(zq, s.ref, a.draft_scale, to) : __builtin_nan("");
            }
            keep = (double)u * q * p.sum < weight(zp, p.ref, a.scale, to) * s.sum;
        }
        const int kept = __builtin_ctzll(~__ballot(keep));   // (lane 63 keeps none)
        if (lane == 0) kept_ = kept;
        if (me == 0 && lane <= a.N && lane != kept) {
            a.out[b * (a.N + 1) + lane] = lane < kept ? x : -1;
            if (a.logprob) {
                double lp = 0.0;
                if (lane < kept) lp = (((double)zp - p.ref) * (a.scale / kVeTable) - log2(p.sum)) * 0.69314718055994530942;
                a.logprob[b * (a.N + 1) + lane] = (float)lp;
            }
        }
        if (me == 0 && lane == 0) a.kept[b] = kept;
    }
    __syncthreads();
    const int kept = kept_;
    const Weights w = weights_of(a, b, kept, n, got[kept], a.draft && kept < n ? got[a.N + 1 + kept] : Sum{0.0, 0.0});
    const auto* const p = logits_of<BF16>(a, b, kept);
    const auto* const q = w.less ? logits_of<BF16>(a, b, a.N + 1 + kept) : p;
    for (int i = me, turn = 0; i < a.blocks; i += a.keepers, turn ^= 1) {
        const double sum = sum64(block_sum<BF16>(a, w, p, q, i * a.block, tid, to));
        if (lane == 0) part[turn][wave] = sum;
        __syncthreads();
        if (tid == 0) a.rest[b * a.blocks + i] = (part[turn][0] + part[turn][1]) + (part[turn][2] + part[turn][3]);
    }
}

// A workgroup finds a row's token: the block that r falls into, then the place in it.
template <bool BF16>
__global__ __launch_bounds__(kVeThreads) void k_verify_draw(VerifyCall a) {
    __shared__ Sum got[2];
    __shared__ double total[2][kVeWaves], before_, table_[kVeTable], again[kVeMaxBlocks];
    __shared__ int block_, last_[kVeWaves];
    __shared__ unsigned long long found;   // the largest: none yet
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave), rows = rows_of(a);
    const int64_t b = blockIdx.x;
    const double r = a.r[b];
    const int i0 = 2 * lane, i1 = i0 + 1;
    double x0 = i0 < a.blocks ? a.rest[b * a.blocks + i0] : 0.0, x1 = i1 < a.blocks ? a.rest[b * a.blocks + i1] : 0.0;
    const int n = drafts_of(a, b), kept = a.kept[b];
    const bool second = a.draft && kept < n;
    const Powers to = make_powers(table_, tid);
    if (tid == 0) found = ~0ull;
    Parts parts = {};
    if (wave == 0 || (wave == 1 && second)) parts = parts_of(a, b * rows + (wave ? a.N + 1 : 0) + kept, lane);
    __syncthreads();
    if (wave < 2) {
        const Sum s = wave == 0 || second ? whole(parts, wave ? a.draft_scale : a.scale, to) : Sum{0.0, 0.0};
        if (lane == 0) got[wave] = s;
    }
    __syncthreads();
    int64_t* const out = a.out + b * (a.N + 1) + kept;
    float* const lp = a.logprob ? a.logprob + b * (a.N + 1) + kept : nullptr;
    if (!is_some(got[0])) {   // no distribution
        if (tid == 0) {
            *out = -1;
            if (lp) *lp = __builtin_nanf("");
        }
        return;
    }
    Weights w = weights_of(a, b, kept, n, got[0], got[1]);
    const auto* const zp = logits_of<BF16>(a, b, kept);
    const auto* zq = w.less ? logits_of<BF16>(a, b, a.N + 1 + kept) : zp;
    double up = scan64(x0 + x1), all = lane64(up, kWave - 1);
    if (!(all > 0.0)) {   // nothing is left (the same in every wave): the target's own weights
        w.less = false, w.without = -1, zq = zp;
        for (int i = 0; i < a.blocks; ++i) {
            const double sum = sum64(block_sum<BF16>(a, w, zp, zq, i * a.block, tid, to));
            if (lane == 0) total[i % 2][wave] = sum;
            __syncthreads();
            if (tid == 0) again[i] = (total[i % 2][0] + total[i % 2][1]) + (total[i % 2][2] + total[i % 2][3]);
        }
        __syncthreads();
        x0 = i0 < a.blocks ? again[i0] : 0.0;
        x1 = i1 < a.blocks ? again[i1] : 0.0;
        up = scan64(x0 + x1);
        all = lane64(up, kWave - 1);
    }
    const double mark = r < 1.0 ? r * all : __builtin_inf();
    if (wave == 0) {
        const double low = up - (x0 + x1);
        const uint64_t hit0 = __ballot(x0 > 0.0 && low + x0 > mark), hit1 = __ballot(x1 > 0.0 && up > mark);
        const uint64_t some0 = __ballot(x0 > 0.0), some1 = __ballot(x1 > 0.0);
        int block;
        if (hit0 | hit1) {
            const int j = __builtin_ctzll(hit0 | hit1);
            block = 2 * j + !(hit0 >> j & 1);
        } else {
            const int j = 63 - __builtin_clzll(some0 | some1);
            block = 2 * j + (int)(some1 >> j & 1);
        }
        const double before = lane64(low, block / 2) + (block % 2 ? lane64(x0, block / 2) : 0.0);
        if (lane == 0) block_ = block, before_ = before;
    }
    __syncthreads();
    double before = before_;
    const int64_t v0 = block_ * a.block, v1 = v0 + a.block < a.V ? v0 + a.block : a.V;
    int last = -1;   // the thread's last place with a weight, from v0
    int turn = 0;
    for (int64_t v = v0; v < v1; v += kVeBlock, turn ^= 1) {
        float p[kVeRun], q[kVeRun];
        double x[kVeRun], sum = 0.0;
        const int64_t at = v + tid * kVeRun;
        load_run<BF16>(p, zp, at, v1);
        if (w.less) load_run<BF16>(q, zq, at, v1);
#pragma unroll
        for (int e = 0; e < kVeRun; ++e) {
            x[e] = w.of(p[e], w.less ? q[e] : 0.f, at + e, to);
            sum += x[e];
            if (x[e] > 0.0) last = (int)(at - v0) + e;
        }
        const double run = scan64(sum);
        if (lane == kWave - 1) total[turn][wave] = run;
        __syncthreads();
        double low = before + (run - sum);
        for (int i = 0; i < wave; ++i) low += total[turn][i];
        const bool hit = sum > 0.0 && low + sum > mark;
        const uint64_t hits = __ballot(hit);
        if (hit && lane == __builtin_ctzll(hits)) {
            int j = -1, most = 0;
#pragma unroll
            for (int e = 0; e < kVeRun; ++e) {
                low += x[e];
                if (x[e] > 0.0) {
                    if (j < 0 && low > mark) j = e;
                    most = e;
                }
            }
            if (j < 0) j = most;   // (the sums round differently one by one)
            atomicMin(&found, (unsigned long long)(at + j));
        }
        for (int i = 0; i < kVeWaves; ++i) before += total[turn][i];
        __syncthreads();
        if (found != ~0ull) break;
    }
    if (found == ~0ull) {   // r or the sums' rounding past the end: the block's last
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) last = max(last, __shfl_xor(last, d));
        if (lane == 0) last_[wave] = last;
        __syncthreads();
        last = max(max(last_[0], last_[1]), max(last_[2], last_[3]));
    }
    if (tid == 0) {
        const int64_t x = found != ~0ull ? (int64_t)found : v0 + last;
        *out = x;
        if (lp) *lp = (float)((((double)get_io<BF16>(zp, x) - w.p.ref) * (a.scale / kVeTable) - log2(w.p.sum)) * 0.69314718055994530942);
    }
}

namespace {

// Waves wanted of the sums' launch, so many that rows without drafts and their neighbours even out (us with
// 8192 / 16384 / 32768: 64 rows of up to 5 drafts x 100003 60 / 57 / 57, 96 of 8 x 32768 38 / 38 / 41).
constexpr int64_t kVeWanted = 16384;
constexpr int64_t kVeKeepers = 2048;   // workgroups wanted of the weights' (with 4096: 60, 38)

int64_t rows_in(const VerifyCall& c) { return c.B * (c.draft ? 2 * c.N + 1 : c.N + 1); }

}  // namespace

void plan_verify(VerifyCall& c) {
    const int64_t rows = rows_in(c), unit = kWave * 16, units = (c.V + unit - 1) / unit;   // of a wave's loads
    int64_t n = kVeWanted / rows;
    if (n > units) n = units;
    if (n > kVeMaxParts) n = kVeMaxParts;
    if (n < 1) n = 1;
    c.per = (units + n - 1) / n * unit;
    c.parts = (int)((c.V + c.per - 1) / c.per);
    const int64_t least = (c.V + kVeBlock - 1) / kVeBlock;
    c.block = (least + kVeMaxBlocks - 1) / kVeMaxBlocks * kVeBlock;
    c.blocks = (int)((c.V + c.block - 1) / c.block);
    const int64_t each = (c.blocks * c.B + kVeKeepers - 1) / kVeKeepers;   // blocks of a workgroup
    c.keepers = (int)(each < c.blocks ? (c.blocks + each - 1) / each : 1);
}

size_t verify_ws_used(const VerifyCall& c) { return 2 * (size_t)rows_in(c) * c.parts + (size_t)c.B * c.blocks; }

size_t verify_ws_doubles(int64_t B, int N, int64_t V) {
    // rows x parts is at most kVeWanted, or the rows where they are more
    VerifyCall c = {};
    c.B = B, c.N = N, c.V = V;
    plan_verify(c);
    const int64_t rows = B * (2 * N + 1);
    return 2 * (size_t)(rows > kVeWanted ? rows : kVeWanted) + (size_t)B * c.blocks;
}

hipError_t launch_verify(VerifyCall c, hipStream_t st) {
    plan_verify(c);
    const int64_t all = rows_in(c) * c.parts;
    c.ref = c.sums + all;
    c.rest = c.ref + all;
    const unsigned sums = (unsigned)((all + kVeWaves - 1) / kVeWaves), keep = (unsigned)(c.B * c.keepers), draw = (unsigned)c.B;
    const auto go = [&](auto bf) {
        constexpr bool BF16 = decltype(bf)::value;
        k_verify_sums<BF16><<<sums, kVeThreads, 0, st>>>(c);
        k_verify_keep<BF16><<<keep, kVeThreads, 0, st>>>(c);
        k_verify_draw<BF16><<<draw, kVeThreads, 0, st>>>(c);
    };
    if (c.io_bf16) go(std::true_type{});
    else go(std::false_type{});
    return hipGetLastError();
}

}  // namespace fi

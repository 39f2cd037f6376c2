// fi_verify.hip -- drafted tokens against the target's probabilities (fi_verify_*).
//
// Everything is held in 64 bits: which token a random number falls on depends
// on running sums of up to 2^31 probabilities, whose borders lie closer than
// fp32 tells apart.
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

constexpr int kVeThreads = 256, kVeWaves = kVeThreads / kWave;
constexpr int kVeRun = 8;                          // logits of a thread that follow one another
constexpr int kVeBlock = kVeThreads * kVeRun;      // a part is a multiple of these
constexpr int kVeMaxParts = 2 * kWave;
constexpr int kVeMaxDrafts = 63, kVeMaxRows = 2 * kVeMaxDrafts + 1;
constexpr double kVeLow = -1100.0;                 // 2^kVeLow = 0
constexpr double kVeNone = -1e300;                 // the reference of a part without a token

// 2^x, x <= 1000, to 2^-45 of itself: n = rint(x), the series of e^{(x - n) ln 2} to the 11th power.
__device__ __forceinline__ double exp2_64(double x) {
    x = fmax(x, kVeLow);
    const double n = rint(x), f = (x - n) * 0.69314718055994530942;
    double p = fma(f, 1.0 / 39916800.0, 1.0 / 3628800.0);
    p = fma(f, p, 1.0 / 362880.0);
    p = fma(f, p, 1.0 / 40320.0);
    p = fma(f, p, 1.0 / 5040.0);
    p = fma(f, p, 1.0 / 720.0);
    p = fma(f, p, 1.0 / 120.0);
    p = fma(f, p, 1.0 / 24.0);
    p = fma(f, p, 1.0 / 6.0);
    p = fma(f, p, 0.5);
    p = fma(f, p, 1.0);
    p = fma(f, p, 1.0);
    return ldexp(p, (int)n);
}
__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d);
    return v;
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

// A wave takes one part of one row of logits: the sum of 2^((z - R) c) with a reference R near the
// largest z (differences first: they are exact, however large the logits are).  A row
// that is no distribution has a sum that is NaN or 0.
template <bool BF16>
__global__ __launch_bounds__(kVeThreads) void k_verify_sums(VerifyCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    using Loose = T __attribute__((ext_vector_type(M::E), aligned(sizeof(T))));
    constexpr int E = M::E, UN = 16 / E, STEP = kWave * E;
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), rows = rows_of(a);
    const int64_t unit = (int64_t)blockIdx.x * kVeWaves + wave, row = unit / a.parts, b = row / rows;
    if (b >= a.B) return;
    const int i = (int)(row - b * rows), n = drafts_of(a, b);
    if (i <= a.N ? i > n : i - a.N - 1 >= n) return;   // no draft there
    const T* const z = logits_of<BF16>(a, b, i);
    const double c = i <= a.N ? a.scale : a.draft_scale;
    const int64_t v0 = (unit - row * a.parts) * a.per, v1 = v0 + a.per < a.V ? v0 + a.per : a.V;
    const float inf = __builtin_inff();
    double R = kVeNone, sum = 0.0;
    bool good = true;
    for (int64_t v = v0; v < v1; v += UN * STEP) {
        Frag f[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int64_t at = v + u * STEP + lane * E;
            if (at + E <= v1) f[u] = *gmem(reinterpret_cast<const Loose*>(z + at));
            else
#pragma unroll
                for (int e = 0; e < E; ++e) f[u][e] = at + e < v1 ? gmem(z)[at + e] : (T)-inf;
        }
        float most = -inf;
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) {
                most = fmaxf(most, (float)f[u][e]);
                good = good && (float)f[u][e] < inf;   // false for NaN
            }
        if (__ballot(most > -inf && ((double)most - R) * c > 64.0)) {
            const double to = (double)wave_max(most);
            sum *= exp2_64((R - to) * c);
            R = to;
        }
#pragma unroll
        for (int u = 0; u < UN; ++u)
#pragma unroll
            for (int e = 0; e < E; ++e) sum += exp2_64(((double)f[u][e] - R) * c);
    }
    sum = wave_sum64(sum);
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
__device__ __forceinline__ Sum whole(const VerifyCall& a, int64_t row, double c, int lane) {
    const double *s = a.sums + row * a.parts, *f = a.ref + row * a.parts;
    double sum[2] = {0.0, 0.0}, ref[2] = {kVeNone, kVeNone};
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (lane + i * kWave < a.parts) sum[i] = s[lane + i * kWave], ref[i] = f[lane + i * kWave];
    double R = fmax(ref[0], ref[1]);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) R = fmax(R, __shfl_xor(R, d));
    return {R, wave_sum64(sum[0] * exp2_64((ref[0] - R) * c) + sum[1] * exp2_64((ref[1] - R) * c))};
}
__device__ __forceinline__ bool is_some(Sum s) { return s.sum > 0.0 && s.sum < __builtin_inf(); }   // false for NaN

// What a row's token is drawn from: w = p, less q or without the certain draft.
struct Weights {
    Sum p, q;
    double cp, cq, ip, iq;   // scales, and 1 / sums
    int64_t without;         // a token left out, or -1
    bool less;               // q is taken off

    // (each product rounded by itself: equal logits leave nothing)
    __device__ __forceinline__ double of(float zp, float zq, int64_t at) const {
#pragma clang fp contract(off)
        double w = exp2_64(((double)zp - p.ref) * cp) * ip;
        if (less) w = fmax(w - exp2_64(((double)zq - q.ref) * cq) * iq, 0.0);
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

// Every workgroup of a row finds how many drafts are kept (the first writes that, the tokens
// and their log probabilities) and adds up its part of the weights that the token is drawn from.
template <bool BF16>
__global__ __launch_bounds__(kVeThreads) void k_verify_keep(VerifyCall a) {
    __shared__ Sum got[kVeMaxRows];
    __shared__ double part[kVeWaves];
    __shared__ int kept_;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, rows = rows_of(a);
    const int64_t b = blockIdx.x / a.parts;
    const int me = blockIdx.x % a.parts, n = drafts_of(a, b);
    for (int i = wave; i < rows; i += kVeWaves)
        if (i <= a.N ? i <= n : i - a.N - 1 < n) {
            const Sum s = whole(a, b * rows + i, i <= a.N ? a.scale : a.draft_scale, lane);
            if (lane == 0) got[i] = s;
        }
    __syncthreads();
    if (wave == 0) {
        bool keep = false;
        double lp = 0.0;
        if (lane < n) {
            const int64_t x = a.tokens[b * a.N + lane];
            const Sum p = got[lane];
            if (x >= 0 && x < a.V && is_some(p)) {
                const double t = ((double)get_io<BF16>(logits_of<BF16>(a, b, lane), x) - p.ref) * a.scale;
                double q = 1.0;
                if (a.draft) {
                    const Sum s = got[a.N + 1 + lane];
                    q = is_some(s) ? exp2_64(((double)get_io<BF16>(logits_of<BF16>(a, b, a.N + 1 + lane), x) - s.ref) * a.draft_scale) / s.sum
                                   : __builtin_nan("");
                }
                keep = (double)a.u[b * a.N + lane] * q < exp2_64(t) / p.sum;
                lp = (t - log2(p.sum)) * 0.69314718055994530942;
            }
        }
        const int kept = __builtin_ctzll(~__ballot(keep));   // (lane 63 keeps none)
        if (lane == 0) kept_ = kept;
        if (me == 0 && lane <= a.N && lane != kept) {
            a.out[b * (a.N + 1) + lane] = lane < kept ? a.tokens[b * a.N + lane] : -1;
            if (a.logprob) a.logprob[b * (a.N + 1) + lane] = lane < kept ? (float)lp : 0.f;
        }
        if (me == 0 && lane == 0) a.kept[b] = kept;
    }
    __syncthreads();
    const int kept = kept_;
    const Weights w = weights_of(a, b, kept, n, got[kept], a.draft && kept < n ? got[a.N + 1 + kept] : Sum{0.0, 0.0});
    const auto* const zp = logits_of<BF16>(a, b, kept);
    const auto* const zq = w.less ? logits_of<BF16>(a, b, a.N + 1 + kept) : zp;
    const int64_t v0 = me * a.per, v1 = v0 + a.per < a.V ? v0 + a.per : a.V;
    double sum = 0.0;
    for (int64_t v = v0 + tid * kVeRun; v < v1; v += kVeBlock) {
        float p[kVeRun], q[kVeRun];
        load_run<BF16>(p, zp, v, v1);
        if (w.less) load_run<BF16>(q, zq, v, v1);
#pragma unroll
        for (int e = 0; e < kVeRun; ++e) sum += w.of(p[e], w.less ? q[e] : 0.f, v + e);
    }
    sum = wave_sum64(sum);
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    if (tid == 0) a.rest[b * a.parts + me] = (part[0] + part[1]) + (part[2] + part[3]);
}

// Inclusive sums over the wave's lanes.
__device__ __forceinline__ double wave_scan64(double v, int lane) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const double x = __shfl_up(v, d);
        if (lane >= d) v += x;
    }
    return v;
}

// A workgroup finds a row's token: the part that r falls into, then the place in it.
template <bool BF16>
__global__ __launch_bounds__(kVeThreads) void k_verify_draw(VerifyCall a) {
    __shared__ Sum got[2];
    __shared__ double total[kVeWaves], whole_, before_;
    __shared__ int part_, last_[kVeWaves];
    __shared__ int64_t found;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, rows = rows_of(a);
    const int64_t b = blockIdx.x;
    const int n = drafts_of(a, b), kept = a.kept[b];
    const bool second = a.draft && kept < n;
    if (wave < 2) {
        Sum s = {0.0, 0.0};
        if (wave == 0 || second) s = whole(a, b * rows + (wave ? a.N + 1 : 0) + kept, wave ? a.draft_scale : a.scale, lane);
        if (lane == 0) got[wave] = s;
    }
    if (tid == 0) found = -1;
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
    const double r = a.r[b];
    if (wave == 0) {
        const int i0 = 2 * lane, i1 = i0 + 1;
        double x0 = i0 < a.parts ? a.rest[b * a.parts + i0] : 0.0, x1 = i1 < a.parts ? a.rest[b * a.parts + i1] : 0.0;
        double up = wave_scan64(x0 + x1, lane), all = __shfl(up, kWave - 1);
        if (!(all > 0.0)) {   // nothing is left: the target's own
            const Sum p = got[0];
            const int64_t at = (b * rows + kept) * a.parts;
            x0 = i0 < a.parts ? a.sums[at + i0] * exp2_64((a.ref[at + i0] - p.ref) * a.scale) / p.sum : 0.0;
            x1 = i1 < a.parts ? a.sums[at + i1] * exp2_64((a.ref[at + i1] - p.ref) * a.scale) / p.sum : 0.0;
            up = wave_scan64(x0 + x1, lane);
            all = -__shfl(up, kWave - 1);   // (the sign says so)
        }
        const double mark = r < 1.0 ? r * fabs(all) : __builtin_inf(), low = up - (x0 + x1);
        const uint64_t hit0 = __ballot(x0 > 0.0 && low + x0 > mark), hit1 = __ballot(x1 > 0.0 && up > mark);
        const uint64_t some0 = __ballot(x0 > 0.0), some1 = __ballot(x1 > 0.0);
        int part;
        if (hit0 | hit1) {
            const int j = __builtin_ctzll(hit0 | hit1);
            part = 2 * j + !(hit0 >> j & 1);
        } else {
            const int j = 63 - __builtin_clzll(some0 | some1);
            part = 2 * j + (int)(some1 >> j & 1);
        }
        const double before = __shfl(low, part / 2) + (part % 2 ? __shfl(x0, part / 2) : 0.0);
        if (lane == 0) part_ = part, whole_ = all, before_ = before;
    }
    __syncthreads();
    if (whole_ < 0.0) w.less = false, w.without = -1;
    const double mark = r < 1.0 ? r * fabs(whole_) : __builtin_inf();
    double before = before_;
    const auto* const zp = logits_of<BF16>(a, b, kept);
    const auto* const zq = w.less ? logits_of<BF16>(a, b, a.N + 1 + kept) : zp;
    const int64_t v0 = part_ * a.per, v1 = v0 + a.per < a.V ? v0 + a.per : a.V;
    int last = -1;   // the thread's last place with a weight, from v0
    for (int64_t v = v0; v < v1; v += kVeBlock) {
        float p[kVeRun], q[kVeRun];
        double x[kVeRun], sum = 0.0;
        const int64_t at = v + tid * kVeRun;
        load_run<BF16>(p, zp, at, v1);
        if (w.less) load_run<BF16>(q, zq, at, v1);
#pragma unroll
        for (int e = 0; e < kVeRun; ++e) {
            x[e] = w.of(p[e], w.less ? q[e] : 0.f, at + e);
            sum += x[e];
            if (x[e] > 0.0) last = (int)(at - v0) + e;
        }
        const double up = wave_scan64(sum, lane);
        if (lane == kWave - 1) total[wave] = up;
        __syncthreads();
        double low = before + (up - sum);
        for (int i = 0; i < wave; ++i) low += total[i];
        const bool hit = sum > 0.0 && low + sum > mark;
        const uint64_t hits = __ballot(hit);
        if (hit && lane == __builtin_ctzll(hits)) {
            int64_t j = -1, most = 0;
#pragma unroll
            for (int e = 0; e < kVeRun; ++e) {
                low += x[e];
                if (x[e] > 0.0) {
                    if (j < 0 && low > mark) j = e;
                    most = e;
                }
            }
            if (j < 0) j = most;   // (the sums round differently one by one)
            atomicMin(reinterpret_cast<unsigned long long*>(&found), (unsigned long long)(at + j));   // -1 is the largest
        }
        for (int i = 0; i < kVeWaves; ++i) before += total[i];
        __syncthreads();
        if (found >= 0) break;
    }
    if (found < 0) {   // r or the sums' rounding past the end: the part's last
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) last = max(last, __shfl_xor(last, d));
        if (lane == 0) last_[wave] = last;
        __syncthreads();
        last = max(max(last_[0], last_[1]), max(last_[2], last_[3]));
    }
    if (tid == 0) {
        const int64_t x = found >= 0 ? found : v0 + last;
        *out = x;
        if (lp) *lp = (float)((((double)get_io<BF16>(zp, x) - w.p.ref) * a.scale - log2(w.p.sum)) * 0.69314718055994530942);
    }
}

namespace {

constexpr int64_t kVeWanted = 4096;   // waves wanted of the sums' launch

}  // namespace

void plan_verify(VerifyCall& c) {
    const int64_t rows = c.B * (c.draft ? 2 * c.N + 1 : c.N + 1), blocks = (c.V + kVeBlock - 1) / kVeBlock;
    int64_t n = kVeWanted / rows;
    if (n > blocks) n = blocks;
    if (n > kVeMaxParts) n = kVeMaxParts;
    if (n < 1) n = 1;
    const int64_t each = (blocks + n - 1) / n;
    c.per = each * kVeBlock;
    c.parts = (int)((blocks + each - 1) / each);
}

size_t verify_ws_used(const VerifyCall& c) {
    const size_t rows = (size_t)c.B * (c.draft ? 2 * c.N + 1 : c.N + 1);
    return (2 * rows + (size_t)c.B) * c.parts;
}

size_t verify_ws_doubles(int64_t B, int N, int64_t, int) {
    // rows x parts is at most kVeWanted, or the rows where they are more; B is at most the rows
    const int64_t rows = B * (2 * N + 1);
    return 3 * (size_t)(rows > kVeWanted ? rows : kVeWanted);
}

hipError_t launch_verify(VerifyCall c, hipStream_t st) {
    plan_verify(c);
    const int64_t rows = c.B * (c.draft ? 2 * c.N + 1 : c.N + 1);
    c.ref = c.sums + rows * c.parts;
    c.rest = c.ref + rows * c.parts;
    const unsigned sums = (unsigned)((rows * c.parts + kVeWaves - 1) / kVeWaves), keep = (unsigned)(c.B * c.parts), draw = (unsigned)c.B;
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

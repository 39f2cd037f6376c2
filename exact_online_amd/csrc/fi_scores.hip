// fi_scores.hip -- log probability of a given token, entropy and the most
// probable tokens of every row of logits (fi_scores_*).
//
// One pass keeps, with a reference m near the largest logit, c = scale log2(e),
// R = m c rounded and t = z c - R (one fused operation, so that large logits
// lose nothing): s = sum 2^t and w = sum t 2^t.  Then, in units of log2,
// lse = R + log2 s and entropy = log2 s - w / s.
#include "fi_opdev.hpp"

namespace fi {

constexpr int kScThreads = 256, kScWaves = kScThreads / kWave;
constexpr int kScUnroll = 4;          // 16-byte loads of a lane in one batch
constexpr int kScBuffer = 96;         // candidates that a wave collects before it ranks them
constexpr int kScEnough = 32;         // ranked after a batch when there are so many
constexpr float kScLow = -16384.f;    // 2^kScLow = 0, and 0 kScLow = 0
constexpr float kScHigh = 16.f;       // t beyond this moves the reference
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

struct Stats {
    float m, s, w;
};

// The scale, and with log2 e: that is infinite for the largest scales, and then no
// reference is within bounds.
struct Scale {
    float s, c;
};
__device__ __forceinline__ Scale scale_of(const ScoresCall& a) { return {a.scale, a.scale * kLog2e}; }

// The scaled reference, rounded by itself everywhere (it is what the sums are
// taken against: m c inside a fused operation would be another number).
__device__ __forceinline__ float reference(float m, Scale k) {
#pragma clang fp contract(off)
    const float r = m * k.c;
    return r;
}
// From 2^24 on R is off m c by more than 1/2, and by more than exp2 can take from 2^31
// on: such logits are taken by differences, t = (z - m) scale log2 e, against m c itself.
__device__ __forceinline__ bool by_reference(float m, Scale k) { return fabsf(reference(m, k)) < 16777216.f; }   // false for NaN
__device__ __forceinline__ float by_difference(float z, float m, Scale k) { return (z - m) * k.s * kLog2e; }
__device__ __forceinline__ float scaled(float z, float m, Scale k) {
    return by_reference(m, k) ? fmaf(z, k.c, -reference(m, k)) : by_difference(z, m, k);
}
__device__ __forceinline__ float scaled_ref(float a, float m, Scale k) {   // of sums by a against those by m
#pragma clang fp contract(off)
    if (by_reference(a, k)) return by_reference(m, k) ? reference(a, k) - reference(m, k) : fmaf(-m, k.c, reference(a, k));
    return by_reference(m, k) ? fmaf(a, k.c, -reference(m, k)) : by_difference(a, m, k);
}

__device__ __forceinline__ Stats join(Stats a, Stats b, Scale k) {
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf(scaled_ref(a.m, m, k), kScLow), db = fmaxf(scaled_ref(b.m, m, k), kScLow);
    const float ea = exp2f(da), eb = exp2f(db);
    return {m, a.s * ea + b.s * eb, ea * (a.w + da * a.s) + eb * (b.w + db * b.s)};
}

// the same sums by another reference
__device__ __forceinline__ Stats moved_to(Stats a, float m, Scale k) {
    const float t = fmaxf(scaled_ref(a.m, m, k), kScLow), e = exp2f(t);
    return {m, a.s * e, e * (a.w + t * a.s)};
}

// sum + x, less what the additions before lost, which this one's loss replaces.
// (One after the other the terms of many equal logits all round the same way:
// 131072 of them in one row put lse off by 3e-5 and the entropy by 2e-4.)
__device__ __forceinline__ void add_to(float& sum, float& lost, float x) {
    const float y = x - lost, t = sum + y;
    lost = (t - sum) - y;
    sum = t;
}
__device__ __forceinline__ Stats join_wave(Stats x, Scale k) {
    x = moved_to(x, wave_max(x.m), k);
    return {x.m, wave_sum(x.s), wave_sum(x.w)};
}

// Alternatives as one number that orders them: the value's bits, then the
// index from the back.  0 is none.
using Key = unsigned long long;
__device__ __forceinline__ uint32_t ordered(float v) {
    const uint32_t u = __float_as_uint(v + 0.f);   // -0 ties with 0
    return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) { return __uint_as_float(o >> 31 ? o & 0x7FFFFFFFu : ~o); }
__device__ __forceinline__ Key key_of(float v, uint32_t id) { return (Key)ordered(v) << 32 | ~id; }

// A threshold that at least k of a wave's values reach and, where ties leave
// one, at most `most`: the more may, the fewer steps of bisection.
__device__ __forceinline__ uint32_t reached_by(uint32_t o, int k, int most) {
    uint32_t lo = 0, hi = 0xFFFFFFFFu;   // lo is reached by k of them, hi + 1 is not
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2 + 1;
        const int n = __popcll(__ballot(o >= mid));
        if (n >= k) {
            lo = mid;
            if (n <= most) break;
        } else hi = mid - 1;
    }
    return lo;
}

// The logit of a row's given token (lane 0; asked for early, as it takes two
// loads one after the other).
struct Target {
    int64_t id;
    float z;
};
template <bool BF16>
__device__ __forceinline__ Target target_of(const ScoresCall& a, int64_t r, int lane) {
    Target t = {-1, 0.f};
    if (lane == 0 && a.targets) {
        t.id = a.targets[r];
        if (t.id >= 0 && t.id < a.V) t.z = get_io<BF16>(a.logits, r * a.ld + t.id);
    }
    return t;
}

// Writes a row's results; lane j < k of the calling wave has alternative j.
__device__ __forceinline__ void scores_out(const ScoresCall& a, int64_t r, Stats x, Key alt, Target t, int lane) {
    const float inf = __builtin_inff(), nan = __builtin_nanf("");
    const bool empty = x.s == 0.f, bad = !(x.s < inf);
    const Scale c = scale_of(a);
    const float l2 = log2f(x.s);
    const auto log_p = [&](float z) {   // (a type's lowest value overflows in units of log2)
        const float t = scaled(z, x.m, c);
        return fabsf(t) < 1e30f ? (t - l2) * kLn2 : fmaf(z - x.m, a.scale, -l2 * kLn2);
    };
    if (lane < a.k) {
        float v = -inf;
        if (alt) v = log_p(value_of((uint32_t)(alt >> 32)));
        a.top[r * a.k + lane] = bad ? nan : v;
        a.top_id[r * a.k + lane] = bad || !alt ? -1 : (int64_t)(uint32_t)~alt;
    }
    if (lane) return;
    if (a.lse) a.lse[r] = bad ? nan : empty ? -inf : by_reference(x.m, c) ? (reference(x.m, c) + l2) * kLn2 : fmaf(x.m, a.scale, l2 * kLn2);
    if (a.entropy) a.entropy[r] = empty ? 0.f : bad ? nan : (l2 - x.w / x.s) * kLn2;
    if (a.logprob) {
        float lp;
        if (t.id < 0) lp = 0.f;
        else if (t.id >= a.V || bad) lp = nan;
        else if (empty) lp = -inf;
        else lp = log_p(t.z);
        a.logprob[r] = lp;
    }
}

// A wave's best k so far, sorted, and the candidates that came after them, in
// LDS (keys[0 .. 32) and keys[32 ..)).  A lane's 16 bytes with a logit that can
// still be among the k go into a queue first (the loop over the logits holds
// only that); the queue's logits are then looked at one a lane, and the
// candidates ranked by counting what is better: no order of arrival is
// needed, and nothing is moved one by one.
template <bool BF16>
struct Best {
    using Frag = typename Mm<BF16>::Frag;
    FI_SHARED Key* keys;
    FI_SHARED Frag* queue;
    FI_SHARED uint32_t* ids;   // of the queue's first logits
    int k, lane;
    int size, count, queued;   // sorted ones, candidates, queue
    Key floor;          // candidates exceed this
    float thr;          // logits of later tokens exceed this (the floor's value)

    __device__ __forceinline__ void rank() {
        if (!count) return;
        constexpr int RUN = 8;   // at once; runs are filled up with none
        if (lane < RUN) keys[kScoresMaxK + count + lane] = 0;
        if (lane >= size && lane < kScoresMaxK) keys[lane] = 0;
        wave_order();
        const Key a = lane < size ? keys[lane] : 0, b = lane < count ? keys[kScoresMaxK + lane] : 0,
                  c = lane + kWave < count ? keys[kScoresMaxK + kWave + lane] : 0;
        int pa = 0, pb = 0, pc = 0;
        const auto better = [&](int from, int to) {
            for (int j = from; j < to; j += RUN)
#pragma unroll
                for (int u = 0; u < RUN; ++u) {
                    const Key o = keys[j + u];
                    pa += o > a;
                    pb += o > b;
                    pc += o > c;
                }
        };
        better(0, size);
        better(kScoresMaxK, kScoresMaxK + count);
        wave_order();
        if (a && pa < k) keys[pa] = a;
        if (b && pb < k) keys[pb] = b;
        if (c && pc < k) keys[pc] = c;
        wave_order();
        size = size + count < k ? size + count : k;
        count = 0;
        if (size == k) {
            const Key last = keys[k - 1];
            const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(last >> 32)),
                           lo = __builtin_amdgcn_readfirstlane((uint32_t)last);
            const Key kth = (Key)hi << 32 | lo;
            if (kth > floor) {
                floor = kth;
                thr = value_of(hi);
            }
        }
    }
    // offers every lane's logit z of token id
    __device__ __forceinline__ void offer(float z, uint32_t id) {
        const Key me = key_of(z, id);
        const bool some = z > -__builtin_inff();   // false for NaN
        uint64_t m = __ballot(some && me > floor);
        if (!m) return;
        if (count + __popcll(m) > kScBuffer) {
            rank();
            m = __ballot(some && me > floor);
        }
        if (m >> lane & 1) keys[kScoresMaxK + count + __popcll(m & (((uint64_t)1 << lane) - 1))] = me;
        count += __popcll(m);
    }
    __device__ __forceinline__ void drain() {
        constexpr int E = Mm<BF16>::E;
        wave_order();
        for (int i = lane; __builtin_amdgcn_readfirstlane(i) < queued * E; i += kWave) {
            const bool some = i < queued * E;
            const FI_SHARED typename Mm<BF16>::T* z = (const FI_SHARED typename Mm<BF16>::T*)queue;
            offer(some ? (float)z[i] : -__builtin_inff(), some ? ids[i / E] + i % E : 0);
        }
        wave_order();
        queued = 0;
    }
    // a lane's logits f from token id, the largest of them z
    __device__ __forceinline__ void enqueue(const Frag& f, float z, uint32_t id) {
        uint64_t m = __ballot(z > thr);
        if (!m) return;
        if (queued + __popcll(m) > kWave) {
            drain();
            m = __ballot(z > thr);
        }
        if (m >> lane & 1) {
            const int at = queued + __popcll(m & (((uint64_t)1 << lane) - 1));
            queue[at] = f;
            ids[at] = id;
        }
        queued += __popcll(m);
    }
};

// A wave takes one part of one row (four of them make a workgroup, and meet
// nowhere); one part: the whole row, and the results go out at once.  A row's
// reductions then cost one wave's steps, once: with a workgroup to a row 4096 x
// 32768 took 76 us.
//
// Measured, bf16: 4096 x 32768, k = 5: 63.6 us (268 MB, 4.2 TB/s; a copy's 4.9 would take
// 55), the vector units 65% busy with an exponential, two fused operations and
// a maximum for each logit; 333 x 100003, nine in ten masked, k = 8: 31.8 us (67 MB), 27 in
// this kernel, where some ten batches a wave do not hide its beginning
// (threshold, first ranking) and end.  fp32, one row of 131072, k = 20: 6.3 us here,
// 4.5 in the join: two launches and their trips to memory.
template <bool BF16>
__global__ __launch_bounds__(kScThreads) void k_scores(ScoresCall a) {
    using M = Mm<BF16>;
    using T = typename M::T;
    using Frag = typename M::Frag;
    constexpr int E = M::E, STEP = kWave * E, BATCH = kScUnroll * STEP;
    __shared__ __align__(16) Key wk[kScWaves][kScoresMaxK + kScBuffer + 8];   // (8: the end of a run)
    __shared__ __align__(16) Frag wq[kScWaves][kWave];
    __shared__ uint32_t wi[kScWaves][kWave];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), k = a.k;
    const Scale c = scale_of(a);
    const float inf = __builtin_inff();
    const int64_t unit = (int64_t)blockIdx.x * kScWaves + wave, r = unit / a.parts;
    if (r >= a.rows) return;
    const int part = (int)(unit - r * a.parts);
    const T* row = static_cast<const T*>(a.logits) + r * a.ld;
    const int64_t v0 = (int64_t)part * a.per, v1 = v0 + a.per < a.V ? v0 + a.per : a.V;

    Stats x = {-__FLT_MAX__, 0.f, 0.f}, lost = x;   // m is the wave's, s and w the lane's; in the additions to them
    Best<BF16> best = {smem_ptr(wk[wave]), smem_ptr(wq[wave]), smem_ptr(wi[wave]), k, lane, 0, 0, 0, 0, -inf};
    const auto load = [&](Frag* f, int64_t v) {
#pragma unroll
        for (int u = 0; u < kScUnroll; ++u) {
            const int64_t at = v + u * STEP + lane * E;
            using Loose = T __attribute__((ext_vector_type(E), aligned(sizeof(T))));
            if (at + E <= v1) f[u] = *gmem(reinterpret_cast<const Loose*>(row + at));
            else
#pragma unroll
                for (int e = 0; e < E; ++e) f[u][e] = at + e < v1 ? gmem(row)[at + e] : (T)-inf;
        }
    };
    Frag now[kScUnroll], next[kScUnroll];
    load(now, v0);
    for (int64_t v = v0; v < v1; v += BATCH) {
        if (v + BATCH < v1) load(next, v + BATCH);
        float big[kScUnroll], most = -inf;
#pragma unroll
        for (int u = 0; u < kScUnroll; ++u) {
            big[u] = (float)now[u][0];
#pragma unroll
            for (int e = 1; e < E; ++e) big[u] = fmaxf(big[u], (float)now[u][e]);
            most = fmaxf(most, big[u]);
        }
        if (v == v0 || __ballot(scaled(most, x.m, c) > kScHigh)) {
            const float m = fmaxf(wave_max(most), x.m);
            x = moved_to(x, m, c);
            lost = moved_to(lost, m, c);
        }
        float s[kScUnroll] = {}, w[kScUnroll] = {};   // the batch's sums
        const auto sums = [&](auto t_of) {
#pragma unroll
            for (int u = 0; u < kScUnroll; ++u)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float t = t_of((float)now[u][e]), p = __builtin_amdgcn_exp2f(t);
                    s[u] += p;
                    w[u] = fmaf(p, fmaxf(t, kScLow), w[u]);   // -inf: 0 (-2^14)
                }
        };
        if (by_reference(x.m, c)) {
            const float ref = reference(x.m, c);
            sums([&](float z) { return fmaf(z, c.c, -ref); });
        } else sums([&](float z) { return by_difference(z, x.m, c); });
        add_to(x.s, lost.s, (s[0] + s[1]) + (s[2] + s[3]));
        add_to(x.w, lost.w, (w[0] + w[1]) + (w[2] + w[3]));
        if (k) {
            if (v == v0) {
                // of the first batch, only what reaches the k-th largest lane or so (95 rows
                // of 54733, k = 32: 19.0 us; up to 3/2 k + 8 lanes 22.8, k exactly 20.1)
                const uint32_t o = reached_by(ordered(most), k, k + k / 8 + 2);
                const float f = value_of(o - (o == 0x80000000u ? 2 : 1));   // the next value below; -0 is 0
                if (o && f > -inf) {                                        // false for NaN bits too
                    best.thr = f;
                    best.floor = ((Key)o << 32) - 1;
                }
            }
#pragma unroll
            for (int u = 0; u < kScUnroll; ++u) best.enqueue(now[u], big[u], (uint32_t)(v + u * STEP + lane * E));
            if (best.queued) {
                best.drain();
                if (v == v0 || best.count >= kScEnough) best.rank();
            }
        }
#pragma unroll
        for (int u = 0; u < kScUnroll; ++u) now[u] = next[u];
    }
    best.rank();
    x.s = wave_sum(x.s - lost.s);
    x.w = wave_sum(x.w - lost.w);
    const Key alt = lane < best.size ? wk[wave][lane] : 0;
    if (a.parts == 1) scores_out(a, r, x, alt, target_of<BF16>(a, r, lane), lane);
    else {
        if (lane == 0) {
            a.pst[unit * 3] = x.m;
            a.pst[unit * 3 + 1] = x.s;
            a.pst[unit * 3 + 2] = x.w;
        }
        if (lane < k) a.pkey[unit * k + lane] = alt;
    }
}

// Joins a row's parts (at most two for each lane of a wave): 4.6 us, a launch
// and its trips to memory; all keys are asked for before the bound on them is
// known.
constexpr int kScMaxParts = 2 * kWave;

template <bool BF16>
__global__ __launch_bounds__(kScThreads) void k_scores_join(ScoresCall a) {
    constexpr int MINE = kScMaxParts * kScoresMaxK / kScThreads, RUN = 8;
    __shared__ __align__(16) Key got[kScMaxParts * kScoresMaxK + RUN];
    __shared__ Key out[kScoresMaxK];
    __shared__ uint32_t least;
    __shared__ int count;
    __shared__ Target given;
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, k = a.k, all = a.parts * k;
    const int64_t r = blockIdx.x;
    const Scale c = scale_of(a);
    const Key* const keys = a.pkey + r * all;
    // one wave joins the sums and writes the results, another bounds the
    // alternatives, a third gets the given token's logit
    Key mine[MINE];
#pragma unroll
    for (int i = 0; i < MINE; ++i)
        if (i * kScThreads < all) mine[i] = i * kScThreads + tid < all ? keys[i * kScThreads + tid] : 0;
    Stats x = {-__FLT_MAX__, 0.f, 0.f};
    if (wave == 0) {
        for (int p = lane; p < a.parts; p += kWave) {
            const float* q = a.pst + (r * a.parts + p) * 3;
            x = join(x, {q[0], q[1], q[2]}, c);
        }
        x = join_wave(x, c);
    } else if (wave == 1) {
        // With the parts' j-th best keys, j = ceil(k / parts), the ceil(k / j)-th of
        // them bounds what can be among the row's k: that many parts have j keys
        // as large (95 rows of 54733, k = 32: 23 us; 37 where half as many more might reach it).
        if (lane < kScoresMaxK) out[lane] = 0;
        if (lane == 0) count = 0;
        if (k) {
            uint32_t head = 0;
            const int j = (k + a.parts - 1) / a.parts;
            for (int p = lane; p < a.parts; p += kWave) {
                const uint32_t h = (uint32_t)(keys[p * k + j - 1] >> 32);
                head = head > h ? head : h;
            }
            const int m = (k + j - 1) / j;
            const uint32_t o = reached_by(head, m, m);
            if (lane == 0) least = o;
        }
    } else if (wave == 2) {
        const Target t = target_of<BF16>(a, r, lane);
        if (lane == 0) given = t;
    }
    __syncthreads();
    if (k) {
#pragma unroll
        for (int i = 0; i < MINE; ++i)
            if (i * kScThreads < all && mine[i] && (uint32_t)(mine[i] >> 32) >= least)
                got[atomicAdd(&count, 1)] = mine[i];   // any order: they are ranked
        __syncthreads();
        const int n = count;
        if (tid < RUN) got[n + tid] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kScThreads) {
            const Key me = got[i];
            int place = 0;
            for (int j = 0; j < n; j += RUN)
#pragma unroll
                for (int u = 0; u < RUN; ++u) place += got[j + u] > me;
            if (place < k) out[place] = me;
        }
        __syncthreads();
    }
    if (wave == 0) scores_out(a, r, x, lane < k ? out[lane] : 0, given, lane);
}

namespace {

// Waves wanted of a launch: two for each SIMD, at most (whole parts of a row: 1025 rows and
// more are one each).  us with 4096 / 2048 / 1024, bf16: 1099
// rows of 9067, k = 5: 18.1 / 17.0 / 16.5; 333 of 100003: 28.8 / 30.9 / 38.3, and with
// k = 32 54.6 / 46.9 / 52.6; 95 of 54733, k = 0: 10.0 / 9.0 / 8.5.
constexpr int kScPartsWanted = 2048;

// Parts that a row of V logits is split into in a call of `rows`: each at
// least a batch of loads of one wave.
int parts_of(int64_t rows, int64_t V, int io_bf16, int64_t* per) {
    const int64_t unit = (int64_t)kWave * (io_bf16 ? 8 : 4);   // logits of one load of a wave
    int64_t n = kScPartsWanted / rows;
    if (n > V / (unit * kScUnroll)) n = V / (unit * kScUnroll);
    if (n > kScMaxParts) n = kScMaxParts;
    if (n < 1) n = 1;
    *per = ((V + n - 1) / n + unit - 1) / unit * unit;
    return (int)((V + *per - 1) / *per);
}

}  // namespace

size_t scores_ws_parts(int64_t rows, int64_t V, int io_bf16) {
    int64_t most = 0, per;
    for (int64_t r = 1; r <= rows && r <= kScPartsWanted / 2; ++r) {
        const int n = parts_of(r, V, io_bf16, &per);
        if (n > 1 && r * n > most) most = r * n;
    }
    return (size_t)most;
}

void plan_scores(ScoresCall& c) { c.parts = parts_of(c.rows, c.V, c.io_bf16, &c.per); }

size_t scores_ws_used(const ScoresCall& c) { return c.parts > 1 ? (size_t)c.rows * c.parts : 0; }

hipError_t launch_scores(ScoresCall c, hipStream_t st) {
    plan_scores(c);
    const ScoresCall all = c;
    constexpr int64_t kRows = (int64_t)1 << 23;   // of one launch, which has at most 2^32 threads
    for (int64_t r = 0; r < all.rows; r += kRows) {
        c.rows = all.rows - r < kRows ? all.rows - r : kRows;
        c.logits = static_cast<const char*>(all.logits) + r * c.ld * (c.io_bf16 ? 2 : 4);
        const auto from = [&](auto* p, int64_t n) { return p ? p + n : p; };
        c.targets = from(all.targets, r);
        c.logprob = from(all.logprob, r);
        c.entropy = from(all.entropy, r);
        c.lse = from(all.lse, r);
        c.top = from(all.top, r * c.k);
        c.top_id = from(all.top_id, r * c.k);
        const unsigned grid = (unsigned)((c.rows * c.parts + kScWaves - 1) / kScWaves);   // several parts only for few rows
        if (c.io_bf16) k_scores<true><<<grid, kScThreads, 0, st>>>(c);
        else k_scores<false><<<grid, kScThreads, 0, st>>>(c);
        if (c.parts > 1) {
            if (c.io_bf16) k_scores_join<true><<<(unsigned)c.rows, kScThreads, 0, st>>>(c);
            else k_scores_join<false><<<(unsigned)c.rows, kScThreads, 0, st>>>(c);
        }
    }
    return hipGetLastError();
}

}  // namespace fi

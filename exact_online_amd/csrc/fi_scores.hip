// fi_scores.hip -- log probability of a given token, entropy and the most
// probable tokens of every row of logits (fi_scores_*).
//
// One pass keeps, with m the largest logit so far and t = (z - m) c, c =
// scale log2(e): s = sum 2^t and w = sum t 2^t.  Then, in units of log2,
// lse = c m + log2 s and entropy = log2 s - w / s.
#include "fi_opdev.hpp"

namespace fi {

constexpr int kScThreads = 256;
constexpr float kScLow = -16384.f;    // 2^kScLow = 0, and 0 kScLow = 0
constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;

struct Stats {
    float m, s, w;
};

__device__ __forceinline__ Stats join(Stats a, Stats b, float c) {
    const float m = fmaxf(a.m, b.m);
    const float da = fmaxf((a.m - m) * c, kScLow), db = fmaxf((b.m - m) * c, kScLow);
    const float ea = exp2f(da), eb = exp2f(db);
    return {m, a.s * ea + b.s * eb, ea * (a.w + da * a.s) + eb * (b.w + db * b.s)};
}

template <bool BF16>
__global__ __launch_bounds__(kScThreads) void k_scores(ScoresCall a) {
    __shared__ Stats st[kScThreads];
    __shared__ float tv[kScThreads];
    __shared__ int64_t ti[kScThreads];
    const int tid = threadIdx.x;
    const float c = a.scale * kLog2e;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        Stats x = {-__FLT_MAX__, 0.f, 0.f};
        for (int64_t j = tid; j < a.V; j += kScThreads) {
            const float z = get_io<BF16>(a.logits, r * a.ld + j);
            if (z > x.m) {
                x = join(x, {z, 0.f, 0.f}, c);
            }
            const float t = (z - x.m) * c, e = exp2f(t);
            x.s += e;
            x.w = fmaf(e, fmaxf(t, kScLow), x.w);
        }
        st[tid] = x;
        __syncthreads();
        for (int d = kScThreads / 2; d > 0; d >>= 1) {
            if (tid < d) st[tid] = join(st[tid], st[tid + d], c);
            __syncthreads();
        }
        x = st[0];
        const bool empty = x.s == 0.f, bad = !(x.s < __builtin_inff());
        const float l2 = log2f(x.s);
        const float lse = empty ? -__builtin_inff() : fmaf(x.m, a.scale, l2 * kLn2);
        if (tid == 0) {
            if (a.lse) a.lse[r] = bad ? __builtin_nanf("") : lse;
            if (a.entropy) a.entropy[r] = empty ? 0.f : bad ? __builtin_nanf("") : (l2 - x.w / x.s) * kLn2;
            if (a.logprob) {
                const int64_t t = a.targets[r];
                float lp;
                if (t < 0) lp = 0.f;
                else if (t >= a.V || bad) lp = __builtin_nanf("");
                else if (empty) lp = -__builtin_inff();
                else lp = fmaf(get_io<BF16>(a.logits, r * a.ld + t) - x.m, a.scale, -l2 * kLn2);
                a.logprob[r] = lp;
            }
        }
        float pv = __builtin_inff();
        int64_t pi = -1;
        for (int k = 0; k < a.k; ++k) {
            // the best of what comes after (pv, pi)
            float bv = -__builtin_inff();
            int64_t bi = -1;
            for (int64_t j = tid; j < a.V; j += kScThreads) {
                const float z = get_io<BF16>(a.logits, r * a.ld + j);
                if ((z < pv || (z == pv && j > pi)) && z > bv) bv = z, bi = j;
            }
            tv[tid] = bv;
            ti[tid] = bi;
            __syncthreads();
            for (int d = kScThreads / 2; d > 0; d >>= 1) {
                if (tid < d) {
                    const float v = tv[tid + d];
                    const int64_t i = ti[tid + d];
                    if (i >= 0 && (ti[tid] < 0 || v > tv[tid] || (v == tv[tid] && i < ti[tid]))) tv[tid] = v, ti[tid] = i;
                }
                __syncthreads();
            }
            pv = tv[0];
            pi = ti[0];
            if (tid == 0) {
                a.top[r * a.k + k] = bad ? __builtin_nanf("") : pi < 0 ? -__builtin_inff() : fmaf(pv - x.m, a.scale, -l2 * kLn2);
                a.top_id[r * a.k + k] = bad ? -1 : pi;
            }
            __syncthreads();
            if (pi < 0) pv = -__builtin_inff();
        }
    }
}

hipError_t launch_scores(const ScoresCall& c, hipStream_t st) {
    const unsigned grid = (unsigned)(c.rows < (1 << 22) ? c.rows : 1 << 22);
    if (c.io_bf16) k_scores<true><<<grid, kScThreads, 0, st>>>(c);
    else k_scores<false><<<grid, kScThreads, 0, st>>>(c);
    return hipGetLastError();
}

}  // namespace fi

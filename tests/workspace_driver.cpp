// Sizes of handles and of calls on them: no call may use more of its handle's
// workspace than the create call allocates (most for all calls that
// the handle takes, of which the longest are not those that use most).
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <random>

#include "fi_operators.h"

using namespace fi;

static std::mt19937_64 rng(7);
static int64_t from(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }
static int64_t spread(int64_t lo, int64_t hi) {   // over the logarithm
    return std::min(hi, (int64_t)std::exp(std::log((double)lo) + (rng() >> 11) * 0x1p-53 * std::log((hi + 1.0) / lo)));
}
static int64_t within(int64_t most) { return from(0, 3) ? spread(1, most) : std::max<int64_t>(1, most - from(0, 3)); }

int main(int argc, char **) {
    const int handles = argc > 1 ? 100 : 6000, calls = 60;
    long split[3] = {};
    for (int h = 0; h < handles; ++h) {
        {
            const int64_t B = spread(1, 600), L = spread(1, 1 << 20), Hkv = spread(1, 64), G = spread(1, 40);
            const int dk = (int)from(1, 256), dv = (int)from(1, 256), bf = (int)from(0, 1);
            const size_t have = lattn_ws_bytes(B, L, (int)(Hkv * G), (int)Hkv, dk, dv, bf);
            for (int i = 0; i < calls; ++i) {
                LattnCall c = {};
                c.B = within(B), c.L = (int)within(L), c.H = (int)(Hkv * G), c.Hkv = (int)Hkv, c.G = (int)G;
                c.dk = dk, c.dv = dv, c.io_bf16 = bf, c.fresh = (int)from(0, 1);
                plan_lattn(c);
                split[0] += lattn_ws_used(c) > 0;
                if (lattn_ws_used(c) > have) {
                    std::printf("lattn: %lld x %lld, %d heads on %d of %d x %d, bf16 %d: %zu of %zu bytes (handle %lld x %lld)\n",
                                (long long)c.B, (long long)c.L, c.H, c.Hkv, dk, dv, bf, lattn_ws_used(c), have, (long long)B, (long long)L);
                    return 1;
                }
            }
        }
        {
            const int64_t M = spread(1, 1 << 20), N = spread(1, 40000), K = spread(1, 200000);
            const int bf = (int)from(0, 1);
            const size_t have = dense_ws_bytes(M, N, K, bf);
            for (int i = 0; i < calls; ++i) {
                DenseCall c = {};
                c.M = within(M), c.N = N, c.K = K, c.io_bf16 = bf;
                plan_dense(c);
                split[1] += dense_ws_used(c) > 0;
                const bool whole = (c.splits - 1) * c.k_split < K && c.splits * c.k_split >= K;   // no part is empty
                if (dense_ws_used(c) > have || !whole) {
                    std::printf("dense: %lld x %lld x %lld, bf16 %d: %zu of %zu bytes, %d parts of %lld (handle %lld)\n", (long long)c.M,
                                (long long)N, (long long)K, bf, dense_ws_used(c), have, c.splits, (long long)c.k_split, (long long)M);
                    return 1;
                }
            }
        }
        {
            const int64_t R = spread(1, 1 << 16), V = spread(1, 1 << 24);
            const int bf = (int)from(0, 1);
            const size_t have = scores_ws_parts(R, V, bf);
            for (int i = 0; i < calls; ++i) {
                ScoresCall c = {};
                c.rows = within(R), c.V = V, c.io_bf16 = bf;
                plan_scores(c);
                split[2] += scores_ws_used(c) > 0;
                if (scores_ws_used(c) > have || (c.parts - 1) * c.per >= V || c.parts * c.per < V) {
                    std::printf("scores: %lld x %lld, bf16 %d: %zu of %zu parts, %d of %lld (handle %lld)\n", (long long)c.rows, (long long)V,
                                bf, scores_ws_used(c), have, c.parts, (long long)c.per, (long long)R);
                    return 1;
                }
            }
        }
    }
    std::printf("ok: %d handles of each kind; calls with workspace %ld, %ld, %ld\n", handles, split[0], split[1], split[2]);
    return 0;
}

// Sizes of handles and of smaller calls on them, of the delta rule and the check of
// drafts: no call may use more of its handle's workspace than the create call allocates, and the plans
// cover what they split.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <random>

#include "fi_operators.h"

using namespace fi;

static std::mt19937_64 rng(11);
static int64_t from(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }
static int64_t spread(int64_t lo, int64_t hi) {   // over the logarithm
    return std::min(hi, (int64_t)std::exp(std::log((double)lo) + (rng() >> 11) * 0x1p-53 * std::log((hi + 1.0) / lo)));
}
static int64_t within(int64_t most) { return from(0, 3) ? spread(1, most) : std::max<int64_t>(1, most - from(0, 3)); }

int main() {
    long split[3] = {}, runs = 0;
    for (int h = 0; h < 6000; ++h) {
        {
            const int64_t B = spread(1, 3000), L = spread(1, 1 << 20), Hk = spread(1, 64), G = spread(1, 5);
            const int dk = (int)from(1, 256), dv = (int)from(1, 256), bf = (int)from(0, 1), Hv = (int)(Hk * G);
            const size_t have = delta_ws_bytes(B, L, Hv, dk, dv, bf);
            for (int i = 0; i < 60; ++i) {
                DeltaCall c = {};
                c.B = within(B), c.L = (int)within(L), c.Hk = (int)Hk, c.Hv = Hv, c.G = (int)G, c.dk = dk, c.dv = dv, c.io_bf16 = bf;
                if (delta_route(c) != DeltaRoute::chunks) {
                    if (delta_ws_used(c) != 0) return 1;
                    continue;
                }
                plan_delta(c);
                const int64_t C = bf ? 64 : 32, all = (c.L + C - 1) / C;
                split[0] += c.nseg > 1;
                runs += c.chunks < all;
                const bool whole = c.chunks >= 1 && c.chunks <= all && (int64_t)(c.nseg - 1) * c.seg_chunks < c.chunks &&
                                   (int64_t)c.nseg * c.seg_chunks >= c.chunks;   // no segment of the longest row is empty
                if (delta_ws_used(c) > have || !whole) {
                    std::printf("delta: %lld x %d, %d heads of %d x %d, bf16 %d: %zu of %zu bytes, %d chunks in %d of %d (handle %lld x %lld)\n",
                                (long long)c.B, c.L, Hv, dk, dv, bf, delta_ws_used(c), have, c.chunks, c.nseg, c.seg_chunks, (long long)B, (long long)L);
                    return 1;
                }
            }
        }
        {
            const int N = (int)from(0, 63);
            const int64_t B = spread(1, kVerifyMaxRows / (2 * N + 1)), V = spread(1, ((int64_t)1 << 31) - 1);
            const size_t have = verify_ws_doubles(B, N, V);
            for (int i = 0; i < 60; ++i) {
                VerifyCall c = {};
                c.B = within(B), c.N = (int)from(0, N), c.V = V;
                c.draft = from(0, 1) ? &c : nullptr;
                plan_verify(c);
                split[1] += c.parts > 1;
                split[2] += c.blocks > 1;
                const bool whole = (int64_t)(c.parts - 1) * c.per < V && c.parts * c.per >= V && (int64_t)(c.blocks - 1) * c.block < V &&
                                   c.blocks * c.block >= V && c.parts <= 128 && c.blocks <= 128 && c.keepers >= 1 && c.keepers <= c.blocks;
                if (verify_ws_used(c) > have || !whole) {
                    std::printf("verify: %lld x %d x %lld: %zu of %zu doubles, %d parts of %lld, %d blocks of %lld (handle %lld x %d)\n",
                                (long long)c.B, c.N, (long long)V, verify_ws_used(c), have, c.parts, (long long)c.per, c.blocks,
                                (long long)c.block, (long long)B, N);
                    return 1;
                }
            }
        }
    }
    std::printf("ok: segments %ld, runs of chunks %ld, parts %ld, blocks %ld\n", split[0], runs, split[1], split[2]);
    return split[0] && runs && split[1] && split[2] ? 0 : 1;
}

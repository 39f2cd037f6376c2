// The parts of the delta rule's workspace for calls of random sizes, odd head sizes most of all: every part lies
// behind the one before, within what the call uses, and what is read in 16-byte units begins at one.
// With three numbers as arguments: handles of random sizes take no more than the header says of fi_delta_create: MB for
// systems, KB for each row and head in their place, MB for segments.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "fi_operators.h"

using namespace fi;

static std::mt19937_64 rng(23);
static int64_t from(int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); }
static int64_t spread(int64_t lo, int64_t hi) {   // over the logarithm
    return std::min(hi, (int64_t)std::exp(std::log((double)lo) + (rng() >> 11) * 0x1p-53 * std::log((hi + 1.0) / lo)));
}

static int bounds(double systems, double each, double segments) {
    double most[2] = {};
    for (int i = 0; i < 2000000; ++i) {
        const int64_t Hv = spread(1, 4096), B = spread(1, kLattnMaxRows / Hv), L = spread(1, (int64_t)1 << 25);
        const int wide = (int)from(0, 3), dk = wide ? (int)from(1, 256) : 256, dv = wide > 1 ? (int)from(1, 256) : 128 << from(0, 1), bf = (int)from(0, 1);
        const double rows = (double)B * Hv, chunks = (double)((L + (bf ? 63 : 31)) / (bf ? 64 : 32)), have = (double)delta_ws_bytes(B, L, (int)Hv, dk, dv, bf);
        const double bound = std::max(systems * 1e6, each * 1e3 * rows) + segments * 1e6 + (rows * chunks > 32768 ? 4.0 * dk * dv * rows : 0.0);
        most[rows > 8192] = std::max(most[rows > 8192], have / bound);
        if (have > bound) {
            std::printf("delta: %lld x %lld, %lld heads of %d x %d, bf16 %d: %.0f bytes, %.0f at most\n", (long long)B, (long long)L, (long long)Hv, dk, dv, bf,
                        have, bound);
            return 1;
        }
    }
    std::printf("ok: at most %.3f and %.3f of the bound\n", most[0], most[1]);
    return most[0] > 0.9 && most[1] > 0.9 ? 0 : 1;   // nor does the header say much more than they take
}

int main(int argc, char** argv) {
    if (argc == 4) return bounds(std::atof(argv[1]), std::atof(argv[2]), std::atof(argv[3]));
    alignas(256) static float base[64];
    long split = 0, carried = 0, odd = 0;
    for (int i = 0; i < 300000; ++i) {
        DeltaCall c = {};
        c.B = spread(1, 1000), c.L = (int)spread(1, 1 << 20), c.Hk = (int)spread(1, 64), c.G = (int)spread(1, 5), c.Hv = c.Hk * c.G;
        c.dk = (int)from(1, 256), c.dv = (int)from(1, 256), c.io_bf16 = (int)from(0, 1);
        if (delta_route(c) != DeltaRoute::chunks) continue;
        plan_delta(c);
        place_delta(c, base);
        const int64_t tasks = c.B * c.Hv, wide = c.dk <= 64 ? 64 : c.dk <= 128 ? 128 : 256, states = (int64_t)c.dk * c.dv;
        const bool segs = c.nseg > 1, carry = (c.L + (c.io_bf16 ? 63 : 31)) / (c.io_bf16 ? 64 : 32) > c.chunks;
        const auto at = [&](const float* p) { return (int64_t)(((uintptr_t)p - (uintptr_t)base) / sizeof(float)); };
        split += segs, carried += carry, odd += segs && tasks * c.nseg * states % 4 != 0;
        bool ok = c.tri == base && (uintptr_t)c.tri % 16 == 0 && at(c.ent) >= tasks * c.chunks && (c.carry != nullptr) == carry;
        int64_t end = at(c.ent);
        if (segs) {
            ok = ok && at(c.move) >= at(c.ent) + tasks * c.nseg * states && (uintptr_t)c.move % 16 == 0;
            end = at(c.move) + tasks * c.nseg * wide * wide;
        }
        if (carry) {
            ok = ok && at(c.carry) >= end;
            end = at(c.carry) + tasks * states;
        }
        if (!ok || end * sizeof(float) > delta_ws_used(c)) {
            std::printf("delta: %lld x %d, %d heads of %d x %d, bf16 %d, %d segments of %d chunks: ent %lld, move %lld, end %lld of %zu bytes\n",
                        (long long)c.B, c.L, c.Hv, c.dk, c.dv, c.io_bf16, c.nseg, c.chunks, (long long)at(c.ent), (long long)at(c.move),
                        (long long)end, delta_ws_used(c));
            return 1;
        }
    }
    std::printf("ok: split %ld, carried %ld, odd %ld\n", split, carried, odd);
    return split && carried && odd ? 0 : 1;
}

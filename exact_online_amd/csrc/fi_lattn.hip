// fi_lattn.hip -- linear attention with a decay per head (fi_lattn_*).
//
// Per row b, key/value head n and position t, lam = exp(ld[n]):
//     S[t] = lam S[t-1] + k[t] v[t]^T,   o[t][h] = scale S[t]^T q[t][h].
#include "fi_opdev.hpp"

namespace fi {

// ------------------------------------------------------------ recurrent form
// A workgroup holds dk x 32 of one (row, head)'s state in registers: thread
// (r, c) = (tid / 8, tid % 8) has the columns 4c .. 4c+3 of the slice and the
// rows r, r + 32, ...  Columns of S never meet, so slices need no exchange.
constexpr int kRecThreads = 256;
constexpr int kRecCols = 32;
constexpr int kRecRows = kRecThreads / (kRecCols / 4);   // rows in one sweep
constexpr int kRecHeads = 8;                             // query heads at a time

template <bool BF16, int RPT>
__global__ __launch_bounds__(kRecThreads) void k_lattn_rec(LattnCall a) {
    __shared__ float ks[kRecRows * RPT], vs[kRecCols], qs[kRecHeads][kRecRows * RPT];
    __shared__ float red[kRecThreads / kWave][kRecHeads][kRecCols];
    const int tid = threadIdx.x, c = tid % (kRecCols / 4), r = tid / (kRecCols / 4);
    const int slices = (a.dv + kRecCols - 1) / kRecCols;
    const int64_t b = blockIdx.x / slices / a.Hkv;
    const int n = blockIdx.x / slices % a.Hkv, col0 = blockIdx.x % slices * kRecCols;
    const int dk = a.dk, dv = a.dv, G = a.G;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;
    const float em1 = expm1f(a.ld[n]);   // lam - 1
    float* const sp = a.state && in ? a.state + (slot * a.Hkv + n) * dk * (int64_t)dv : nullptr;

    float S[RPT][4];
    for (int i = 0; i < RPT; ++i)
        for (int j = 0; j < 4; ++j) {
            const int row = r + i * kRecRows, col = col0 + 4 * c + j;
            S[i][j] = !a.fresh && sp && row < dk && col < dv ? sp[row * (int64_t)dv + col] : 0.f;
        }
    for (int t = 0; t < len; ++t) {
        const int64_t kb = b * a.k.row + t * a.k.pos + n * a.k.head, vb = b * a.v.row + t * a.v.pos + n * a.v.head;
        for (int i = tid; i < kRecRows * RPT; i += kRecThreads) ks[i] = i < dk ? get_io<BF16>(a.k.p, kb + i) : 0.f;
        if (tid < kRecCols) vs[tid] = col0 + tid < dv ? get_io<BF16>(a.v.p, vb + col0 + tid) : 0.f;
        __syncthreads();
        // S + (lam - 1) S rather than lam S: the rounding of lam (up to 2^-25
        // of S a step, always to one side) would add up over long memories
        for (int i = 0; i < RPT; ++i)
            for (int j = 0; j < 4; ++j)
                S[i][j] = fmaf(ks[r + i * kRecRows], vs[4 * c + j], fmaf(em1, S[i][j], S[i][j]));
        for (int g0 = 0; g0 < G; g0 += kRecHeads) {
            const int gn = G - g0 < kRecHeads ? G - g0 : kRecHeads;
            __syncthreads();
            for (int i = tid; i < gn * kRecRows * RPT; i += kRecThreads) {
                const int g = i / (kRecRows * RPT), row = i % (kRecRows * RPT);
                qs[g][row] = row < dk ? get_io<BF16>(a.q.p, b * a.q.row + t * a.q.pos + (n * G + g0 + g) * a.q.head + row) : 0.f;
            }
            __syncthreads();
            for (int g = 0; g < gn; ++g)
                for (int j = 0; j < 4; ++j) {
                    float p = 0.f;
                    for (int i = 0; i < RPT; ++i) p = fmaf(qs[g][r + i * kRecRows], S[i][j], p);
                    for (int d = 8; d < kWave; d <<= 1) p += __shfl_xor(p, d);
                    if (tid % kWave < 8) red[tid / kWave][g][4 * c + j] = p;
                }
            __syncthreads();
            for (int i = tid; i < gn * kRecCols; i += kRecThreads) {
                const int g = i / kRecCols, col = i % kRecCols;
                const float o = red[0][g][col] + red[1][g][col] + red[2][g][col] + red[3][g][col];
                if (col0 + col < dv)
                    put_io<BF16>(a.o.p, b * a.o.row + t * a.o.pos + (n * G + g0 + g) * a.o.head + col0 + col, a.scale * o);
            }
        }
        __syncthreads();
    }
    for (int64_t i = (int64_t)len * G * kRecCols + tid; i < (int64_t)a.L * G * kRecCols; i += kRecThreads) {
        const int col = i % kRecCols, g = i / kRecCols % G, t = i / kRecCols / G;
        if (col0 + col < dv) put_io<BF16>(a.o.p, b * a.o.row + t * a.o.pos + (n * G + g) * a.o.head + col0 + col, 0.f);
    }
    if (sp)
        for (int i = 0; i < RPT; ++i)
            for (int j = 0; j < 4; ++j) {
                const int row = r + i * kRecRows, col = col0 + 4 * c + j;
                if (row < dk && col < dv) sp[row * (int64_t)dv + col] = S[i][j];
            }
}

hipError_t launch_lattn_rec(const LattnCall& c, hipStream_t st) {
    const bool small = c.dk <= 4 * kRecRows;
    const dim3 grid((unsigned)((c.dv + kRecCols - 1) / kRecCols * c.Hkv * c.B));   // B Hkv <= kLattnMaxRows
    if (c.io_bf16) {
        if (small) k_lattn_rec<true, 4><<<grid, kRecThreads, 0, st>>>(c);
        else k_lattn_rec<true, 8><<<grid, kRecThreads, 0, st>>>(c);
    } else {
        if (small) k_lattn_rec<false, 4><<<grid, kRecThreads, 0, st>>>(c);
        else k_lattn_rec<false, 8><<<grid, kRecThreads, 0, st>>>(c);
    }
    return hipGetLastError();
}

}  // namespace fi

// fi_dense.hip -- dense product with bias, activation and residual (fi_dense_*):
//     y[m][n] = act(sum_k x[m][k] w[n][k] + bias[n]) + res[m][n].
#include "fi_opdev.hpp"

namespace fi {

constexpr int kDsTile = 64, kDsK = 16, kDsThreads = 256;

template <bool IO, bool OUT, int ACT>
__global__ __launch_bounds__(kDsThreads) void k_dense(DenseCall a) {
    __shared__ float xs[kDsK][kDsTile + 1], ws[kDsK][kDsTile + 1];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const int64_t tn = (a.N + kDsTile - 1) / kDsTile, tiles = tn * ((a.M + kDsTile - 1) / kDsTile);
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t m0 = tile / tn * kDsTile, n0 = tile % tn * kDsTile;
        float acc[4][4] = {};
        for (int64_t k0 = 0; k0 < a.K; k0 += kDsK) {
            for (int i = tid; i < kDsTile * kDsK; i += kDsThreads) {
                const int r = i / kDsK, k = i % kDsK;
                xs[k][r] = m0 + r < a.M && k0 + k < a.K ? get_io<IO>(a.x, (m0 + r) * a.ldx + k0 + k) : 0.f;
                ws[k][r] = n0 + r < a.N && k0 + k < a.K ? get_io<IO>(a.w, (n0 + r) * a.ldw + k0 + k) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < kDsK; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[k][ty + 16 * i], ws[k][tx + 16 * j], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m >= a.M || n >= a.N) continue;
                float v = acc[i][j] + (a.bias ? get_io<IO>(a.bias, n) : 0.f);
                v = activate<ACT>(v) + (a.res ? get_io<OUT>(a.res, m * a.ldr + n) : 0.f);
                put_io<OUT>(a.y, m * a.ldy + n, v);
            }
    }
}

template <bool IO, bool OUT>
static void dense_act(const DenseCall& c, unsigned grid, hipStream_t st) {
    if (c.act == 0) k_dense<IO, OUT, 0><<<grid, kDsThreads, 0, st>>>(c);
    else if (c.act == 1) k_dense<IO, OUT, 1><<<grid, kDsThreads, 0, st>>>(c);
    else k_dense<IO, OUT, 2><<<grid, kDsThreads, 0, st>>>(c);
}

hipError_t launch_dense(const DenseCall& c, hipStream_t st) {
    const int64_t tiles = ((c.N + kDsTile - 1) / kDsTile) * ((c.M + kDsTile - 1) / kDsTile);
    const unsigned grid = (unsigned)(tiles < (1 << 22) ? tiles : 1 << 22);
    if (c.io_bf16) c.out_bf16 ? dense_act<true, true>(c, grid, st) : dense_act<true, false>(c, grid, st);
    else c.out_bf16 ? dense_act<false, true>(c, grid, st) : dense_act<false, false>(c, grid, st);
    return hipGetLastError();
}

}  // namespace fi

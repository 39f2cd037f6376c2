// fi_delta.hip -- the gated delta rule (fi_delta_*).
//
// Per row b, value head n and position t, a = exp(log_decay[t]):
//     u[t] = beta[t] (v[t] - a S[t-1]^T k[t]),   S[t] = a S[t-1] + k[t] u[t]^T,   o[t] = scale S[t]^T q[t].
#include <type_traits>

#include "fi_opdev.hpp"

namespace fi {

// ------------------------------------------------------------ recurrent form
// Position by position: a workgroup has dk x 32 of one (row, head)'s state in its
// registers, thread (r, c) = (tid / 8, tid % 8) the columns 4c .. 4c+3 of the
// slice and the rows r, r + 32, ...: columns of S never meet, so slices need no
// exchange, and rows of the slice are whole lines of memory.  Both products
// with the state before the position are formed at once, S^T k and S^T q; then
// o = a S^T q + (k . q) u needs no second pass over S.
constexpr int kDsThreads = 256, kDsWaves = kDsThreads / kWave;
constexpr int kDsCols = 32;
constexpr int kDsRows = kDsThreads / (kDsCols / 4);   // rows in one sweep

template <bool BF16, int RPT, bool VEC>
__global__ __launch_bounds__(kDsThreads) void k_delta_step(DeltaCall a) {
    constexpr int ROWS = kDsRows * RPT;
    __shared__ float ks[2][ROWS], qs[2][ROWS];
    __shared__ __align__(16) float vs[2][kDsCols], red[2][kDsWaves][2][kDsCols];   // read in 16-byte units
    __shared__ float kqs[2][kDsWaves];
    const int tid = threadIdx.x, c = tid % (kDsCols / 4), r = tid / (kDsCols / 4), wave = tid / kWave;
    const int slices = (a.dv + kDsCols - 1) / kDsCols;
    const int64_t b = blockIdx.x / slices / a.Hv;
    const int n = blockIdx.x / slices % a.Hv, col0 = blockIdx.x % slices * kDsCols;
    const int dk = a.dk, dv = a.dv;
    const int64_t slot = a.slots ? a.slots[b] : b;
    const bool in = slot >= 0 && slot < a.n_slots;
    int len = a.lens ? a.lens[b] : a.L;
    len = in ? (len < 0 ? 0 : len > a.L ? a.L : len) : 0;
    const int col = col0 + 4 * c, left = dv - col;   // columns of the state from the thread's first on

    float* const sp = in && a.state ? a.state + (slot * a.Hv + n) * dk * (int64_t)dv + r * dv + col : nullptr;
    V4 S[RPT] = {};
    if (sp && !a.fresh) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (r + i * kDsRows < dk) {
                const FI_GLOBAL float* p = gmem(sp + i * kDsRows * dv);
                if constexpr (VEC) {
                    if (left > 0) S[i] = *reinterpret_cast<const FI_GLOBAL V4*>(p);
                } else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) S[i][j] = p[j];
            }
    }
    const int64_t kb = b * a.k.row + n / a.G * a.k.head, qb = b * a.q.row + n / a.G * a.q.head, vb = b * a.v.row + n * a.v.head + col0;
    const float* const ldp = static_cast<const float*>(a.ld.p) + b * a.ld.row + n * a.ld.head;
    const float* const bp = static_cast<const float*>(a.beta.p) + b * a.beta.row + n * a.beta.head;
    const int64_t ob = b * a.o.row + n * a.o.head + col;
    // the next position's: asked for a position ahead
    float nk = 0.f, nq = 0.f, nv = 0.f, nld = 0.f, nbeta = 0.f;
    const auto ask = [&](int64_t t) {
        if (tid < dk) {
            nk = get_io<BF16>(a.k.p, kb + t * a.k.pos + tid);
            nq = get_io<BF16>(a.q.p, qb + t * a.q.pos + tid);
        }
        if (tid < kDsCols && col0 + tid < dv) nv = get_io<BF16>(a.v.p, vb + t * a.v.pos + tid);
        nld = gmem(ldp)[t * a.ld.pos];
        nbeta = gmem(bp)[t * a.beta.pos];
    };
    if (len > 0) ask(0);
    for (int t = 0; t < len; ++t) {
        const int at = t % 2;
        if (tid < ROWS) ks[at][tid] = nk, qs[at][tid] = nq;
        if (tid < kDsCols) vs[at][tid] = nv;
        const float em1 = expm1f(nld), beta = nbeta;   // a - 1
        __syncthreads();
        if (t + 1 < len) ask(t + 1);
        V4 sk = {0.f, 0.f, 0.f, 0.f}, sq = sk;
        float kq = 0.f;
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float k = ks[at][r + i * kDsRows], q = qs[at][r + i * kDsRows];
            kq = fmaf(k, q, kq);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // a S as S + (a - 1) S: the rounding of a (up to 2^-25 of S a step, always
                // to one side) would add up over long memories
                S[i][j] = fmaf(em1, S[i][j], S[i][j]);
                sk[j] = fmaf(k, S[i][j], sk[j]);
                sq[j] = fmaf(q, S[i][j], sq[j]);
            }
        }
#pragma unroll
        for (int d = 8; d < kWave; d <<= 1) {
            kq += __shfl_xor(kq, d);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sk[j] += __shfl_xor(sk[j], d);
                sq[j] += __shfl_xor(sq[j], d);
            }
        }
        if (tid % kWave < 8) {
            *smem_ptr(reinterpret_cast<V4*>(&red[at][wave][0][4 * c])) = sk;
            *smem_ptr(reinterpret_cast<V4*>(&red[at][wave][1][4 * c])) = sq;
            if (c == 0) kqs[at][wave] = kq;
        }
        __syncthreads();
        sk = sq = {0.f, 0.f, 0.f, 0.f};
        kq = 0.f;
#pragma unroll
        for (int w = 0; w < kDsWaves; ++w) {
            sk += *smem_ptr(reinterpret_cast<const V4*>(&red[at][w][0][4 * c]));
            sq += *smem_ptr(reinterpret_cast<const V4*>(&red[at][w][1][4 * c]));
            kq += kqs[at][w];
        }
        const V4 u = beta * (*smem_ptr(reinterpret_cast<const V4*>(&vs[at][4 * c])) - sk);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const float k = ks[at][r + i * kDsRows];
#pragma unroll
            for (int j = 0; j < 4; ++j) S[i][j] = fmaf(k, u[j], S[i][j]);
        }
        if (r == 0)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) put_io<BF16>(a.o.p, ob + t * a.o.pos + j, a.scale * fmaf(kq, u[j], sq[j]));
    }
    if (sp && !a.hold && (len > 0 || a.fresh)) {
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            if (r + i * kDsRows < dk) {
                FI_GLOBAL float* p = gmem(sp + i * kDsRows * dv);
                if constexpr (VEC) {
                    if (left > 0) *reinterpret_cast<FI_GLOBAL V4*>(p) = S[i];
                } else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (j < left) p[j] = S[i][j];
            }
    }
    for (int t = len + r; t < a.L; t += kDsRows)   // o is zero past the row's end
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) put_io<BF16>(a.o.p, ob + t * a.o.pos + j, 0.f);
}

hipError_t launch_delta_step(const DeltaCall& c, hipStream_t st) {
    const bool small = c.dk <= 4 * kDsRows, vec = c.dv % 4 == 0;   // the state's rows are whole 16-byte units
    const dim3 grid((unsigned)((c.dv + kDsCols - 1) / kDsCols * c.Hv * c.B));   // B Hv <= kLattnMaxRows
    const auto go = [&](auto bf, auto rpt) {
        constexpr bool BF16 = decltype(bf)::value;
        constexpr int RPT = decltype(rpt)::value;
        if (vec) k_delta_step<BF16, RPT, true><<<grid, kDsThreads, 0, st>>>(c);
        else k_delta_step<BF16, RPT, false><<<grid, kDsThreads, 0, st>>>(c);
    };
    using std::integral_constant;
    if (c.io_bf16 && small) go(std::true_type{}, integral_constant<int, 4>{});
    else if (c.io_bf16) go(std::true_type{}, integral_constant<int, 8>{});
    else if (small) go(std::false_type{}, integral_constant<int, 4>{});
    else go(std::false_type{}, integral_constant<int, 8>{});
    return hipGetLastError();
}

}  // namespace fi

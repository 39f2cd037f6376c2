// fi_opdev.hpp -- device helpers shared by the operators around the mixers.
#pragma once

#include "fi_device.hpp"
#include "fi_operators.h"

namespace fi {

using BF = __bf16;

// One element of an array of io type (bf16 or fp32), as fp32, and back
// (round to nearest even; a NaN stays one).
template <bool BF16>
__device__ __forceinline__ float get_io(const void* p, int64_t i) {
    if constexpr (BF16) return (float)gmem(static_cast<const BF*>(p))[i];
    else return gmem(static_cast<const float*>(p))[i];
}
template <bool BF16>
__device__ __forceinline__ void put_io(void* p, int64_t i, float v) {
    if constexpr (BF16) gmem(static_cast<BF*>(p))[i] = (BF)v;
    else gmem(static_cast<float*>(p))[i] = v;
}

// lam^n = exp(n ld), n >= 0; lam^0 = 1 for lam = 0 (ld = -inf) too
__device__ __forceinline__ float decay_pow(float ld, float n) { return n == 0.f ? 1.f : expf(n * ld); }

// The blocks' activations: 0 GELU (exact), 1 tanh, 2 identity.
template <int ACT>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == 0) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    else if constexpr (ACT == 1) return tanhf(v);
    else return v;
}

using BF8 = BF __attribute__((ext_vector_type(8)));
using BF4 = BF __attribute__((ext_vector_type(4)));
using S4 = short __attribute__((ext_vector_type(4)));

// Operands of the matrix cores, 16 x KB each: lane l has row (column) l % 16
// and, with g = l / 16, the E values k(g, e) of the KB long axis.  Products
// sum over k, so any k(g, e) serves that both operands share.  The result has
// column l % 16 and rows 4 g .. 4 g + 3.
template <bool BF16>
struct Mm;
template <>
struct Mm<true> {
    using T = BF;
    static constexpr int KB = 32, E = 8;
    using Frag = BF8;
    static __device__ __forceinline__ V4 mma(Frag a, Frag b, V4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <>
struct Mm<false> {
    using T = float;
    static constexpr int KB = 16, E = 4;
    using Frag = V4;
    static __device__ __forceinline__ V4 mma(Frag a, Frag b, V4 c) {
        for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
};

// 16 bytes of a row at any alignment: elements c .. c + E - 1 of the row at p
// that lie below d, zero elsewhere
template <bool BF16>
__device__ __forceinline__ typename Mm<BF16>::Frag load_loose(const typename Mm<BF16>::T* p, int64_t c, int64_t d) {
    using M = Mm<BF16>;
    using Loose = typename M::T __attribute__((ext_vector_type(M::E), aligned(sizeof(typename M::T))));
    typename M::Frag u = {};
    if (c + M::E <= d) u = *gmem(reinterpret_cast<const Loose*>(p + c));
    else {
#pragma unroll
        for (int e = 0; e < M::E; ++e)
            if (c + e < d) u[e] = gmem(p)[c + e];
    }
    return u;
}

}  // namespace fi

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

// A wave's own LDS operations before this come before those after it (they
// are performed in order; the compiler has to keep them so).
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A wave's sum (largest value) of v, in every lane: neighbours, quads, halves
// and rows of 16 lanes exchange through the data-parallel moves, the rows'
// totals through scalars.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}
template <class F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
    v = f(v, moved<0xB1>(v));    // lanes 1, 0, 3, 2
    v = f(v, moved<0x4E>(v));    // lanes 2, 3, 0, 1
    v = f(v, moved<0x141>(v));   // half rows mirrored
    v = f(v, moved<0x140>(v));   // rows mirrored
    const auto lane = [&](int l) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), l)); };
    return f(f(lane(0), lane(16)), f(lane(32), lane(48)));
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}

// lam^n = exp(n ld), n >= 0; lam^0 = 1 for lam = 0 (ld = -inf) too
__device__ __forceinline__ float decay_pow(float ld, float n) { return n == 0.f ? 1.f : expf(n * ld); }

// GELU, v Phi(v) = max(v, 0) - |v| h, h = Phi(-|v|) = e^{-v^2/2} t Q(t), t = 1 /
// (1 + 0.305 |v|): Phi(-x) e^{x^2/2} / t is smooth in t up to t = 0, and Q its
// best polynomial of degree 7 there in the relative error, 9.4e-8 (fitted by
// reweighted least squares against erfcx in 64 bits, |v| to 14).  h is off
// by (6 + v^2) 2^-23 of itself with fp32's roundings, so that the negative side,
// which is made of it, keeps its digits.  Without branches: 15 operations and two of
// the transcendental unit (the library's erff cost three times that).  |v|
// is bounded in the last product only: h is 0 there, or NaN with v.
__device__ __forceinline__ float gelu(float v) {
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(v), 0.305f, 1.f));
    const float s = v * 0.84932180028801904f;   // e^{-v^2 / 2} = 2^{-s^2}
    const float e = __builtin_amdgcn_exp2f(-(s * s));
    float q = fmaf(t, 0.036699194461107254f, -0.15298831462860107f);
    q = fmaf(t, q, 0.1857168972492218f);
    q = fmaf(t, q, -0.03797682374715805f);
    q = fmaf(t, q, 0.12102168053388596f);
    q = fmaf(t, q, 0.10342086851596832f);
    q = fmaf(t, q, 0.12246681749820709f);
    q = fmaf(t, q, 0.12163973599672318f);
    return fmaf(-fminf(fabsf(v), 1e6f), q * t * e, fmaxf(v, 0.f));
}

// tanh |v| = 1 - 2 / (1 + e^{2 |v|}), and for small v, where that cancels, its
// series to v^9 (the next term is 5e-8 v at the seam).
__device__ __forceinline__ float tanh_flat(float v) {
    const float x = fabsf(v), s = v * v;
    const float big = copysignf(fmaf(-2.f, __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(x * 2.8853900817779268f)), 1.f), v);
    float q = fmaf(s, 62.f / 2835.f, -17.f / 315.f);
    q = fmaf(s, q, 2.f / 15.f);
    q = fmaf(s, q, -1.f / 3.f);
    return x < 0.3f ? fmaf(v * s, q, v) : big;
}

// The blocks' activations: 0 GELU, 1 tanh, 2 identity.
__device__ __forceinline__ float activate(float v, int act) {
    return act == 0 ? gelu(v) : act == 1 ? tanh_flat(v) : v;
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

// 16 bytes at any alignment, where the element after them can be read too.
// Loads of 16 bytes from places that are not whole words take twice as long
// (one row, 4096 x 4095 bf16: 17 us, 8.4 with rows of whole words): from such a
// place bf16's first element by itself, the others and the next one in words
// (11.6).
template <bool BF16>
__device__ __forceinline__ typename Mm<BF16>::Frag load_by_words(const typename Mm<BF16>::T* p) {
    using M = Mm<BF16>;
    using Words = uint32_t __attribute__((ext_vector_type(4), aligned(4)));
    if constexpr (BF16) {
        const bool odd = reinterpret_cast<uintptr_t>(p) % 4 != 0;
        const uint32_t first = *gmem(reinterpret_cast<const uint16_t*>(p));
        const Words w = *gmem(reinterpret_cast<const Words*>(p + odd));
        const uint32_t moved[4] = {w.x << 16 | first, __builtin_amdgcn_alignbit(w.y, w.x, 16),
                                   __builtin_amdgcn_alignbit(w.z, w.y, 16), __builtin_amdgcn_alignbit(w.w, w.z, 16)};
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = odd ? moved[i] : w[i];
        return __builtin_bit_cast(typename M::Frag, u);
    } else return __builtin_bit_cast(typename M::Frag, *gmem(reinterpret_cast<const Words*>(p)));
}

}  // namespace fi

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

}  // namespace fi

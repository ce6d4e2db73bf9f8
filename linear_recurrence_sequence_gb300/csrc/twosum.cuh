// Sums in two floats (two-sum: the exact rounding error of an addition by
// further additions; Knuth, The Art of Computer Programming, vol. 2, 4.2.2).
#pragma once

#include "common.cuh"

namespace lrs {

// A sum in two floats: the rounding of hi is kept in lo by the exact difference
// (two-sum), so the sum is right to its last FP32 bit without FP64 arithmetic,
// whose latency here is some tenths of a microsecond an operation.
struct TwoSum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float q, float q_lo = 0.f) {
        const float t = __fadd_rn(hi, q), b = __fsub_rn(t, hi);
        lo = __fadd_rn(__fadd_rn(lo, q_lo), __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(q, b)));
        hi = t;
    }
    // a sum that overflowed has no difference to add
    __device__ __forceinline__ float value() const { return isfinite(hi) ? hi + lo : hi; }
};
__device__ __forceinline__ TwoSum warp_sum(TwoSum v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v.add(__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o));
    return v;
}

}  // namespace lrs

// The rotary angle, for the kernels that turn heads.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace w8a8 {
namespace {

constexpr int kMaxPairs = 128;  // heads of at most 256 elements

// The turn per position of a frequency f (radians), as a multiple of 2^-64 turns.
__device__ __forceinline__ uint64_t turn_step(double f) {
    // f / (2 pi) as a sum of two doubles (1 / (2 pi) = kHi + kLo), whole turns off
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    constexpr double k64 = 18446744073709551616.0;
    // of |f|: 1 - t of a small t would not be exact
    const double a = __longlong_as_double(__double_as_longlong(f) & 0x7FFFFFFFFFFFFFFFll);
    double t = a * kHi;
    const double e = fma(a, kHi, -t) + a * kLo;
    t -= floor(t);
    const uint64_t step = static_cast<uint64_t>(t * k64) + static_cast<uint64_t>(static_cast<int64_t>(e * k64));
    const uint64_t back = __double_as_longlong(f) >> 63;  // all ones for a negative f
    return (step ^ back) - back;
}

// The angle at position p in half turns, in [-1, 1).
__device__ __forceinline__ float half_turns_of(int64_t p, uint64_t step) {
    const uint64_t turn = static_cast<uint64_t>(p) * step;
    return static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
}
__device__ __forceinline__ float half_turns(int64_t p, double f) { return half_turns_of(p, turn_step(f)); }

}  // namespace
}  // namespace w8a8

// The rotary angle, and the cache rows of tokens, for the kernels that turn heads.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "operators.h"

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

// Where K and V of token t go, in elements from k_out and v_out; a slot outside the
// cache: nowhere.  kPages: caches in pages, where page_size is not 0.
struct CacheRow {
    int64_t k, v;
    bool store;
};
template <bool kPages>
__device__ __forceinline__ CacheRow cache_row(const RotaryArgs& p, int64_t t) {
    if (!p.slots) return {t * p.k_out.token, 0, true};  // (and no V)
    const int64_t slot = p.slots[t];
    const bool store = slot >= 0 && slot < p.cache_rows;
    if (!kPages) return {slot * p.k_out.token, slot * p.v_out.token, store};
    int64_t page = 0, row = slot;
    if (p.page_size && store) {
        page = (slot >> 31) ? slot / p.page_size : static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.page_size);
        row = slot - page * p.page_size;
    }
    return {page * p.k_page + row * p.k_out.token, page * p.v_page + row * p.v_out.token, store};
}

}  // namespace
}  // namespace w8a8

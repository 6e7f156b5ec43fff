// Rotary positions of Q and K heads, in place, out of place, or (for a token
// that joins a cache) with K and V written straight to their cache rows.
//
// Pair k of a head turns by the angle p f_k (p the token's position, f_k the
// pair's frequency in radians per position, a 64-bit number):
//   half layout         (x_k, x_{k + r/2}),   interleaved   (x_2k, x_{2k+1}),
//   (x, y) -> amp (x cos a - y sin a, y cos a + x sin a);
// elements past the rotated part r of the head are copied.
//
// The angle is held in turns as a 64-bit fraction: f_k / 2 pi as an integer
// multiple of 2^-64 times the integer position, modulo 2^64, is the place on
// the circle with the whole turns gone, off by 2^-64 p turns: a far position
// costs nothing (binary32 p f_k is off by 2^-24 p f_k radians: 0.06 at
// p = 10^6).  Its top 32 bits go to sincospif.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pair16.cuh"
#include "ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kRotThreads = 128;
constexpr int kMaxPairs = 128;  // heads of at most 256 elements

// The angle p f in half turns, in [-1, 1).
__device__ __forceinline__ float half_turns(int64_t p, double f) {
    // f / (2 pi) as a sum of two doubles (1 / (2 pi) = kHi + kLo), whole turns off
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    constexpr double k64 = 18446744073709551616.0;
    double t = f * kHi;
    const double e = fma(f, kHi, -t) + f * kLo;
    t -= floor(t);
    const uint64_t step = static_cast<uint64_t>(t * k64) + static_cast<uint64_t>(static_cast<int64_t>(e * k64));
    const uint64_t turn = static_cast<uint64_t>(p) * step;
    return static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
}

// Rotate 8 pairs: the half layout holds the x of pairs 0..7 in a and the y in
// b; the interleaved one x0 y0 x1 y1 ... across a then b.
template <typename T, bool kHalf>
__device__ __forceinline__ void rotate8(uint4& a, uint4& b, const float2* cs) {
    uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (kHalf) {
            const float2 x = Pair16<T>::unpack(u[i]), y = Pair16<T>::unpack(v[i]);
            const float2 t0 = cs[2 * i], t1 = cs[2 * i + 1];
            u[i] = Pair16<T>::pack(fmaf(x.x, t0.x, -(y.x * t0.y)), fmaf(x.y, t1.x, -(y.y * t1.y)));
            v[i] = Pair16<T>::pack(fmaf(y.x, t0.x, x.x * t0.y), fmaf(y.y, t1.x, x.y * t1.y));
        } else {
            const float2 x = Pair16<T>::unpack(u[i]), y = Pair16<T>::unpack(v[i]);
            const float2 t0 = cs[i], t1 = cs[4 + i];
            u[i] = Pair16<T>::pack(fmaf(x.x, t0.x, -(x.y * t0.y)), fmaf(x.y, t0.x, x.x * t0.y));
            v[i] = Pair16<T>::pack(fmaf(y.x, t1.x, -(y.y * t1.y)), fmaf(y.y, t1.x, y.x * t1.y));
        }
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
    b = make_uint4(v[0], v[1], v[2], v[3]);
}

// One CTA per token: the angles of its pairs once, in shared memory, then all
// heads of Q and K.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs p) {
    __shared__ float2 cs[kMaxPairs];
    const int64_t t = blockIdx.x;
    const int pairs = p.rot >> 1;
    const int64_t pos = p.positions[t];
    for (int i = threadIdx.x; i < pairs; i += kRotThreads) {
        float s, c;
        sincospif(half_turns(pos, p.freqs[i]), &s, &c);
        cs[i] = make_float2(c * p.amplitude, p.inverse ? -(s * p.amplitude) : s * p.amplitude);
    }
    __syncthreads();
    // the cache row of this token's K and V; outside the cache: not stored
    int64_t kt = t;
    bool store_k = true;
    if (p.slots) {
        kt = p.slots[t];
        store_k = kt >= 0 && kt < p.cache_rows;
    }
    const int per_head = p.rot >> 4;         // units of 8 pairs
    const int rest = (p.dim - p.rot) >> 3;   // 16-byte chunks past the rotated part
    auto side = [&](const Heads& in, const Heads& out, int64_t to) {
        const T* src = static_cast<const T*>(in.ptr) + t * in.token;
        T* dst = static_cast<T*>(const_cast<void*>(out.ptr)) + to * out.token;
        for (int u = threadIdx.x; u < in.heads * per_head; u += kRotThreads) {
            const int h = u / per_head, k = u - h * per_head;
            const int ia = kHalf ? 8 * k : 16 * k, ib = kHalf ? pairs + 8 * k : 16 * k + 8;
            uint4 a = *reinterpret_cast<const uint4*>(src + h * in.head + ia);
            uint4 b = *reinterpret_cast<const uint4*>(src + h * in.head + ib);
            rotate8<T, kHalf>(a, b, cs + 8 * k);
            *reinterpret_cast<uint4*>(dst + h * out.head + ia) = a;
            *reinterpret_cast<uint4*>(dst + h * out.head + ib) = b;
        }
        for (int u = threadIdx.x; u < in.heads * rest; u += kRotThreads) {
            const int h = u / rest, i = p.rot + 8 * (u - h * rest);
            *reinterpret_cast<uint4*>(dst + h * out.head + i) =
                *reinterpret_cast<const uint4*>(src + h * in.head + i);
        }
    };
    side(p.q, p.q_out, t);
    if (store_k) side(p.k, p.k_out, kt);
    if (store_k && p.v.ptr) {
        const int chunks = p.dim >> 3;
        const T* src = static_cast<const T*>(p.v.ptr) + t * p.v.token;
        T* dst = static_cast<T*>(const_cast<void*>(p.v_out.ptr)) + kt * p.v_out.token;
        for (int u = threadIdx.x; u < p.v.heads * chunks; u += kRotThreads) {
            const int h = u / chunks, i = 8 * (u - h * chunks);
            *reinterpret_cast<uint4*>(dst + h * p.v_out.head + i) =
                *reinterpret_cast<const uint4*>(src + h * p.v.head + i);
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, bool half, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.tokens));
    if (dtype == kBf16) {
        if (half) rotary_kernel<__nv_bfloat16, true><<<grid, kRotThreads, 0, st>>>(a);
        else rotary_kernel<__nv_bfloat16, false><<<grid, kRotThreads, 0, st>>>(a);
    } else {
        if (half) rotary_kernel<__half, true><<<grid, kRotThreads, 0, st>>>(a);
        else rotary_kernel<__half, false><<<grid, kRotThreads, 0, st>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace w8a8

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
// the circle with the whole turns gone, off by at most 2^-63 |p| turns (two
// numbers cut to multiples of 2^-64): nothing beside binary32 up to p = 2^38
// (binary32 p f_k is off by 2^-24 p f_k radians: 0.06 at p = 10^6).  Its top 32
// bits go to sincospif.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "operators.h"
#include "pair16.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace w8a8 {

namespace {

// Rotate 8 pairs: the half layout holds the x of pairs 0..7 in a and the y in
// b; the interleaved one x0 y0 x1 y1 ... across a then b.  cs: (cos, sin) of
// pairs 0 and 1, `step` further on of 2 and 3, and so on.
template <typename T, bool kHalf>
__device__ __forceinline__ void rotate8(uint4& a, uint4& b, const float4* cs, int step) {
    uint32_t u[4] = {a.x, a.y, a.z, a.w}, v[4] = {b.x, b.y, b.z, b.w};
    auto turn = [](uint32_t& w, float c, float s) {  // x y of one pair
        const float2 x = Pair16<T>::unpack(w);
        w = Pair16<T>::pack(fmaf(x.x, c, -(x.y * s)), fmaf(x.y, c, x.x * s));
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 t = cs[i * step];
        if (kHalf) {
            const float2 x = Pair16<T>::unpack(u[i]), y = Pair16<T>::unpack(v[i]);
            u[i] = Pair16<T>::pack(fmaf(x.x, t.x, -(y.x * t.y)), fmaf(x.y, t.z, -(y.y * t.w)));
            v[i] = Pair16<T>::pack(fmaf(y.x, t.x, x.x * t.y), fmaf(y.y, t.z, x.y * t.w));
        } else {
            turn(i < 2 ? u[2 * i] : v[2 * i - 4], t.x, t.y);
            turn(i < 2 ? u[2 * i + 1] : v[2 * i - 3], t.z, t.w);
        }
    }
    a = make_uint4(u[0], u[1], u[2], u[3]);
    b = make_uint4(v[0], v[1], v[2], v[3]);
}

constexpr int kAtOnce = 3;  // units of a thread in flight

// One CTA per token.  The angles of its pairs are computed once, in shared
// memory, while the first units of Q and K (8 pairs of a head each) are on
// their way to registers; bytes bound it: 32768 tokens x (40 + 8) heads x 128
// take 117 us, the copy bandwidth (126 with the angles in order, where the units
// of eight neighbouring threads share two banks; 4 units in flight, or the loads
// after the angles, were 5% slower).
template <typename T, bool kHalf, int kRotThreads, bool kPages>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const RotaryArgs p) {
    // two pairs each: those of a unit lie a head's units apart, so that the units of
    // neighbouring threads fall into different banks
    __shared__ float4 cs[kMaxPairs / 2];
    const int64_t t = blockIdx.x;
    const int pairs = p.rot >> 1;
    const CacheRow row = cache_row<kPages>(p, t);
    const int per_head = p.rot >> 4;  // units of a head
    const int q_units = p.q.heads * per_head, units = q_units + (row.store ? p.k.heads * per_head : 0);
    const T* q_src = static_cast<const T*>(p.q.ptr) + t * p.q.token;
    const T* k_src = static_cast<const T*>(p.k.ptr) + t * p.k.token;
    T* q_dst = static_cast<T*>(const_cast<void*>(p.q_out.ptr)) + t * p.q_out.token;
    T* k_dst = static_cast<T*>(const_cast<void*>(p.k_out.ptr)) + row.k;

    bool angles = false;
    for (int u0 = threadIdx.x; !angles || u0 < units; u0 += kAtOnce * kRotThreads) {
        uint4 a[kAtOnce], b[kAtOnce];
        T* dst[kAtOnce];
        int unit[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int u = u0 + i * kRotThreads;
            dst[i] = nullptr;
            if (u >= units) continue;
            const bool is_q = u < q_units;
            const int v = is_q ? u : u - q_units, h = v / per_head, k = v - h * per_head;
            const T* src = is_q ? q_src + h * p.q.head : k_src + h * p.k.head;
            unit[i] = k;
            const int at = kHalf ? 8 * k : 16 * k;
            dst[i] = (is_q ? q_dst + h * p.q_out.head : k_dst + h * p.k_out.head) + at;
            a[i] = *reinterpret_cast<const uint4*>(src + at);
            b[i] = *reinterpret_cast<const uint4*>(src + at + (kHalf ? pairs : 8));
        }
        if (!angles) {
            const int64_t pos = p.positions[t];
            for (int i = threadIdx.x; i < pairs; i += kRotThreads) {
                float s, c;
                sincospif(half_turns(pos, p.freqs[i]), &s, &c);
                reinterpret_cast<float2*>(cs)[2 * ((i >> 1 & 3) * per_head + (i >> 3)) + (i & 1)] =
                    make_float2(c * p.amplitude, p.inverse ? -(s * p.amplitude) : s * p.amplitude);
            }
            __syncthreads();
            angles = true;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            if (!dst[i]) continue;
            rotate8<T, kHalf>(a[i], b[i], cs + unit[i], per_head);
            *reinterpret_cast<uint4*>(dst[i]) = a[i];
            *reinterpret_cast<uint4*>(dst[i] + (kHalf ? pairs : 8)) = b[i];
        }
    }

    // 16-byte chunks that are only copied: past the rotated part, and V
    auto copy = [&](const T* src, T* dst, int heads, int64_t from, int64_t to, int first, int chunks) {
        const int all = heads * chunks;
        for (int u0 = threadIdx.x; u0 < all; u0 += kAtOnce * kRotThreads) {
            uint4 w[kAtOnce];
            T* at[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int u = u0 + i * kRotThreads;
                at[i] = nullptr;
                if (u >= all) continue;
                const int h = u / chunks, c = first + 8 * (u - h * chunks);
                w[i] = *reinterpret_cast<const uint4*>(src + h * from + c);
                at[i] = dst + h * to + c;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (at[i]) *reinterpret_cast<uint4*>(at[i]) = w[i];
        }
    };
    const int rest = (p.dim - p.rot) >> 3;
    if (rest) copy(q_src, q_dst, p.q.heads, p.q.head, p.q_out.head, p.rot, rest);
    if (rest && row.store) copy(k_src, k_dst, p.k.heads, p.k.head, p.k_out.head, p.rot, rest);
    if (row.store && p.v.ptr)
        copy(static_cast<const T*>(p.v.ptr) + t * p.v.token,
             static_cast<T*>(const_cast<void*>(p.v_out.ptr)) + row.v, p.v.heads, p.v.head, p.v_out.head, 0, p.dim >> 3);
}

template <int kRotThreads, bool kPages>
void launch_threads(const RotaryArgs& a, int dtype, bool half, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.tokens));
    if (dtype == kBf16) {
        if (half) rotary_kernel<__nv_bfloat16, true, kRotThreads, kPages><<<grid, kRotThreads, 0, st>>>(a);
        else rotary_kernel<__nv_bfloat16, false, kRotThreads, kPages><<<grid, kRotThreads, 0, st>>>(a);
    } else {
        if (half) rotary_kernel<__half, true, kRotThreads, kPages><<<grid, kRotThreads, 0, st>>>(a);
        else rotary_kernel<__half, false, kRotThreads, kPages><<<grid, kRotThreads, 0, st>>>(a);
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, bool half, int num_sms, cudaStream_t st) {
    // 64 threads where a token has no more units than they keep in flight, so that
    // more tokens are on their way (8192 tokens x 48 heads of 64 15.9 us against 18.8
    // with 128, half of heads of 128 33.1 against 36.2; whole heads of 128 32.9 against
    // 32.1), and where eight CTAs of 128 per SM would not hold all tokens (1500 tokens
    // 4.8 against 5.4, 1000 4.1 against 4.0)
    const int units = (a.q.heads + a.k.heads) * (a.rot >> 4);
    const bool narrow = units <= 64 * kAtOnce && a.tokens > static_cast<int64_t>(num_sms) * 8;
    // Pages by kernels of their own: the division, and two places of a row, cost 7 to 24%
    // (4096 tokens of 40 heads on 8 x 128 21.9 us against 20.5, 64 of them 3.5 against 3.2,
    // 1200 with half of each head turned 8.5 against 6.8), and 3 to 34% where caches of rows
    // took the same code.
    if (a.page_size) {
        if (narrow) launch_threads<64, true>(a, dtype, half, st);
        else launch_threads<128, true>(a, dtype, half, st);
    } else {
        if (narrow) launch_threads<64, false>(a, dtype, half, st);
        else launch_threads<128, false>(a, dtype, half, st);
    }
    return cudaGetLastError();
}

}  // namespace w8a8

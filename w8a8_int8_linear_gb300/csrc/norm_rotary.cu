// Norms of the query and key heads with their rotary positions, and (for tokens
// that join a cache) K and V written straight to their cache rows:
//   y = x / sqrt(mean(x^2) + eps) * gamma, or with the mean taken off first,
//   then pair k of the head turns by p f_k (rotary.cuh),
// in binary32 from the input to the one rounding of the result.
//
// 16 elements of a head (8 of its pairs, or what follows the turned part) are a
// thread's, two to a 64-bit register: the 1 to 16 neighbouring threads that hold a
// head add up its squares by shuffles, so a head is read once and stays in registers.
// Gamma, cos and sin are multiplied together once per token, in shared memory:
// element z of a pair (z, w) becomes r (z a + w b), r the reciprocal root.
//
// Bytes bound it.  A CTA takes a token at a time, so that few tokens go to as many
// SMs; the turn per position of each frequency, which takes 64-bit floating point,
// is computed once per CTA (gamma, cos and sin from their own places for every head,
// and the 64-bit steps for every token: 67.5 us against 57).  16384 tokens x 40 heads of
// 128 take 57 us (0.87 of the copy bandwidth; x 48 heads 65, 0.93), 8000 tokens of 32
// heads on 8 into pages 35, 48 single tokens 4.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "operators.h"
#include "pair16.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace w8a8 {

namespace {

constexpr int kResident = 1024;  // threads of an SM
constexpr int kAtOnce = 3;  // heads of a thread in flight
constexpr int kUnits = 16;  // threads of the largest heads
constexpr int kUnit = 20;   // floats from a thread's 16 factors to the next one's: other banks

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, uint64_t* z) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Pair16<T>::unpack(u[i]);
        z[i] = f2_pack(f.x, f.y);
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const uint64_t* z) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float a, b;
        f2_unpack(z[i], a, b);
        u[i] = Pair16<T>::pack(a, b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ uint64_t f2_swap(uint64_t z) {
    float a, b;
    f2_unpack(z, a, b);
    return f2_pack(b, a);
}
__device__ __forceinline__ float f2_sum(uint64_t z) {
    float a, b;
    f2_unpack(z, a, b);
    return a + b;
}

__device__ __forceinline__ float sum_of(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The factors of a token for Q and K: of an element, and of its partner.
struct Factors {
    float own[2][kUnits * kUnit], partner[2][kUnits * kUnit];
};

// lanes: threads of a head, a power of two.
template <typename T, bool kHalf, int kThreads>
__global__ void __launch_bounds__(kThreads, kResident / kThreads)
    norm_rotary_kernel(const __grid_constant__ NormRotaryArgs a, const int lanes) {
    __shared__ uint64_t steps[kMaxPairs];
    __shared__ __align__(16) Factors factors[2];  // of this token and the one before
    const RotaryArgs& p = a.r;
    const int pairs = p.rot >> 1;
    // gamma, where it is one for all heads
    const auto gamma_of = [&](int side, int e) {
        const HeadNorm& n = side ? a.k_norm : a.q_norm;
        return n.gamma && n.stride == 0 ? static_cast<float>(static_cast<const T*>(n.gamma)[e]) : 1.0f;
    };
    for (int i = threadIdx.x; i < pairs; i += kThreads) steps[i] = turn_step(p.freqs[i]);
    for (int e = p.rot + threadIdx.x; e < p.dim; e += kThreads)  // what does not turn
        for (int i = 0; i < 4; ++i) {
            const int at = (e >> 4) * kUnit + (e & 15);
            factors[i >> 1].own[i & 1][at] = gamma_of(i & 1, e);
            factors[i >> 1].partner[i & 1][at] = 0.0f;
        }
    __syncthreads();

    // this thread's two chunks of 8 elements
    const int unit = threadIdx.x & (lanes - 1), per_pass = kThreads / lanes, of_pass = threadIdx.x / lanes;
    const bool turns = unit < p.rot >> 4;
    const int c0 = kHalf && turns ? 8 * unit : 16 * unit, c1 = kHalf && turns ? c0 + pairs : c0 + 8;
    const bool has0 = c0 < p.dim, has1 = c1 < p.dim;
    const float inv_dim = 1.0f / p.dim;

    for (int64_t t = blockIdx.x, turn = 0; t < p.tokens; t += gridDim.x, turn ^= 1) {
        Factors& f = factors[turn];
        const CacheRow at = cache_row<true>(p, t);
        // heads of Q, then of K, then of V
        const int q_heads = p.q.heads, qk_heads = q_heads + p.k.heads;
        const int heads = at.store ? qk_heads + p.v.heads : q_heads;
        const T* q_src = static_cast<const T*>(p.q.ptr) + t * p.q.token;
        const T* k_src = static_cast<const T*>(p.k.ptr) + t * p.k.token;
        const T* v_src = static_cast<const T*>(p.v.ptr) + t * p.v.token;
        T* q_dst = static_cast<T*>(const_cast<void*>(p.q_out.ptr)) + t * p.q_out.token;
        T* k_dst = static_cast<T*>(const_cast<void*>(p.k_out.ptr)) + at.k;
        T* v_dst = static_cast<T*>(const_cast<void*>(p.v_out.ptr)) + at.v;

        bool ready = false;
        // (all threads of a warp take every pass: the shuffles are theirs together)
#pragma unroll 1
        for (int h0 = 0; !ready || h0 < heads; h0 += kAtOnce * per_pass) {
            uint4 w0[kAtOnce], w1[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const int h = h0 + i * per_pass + of_pass;
                w0[i] = w1[i] = make_uint4(0, 0, 0, 0);
                if (h >= heads) continue;
                const T* src = h < q_heads    ? q_src + h * p.q.head
                               : h < qk_heads ? k_src + (h - q_heads) * p.k.head
                                              : v_src + (h - qk_heads) * p.v.head;
                if (has0) w0[i] = *reinterpret_cast<const uint4*>(src + c0);
                if (has1) w1[i] = *reinterpret_cast<const uint4*>(src + c1);
            }
            if (!ready) {
                const int64_t pos = p.positions[t];
                for (int i = threadIdx.x; i < pairs; i += kThreads) {
                    float s, c;
                    sincospif(half_turns_of(pos, steps[i]), &s, &c);
                    c *= p.amplitude;
                    s *= p.amplitude;
                    // the pair's elements x and y, and their places
                    const int x = kHalf ? i : 2 * i, y = kHalf ? i + pairs : 2 * i + 1;
                    const int px = (i >> 3) * kUnit + (kHalf ? i & 7 : 2 * (i & 7)), py = px + (kHalf ? 8 : 1);
#pragma unroll
                    for (int side = 0; side < 2; ++side) {
                        const float gx = gamma_of(side, x), gy = gamma_of(side, y);
                        f.own[side][px] = gx * c;
                        f.partner[side][px] = -(gy * s);
                        f.own[side][py] = gy * c;
                        f.partner[side][py] = gx * s;
                    }
                }
                __syncthreads();
                ready = true;
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (h0 + i * per_pass >= heads) break;
                const int h = h0 + i * per_pass + of_pass;
                uint64_t z[8];
                unpack8<T>(w0[i], z);
                unpack8<T>(w1[i], z + 4);
                if (a.layer) {
                    uint64_t s = z[0];
#pragma unroll
                    for (int e = 1; e < 8; ++e) s = f2_add(s, z[e]);
                    const float mean = sum_of(f2_sum(s), lanes) * inv_dim;
                    const uint64_t m = f2_pack(-mean, -mean);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < 4 ? has0 : has1) z[e] = f2_add(z[e], m);
                }
                uint64_t s = f2_mul(z[0], z[0]);
#pragma unroll
                for (int e = 1; e < 8; ++e) s = f2_fma(z[e], z[e], s);
                const float r = rsqrtf(sum_of(f2_sum(s), lanes) * inv_dim + a.eps);
                if (h >= heads || !has0) continue;
                if (h >= qk_heads) {  // V as it is
                    T* to = v_dst + (h - qk_heads) * p.v_out.head;
                    *reinterpret_cast<uint4*>(to + c0) = w0[i];
                    if (has1) *reinterpret_cast<uint4*>(to + c1) = w1[i];
                    continue;
                }
                const int side = h >= q_heads, kh = side ? h - q_heads : h;
                const HeadNorm& norm = side ? a.k_norm : a.q_norm;
                if (norm.stride && norm.gamma) {  // a row of gamma for each head
                    const T* gamma = static_cast<const T*>(norm.gamma) + kh * norm.stride;
                    uint64_t g[8];
                    unpack8<T>(*reinterpret_cast<const uint4*>(gamma + c0), g);
                    unpack8<T>(has1 ? *reinterpret_cast<const uint4*>(gamma + c1) : make_uint4(0, 0, 0, 0), g + 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[e] = f2_mul(z[e], g[e]);
                }
                const uint64_t r2 = f2_pack(r, r);
                const ulonglong2* own = reinterpret_cast<const ulonglong2*>(f.own[side] + unit * kUnit);
                const ulonglong2* partner = reinterpret_cast<const ulonglong2*>(f.partner[side] + unit * kUnit);
                uint64_t y[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const ulonglong2 za = own[e >> 1], zb = partner[e >> 1];
                    const uint64_t w = kHalf ? z[(e + 4) & 7] : f2_swap(z[e]);
                    const uint64_t w1 = kHalf ? z[(e + 5) & 7] : f2_swap(z[e + 1]);
                    y[e] = f2_mul(f2_fma(z[e], za.x, f2_mul(w, zb.x)), r2);
                    y[e + 1] = f2_mul(f2_fma(z[e + 1], za.y, f2_mul(w1, zb.y)), r2);
                }
                T* to = side ? k_dst + kh * p.k_out.head : q_dst + kh * p.q_out.head;
                *reinterpret_cast<uint4*>(to + c0) = pack8<T>(y);
                if (has1) *reinterpret_cast<uint4*>(to + c1) = pack8<T>(y + 4);
            }
        }
    }
}

template <typename T, bool kHalf>
cudaError_t launch(const NormRotaryArgs& a, int num_sms, cudaStream_t st) {
    int lanes = 1;
    while (16 * lanes < a.r.dim) lanes *= 2;
    // 64 threads where a token has no more than they keep in flight
    const int threads = (a.r.q.heads + a.r.k.heads + a.r.v.heads) * lanes <= 64 * kAtOnce ? 64 : 128;
    const unsigned ctas = static_cast<unsigned>(std::min<int64_t>(a.r.tokens, num_sms * (kResident / threads)));
    if (threads == 64) norm_rotary_kernel<T, kHalf, 64><<<ctas, 64, 0, st>>>(a, lanes);
    else norm_rotary_kernel<T, kHalf, 128><<<ctas, 128, 0, st>>>(a, lanes);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rotary(const NormRotaryArgs& a, int dtype, bool half, int num_sms, cudaStream_t st) {
    if (dtype == kBf16)
        return half ? launch<__nv_bfloat16, true>(a, num_sms, st) : launch<__nv_bfloat16, false>(a, num_sms, st);
    return half ? launch<__half, true>(a, num_sms, st) : launch<__half, false>(a, num_sms, st);
}

}  // namespace w8a8

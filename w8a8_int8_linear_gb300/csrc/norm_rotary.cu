// Norms of the query and key heads with their rotary positions, and (for tokens
// that join a cache) K and V written straight to their cache rows:
//   y = x / sqrt(mean(x^2) + eps) * gamma, or with the mean taken off first,
//   then pair k of the head turns by p f_k (rotary.cuh),
// in binary32 from the input to the one rounding of the result.
//
// One CTA per token.  16 elements of a head (8 of its pairs, or what follows the
// turned part) are a thread's: the 2, 4, 8 or 16 neighbouring threads that hold a
// head add up its squares by shuffles, so a head is read once and stays in
// registers.  Bytes bound it.
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

constexpr int kThreads = 128;
constexpr int kAtOnce = 3;  // heads of a thread in flight

template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[16], int at) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = Pair16<T>::unpack(u[i]);
        x[at + 2 * i] = f.x;
        x[at + 2 * i + 1] = f.y;
    }
}
template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&x)[16], int at) {
    return make_uint4(Pair16<T>::pack(x[at], x[at + 1]), Pair16<T>::pack(x[at + 2], x[at + 3]),
                      Pair16<T>::pack(x[at + 4], x[at + 5]), Pair16<T>::pack(x[at + 6], x[at + 7]));
}

__device__ __forceinline__ float sum_of(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// lanes: threads of a head, a power of two.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kThreads) norm_rotary_kernel(const __grid_constant__ NormRotaryArgs a, const int lanes) {
    // two pairs each: those of a unit lie a head's units apart, so that the units of
    // neighbouring threads fall into different banks
    __shared__ float4 cs[kMaxPairs / 2];
    const RotaryArgs& p = a.r;
    const int64_t t = blockIdx.x;
    const int pairs = p.rot >> 1, per_head = p.rot >> 4;
    // where this token's K and V go; a slot outside the cache: nowhere
    int64_t k_at = t * p.k_out.token, v_at = 0;
    bool store_k = true;
    if (p.slots) {
        const int64_t slot = p.slots[t];
        store_k = slot >= 0 && slot < p.cache_rows;
        int64_t page = 0, row = slot;
        if (a.page_size && store_k) {
            page = (slot >> 31) ? slot / a.page_size
                                : static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.page_size);
            row = slot - page * a.page_size;
        }
        k_at = page * a.k_page + row * p.k_out.token;
        v_at = page * a.v_page + row * p.v_out.token;
    }
    const int q_heads = p.q.heads, heads = q_heads + (store_k ? p.k.heads : 0);
    const T* q_src = static_cast<const T*>(p.q.ptr) + t * p.q.token;
    const T* k_src = static_cast<const T*>(p.k.ptr) + t * p.k.token;
    T* q_dst = static_cast<T*>(const_cast<void*>(p.q_out.ptr)) + t * p.q_out.token;
    T* k_dst = static_cast<T*>(const_cast<void*>(p.k_out.ptr)) + k_at;

    // this thread's two chunks of 8 elements
    const int unit = threadIdx.x & (lanes - 1), per_pass = kThreads / lanes;
    const bool turns = unit < per_head;
    const int c0 = kHalf && turns ? 8 * unit : 16 * unit, c1 = kHalf && turns ? c0 + pairs : c0 + 8;
    const bool has0 = c0 < p.dim, has1 = c1 < p.dim;
    const float inv_dim = 1.0f / p.dim;

    bool angles = false;
    // (all threads of a warp take every step: the shuffles are theirs together)
    for (int h0 = 0; !angles || h0 < heads; h0 += kAtOnce * per_pass) {
        uint4 w0[kAtOnce], w1[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int h = h0 + i * per_pass + threadIdx.x / lanes;
            w0[i] = w1[i] = make_uint4(0, 0, 0, 0);
            if (h >= heads) continue;
            const T* src = h < q_heads ? q_src + h * p.q.head : k_src + (h - q_heads) * p.k.head;
            if (has0) w0[i] = *reinterpret_cast<const uint4*>(src + c0);
            if (has1) w1[i] = *reinterpret_cast<const uint4*>(src + c1);
        }
        if (!angles) {
            const int64_t pos = p.positions[t];
            for (int i = threadIdx.x; i < pairs; i += kThreads) {
                float s, c;
                sincospif(half_turns(pos, p.freqs[i]), &s, &c);
                reinterpret_cast<float2*>(cs)[2 * ((i >> 1 & 3) * per_head + (i >> 3)) + (i & 1)] =
                    make_float2(c * p.amplitude, s * p.amplitude);
            }
            __syncthreads();
            angles = true;
        }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int h = h0 + i * per_pass + threadIdx.x / lanes;
            float x[16];
            unpack8<T>(w0[i], x, 0);
            unpack8<T>(w1[i], x, 8);
            if (a.layer) {
                float s = 0.0f;
#pragma unroll
                for (int e = 0; e < 16; ++e) s += x[e];
                const float mean = sum_of(s, lanes) * inv_dim;
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (e < 8 ? has0 : has1) x[e] -= mean;
            }
            float s = 0.0f;
#pragma unroll
            for (int e = 0; e < 16; ++e) s = fmaf(x[e], x[e], s);
            const float r = rsqrtf(sum_of(s, lanes) * inv_dim + a.eps);
            if (h >= heads || !has0) continue;
            const bool is_q = h < q_heads;
            const HeadNorm& norm = is_q ? a.q_norm : a.k_norm;
            const int kh = is_q ? h : h - q_heads;
            if (norm.gamma) {
                const T* gamma = static_cast<const T*>(norm.gamma) + kh * norm.stride;
                float g[16];
                unpack8<T>(*reinterpret_cast<const uint4*>(gamma + c0), g, 0);
                unpack8<T>(has1 ? *reinterpret_cast<const uint4*>(gamma + c1) : make_uint4(0, 0, 0, 0), g, 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] = x[e] * r * g[e];
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) x[e] *= r;
            }
            if (turns) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float2 c = reinterpret_cast<const float2*>(cs)[2 * ((k >> 1) * per_head + unit) + (k & 1)];
                    float& u = x[kHalf ? k : 2 * k];
                    float& v = x[kHalf ? 8 + k : 2 * k + 1];
                    const float u1 = fmaf(u, c.x, -(v * c.y)), v1 = fmaf(v, c.x, u * c.y);
                    u = u1;
                    v = v1;
                }
            }
            T* dst = is_q ? q_dst + kh * p.q_out.head : k_dst + kh * p.k_out.head;
            *reinterpret_cast<uint4*>(dst + c0) = pack8<T>(x, 0);
            if (has1) *reinterpret_cast<uint4*>(dst + c1) = pack8<T>(x, 8);
        }
    }

    if (!p.v.ptr || !store_k) return;
    const T* v_src = static_cast<const T*>(p.v.ptr) + t * p.v.token;
    T* v_dst = static_cast<T*>(const_cast<void*>(p.v_out.ptr)) + v_at;
    const int chunks = p.dim >> 3, all = p.v.heads * chunks;
    for (int u = threadIdx.x; u < all; u += kThreads) {
        const int h = u / chunks, c = 8 * (u - h * chunks);
        *reinterpret_cast<uint4*>(v_dst + h * p.v_out.head + c) =
            *reinterpret_cast<const uint4*>(v_src + h * p.v.head + c);
    }
}

}  // namespace

cudaError_t launch_norm_rotary(const NormRotaryArgs& a, int dtype, bool half, int, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.r.tokens));
    int lanes = 1;
    while (16 * lanes < a.r.dim) lanes *= 2;
    if (dtype == kBf16) {
        if (half) norm_rotary_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, st>>>(a, lanes);
        else norm_rotary_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, st>>>(a, lanes);
    } else {
        if (half) norm_rotary_kernel<__half, true><<<grid, kThreads, 0, st>>>(a, lanes);
        else norm_rotary_kernel<__half, false><<<grid, kThreads, 0, st>>>(a, lanes);
    }
    return cudaGetLastError();
}

}  // namespace w8a8

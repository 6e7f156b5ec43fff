// What stands between a transformer block's output projection and the next
// block's first Linear, in one pass over the rows: the norm after the block
// (on the branch), its gate, the residual sum, the norm before the next block,
// its modulation, and the per-token int8 quantization of the W8A8 Linear
// ("TurboDiffusion Integration Notes", section "Reused Components": FastNorm
// with the modulation / residual helpers; W8A8 + FastNorm is the one combined
// stage of section "End-to-End Result").
//
//   b' = b / sqrt(S(b*b)/K + eps) * branch_gamma      (only with branch_gamma)
//   h  = alpha * x + gate * b'                        (stored in x's type)
//   n  = (h - mu) / sqrt(S((h - mu)^2)/K + eps) * gamma + beta
//                                                     (mu = 0 for RMSNorm)
//   y  = n * (1 + mod_scale) + mod_shift
//   sx = max|y| / 127, code = clamp(rne(y * (1/sx)), -127, 127)
//
// Everything between the loads and the stores is binary32: the norm goes on
// from the unrounded h, and the quantization takes the unrounded y (rounding
// either to bf16 first would only add its half step, 2^-8, to the error).
// One CTA per row; the row stays in registers between the reductions.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "pair16.cuh"
#include "ptx.cuh"
#include "quant_core.cuh"

namespace w8a8 {

namespace {

using P16 = Pair16<__nv_bfloat16>;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Sum (or maximum) over the CTA; every thread gets it.  `red` is this
// reduction's own scratch, so one barrier suffices; the order is fixed.
template <bool kMax>
__device__ __forceinline__ float block_reduce(float v, float* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    v = kMax ? warp_max(v) : warp_sum(v);
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < warps ? red[lane] : 0.0f;
    return kMax ? warp_max(v) : warp_sum(v);
}

__device__ __forceinline__ void load8(const void* base, int64_t chunk, float (&v)[8]) {
    const uint4 w = __ldg(static_cast<const uint4*>(base) + chunk);
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = P16::unpack(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(P16::pack(v[0], v[1]), P16::pack(v[2], v[3]), P16::pack(v[4], v[5]), P16::pack(v[6], v[7]));
}

// C chunks of 8 elements per thread, chunk threadIdx.x + i * blockDim.x.
template <int C, bool kF32>
__global__ void __launch_bounds__(256) residual_norm_kernel(const ResidualNormArgs p) {
    __shared__ float red[4][32];
    const int64_t row = blockIdx.x;
    const int chunks = static_cast<int>(p.K >> 3);
    const int64_t base = row * chunks;
    const int64_t group = p.rows_per_group ? row / p.rows_per_group : 0;
    const int64_t mod = group * (p.mod_stride >> 3);
    const float inv_k = 1.0f / static_cast<float>(p.K);
    float h[C][8];
    float x[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = x[i][j] = 0.0f;
        if (c >= chunks) continue;
        load8(p.B, base + c, h[i]);
        if (kF32) {
            const float4* s = static_cast<const float4*>(p.X) + 2 * (base + c);
            const float4 u = s[0], v = s[1];
            x[i][0] = u.x; x[i][1] = u.y; x[i][2] = u.z; x[i][3] = u.w;
            x[i][4] = v.x; x[i][5] = v.y; x[i][6] = v.z; x[i][7] = v.w;
        } else {
            // not through the read-only path: H may be X itself
            const uint4 w = static_cast<const uint4*>(p.X)[base + c];
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = P16::unpack(u[j]);
                x[i][2 * j] = f.x;
                x[i][2 * j + 1] = f.y;
            }
        }
    }
    if (p.branch_gamma) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
        const float r = __frcp_rn(__fsqrt_rn(fmaf(block_reduce<false>(s, red[0]), inv_k, p.eps)));
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= chunks) continue;
            float g[8];
            load8(p.branch_gamma, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * r * g[j];
        }
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= chunks) continue;
        if (p.gate) {
            float g[8];
            load8(p.gate, mod + c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            h[i][j] = fmaf(p.alpha, x[i][j], h[i][j]);
            s += p.layer ? h[i][j] : h[i][j] * h[i][j];
        }
        if (kF32) {
            float4* d = static_cast<float4*>(p.H) + 2 * (base + c);
            d[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
            d[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
        } else {
            static_cast<uint4*>(p.H)[base + c] = pack8(h[i]);
        }
    }
    s = block_reduce<false>(s, red[1]);
    float mu = 0.0f;
    if (p.layer) {  // the variance about the mean, from the values in registers
        mu = s * inv_k;
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            if (static_cast<int>(threadIdx.x + i * blockDim.x) >= chunks) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(h[i][j] - mu, h[i][j] - mu, s);
        }
        s = block_reduce<false>(s, red[2]);
    }
    const float r = __frcp_rn(__fsqrt_rn(fmaf(s, inv_k, p.eps)));
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= chunks) continue;
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) h[i][j] = (h[i][j] - mu) * r;
        if (p.gamma) {
            load8(p.gamma, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] *= g[j];
        }
        if (p.beta) {
            load8(p.beta, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += g[j];
        }
        if (p.mod_scale) {
            load8(p.mod_scale, mod + c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = fmaf(h[i][j], g[j], h[i][j]);
        }
        if (p.mod_shift) {
            load8(p.mod_shift, mod + c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] += g[j];
        }
        if (p.Y) static_cast<uint4*>(p.Y)[base + c] = pack8(h[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[i][j]));
    }
    if (!p.sx) return;
    const RowScale sc = make_scale_div(block_reduce<true>(top, red[3]));
    if (threadIdx.x == 0) p.sx[row] = sc.s;
#pragma unroll
    for (int i = 0; i < C; ++i) {
        const int c = threadIdx.x + i * blockDim.x;
        if (c >= chunks) continue;
        float q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[j] = sc.exact ? static_cast<float>(quant_exact(h[i][j], sc.s))
                            : fminf(fmaxf(rintf(h[i][j] * sc.inv), -kQMax), kQMax);
        if (p.Ximg) {
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] += 0.0f;  // the code 0 has one image, +0
            static_cast<uint4*>(p.Ximg)[base + c] = pack8(q);
        }
        if (p.Xq) {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 8; ++j)
                w[j >> 2] |= (static_cast<uint32_t>(static_cast<int>(q[j])) & 0xFFu) << (8 * (j & 3));
            reinterpret_cast<uint2*>(p.Xq)[base + c] = make_uint2(w[0], w[1]);
        }
    }
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, bool f32, cudaStream_t st) {
    const int chunks = static_cast<int>(a.K >> 3);
    const dim3 grid(static_cast<unsigned>(a.M));
    auto threads = [&](int c) { return 32 * ((chunks + 32 * c - 1) / (32 * c)); };
    auto launch = [&](auto kern, int c) { kern<<<grid, threads(c), 0, st>>>(a); };
    if (chunks <= 256) f32 ? launch(residual_norm_kernel<1, true>, 1) : launch(residual_norm_kernel<1, false>, 1);
    else if (chunks <= 1024) f32 ? launch(residual_norm_kernel<4, true>, 4) : launch(residual_norm_kernel<4, false>, 4);
    else f32 ? launch(residual_norm_kernel<8, true>, 8) : launch(residual_norm_kernel<8, false>, 8);
    return cudaGetLastError();
}

}  // namespace w8a8

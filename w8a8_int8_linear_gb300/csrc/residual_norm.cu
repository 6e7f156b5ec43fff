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
//   sx = max|y| / 127, code = rne(y * (1/sx))
//
// Everything between the loads and the stores is binary32: the norm goes on
// from the unrounded h, and the quantization takes the unrounded y (rounding
// either to bf16 first would only add its half step, 2^-8, to the error).
//
// With r the reciprocal root and v = (h - mu) * gamma, y = v * r where nothing
// else is asked for, and max|y| = r * max|v|: the sum of squares and the maximum
// then go through one reduction over the CTA.
//
// Bytes bound it (read x and b, write h and y or the image: 8 bytes an
// element), and a row passes one to four reductions between its loads and its
// stores.  With many rows a CTA therefore takes rows in a loop and bulk copies
// keep its next rows on the way to shared memory while it works on the present
// one; with few rows each CTA loads its row directly.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "operators.h"
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
// Maxima that a NaN stays in: a row that has one somewhere gets the scale NaN, and
// the Linear after it gives NaN rather than its bias.
__device__ __forceinline__ float warp_max_abs(float v) {
    float m;
    asm volatile("redux.sync.max.abs.NaN.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}
__device__ __forceinline__ float max_abs(float top, float v) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(top), "f"(fabsf(v)));
    return m;
}

// Sum of a (kSum) and maximum of |b| (kMax) over the CTA; every thread gets
// both.  `red` is this reduction's own scratch, so one barrier suffices; the
// order is fixed.
template <bool kSum, bool kMax>
__device__ __forceinline__ float2 block_reduce(float a, float b, float2* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (kSum) a = warp_sum(a);
    if (kMax) b = warp_max_abs(b);
    if (lane == 0) red[warp] = make_float2(a, b);
    __syncthreads();
    float2 v = lane < warps ? red[lane] : make_float2(0.0f, 0.0f);
    if (kSum) v.x = warp_sum(v.x);
    if (kMax) v.y = warp_max_abs(v.y);
    return v;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = P16::unpack(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void load8(const void* base, int64_t chunk, float (&v)[8]) {
    unpack8(__ldg(static_cast<const uint4*>(base) + chunk), v);
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return make_uint4(P16::pack(v[0], v[1]), P16::pack(v[2], v[3]), P16::pack(v[4], v[5]), P16::pack(v[6], v[7]));
}

constexpr int kMaxStages = 3;
constexpr int kRingBytes = 200 * 1024;

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...: C chunks of 8 elements per
// thread, chunk threadIdx.x + i * blockDim.x.  kRing: rows come through
// `stages` shared-memory buffers (x, then b), else straight from memory.
// kOptions: with a branch norm, gate, modulation or beta; without, the code
// for them does not cost the common form its registers.
template <int C, bool kF32, bool kRing, bool kOptions>
__global__ void __launch_bounds__(1024, 1) residual_norm_kernel(const ResidualNormArgs args, int stages) {
    ResidualNormArgs p = args;
    if (!kOptions) {
        p.branch_gamma = p.beta = p.gate = p.mod_scale = p.mod_shift = nullptr;
        p.rows_per_group = 0;
    }
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float2 red[2][4][32];
    __shared__ uint64_t full[kMaxStages];
    constexpr int kXBytes = kF32 ? 4 : 2;
    const int chunks = static_cast<int>(p.K >> 3);
    const uint32_t x_bytes = static_cast<uint32_t>(p.K) * kXBytes, b_bytes = static_cast<uint32_t>(p.K) * 2;
    const float inv_k = 1.0f / static_cast<float>(p.K);

    auto fetch = [&](int64_t row, int st) {
        uint8_t* dst = ring + static_cast<size_t>(st) * (x_bytes + b_bytes);
        mbar_arrive_expect_tx(&full[st], x_bytes + b_bytes);
        bulk_load(dst, static_cast<const uint8_t*>(p.X) + row * x_bytes, x_bytes, &full[st]);
        bulk_load(dst + x_bytes, static_cast<const uint8_t*>(p.B) + row * b_bytes, b_bytes, &full[st]);
    };
    if (kRing) {
        if (threadIdx.x == 0) {
            for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
            fence_mbarrier_init();
            for (int i = 0; i < stages; ++i) {
                const int64_t row = blockIdx.x + static_cast<int64_t>(i) * gridDim.x;
                if (row < p.M) fetch(row, i);
            }
        }
        __syncthreads();
    }

    // The options' values for this thread's columns stay in registers where they
    // are few (a CTA's rows ascend, so it meets each group of rows once): fetched
    // row by row they do not stay in L1 beside the ring, and the row waits for them.
    constexpr bool kHold = kOptions && C == 1;
    uint4 branch_w, gate_w, gamma_w, beta_w, scale_w, shift_w;
    const auto hold = [&](const void* base, int64_t chunk, uint4& w) {
        if (kHold && base && threadIdx.x < chunks) w = __ldg(static_cast<const uint4*>(base) + chunk + threadIdx.x);
    };
    hold(p.branch_gamma, 0, branch_w);
    hold(p.gamma, 0, gamma_w);
    hold(p.beta, 0, beta_w);
    // modulation: the chunk where the present rows' starts, and the row where they end
    int64_t mod = 0, mod_end = 0;
    // chunk `chunk` of base, or what is held of it
    auto option = [&](const void* base, int64_t chunk, const uint4& w, float(&v)[8]) {
        if (kHold)
            unpack8(w, v);
        else
            load8(base, chunk, v);
    };

    int st = 0, phase = 0, odd = 0;
    for (int64_t row = blockIdx.x; row < p.M; row += gridDim.x, odd ^= 1) {
        const int64_t base = row * chunks;
        if (kOptions && row >= mod_end) {
            const int64_t group = p.rows_per_group ? row / p.rows_per_group : 0;
            mod_end = p.rows_per_group ? (group + 1) * p.rows_per_group : p.M;
            mod = group * (p.mod_stride >> 3);
            hold(p.gate, mod, gate_w);
            hold(p.mod_scale, mod, scale_w);
            hold(p.mod_shift, mod, shift_w);
        }
        if (kRing && !mbar_wait(&full[st], phase, 80)) {
            // recorded; the copies still on their way land before the CTA ends
            if (threadIdx.x == 0)
                for (int i = 1; i < stages; ++i) {
                    const int at = (st + i) % stages;
                    if (row + static_cast<int64_t>(i) * gridDim.x < p.M)
                        mbar_wait(&full[at], at > st ? phase : phase ^ 1, 80);
                }
            return;
        }
        const uint8_t* buf = ring + static_cast<size_t>(st) * (x_bytes + b_bytes);
        // x not through the read-only path: H may be X itself
        const uint4* xs = kRing ? reinterpret_cast<const uint4*>(buf)
                                : reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.X) + row * x_bytes);
        const uint4* bs = kRing ? reinterpret_cast<const uint4*>(buf + x_bytes)
                                : reinterpret_cast<const uint4*>(p.B) + base;
        constexpr int kX = kF32 ? 2 : 1;
        uint4 xw[C][kX], bw[C];
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            bw[i] = c < chunks ? bs[c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int k = 0; k < kX; ++k) xw[i][k] = c < chunks ? xs[kX * c + k] : make_uint4(0, 0, 0, 0);
        }
        float h[C][8];
        bool fetched = !kRing;
        // after the first reduction's barrier every thread has read its part of
        // the buffer: the row that goes there next can be fetched
        auto refill = [&]() {
            if (!fetched && threadIdx.x == 0) {
                const int64_t next = row + static_cast<int64_t>(stages) * gridDim.x;
                if (next < p.M) fetch(next, st);
            }
            fetched = true;
        };
        float branch = 1.0f;  // reciprocal root of the branch's mean square
        if (p.branch_gamma) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                unpack8(bw[i], h[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
            }
            branch = __frcp_rn(__fsqrt_rn(fmaf(block_reduce<true, false>(s, 0.0f, red[odd][0]).x, inv_k, p.eps)));
            refill();
        }
        // h; RMSNorm's v right away
        auto scaled = [&](int c, float(&v)[8]) {  // d -> v
            if (!p.gamma) return;
            float g[8];
            option(p.gamma, c, gamma_w, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= g[j];
        };
        float s = 0.0f, top = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= chunks) continue;
            unpack8(bw[i], h[i]);
            float g[8];
            if (p.branch_gamma) {
                option(p.branch_gamma, c, branch_w, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * branch * g[j];
            }
            if (p.gate) {
                option(p.gate, mod + c, gate_w, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = h[i][j] * g[j];
            }
            if (kF32) {
                const uint4 u = xw[i][0], v = xw[i][kX - 1];
                g[0] = __uint_as_float(u.x); g[1] = __uint_as_float(u.y);
                g[2] = __uint_as_float(u.z); g[3] = __uint_as_float(u.w);
                g[4] = __uint_as_float(v.x); g[5] = __uint_as_float(v.y);
                g[6] = __uint_as_float(v.z); g[7] = __uint_as_float(v.w);
            } else {
                unpack8(xw[i][0], g);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = fmaf(p.alpha, g[j], h[i][j]);
            if (kF32) {
                float4* d = static_cast<float4*>(p.H) + 2 * (base + c);
                d[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
                d[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
            } else {
                static_cast<uint4*>(p.H)[base + c] = pack8(h[i]);
            }
            if (p.layer) {
#pragma unroll
                for (int j = 0; j < 8; ++j) s += h[i][j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) s = fmaf(h[i][j], h[i][j], s);
                if (!kOptions) {
                    scaled(c, h[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max_abs(top, h[i][j]);
                }
            }
        }
        float2 all = p.layer || kOptions ? block_reduce<true, false>(s, 0.0f, red[odd][1])
                                         : block_reduce<true, true>(s, top, red[odd][1]);
        refill();
        if (p.layer) {  // the variance about the mean, from the values in registers
            const float mu = all.x * inv_k;
            s = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= chunks) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    h[i][j] -= mu;
                    s = fmaf(h[i][j], h[i][j], s);
                }
                if (!kOptions) {
                    scaled(c, h[i]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max_abs(top, h[i][j]);
                }
            }
            all = block_reduce<true, !kOptions>(s, top, red[odd][2]);
        }
        if (kRing && ++st == stages) {
            st = 0;
            phase ^= 1;
        }
        const float r = __frcp_rn(__fsqrt_rn(fmaf(all.x, inv_k, p.eps)));
        float peak = all.y * r;
        if (kOptions) {
            top = 0.0f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c >= chunks) continue;
                float g[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] *= r;
                scaled(c, h[i]);
                if (p.beta) {
                    option(p.beta, c, beta_w, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += g[j];
                }
                if (p.mod_scale) {
                    option(p.mod_scale, mod + c, scale_w, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] = fmaf(h[i][j], g[j], h[i][j]);
                }
                if (p.mod_shift) {
                    option(p.mod_shift, mod + c, shift_w, g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += g[j];
                }
                if (p.sx) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max_abs(top, h[i][j]);
                }
            }
            if (p.sx) peak = block_reduce<false, true>(0.0f, top, red[odd][3]).y;
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] *= r;
        }
        if (p.Y) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
                const int c = threadIdx.x + i * blockDim.x;
                if (c < chunks) static_cast<uint4*>(p.Y)[base + c] = pack8(h[i]);
            }
        }
        if (!p.sx) continue;
        const RowScale sc = make_scale_div(peak);
        if (threadIdx.x == 0) p.sx[row] = sc.s;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int c = threadIdx.x + i * blockDim.x;
            if (c >= chunks) continue;
            // rne(y / sx) + 1.5 * 2^23, the code in the low byte; never above 127, as
            // max|y| / sx is within a few roundings of 127
            float q[8];
            if (sc.exact) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = static_cast<float>(quant_exact(h[i][j], sc.s)) + kRoundMagic;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] = fmaf(h[i][j], sc.inv, kRoundMagic);
            }
            if (p.Xq) {
                uint32_t u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(q[j]);
                reinterpret_cast<uint2*>(p.Xq)[base + c] = make_uint2(
                    __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410));
            }
            if (p.Ximg) {
#pragma unroll
                for (int j = 0; j < 8; ++j) q[j] -= kRoundMagic;  // the code 0 is +0
                static_cast<uint4*>(p.Ximg)[base + c] = pack8(q);
            }
        }
    }
}

template <int C, bool kF32, bool kOptions>
cudaError_t launch_rows(const ResidualNormArgs& a, int num_sms, cudaStream_t st) {
    const int chunks = static_cast<int>(a.K >> 3);
    const int threads = 32 * ((chunks + 32 * C - 1) / (32 * C));
    const int row_bytes = static_cast<int>(a.K) * (kF32 ? 6 : 4);
    // Fewer rows in flight are better where little is computed between load and
    // store, more where a row passes several reductions.  Measured, CTAs x buffers:
    // 32768 x 5120 to the image 209 us at 2 x 3 (228 at 3 x 2, 235 at 4 x 2), 32768
    // x 4096 166 at 3 x 3 (189 at 4 x 2), x 8192 321 at 2 x 3 (356 at 3 x 2); with
    // a branch norm 16384 x 5120 116 at 3 x 2 (132 at 2 x 3), 4096 x 4096 32 at 4 x 2
    // (45 at 2 x 3).  So too where an SM has few rows to
    // share out: 4096 x 4096 to the image 22.8 at 4 x 2 (25.5 at 3 x 3).
    const bool many = kOptions || a.M < static_cast<int64_t>(num_sms) * 32;
    int per_sm = many ? 1024 / threads : (768 + threads / 2) / threads;
    if (per_sm > 16) per_sm = 16;
    if (per_sm < 1) per_sm = 1;
    int stages = many ? 2 : 3;
    while (per_sm > 1 && per_sm * stages * row_bytes > kRingBytes) --per_sm;
    if (stages * row_bytes > kRingBytes) stages = 2;
    if (a.M <= static_cast<int64_t>(num_sms) * per_sm) {
        residual_norm_kernel<C, kF32, false, kOptions><<<static_cast<unsigned>(a.M), threads, 0, st>>>(a, 0);
        return cudaGetLastError();
    }
    static bool allowed[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !allowed[dev]) {
        e = cudaFuncSetAttribute(residual_norm_kernel<C, kF32, true, kOptions>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
        if (e != cudaSuccess) return e;
        if (dev < 64) allowed[dev] = true;
    }
    residual_norm_kernel<C, kF32, true, kOptions>
        <<<num_sms * per_sm, threads, static_cast<size_t>(stages) * row_bytes, st>>>(a, stages);
    return cudaGetLastError();
}

template <bool kF32, bool kOptions>
cudaError_t launch_width(const ResidualNormArgs& a, int num_sms, cudaStream_t st) {
    // Narrow CTAs, so that more rows are on their way through their reductions: two
    // chunks a thread from 512 elements on (16384 x 2048 with a branch norm 56 us
    // against 72 with one, x 1024 32 against 38; x 512 21 with one against 23).  One
    // chunk where the options are then held in registers and a CTA keeps them for
    // several rows, if rows are long in bytes (fp32 x, gate, scale and shift: 4096 x
    // 4096 37 us against 47 with two chunks, 4096 x 8192 71 against 87, 1000 x 4096
    // 11.4 against 12.6; 600 x 4096 8.0 against 7.1).  In bf16 a row leaves less time
    // than the fewer, wider CTAs take to reduce it (16384 x 5120 with a branch norm
    // 172 against 116).
    const bool wide = kF32 && kOptions && a.K <= 8192 && a.M >= static_cast<int64_t>(num_sms) * 6;
    return wide || a.K <= 512 ? launch_rows<1, kF32, kOptions>(a, num_sms, st)
                              : launch_rows<2, kF32, kOptions>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_residual_norm(const ResidualNormArgs& a, bool f32, int num_sms, cudaStream_t st) {
    const bool options = a.branch_gamma || a.beta || a.gate || a.mod_scale || a.mod_shift;
    if (f32) return options ? launch_width<true, true>(a, num_sms, st) : launch_width<true, false>(a, num_sms, st);
    return options ? launch_width<false, true>(a, num_sms, st) : launch_width<false, false>(a, num_sms, st);
}

cudaError_t residual_norm_read_device_error(unsigned int* code) {
    unsigned int v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_device_error, &z, sizeof z);
    *code = v;
    return e;
}

}  // namespace w8a8

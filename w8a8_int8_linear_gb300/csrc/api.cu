// C ABI of the W8A8 INT8 Linear library (declared in include/w8a8.h):
// argument checks, device checks, workspace carving and kernel launches.
// Every check runs before anything is enqueued, so a rejected call leaves
// all outputs untouched.
#include <algorithm>
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdint>
#include <mutex>

#include "../../include/w8a8.h"
#include "device_errors.h"
#include "gemv.h"
#include "kernels.h"
#include "operators.h"

namespace {

constexpr int64_t kMaxK = 131072;  // 127 * 127 * K must stay below 2^31
constexpr int kMaxDevices = 64;
// Rows of queries (times the heads of a group) and of keys: the attention kernels count them
// in 32 bits, rounded up to whole tiles.
constexpr int64_t kMostRows = INT32_MAX - 1024;

struct DeviceInfo {
    bool ok;
    int num_sms;
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
std::atomic<bool> g_dev_known[kMaxDevices];
void* g_encode = nullptr;
thread_local char t_detail[256] = "";
thread_local cudaEvent_t t_gemm_start = nullptr;
thread_local cudaEvent_t t_gemm_end = nullptr;

void set_detail(const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(t_detail, sizeof t_detail, fmt, ap);
    va_end(ap);
}

w8a8_status cuda_fail(const char* what, cudaError_t e) {
    set_detail("%s: %s", what, cudaGetErrorString(e));
    return W8A8_ERR_CUDA;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Workspace of the GEMM on bf16 operand images: the images of Xq and Wq and
// the int32 partial sums of the K splits.
size_t image_gemm_need(int64_t M, int64_t N, int64_t K) {
    return align256(static_cast<size_t>(M) * K * 2) + align256(static_cast<size_t>(N) * K * 2) +
           align256(w8a8::splitk_partial_bytes(M, N, K));
}

// Current device must be compute capability 10.3.
w8a8_status current_device(DeviceInfo* out) {
    int dev = 0;
    cudaError_t ge = cudaGetDevice(&dev);
    if (ge != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("cudaGetDevice", ge);
    }
    if (dev < 0 || dev >= kMaxDevices) return W8A8_ERR_UNSUPPORTED_DEVICE;
    if (!g_dev_known[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_dev_known[dev].load(std::memory_order_relaxed)) {
            int major = 0, minor = 0, sms = 0;
            if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
                cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
                cudaGetLastError();
                set_detail("cudaDeviceGetAttribute failed on device %d", dev);
                return W8A8_ERR_CUDA;
            }
            g_dev[dev].ok = (major == 10 && minor == 3);
            g_dev[dev].num_sms = sms;
            g_dev_known[dev].store(true, std::memory_order_release);
        }
    }
    *out = g_dev[dev];
    return out->ok ? W8A8_OK : W8A8_ERR_UNSUPPORTED_DEVICE;
}

void* encode_fn() {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        cudaDriverEntryPointQueryResult q;
        void* fn = nullptr;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e == cudaSuccess && q == cudaDriverEntryPointSuccess && fn) {
            g_encode = fn;
        } else {
            cudaGetLastError();
            set_detail("cudaGetDriverEntryPointByVersion(cuTensorMapEncodeTiled): %s, query result %d",
                       cudaGetErrorString(e), (int)q);
        }
    }
    return g_encode;
}

w8a8_status from_cuda(cudaError_t e, const char* what = "kernel launch") {
    return e == cudaSuccess ? W8A8_OK : cuda_fail(what, e);
}

w8a8_status check_k(int64_t K, bool block) {
    if (K <= 0) return W8A8_ERR_INVALID_ARG;
    if (K % 16 != 0 || K > kMaxK) return W8A8_ERR_SHAPE;
    if (block && K % 128 != 0) return W8A8_ERR_SHAPE;
    return W8A8_OK;
}

// Workspace bytes the post-scale GEMM (int8 codes in) uses for this shape:
// none for the few-token GEMV; when the GEMM streams the int8 codes itself
// (M <= 288), the fp16 image of Xq and, where K may be split, int32 sums and
// counters; else the bf16 images of Xq and Wq plus the partial sums of the
// K splits.  M, N, K > 0.
size_t postscale_gemm_need(int64_t M, int64_t N, int64_t K) {
    if (w8a8::gemv_takes(M, K)) return 0;
    if (w8a8::gemm_takes_int8(w8a8::kEpiPostscaleBf16, M)) return w8a8::s8_workspace_bytes(M, N, K);
    return image_gemm_need(M, N, K);
}

// Shared checks of the GEMM entry points.  need_sx/need_sw: scale pointers
// used by this variant.
w8a8_status check_gemm(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, const void* bias,
                       const void* out, int64_t M, int64_t N, int64_t K, bool block, bool need_scales,
                       const void* ws, size_t ws_bytes, DeviceInfo* dev, bool* nothing_to_do) {
    *nothing_to_do = false;
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, block);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) {
        *nothing_to_do = true;
        return W8A8_OK;
    }
    if (!Xq || !Wq || !out || (need_scales && (!sx || !sw))) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(Xq) || !aligned16(Wq) || !aligned16(out) || (sx && !aligned16(sx)) ||
        (sw && !aligned16(sw)) || (bias && !aligned16(bias)))
        return W8A8_ERR_ALIGNMENT;
    const size_t need = block ? w8a8_gemm_workspace_size(M, N, K) : postscale_gemm_need(M, N, K);
    if (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need)) return W8A8_ERR_WORKSPACE;
    return current_device(dev);
}

// GEMM on bf16 operand images, with the timing hook around the launch.
w8a8_status run_gemm_images(int epi, const void* Ab, const void* Bb, const float* sx, const float* sw,
                            const void* bias, void* out, int64_t M, int64_t N, int64_t K, void* partial,
                            const DeviceInfo& dev, cudaStream_t st, float* sg = nullptr,
                            bool weights_settled = false, bool int8_operands = false,
                            bool tokens_widened = false) {
    void* enc = encode_fn();
    if (!enc) return W8A8_ERR_CUDA;
    w8a8::GemmArgs a;
    a.sx = sx;
    a.sw = sw;
    a.bias = bias;
    a.out = out;
    a.M = M;
    a.N = N;
    a.K = K;
    a.partial = static_cast<int32_t*>(partial);
    a.sg = sg;
    a.weights_settled = weights_settled;
    a.int8_operands = int8_operands;
    a.tokens_widened = tokens_widened;
    cudaError_t e;
    if (t_gemm_start && (e = cudaEventRecord(t_gemm_start, st)) != cudaSuccess) return cuda_fail("event", e);
    e = w8a8::launch_gemm(epi, Ab, Bb, a, dev.num_sms, enc, st, t_detail, sizeof t_detail);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return W8A8_ERR_CUDA;
    }
    if (t_gemm_end && (e = cudaEventRecord(t_gemm_end, st)) != cudaSuccess) return cuda_fail("event", e);
    return W8A8_OK;
}

// Checks and launches of the fused Linear entry points.
w8a8_status run_linear(bool block, const void* X, const void* Wimg, const float* sw, const void* bias, void* Y,
                       int64_t M, int64_t N, int64_t K, float* sx, int8_t* Xq, void* ws, size_t ws_bytes,
                       cudaStream_t st) {
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, block);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    if (!X || !Wimg || !sw || !Y || !sx) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Wimg) || !aligned16(sw) || !aligned16(Y) || !aligned16(sx) ||
        (Xq && !aligned16(Xq)) || (bias && !aligned16(bias)))
        return W8A8_ERR_ALIGNMENT;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < w8a8_linear_workspace_size(M, N, K))
        return W8A8_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    cudaError_t e = block ? w8a8::launch_quant_act_block(X, M, K, Xq, ws, sx, dev.num_sms, st)
                          : w8a8::launch_quant_rows(X, M, K, Xq, ws, sx, dev.num_sms, st);
    if (e != cudaSuccess) return cuda_fail("activation quant launch", e);
    void* partial = static_cast<uint8_t*>(ws) + align256(static_cast<size_t>(M) * K * 2);
    // Wimg predates the quantization kernel just launched (which waited for
    // all earlier work), so the GEMM may start reading it before that kernel ends.
    return run_gemm_images(block ? w8a8::kEpiBlockwiseBf16 : w8a8::kEpiPostscaleBf16, ws, Wimg, sx, sw, bias, Y, M,
                           N, K, partial, dev, st, nullptr, true);
}

// Checks and launches of the fused FFN up-projection (quant, GEMM with the
// GELU + 1x128 quantization epilogue).
w8a8_status run_linear_gelu_quant(const void* X, const void* Wimg, const float* sw, const void* bias, void* Gimg,
                                  float* sg, int64_t M, int64_t N, int64_t K, float* sx, int8_t* Xq, void* ws,
                                  size_t ws_bytes, cudaStream_t st) {
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, false);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX || N % 128 != 0) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    if (!X || !Wimg || !sw || !Gimg || !sg || !sx) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Wimg) || !aligned16(sw) || !aligned16(Gimg) || !aligned16(sg) ||
        !aligned16(sx) || (Xq && !aligned16(Xq)) || (bias && !aligned16(bias)))
        return W8A8_ERR_ALIGNMENT;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < w8a8_linear_workspace_size(M, N, K))
        return W8A8_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    cudaError_t e = w8a8::launch_quant_rows(X, M, K, Xq, ws, sx, dev.num_sms, st);
    if (e != cudaSuccess) return cuda_fail("activation quant launch", e);
    return run_gemm_images(w8a8::kEpiGeluQuant, ws, Wimg, sx, sw, bias, Gimg, M, N, K, nullptr, dev, st, sg, true);
}

// Few-token post-scale GEMM on the CUDA cores (with the per-token
// quantization folded in when X is given instead of Xq), with the timing hook
// around the launch.
w8a8_status run_gemv(int epi, const void* X, const int8_t* Xq, float* sx, int8_t* Xq_out, const int8_t* Wq,
                     const float* sw, const void* bias, void* out, int64_t M, int64_t N, int64_t K,
                     bool weights_settled, const DeviceInfo& dev, cudaStream_t st) {
    cudaError_t e;
    if (t_gemm_start && (e = cudaEventRecord(t_gemm_start, st)) != cudaSuccess) return cuda_fail("event", e);
    e = X ? w8a8::launch_gemv_s8_quant(X, sx, Xq_out, Wq, sw, bias, out, M, N, K, dev.num_sms, st)
          : w8a8::launch_gemv_s8(epi, Xq, sx, Wq, sw, bias, out, M, N, K, weights_settled, dev.num_sms, st);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("few-token GEMV launch", e);
    }
    if (t_gemm_end && (e = cudaEventRecord(t_gemm_end, st)) != cudaSuccess) return cuda_fail("event", e);
    return W8A8_OK;
}

bool takes_gemv(int epi, int64_t M, int64_t K) {
    return (epi == w8a8::kEpiPostscaleBf16 || epi == w8a8::kEpiPostscaleS32) && w8a8::gemv_takes(M, K);
}

w8a8_status run_gemm(int epi, const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw,
                     const void* bias, void* out, int64_t M, int64_t N, int64_t K, void* ws, const DeviceInfo& dev,
                     cudaStream_t st, bool weights_settled = false) {
    // a handful of tokens: a GEMV streaming the int8 weight codes
    if (takes_gemv(epi, M, K))
        return run_gemv(epi, nullptr, Xq, const_cast<float*>(sx), nullptr, Wq, sw, bias, out, M, N, K,
                        weights_settled, dev, st);
    void* enc = encode_fn();
    if (!enc) return W8A8_ERR_CUDA;
    uint8_t* w = static_cast<uint8_t*>(ws);
    if (w8a8::gemm_takes_int8(epi, M)) {
        // few tokens: the GEMM streams the int8 codes itself, no images
        return run_gemm_images(epi, Xq, Wq, sx, sw, bias, out, M, N, K, w, dev, st, nullptr, weights_settled, true);
    }
    void* Ab = w;
    void* Bb = w + align256(static_cast<size_t>(M) * K * 2);
    void* partial = static_cast<uint8_t*>(Bb) + align256(static_cast<size_t>(N) * K * 2);
    cudaError_t e = w8a8::launch_expand_s8_bf16(Xq, M * K, Ab, dev.num_sms, st);
    if (e != cudaSuccess) return cuda_fail("expand Xq launch", e);
    e = w8a8::launch_expand_s8_bf16(Wq, N * K, Bb, dev.num_sms, st);
    if (e != cudaSuccess) return cuda_fail("expand Wq launch", e);
    return run_gemm_images(epi, Ab, Bb, sx, sw, bias, out, M, N, K, partial, dev, st);
}

bool linear_codes_fused(int64_t M, int64_t K) { return w8a8::gemv_takes(M, K) && M <= w8a8::kGemvFusedMaxTokens; }

// The one-kernel GEMV path needs no workspace; otherwise the codes of X, plus
// the GEMM's workspace unless the GEMM is the GEMV.
size_t linear_codes_workspace(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0 || linear_codes_fused(M, K)) return 0;
    return align256(static_cast<size_t>(M) * K) + postscale_gemm_need(M, N, K);
}

// Checks and launches of the fused Linear on int8 weight codes: per-token
// quantization of X, then the post-scale GEMM on the codes.
w8a8_status run_linear_codes(const void* X, const int8_t* Wq, const float* sw, const void* bias, void* Y, int64_t M,
                             int64_t N, int64_t K, float* sx, int8_t* Xq, void* ws, size_t ws_bytes,
                             cudaStream_t st) {
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, false);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    if (!X || !Wq || !sw || !Y || !sx) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Wq) || !aligned16(sw) || !aligned16(Y) || !aligned16(sx) ||
        (Xq && !aligned16(Xq)) || (bias && !aligned16(bias)))
        return W8A8_ERR_ALIGNMENT;
    const size_t need = linear_codes_workspace(M, N, K);
    if (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || ws_bytes < need))
        return W8A8_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    // one or two tokens: one kernel quantizes X in every CTA and streams the weight codes
    if (linear_codes_fused(M, K))
        return run_gemv(w8a8::kEpiPostscaleBf16, X, nullptr, sx, Xq, Wq, sw, bias, Y, M, N, K, false, dev, st);
    int8_t* q = Xq ? Xq : static_cast<int8_t*>(ws);
    uint8_t* rest = static_cast<uint8_t*>(ws) + align256(static_cast<size_t>(M) * K);
    if (!w8a8::gemv_takes(M, K) && w8a8::gemm_takes_int8(w8a8::kEpiPostscaleBf16, M) &&
        w8a8::quant_tokens_f16_takes(K)) {
        // few tokens on the int8-operand GEMM: the quantization kernel also
        // writes the GEMM's fp16 token image and zeroes its split-K sums
        size_t zoff = 0, zbytes = 0;
        w8a8::s8_scratch_zero(M, N, K, dev.num_sms, &zoff, &zbytes);
        cudaError_t e = w8a8::launch_quant_tokens_f16(X, M, K, Xq, rest, sx, rest + zoff, zbytes, st);
        if (e != cudaSuccess) return cuda_fail("activation quant launch", e);
        return run_gemm_images(w8a8::kEpiPostscaleBf16, Xq, Wq, sx, sw, bias, Y, M, N, K, rest, dev, st, nullptr,
                               true, true, true);
    }
    cudaError_t e = w8a8::launch_quant_rows(X, M, K, q, nullptr, sx, dev.num_sms, st);
    if (e != cudaSuccess) return cuda_fail("activation quant launch", e);
    // Wq predates the quantization kernel just launched (which waited for all
    // earlier work), so the GEMM may start reading it before that kernel ends.
    return run_gemm(w8a8::kEpiPostscaleBf16, q, sx, Wq, sw, bias, Y, M, N, K, rest, dev, st, true);
}

// Scratch of the allocation-free GEMM entry point: a fixed device array,
// loaded with the library on every device that uses it and held until the
// process exits.  The name is a host-side stand-in; its device address comes
// from cudaGetSymbolAddress, taken once per device with that device current.
constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;  // 64 MiB
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];
void* g_noalloc_ptr[kMaxDevices];
std::atomic<bool> g_noalloc_ready[kMaxDevices];

w8a8_status noalloc_scratch(void** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return cuda_fail("cudaGetDevice", e);
    }
    if (dev < 0 || dev >= kMaxDevices) return W8A8_ERR_UNSUPPORTED_DEVICE;
    if (!g_noalloc_ready[dev].load(std::memory_order_acquire)) {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!g_noalloc_ready[dev].load(std::memory_order_relaxed)) {
            void* p = nullptr;
            e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
            if (e != cudaSuccess || p == nullptr) {
                cudaGetLastError();
                return cuda_fail("cudaGetSymbolAddress(no-alloc scratch)", e);
            }
            g_noalloc_ptr[dev] = p;
            g_noalloc_ready[dev].store(true, std::memory_order_release);
        }
    }
    *out = g_noalloc_ptr[dev];
    return W8A8_OK;
}

}  // namespace

extern "C" {

const char* w8a8_status_string(w8a8_status s) {
    switch (s) {
        case W8A8_OK: return "W8A8_OK";
        case W8A8_ERR_INVALID_ARG: return "W8A8_ERR_INVALID_ARG: null pointer, bad mode or negative size";
        case W8A8_ERR_ALIGNMENT: return "W8A8_ERR_ALIGNMENT: a pointer is not 16-byte aligned";
        case W8A8_ERR_SHAPE: return "W8A8_ERR_SHAPE: K must be a positive multiple of 16 (128 for blocks), <= 131072";
        case W8A8_ERR_UNSUPPORTED_DEVICE: return "W8A8_ERR_UNSUPPORTED_DEVICE: current device is not sm_103";
        case W8A8_ERR_CUDA: return "W8A8_ERR_CUDA: a CUDA call failed";
        case W8A8_ERR_TIMEOUT: return "W8A8_ERR_TIMEOUT: a device-side bounded wait ran out";
        case W8A8_ERR_WORKSPACE: return "W8A8_ERR_WORKSPACE: workspace missing, unaligned or too small";
    }
    return "unknown w8a8_status";
}

w8a8_status w8a8_quantize_weight(const void* W, int64_t N, int64_t K, w8a8_scale_mode mode, int8_t* Wq,
                                 float* sw, void* stream) {
    if (mode != W8A8_SCALE_PER_ROW && mode != W8A8_SCALE_BLOCK) return W8A8_ERR_INVALID_ARG;
    if (N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, mode == W8A8_SCALE_BLOCK);
    if (s != W8A8_OK) return s;
    if (N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (N == 0) return W8A8_OK;
    if (!W || !Wq || !sw) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(W) || !aligned16(Wq) || !aligned16(sw)) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (mode == W8A8_SCALE_PER_ROW) return from_cuda(w8a8::launch_quant_rows(W, N, K, Wq, nullptr, sw, dev.num_sms, st));
    if ((N + 127) / 128 > 65535) return W8A8_ERR_SHAPE;
    return from_cuda(w8a8::launch_quant_weight_block(W, N, K, Wq, sw, st));
}

w8a8_status w8a8_quantize_act(const void* X, int64_t M, int64_t K, w8a8_scale_mode mode, int8_t* Xq, float* sx,
                              void* stream) {
    if (mode != W8A8_SCALE_PER_ROW && mode != W8A8_SCALE_BLOCK) return W8A8_ERR_INVALID_ARG;
    if (M < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, mode == W8A8_SCALE_BLOCK);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0) return W8A8_OK;
    if (!X || !Xq || !sx) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(X) || !aligned16(Xq) || !aligned16(sx)) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (mode == W8A8_SCALE_PER_ROW) return from_cuda(w8a8::launch_quant_rows(X, M, K, Xq, nullptr, sx, dev.num_sms, st));
    return from_cuda(w8a8::launch_quant_act_block(X, M, K, Xq, nullptr, sx, dev.num_sms, st));
}

w8a8_status w8a8_pack_weight(const int8_t* Wq, int64_t N, int64_t K, void* Wimg, void* stream) {
    if (N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, false);
    if (s != W8A8_OK) return s;
    if (N == 0) return W8A8_OK;
    if (!Wq || !Wimg) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(Wq) || !aligned16(Wimg)) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    return from_cuda(w8a8::launch_expand_s8_bf16(Wq, N * K, Wimg, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

size_t w8a8_linear_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    return align256(static_cast<size_t>(M) * K * 2) + align256(w8a8::splitk_partial_bytes(M, N, K));
}

w8a8_status w8a8_linear_postscale(const void* X, const void* Wimg, const float* sw, const void* bias, void* Y,
                                  int64_t M, int64_t N, int64_t K, float* sx, int8_t* Xq, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    return run_linear(false, X, Wimg, sw, bias, Y, M, N, K, sx, Xq, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream));
}

size_t w8a8_linear_codes_workspace_size(int64_t M, int64_t N, int64_t K) { return linear_codes_workspace(M, N, K); }

w8a8_status w8a8_linear_postscale_codes(const void* X, const int8_t* Wq, const float* sw, const void* bias, void* Y,
                                        int64_t M, int64_t N, int64_t K, float* sx, int8_t* Xq, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    return run_linear_codes(X, Wq, sw, bias, Y, M, N, K, sx, Xq, workspace, workspace_bytes,
                            static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_linear_blockwise(const void* X, const void* Wimg, const float* sw, const void* bias, void* Y,
                                  int64_t M, int64_t N, int64_t K, float* sx, int8_t* Xq, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    return run_linear(true, X, Wimg, sw, bias, Y, M, N, K, sx, Xq, workspace, workspace_bytes,
                      static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_linear_postscale_gelu_quant(const void* X, const void* Wimg, const float* sw, const void* bias,
                                             void* Gimg, float* sg, int64_t M, int64_t N, int64_t K, float* sx,
                                             int8_t* Xq, void* workspace, size_t workspace_bytes, void* stream) {
    return run_linear_gelu_quant(X, Wimg, sw, bias, Gimg, sg, M, N, K, sx, Xq, workspace, workspace_bytes,
                                 static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_gemm_blockwise_images(const void* Ximg, const float* sx, const void* Wimg, const float* sw,
                                       const void* bias, void* Y, int64_t M, int64_t N, int64_t K, void* stream) {
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, true);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    if (!Ximg || !sx || !Wimg || !sw || !Y) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(Ximg) || !aligned16(sx) || !aligned16(Wimg) || !aligned16(sw) || !aligned16(Y) ||
        (bias && !aligned16(bias)))
        return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    return run_gemm_images(w8a8::kEpiBlockwiseBf16, Ximg, Wimg, sx, sw, bias, Y, M, N, K, nullptr, dev,
                           static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_norm_quant(const void* X, const void* gamma, const void* beta, float eps, w8a8_norm_kind kind,
                            int64_t M, int64_t K, void* Y, int8_t* Xq, void* Ximg, float* sx, void* stream) {
    if (M < 0 || K <= 0) return W8A8_ERR_INVALID_ARG;
    if (kind != W8A8_NORM_RMS && kind != W8A8_NORM_LAYER) return W8A8_ERR_INVALID_ARG;
    if (K % 8 != 0 || K > 16384 || M > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0) return W8A8_OK;
    if (!X || !sx) return W8A8_ERR_INVALID_ARG;
    if (!(eps >= 0.0f)) return W8A8_ERR_INVALID_ARG;  // also rejects NaN
    if (!aligned16(X) || !aligned16(sx) || (gamma && !aligned16(gamma)) || (beta && !aligned16(beta)) ||
        (Y && !aligned16(Y)) || (Xq && !aligned16(Xq)) || (Ximg && !aligned16(Ximg)))
        return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    return from_cuda(w8a8::launch_norm_quant(X, gamma, beta, eps, kind == W8A8_NORM_LAYER ? 1 : 0, M, K, Y, Xq, Ximg,
                                             sx, static_cast<cudaStream_t>(stream)));
}

size_t w8a8_splitk_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    return align256(w8a8::splitk_partial_bytes(M, N, K));
}

w8a8_status w8a8_gemm_postscale_images(const void* Ximg, const float* sx, const void* Wimg, const float* sw,
                                       const void* bias, void* Y, int64_t M, int64_t N, int64_t K, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, false);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    if (!Ximg || !sx || !Wimg || !sw || !Y) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(Ximg) || !aligned16(sx) || !aligned16(Wimg) || !aligned16(sw) || !aligned16(Y) ||
        (bias && !aligned16(bias)))
        return W8A8_ERR_ALIGNMENT;
    const size_t need = w8a8_splitk_workspace_size(M, N, K);
    if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || workspace_bytes < need))
        return W8A8_ERR_WORKSPACE;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    return run_gemm_images(w8a8::kEpiPostscaleBf16, Ximg, Wimg, sx, sw, bias, Y, M, N, K, workspace, dev,
                           static_cast<cudaStream_t>(stream));
}

size_t w8a8_gemm_workspace_size(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return 0;
    const size_t img = image_gemm_need(M, N, K);
    const size_t s8 = w8a8::gemm_takes_int8(w8a8::kEpiPostscaleBf16, M) ? w8a8::s8_workspace_bytes(M, N, K) : 0;
    return img > s8 ? img : s8;
}

w8a8_status w8a8_gemm_postscale(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw,
                                const void* bias, void* Y, int64_t M, int64_t N, int64_t K, void* workspace,
                                size_t workspace_bytes, void* stream) {
    DeviceInfo dev;
    bool none;
    w8a8_status s =
        check_gemm(Xq, sx, Wq, sw, bias, Y, M, N, K, false, true, workspace, workspace_bytes, &dev, &none);
    if (s != W8A8_OK || none) return s;
    return run_gemm(w8a8::kEpiPostscaleBf16, Xq, sx, Wq, sw, bias, Y, M, N, K, workspace, dev,
                    static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_gemm_blockwise(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw,
                                const void* bias, void* Y, int64_t M, int64_t N, int64_t K, void* workspace,
                                size_t workspace_bytes, void* stream) {
    DeviceInfo dev;
    bool none;
    w8a8_status s =
        check_gemm(Xq, sx, Wq, sw, bias, Y, M, N, K, true, true, workspace, workspace_bytes, &dev, &none);
    if (s != W8A8_OK || none) return s;
    return run_gemm(w8a8::kEpiBlockwiseBf16, Xq, sx, Wq, sw, bias, Y, M, N, K, workspace, dev,
                    static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_gemm_postscale_noalloc(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw,
                                        const void* bias, void* Y, int64_t M, int64_t N, int64_t K, void* stream) {
    if (M < 0 || N < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_k(K, false);
    if (s != W8A8_OK) return s;
    if (M > INT32_MAX || N > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0 || N == 0) return W8A8_OK;
    const size_t need = postscale_gemm_need(M, N, K);
    if (need > kNoAllocScratchBytes) {
        set_detail("shape %lld x %lld x %lld needs %zu bytes of scratch; the fixed no-alloc scratch holds %zu",
                   (long long)M, (long long)N, (long long)K, need, kNoAllocScratchBytes);
        return W8A8_ERR_WORKSPACE;
    }
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    void* scratch = nullptr;
    if ((s = noalloc_scratch(&scratch)) != W8A8_OK) return s;
    bool none;
    s = check_gemm(Xq, sx, Wq, sw, bias, Y, M, N, K, false, true, scratch, kNoAllocScratchBytes, &dev, &none);
    if (s != W8A8_OK || none) return s;
    return run_gemm(w8a8::kEpiPostscaleBf16, Xq, sx, Wq, sw, bias, Y, M, N, K, scratch, dev,
                    static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_gemm_postscale_s32(const int8_t* Xq, const int8_t* Wq, int32_t* acc, int64_t M, int64_t N,
                                    int64_t K, void* workspace, size_t workspace_bytes, void* stream) {
    DeviceInfo dev;
    bool none;
    w8a8_status s = check_gemm(Xq, nullptr, Wq, nullptr, nullptr, acc, M, N, K, false, false, workspace,
                               workspace_bytes, &dev, &none);
    if (s != W8A8_OK || none) return s;
    return run_gemm(w8a8::kEpiPostscaleS32, Xq, nullptr, Wq, nullptr, nullptr, acc, M, N, K, workspace, dev,
                    static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_gemm_blockwise_f32(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw,
                                    float* acc, int64_t M, int64_t N, int64_t K, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    DeviceInfo dev;
    bool none;
    w8a8_status s = check_gemm(Xq, sx, Wq, sw, nullptr, acc, M, N, K, true, true, workspace, workspace_bytes,
                               &dev, &none);
    if (s != W8A8_OK || none) return s;
    return run_gemm(w8a8::kEpiBlockwiseF32, Xq, sx, Wq, sw, nullptr, acc, M, N, K, workspace, dev,
                    static_cast<cudaStream_t>(stream));
}

size_t w8a8_attention_workspace_size(void) {
    DeviceInfo dev;
    return current_device(&dev) == W8A8_OK ? w8a8::attention_workspace_bytes(dev.num_sms) : 0;
}

size_t w8a8_attention_workspace_zeroed(void) {
    DeviceInfo dev;
    return current_device(&dev) == W8A8_OK ? w8a8::attention_counter_bytes(dev.num_sms) : 0;
}

w8a8_status w8a8_attention(const void* Q, const void* K, const void* V, void* O, float* lse, const int32_t* cu_q,
                           const int32_t* cu_k, const int32_t* k_lens, w8a8_dtype dtype, int64_t batch, int64_t Tq,
                           int64_t Tk, int64_t Hq, int64_t Hk, int64_t D, int64_t q_token, int64_t q_head,
                           int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, int64_t o_token,
                           int64_t o_head, float scale, int causal, void* workspace, size_t workspace_bytes,
                           void* stream) {
    if (dtype != W8A8_BF16 && dtype != W8A8_FP16) return W8A8_ERR_INVALID_ARG;
    if (batch < 0 || Tq < 0 || Tk < 0 || Hq <= 0 || Hk <= 0 || D <= 0) return W8A8_ERR_INVALID_ARG;
    const double scale_log2 = static_cast<double>(scale) * 1.4426950408889634;  // the kernels' exponentials are 2^x
    if (!(scale > 0.0f) || !(scale_log2 <= 3.4e38)) return W8A8_ERR_INVALID_ARG;  // also rejects NaN
    if (D % 8 != 0 || D > 128 || Hq % Hk != 0 || Hq > 65535 || Tq > kMostRows || Tk > kMostRows ||
        batch > INT32_MAX || Tq * (Hq / Hk) > kMostRows)
        return W8A8_ERR_SHAPE;
    if (batch == 0 || Tq == 0) return W8A8_OK;
    if ((!cu_q && Tq % batch != 0) || (!cu_k && Tk % batch != 0)) return W8A8_ERR_SHAPE;
    if (!Q || !O || (Tk > 0 && (!K || !V))) return W8A8_ERR_INVALID_ARG;
    const int64_t strides[8] = {q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head};
    for (int64_t v : strides)
        if (v <= 0 || v >= (int64_t(1) << 39) || v % 8 != 0) return W8A8_ERR_ALIGNMENT;
    if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O) || !aligned4(lse) || !aligned4(cu_q) ||
        !aligned4(cu_k) || !aligned4(k_lens))
        return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < w8a8::attention_workspace_bytes(dev.num_sms))
        return W8A8_ERR_WORKSPACE;
    w8a8::AttentionArgs a{};
    a.q = Q;
    a.k = K;
    a.v = V;
    a.o = O;
    a.lse = lse;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.k_lens = k_lens;
    a.batch = static_cast<int>(batch);
    a.Tq = static_cast<int>(Tq);
    a.Tk = static_cast<int>(Tk);
    a.Hq = static_cast<int>(Hq);
    a.Hk = static_cast<int>(Hk);
    a.D = static_cast<int>(D);
    a.group = static_cast<int>(Hq / Hk);
    a.q_token = q_token;
    a.q_head = q_head;
    a.k_token = k_token;
    a.k_head = k_head;
    a.v_token = v_token;
    a.v_head = v_head;
    a.o_token = o_token;
    a.o_head = o_head;
    a.scale_log2 = static_cast<float>(scale_log2);
    a.causal = causal != 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    void* enc = encode_fn();
    if (!enc) return W8A8_ERR_CUDA;
    t_detail[0] = 0;
    const auto launch =
        w8a8::attention_splits(a, dev.num_sms) ? w8a8::launch_attention_split : w8a8::launch_attention_prompt;
    const cudaError_t e = launch(a, dtype, dev.num_sms, workspace, enc, st, t_detail, sizeof t_detail);
    if (e == cudaSuccess) return W8A8_OK;
    cudaGetLastError();
    return t_detail[0] ? W8A8_ERR_CUDA : cuda_fail("attention launch", e);
}

}  // extern "C"

namespace {

// Checks shared by the rotary entry points; *none: there is nothing to do.
w8a8_status check_rotary(const w8a8::RotaryArgs& a, w8a8_dtype dtype, w8a8_rotary_layout layout, int64_t D, int64_t rot,
                         bool* none) {
    *none = false;
    if (dtype != W8A8_BF16 && dtype != W8A8_FP16) return W8A8_ERR_INVALID_ARG;
    if (layout != W8A8_ROTARY_HALF && layout != W8A8_ROTARY_INTERLEAVED) return W8A8_ERR_INVALID_ARG;
    if (a.tokens < 0 || a.cache_rows < 0 || a.q.heads < 0 || a.k.heads < 0 || D <= 0 || rot <= 0)
        return W8A8_ERR_INVALID_ARG;
    if (!(fabsf(a.amplitude) <= 3.0e38f)) return W8A8_ERR_INVALID_ARG;
    if (D % 8 != 0 || D > 256 || rot % 16 != 0 || rot > D || a.tokens > INT32_MAX) return W8A8_ERR_SHAPE;
    *none = a.tokens == 0 || (a.q.heads == 0 && a.k.heads == 0);
    if (*none) return W8A8_OK;
    if (!a.positions || !a.freqs) return W8A8_ERR_INVALID_ARG;
    const w8a8::Heads* sides[6] = {&a.q, &a.q_out, &a.k, &a.k_out, &a.v, &a.v_out};
    for (const w8a8::Heads* h : sides) {
        if (h->heads == 0) continue;
        if (!h->ptr) return W8A8_ERR_INVALID_ARG;
        if (h->token < 0 || h->head < 0 || h->token % 8 != 0 || h->head % 8 != 0 || !aligned16(h->ptr))
            return W8A8_ERR_ALIGNMENT;
        // rows of an output that lie on one another
        if ((h == &a.q_out || h == &a.k_out || h == &a.v_out) &&
            ((h->token == 0 && a.tokens > 1) || (h->head == 0 && h->heads > 1)))
            return W8A8_ERR_INVALID_ARG;
    }
    if ((reinterpret_cast<uintptr_t>(a.positions) & 7u) || (reinterpret_cast<uintptr_t>(a.slots) & 7u) ||
        (reinterpret_cast<uintptr_t>(a.freqs) & 7u))
        return W8A8_ERR_ALIGNMENT;
    return W8A8_OK;
}

w8a8_status run_rotary(const w8a8::RotaryArgs& a, w8a8_dtype dtype, w8a8_rotary_layout layout, int64_t D, int64_t rot,
                       cudaStream_t st) {
    bool none;
    w8a8_status s = check_rotary(a, dtype, layout, D, rot, &none);
    if (s != W8A8_OK || none) return s;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    return from_cuda(w8a8::launch_rotary(a, dtype, layout == W8A8_ROTARY_HALF, dev.num_sms, st), "rotary launch");
}

// Checks of what an append has besides, before check_rotary.
w8a8_status check_append(int64_t T, int64_t Hq, int64_t Hk, int64_t cache_rows, int64_t page_size, int64_t kc_page,
                         int64_t vc_page, const int64_t* slots) {
    if (Hq > 65535 || Hk > 65535) return W8A8_ERR_SHAPE;
    if (Hk <= 0 || page_size < 0) return W8A8_ERR_INVALID_ARG;
    if (T > 0 && !slots) return W8A8_ERR_INVALID_ARG;
    if (page_size > INT32_MAX) return W8A8_ERR_SHAPE;
    if (page_size > 0) {
        if (kc_page < 0 || vc_page < 0 || kc_page % 8 != 0 || vc_page % 8 != 0) return W8A8_ERR_ALIGNMENT;
        if ((kc_page == 0 || vc_page == 0) && cache_rows > page_size) return W8A8_ERR_INVALID_ARG;  // on one another
    }
    return W8A8_OK;
}

struct HeadNorms {
    const void* q_gamma;
    int64_t q_gamma_head;
    const void* k_gamma;
    int64_t k_gamma_head;
    float eps;
    w8a8_norm_kind kind;
};

w8a8_status run_norm_rotary(w8a8::NormRotaryArgs& a, const HeadNorms& n, w8a8_dtype dtype, w8a8_rotary_layout layout,
                            int64_t D, int64_t rot, cudaStream_t st) {
    if (n.kind != W8A8_NORM_RMS && n.kind != W8A8_NORM_LAYER) return W8A8_ERR_INVALID_ARG;
    if (!(n.eps >= 0.0f)) return W8A8_ERR_INVALID_ARG;  // also rejects NaN
    if (n.q_gamma_head < 0 || n.k_gamma_head < 0) return W8A8_ERR_INVALID_ARG;
    bool none;
    w8a8_status s = check_rotary(a.r, dtype, layout, D, rot, &none);
    if (s != W8A8_OK || none) return s;
    if (!aligned16(n.q_gamma) || !aligned16(n.k_gamma) || n.q_gamma_head % 8 != 0 || n.k_gamma_head % 8 != 0)
        return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    a.q_norm = {n.q_gamma, n.q_gamma_head};
    a.k_norm = {n.k_gamma, n.k_gamma_head};
    a.eps = n.eps;
    a.layer = n.kind == W8A8_NORM_LAYER;
    return from_cuda(w8a8::launch_norm_rotary(a, dtype, layout == W8A8_ROTARY_HALF, dev.num_sms, st),
                     "head norm launch");
}

w8a8_status check_caches(void* const* caches, const int64_t* strides, int64_t n_caches, int64_t pages,
                         int64_t page_bytes) {
    if (n_caches < 0 || pages < 0 || page_bytes <= 0) return W8A8_ERR_INVALID_ARG;
    if (pages > INT32_MAX || page_bytes > (int64_t(1) << 32)) return W8A8_ERR_SHAPE;
    if (n_caches > 0 && (!caches || !strides)) return W8A8_ERR_INVALID_ARG;
    if (page_bytes % 16 != 0) return W8A8_ERR_ALIGNMENT;
    for (int64_t i = 0; i < n_caches; ++i) {
        if (pages > 0 && !caches[i]) return W8A8_ERR_INVALID_ARG;
        if (!aligned16(caches[i]) || strides[i] % 16 != 0) return W8A8_ERR_ALIGNMENT;
        if (pages > 1 && strides[i] < page_bytes) return W8A8_ERR_INVALID_ARG;  // on one another
    }
    return W8A8_OK;
}

// As many launches as the caches need.  (The later ones of a fork read the sources' rows and
// lengths again, which the first has left alone: no destination is a source.)
template <typename F>
w8a8_status for_caches(void* const* caches, const int64_t* strides, int64_t n_caches, int64_t pages, int64_t page_bytes,
                       F launch) {
    w8a8::PageCaches c{};
    c.pages = static_cast<int>(pages);
    c.page_bytes = page_bytes;
    for (int64_t first = 0; first < n_caches; first += c.count) {
        c.count = static_cast<int>(std::min<int64_t>(n_caches - first, w8a8::PageCaches::kMost));
        for (int i = 0; i < c.count; ++i) {
            c.base[i] = caches[first + i];
            c.stride[i] = strides[first + i];
        }
        const w8a8_status s = from_cuda(launch(c, first == 0), "pages launch");
        if (s != W8A8_OK) return s;
    }
    return W8A8_OK;
}

}  // namespace

extern "C" {

w8a8_status w8a8_rotary(const void* Q, const void* K, void* Q_out, void* K_out, w8a8_dtype dtype, int64_t T,
                        int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t q_token, int64_t q_head,
                        int64_t k_token, int64_t k_head, int64_t qo_token, int64_t qo_head, int64_t ko_token,
                        int64_t ko_head, const int64_t* positions, const double* freqs, float amplitude,
                        w8a8_rotary_layout layout, int inverse, void* stream) {
    if (Hq > 65535 || Hk > 65535) return W8A8_ERR_SHAPE;
    const int hq = static_cast<int>(Hq), hk = static_cast<int>(Hk);
    w8a8::RotaryArgs a{};
    a.q = {Q, q_token, q_head, hq};
    a.q_out = {Q_out, qo_token, qo_head, hq};
    a.k = {K, k_token, k_head, hk};
    a.k_out = {K_out, ko_token, ko_head, hk};
    a.positions = positions;
    a.tokens = T;
    a.freqs = freqs;
    a.dim = static_cast<int>(D);
    a.rot = static_cast<int>(rot);
    a.inverse = inverse != 0;
    a.amplitude = amplitude;
    return run_rotary(a, dtype, layout, D, rot, static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_rotary_append_pages(const void* Q, const void* K, const void* V, void* Q_out, void* K_cache,
                                     void* V_cache, w8a8_dtype dtype, int64_t T, int64_t Hq, int64_t Hk, int64_t D,
                                     int64_t rot, int64_t cache_rows, int64_t page_size, int64_t q_token,
                                     int64_t q_head, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                                     int64_t qo_token, int64_t qo_head, int64_t kc_page, int64_t kc_token,
                                     int64_t kc_head, int64_t vc_page, int64_t vc_token, int64_t vc_head,
                                     const int64_t* positions, const int64_t* slots, const double* freqs,
                                     float amplitude, w8a8_rotary_layout layout, void* stream) {
    w8a8_status s = check_append(T, Hq, Hk, cache_rows, page_size, kc_page, vc_page, slots);
    if (s != W8A8_OK) return s;
    // pages right behind one another are rows, for which there is the faster kernel
    if (page_size > 0 && kc_page % page_size == 0 && kc_page / page_size == kc_token && vc_page % page_size == 0 &&
        vc_page / page_size == vc_token)
        page_size = 0;
    const int hq = static_cast<int>(Hq), hk = static_cast<int>(Hk);
    w8a8::RotaryArgs a{};
    a.q = {Q, q_token, q_head, hq};
    a.q_out = {Q_out, qo_token, qo_head, hq};
    a.k = {K, k_token, k_head, hk};
    a.k_out = {K_cache, kc_token, kc_head, hk};
    a.v = {V, v_token, v_head, hk};
    a.v_out = {V_cache, vc_token, vc_head, hk};
    a.positions = positions;
    a.slots = slots;
    a.tokens = T;
    a.cache_rows = cache_rows;
    a.page_size = page_size;
    a.k_page = kc_page;
    a.v_page = vc_page;
    a.freqs = freqs;
    a.dim = static_cast<int>(D);
    a.rot = static_cast<int>(rot);
    a.amplitude = amplitude;
    return run_rotary(a, dtype, layout, D, rot, static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_rotary_append(const void* Q, const void* K, const void* V, void* Q_out, void* K_cache, void* V_cache,
                               w8a8_dtype dtype, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t rot,
                               int64_t cache_rows, int64_t q_token, int64_t q_head, int64_t k_token, int64_t k_head,
                               int64_t v_token, int64_t v_head, int64_t qo_token, int64_t qo_head, int64_t kc_token,
                               int64_t kc_head, int64_t vc_token, int64_t vc_head, const int64_t* positions,
                               const int64_t* slots, const double* freqs, float amplitude, w8a8_rotary_layout layout,
                               void* stream) {
    return w8a8_rotary_append_pages(Q, K, V, Q_out, K_cache, V_cache, dtype, T, Hq, Hk, D, rot, cache_rows, 0, q_token,
                                    q_head, k_token, k_head, v_token, v_head, qo_token, qo_head, 0, kc_token, kc_head,
                                    0, vc_token, vc_head, positions, slots, freqs, amplitude, layout, stream);
}

w8a8_status w8a8_qk_norm_rotary(const void* Q, const void* K, void* Q_out, void* K_out, w8a8_dtype dtype, int64_t T,
                                int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t q_token, int64_t q_head,
                                int64_t k_token, int64_t k_head, int64_t qo_token, int64_t qo_head, int64_t ko_token,
                                int64_t ko_head, const void* q_gamma, int64_t q_gamma_head, const void* k_gamma,
                                int64_t k_gamma_head, float eps, w8a8_norm_kind kind, const int64_t* positions,
                                const double* freqs, float amplitude, w8a8_rotary_layout layout, void* stream) {
    if (Hq > 65535 || Hk > 65535) return W8A8_ERR_SHAPE;
    const int hq = static_cast<int>(Hq), hk = static_cast<int>(Hk);
    w8a8::NormRotaryArgs a{};
    a.r.q = {Q, q_token, q_head, hq};
    a.r.q_out = {Q_out, qo_token, qo_head, hq};
    a.r.k = {K, k_token, k_head, hk};
    a.r.k_out = {K_out, ko_token, ko_head, hk};
    a.r.positions = positions;
    a.r.tokens = T;
    a.r.freqs = freqs;
    a.r.dim = static_cast<int>(D);
    a.r.rot = static_cast<int>(rot);
    a.r.amplitude = amplitude;
    const HeadNorms n = {q_gamma, q_gamma_head, k_gamma, k_gamma_head, eps, kind};
    return run_norm_rotary(a, n, dtype, layout, D, rot, static_cast<cudaStream_t>(stream));
}

w8a8_status w8a8_qk_norm_rotary_append(
    const void* Q, const void* K, const void* V, void* Q_out, void* K_cache, void* V_cache, w8a8_dtype dtype, int64_t T,
    int64_t Hq, int64_t Hk, int64_t D, int64_t rot, int64_t cache_rows, int64_t page_size, int64_t q_token,
    int64_t q_head, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, int64_t qo_token, int64_t qo_head,
    int64_t kc_page, int64_t kc_token, int64_t kc_head, int64_t vc_page, int64_t vc_token, int64_t vc_head,
    const void* q_gamma, int64_t q_gamma_head, const void* k_gamma, int64_t k_gamma_head, float eps, w8a8_norm_kind kind,
    const int64_t* positions, const int64_t* slots, const double* freqs, float amplitude, w8a8_rotary_layout layout,
    void* stream) {
    w8a8_status s = check_append(T, Hq, Hk, cache_rows, page_size, kc_page, vc_page, slots);
    if (s != W8A8_OK) return s;
    const int hq = static_cast<int>(Hq), hk = static_cast<int>(Hk);
    w8a8::NormRotaryArgs a{};
    a.r.q = {Q, q_token, q_head, hq};
    a.r.q_out = {Q_out, qo_token, qo_head, hq};
    a.r.k = {K, k_token, k_head, hk};
    a.r.k_out = {K_cache, kc_token, kc_head, hk};
    a.r.v = {V, v_token, v_head, hk};
    a.r.v_out = {V_cache, vc_token, vc_head, hk};
    a.r.positions = positions;
    a.r.slots = slots;
    a.r.tokens = T;
    a.r.cache_rows = cache_rows;
    a.r.freqs = freqs;
    a.r.dim = static_cast<int>(D);
    a.r.rot = static_cast<int>(rot);
    a.r.amplitude = amplitude;
    a.r.page_size = page_size;
    a.r.k_page = kc_page;
    a.r.v_page = vc_page;
    const HeadNorms n = {q_gamma, q_gamma_head, k_gamma, k_gamma_head, eps, kind};
    return run_norm_rotary(a, n, dtype, layout, D, rot, static_cast<cudaStream_t>(stream));
}

size_t w8a8_paged_attention_workspace_size(void) {
    DeviceInfo dev;
    return current_device(&dev) == W8A8_OK ? w8a8::paged_attention_workspace_bytes(dev.num_sms) : 0;
}

w8a8_status w8a8_paged_attention(
    const void* Q, const void* K_pages, const void* V_pages, void* O, float* lse, const int32_t* cu_q,
    const int32_t* page_table, const int32_t* k_lens, w8a8_dtype dtype, int64_t batch, int64_t Tq, int64_t max_queries,
    int64_t pages, int64_t page_size, int64_t max_pages, int64_t table_stride, int64_t Hq, int64_t Hk, int64_t D,
    int64_t q_token, int64_t q_head, int64_t k_page, int64_t k_token, int64_t k_head, int64_t v_page, int64_t v_token,
    int64_t v_head, int64_t o_token, int64_t o_head, float scale, int causal, void* workspace, size_t workspace_bytes,
    void* stream) {
    if (dtype != W8A8_BF16 && dtype != W8A8_FP16) return W8A8_ERR_INVALID_ARG;
    if (batch < 0 || Tq < 0 || max_queries < 0 || pages < 0 || page_size <= 0 || max_pages < 0 || table_stride < 0 ||
        Hq <= 0 || Hk <= 0 || D <= 0)
        return W8A8_ERR_INVALID_ARG;
    const double scale_log2 = static_cast<double>(scale) * 1.4426950408889634;  // the kernels' exponentials are 2^x
    if (!(scale > 0.0f) || !(scale_log2 <= 3.4e38)) return W8A8_ERR_INVALID_ARG;  // also rejects NaN
    if (D % 8 != 0 || D > 128 || Hq % Hk != 0 || Hq > 65535 || Tq > kMostRows || batch > INT32_MAX ||
        Tq * (Hq / Hk) > kMostRows)
        return W8A8_ERR_SHAPE;
    if (page_size % 8 != 0 || page_size > (1 << 20) || pages >= INT32_MAX || max_pages > kMostRows / page_size ||
        table_stride > INT32_MAX)
        return W8A8_ERR_SHAPE;
    if (batch == 0 || Tq == 0) return W8A8_OK;
    if (!cu_q && Tq % batch != 0) return W8A8_ERR_SHAPE;
    if (!Q || !O || !k_lens || (max_pages > 0 && !page_table) || (pages > 0 && (!K_pages || !V_pages)))
        return W8A8_ERR_INVALID_ARG;
    const int64_t strides[10] = {q_token, q_head, k_page, k_token, k_head, v_page, v_token, v_head, o_token, o_head};
    for (int64_t v : strides)
        if (v <= 0 || v >= (int64_t(1) << 39) || v % 8 != 0) return W8A8_ERR_ALIGNMENT;
    if (!aligned16(Q) || !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(O) || !aligned4(lse) ||
        !aligned4(cu_q) || !aligned4(page_table) || !aligned4(k_lens))
        return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < w8a8::paged_attention_workspace_bytes(dev.num_sms))
        return W8A8_ERR_WORKSPACE;
    w8a8::AttentionArgs a{};
    a.q = Q;
    a.k = K_pages;
    a.v = V_pages;
    a.o = O;
    a.lse = lse;
    a.cu_q = cu_q;
    a.k_lens = k_lens;
    a.page_table = page_table;
    a.table_stride = table_stride;
    a.k_page = k_page;
    a.v_page = v_page;
    a.pages = static_cast<int>(pages);
    a.page_size = static_cast<int>(page_size);
    a.max_pages = pages > 0 ? static_cast<int>(max_pages) : 0;  // a cache of no pages has no keys
    a.batch = static_cast<int>(batch);
    a.Tq = static_cast<int>(Tq);
    a.Hq = static_cast<int>(Hq);
    a.Hk = static_cast<int>(Hk);
    a.D = static_cast<int>(D);
    a.group = static_cast<int>(Hq / Hk);
    a.q_token = q_token;
    a.q_head = q_head;
    a.k_token = k_token;
    a.k_head = k_head;
    a.v_token = v_token;
    a.v_head = v_head;
    a.o_token = o_token;
    a.o_head = o_head;
    a.scale_log2 = static_cast<float>(scale_log2);
    a.causal = causal != 0;
    // Which kernel serves the call.  As many rows as sequences, without a word about them,
    // are single tokens, or a chunk in a batch padded with idle sequences.  Taken for single
    // tokens, a chunk has its keys read again for every 16 packed rows, and taken for a
    // chunk, single tokens pay for 128 rows each.  Few rows lose little by the first and
    // much by the second (us, kernel of few queries against that of many, 32 heads on 8 x
    // 128: a chunk of 16 over 2000 keys 15 against 22, over 33000 88 against 38; 16 single
    // tokens over up to 300 keys 9 against 19, up to 30000 159 against 167), many rows the
    // other way round (512 tokens over 33280 keys 1426 against 195, 200 over 2000 53 against
    // 30; 48 single ones over up to 8192 130 against 141, 256 up to 1000 104 against 140).
    int64_t most = cu_q ? Tq : Tq / batch;
    if (max_queries > 0)
        most = std::min(max_queries, most);
    else if (cu_q && Tq == batch && Tq * (Hq / Hk) <= 64)
        most = 1;
    void* enc = encode_fn();
    if (!enc) return W8A8_ERR_CUDA;
    t_detail[0] = 0;
    const cudaError_t e = w8a8::launch_paged_attention(a, static_cast<int>(most), dtype, dev.num_sms, workspace, enc,
                                                       static_cast<cudaStream_t>(stream), t_detail, sizeof t_detail);
    if (e == cudaSuccess) return W8A8_OK;
    cudaGetLastError();
    return t_detail[0] ? W8A8_ERR_CUDA : cuda_fail("paged attention launch", e);
}

w8a8_status w8a8_copy_pages(void* const* caches, const int64_t* strides, int64_t n_caches, int64_t pages,
                            int64_t page_bytes, const int32_t* src, const int32_t* dst, int64_t n, void* stream) {
    if (n < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_caches(caches, strides, n_caches, pages, page_bytes);
    if (s != W8A8_OK) return s;
    if (n == 0 || n_caches == 0 || pages == 0) return W8A8_OK;
    if (!src || !dst) return W8A8_ERR_INVALID_ARG;
    if (!aligned4(src) || !aligned4(dst)) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    return for_caches(caches, strides, n_caches, pages, page_bytes, [&](const w8a8::PageCaches& c, bool) {
        return w8a8::launch_copy_pages(c, src, dst, n, static_cast<cudaStream_t>(stream));
    });
}

w8a8_status w8a8_fork_sequences(void* const* caches, const int64_t* strides, int64_t n_caches, int64_t pages,
                                int64_t page_bytes, int64_t page_size, int32_t* page_table, int64_t rows,
                                int64_t max_pages, int64_t table_stride, int32_t* k_lens, const int32_t* src,
                                const int32_t* dst, const int32_t* new_pages, int64_t n, void* stream) {
    if (n < 0 || rows < 0 || max_pages < 0 || page_size <= 0 || table_stride < 0) return W8A8_ERR_INVALID_ARG;
    w8a8_status s = check_caches(caches, strides, n_caches, pages, page_bytes);
    if (s != W8A8_OK) return s;
    if (rows > INT32_MAX || page_size > INT32_MAX || max_pages > INT32_MAX / page_size || table_stride > INT32_MAX)
        return W8A8_ERR_SHAPE;
    if (n == 0 || n_caches == 0 || pages == 0 || rows == 0) return W8A8_OK;
    if (!k_lens || !src || !dst || !new_pages || (max_pages > 0 && !page_table)) return W8A8_ERR_INVALID_ARG;
    if (table_stride < max_pages && rows > 1) return W8A8_ERR_INVALID_ARG;
    if (!aligned4(page_table) || !aligned4(k_lens) || !aligned4(src) || !aligned4(dst) || !aligned4(new_pages))
        return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    if ((s = current_device(&dev)) != W8A8_OK) return s;
    w8a8::ForkArgs f{};
    f.table = page_table;
    f.table_stride = table_stride;
    f.k_lens = k_lens;
    f.src = src;
    f.dst = dst;
    f.page = new_pages;
    f.n = n;
    f.rows = static_cast<int>(rows);
    f.max_pages = static_cast<int>(max_pages);
    f.page_size = static_cast<int>(page_size);
    return for_caches(caches, strides, n_caches, pages, page_bytes, [&](const w8a8::PageCaches& c, bool first) {
        f.tables = first;
        return w8a8::launch_fork_sequences(c, f, static_cast<cudaStream_t>(stream));
    });
}

w8a8_status w8a8_residual_norm_quant(const void* X, const void* B, void* H, w8a8_dtype x_dtype,
                                     const void* branch_gamma, const void* gamma, const void* beta, const void* gate,
                                     const void* mod_scale, const void* mod_shift, int64_t mod_stride,
                                     int64_t rows_per_group, float alpha, float eps, w8a8_norm_kind kind, int64_t M,
                                     int64_t K, void* Y, int8_t* Xq, void* Ximg, float* sx, void* stream) {
    if (x_dtype != W8A8_BF16 && x_dtype != W8A8_FP32) return W8A8_ERR_INVALID_ARG;
    if (kind != W8A8_NORM_RMS && kind != W8A8_NORM_LAYER) return W8A8_ERR_INVALID_ARG;
    if (M < 0 || K <= 0 || rows_per_group < 0 || mod_stride < 0) return W8A8_ERR_INVALID_ARG;
    if (!(eps >= 0.0f) || !(fabsf(alpha) <= 3.0e38f)) return W8A8_ERR_INVALID_ARG;  // also rejects NaN
    if (K % 8 != 0 || K > 16384 || M > INT32_MAX) return W8A8_ERR_SHAPE;
    if (M == 0) return W8A8_OK;
    if (!X || !B || !H || ((Xq || Ximg) && !sx) || (sx && !Xq && !Ximg)) return W8A8_ERR_INVALID_ARG;
    const void* vectors[13] = {X, B, H, branch_gamma, gamma, beta, gate, mod_scale, mod_shift, Y, Xq, Ximg, sx};
    for (const void* v : vectors)
        if (!aligned16(v)) return W8A8_ERR_ALIGNMENT;
    if (mod_stride % 8 != 0) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    w8a8::ResidualNormArgs a{};
    a.X = X;
    a.B = B;
    a.H = H;
    a.branch_gamma = branch_gamma;
    a.gamma = gamma;
    a.beta = beta;
    a.gate = gate;
    a.mod_scale = mod_scale;
    a.mod_shift = mod_shift;
    a.mod_stride = mod_stride;
    a.rows_per_group = rows_per_group;
    a.M = M;
    a.K = K;
    a.alpha = alpha;
    a.eps = eps;
    a.layer = kind == W8A8_NORM_LAYER;
    a.Y = Y;
    a.Xq = Xq;
    a.Ximg = Ximg;
    a.sx = sx;
    return from_cuda(w8a8::launch_residual_norm(a, x_dtype == W8A8_FP32, dev.num_sms, static_cast<cudaStream_t>(stream)),
                     "residual norm launch");
}

w8a8_status w8a8_gelu_bf16(const void* Y, int64_t n, void* G, void* stream) {
    if (n < 0) return W8A8_ERR_INVALID_ARG;
    if (n % 8 != 0) return W8A8_ERR_SHAPE;
    if (n == 0) return W8A8_OK;
    if (!Y || !G) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(Y) || !aligned16(G)) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    return from_cuda(w8a8::launch_gelu_bf16(Y, n, G, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

w8a8_status w8a8_get_device_error(int* code) {
    if (!code) return W8A8_ERR_INVALID_ARG;
    *code = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) {
        cudaGetLastError();
        return W8A8_ERR_CUDA;
    }
    cudaError_t (*const readers[])(unsigned int*) = {
        w8a8::gemm_read_device_error,      w8a8::gemm_s8_read_device_error,         w8a8::quant_read_device_error,
        w8a8::attention_read_device_error, w8a8::attention_split_read_device_error, w8a8::residual_norm_read_device_error,
        w8a8::attention_paged_read_device_error};
    unsigned int v = 0;
    if (w8a8::read_device_errors(readers, &v) != cudaSuccess) return W8A8_ERR_CUDA;
    *code = static_cast<int>(v);
    if (v >= w8a8::kDeviceErrorTimeoutBase) return W8A8_ERR_TIMEOUT;
    return v ? W8A8_ERR_CUDA : W8A8_OK;
}

w8a8_status w8a8_probe_wait_timeout(void* stream) {
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    return from_cuda(w8a8::launch_wait_timeout_probe(static_cast<cudaStream_t>(stream)));
}

const char* w8a8_last_error_detail(void) { return t_detail; }

w8a8_status w8a8_set_gemm_timing_events(void* start, void* end) {
    if ((start == nullptr) != (end == nullptr)) return W8A8_ERR_INVALID_ARG;
    t_gemm_start = static_cast<cudaEvent_t>(start);
    t_gemm_end = static_cast<cudaEvent_t>(end);
    return W8A8_OK;
}

w8a8_status w8a8_measure_imma_peak(double* tops, void* stream) {
    if (!tops) return W8A8_ERR_INVALID_ARG;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    return from_cuda(w8a8::measure_imma_peak(tops, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

w8a8_status w8a8_stream_floor(const void* src, int64_t n, void* dst, void* stream) {
    if (n < 0) return W8A8_ERR_INVALID_ARG;
    if (n % 8 != 0) return W8A8_ERR_SHAPE;
    if (n == 0) return W8A8_OK;
    if (!src || !dst) return W8A8_ERR_INVALID_ARG;
    if (!aligned16(src) || !aligned16(dst)) return W8A8_ERR_ALIGNMENT;
    DeviceInfo dev;
    w8a8_status s = current_device(&dev);
    if (s != W8A8_OK) return s;
    return from_cuda(w8a8::launch_stream_floor(src, n, dst, dev.num_sms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

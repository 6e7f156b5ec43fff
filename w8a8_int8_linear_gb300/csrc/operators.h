// Host-side launcher interface between the C ABI (api.cu) and the kernels of the
// operators between the Linears (attention, rotary positions, residual norm).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace w8a8 {

// Element types of the operators that take more than one.
enum ElementType : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

// Attention of packed sequences.  Strides count elements; rows are tokens.
struct AttentionArgs {
    const void *q, *k, *v;  // [Tq, Hq, D], [Tk, Hk, D], [Tk, Hk, D]
    void* o;                // [Tq, Hq, D]
    float* lse;             // [Tq, Hq] or nullptr
    const int *cu_q, *cu_k; // [batch + 1] first rows, or nullptr: equal parts of Tq / Tk
    const int* k_lens;      // [batch] keys in use of each sequence's part, or nullptr: all
    int batch, Tq, Tk, Hq, Hk, D, group;  // group = Hq / Hk
    int64_t q_token, q_head, k_token, k_head, v_token, v_head, o_token, o_head;
    float scale_log2;       // scale * log2(e)
    int causal;
    // filled in by the launchers
    int* counters;
    float* partial;
    int join_rounds;         // of the split kernel's threads over the rows of an item
    int side_heads;
};
size_t attention_workspace_bytes(int num_sms);
// The workspace's counters (its first attention_counter_bytes) are zero
// before the first call; every call leaves them zero.
size_t attention_counter_bytes(int num_sms);
// Two kernels: for few queries per sequence, with the keys split over the CTAs,
// and for many on the tensor cores (attention_splits says which).  `encode_fn` is the
// driver's cuTensorMapEncodeTiled.  On failure a one-line description may be
// written to `detail` (size `n`).
cudaError_t launch_attention_split(const AttentionArgs& a, int dtype, int num_sms, void* workspace, void* encode_fn,
                                   cudaStream_t st, char* detail, size_t n);
bool attention_splits(const AttentionArgs& a, int num_sms);
cudaError_t launch_attention_prompt(const AttentionArgs& a, int dtype, int num_sms, void* workspace, void* encode_fn,
                                    cudaStream_t st, char* detail, size_t n);
// Tensor map of [rows, heads, dim] 16-bit elements (strides in elements) with
// boxes of 64 x box_heads x box_rows, 128-byte swizzled; elements outside are 0.
cudaError_t encode_heads(void* encode_fn, CUtensorMap* map, char name, const void* ptr, int dtype, int rows, int heads,
                         int dim, int64_t token, int64_t head, int box_heads, int box_rows, char* detail, size_t n);
cudaError_t attention_read_device_error(unsigned int* code);
cudaError_t attention_split_read_device_error(unsigned int* code);

// One [rows, heads, dim] side of the rotary kernel; strides count elements.
struct Heads {
    const void* ptr;
    int64_t token, head;
    int heads;
};
struct RotaryArgs {
    Heads q, k, v, q_out, k_out, v_out;  // v.ptr nullptr: no V
    const int64_t* positions;            // [tokens]
    const int64_t* slots;                // [tokens] rows of k_out / v_out, or nullptr: the token's own row
    int64_t tokens, cache_rows;
    const double* freqs;                 // [rot / 2]
    int dim, rot, inverse;
    float amplitude;
};
cudaError_t launch_rotary(const RotaryArgs& a, int dtype, bool half, int num_sms, cudaStream_t st);

// Branch norm, gate, residual, norm, modulation and quantization of [M, K]
// rows; every pointer after B but H may be nullptr.
struct ResidualNormArgs {
    const void *X, *B;  // X, H: bf16 or fp32; B bf16
    void* H;
    const void *branch_gamma, *gamma, *beta;    // bf16 [K]
    const void *gate, *mod_scale, *mod_shift;   // bf16 [groups, K], rows mod_stride apart
    int64_t mod_stride, rows_per_group, M, K;
    float alpha, eps;
    int layer;
    void* Y;
    int8_t* Xq;
    void* Ximg;
    float* sx;
};
cudaError_t launch_residual_norm(const ResidualNormArgs& a, bool f32, int num_sms, cudaStream_t st);
cudaError_t residual_norm_read_device_error(unsigned int* code);

}  // namespace w8a8

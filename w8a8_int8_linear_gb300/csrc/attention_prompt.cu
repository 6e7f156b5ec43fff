// Attention of many queries per sequence, keys in rows: the launch of the kernel in
// attention_prompt.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "attention_prompt.cuh"

namespace w8a8 {

namespace {

template <typename T, int DP>
cudaError_t launch_prompt_typed(const CUtensorMap (&map)[3], const AttentionArgs& a, int grid, cudaStream_t st) {
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(attention_prompt_kernel<T, DP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PromptSmem<DP>::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    attention_prompt_kernel<T, DP, false><<<grid, kThreads, PromptSmem<DP>::kTotal, st>>>(map[0], map[1], map[2], a);
    return cudaGetLastError();
}

// An upper bound on the items of any split of the rows into sequences.
int64_t most_items(const AttentionArgs& a) {
    return (static_cast<int64_t>(a.Tq) / (2 * (kTileRows / a.group)) + a.batch) * a.Hk;
}

}  // namespace

cudaError_t launch_attention_prompt(const AttentionArgs& args, int dtype, int num_sms, void* workspace,
                                    void* encode_fn, cudaStream_t st, char* detail, size_t n) {
    AttentionArgs a = args;
    a.counters = static_cast<int*>(workspace);
    CUtensorMap map[3];
    constexpr int kKeyBox = kKeyTile;
    cudaError_t e = encode_heads(encode_fn, &map[0], 'Q', a.q, dtype, a.Tq, a.Hq, a.D, a.q_token, a.q_head, a.group,
                                 kTileRows / a.group, detail, n);
    if (e == cudaSuccess)
        e = encode_heads(encode_fn, &map[1], 'K', a.k, dtype, a.Tk, a.Hk, a.D, a.k_token, a.k_head, 1, kKeyBox, detail,
                         n);
    if (e == cudaSuccess)
        e = encode_heads(encode_fn, &map[2], 'V', a.v, dtype, a.Tk, a.Hk, a.D, a.v_token, a.v_head, 1, kKeyBox, detail,
                         n);
    if (e != cudaSuccess) return e;
    const int64_t items = 2 * most_items(a);  // taken apart
    const int grid = items < num_sms ? static_cast<int>(items) : num_sms;
    if (dtype == kBf16)
        return a.D <= 64 ? launch_prompt_typed<__nv_bfloat16, 64>(map, a, grid, st)
                         : launch_prompt_typed<__nv_bfloat16, 128>(map, a, grid, st);
    return a.D <= 64 ? launch_prompt_typed<__half, 64>(map, a, grid, st)
                     : launch_prompt_typed<__half, 128>(map, a, grid, st);
}

cudaError_t attention_read_device_error(unsigned int* code) {
    unsigned int v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_device_error, &z, sizeof z);
    *code = v;
    return e;
}

}  // namespace w8a8

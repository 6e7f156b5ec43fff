// Attention of new tokens over a cache in pages.
//
// Sequences with up to 16 packed rows (queries x heads of a group) go to the kernel
// of few queries (attention.cu), which the keys' bytes bound; those with more to
// the tensor cores (attention_prompt.cuh), with the keys of an item cut into
// pieces so that all SMs have the same share whatever the lengths; a third kernel
// joins the pieces, in the order of their keys, row by row:
//   M = max M_i,  l = sum 2^(M_i - M) l_i,  o = sum 2^(M_i - M) o_i / l.
// The lengths stay on the device.  Where the host does not know that one kernel
// serves all, both run, each on its own sequences and the second starting on the
// SMs that the first leaves.
#include <cuda.h>

#include <algorithm>
#include <numeric>

#include "attention_prompt.cuh"

namespace w8a8 {

namespace {

constexpr int kFewRows = 16;

// One thread per row and 16 columns of a CTA's item.
template <typename T, int DP>
__global__ void __launch_bounds__(kTileRows) join_kernel(const AttentionArgs p) {
    grid_dependency_wait();
    const Join it = static_cast<const Join*>(p.joins)[blockIdx.x];
    if (it.last < 0) return;
    constexpr int kQuads = 4, kParts = DP / (4 * kQuads);
    const int t = blockIdx.y / kParts, quad = blockIdx.y % kParts * kQuads, row = threadIdx.x;
    const int tile_tokens = kTileRows / p.group, token = it.token0 + t * tile_tokens + row / p.group;
    if (t >= it.tiles || row >= tile_tokens * p.group || token >= it.n) return;
    const int side = blockIdx.x % p.side_heads, first = blockIdx.x / p.side_heads;
    // the first piece is in its CTA's slot 1, the others in slot 0
    const auto part = [&](int x) {
        const int64_t slot = 2 * (static_cast<int64_t>(x) * p.side_heads + side) + (x == first);
        return p.partial + (2 * slot + t) * kTilePart<DP>;
    };
    float top = -INFINITY, l = 0.0f;
    float4 o[kQuads];
#pragma unroll
    for (int i = 0; i < kQuads; ++i) o[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const auto weight = [](float m, float to) { return m == to ? 1.0f : exp2_approx(m - to); };
#pragma unroll 2
    for (int x = first; x <= it.last; ++x) {
        const float* src = part(x);
        const float m = __ldcg(src + row), l1 = __ldcg(src + kTileRows + row);
        float4 v[kQuads];
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            v[i] = __ldcg(reinterpret_cast<const float4*>(src + 2 * kTileRows) + (quad + i) * kTileRows + row);
        const float to = fmaxf(top, m), f0 = weight(top, to), f1 = weight(m, to);
        top = to;
        l = l * f0 + l1 * f1;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
            o[i] = make_float4(o[i].x * f0 + v[i].x * f1, o[i].y * f0 + v[i].y * f1, o[i].z * f0 + v[i].z * f1,
                               o[i].w * f0 + v[i].w * f1);
    }
    const bool sees = !p.causal || token + it.m - it.n >= 0;  // (a joined item has keys)
    const float inv = sees ? __frcp_rn(l) : 0.0f;
    const int head = it.hk * p.group + row % p.group;
    T* to = static_cast<T*>(p.o) + static_cast<int64_t>(it.q0 + token) * p.o_token + static_cast<int64_t>(head) * p.o_head;
#pragma unroll
    for (int i = 0; i < kQuads; i += 2) {
        const int col = 4 * (quad + i);
        if (col >= p.D) break;
        *reinterpret_cast<uint4*>(to + col) =
            sees ? make_uint4(Pair16<T>::pack(o[i].x * inv, o[i].y * inv), Pair16<T>::pack(o[i].z * inv, o[i].w * inv),
                              Pair16<T>::pack(o[i + 1].x * inv, o[i + 1].y * inv),
                              Pair16<T>::pack(o[i + 1].z * inv, o[i + 1].w * inv))
                 : make_uint4(0, 0, 0, 0);
    }
    if (p.lse && blockIdx.y % kParts == 0)
        p.lse[static_cast<int64_t>(it.q0 + token) * p.Hq + head] =
            sees ? (log2f(l) + (top == -INFINITY ? 0.0f : top - kShift<T>)) * kLn2 : -INFINITY;
}

// After the kernel before it in the stream has started everywhere.
template <typename... P, typename... A>
cudaError_t launch_beside(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, bool beside,
                          const A&... args) {
    cudaLaunchAttribute attribute{};
    attribute.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attribute.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = grid;
    config.blockDim = dim3(threads);
    config.dynamicSmemBytes = smem;
    config.stream = st;
    config.attrs = &attribute;
    config.numAttrs = beside;
    return cudaLaunchKernelEx(&config, kernel, args...);
}

template <typename T, int DP>
cudaError_t launch_pieces(const CUtensorMap (&map)[3], const AttentionArgs& a, int num_sms, bool beside, cudaStream_t st) {
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(attention_prompt_kernel<T, DP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PromptSmem<DP>::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    const unsigned ctas = num_sms / a.side_heads * a.side_heads;
    e = launch_beside(attention_prompt_kernel<T, DP, true>, dim3(ctas), kThreads, PromptSmem<DP>::kTotal, st, beside,
                      map[0], map[1], map[2], a);
    if (e != cudaSuccess) return e;
    return launch_beside(join_kernel<T, DP>, dim3(ctas, 2 * DP / 16), kTileRows, 0, st, true, a);
}

size_t joins_bytes(int num_sms) { return (sizeof(Join) * num_sms + 255) / 256 * 256; }

}  // namespace

// The few queries' workspace, what there is to join, and two pieces a CTA.
size_t paged_attention_workspace_bytes(int num_sms) {
    return attention_workspace_bytes(num_sms) + joins_bytes(num_sms) +
           static_cast<size_t>(num_sms) * 2 * 2 * kTilePart<128> * 4;
}

cudaError_t launch_paged_attention(const AttentionArgs& args, int max_queries, int dtype, int num_sms, void* workspace,
                                   void* encode_fn, cudaStream_t st, char* detail, size_t n) {
    AttentionArgs a = args;
    const int rows = max_queries * a.group;
    a.few_rows = 0;
    a.most_rows = 0x7FFFFFFF;
    a.expected_rows = rows;
    // groups of more heads than a tile has rows, and caches without keys, have only the first kernel
    if (rows <= kFewRows || a.group > kTileRows || a.max_pages == 0)
        return launch_attention_split(a, dtype, num_sms, workspace, encode_fn, st, detail, n);
    const bool both = a.cu_q != nullptr;
    if (both) {
        a.most_rows = a.expected_rows = kFewRows;
        const cudaError_t e = launch_attention_split(a, dtype, num_sms, workspace, encode_fn, st, detail, n);
        if (e != cudaSuccess) return e;
        a.few_rows = kFewRows;
        a.most_rows = 0x7FFFFFFF;
    }
    uint8_t* at = static_cast<uint8_t*>(workspace) + attention_workspace_bytes(num_sms);
    a.joins = at;
    a.partial = reinterpret_cast<float*>(at + joins_bytes(num_sms));
    a.side_heads = side_heads(a.Hk);
    a.box = std::gcd(a.page_size, kKeyTile);
    CUtensorMap map[3];
    cudaError_t e = encode_heads(encode_fn, &map[0], 'Q', a.q, dtype, a.Tq, a.Hq, a.D, a.q_token, a.q_head, a.group,
                                 kTileRows / a.group, detail, n);
    if (e == cudaSuccess)
        e = encode_pages(encode_fn, &map[1], 'K', a.k, dtype, a.pages, a.page_size, a.Hk, a.D, a.k_page, a.k_token,
                         a.k_head, a.box, detail, n);
    if (e == cudaSuccess)
        e = encode_pages(encode_fn, &map[2], 'V', a.v, dtype, a.pages, a.page_size, a.Hk, a.D, a.v_page, a.v_token,
                         a.v_head, a.box, detail, n);
    if (e != cudaSuccess) return e;
    if (dtype == kBf16)
        return a.D <= 64 ? launch_pieces<__nv_bfloat16, 64>(map, a, num_sms, both, st)
                         : launch_pieces<__nv_bfloat16, 128>(map, a, num_sms, both, st);
    return a.D <= 64 ? launch_pieces<__half, 64>(map, a, num_sms, both, st)
                     : launch_pieces<__half, 128>(map, a, num_sms, both, st);
}

cudaError_t attention_paged_read_device_error(unsigned int* code) {
    unsigned int v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_device_error, &z, sizeof z);
    *code = v;
    return e;
}

}  // namespace w8a8

// Attention of new tokens over a cache in pages.
//
// Where no sequence has more than 16 packed rows (queries x heads of a group), the
// kernel of few queries (attention.cu) serves the call: the keys' bytes bound it.
// Otherwise the tensor cores do (attention_prompt.cuh), with the keys of an item cut
// into pieces so that all SMs have the same share whatever the lengths, and sequences
// of few and of many queries run beside each other; a second kernel joins the
// pieces, in the order of their keys, row by row:
//   M = max M_i,  l = sum 2^(M_i - M) l_i,  o = sum 2^(M_i - M) o_i / l.
// The lengths stay on the device.
#include <cuda.h>

#include <algorithm>
#include <numeric>

#include "attention_prompt.cuh"

namespace w8a8 {

namespace {

constexpr int kFewRows = 16;

constexpr int kJoinThreads = 128;
constexpr int kJoinParts = 8;  // blocks of a seat

// Rows row, row + step, ... below `end` of an item, kRows of them and kPieces pieces on
// their way at once; DP / 4 lanes to a row, this one's columns 4 lane, ... .
template <typename T, int DP, int kRows, int kPieces>
__device__ __forceinline__ void join_rows(const AttentionArgs& p, const Join& it, int side, int row, int end, int step,
                                          int lane) {
    const auto weight = [](float m, float to) { return m == to ? 1.0f : exp2_approx(m - to); };
    for (; row < end; row += kRows * step) {
        float top[kRows], l[kRows];
        float4 o[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            top[r] = -INFINITY;
            l[r] = 0.0f;
            o[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll 1
        for (int x0 = it.first; x0 <= it.last; x0 += kPieces) {
            float2 stats[kPieces][kRows];
            float4 v[kPieces][kRows];
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                // the first piece is in its CTA's slot 1, the others in slot 0
                const int64_t slot = 2 * (static_cast<int64_t>(x0 + i) * p.side_heads + side) + (x0 + i == it.first);
                const float* src = p.partial + 2 * slot * kTilePart<DP>;
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int at = row + r * step, t = at / kTileRows, in_tile = at % kTileRows;
                    stats[i][r] = make_float2(-INFINITY, 0.0f);
                    v[i][r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (x0 + i > it.last || at >= end) continue;
                    const float* of_tile = src + t * kTilePart<DP>;
                    stats[i][r] = __ldcg(reinterpret_cast<const float2*>(of_tile) + in_tile);
                    v[i][r] = __ldcg(reinterpret_cast<const float4*>(of_tile + 2 * kTileRows + in_tile * DP) + lane);
                }
            }
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                float to = top[r];
#pragma unroll
                for (int i = 0; i < kPieces; ++i) to = fmaxf(to, stats[i][r].x);
                const float f = weight(top[r], to);
                top[r] = to;
                l[r] *= f;
                o[r] = make_float4(o[r].x * f, o[r].y * f, o[r].z * f, o[r].w * f);
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const float w = weight(stats[i][r].x, to);
                    const float4 u = v[i][r];
                    l[r] += stats[i][r].y * w;
                    o[r] = make_float4(o[r].x + u.x * w, o[r].y + u.y * w, o[r].z + u.z * w, o[r].w + u.w * w);
                }
            }
        }
        const int tile_tokens = kTileRows / p.group;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const int at = row + r * step, in_tile = at % kTileRows;
            const int token = it.token0 + at / kTileRows * tile_tokens + in_tile / p.group;
            if (at >= end || in_tile >= tile_tokens * p.group || token >= it.n) continue;
            const int head = it.hk * p.group + in_tile % p.group;
            const bool sees = !p.causal || token + it.m - it.n >= 0;  // (a joined item has keys)
            const float inv = sees ? __frcp_rn(l[r]) : 0.0f;
            if (4 * lane < p.D)
                *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + static_cast<int64_t>(it.q0 + token) * p.o_token +
                                          static_cast<int64_t>(head) * p.o_head + 4 * lane) =
                    sees ? make_uint2(Pair16<T>::pack(o[r].x * inv, o[r].y * inv),
                                      Pair16<T>::pack(o[r].z * inv, o[r].w * inv))
                         : make_uint2(0, 0);
            if (p.lse && lane == 0)
                p.lse[static_cast<int64_t>(it.q0 + token) * p.Hq + head] =
                    sees ? (log2f(l[r]) + (top[r] == -INFINITY ? 0.0f : top[r] - kShift<T>)) * kLn2 : -INFINITY;
        }
    }
}

// The pieces of an item share its join: its rows are dealt out over the blocks of
// their seats, so that every block reads the same bytes however many pieces an item has.
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads, 6) join_kernel(const AttentionArgs p) {
    const int seat = blockIdx.x / kJoinParts, part = blockIdx.x % kJoinParts;
    const int cta = seat >> 1, side = cta % p.side_heads;
    constexpr int kLanes = DP / 4, kAtOnce = kJoinThreads / kLanes;
    const int lane = threadIdx.x % kLanes;
    grid_dependency_wait();
    const Join it = static_cast<const Join*>(p.joins)[seat];
    if (it.last < 0) return;
    const int pieces = it.last - it.first + 1, shares = pieces * kJoinParts;
    const int share = (cta / p.side_heads - it.first) * kJoinParts + part, rows = it.tiles * kTileRows;
    const int first = rows * share / shares + threadIdx.x / kLanes, end = rows * (share + 1) / shares;
    if (pieces <= 2) join_rows<T, DP, 4, 2>(p, it, side, first, end, kAtOnce, lane);
    else if (pieces <= 4) join_rows<T, DP, 2, 4>(p, it, side, first, end, kAtOnce, lane);
    else join_rows<T, DP, 1, 8>(p, it, side, first, end, kAtOnce, lane);
}

template <typename T, int DP>
cudaError_t launch_pieces(const CUtensorMap (&map)[3], const AttentionArgs& a, int num_sms, cudaStream_t st) {
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
    attention_prompt_kernel<T, DP, true><<<ctas, kThreads, PromptSmem<DP>::kTotal, st>>>(map[0], map[1], map[2], a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // the join's blocks are in place when the pieces are done
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t config{};
    config.gridDim = dim3(2 * ctas * kJoinParts);
    config.blockDim = dim3(kJoinThreads);
    config.stream = st;
    config.attrs = &early;
    config.numAttrs = 1;
    return cudaLaunchKernelEx(&config, join_kernel<T, DP>, a);
}

size_t joins_bytes(int num_sms) { return (2 * sizeof(Join) * num_sms + 255) / 256 * 256; }

}  // namespace

// The few queries' workspace, what there is to join, and two pieces a CTA.
size_t paged_attention_workspace_bytes(int num_sms) {
    return attention_workspace_bytes(num_sms) + joins_bytes(num_sms) +
           static_cast<size_t>(num_sms) * 2 * 2 * kTilePart<128> * 4;
}

cudaError_t launch_paged_attention(const AttentionArgs& args, int max_queries, int dtype, int num_sms, void* workspace,
                                   void* encode_fn, cudaStream_t st, char* detail, size_t n) {
    AttentionArgs a = args;
    a.expected_rows = max_queries * a.group;
    // groups of more heads than a tile has rows, and caches without keys, have only the first kernel
    if (a.expected_rows <= kFewRows || a.group > kTileRows || a.max_pages == 0)
        return launch_attention_split(a, dtype, num_sms, workspace, encode_fn, st, detail, n);
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
        return a.D <= 64 ? launch_pieces<__nv_bfloat16, 64>(map, a, num_sms, st)
                         : launch_pieces<__nv_bfloat16, 128>(map, a, num_sms, st);
    return a.D <= 64 ? launch_pieces<__half, 64>(map, a, num_sms, st)
                     : launch_pieces<__half, 128>(map, a, num_sms, st);
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

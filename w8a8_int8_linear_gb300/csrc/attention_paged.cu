// Attention of new tokens over a cache in pages.
//
// Where no sequence has more than 16 packed rows (queries x heads of a group; 32, where
// the table has room for few keys), the kernel of few queries (attention.cu) serves the
// call: the keys' bytes bound it.
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

// The pieces of an item share its join: its rows are dealt out over the blocks of
// their seats, so that every block reads the same bytes however many pieces an item
// has.  DP / 4 lanes to a row, four columns each.  The code is kept short: it is
// fetched from DRAM every time, as keys have driven it out of L2, and written out for
// few and many pieces (4 KB more) it took 3 to 5 us longer.
template <typename T, int DP>
__global__ void __launch_bounds__(kJoinThreads, 8) join_kernel(const AttentionArgs p) {
    constexpr int kLanes = DP / 4, kAtOnce = 4;  // pieces on their way
    grid_dependency_wait();
    const int seat = blockIdx.x / kJoinParts, cta = seat >> 1;
    const Join it = static_cast<const Join*>(p.joins)[seat];
    if (it.last < 0) return;
    const int side = cta % p.side_heads, pieces = it.last - it.first + 1, shares = pieces * kJoinParts;
    const int share = (cta / p.side_heads - it.first) * kJoinParts + blockIdx.x % kJoinParts;
    const int rows = it.tiles * kTileRows, end = rows * (share + 1) / shares, lane = threadIdx.x % kLanes;
    const int tile_tokens = kTileRows / p.group;
    // the first piece is in its CTA's slot 1, the others in slot 0
    const int64_t step = static_cast<int64_t>(4 * p.side_heads) * kTilePart<DP>;
    const float* from = p.partial + it.first * step + 4 * side * kTilePart<DP>;
#pragma unroll 1
    for (int row = rows * share / shares + threadIdx.x / kLanes; row < end; row += kJoinThreads / kLanes) {
        const int t = row / kTileRows, r = row % kTileRows, token = it.token0 + t * tile_tokens + r / p.group;
        if (r >= tile_tokens * p.group || token >= it.n) continue;
        const float* src = from + t * kTilePart<DP>;
        float top = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 1
        for (int x0 = 0; x0 < pieces; x0 += kAtOnce, src += kAtOnce * step) {
            float2 stats[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float* part = src + i * step + (x0 + i == 0 ? 2 * kTilePart<DP> : 0);
                stats[i] = make_float2(-INFINITY, 0.0f);
                v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (x0 + i < pieces) {
                    stats[i] = __ldcg(reinterpret_cast<const float2*>(part) + r);
                    v[i] = __ldcg(reinterpret_cast<const float4*>(part + 2 * kTileRows + r * DP) + lane);
                }
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const float to = fmaxf(top, stats[i].x);
                const float f = top == to ? 1.0f : exp2_approx(top - to);
                const float w = stats[i].x == to ? 1.0f : exp2_approx(stats[i].x - to);
                top = to;
                l = l * f + stats[i].y * w;
                o = make_float4(o.x * f + v[i].x * w, o.y * f + v[i].y * w, o.z * f + v[i].z * w, o.w * f + v[i].w * w);
            }
        }
        const bool sees = !p.causal || token - it.n + it.m >= 0;  // (a joined item has keys)
        const float inv = sees ? __frcp_rn(l) : 0.0f;
        const int head = it.hk * p.group + r % p.group;
        const int64_t at = it.q0 + token;
        if (4 * lane < p.D)
            *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + at * p.o_token + head * p.o_head + 4 * lane) =
                sees ? make_uint2(Pair16<T>::pack(o.x * inv, o.y * inv), Pair16<T>::pack(o.z * inv, o.w * inv))
                     : make_uint2(0, 0);
        if (p.lse && lane == 0)
            p.lse[at * p.Hq + head] =
                sees ? (log2f(l) + (top == -INFINITY ? 0.0f : top - kShift<T>)) * kLn2 : -INFINITY;
    }
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
    // Up to 16 rows the kernel of few queries reads each key once for one MMA tile.  With
    // two such tiles it is the better one while the table has room for few keys, as it
    // starts and ends faster (us, 40 heads on 8 x 128, 4 queries each: 4 sequences of 500
    // keys 13.5 against 17.5, 16 of 500 15.6 against 22; 16 of 2000 46 against 38, 4 of
    // 8000 46 against 36).  Groups of more heads than a tile has rows, and caches without
    // keys, have only that kernel.
    const double keys = static_cast<double>(a.batch) * a.Hk * a.max_pages * a.page_size;
    const bool few = a.expected_rows <= kFewRows || (a.expected_rows <= 2 * kFewRows && keys <= 131072);
    if (few || a.group > kTileRows || a.max_pages == 0)
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

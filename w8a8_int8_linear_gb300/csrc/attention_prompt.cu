// Attention of many queries per sequence on the tensor cores (tcgen05):
// O = softmax(scale Q K^T) V per sequence and head, causal or full, heads in
// groups over the KV heads.
//
// An item is two tiles of 128 packed rows of one KV head.  Row r of a tile is
// (query r / G, head r % G of the group), for the 128 / G queries that fit, so
// a group's heads share the keys that pass through shared memory, short
// sequences still fill tiles, and a causal tile spans few positions.  Keys
// stream in tiles of 128.  For tile t and key tile j
//   S = Q_t K_j^T        operands in shared memory, S (128 x 128, binary32) in TMEM
//   P = 2^(scale log2(e) S - M), in the inputs' type, over S's own columns
//   O_t += P V_j         P from TMEM, V_j (keys x D, D contiguous) as the
//                        MN-major operand, O_t in TMEM
//
// CTAs are persistent, one per SM: each takes items (the longest of a sequence
// first) from a counter.  Warps 0-3 and 4-7 are the softmax of tile 0 and 1
// (one thread per row, which also finishes O), warp 8 issues the MMAs, warp 9
// finds items and issues the TMA loads of Q, K and V, warps 10-11 clean V
// (below).  Loads and first products of the next item run while the softmax
// warps finish the present one.
//
// The tiles' steps alternate: step n of an item is (tile n mod T, key tile
// n / T), T = 2, or 1 where the second tile has no rows.  S and P of a step lie
// in one of B buffers in TMEM, in turn, and the MMA thread issues PV of step n
// and then S of step n + B into the same buffer: MMAs of one thread execute in
// order, so S may overwrite P.  O of both tiles takes 2 D of TMEM's 512 columns
// and a buffer 128: B = 2 for D = 128 (while one tile's softmax runs, the other
// tile's two products run) and 3 for D = 64 (a tile's next S is there before
// its softmax ends).
//
// M is any reference near the row's maximum: softmax does not change with
// it.  It moves only when a score exceeds it by more than 2^8 in weight; only
// then is O_t rescaled (by the softmax threads, between products).  Sums and O
// stay binary32; P's rounding to 16 bits is half a step of each weight, as in
// the output.  In fp16 M lies 7 lower, so that weights reach 2^15 and only those
// below 2^-14 (2^-21 of the row's largest at most) lose bits, of 2^-25 (2^-32 of
// it).  The two halves of P go to the second product one after the other.
//
// Bound by the tensor cores: for D = 128 two tiles alternate at 0.95 of their
// rate while key tiles stream (2900 clocks a pair of tiles).  An item costs about
// 4000 clocks besides (the last softmax, the last product, O on its way out, 64 KB
// at the 64 bytes a clock that an SM stores), and so do the causal tiles' unseen
// half and the last wave.  Measured in bursts of 12 calls (2070 MHz): 8192 tokens
// causal, 40 heads on 8 of 128, 435 us, 1580 TFLOP/s (in a longer loop, under the
// power cap, 473 us, 1450); 16384 x 8 heads full 650 us, 1690 TFLOP/s.  For D = 64
// a key tile's products take half as long and its softmax does not: 4096 x 32
// heads full 129 to 136 us, 1010 to 1060 TFLOP/s.
//
// A weight of 0 does not hide a non-finite V (0 * inf = NaN).  In the key tiles
// that some row does not see completely, warps 10-11 therefore replace the
// non-finite values of V by 0 before the product; if one of them belonged to
// the sequence, the rows that do see it get it added at the end.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <type_traits>

#include "attention.cuh"
#include "pair16.cuh"
#include "ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kTileRows = 128;
constexpr int kKeyTile = 128;
constexpr int kThreads = 384;
constexpr int kSoftmaxWarps = 8;
constexpr float kSlack = 8.0f;  // log2 of the weight that moves the reference
template <typename T>
constexpr float kShift = std::is_same<T, __half>::value ? 7.0f : 0.0f;  // log2 of the weight at the reference
constexpr int kChunkBytes = 128 * 128;  // 128 rows of 64 16-bit elements

template <int DP>
struct PromptSmem {
    static constexpr int kChunks = DP / 64;
    static constexpr int kTileBytes = kChunks * kChunkBytes;  // a Q, K or V tile
    static constexpr int kStages = DP == 128 ? 4 : 8;
    static constexpr int kPipe = 2 * kTileBytes;
    static constexpr int kOut = kPipe + kStages * kTileBytes;  // 32 rows of 64 outputs for each softmax warp
    static constexpr int kOutBytes = 32 * 128;
    static constexpr int kBars = kOut + kSoftmaxWarps * kOutBytes;
    static constexpr int kTotal = kBars + 768;
    static constexpr int kBuffers = DP == 128 ? 2 : 3;  // of S and P in TMEM
    static constexpr int kOutputs = 128 * kBuffers;     // TMEM column of tile 0's O
};

// What the warps need of an item.
struct Item {
    int q0, n, k0, m;   // the sequence
    int hk, token0;     // KV head, first query of tile 0
    int tiles;          // tiles with rows: 1 or 2
    int keys;           // key tiles that some row sees
    int edge;           // key tiles from here on are not seen completely by every row
    int bad;            // a non-finite V of the sequence was taken out
    int any;            // 0: no more items
};

struct Bars {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t q_full[2], q_empty[2];
    // S and PV of a tile's own step k complete s_full and pv_done[tile][k mod 4];
    // P of a buffer's round, p_full
    uint64_t s_full[2][4], pv_done[2][4], p_full[3][2];
    // the V tiles to be cleaned: issued (so that the stage's barrier is in this
    // load's phase, not an older one of the same parity) and done; a slot per V
    // in the ring, as the cleaners run up to three tiles ahead of the products
    uint64_t v_issued[4], v_clean[4];
    uint64_t item_full[2], item_empty[2], done;
    uint32_t tmem;
    Item items[2];
};
static_assert(sizeof(Bars) <= 768, "barriers fit their room");

// Shared-memory operand descriptors with the 128-byte swizzle, low words built
// from an address by adding (address >> 4); the high word is the same for all:
// 1024 bytes between groups of 8 rows, descriptor version 1, swizzle type 2.
// K-major (Q and K): rows of 64 elements of D, the leading offset is unused.
// MN-major (V as the second product's B, N = D): 64 elements of D per 128-byte
// row, rows are keys; leading offset from one 64-wide column block to the next.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kDescKMajor = 1u << 16;
constexpr uint32_t kDescMnMajor = static_cast<uint32_t>(kChunkBytes >> 4) << 16;

__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
__device__ __forceinline__ void mma_output(uint32_t d, uint32_t a, uint32_t b_low, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "mov.b64 b, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_low), "r"(kDescHigh), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// A place in the ring of S stages and the parity of its present round.
template <int S>
struct Ring {
    int st = 0, ph = 0;
    __device__ __forceinline__ void next(int n = 1) {
        st += n;
        if (st >= S) {
            st -= S;
            ph ^= 1;
        }
    }
    __device__ __forceinline__ void skip(int n) {
        const int rounds = (st + n) / S;
        st += n - rounds * S;
        ph ^= rounds & 1;
    }
};

// An item's loads come in the order K_0 K_1 V_0 K_2 V_1 ... K_{J-1} V_{J-2}
// V_{J-1}: load i is K or V of key tile load_tile(i).
__device__ __forceinline__ bool load_is_v(int i, int jmax) { return i == 2 * jmax - 1 || (i > 0 && (i & 1) == 0); }
__device__ __forceinline__ int load_tile(int i, int jmax) {
    return i == 2 * jmax - 1 ? jmax - 1 : (i & 1) ? (i + 1) >> 1 : i == 0 ? 0 : (i >> 1) - 1;
}
__device__ __forceinline__ int load_of_v(int j, int jmax) { return j < jmax - 1 ? 2 * j + 2 : 2 * jmax - 1; }

template <typename T>
constexpr uint32_t prompt_idesc(uint32_t n, bool b_mn_major) {
    return (std::is_same<T, __half>::value ? idesc_f16_f32(128, n) : idesc_bf16_f32(128, n)) |
           (b_mn_major ? 1u << 16 : 0u);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The items of a call, by one warp.  They go through the sequences, those with
// the most keys first (up to 32 sequences), each from its last rows (the most
// keys) to its first, KV heads innermost, two tiles an item.  Full attention
// has items of one size: what is left over from whole rounds of CTAs, if its
// tiles fit one round, is taken apart into them (a tile alone takes 0.6 to 0.7
// of an item's time): 16384 queries x 8 heads 717 -> 650 us, 4096 x 32 193 ->
// 180.  Causal items end short, and there this costs 1 to 3%.
struct Items {
    int sequence_of;  // of this lane, in order
    int mine, incl;   // items of this lane's sequence, and of all up to it
    int all;          // pairs of tiles
    int apart, until; // those from `apart` to `until` are taken apart
    int tile_tokens, key_tile;

    // items of sequences b0 .. b0 + 31 (in order for b0 = 0)
    __device__ __forceinline__ void count(const AttentionArgs& p, int b0, int b) {
        const int lane = threadIdx.x & 31;
        mine = b0 + lane < p.batch ? (sequence(p, b).n + 2 * tile_tokens - 1) / (2 * tile_tokens) * p.Hk : 0;
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
    }

    __device__ __forceinline__ void start(const AttentionArgs& p, int tokens, int keys) {
        const int lane = threadIdx.x & 31;
        tile_tokens = tokens;
        key_tile = keys;
        sequence_of = lane;
        if (p.batch > 1 && p.batch <= 32) {
            // place of this lane's sequence among the others, then the sequence of this place
            const int m = lane < p.batch ? sequence(p, lane).m : -1;
            int place = 0;
            for (int i = 0; i < 32; ++i) {
                const int other = __shfl_sync(0xffffffffu, m, i);
                place += other > m || (other == m && i < lane);
            }
            for (int i = 0; i < 32; ++i)
                if (__shfl_sync(0xffffffffu, place, i) == lane) sequence_of = i;
        }
        all = 0;
        for (int b0 = (p.batch - 1) / 32 * 32; b0 >= 0; b0 -= 32) {
            count(p, b0, b0 ? b0 + lane : sequence_of);
            all += __shfl_sync(0xffffffffu, incl, 31);
        }
        const int ctas = gridDim.x, over = all % ctas;
        apart = all - over;
        until = !p.causal && over <= ctas / 2 ? all : apart;
    }

    __device__ __forceinline__ Item find(const AttentionArgs& p, int index) {
        const int lane = threadIdx.x & 31;
        int half = -1;  // both tiles
        if (index >= apart) {
            const int i = index - apart;
            if (i < 2 * (until - apart)) {
                index = apart + i / 2;
                half = i & 1;
            } else {
                index -= until - apart;
            }
        }
        Item it{};
        if (index >= all) return it;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            if (p.batch > 32) count(p, b0, b0 ? b0 + lane : sequence_of);
            const unsigned hit = __ballot_sync(0xffffffffu, incl > index);
            if (hit) {
                const int l = __ffs(hit) - 1;
                const int local = index - __shfl_sync(0xffffffffu, incl - mine, l);
                const int blocks = __shfl_sync(0xffffffffu, mine, l) / p.Hk;
                const Sequence s = sequence(p, b0 ? b0 + l : __shfl_sync(0xffffffffu, sequence_of, l));
                it.any = 1;
                it.q0 = s.q0;
                it.n = s.n;
                it.k0 = s.k0;
                it.m = s.m;
                it.hk = local % p.Hk;
                it.token0 = (blocks - 1 - local / p.Hk) * 2 * tile_tokens + max(half, 0) * tile_tokens;
                it.tiles = half < 0 && it.token0 + tile_tokens < s.n ? 2 : 1;
                const int last = min(it.token0 + it.tiles * tile_tokens, s.n) - 1;
                auto limit = [&](int token) { return p.causal ? clampi(token + s.m - s.n + 1, 0, s.m) : s.m; };
                it.edge = limit(it.token0) / key_tile;
                // (the second tile of an item taken apart may have no rows)
                it.keys = it.token0 <= last ? (limit(last) + key_tile - 1) / key_tile : 0;
                return it;
            }
            index -= __shfl_sync(0xffffffffu, incl, 31);
        }
        return it;
    }
};

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const AttentionArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = PromptSmem<DP>;
    constexpr int S = L::kStages;
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles start at multiples of 1024
        if (threadIdx.x == 0) record_device_error(1);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tile_tokens = kTileRows / p.group;

    if (warp == kSoftmaxWarps) {
        if (lane == 0) {
            for (int i = 0; i < S; ++i) {
                mbar_init(&bars->kv_full[i], 1);
                mbar_init(&bars->kv_empty[i], 1);
            }
            for (int t = 0; t < 2; ++t) {
                mbar_init(&bars->q_full[t], 1);
                mbar_init(&bars->q_empty[t], 1);
                mbar_init(&bars->item_full[t], 1);
                mbar_init(&bars->item_empty[t], kSoftmaxWarps + 3);  // and MMA, 2 cleaners
            }
            for (int i = 0; i < 8; ++i) {
                mbar_init(&bars->s_full[i >> 2][i & 3], 1);
                mbar_init(&bars->pv_done[i >> 2][i & 3], 1);
            }
            for (int i = 0; i < 3; ++i) {
                mbar_init(&bars->p_full[i][0], kSoftmaxWarps / 2);
                mbar_init(&bars->p_full[i][1], kSoftmaxWarps / 2);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&bars->v_issued[i], 1);
                mbar_init(&bars->v_clean[i], 2);
            }
            mbar_init(&bars->done, 1);
            fence_mbarrier_init();
        }
        __syncwarp();
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    const uint32_t pipe = smem_u32(smem) + L::kPipe;

    auto leave_item = [&](int at) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->item_empty[at & 1]);
    };

    if (warp >= kSoftmaxWarps) {
        regs_dec<72>();
        if (warp == kSoftmaxWarps + 1) {
            // ---- items and TMA loads: K_0 Q_0 Q_1 K_1 V_0 ...
            if (elect_one_sync()) {
                tma_prefetch_desc(&tmQ);
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            const uint32_t q_bytes = L::kChunks * tile_tokens * p.group * 128;
            Items items;
            items.start(p, tile_tokens, kKeyTile);
            int index = blockIdx.x, edges = 0;
            int q_ph[2] = {1, 1};  // a fresh barrier lets the first wait through
            Ring<S> r;
            r.ph = 1;
            bool ok = true;
            for (int at = 0; ok; ++at) {
                Item it = items.find(p, index);
                if (!mbar_wait(&bars->item_empty[at & 1], ((at >> 1) & 1) ^ 1, 60)) {
                    it.any = 0;
                    ok = false;
                }
                if (lane == 0) {
                    bars->items[at & 1] = it;
                    mbar_arrive(&bars->item_full[at & 1]);
                }
                if (!it.any) break;
                if (lane == 0) index = atomicAdd(p.counters, 1);
                const int jmax = it.keys;
                for (int i = 0; i < 2 * jmax; ++i) {
                    const int j = load_tile(i, jmax);
                    const bool is_v = load_is_v(i, jmax);
                    ok = mbar_wait(&bars->kv_empty[r.st], r.ph, 61);
                    if (!ok) break;
                    if (elect_one_sync()) {
                        mbar_arrive_expect_tx(&bars->kv_full[r.st], L::kTileBytes);
                        const void* map = is_v ? static_cast<const void*>(&tmV) : static_cast<const void*>(&tmK);
#pragma unroll
                        for (int c = 0; c < L::kChunks; ++c)
                            tma_load_3d(pipe + r.st * L::kTileBytes + c * kChunkBytes, map, &bars->kv_full[r.st],
                                        64 * c, it.hk, it.k0 + j * kKeyTile);
                        if (is_v && j >= it.edge) mbar_arrive(&bars->v_issued[(edges + j - it.edge) & 3]);
                    }
                    r.next();
                    if (i == 0) {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            if (t >= it.tiles) continue;
                            ok = ok && mbar_wait(&bars->q_empty[t], q_ph[t], 62);
                            q_ph[t] ^= 1;
                            if (ok && elect_one_sync()) {
                                mbar_arrive_expect_tx(&bars->q_full[t], q_bytes);
#pragma unroll
                                for (int c = 0; c < L::kChunks; ++c)
                                    tma_load_3d(smem_u32(smem) + t * L::kTileBytes + c * kChunkBytes, &tmQ,
                                                &bars->q_full[t], 64 * c, it.hk * p.group,
                                                it.q0 + it.token0 + t * tile_tokens);
                            }
                        }
                        if (!ok) break;
                    }
                }
                edges += max(0, jmax - it.edge);
                index = static_cast<int>(gridDim.x) + __shfl_sync(0xffffffffu, index, 0);
            }
            // nothing is in flight into this CTA's shared memory when it ends
            // (a stage's last load is complete when its barrier has left that round;
            // a stage never loaded has parity 1 behind it)
            for (int i = 0; i < S; ++i) {
                mbar_wait(&bars->kv_full[r.st], r.ph, 61);
                r.next();
            }
            for (int t = 0; t < 2; ++t) mbar_wait(&bars->q_full[t], q_ph[t], 62);
            // the last CTA to run out of items leaves the counters at zero
            if (lane == 0) {
                __threadfence();
                if (atomicAdd(p.counters + 1, 1) == static_cast<int>(gridDim.x) - 1) {
                    p.counters[0] = 0;
                    p.counters[1] = 0;
                }
            }
        } else if (warp == kSoftmaxWarps) {
            // ---- MMA issuer, one thread throughout (so that the MMAs' operands are uniform)
            if (elect_one_sync()) {
                constexpr int NB = L::kBuffers, kTileLow = L::kTileBytes >> 4;
                const uint32_t q_low = (smem_u32(smem) >> 4) | kDescKMajor, kv_low = pipe >> 4;
                int q_ph = 0, edges = 0, buf = 0, p_ph = 0, own[2] = {0, 0}, pv_own[2] = {0, 0};
                Ring<S> r;  // the item's first load
                bool ok = true;
                // all steps of an item with kT tiles
                auto run = [&](auto tc, int J, int edge) {
                    constexpr int kT = decltype(tc)::value;
                    Ring<S> rk = r, rv = r;  // the next K and V to use
                    rv.next(load_of_v(0, J));
                    auto scores = [&](int t, int j, int to) {
                        const uint32_t a = q_low + t * kTileLow, b = (kv_low + rk.st * kTileLow) | kDescKMajor;
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            const uint32_t off = ((k >> 2) * kChunkBytes + (k & 3) * 32) >> 4;
                            mma_scores(tmem + 128 * to, a + off, b + off, prompt_idesc<T>(kKeyTile, false), k > 0);
                        }
                        mma_commit(&bars->s_full[t][own[t] & 3]);
                        ++own[t];
                        if (j + 1 == J) mma_commit(&bars->q_empty[t]);
                        if (t == kT - 1) {
                            mma_commit(&bars->kv_empty[rk.st]);
                            rk.next(j == 0 ? 1 : 2);
                        }
                    };
#pragma unroll
                    for (int n = 0; n < NB; ++n) {
                        const int t = n % kT, j = n / kT;
                        if (j >= J) break;
                        if (t == 0 && !(ok = mbar_wait(&bars->kv_full[rk.st], rk.ph, 64))) return;
                        if (j == 0 && !(ok = mbar_wait(&bars->q_full[t], (q_ph >> t) & 1, 65))) return;
                        tc_fence_after();
                        const int to = buf + n;
                        scores(t, j, to >= NB ? to - NB : to);
                    }
                    q_ph ^= (1 << kT) - 1;
                    for (int j = 0; j < J; ++j) {
                        if (!(ok = mbar_wait(&bars->kv_full[rv.st], rv.ph, 66))) return;
                        if (j >= edge) {
                            if (!(ok = mbar_wait(&bars->v_clean[edges & 3], (edges >> 2) & 1, 67))) return;
                            ++edges;
                        }
                        const uint32_t v_low = (kv_low + rv.st * kTileLow) | kDescMnMajor;
#pragma unroll
                        for (int t = 0; t < kT; ++t) {
                            // S of step n + NB: (nt, nj)
                            const int nt = (t + NB) % kT, nj = j + (t + NB) / kT;
                            if (nt == 0 && nj < J && !(ok = mbar_wait(&bars->kv_full[rk.st], rk.ph, 68))) return;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                if (!(ok = mbar_wait(&bars->p_full[buf][half], (p_ph >> buf) & 1, 69))) return;
                                tc_fence_after();
#pragma unroll
                                for (int k = 4 * half; k < 4 * half + 4; ++k)
                                    mma_output(tmem + L::kOutputs + t * DP, tmem + 128 * buf + 8 * k,
                                               v_low + k * (2048 >> 4), prompt_idesc<T>(DP, true), j + k > 0);
                            }
                            if (nj < J) scores(nt, nj, buf);
                            mma_commit(&bars->pv_done[t][pv_own[t] & 3]);
                            ++pv_own[t];
                            p_ph ^= 1 << buf;
                            if (++buf == NB) buf = 0;
                        }
                        mma_commit(&bars->kv_empty[rv.st]);
                        rv.next(load_of_v(j + 1, J) - load_of_v(j, J));
                    }
                };
                for (int at = 0; ok; ++at) {
                    if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 63)) break;
                    const volatile Item& it = bars->items[at & 1];
                    const int any = it.any, two = it.tiles > 1, J = it.keys, edge = it.edge;
                    if (!any) break;
                    mbar_arrive(&bars->item_empty[at & 1]);
                    if (J == 0) continue;
                    if (two) run(std::integral_constant<int, 2>{}, J, edge);
                    else run(std::integral_constant<int, 1>{}, J, edge);
                    r.skip(2 * J);
                }
            // every commit has arrived before the CTA ends
            mma_commit(&bars->done);
            mbar_wait(&bars->done, 0, 70);
            }
            __syncwarp();
        } else {
            // ---- V cleaners: key tiles from `edge` on
            const int me = threadIdx.x - 32 * (kSoftmaxWarps + 2);  // 0..63
            int ld = 0, edges = 0;
            bool ok = true;
            for (int at = 0; ok; ++at) {
                if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 71)) break;
                volatile Item& it = bars->items[at & 1];
                if (!it.any) break;
                const int jmax = it.keys;
                for (int j = it.edge; j < jmax && ok; ++j, ++edges) {
                    const int lv = ld + load_of_v(j, jmax);
                    ok = mbar_wait(&bars->v_issued[edges & 3], (edges >> 2) & 1, 72) &&
                         mbar_wait(&bars->kv_full[lv % S], (lv / S) & 1, 73);
                    if (!ok) break;
                    const uint32_t v = pipe + (lv % S) * L::kTileBytes;
                    constexpr int kAtOnce = 8;  // loads in flight: one by one they would bound an item's end
                    static_assert(L::kTileBytes % (16 * 64 * kAtOnce) == 0, "whole rounds");
                    for (int c0 = me; c0 < L::kTileBytes / 16; c0 += 64 * kAtOnce) {
                        uint4 w[kAtOnce];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i)
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                                         : "r"(v + 16 * (c0 + 64 * i)));
                        bool some = false;
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) some |= any_non_finite<T>(w[i]);
                        if (!some) continue;
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            if (!any_non_finite<T>(w[i])) continue;
                            const int c = c0 + 64 * i;
                            constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
                            uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                if ((u[k] & e) == e) u[k] &= 0xFFFF0000u;
                                if (((u[k] >> 16) & e) == e) u[k] &= 0x0000FFFFu;
                            }
                            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(v + 16 * c), "r"(u[0]),
                                         "r"(u[1]), "r"(u[2]), "r"(u[3])
                                         : "memory");
                            const int key = j * kKeyTile + ((c >> 3) & 127);
                            if (key < it.m) it.bad = 1;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->v_clean[edges & 3]);
                }
                ld += 2 * jmax;
                leave_item(at);
            }
        }
    } else {
        // ---- softmax, one thread per row
        regs_inc<208>();
        const int t = warp >> 2, wq = warp & 3;
        const int row = wq * 32 + lane;
        const int row_token = t * tile_tokens + row / p.group, row_head = row % p.group;
        const bool used = row < tile_tokens * p.group;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t to = tmem + lanes + L::kOutputs + t * DP;
        const float c = p.scale_log2;
        const uint64_t c2 = f2_pack(c, c);
        int steps = 0, own = 0;  // steps of both tiles before this item (mod the buffers), of this tile
        bool ok = true;
        for (int at = 0; ok; ++at) {
            if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 74)) break;
            const volatile Item& it = bars->items[at & 1];
            if (!it.any) break;
            int lim, warp_lim;
            {
                const int n = it.n, m = it.m, token = it.token0 + row_token;
                const bool valid = used && t < it.tiles && token < n;
                lim = valid ? (p.causal ? clampi(token + m - n + 1, 0, m) : m) : 0;
                warp_lim = __reduce_min_sync(0xffffffffu, valid ? lim : m);
            }
            const int both = it.tiles, tiles = t < both ? it.keys : 0;
            float ref = -INFINITY;
            auto base_of = [](float r) { return r == -INFINITY ? 0.0f : kShift<T> - r; };
            uint64_t sum2 = f2_pack(0.0f, 0.0f);
            for (int j = 0; j < tiles; ++j, ++own) {
                const int buf = (steps + j * both + t) % L::kBuffers;
                const uint32_t ts = tmem + lanes + 128 * buf;
                ok = mbar_wait(&bars->s_full[t][own & 3], (own >> 2) & 1, 75);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, v[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_wait_ld_regs32(v[i]);
                if (warp_lim < (j + 1) * kKeyTile) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int left = lim - j * kKeyTile - 32 * i;  // columns this row sees
                        if (!__any_sync(0xffffffffu, left < 32)) continue;
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (k >= left) v[i][k] = 0xFF800000u;  // -inf
                    }
                }
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int k = 0; k < 32; k += 2)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        m[i] = max3(m[i], __uint_as_float(v[i][k]), __uint_as_float(v[i][k + 1]));
                const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
                if (j == 0) {
                    ref = top;
                } else {
                    const bool moves = top > ref + kSlack;  // also from -inf
                    if (__any_sync(0xffffffffu, moves)) {
                        const float f = moves ? exp2_approx((kShift<T> - top) - (kShift<T> - ref)) : 1.0f;
                        if (moves) ref = top;
                        sum2 = f2_mul(sum2, f2_pack(f, f));
                        // S of this step says nothing of the product before it
                        ok = mbar_wait(&bars->pv_done[t][(own - 1) & 3], ((own - 1) >> 2) & 1, 77);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int i = 0; i < DP / 16; ++i) {
                            uint32_t o[16];
                            tmem_ld_32x32b_x16(to + 16 * i, o);
                            tmem_wait_ld_regs(o);
#pragma unroll
                            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f);
                            tmem_st_32x32b_x16(to + 16 * i, o);
                        }
                    }
                }
                const float base = base_of(ref);
                const uint64_t base2 = f2_pack(base, base);
                uint64_t part2[2] = {sum2, f2_pack(0.0f, 0.0f)};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float a, b;
                        f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i][k]), __uint_as_float(v[i][k + 1])), c2, base2), a,
                                  b);
                        a = exp2_approx(a);
                        b = exp2_approx(b);
                        part2[(k >> 1) & 1] = f2_add(part2[(k >> 1) & 1], f2_pack(a, b));
                        w[k >> 1] = Pair16<T>::pack(a, b);
                    }
                    tmem_st_32x32b_x16(ts + 16 * i, w);
                    if (i & 1) {  // half of P: its product can start
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->p_full[buf][i >> 1]);
                    }
                }
                sum2 = f2_add(part2[0], part2[1]);
            }

            steps = (steps + both * it.keys) % L::kBuffers;

            // ---- O / sum to memory
            float l0, l1;
            f2_unpack(sum2, l0, l1);
            const float l = l0 + l1;
            const float inv = lim > 0 ? __frcp_rn(l) : 0.0f;
            // where the rows go: through shared memory, so that eight lanes write 128
            // bytes of a row, this lane 16 bytes of rows sub, sub + 4, ...
            const int q0 = it.q0, k0 = it.k0, hk = it.hk, token = it.token0 + row_token, edge = it.edge;
            const bool valid = used && t < it.tiles && token < it.n;
            const int head = hk * p.group + row_head;
            const int sub = lane >> 3, ch = lane & 7;
            const int64_t mine = static_cast<int64_t>(q0 + token) * p.o_token + static_cast<int64_t>(head) * p.o_head;
            const uint32_t valid_rows = __ballot_sync(0xffffffffu, valid) >> sub;
            int64_t to_row[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) to_row[x] = __shfl_sync(0xffffffffu, mine, 4 * x + sub) + 8 * ch;
            if (tiles > 0) ok = ok && mbar_wait(&bars->pv_done[t][(own - 1) & 3], ((own - 1) >> 2) & 1, 76);
            if (!ok) break;
            tc_fence_after();
            const int bad = tiles > 0 ? it.bad : 0;
            leave_item(at);
            const uint32_t stage = smem_u32(smem) + L::kOut + warp * L::kOutBytes;
#pragma unroll 1
            for (int i = 0; i < DP / 64; ++i) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t o[32];
                    if (tiles > 0) {
                        tmem_ld_32x32b_x32(to + 64 * i + 32 * q, o);
                        tmem_wait_ld_regs32(o);
                    }
                    if (bad) {
                        for (int key = edge * kKeyTile; key < lim; ++key) {
                            const T* src = static_cast<const T*>(p.v) + static_cast<int64_t>(k0 + key) * p.v_token +
                                           static_cast<int64_t>(hk) * p.v_head + 64 * i + 32 * q;
#pragma unroll
                            for (int x = 0; x < 32; ++x) {
                                if (64 * i + 32 * q + x >= p.D) continue;
                                const float val = static_cast<float>(src[x]);
                                if (!isfinite(val)) o[x] = __float_as_uint(__uint_as_float(o[x]) + val);
                            }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t w[4];
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            w[x] = lim > 0 ? Pair16<T>::pack(__uint_as_float(o[8 * h + 2 * x]) * inv,
                                                             __uint_as_float(o[8 * h + 2 * x + 1]) * inv)
                                           : 0u;
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         stage + lane * 128 + (((4 * q + h) ^ (lane & 7)) << 4)),
                                     "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                                     : "memory");
                    }
                }
                __syncwarp();
                uint4 w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w[x].x), "=r"(w[x].y), "=r"(w[x].z), "=r"(w[x].w)
                                 : "r"(stage + (4 * x + sub) * 128 + ((ch ^ ((4 * x + sub) & 7)) << 4)));
                if (64 * i + 8 * ch < p.D) {
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (valid_rows >> (4 * x) & 1) *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + to_row[x] + 64 * i) = w[x];
                }
                __syncwarp();
            }
            if (p.lse && valid)
                p.lse[static_cast<int64_t>(q0 + token) * p.Hq + head] =
                    lim > 0 ? (log2f(l) - base_of(ref)) * kLn2 : -INFINITY;
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == kSoftmaxWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int DP>
cudaError_t launch_prompt_typed(const CUtensorMap (&map)[3], const AttentionArgs& a, int grid, cudaStream_t st) {
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(attention_prompt_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PromptSmem<DP>::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    attention_prompt_kernel<T, DP><<<grid, kThreads, PromptSmem<DP>::kTotal, st>>>(map[0], map[1], map[2], a);
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

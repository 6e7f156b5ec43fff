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
// Keys in pages (kPaged, attention_paged.cu) come by boxes of a page, K's and V's from a
// warp each (9 and 10), the cleaning from warp 11; an item is then a piece of its key tiles
// (Pieces), which may begin in their middle, and leaves its reference, sum and output to
// a join where it is not all.  512 tokens of 40 heads on 8 x 128 over 33280 keys: 256 us
// with the join, 67% of the tensor pipe's cycles; 16 x 5 tokens of 28 heads on 4 over 22
// to 7544 keys 36 us, of which 20 at 0.9 of the copy bandwidth.
//
// A weight of 0 does not hide a non-finite V (0 * inf = NaN).  In the key tiles
// that some row does not see completely, warps 10-11 therefore replace the
// non-finite values of V by 0 before the product; if one of them belonged to
// the sequence, the rows that do see it get it added at the end.
#pragma once
#include <cuda.h>

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
    static constexpr int kHanded = kBars + 768;  // reference and sum of 128 rows
    static constexpr int kTotal = kHanded + 1024;
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
    // keys in pages: an item is a piece of the key tiles; `keys` and `edge` count from the
    // first, j0
    int b, j0;
    int slot;           // where its partial result goes; -1: the piece is all there is
    int last_tile;      // of the whole item
    int seen;           // keys of the sequence that every row sees
    int turn;           // the first of its key tiles to be taken, at most `edge`; they go round
    // key tile of step j
    __device__ __forceinline__ static int tile_of(int j, int turn, int keys) {
        return j + turn < keys ? j + turn : j + turn - keys;
    }
};

// What the join of an item's pieces needs of it: a seat for each piece, two a CTA
// (slot 0: the end of an item that an earlier CTA began, or its middle; slot 1: the
// beginning of one that a later CTA goes on with).
struct Join {
    int q0, n, m, hk, token0, tiles;
    int first, last;    // ranges of the first and the last piece; last < 0: no piece
};
// The partial result of a piece, for each of its two tiles: (reference, sum) of the
// 128 rows, then their outputs [128][DP].
template <int DP>
constexpr int kTilePart = kTileRows * (DP + 2);

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
    // a tile alone: the second half's reference, sum and O are there, and have been read
    uint64_t handed[4], taken[4];
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

// The pieces of a call over pages, by one warp.  An item (two tiles of rows of a
// sequence and KV head, or the last one) has as many key tiles as some of its rows
// see.  All items are laid end to end, sequences outermost, then groups of
// `side_heads` KV heads (the CTAs side by side take the same range for each of them),
// then rows, and cut into equal ranges, one per CTA.  A key tile counts a unit for
// each tile of rows, and an item's end kEnds.
struct Pieces {
    static constexpr int kEnds = 6;
    // Items of few key tiles are not cut: a piece's end and the join cost as much (32 heads
    // on 8 x 128: prompts of 300 and 200 tokens 17 us against 23, one of 1000 24 against 32,
    // 8 x 64 tokens over 300 to 800 keys 23 against 28; 40 heads, 100 tokens over 1500 and
    // 100 over 1000 30 against 26).
    static constexpr int kWhole = 8;
    int64_t w, w_end, per, item_start;     // what is left of the range: [w, w_end)
    int b, blocks, groups, hg, block, at;  // at: where w_end is in the item's part of the line
    int tiles, each, line;                 // the item's key tiles, units of one, its part of the line
    Sequence s;
    int pair_tokens, side, range;
    int passed;                            // key tiles of this CTA so far

    __device__ __forceinline__ int limit(const AttentionArgs& p, const Sequence& q, int token) const {
        return p.causal ? clampi(token - q.n + q.m + 1, 0, q.m) : q.m;
    }
    __device__ __forceinline__ int tiles_of(const AttentionArgs& p, const Sequence& q, int i) const {
        return (limit(p, q, min((i + 1) * pair_tokens, q.n) - 1) + kKeyTile - 1) / kKeyTile;
    }
    __device__ __forceinline__ int units_of(const Sequence& q, int i) const {
        return i * pair_tokens + pair_tokens / 2 < q.n ? 2 : 1;
    }
    __device__ __forceinline__ int line_of(const AttentionArgs& p, const Sequence& q, int i) const {
        return max(tiles_of(p, q, i), 1) * units_of(q, i) + kEnds;
    }
    __device__ __forceinline__ int blocks_of(const Sequence& q) const { return (q.n + pair_tokens - 1) / pair_tokens; }
    // this lane's sequence's line, and inclusive over the lanes
    __device__ __forceinline__ void lines(const AttentionArgs& p, int b0, int64_t& mine, int64_t& incl) const {
        const int lane = threadIdx.x & 31;
        mine = 0;
        if (b0 + lane < p.batch) {
            const Sequence q = sequence<true>(p, b0 + lane);
            const int n = blocks_of(q);
            for (int i = 0; i < n; ++i) mine += line_of(p, q, i);
        }
        mine *= groups;
        incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
    }
    __device__ __forceinline__ void item(const AttentionArgs& p) {
        tiles = tiles_of(p, s, block);
        each = units_of(s, block);
        line = max(tiles, 1) * each + kEnds;
    }

    // false: nothing for this CTA
    __device__ __forceinline__ bool start(const AttentionArgs& p, int tile_tokens) {
        const int lane = threadIdx.x & 31;
        pair_tokens = 2 * tile_tokens;
        side = blockIdx.x % p.side_heads;
        range = blockIdx.x / p.side_heads;
        groups = p.Hk / p.side_heads;
        const int ranges = gridDim.x / p.side_heads;
        int64_t mine, incl, total = 0;
        if (p.batch == 1) {  // by all lanes
            const Sequence q = sequence<true>(p, 0);
            const int n = blocks_of(q);
            mine = 0;
            for (int i = lane; i < n; i += 32) mine += line_of(p, q, i);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
            mine *= groups;
            incl = total = mine;
        } else {
            for (int b0 = (p.batch - 1) / 32 * 32; b0 >= 0; b0 -= 32) {
                lines(p, b0, mine, incl);
                total += __shfl_sync(0xffffffffu, incl, 31);
            }
        }
        per = max(static_cast<int64_t>(2 + kEnds), quotient(total + ranges - 1, ranges));
        w = per * range;
        w_end = min(total, w + per);
        passed = 0;
        if (w >= w_end) return false;
        int64_t left = w_end - 1;
        for (int b0 = 0;; b0 += 32) {
            if (b0 > 0) lines(p, b0, mine, incl);
            const unsigned hit = __ballot_sync(0xffffffffu, incl > left);
            if (hit) {
                const int l = __ffs(hit) - 1;
                left -= __shfl_sync(0xffffffffu, incl - mine, l);
                b = b0 + l;
                mine = __shfl_sync(0xffffffffu, mine, l);
                break;
            }
            left -= __shfl_sync(0xffffffffu, incl, 31);
        }
        s = sequence<true>(p, b);
        blocks = blocks_of(s);
        hg = 0;
        if (groups > 1) {
            const int64_t of_group = quotient(mine, groups);
            hg = static_cast<int>(quotient(left, of_group));
            left -= hg * of_group;
        }
        for (int i0 = 0;; i0 += 32) {
            const int one = i0 + lane < blocks ? line_of(p, s, i0 + lane) : 0;
            int sum = one;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += t;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, sum > left);
            if (hit) {
                const int l = __ffs(hit) - 1;
                block = i0 + l;
                at = static_cast<int>(left) - __shfl_sync(0xffffffffu, sum - one, l) + 1;
                break;
            }
            left -= __shfl_sync(0xffffffffu, sum, 31);
        }
        item(p);
        return true;
    }

    __device__ __forceinline__ void previous_item(const AttentionArgs& p) {
        if (--block < 0) {
            if (--hg < 0) {
                do {
                    s = sequence<true>(p, --b);
                    blocks = blocks_of(s);
                } while (blocks == 0);
                hg = groups - 1;
            }
            block = blocks - 1;
        }
        item(p);
        at = line;
    }

    // The next piece, from the range's end to its beginning; any = 0 when there is none.
    __device__ __forceinline__ Item next(const AttentionArgs& p) {
        Item it{};
        while (w < w_end) {
            const int begin = static_cast<int>(max(static_cast<int64_t>(0), at - (w_end - w)));
            // a key tile belongs to the range that its first unit lies in
            const int most = max(tiles, 1);
            int from = (begin + each - 1) / each, to = min((at + each - 1) / each, most);
            if (tiles <= kWhole) {  // not worth a join: all of it where it begins
                from = begin == 0 ? 0 : most;
                to = most;
            }
            const bool some = from < to;
            if (some) {
                it.any = 1;
                it.q0 = s.q0;
                it.n = s.n;
                it.m = s.m;
                it.b = b;
                it.hk = hg * p.side_heads + side;
                it.token0 = block * pair_tokens;
                it.tiles = each;
                it.j0 = from;
                it.keys = min(to, tiles) - from;
                it.seen = limit(p, s, it.token0);
                it.edge = clampi(it.seen / kKeyTile - from, 0, it.keys);
                it.slot = from == 0 && to == most ? -1 : 2 * blockIdx.x + (from == 0);
                item_start = w_end - at;
                it.last_tile = most - 1;
                if (turns(p)) it.turn = min(turn(from, it.keys), it.edge);
                passed += it.keys + kEnds / 2;
            }
            w_end -= at - begin;
            at = begin;
            if (at == 0 && w < w_end) previous_item(p);
            if (some) break;
        }
        return it;
    }

    // Where a piece begins with its key tiles, so that the CTAs that take the items of one
    // KV head (whose pieces lie in different places) pass the same keys at about the same
    // time and find them in L2: fronts as far apart as a CTA gets, that all started with
    // the call.  (A range that begins in one item and ends in the next takes the end first:
    // those are the next item's first keys.)  Where the items of a sequence are about as
    // long as each other and its keys fill a good part of L2: 512 tokens, 40 heads on 8 x
    // 128, over 33280 keys 275 -> 256 us, over 131072 1010 -> 890, over 8192 99 -> 93; the
    // items of a whole prompt, which differ, lose 2%.
    __device__ __forceinline__ bool turns(const AttentionArgs& p) const {
        return blocks > 1 && 4 * tiles >= 3 * tiles_of(p, s, blocks - 1) &&
               static_cast<int64_t>(s.m) * p.Hk * p.D * 4 >= (int64_t{32} << 20);
    }
    __device__ __forceinline__ int turn(int from, int keys) const {
        const int range_tiles = max(1, static_cast<int>(per >> (each - 1)));
        const int fronts = max(1, (tiles + range_tiles / 2) / range_tiles), apart = max(1, tiles / fronts);
        int ahead = (passed - from) % apart;
        if (ahead < 0) ahead += apart;
        return ahead < keys ? ahead : 0;
    }

    // The seat of a piece at its item's join: the ranges in which its first and its
    // last key tile begin.
    __device__ __forceinline__ Join seat(const Item& it) const {
        return {it.q0, it.n, it.m, it.hk, it.token0, it.tiles, static_cast<int>(quotient(item_start, per)),
                static_cast<int>(quotient(item_start + it.last_tile * it.tiles, per))};
    }
};

template <typename T, int DP, bool kPaged>
__global__ void __launch_bounds__(kThreads, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const AttentionArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    using L = PromptSmem<DP>;
    constexpr int S = L::kStages;
    if (kPaged) grid_launch_dependents();  // the join, which waits for this grid's end
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
    if (smem_u32(smem) & 1023u) {  // the swizzled tiles start at multiples of 1024
        if (threadIdx.x == 0) record_device_error(1);
        if (kPaged && threadIdx.x < 2) static_cast<Join*>(p.joins)[2 * blockIdx.x + threadIdx.x].last = -1;
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
                mbar_init(&bars->v_clean[i], kPaged ? 1 : 2);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&bars->handed[i], 1);
                mbar_init(&bars->taken[i], 1);
            }
            mbar_init(&bars->done, 1);
            fence_mbarrier_init();
        }
        __syncwarp();
        tmem_alloc(&bars->tmem, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    Pieces pieces;
    bool some = true;
    Join* joins = static_cast<Join*>(p.joins) + 2 * blockIdx.x;
    if (kPaged && warp == kSoftmaxWarps + 1) {
        if (elect_one_sync()) {
            tma_prefetch_desc(&tmQ);
            tma_prefetch_desc(&tmK);
            tma_prefetch_desc(&tmV);
        }
        if (lane == 0) joins[0].last = joins[1].last = -1;
        some = pieces.start(p, tile_tokens);
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
        regs_dec<kPaged ? 88 : 72>();  // (168 a thread at launch: 8 warps of 208 and 4 of 88)
        if (warp == kSoftmaxWarps + 1) {
            // ---- items and TMA loads: K_0 Q_0 Q_1 K_1 V_0 ...
            if (!kPaged && elect_one_sync()) {
                tma_prefetch_desc(&tmQ);
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
            }
            const uint32_t q_bytes = L::kChunks * tile_tokens * p.group * 128;
            Items items;
            if (!kPaged) items.start(p, tile_tokens, kKeyTile);
            int index = blockIdx.x, edges = 0;
            int q_ph[2] = {1, 1};  // a fresh barrier lets the first wait through
            Ring<S> r;
            r.ph = 1;
            bool ok = true;
            for (int at = 0; ok; ++at) {
                Item it{};
                if (!kPaged) it = items.find(p, index);
                else if (some) it = pieces.next(p);
                if (!mbar_wait(&bars->item_empty[at & 1], ((at >> 1) & 1) ^ 1, 60)) {
                    it.any = 0;
                    ok = false;
                }
                if (lane == 0) {
                    bars->items[at & 1] = it;
                    mbar_arrive(&bars->item_full[at & 1]);
                }
                if (!it.any) break;
                if (!kPaged && lane == 0) index = atomicAdd(p.counters, 1);
                const int jmax = it.keys;
                Boxes<kKeyTile> boxes;
                if (kPaged && jmax > 0) boxes.start(p, it.b, it.m, it.j0, jmax, it.turn);
                for (int i = 0; i < 2 * jmax; ++i) {
                    const int j = load_tile(i, jmax);
                    const bool is_v = load_is_v(i, jmax);
                    if (kPaged && is_v) {  // another warp's
                        r.next();
                        continue;
                    }
                    ok = mbar_wait(&bars->kv_empty[r.st], r.ph, 61);
                    if (!ok) break;
                    const void* map = is_v ? static_cast<const void*>(&tmV) : static_cast<const void*>(&tmK);
                    if (kPaged) {
                        boxes.step(p);
                        if (elect_one_sync()) mbar_arrive_expect_tx(&bars->kv_full[r.st], L::kTileBytes);
                        boxes.each([&](int x, int row, int page) {
                            const uint32_t dst = pipe + r.st * L::kTileBytes + x * p.box * 128;
#pragma unroll
                            for (int c = 0; c < L::kChunks; ++c)
                                tma_load_page(dst + c * kChunkBytes, &tmK, &bars->kv_full[r.st], 64 * c, it.hk, row, page);
                        });
                    } else if (elect_one_sync()) {
                        mbar_arrive_expect_tx(&bars->kv_full[r.st], L::kTileBytes);
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
                if (kPaged && lane == 0 && it.slot >= 0) joins[it.slot & 1] = pieces.seat(it);
                if (!kPaged) index = static_cast<int>(gridDim.x) + __shfl_sync(0xffffffffu, index, 0);
            }
            // nothing is in flight into this CTA's shared memory when it ends
            // (a stage's last load is complete when its barrier has left that round;
            // a stage never loaded has parity 1 behind it)
            for (int i = 0; i < S; ++i) {
                mbar_wait(&bars->kv_full[r.st], r.ph, 61);
                r.next();
            }
            for (int t = 0; t < 2; ++t) mbar_wait(&bars->q_full[t], q_ph[t], 62);
            if (!kPaged && lane == 0) {  // the last CTA to run out of items leaves the counters at zero
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
                auto run = [&](auto tc, int J, int edge, int past) {
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
                        if (j >= edge && (!kPaged || j < past)) {
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
                // a tile alone: its key tiles go to O of tile 0 and of tile 1 in turn
                auto run_alone = [&](int J, int edge, int past) {
                    Ring<S> rk = r, rv = r;
                    rv.next(load_of_v(0, J));
                    auto scores = [&](int j, int to) {
                        const uint32_t b = (kv_low + rk.st * kTileLow) | kDescKMajor;
#pragma unroll
                        for (int k = 0; k < DP / 16; ++k) {
                            const uint32_t off = ((k >> 2) * kChunkBytes + (k & 3) * 32) >> 4;
                            mma_scores(tmem + 128 * to, q_low + off, b + off, prompt_idesc<T>(kKeyTile, false), k > 0);
                        }
                        mma_commit(&bars->s_full[j & 1][own[j & 1] & 3]);
                        ++own[j & 1];
                        if (j + 1 == J) mma_commit(&bars->q_empty[0]);
                        mma_commit(&bars->kv_empty[rk.st]);
                        rk.next(j == 0 ? 1 : 2);
                    };
                    for (int j = 0; j < NB && j < J; ++j) {
                        if (!(ok = mbar_wait(&bars->kv_full[rk.st], rk.ph, 64))) return;
                        if (j == 0 && !(ok = mbar_wait(&bars->q_full[0], q_ph & 1, 65))) return;
                        tc_fence_after();
                        const int to = buf + j;
                        scores(j, to >= NB ? to - NB : to);
                    }
                    q_ph ^= 1;
                    for (int j = 0; j < J; ++j) {
                        if (!(ok = mbar_wait(&bars->kv_full[rv.st], rv.ph, 66))) return;
                        if (j >= edge && j < past) {
                            if (!(ok = mbar_wait(&bars->v_clean[edges & 3], (edges >> 2) & 1, 67))) return;
                            ++edges;
                        }
                        const uint32_t v_low = (kv_low + rv.st * kTileLow) | kDescMnMajor;
                        const int t = j & 1;
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            if (!(ok = mbar_wait(&bars->p_full[buf][half], (p_ph >> buf) & 1, 69))) return;
                            tc_fence_after();
#pragma unroll
                            for (int k = 4 * half; k < 4 * half + 4; ++k)
                                mma_output(tmem + L::kOutputs + t * DP, tmem + 128 * buf + 8 * k,
                                           v_low + k * (2048 >> 4), prompt_idesc<T>(DP, true), j > 1 || k > 0);
                        }
                        mma_commit(&bars->pv_done[t][pv_own[t] & 3]);
                        ++pv_own[t];
                        mma_commit(&bars->kv_empty[rv.st]);
                        rv.next(load_of_v(j + 1, J) - load_of_v(j, J));
                        if (j + NB < J) {
                            if (!(ok = mbar_wait(&bars->kv_full[rk.st], rk.ph, 68))) return;
                            tc_fence_after();
                            scores(j + NB, buf);
                        }
                        p_ph ^= 1 << buf;
                        if (++buf == NB) buf = 0;
                    }
                };
                for (int at = 0; ok; ++at) {
                    if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 63)) break;
                    const volatile Item& it = bars->items[at & 1];
                    const int any = it.any, two = it.tiles > 1, J = it.keys, turn = kPaged ? it.turn : 0;
                    const int edge = it.edge - turn, past = J - turn;  // steps of the tiles from edge on
                    if (!any) break;
                    mbar_arrive(&bars->item_empty[at & 1]);
                    if (J == 0) continue;
                    if (two) run(std::integral_constant<int, 2>{}, J, edge, past);
                    else if (kPaged) run_alone(J, edge, past);
                    else run(std::integral_constant<int, 1>{}, J, edge, past);
                    r.skip(2 * J);
                }
            // every commit has arrived before the CTA ends
            mma_commit(&bars->done);
            mbar_wait(&bars->done, 0, 70);
            }
            __syncwarp();
        } else if (kPaged && warp == kSoftmaxWarps + 2) {
            // ---- V from pages (the copies of one warp alone would bound short tiles)
            Ring<S> r;
            r.ph = 1;
            int edges = 0;
            bool ok = true;
            for (int at = 0; ok; ++at) {
                if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 81)) break;
                const volatile Item& it = bars->items[at & 1];
                if (!it.any) break;
                const int jmax = it.keys, hk = it.hk, edge = it.edge, turn = it.turn;
                Boxes<kKeyTile> boxes;
                if (jmax > 0) boxes.start(p, it.b, it.m, it.j0, jmax, turn);
                leave_item(at);
                for (int i = 0; i < 2 * jmax; ++i, r.next()) {
                    if (!load_is_v(i, jmax)) continue;
                    ok = mbar_wait(&bars->kv_empty[r.st], r.ph, 82);
                    if (!ok) break;
                    const int j = load_tile(i, jmax), tile = Item::tile_of(j, turn, jmax);
                    boxes.step(p);
                    if (elect_one_sync()) mbar_arrive_expect_tx(&bars->kv_full[r.st], L::kTileBytes);
                    boxes.each([&](int x, int row, int page) {
                        const uint32_t dst = pipe + r.st * L::kTileBytes + x * p.box * 128;
#pragma unroll
                        for (int c = 0; c < L::kChunks; ++c)
                            tma_load_page(dst + c * kChunkBytes, &tmV, &bars->kv_full[r.st], 64 * c, hk, row, page);
                    });
                    if (tile < edge) continue;
                    if (elect_one_sync()) mbar_arrive(&bars->v_issued[edges & 3]);
                    ++edges;
                }
            }
            for (int i = 0; i < S; ++i) {  // nothing is in flight when the CTA ends
                mbar_wait(&bars->kv_full[r.st], r.ph, 82);
                r.next();
            }
        } else {
            // ---- V cleaners: key tiles from `edge` on
            constexpr int kCleaners = kPaged ? 32 : 64;
            const int me = threadIdx.x - 32 * (kSoftmaxWarps + 4) + kCleaners;  // 0 .. kCleaners - 1
            int ld = 0, edges = 0;
            bool ok = true;
            for (int at = 0; ok; ++at) {
                if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 71)) break;
                volatile Item& it = bars->items[at & 1];
                if (!it.any) break;
                const int jmax = it.keys;
                for (int j = kPaged ? 0 : it.edge; j < jmax && ok; ++j) {
                    const int tile = kPaged ? Item::tile_of(j, it.turn, jmax) : j;
                    if (tile < it.edge) continue;
                    const int lv = ld + load_of_v(j, jmax);
                    ok = mbar_wait(&bars->v_issued[edges & 3], (edges >> 2) & 1, 72) &&
                         mbar_wait(&bars->kv_full[lv % S], (lv / S) & 1, 73);
                    if (!ok) break;
                    const uint32_t v = pipe + (lv % S) * L::kTileBytes;
                    constexpr int kAtOnce = 8;  // loads in flight: one by one they would bound an item's end
                    static_assert(L::kTileBytes % (16 * kCleaners * kAtOnce) == 0, "whole rounds");
                    for (int c0 = me; c0 < L::kTileBytes / 16; c0 += kCleaners * kAtOnce) {
                        // 32 keys at a time, from those on that some row does not see
                        static_assert(!kPaged || kCleaners * kAtOnce == 32 * 8, "32 keys");
                        if (kPaged && (it.j0 + tile) * kKeyTile + ((c0 - me) / 8 & 127) + 32 <= it.seen) continue;
                        uint4 w[kAtOnce];
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i)
                            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w[i].x), "=r"(w[i].y), "=r"(w[i].z), "=r"(w[i].w)
                                         : "r"(v + 16 * (c0 + kCleaners * i)));
                        bool some = false;
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) some |= any_non_finite<T>(w[i]);
                        if (!some) continue;
#pragma unroll
                        for (int i = 0; i < kAtOnce; ++i) {
                            if (!any_non_finite<T>(w[i])) continue;
                            const int c = c0 + kCleaners * i;
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
                            const int key = (kPaged ? it.j0 + tile : j) * kKeyTile + ((c >> 3) & 127);
                            if (key < it.m) it.bad = 1;
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->v_clean[edges & 3]);
                    ++edges;
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
        int alones = 0;          // tiles alone so far
        int steps = 0, own = 0;  // steps of both tiles before this item (mod the buffers), of this tile
        bool ok = true;
        for (int at = 0; ok; ++at) {
            if (!mbar_wait(&bars->item_full[at & 1], (at >> 1) & 1, 74)) break;
            const volatile Item& it = bars->items[at & 1];
            if (!it.any) break;
            // a tile alone: both groups' rows are its rows, and the key tiles theirs in turn
            const int both = it.tiles;
            const bool alone = kPaged && both == 1;
            const int j_first = alone ? t : 0, j_step = alone ? 2 : 1;
            const int my_token = alone ? row / p.group : row_token;
            int lim, warp_lim, sees;  // limits from the first key of the item
            {
                const int n = it.n, m = it.m, token = it.token0 + my_token;
                const bool valid = used && (alone || t < both) && token < n;
                lim = valid ? (p.causal ? clampi(token - n + m + 1, 0, m) : m) : 0;
                warp_lim = __reduce_min_sync(0xffffffffu, valid ? lim : m);
                sees = lim;
                if (kPaged) {
                    lim -= it.j0 * kKeyTile;
                    warp_lim -= it.j0 * kKeyTile;
                }
            }
            const int tiles = alone || t < both ? it.keys : 0;
            // first key of the step's tile, from the item's first one
            int key0 = kPaged ? Item::tile_of(j_first, it.turn, it.keys) * kKeyTile : 0;
            float ref = -INFINITY;
            auto base_of = [](float r) { return r == -INFINITY ? 0.0f : kShift<T> - r; };
            uint64_t sum2 = f2_pack(0.0f, 0.0f);
            for (int j = j_first; j < tiles; j += j_step, ++own) {
                const int buf = (steps + (alone ? j : j * both + t)) % L::kBuffers;
                const uint32_t ts = tmem + lanes + 128 * buf;
                ok = mbar_wait(&bars->s_full[t][own & 3], (own >> 2) & 1, 75);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[4][32];
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, v[i]);
#pragma unroll
                for (int i = 0; i < 4; ++i) tmem_wait_ld_regs32(v[i]);
                if (!kPaged) key0 = j * kKeyTile;
                if (warp_lim < key0 + kKeyTile) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int left = lim - key0 - 32 * i;  // columns this row sees
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
                if (j == j_first) {
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
                if (kPaged) {
                    key0 += j_step * kKeyTile;
                    if (key0 >= tiles * kKeyTile) key0 -= tiles * kKeyTile;
                }
            }

            steps = (steps + both * it.keys) % L::kBuffers;

            // ---- O / sum to memory
            float l0, l1;
            f2_unpack(sum2, l0, l1);
            float l = l0 + l1;
            float f0 = 1.0f, f1 = 0.0f;  // weights of this group's O and the other's, of a tile alone
            if (alone) {
                float2* row_of = reinterpret_cast<float2*>(smem + L::kHanded) + row;
                if (t == 1) {
                    if (tiles > 1) ok = ok && mbar_wait(&bars->pv_done[1][(own - 1) & 3], ((own - 1) >> 2) & 1, 78);
                    if (!ok) break;
                    *row_of = make_float2(ref, l);
                    leave_item(at);
                    tc_fence_before();
                    if (lane == 0) mbar_arrive(&bars->handed[wq]);
                    ok = mbar_wait(&bars->taken[wq], alones & 1, 79);
                    ++alones;
                    continue;
                }
                ok = ok && mbar_wait(&bars->handed[wq], alones & 1, 80);
                if (!ok) break;
                ++alones;
                const float2 other = *row_of;
                const float to_ref = fmaxf(ref, other.x);
                f0 = ref == to_ref ? 1.0f : exp2_approx(ref - to_ref);
                f1 = other.x == to_ref ? 1.0f : exp2_approx(other.x - to_ref);
                ref = to_ref;
                l = l * f0 + other.y * f1;
            }
            const float inv = sees > 0 ? __frcp_rn(l) : 0.0f;
            // where the rows go: through shared memory, so that eight lanes write 128
            // bytes of a row, this lane 16 bytes of rows sub, sub + 4, ...
            const int q0 = it.q0, k0 = it.k0, hk = it.hk, token = it.token0 + row_token, edge = it.edge;
            const bool valid = used && t < it.tiles && token < it.n;
            const int first = kPaged ? it.j0 * kKeyTile : 0, b = kPaged ? it.b : 0, slot = kPaged ? it.slot : -1;
            const int seen_end = kPaged ? min(lim, it.keys * kKeyTile) : lim;
            const int head = hk * p.group + row_head;
            const int sub = lane >> 3, ch = lane & 7;
            const uint32_t valid_rows = __ballot_sync(0xffffffffu, valid) >> sub;
            int64_t mine = static_cast<int64_t>(q0 + token) * p.o_token + static_cast<int64_t>(head) * p.o_head;
            int64_t to_row[8];  // elements, or over pages an address
            float* part = nullptr;
            if constexpr (kPaged) {
                part = p.partial + (2 * static_cast<int64_t>(slot) + t) * kTilePart<DP>;
                mine = reinterpret_cast<int64_t>(slot >= 0 ? static_cast<void*>(part + 2 * kTileRows + row * DP)
                                                           : static_cast<void*>(static_cast<T*>(p.o) + mine));
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) to_row[x] = __shfl_sync(0xffffffffu, mine, 4 * x + sub) + (kPaged ? 0 : 8 * ch);
            if (tiles > 0) ok = ok && mbar_wait(&bars->pv_done[t][(own - 1) & 3], ((own - 1) >> 2) & 1, 76);
            if (!ok) break;
            tc_fence_after();
            const int bad = tiles > 0 ? it.bad : 0;
            leave_item(at);
            const uint32_t stage = smem_u32(smem) + L::kOut + warp * L::kOutBytes;
            if constexpr (kPaged) {
                // A whole item's rows in the type, or a piece's in binary32 for the join, 32
                // columns at a time in one loop: an item's end is run seldom, and fetching
                // its code takes as long as running it (6 us for the first end on an SM
                // when the loop was written out for both).
                const float scale = slot >= 0 ? 1.0f : inv;
#pragma unroll 1
                for (int c = 0; c < DP / 32; ++c) {
                    uint32_t o[32];
                    if (tiles > 0) {
                        tmem_ld_32x32b_x32(to + 32 * c, o);
                        tmem_wait_ld_regs32(o);
                        if (alone && tiles > 1) {
                            uint32_t o1[32];
                            tmem_ld_32x32b_x32(to + DP + 32 * c, o1);
                            tmem_wait_ld_regs32(o1);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                o[x] = __float_as_uint(__uint_as_float(o[x]) * f0 + __uint_as_float(o1[x]) * f1);
                        }
                    }
                    if (alone && 32 * c + 32 == DP) {  // O of the other group has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars->taken[wq]);
                    }
                    const bool some = tiles > 0 && (sees > 0 || slot >= 0);
#pragma unroll
                    for (int x = 0; x < 8; ++x) {
                        float f[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) f[y] = some ? __uint_as_float(o[4 * x + y]) * scale : 0.0f;
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         stage + lane * 128 + ((x ^ (lane & 7)) << 4)),
                                     "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3])
                                     : "memory");
                    }
                    if (bad) {  // the non-finite values that this row sees, in its places
#pragma unroll 1
                        for (int key = edge * kKeyTile; key < seen_end; ++key) {
                            const unsigned at_key = first + key, size = p.page_size;
                            const int page = page_of(p, entry_of(p, b, at_key / size));
                            if (page == p.pages) continue;  // zeros
                            const T* src = static_cast<const T*>(p.v) + page * p.v_page + at_key % size * p.v_token +
                                           hk * p.v_head + 32 * c;
#pragma unroll 1
                            for (int x = 0; x < 32 && 32 * c + x < p.D; ++x) {
                                const float val = static_cast<float>(src[x]);
                                if (isfinite(val)) continue;
                                const uint32_t place = stage + lane * 128 + (((x >> 2) ^ (lane & 7)) << 4) + 4 * (x & 3);
                                float f;
                                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(place) : "memory");
                                asm volatile("st.shared.f32 [%0], %1;" ::"r"(place), "f"(f + val) : "memory");
                            }
                        }
                    }
                    __syncwarp();
                    float4 w[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(w[x].x), "=f"(w[x].y), "=f"(w[x].z), "=f"(w[x].w)
                                     : "r"(stage + (4 * x + sub) * 128 + ((ch ^ ((4 * x + sub) & 7)) << 4)));
                    if (slot >= 0) {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (valid_rows >> (4 * x) & 1)
                                reinterpret_cast<float4*>(to_row[x])[8 * c + ch] = w[x];
                    } else if (32 * c + 4 * ch < p.D) {
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            if (valid_rows >> (4 * x) & 1)
                                reinterpret_cast<uint2*>(to_row[x])[8 * c + ch] =
                                    make_uint2(Pair16<T>::pack(w[x].x, w[x].y), Pair16<T>::pack(w[x].z, w[x].w));
                    }
                    __syncwarp();
                }
                if (valid && slot >= 0) *reinterpret_cast<float2*>(part + 2 * row) = make_float2(ref, l);
            } else {
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
                            if (valid_rows >> (4 * x) & 1)
                                *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + to_row[x] + 64 * i) = w[x];
                    }
                    __syncwarp();
                }
            }
            if (p.lse && valid && slot < 0)
                p.lse[static_cast<int64_t>(q0 + token) * p.Hq + head] =
                    sees > 0 ? (log2f(l) - base_of(ref)) * kLn2 : -INFINITY;
            tc_fence_before();
        }
    }
    __syncthreads();
    if (warp == kSoftmaxWarps) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace
}  // namespace w8a8


// Attention of a few queries per sequence over long caches:
// o_i = sum_j softmax_j(scale q_i k_j) v_j with grouped heads.
//
// One query of a group of G heads reads each K and V value once for G
// multiply-adds, so the keys' bytes bound it: the G heads (and the n queries)
// that share a KV head form the rows of up to four warp MMA tiles (16 x 16 x 8)
// and the keys stream through shared memory once.
//
// The row blocks of all sequences are laid end to end, each as its tiles of 64
// keys, and cut into equal ranges whatever the lengths are; the lengths stay on
// the device.  CTAs that run side by side take the same range for neighbouring
// KV heads (up to 8), so that they read whole rows of the cache.  One CTA per
// SM (or two of half the size): its last warp keeps the ring of key tiles full by
// TMA, also across items; warps 0-3 and 4-7 take the tiles in turn, each warp its
// own 16 rows and its own part of the tile's keys with an online softmax of its
// own (no barrier while keys stream), and are joined at the end of an item.  An
// item that spans CTAs leaves (max, sum, unnormalized output) per piece in the
// workspace; the CTA that arrives last joins the pieces in key order, so the
// result does not depend on the order of arrival.
//
// Measured with single queries, heads of 128, bf16: 131072 + 99991 keys of 8 KV
// heads 139 us (the copy bandwidth), 64 sequences of 1 to 4096 keys 88 us (0.88: items
// start and end all along the way), 4 sequences of 77 to 513 keys 9.8 us (launch,
// one tile's latency, the join).
//
//   softmax:  t = scale log2(e) s;  running max M, sum L, O in binary32,
//             p = 2^(t - M); P enters the second product rounded to the
//             inputs' type (half a step, 2^-8 for bf16, of each p: the same
//             size as the output's own rounding, the sums stay binary32), in
//             fp16 times 2^15, so that only weights below 2^-29 lose bits of it
//             (2^-40 of a row's largest at most; 8 multiplications a step of 16
//             keys, exact ones).
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <type_traits>

#include "attention.cuh"
#include "pair16.cuh"
#include "ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kWarps = 4;      // of a group
constexpr int kKeys = 16;      // keys of a step
constexpr int kTile = 64;
constexpr int threads_of(int G) { return G * kWarps * 32 + 32; }

// R: packed (query, head) rows of an item: 16, 32 or 64.  The four warps of a
// group are R / 16 tiles of rows by 64 / R parts of the keys.
// G: groups of a CTA, which take its tiles in turn.  2: one CTA per SM; 1: two,
// with half the ring each.
template <int DP, int R, int G>
struct SplitSmem {
    static constexpr int kChunk = kTile * 128;  // 64 elements of each key, 128-byte swizzled
    static constexpr int kKv = DP / 64 * kChunk;
    static constexpr int kStage = 2 * kKv;      // K, then V
    // even: a stage is always the same group's, whose waits then see every round of its barrier
    static constexpr int kStages = (DP == 128 ? 2 : 4) * G;
    static_assert(kStages % G == 0, "one group per stage");
    static constexpr int kJoin = kStages * kStage;  // (max, sum, output) of every warp
    // rows 8 floats further apart than they are long: the 8 rows that a warp writes at
    // once fall into different banks
    static constexpr int kJoinRow = DP + 8, kSlot = 16 * (2 + kJoinRow);
    static constexpr int kQ = kJoin + G * kWarps * kSlot * 4;
    static constexpr int kBars = kQ + R * DP * 2;
    static constexpr int kTotal = kBars + 2 * kStages * 8;
};

// Byte offset of 16-byte chunk c of row r of a tile as TMA writes it, and of a
// [rows][DP] tile of Q: chunks permuted by the row, so that eight rows of one
// chunk column fall into different banks.
__device__ __forceinline__ uint32_t kv_at(int r, int c) {
    return static_cast<uint32_t>((c >> 3) * kTile * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
template <int DP>
__device__ __forceinline__ uint32_t q_at(int r, int c) {
    return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

// Partial result of one piece of an item: [R] maxima, [R] sums, [R][DP] outputs.
template <int DP, int R>
constexpr int kPartFloats = R * (DP + 2);

// Where a linear tile index lies: sequence, head group and row block, tile.
struct Cursor {
    int b;
    Sequence s;
    int blocks;    // R-row blocks of the sequence
    int tiles;     // key tiles of one block
    int item;      // head group * blocks + block
    int tile;
};

template <int R>
__device__ __forceinline__ int blocks_of(const AttentionArgs& p, const Sequence& s) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.group + R - 1) / R);
}
__device__ __forceinline__ int tiles_of(const Sequence& s) { return max(1, (s.m + kTile - 1) / kTile); }

// Tiles of the 32 sequences from b0 on: this lane's, and inclusive over the
// lanes; `most` becomes the most of one item.
template <int R>
__device__ __forceinline__ void tiles_from(const AttentionArgs& p, int b0, int64_t& mine, int64_t& incl, int& most) {
    const int lane = threadIdx.x & 31;
    mine = 0;
    if (b0 + lane < p.batch) {
        const Sequence s = sequence(p, b0 + lane);
        mine = static_cast<int64_t>(blocks_of<R>(p, s)) * (p.Hk / p.side_heads) * tiles_of(s);
        most = max(most, tiles_of(s));
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
}

__device__ __forceinline__ float sqrt_approx(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a / b for positive a and b, in 32 bits where a allows.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

template <typename T, int DP, int R, int G>
__global__ void __launch_bounds__(threads_of(G), 3 - G)
    attention_split_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const AttentionArgs p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ int last_flag;
    using L = SplitSmem<DP, R, G>;
    constexpr int S = L::kStages, kConsumers = threads_of(G) - 32;
    constexpr int kRowTiles = R / 16, kParts = kWarps / kRowTiles;
    constexpr int kChunks = DP / 8;   // 16-byte chunks of a row
    constexpr int kDT = DP / 8;       // 8-wide output column tiles
    constexpr float kScale = std::is_same<T, __half>::value ? 32768.0f : 1.0f;  // of p and O, not of the sum
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kBars);
    uint64_t* empty = full + S;
    float* join = reinterpret_cast<float*>(smem + L::kJoin);

    if (smem_u32(smem) & 1023u) {  // the swizzled tiles start at multiples of 1024
        if (threadIdx.x == 0) record_device_error(1);
        return;
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kWarps);
        }
        fence_mbarrier_init();
    }

    // this CTA's range of tiles, found by every warp on its own; the first 32
    // sequences' counts stay
    const int side = blockIdx.x % p.side_heads, range = blockIdx.x / p.side_heads, ranges = gridDim.x / p.side_heads;
    const int head_groups = p.Hk / p.side_heads;
    Sequence own = {0, 0, 0, 0};  // this lane's, of up to 32
    if (p.batch <= 32 && lane < p.batch) own = sequence(p, lane);
    const int blocks = blocks_of<R>(p, own), items = blocks * head_groups, tiles = tiles_of(own);
    int64_t mine = static_cast<int64_t>(items) * tiles, incl, total;
    int most = tiles;
    const bool few = p.batch <= 32 && !__any_sync(0xffffffffu, mine > 1 << 24);  // fits 32 bits
    if (few) {
        total = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine));
    } else {
        tiles_from<R>(p, 0, mine, incl, most);
        total = __shfl_sync(0xffffffffu, incl, 31);
        for (int b0 = 32; b0 < p.batch; b0 += 32) {
            int64_t m2, i2;
            tiles_from<R>(p, b0, m2, i2, most);
            total += __shfl_sync(0xffffffffu, i2, 31);
        }
    }
    // A piece takes a CTA 0.35 us a tile (of 16 rows; 64 rows four times that), and the
    // join 0.08 us a piece for each of its rounds over the rows: few tiles are not cut
    // into more pieces than that is worth (12 heads on 1, one sequence of 4871 keys 14
    // us against 24).
    const int least = max(1, static_cast<int>(sqrt_approx(0.23f * 16 / R * p.join_rounds * __reduce_max_sync(0xffffffffu, most))));
    int64_t per = max(static_cast<int64_t>(least), quotient(total + ranges - 1, ranges));
    // A CTA whose range ends one item and begins another takes 3 us longer: where
    // there are few tiles, ranges of a few more that start with the items are better
    // (8 sequences of 300 keys 10.8 us against 13.3).  An item then takes whole ranges
    // of the line of tiles.
    int line = tiles;  // an item's part of the line
    bool apart = false;
    if (few) {
        if (total <= 64 * ranges) {
            for (int wide = static_cast<int>(per), end = wide + 4; wide <= end; ++wide) {
                const int pieces = (tiles + wide - 1) / wide;
                if (__reduce_add_sync(0xffffffffu, static_cast<unsigned>(items * pieces)) > static_cast<unsigned>(ranges))
                    continue;
                apart = true;
                per = wide;
                line = pieces * wide;
                break;
            }
        }
        const int n = items * line;
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += t;
        }
        mine = n;
        incl = sum;
        total = __shfl_sync(0xffffffffu, sum, 31);
    }
    int64_t w = per * range;
    int64_t w_end = min(total, w + per);
    if (w >= w_end) return;
    Cursor c;
    {  // the cursor of tile w
        int64_t left = w;
        for (int b0 = 0;; b0 += 32) {
            if (b0 > 0) tiles_from<R>(p, b0, mine, incl, most);
            const unsigned hit = __ballot_sync(0xffffffffu, incl > left);
            if (hit) {
                const int l = __ffs(hit) - 1;
                left -= __shfl_sync(0xffffffffu, incl - mine, l);
                c.b = b0 + l;
                break;
            }
            left -= __shfl_sync(0xffffffffu, incl, 31);
        }
        if (few) {
            const auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, c.b); };
            c.s = {of(own.q0), of(own.n), of(own.k0), of(own.m)};
            c.blocks = of(blocks);
            c.tiles = of(tiles);
            line = of(line);
        } else {
            c.s = sequence(p, c.b);
            c.blocks = blocks_of<R>(p, c.s);
            line = c.tiles = tiles_of(c.s);
        }
        c.item = static_cast<int>(quotient(left, line));
        c.tile = static_cast<int>(left - static_cast<int64_t>(c.item) * line);
        if (apart) w_end = w + min(per, static_cast<int64_t>(c.tiles - c.tile));
    }
    __syncthreads();

    // The next piece: tiles [c.tile, t_end) of item c.item; false at the end.
    auto next_piece = [&](int t_end) {
        w += t_end - c.tile;
        c.tile = 0;
        if (w >= w_end) return false;
        if (++c.item >= c.blocks * head_groups) {
            c.item = 0;
            do {
                if (++c.b >= p.batch) return false;
                c.s = sequence(p, c.b);
                c.blocks = blocks_of<R>(p, c.s);
                c.tiles = tiles_of(c.s);
            } while (c.blocks == 0);
        }
        return true;
    };
    auto piece_end = [&]() { return static_cast<int>(min(static_cast<int64_t>(c.tiles), c.tile + (w_end - w))); };
    // keys that packed row pr of the sequence sees: [0, limit)
    auto limit = [&](int pr) { return p.causal ? clampi(pr / p.group + c.s.m - c.s.n + 1, 0, c.s.m) : c.s.m; };
    // tiles of the piece that some row sees end here
    auto seen_end = [&](int rb, int t_end) {
        const int last = min((rb + 1) * R, c.s.n * p.group) - 1;
        return min(t_end, (limit(last) + kTile - 1) / kTile);
    };

    int st = 0, ph = 0;  // ring place of the next tile
    auto next_stage = [&]() {
        if (++st == S) {
            st = 0;
            ph ^= 1;
        }
    };

    if (warp == G * kWarps) {
        // ---- producer
        bool ok = true;
        int loaded = 0;
        for (bool more = true; more && ok;) {
            const int t_end = piece_end(), hg = c.item / c.blocks, rb = c.item - hg * c.blocks;
            const int end = seen_end(rb, t_end), hk = hg * p.side_heads + side;
            for (int t = c.tile; t < end; ++t) {
                ok = mbar_wait(&empty[st], ph ^ 1, 50);
                if (!ok) break;
                if (elect_one_sync()) {
                    mbar_arrive_expect_tx(&full[st], L::kStage);
                    const uint32_t dst = smem_u32(smem) + st * L::kStage;
#pragma unroll
                    for (int x = 0; x < DP / 64; ++x) {
                        tma_load_3d(dst + x * L::kChunk, &tmK, &full[st], 64 * x, hk, c.s.k0 + t * kTile);
                        tma_load_3d(dst + L::kKv + x * L::kChunk, &tmV, &full[st], 64 * x, hk, c.s.k0 + t * kTile);
                    }
                }
                ++loaded;
                next_stage();
            }
            more = next_piece(t_end);
        }
        // nothing is in flight into this CTA's shared memory when it ends: the
        // last round of every stage that was loaded
        for (int i = 0; i < min(S, loaded); ++i) {
            if (--st < 0) {
                st = S - 1;
                ph ^= 1;
            }
            mbar_wait(&full[st], ph, 51);
        }
        return;
    }

    // ---- consumers
    const int group = warp / kWarps, sub = warp % kWarps;
    const int my_row = 16 * (sub % kRowTiles), my_keys = sub / kRowTiles * (kTile / kParts);  // of an item, of a tile
    bool ok = true;
    int turn = 0;  // group of the next tile
    for (bool more = true; more;) {
        const int t_begin = c.tile, t_end = piece_end();
        const int64_t item_start = w - t_begin;
        const int hg = c.item / c.blocks, rb = c.item - hg * c.blocks, hk = hg * p.side_heads + side;
        const Sequence s = c.s;
        const int rows = min(R, s.n * p.group - rb * R);
        const int lim_low = limit(rb * R), end = seen_end(rb, t_end);

        // Q rows to shared memory
        for (int u = threadIdx.x; u < R * kChunks; u += kConsumers) {
            const int r = u / kChunks, ch = u % kChunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && 8 * ch < p.D) {
                const int pr = rb * R + r, i = pr / p.group, g = pr - i * p.group;
                v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                    static_cast<int64_t>(s.q0 + i) * p.q_token +
                                                    static_cast<int64_t>(hk * p.group + g) * p.q_head + 8 * ch);
            }
            *reinterpret_cast<uint4*>(smem + L::kQ + q_at<DP>(r, ch)) = v;
        }
        float o[kDT][4], mx[2], sum[2];
        int lim[2];
#pragma unroll
        for (int j = 0; j < kDT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = my_row + (lane >> 2) + 8 * h;
            mx[h] = -INFINITY;
            sum[h] = 0.0f;
            lim[h] = r < rows ? limit(rb * R + r) : 0;
        }
        named_bar_sync(1, kConsumers);
        uint32_t qf[DP / 16][4];
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
            ldmatrix4(qf[kk], smem_u32(smem) + L::kQ + q_at<DP>(my_row + (lane & 15), 2 * kk + (lane >> 4)));

#pragma unroll 1
        for (int t = t_begin; t < end; ++t, turn ^= 1, next_stage()) {
            if (G > 1 && turn != group) continue;
            ok = ok && mbar_wait(&full[st], ph, 52);
            const uint32_t ks = smem_u32(smem) + st * L::kStage, vs = ks + L::kKv;
#pragma unroll 1
            for (int row0 = my_keys; row0 < my_keys + kTile / kParts; row0 += kKeys) {
                const int key0 = t * kTile + row0;
                float sc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
                for (int kk = 0; kk < DP / 16; ++kk) {
                    uint32_t kf[4];
                    ldmatrix4(kf, ks + kv_at(row0 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
                    mma16816<T>(sc[0], qf[kk], kf[0], kf[1]);
                    mma16816<T>(sc[1], qf[kk], kf[2], kf[3]);
                }
                const int col = key0 + 2 * (lane & 3);
                float tm[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[j][e] = col + 8 * j + (e & 1) < lim[e >> 1] ? sc[j][e] * p.scale_log2 : -INFINITY;
                        tm[e >> 1] = fmaxf(tm[e >> 1], sc[j][e]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 1));
                    tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 2));
                }
                const bool grows = tm[0] > mx[0] || tm[1] > mx[1];
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float m = fmaxf(mx[h], tm[h]);
                        const float f = m == mx[h] ? 1.0f : exp2_approx(mx[h] - m);
                        mx[h] = m;
                        sum[h] *= f;
#pragma unroll
                        for (int j = 0; j < kDT; ++j) {
                            o[j][2 * h] *= f;
                            o[j][2 * h + 1] *= f;
                        }
                    }
                }
                const float base[2] = {mx[0] == -INFINITY ? 0.0f : mx[0], mx[1] == -INFINITY ? 0.0f : mx[1]};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[j][e] = exp2_approx(sc[j][e] - base[e >> 1]);
                        sum[e >> 1] += sc[j][e];
                    }
                // A key that only some of the rows see (or none: past the length)
                // must not reach the others through 0 * inf: such keys with a
                // non-finite V go one by one.
                bool apart = false;
                if (key0 + kKeys > lim_low) {
                    bool bad = false;
                    for (int u = lane; u < kKeys * kChunks; u += 32) {
                        uint4 v;
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                     : "r"(vs + kv_at(row0 + u / kChunks, u % kChunks)));
                        bad |= any_non_finite<T>(v);
                    }
                    apart = __any_sync(0xffffffffu, bad);
                }
                if (!apart) {
                    uint32_t pf[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pf[i] = Pair16<T>::pack(sc[i >> 1][2 * (i & 1)] * kScale, sc[i >> 1][2 * (i & 1) + 1] * kScale);
#pragma unroll
                    for (int j = 0; j < kDT; j += 2) {
                        uint32_t vf[4];
                        ldmatrix4_trans(vf, vs + kv_at(row0 + (lane & 7) + ((lane >> 3) & 1) * 8, j + (lane >> 4)));
                        mma16816<T>(o[j], pf, vf[0], vf[1]);
                        mma16816<T>(o[j + 1], pf, vf[2], vf[3]);
                    }
                } else {
#pragma unroll 1
                    for (int k = 0; k < kKeys; ++k) {
                        // p of rows lane/4 and lane/4 + 8 at key k
                        const int from = (lane & ~3) | ((k & 7) >> 1);
                        auto pick = [&](int e) {
                            const float even = k & 8 ? sc[1][e] : sc[0][e];
                            const float odd = k & 8 ? sc[1][e + 1] : sc[0][e + 1];
                            return __shfl_sync(0xffffffffu, k & 1 ? odd : even, from);
                        };
                        const float p0 = pick(0) * kScale, p1 = pick(2) * kScale;
                        const bool s0 = key0 + k < lim[0], s1 = key0 + k < lim[1];
#pragma unroll
                        for (int j = 0; j < kDT; ++j) {
                            uint32_t w32;
                            asm volatile("ld.shared.u32 %0, [%1];"
                                         : "=r"(w32)
                                         : "r"(vs + kv_at(row0 + k, j) + 4 * (lane & 3)));
                            const float2 v = Pair16<T>::unpack(w32);
                            if (s0) {
                                o[j][0] = fmaf(p0, v.x, o[j][0]);
                                o[j][1] = fmaf(p0, v.y, o[j][1]);
                            }
                            if (s1) {
                                o[j][2] = fmaf(p1, v.x, o[j][2]);
                                o[j][3] = fmaf(p1, v.y, o[j][3]);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
        }

        // ---- join: every warp's rows to shared memory, then each thread its share of a
        // row from the warps that have a part of it
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        }
        // a warp's [16] maxima, [16] sums, [16][kJoinRow] outputs
        constexpr int kSlot = L::kSlot, kJoinRow = L::kJoinRow;
        float* slot = join + warp * kSlot;
        // (the piece before has been read: its readers came through the barrier after Q)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = 8 * h + (lane >> 2);
            if ((lane & 3) == 0) {
                slot[r] = mx[h];
                slot[16 + r] = sum[h];
            }
#pragma unroll
            for (int j = 0; j < kDT; ++j)
                *reinterpret_cast<float2*>(slot + 32 + r * kJoinRow + 8 * j + 2 * (lane & 3)) =
                    make_float2(o[j][2 * h], o[j][2 * h + 1]);
        }
        named_bar_sync(1, kConsumers);

        // A thread takes four columns of a row, of the rows that there are.
        constexpr int kQuads = DP / 4, kPart = kPartFloats<DP, R>;
        const bool whole = t_begin == 0 && t_end == c.tiles;
        float* part = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (t_begin == 0 ? 1 : 0)) * kPart;
        struct Row {
            float m = -INFINITY, l = 0.0f;
            float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
            __device__ void add(float m1, float l1, const float4& v1, float f0, float f1) {
                m = m1;
                l = l * f0 + l1 * f1;
                v = make_float4(v.x * f0 + v1.x * f1, v.y * f0 + v1.y * f1, v.z * f0 + v1.z * f1, v.w * f0 + v1.w * f1);
            }
        };
        auto weight = [](float m, float top) { return m == top ? 1.0f : exp2_approx(m - top); };
        auto store = [&](const Row& row, int r, int col) {
            const int pr = rb * R + r, i = pr / p.group, g = pr - i * p.group, head = hk * p.group + g;
            const bool sees = limit(pr) > 0;
            // (a row that sees keys of no weight is 0 / 0)
            const float inv = sees ? __frcp_rn(row.l) * (1.0f / kScale) : 0.0f;
            if (col < p.D)
                *reinterpret_cast<uint2*>(static_cast<T*>(p.o) + static_cast<int64_t>(s.q0 + i) * p.o_token +
                                          static_cast<int64_t>(head) * p.o_head + col) =
                    sees ? make_uint2(Pair16<T>::pack(row.v.x * inv, row.v.y * inv),
                                      Pair16<T>::pack(row.v.z * inv, row.v.w * inv))
                         : make_uint2(0, 0);
            if (p.lse && col == 0)
                p.lse[static_cast<int64_t>(s.q0 + i) * p.Hq + head] =
                    sees ? (row.m + log2f(row.l)) * kLn2 : -INFINITY;
        };
#pragma unroll 1
        for (int e = threadIdx.x; e < rows * kQuads; e += kConsumers) {
            const int r = e / kQuads, col = 4 * (e % kQuads);
            Row row;
#pragma unroll
            for (int x = 0; x < G * kParts; ++x) {
                const float* pm = join + (x * kRowTiles + r / 16) * kSlot;
                const float m = pm[r % 16], top = fmaxf(row.m, m);
                row.add(top, pm[16 + r % 16], *reinterpret_cast<const float4*>(pm + 32 + r % 16 * kJoinRow + col),
                        weight(row.m, top), weight(m, top));
            }
            if (whole) {
                store(row, r, col);
            } else {
                *reinterpret_cast<float4*>(part + 2 * R + r * DP + col) = row.v;
                if (col == 0) {
                    part[r] = row.m;
                    part[R + r] = row.l;
                }
            }
        }
        if (!whole) {
            // the last piece to arrive joins all, in the order of their keys
            __threadfence();
            named_bar_sync(1, kConsumers);
            const int first = static_cast<int>(quotient(item_start, per));
            const int last = static_cast<int>(quotient(item_start + c.tiles - 1, per));
            int* counter = p.counters + first * p.side_heads + side;
            if (threadIdx.x == 0) last_flag = atomicAdd(counter, 1) == last - first;
            named_bar_sync(1, kConsumers);
            if (last_flag) {
                __threadfence();
                constexpr int kBatch = 10;  // pieces on their way at once
#pragma unroll 1
                for (int e = threadIdx.x; e < rows * kQuads; e += kConsumers) {
                    const int r = e / kQuads, col = 4 * (e % kQuads);
                    Row row;
#pragma unroll 1
                    for (int x0 = first; x0 <= last; x0 += kBatch) {
                        float m[kBatch], l[kBatch];
                        float4 v[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            m[i] = -INFINITY;
                            l[i] = 0.0f;
                            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (x0 + i > last) continue;
                            // the first piece starts at the item's tile 0
                            const float* src =
                                p.partial +
                                (2 * (static_cast<int64_t>(x0 + i) * p.side_heads + side) + (x0 + i == first)) * kPart;
                            m[i] = __ldcg(src + r);
                            l[i] = __ldcg(src + R + r);
                            v[i] = __ldcg(reinterpret_cast<const float4*>(src + 2 * R + r * DP + col));
                        }
                        float top = row.m;
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) top = fmaxf(top, m[i]);
                        float f = weight(row.m, top);
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) {
                            row.add(top, l[i], v[i], f, weight(m[i], top));
                            f = 1.0f;
                        }
                    }
                    store(row, r, col);
                }
                if (threadIdx.x == 0) *counter = 0;  // ready for the next call
            }
        }
        more = next_piece(t_end);
    }
}

template <typename T, int DP, int R, int G>
cudaError_t launch_split_rows(const CUtensorMap (&map)[2], const AttentionArgs& a, int num_sms, cudaStream_t st) {
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(attention_split_kernel<T, DP, R, G>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SplitSmem<DP, R, G>::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    const int ctas = (3 - G) * num_sms / a.side_heads * a.side_heads;
    attention_split_kernel<T, DP, R, G><<<ctas, threads_of(G), SplitSmem<DP, R, G>::kTotal, st>>>(map[0], map[1], a);
    return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t launch_split(const CUtensorMap (&map)[2], const AttentionArgs& a, int num_sms, cudaStream_t st) {
    // as many rows an item as a sequence has, so that its keys are read once
    const int64_t rows = static_cast<int64_t>(a.Tq) * a.group;
    if (rows <= 16 * static_cast<int64_t>(a.batch)) {
        // Two CTAs per SM where they get several items each: one starts and ends an
        // item while the other's keys stream (us, against one CTA, at heads of 128, 8
        // KV heads: 64 sequences of 60 keys 10.6 against 16.4, 256 of 500 96 against
        // 104, 64 of 1 to 4096 87 against 89).  Not where items are cut over the CTAs,
        // into twice as many pieces (16 of 8192 86 against 84, on 1 KV head 27 against
        // 24, 4 of 500 9.8 against 9.5).
        const int64_t items = static_cast<int64_t>(a.batch) * (a.Hk / a.side_heads);
        if (2 * items >= 3 * (num_sms / a.side_heads)) return launch_split_rows<T, DP, 16, 1>(map, a, num_sms, st);
        return launch_split_rows<T, DP, 16, 2>(map, a, num_sms, st);
    }
    if (rows <= 32 * static_cast<int64_t>(a.batch)) return launch_split_rows<T, DP, 32, 2>(map, a, num_sms, st);
    return launch_split_rows<T, DP, 64, 2>(map, a, num_sms, st);
}

// Heads that run side by side: the largest divisor of Hk up to 8.
int side_heads(int Hk) {
    for (int h = 8; h > 1; --h)
        if (Hk % h == 0) return h;
    return 1;
}

}  // namespace

// a counter for each of up to two CTAs per SM
size_t attention_counter_bytes(int num_sms) { return (static_cast<size_t>(num_sms) * 8 + 255) / 256 * 256; }

// two pieces a CTA, of 64 rows, or of 16 where two CTAs run per SM
size_t attention_workspace_bytes(int num_sms) {
    return attention_counter_bytes(num_sms) + static_cast<size_t>(num_sms) * 2 * kPartFloats<128, 64> * 4;
}

// Whether to split the keys over the CTAs rather than run the prompt kernel:
// always up to one MMA tile of rows per sequence (the keys' bytes bound it) and
// where there are no keys, which the split kernel runs without loading any;
// above, by what a key costs.  The prompt kernel takes 7 to 11 ns a key for each
// wave of items (a pair of 128-row tiles per SM), the split kernel 0.13 ns for each
// block of 64 rows, and 2 us more around them; the rule takes 7.  Measured at 40 query heads on 8
// KV heads x 128: 1 sequence x 64 queries over 32768 keys 202 us split against
// 357, 4 x 8 over 32768 163 against 236, 4 x 16 293 against 236, 16 x 8 over
// 4096 98 against 49, 1 x 4 over 512 13.7 against 11.3.
bool attention_splits(const AttentionArgs& a, int num_sms) {
    const int64_t rows = static_cast<int64_t>(a.Tq) * a.group, batch = a.batch;
    if (rows <= 16 * batch || a.Tk == 0) return true;  // (there is no tensor map of no keys)
    if (a.group > 128 || a.Tk < 1024 * batch) return a.group > 128;
    const int64_t blocks = (rows + 64 * batch - 1) / (64 * batch) * batch * a.Hk;
    const int64_t tokens = 2 * (128 / a.group);  // of an item of the prompt kernel
    const int64_t items = (a.Tq + tokens * batch - 1) / (tokens * batch) * batch * a.Hk;
    return blocks < 54 * ((items + num_sms - 1) / num_sms);
}

cudaError_t encode_heads(void* encode_fn, CUtensorMap* map, char name, const void* ptr, int dtype, int rows, int heads,
                         int dim, int64_t token, int64_t head, int box_heads, int box_rows, char* detail, size_t n) {
    cuuint64_t dims[3] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(token) * 2};
    cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(encode_fn)(
        map, dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
        const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return cudaSuccess;
    snprintf(detail, n, "cuTensorMapEncodeTiled(%c: %d x %d x %d) returned %d", name, rows, heads, dim,
             static_cast<int>(r));
    return cudaErrorInvalidValue;
}

cudaError_t launch_attention_split(const AttentionArgs& args, int dtype, int num_sms, void* workspace, void* encode_fn,
                                   cudaStream_t st, char* detail, size_t n) {
    AttentionArgs a = args;
    a.counters = static_cast<int*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attention_counter_bytes(num_sms));
    a.side_heads = side_heads(a.Hk);
    // rows of an item x 32 (16) quads of columns, over the 256 threads of a CTA
    const int64_t rows = (static_cast<int64_t>(a.Tq) * a.group + a.batch - 1) / a.batch;
    a.join_rounds = static_cast<int>(((rows < 64 ? rows : 64) * (a.D <= 64 ? 16 : 32) + 255) / 256);
    CUtensorMap map[2] = {};  // without keys, nothing is loaded
    if (a.Tk > 0) {
        cudaError_t e = encode_heads(encode_fn, &map[0], 'K', a.k, dtype, a.Tk, a.Hk, a.D, a.k_token, a.k_head, 1,
                                     kTile, detail, n);
        if (e == cudaSuccess)
            e = encode_heads(encode_fn, &map[1], 'V', a.v, dtype, a.Tk, a.Hk, a.D, a.v_token, a.v_head, 1, kTile,
                             detail, n);
        if (e != cudaSuccess) return e;
    }
    if (dtype == kBf16)
        return a.D <= 64 ? launch_split<__nv_bfloat16, 64>(map, a, num_sms, st)
                         : launch_split<__nv_bfloat16, 128>(map, a, num_sms, st);
    return a.D <= 64 ? launch_split<__half, 64>(map, a, num_sms, st) : launch_split<__half, 128>(map, a, num_sms, st);
}

cudaError_t attention_split_read_device_error(unsigned int* code) {
    unsigned int v = 0, z = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_device_error, sizeof v);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyToSymbol(g_device_error, &z, sizeof z);
    *code = v;
    return e;
}

}  // namespace w8a8

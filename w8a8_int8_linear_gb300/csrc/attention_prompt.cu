// Attention of many queries per sequence on the tensor cores (tcgen05):
// O = softmax(scale Q K^T) V per sequence and head, causal or full, heads in
// groups over the KV heads.
//
// A CTA owns two tiles of 128 packed rows of one KV head.  Row r of a
// sequence is (query r / G, head r % G of the group), so a group's heads share
// the keys that pass through shared memory, short sequences still fill tiles,
// and a causal tile spans 128 / G positions.  Keys stream in tiles of 128.
// For tile t and key tile j
//   S = Q_t K_j^T        operands in shared memory, S (128 x 128, binary32) in TMEM
//   P = 2^(scale log2(e) S - M), in the inputs' type, over S's own columns
//   O_t += P V_j         P from TMEM, V_j (keys x D, D contiguous) as the
//                        MN-major operand, O_t in TMEM
// Roles: warps 0-3 and 4-7 are the softmax of tile 0 and 1 (one thread per
// row, which also loads Q and finishes O), warp 8 issues the MMAs, warp 9 the
// TMA loads, warps 10-11 clean V (below).  While one tile's softmax runs, the
// other tile's two products run: PV_0(j) S_0(j+1) PV_1(j) S_1(j+1).  MMAs of
// one thread execute in order, so S_t(j+1) may overwrite P_t(j), and the commit
// after S_t(j+1) also says that O_t holds all products up to j.
//
// M is any reference near the row's maximum: softmax does not change with
// it.  It moves only when a score exceeds it by more than 2^8 in weight; only
// then is O_t rescaled (by the softmax threads, between products).  Sums and O
// stay binary32; P's rounding to 16 bits is half a step of each weight, as in
// the output.
//
// A weight of 0 does not hide a non-finite V (0 * inf = NaN).  In the key tiles
// that some row does not see completely, warps 10-11 therefore replace the
// non-finite values of V by 0 before the product; if one of them belonged to
// the sequence, the rows that do see it get it added at the end.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstdio>
#include <type_traits>

#include "attention.cuh"
#include "pair16.cuh"
#include "ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kTileRows = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kKeyTile = 128;
constexpr int kThreads = 384;
constexpr float kSlack = 8.0f;  // log2 of the weight that moves the reference
constexpr int kChunkBytes = 128 * 128;  // 128 rows of 64 16-bit elements

template <int DP>
struct PromptSmem {
    static constexpr int kChunks = DP / 64;
    static constexpr int kTileBytes = kChunks * kChunkBytes;  // a Q, K or V tile
    static constexpr int kStages = DP == 128 ? 5 : 8;
    static constexpr int kPipe = 2 * kTileBytes;
    static constexpr int kBars = kPipe + kStages * kTileBytes;
    static constexpr int kTotal = kBars + 384 + 1024;  // and room to align to 1024
};

struct Bars {
    uint64_t kv_full[8], kv_empty[8];
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    // the V tiles to be cleaned: issued (so that the stage's barrier is in this
    // load's phase, not an older one of the same parity) and done; a slot per V
    // in the ring, as the cleaners run up to three tiles ahead of the products
    uint64_t v_issued[4], v_clean[4];
    uint32_t tmem;
    int bad;
};
static_assert(sizeof(Bars) <= 384, "barriers fit their room");

__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// 128-byte-swizzled operand whose M/N elements are contiguous (V as the
// second product's B: N = D): 64 elements per 128-byte row, rows are keys.
// Leading byte offset: from one 64-wide column block to the next; stride byte
// offset: from 8 keys to the next 8.
__device__ __forceinline__ uint64_t smem_desc_mnmajor_sw128(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
    d |= static_cast<uint64_t>(kChunkBytes >> 4) << 16;
    d |= static_cast<uint64_t>(1024u >> 4) << 32;
    d |= static_cast<uint64_t>(1u) << 46;
    d |= static_cast<uint64_t>(2u) << 61;
    return d;
}

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

// Byte offset of 16-byte chunk ch of row r in a tile as TMA writes it.
__device__ __forceinline__ uint32_t tile_at(int r, int ch) {
    return static_cast<uint32_t>((ch >> 3) * kChunkBytes + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}

// The item of this CTA: rows [row0, row0 + 256) of KV head hk of sequence s.
// A sequence's items run from its last rows (the most keys) to its first.
struct Item {
    bool any;
    Sequence s;
    int hk, row0;
};

__device__ __forceinline__ Item find_item(const AttentionArgs& p, int index) {
    const int lane = threadIdx.x & 31;
    Item it{};
    int64_t before = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        int64_t mine = 0;
        if (b0 + lane < p.batch) {
            const Sequence s = sequence(p, b0 + lane);
            mine = (static_cast<int64_t>(s.n) * p.group + kItemRows - 1) / kItemRows * p.Hk;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl > index);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int local = static_cast<int>(index - (before + __shfl_sync(0xffffffffu, incl - mine, l)));
            const int blocks = static_cast<int>(__shfl_sync(0xffffffffu, mine, l)) / p.Hk;
            it.any = true;
            it.s = sequence(p, b0 + l);
            it.hk = local % p.Hk;
            it.row0 = (blocks - 1 - local / p.Hk) * kItemRows;
            return it;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return it;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const AttentionArgs p) {
    extern __shared__ uint8_t raw[];
    using L = PromptSmem<DP>;
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + L::kBars);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const Item it = find_item(p, blockIdx.x);
    if (!it.any) return;  // the whole CTA
    const Sequence s = it.s;
    const int rows_end = s.n * p.group;  // packed rows of the sequence
    auto limit = [&](int pr) {  // keys that packed row pr sees: [0, limit)
        return p.causal ? clampi(pr / p.group + s.m - s.n + 1, 0, s.m) : s.m;
    };
    int tiles[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = it.row0 + t * kTileRows;
        const int last = min(first + kTileRows, rows_end) - 1;
        tiles[t] = first <= last ? (limit(last) + kKeyTile - 1) / kKeyTile : 0;
    }
    const int jmax = max(tiles[0], tiles[1]);
    const int edge = limit(it.row0) / kKeyTile;  // key tiles from here on are not seen completely by every row

    if (warp == 8) {
        if (lane == 0) {
            for (int i = 0; i < L::kStages; ++i) {
                mbar_init(&bars->kv_full[i], 1);
                mbar_init(&bars->kv_empty[i], 1);
            }
            for (int t = 0; t < 2; ++t) {
                mbar_init(&bars->q_full[t], 4);
                mbar_init(&bars->s_full[t], 1);
                mbar_init(&bars->p_full[t], 4);
                mbar_init(&bars->o_full[t], 1);
            }
            for (int i = 0; i < 4; ++i) {
                mbar_init(&bars->v_issued[i], 1);
                mbar_init(&bars->v_clean[i], 2);
            }
            bars->bad = 0;
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

    if (warp >= 8) {
        regs_dec<72>();
        if (warp == 9) {
            // ---- TMA producer: K_0 V_0 K_1 V_1 ...
            if (elect_one_sync()) {
                tma_prefetch_desc(&tmK);
                tma_prefetch_desc(&tmV);
                int ld = 0;
                for (; ld < 2 * jmax; ++ld) {
                    const int st = ld % L::kStages;
                    if (ld >= L::kStages && !mbar_wait(&bars->kv_empty[st], (ld / L::kStages - 1) & 1, 60)) break;
                    mbar_arrive_expect_tx(&bars->kv_full[st], L::kTileBytes);
                    const void* map = (ld & 1) ? static_cast<const void*>(&tmV) : static_cast<const void*>(&tmK);
#pragma unroll
                    for (int c = 0; c < L::kChunks; ++c)
                        tma_load_3d(pipe + st * L::kTileBytes + c * kChunkBytes, map, &bars->kv_full[st], 64 * c,
                                    it.hk, s.k0 + (ld >> 1) * kKeyTile);
                    if ((ld & 1) && (ld >> 1) >= edge) mbar_arrive(&bars->v_issued[((ld >> 1) - edge) & 3]);
                }
                // nothing is in flight into this CTA's shared memory when it ends
                for (int i = max(0, ld - L::kStages); i < ld; ++i)
                    mbar_wait(&bars->kv_full[i % L::kStages], (i / L::kStages) & 1, 60);
            }
        } else if (warp == 8) {
            // ---- MMA issuer
            const bool leader = elect_one_sync();
            auto scores = [&](int t, int ld) {
                if (!leader) return;
                const uint32_t a = smem_u32(smem) + t * L::kTileBytes;
                const uint32_t b = pipe + (ld % L::kStages) * L::kTileBytes;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const uint32_t at = (k >> 2) * kChunkBytes + (k & 3) * 32;
                    mma_bf16_ss(tmem + t * 128, smem_desc_kmajor_sw128(a + at), smem_desc_kmajor_sw128(b + at),
                                prompt_idesc<T>(kKeyTile, false), k > 0);
                }
                mma_commit(&bars->s_full[t]);
            };
            bool ok = jmax > 0 && mbar_wait(&bars->kv_full[0], 0, 61);
            for (int t = 0; t < 2 && ok; ++t)
                if (tiles[t] > 0) {
                    ok = mbar_wait(&bars->q_full[t], 0, 62);
                    tc_fence_after();
                    if (ok) scores(t, 0);
                }
            // a stage is released only to a load that will come
            if (ok && leader && L::kStages < 2 * jmax) mma_commit(&bars->kv_empty[0]);
            for (int j = 0; j < jmax && ok; ++j) {
                const int lv = 2 * j + 1, lk = 2 * j + 2;
                ok = mbar_wait(&bars->kv_full[lv % L::kStages], (lv / L::kStages) & 1, 63);
                if (ok && j >= edge) ok = mbar_wait(&bars->v_clean[(j - edge) & 3], ((j - edge) >> 2) & 1, 64);
                if (ok && j + 1 < jmax) ok = mbar_wait(&bars->kv_full[lk % L::kStages], (lk / L::kStages) & 1, 65);
                for (int t = 0; t < 2 && ok; ++t) {
                    if (j >= tiles[t]) continue;
                    ok = mbar_wait(&bars->p_full[t], j & 1, 66);
                    if (!ok) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t b = pipe + (lv % L::kStages) * L::kTileBytes;
#pragma unroll
                        for (int k = 0; k < kKeyTile / 16; ++k)
                            mma_f16_ts(tmem + 256 + t * 128, tmem + t * 128 + 8 * k,
                                       smem_desc_mnmajor_sw128(b + k * 2048), prompt_idesc<T>(DP, true), j + k > 0);
                    }
                    if (j + 1 < tiles[t]) scores(t, lk);
                    else if (leader) mma_commit(&bars->o_full[t]);
                }
                if (ok && leader) {
                    if (lv + L::kStages < 2 * jmax) mma_commit(&bars->kv_empty[lv % L::kStages]);
                    if (lk + L::kStages < 2 * jmax) mma_commit(&bars->kv_empty[lk % L::kStages]);
                }
            }
        } else {
            // ---- V cleaners: key tiles from `edge` on
            const int me = threadIdx.x - 320;  // 0..63
            bool ok = true;
            for (int j = edge; j < jmax && ok; ++j) {
                const int lv = 2 * j + 1;
                ok = mbar_wait(&bars->v_issued[(j - edge) & 3], ((j - edge) >> 2) & 1, 67) &&
                     mbar_wait(&bars->kv_full[lv % L::kStages], (lv / L::kStages) & 1, 67);
                if (!ok) break;
                const uint32_t v = pipe + (lv % L::kStages) * L::kTileBytes;
#pragma unroll 4
                for (int c = me; c < L::kTileBytes / 16; c += 64) {
                    uint4 w;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                 : "r"(v + 16 * c));
                    if (any_non_finite<T>(w)) {
                        constexpr uint32_t e = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
                        uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if ((u[i] & e) == e) u[i] &= 0xFFFF0000u;
                            if (((u[i] >> 16) & e) == e) u[i] &= 0x0000FFFFu;
                        }
                        asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(v + 16 * c), "r"(u[0]),
                                     "r"(u[1]), "r"(u[2]), "r"(u[3])
                                     : "memory");
                        const int key = j * kKeyTile + ((c >> 3) & 127);
                        if (key < s.m) *reinterpret_cast<volatile int*>(&bars->bad) = 1;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->v_clean[(j - edge) & 3]);
            }
        }
    } else {
        // ---- softmax, one thread per row
        regs_inc<208>();
        const int t = warp >> 2, wq = warp & 3;
        const int pr = it.row0 + t * kTileRows + wq * 32 + lane;
        const bool valid = pr < rows_end;
        const int query = pr / p.group, head = it.hk * p.group + (pr - query * p.group);
        const int lim = valid ? limit(pr) : 0;
        const int warp_lim = __reduce_min_sync(0xffffffffu, valid ? lim : s.m);
        const uint32_t qtile = smem_u32(smem) + t * L::kTileBytes;
        const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
        const uint32_t ts = tmem + lanes + t * 128, to = tmem + lanes + 256 + t * 128;
        constexpr int kRowChunks = DP / 8, kRowsAtOnce = 32 / kRowChunks;
        const int sub = lane / kRowChunks, ch = lane % kRowChunks;

        {  // Q rows of this warp
            const int64_t at = static_cast<int64_t>(s.q0 + query) * p.q_token + static_cast<int64_t>(head) * p.q_head;
#pragma unroll 8
            for (int r0 = 0; r0 < 32; r0 += kRowsAtOnce) {
                const int r = r0 + sub;
                const int64_t src = __shfl_sync(0xffffffffu, at, r);
                const bool take = __shfl_sync(0xffffffffu, valid, r) && 8 * ch < p.D;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (take) w = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) + src + 8 * ch);
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(qtile + tile_at(wq * 32 + r, ch)),
                             "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w)
                             : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->q_full[t]);
        }

        const float c = p.scale_log2;
        const uint64_t c2 = f2_pack(c, c);
        float ref = -INFINITY;
        uint64_t sum2 = f2_pack(0.0f, 0.0f);
        bool ok = true;
        for (int j = 0; j < tiles[t]; ++j) {
            ok = mbar_wait(&bars->s_full[t], j & 1, 68);
            if (!ok) break;
            tc_fence_after();
            uint32_t v[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, v[i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_wait_ld_regs32(v[i]);
            const int left = lim - j * kKeyTile;  // columns this row sees
            if (warp_lim < (j + 1) * kKeyTile) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int x = 0; x < 32; ++x)
                        if (32 * i + x >= left) v[i][x] = 0xFF800000u;  // -inf
            }
            float m0 = -INFINITY, m1 = -INFINITY, m2 = -INFINITY, m3 = -INFINITY;
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
                m0 = max3(m0, __uint_as_float(v[0][x]), __uint_as_float(v[0][x + 1]));
                m1 = max3(m1, __uint_as_float(v[1][x]), __uint_as_float(v[1][x + 1]));
                m2 = max3(m2, __uint_as_float(v[2][x]), __uint_as_float(v[2][x + 1]));
                m3 = max3(m3, __uint_as_float(v[3][x]), __uint_as_float(v[3][x + 1]));
            }
            const float top = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * c;
            if (j == 0) {
                ref = top;
            } else {
                const bool moves = top > ref + kSlack;  // also from -inf
                if (__any_sync(0xffffffffu, moves)) {
                    const float f = moves ? exp2_approx(ref - top) : 1.0f;
                    if (moves) ref = top;
                    const uint64_t f2 = f2_pack(f, f);
                    sum2 = f2_mul(sum2, f2);
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
            const float base = ref == -INFINITY ? 0.0f : -ref;
            const uint64_t base2 = f2_pack(base, base);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[16];
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                    float a, b;
                    f2_unpack(f2_fma(f2_pack(__uint_as_float(v[i][x]), __uint_as_float(v[i][x + 1])), c2, base2), a, b);
                    a = exp2_approx(a);
                    b = exp2_approx(b);
                    sum2 = f2_add(sum2, f2_pack(a, b));
                    w[x >> 1] = Pair16<T>::pack(a, b);
                }
                tmem_st_32x32b_x16(ts + 16 * i, w);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_full[t]);
        }

        // ---- O / sum, through this warp's rows of the Q tile, to memory
        float l0, l1;
        f2_unpack(sum2, l0, l1);
        const float l = l0 + l1;
        if (tiles[t] > 0 && ok) ok = mbar_wait(&bars->o_full[t], 0, 69);
        tc_fence_after();
        const int bad = tiles[t] > 0 ? *reinterpret_cast<volatile int*>(&bars->bad) : 0;
        const float inv = lim > 0 ? __frcp_rn(l) : 0.0f;
        if (ok) {
#pragma unroll 1
            for (int i = 0; i < DP / 16; ++i) {
                uint32_t o[16];
                if (tiles[t] > 0) {
                    tmem_ld_32x32b_x16(to + 16 * i, o);
                    tmem_wait_ld_regs(o);
                }
                if (bad) {
                    for (int key = edge * kKeyTile; key < lim; ++key) {
                        const T* src = static_cast<const T*>(p.v) + static_cast<int64_t>(s.k0 + key) * p.v_token +
                                       static_cast<int64_t>(it.hk) * p.v_head + 16 * i;
#pragma unroll
                        for (int x = 0; x < 16; ++x) {
                            if (16 * i + x >= p.D) continue;
                            const float val = static_cast<float>(src[x]);
                            if (!isfinite(val)) o[x] = __float_as_uint(__uint_as_float(o[x]) + val);
                        }
                    }
                }
                uint32_t w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    w[x] = lim > 0 ? Pair16<T>::pack(__uint_as_float(o[2 * x]) * inv, __uint_as_float(o[2 * x + 1]) * inv)
                                   : 0u;
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     qtile + tile_at(wq * 32 + lane, 2 * i + h)),
                                 "r"(w[4 * h]), "r"(w[4 * h + 1]), "r"(w[4 * h + 2]), "r"(w[4 * h + 3])
                                 : "memory");
            }
            __syncwarp();
            const int64_t at = static_cast<int64_t>(s.q0 + query) * p.o_token + static_cast<int64_t>(head) * p.o_head;
#pragma unroll 4
            for (int r0 = 0; r0 < 32; r0 += kRowsAtOnce) {
                const int r = r0 + sub;
                const int64_t dst = __shfl_sync(0xffffffffu, at, r);
                const bool take = __shfl_sync(0xffffffffu, valid, r) && 8 * ch < p.D;
                uint4 w;
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                             : "r"(qtile + tile_at(wq * 32 + r, ch))
                             : "memory");
                if (take) *reinterpret_cast<uint4*>(static_cast<T*>(p.o) + dst + 8 * ch) = w;
            }
            if (p.lse && valid)
                p.lse[static_cast<int64_t>(s.q0 + query) * p.Hq + head] =
                    lim > 0 ? ((ref == -INFINITY ? 0.0f : ref) + log2f(l)) * kLn2 : -INFINITY;
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <typename T, int DP>
cudaError_t launch_prompt_typed(const CUtensorMap& tmK, const CUtensorMap& tmV, const AttentionArgs& a, int grid,
                                cudaStream_t st) {
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
    attention_prompt_kernel<T, DP><<<grid, kThreads, PromptSmem<DP>::kTotal, st>>>(tmK, tmV, a);
    return cudaGetLastError();
}

}  // namespace

bool attention_prompt_takes(const AttentionArgs& a) {
    // TMA strides are positive and below 2^40 bytes
    const int64_t s[4] = {a.k_token, a.k_head, a.v_token, a.v_head};
    for (int64_t v : s)
        if (v <= 0 || v >= int64_t(1) << 39) return false;
    const int64_t items = (static_cast<int64_t>(a.Tq) * a.group / kItemRows + a.batch) * a.Hk;
    return a.Tk > 0 && items <= INT32_MAX && static_cast<int64_t>(a.Tq) * a.group <= INT32_MAX;
}

cudaError_t launch_attention_prompt(const AttentionArgs& a, int dtype, void* encode_fn, cudaStream_t st, char* detail,
                                    size_t n) {
    auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(encode_fn);
    CUtensorMap map[2];
    for (int i = 0; i < 2; ++i) {
        const void* ptr = i ? a.v : a.k;
        const int64_t token = i ? a.v_token : a.k_token, head = i ? a.v_head : a.k_head;
        cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.D), static_cast<cuuint64_t>(a.Hk),
                              static_cast<cuuint64_t>(a.Tk)};
        cuuint64_t strides[2] = {static_cast<cuuint64_t>(head) * 2, static_cast<cuuint64_t>(token) * 2};
        cuuint32_t box[3] = {64, 1, kKeyTile};
        cuuint32_t estr[3] = {1, 1, 1};
        const CUresult r = encode(&map[i], dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                                  3, const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
        if (r != CUDA_SUCCESS) {
            snprintf(detail, n, "cuTensorMapEncodeTiled(%s: %d x %d x %d) returned %d", i ? "V" : "K", a.Tk, a.Hk, a.D,
                     static_cast<int>(r));
            return cudaErrorInvalidValue;
        }
    }
    // an upper bound on the items of any split of the rows into sequences
    const int grid = static_cast<int>((static_cast<int64_t>(a.Tq) * a.group / kItemRows + a.batch) * a.Hk);
    if (dtype == kBf16)
        return a.D <= 64 ? launch_prompt_typed<__nv_bfloat16, 64>(map[0], map[1], a, grid, st)
                         : launch_prompt_typed<__nv_bfloat16, 128>(map[0], map[1], a, grid, st);
    return a.D <= 64 ? launch_prompt_typed<__half, 64>(map[0], map[1], a, grid, st)
                     : launch_prompt_typed<__half, 128>(map[0], map[1], a, grid, st);
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

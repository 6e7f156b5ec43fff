// Attention of a few queries per sequence over long caches:
// o_i = sum_j softmax_j(scale q_i k_j) v_j with grouped heads.
//
// One query of a group of G heads reads each K and V value once for G
// multiply-adds, so the keys' bytes bound it: the G heads (and the n queries)
// that share a KV head form the rows of one or two warp MMA tiles (16 x 16 x 8)
// and the keys stream through shared memory once.
//
// The row blocks of all sequences are laid end to end, each as its tiles of 64
// keys, and cut into equal ranges whatever the lengths are; the lengths stay on
// the device.  CTA c takes range c / Hk for KV head c mod Hk, so that the CTAs
// that run side by side read the neighbouring heads of the same keys (whole
// rows of the cache).  Within a CTA each warp runs its own online softmax over
// its own 16 keys of every tile (no barrier while keys stream), and the four
// are joined at the end of an item.  An item that spans CTAs leaves (max, sum,
// unnormalized output) per piece in the workspace; the CTA that arrives last
// joins the pieces in key order, so the result does not depend on the order of
// arrival.
//
//   softmax:  t = scale log2(e) s;  running max M, sum L, O in binary32,
//             p = 2^(t - M); P enters the second product rounded to the
//             inputs' type (half a step, 2^-8 for bf16, of each p: the same
//             size as the output's own rounding, the sums stay binary32).
#include <cfloat>
#include <type_traits>

#include "attention.cuh"
#include "pair16.cuh"
#include "ptx.cuh"

namespace w8a8 {

namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;      // keys of a warp per tile
constexpr int kTile = kWarps * kKeys;
constexpr int kStages = 3;

// R: packed (query, head) rows of an item, 16 or 32.
template <int DP, int R>
struct SplitSmem {
    static constexpr int kStageBytes = 2 * kKeys * DP * 2;  // K and V of one warp
    static constexpr int kPipe = kWarps * kStages * kStageBytes;
    static constexpr int kQ = R * DP * 2;
    static constexpr int kJoin = kWarps * R * (DP + 2) * 4;  // reuses the pipe
    static constexpr int kTotal = (kPipe > kJoin ? kPipe : kJoin) + kQ;
};

// Byte offset of 16-byte chunk c of row r in a [rows][DP] tile: chunks
// permuted by the row, so that eight rows of one chunk column fall into
// different banks.
template <int DP>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

// Partial result of one piece of an item: [R] maxima, [R] sums, [R][DP] outputs.
template <int DP, int R>
constexpr int kPartFloats = R * (DP + 2);

// Where a linear tile index lies: sequence, row block, tile of the block.
struct Cursor {
    int b;
    Sequence s;
    int blocks;    // R-row blocks of the sequence
    int tiles;     // key tiles of one block
    int block;
    int tile;
};

template <int R>
__device__ __forceinline__ int blocks_of(const AttentionArgs& p, const Sequence& s) {
    return static_cast<int>((static_cast<int64_t>(s.n) * p.group + R - 1) / R);
}
__device__ __forceinline__ int tiles_of(const Sequence& s) { return max(1, (s.m + kTile - 1) / kTile); }

// Tiles of the 32 sequences from b0 on: this lane's, and inclusive over the lanes.
template <int R>
__device__ __forceinline__ void tiles_from(const AttentionArgs& p, int b0, int64_t& mine, int64_t& incl) {
    const int lane = threadIdx.x & 31;
    mine = 0;
    if (b0 + lane < p.batch) {
        const Sequence s = sequence(p, b0 + lane);
        mine = static_cast<int64_t>(blocks_of<R>(p, s)) * tiles_of(s);
    }
    incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
}

template <typename T, int DP, int R>
__global__ void __launch_bounds__(kWarps * 32, 2) attention_split_kernel(const AttentionArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int last_flag;
    using L = SplitSmem<DP, R>;
    constexpr int kMT = R / 16;       // MMA tiles of rows
    constexpr int kChunks = DP / 8;   // 16-byte chunks of a row
    constexpr int kDT = DP / 8;       // 8-wide output column tiles
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dchunks = p.D >> 3;
    uint8_t* q_smem = smem + L::kTotal - L::kQ;
    uint8_t* pipe = smem + warp * kStages * L::kStageBytes;
    float* join = reinterpret_cast<float*>(smem);

    const int hk = blockIdx.x % p.Hk, range = blockIdx.x / p.Hk, ranges = gridDim.x / p.Hk;
    // all tiles, by every warp on its own; the first 32 sequences' counts stay
    int64_t mine, incl;
    tiles_from<R>(p, 0, mine, incl);
    int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    for (int b0 = 32; b0 < p.batch; b0 += 32) {
        int64_t m2, i2;
        tiles_from<R>(p, b0, m2, i2);
        total += __shfl_sync(0xffffffffu, i2, 31);
    }
    const int64_t per = max(static_cast<int64_t>(p.min_tiles), (total + ranges - 1) / ranges);
    int64_t w = per * range;
    const int64_t w_end = min(total, w + per);
    if (w >= w_end) return;
    Cursor c;
    {  // the cursor of tile w
        int64_t left = w;
        for (int b0 = 0;; b0 += 32) {
            if (b0 > 0) tiles_from<R>(p, b0, mine, incl);
            const unsigned hit = __ballot_sync(0xffffffffu, incl > left);
            if (hit) {
                const int l = __ffs(hit) - 1;
                left -= __shfl_sync(0xffffffffu, incl - mine, l);
                c.b = b0 + l;
                break;
            }
            left -= __shfl_sync(0xffffffffu, incl, 31);
        }
        c.s = sequence(p, c.b);
        c.blocks = blocks_of<R>(p, c.s);
        c.tiles = tiles_of(c.s);
        c.block = static_cast<int>(left / c.tiles);
        c.tile = static_cast<int>(left - static_cast<int64_t>(c.block) * c.tiles);
    }

    while (w < w_end) {
        // ---- one piece: tiles [c.tile, t_end) of row block c.block of sequence c.b
        const int t_begin = c.tile;
        const int t_end = static_cast<int>(min(static_cast<int64_t>(c.tiles), t_begin + (w_end - w)));
        const int64_t item_start = w - t_begin;
        const int rb = c.block;
        const Sequence s = c.s;
        const int rows = min(R, s.n * p.group - rb * R);
        const T* kbase = static_cast<const T*>(p.k) + static_cast<int64_t>(hk) * p.k_head;
        const T* vbase = static_cast<const T*>(p.v) + static_cast<int64_t>(hk) * p.v_head;

        // keys a packed row may see: [0, lim)
        auto limit = [&](int r) {
            if (r >= rows) return 0;
            const int i = (rb * R + r) / p.group;
            return p.causal ? clampi(i + s.m - s.n + 1, 0, s.m) : s.m;
        };
        const int lim_top = limit(rows - 1), lim_low = limit(0);

        auto issue = [&](int t) {
            const int key0 = t * kTile + warp * kKeys;
            if (t < t_end && key0 < lim_top) {
                uint8_t* st = pipe + ((t - t_begin) % kStages) * L::kStageBytes;
#pragma unroll
                for (int u = lane; u < kKeys * kChunks; u += 32) {
                    const int r = u / kChunks, ch = u % kChunks;
                    const int key = key0 + r;
                    const bool take = key < lim_top && ch < dchunks;
                    const int64_t tok = s.k0 + (take ? key : 0);
                    const int col = take ? 8 * ch : 0;
                    const T* ks = kbase + (take ? tok * p.k_token + col : 0);
                    const T* vs = vbase + (take ? tok * p.v_token + col : 0);
                    cp_async16(smem_u32(st) + swz<DP>(r, ch), ks, take);
                    cp_async16(smem_u32(st) + kKeys * DP * 2 + swz<DP>(r, ch), vs, take);
                }
            }
            cp_async_commit();
        };

        __syncthreads();  // the previous piece's join is done
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(t_begin + i);
        // Q rows to shared memory while the first keys are on their way
        for (int u = threadIdx.x; u < R * kChunks; u += kWarps * 32) {
            const int r = u / kChunks, ch = u % kChunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && ch < dchunks) {
                const int pr = rb * R + r, i = pr / p.group, g = pr - i * p.group;
                v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                    static_cast<int64_t>(s.q0 + i) * p.q_token +
                                                    static_cast<int64_t>(hk * p.group + g) * p.q_head + 8 * ch);
            }
            *reinterpret_cast<uint4*>(q_smem + swz<DP>(r, ch)) = v;
        }
        __syncthreads();
        uint32_t qf[kMT][DP / 16][4];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk)
                ldmatrix4(qf[mt][kk], smem_u32(q_smem) + swz<DP>(16 * mt + (lane & 15), 2 * kk + (lane >> 4)));

        float o[kMT][kDT][4], mx[kMT][2], sum[kMT][2];
        int lim[kMT][2];
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt) {
#pragma unroll
            for (int j = 0; j < kDT; ++j) o[mt][j][0] = o[mt][j][1] = o[mt][j][2] = o[mt][j][3] = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mx[mt][h] = -INFINITY;
                sum[mt][h] = 0.0f;
                lim[mt][h] = limit(16 * mt + (lane >> 2) + 8 * h);
            }
        }
        for (int t = t_begin; t < t_end; ++t) {
            __syncwarp();  // every lane is done with the stage that issue() refills
            issue(t + kStages - 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const int key0 = t * kTile + warp * kKeys;
            if (key0 >= lim_top) continue;
            const uint32_t ks = smem_u32(pipe + ((t - t_begin) % kStages) * L::kStageBytes);
            const uint32_t vs = ks + kKeys * DP * 2;
            float sc[kMT][2][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
                for (int j = 0; j < 2; ++j) sc[mt][j][0] = sc[mt][j][1] = sc[mt][j][2] = sc[mt][j][3] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                uint32_t kf[4];
                ldmatrix4(kf, ks + swz<DP>((lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) {
                    mma16816<T>(sc[mt][0], qf[mt][kk], kf[0], kf[1]);
                    mma16816<T>(sc[mt][1], qf[mt][kk], kf[2], kf[3]);
                }
            }
            const int col = key0 + 2 * (lane & 3);
            // A key that only some of the rows see must not reach the others
            // through 0 * inf: such a tile with a non-finite V goes key by key.
            bool apart = false;
            if (key0 + kKeys > lim_low) {
                bool bad = false;
                for (int u = lane; u < kKeys * kChunks; u += 32) {
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(vs + swz<DP>(u / kChunks, u % kChunks)));
                    bad |= any_non_finite<T>(v);
                }
                apart = __any_sync(0xffffffffu, bad);
            }
            uint32_t pf[kMT][4];
#pragma unroll
            for (int mt = 0; mt < kMT; ++mt) {
                float tm[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[mt][j][e] =
                            col + 8 * j + (e & 1) < lim[mt][e >> 1] ? sc[mt][j][e] * p.scale_log2 : -INFINITY;
                        tm[e >> 1] = fmaxf(tm[e >> 1], sc[mt][j][e]);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 1));
                    tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 2));
                }
                const bool grows = tm[0] > mx[mt][0] || tm[1] > mx[mt][1];
                if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float m = fmaxf(mx[mt][h], tm[h]);
                        const float f = m == mx[mt][h] ? 1.0f : exp2_approx(mx[mt][h] - m);
                        mx[mt][h] = m;
                        sum[mt][h] *= f;
#pragma unroll
                        for (int j = 0; j < kDT; ++j) {
                            o[mt][j][2 * h] *= f;
                            o[mt][j][2 * h + 1] *= f;
                        }
                    }
                }
                const float base[2] = {mx[mt][0] == -INFINITY ? 0.0f : mx[mt][0],
                                       mx[mt][1] == -INFINITY ? 0.0f : mx[mt][1]};
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sc[mt][j][e] = exp2_approx(sc[mt][j][e] - base[e >> 1]);
                        sum[mt][e >> 1] += sc[mt][j][e];
                    }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        pf[mt][2 * j + h] = Pair16<T>::pack(sc[mt][j][2 * h], sc[mt][j][2 * h + 1]);
            }
            if (!apart) {
#pragma unroll
                for (int j = 0; j < kDT; j += 2) {
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, vs + swz<DP>((lane & 7) + ((lane >> 3) & 1) * 8, j + (lane >> 4)));
#pragma unroll
                    for (int mt = 0; mt < kMT; ++mt) {
                        mma16816<T>(o[mt][j], pf[mt], vf[0], vf[1]);
                        mma16816<T>(o[mt][j + 1], pf[mt], vf[2], vf[3]);
                    }
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt)
#pragma unroll 1
                    for (int k = 0; k < kKeys; ++k) {
                        // p of rows lane/4 and lane/4 + 8 at key k
                        const int from = (lane & ~3) | ((k & 7) >> 1);
                        auto pick = [&](int e) {
                            const float even = k & 8 ? sc[mt][1][e] : sc[mt][0][e];
                            const float odd = k & 8 ? sc[mt][1][e + 1] : sc[mt][0][e + 1];
                            return __shfl_sync(0xffffffffu, k & 1 ? odd : even, from);
                        };
                        const float p0 = pick(0), p1 = pick(2);
                        const bool s0 = key0 + k < lim[mt][0], s1 = key0 + k < lim[mt][1];
#pragma unroll
                        for (int j = 0; j < kDT; ++j) {
                            uint32_t w32;
                            asm volatile("ld.shared.u32 %0, [%1];"
                                         : "=r"(w32)
                                         : "r"(vs + swz<DP>(k, j) + 4 * (lane & 3)));
                            const float2 v = Pair16<T>::unpack(w32);
                            if (s0) {
                                o[mt][j][0] = fmaf(p0, v.x, o[mt][j][0]);
                                o[mt][j][1] = fmaf(p0, v.y, o[mt][j][1]);
                            }
                            if (s1) {
                                o[mt][j][2] = fmaf(p1, v.x, o[mt][j][2]);
                                o[mt][j][3] = fmaf(p1, v.y, o[mt][j][3]);
                            }
                        }
                    }
            }
        }
        cp_async_wait<0>();
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                sum[mt][h] += __shfl_xor_sync(0xffffffffu, sum[mt][h], 1);
                sum[mt][h] += __shfl_xor_sync(0xffffffffu, sum[mt][h], 2);
            }

        // ---- join the four warps
        __syncthreads();
        float* jm = join + warp * R * (DP + 2);
        float* jl = jm + R;
        float* jo = jl + R;
#pragma unroll
        for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = 16 * mt + 8 * h + (lane >> 2);
                if ((lane & 3) == 0) {
                    jm[r] = mx[mt][h];
                    jl[r] = sum[mt][h];
                }
#pragma unroll
                for (int j = 0; j < kDT; ++j)
                    *reinterpret_cast<float2*>(jo + r * DP + 8 * j + 2 * (lane & 3)) =
                        make_float2(o[mt][j][2 * h], o[mt][j][2 * h + 1]);
            }
        __syncthreads();

        // thread: row threadIdx.x / kPer, columns in pairs kPer apart
        constexpr int kPer = kWarps * 32 / R, kPairs = DP / 2 / kPer;
        const int jr = threadIdx.x / kPer, jc = 2 * (threadIdx.x % kPer);
        const bool whole = t_begin == 0 && t_end == c.tiles;
        float om = -INFINITY, ol = 0.0f;
        float2 ov[kPairs];
        auto clear = [&]() {
            om = -INFINITY;
            ol = 0.0f;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) ov[i] = make_float2(0.0f, 0.0f);
        };
        auto join_into = [&](float m, float l, const float2(&v)[kPairs]) {
            const float nm = fmaxf(om, m);
            const float f0 = om == nm ? 1.0f : exp2_approx(om - nm);
            const float f1 = m == nm ? 1.0f : exp2_approx(m - nm);
            ol = ol * f0 + l * f1;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                ov[i].x = ov[i].x * f0 + v[i].x * f1;
                ov[i].y = ov[i].y * f0 + v[i].y * f1;
            }
            om = nm;
        };
        clear();
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float* pm = join + x * R * (DP + 2);
            float2 v[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                v[i] = *reinterpret_cast<const float2*>(pm + 2 * R + jr * DP + jc + 2 * kPer * i);
            join_into(pm[jr], pm[R + jr], v);
        }

        auto store = [&]() {
            if (jr >= rows) return;
            const int pr = rb * R + jr, i = pr / p.group, g = pr - i * p.group, head = hk * p.group + g;
            const bool sees = limit(jr) > 0;
            const float inv = sees ? __frcp_rn(ol) : 0.0f;  // a row that sees keys of no weight is 0 / 0
            T* dst = static_cast<T*>(p.o) + static_cast<int64_t>(s.q0 + i) * p.o_token +
                     static_cast<int64_t>(head) * p.o_head;
#pragma unroll
            for (int x = 0; x < kPairs; ++x) {
                const int cc = jc + 2 * kPer * x;
                if (cc < p.D)
                    *reinterpret_cast<uint32_t*>(dst + cc) =
                        sees ? Pair16<T>::pack(ov[x].x * inv, ov[x].y * inv) : 0u;
            }
            if (p.lse && jc == 0)
                p.lse[static_cast<int64_t>(s.q0 + i) * p.Hq + head] = sees ? (om + log2f(ol)) * kLn2 : -INFINITY;
        };

        if (whole) {
            store();
        } else {
            // this piece's partial result, then the last piece to arrive joins all
            constexpr int kPart = kPartFloats<DP, R>;
            float* part = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (t_begin == 0 ? 1 : 0)) * kPart;
            if (jc == 0) {
                part[jr] = om;
                part[R + jr] = ol;
            }
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                *reinterpret_cast<float2*>(part + 2 * R + jr * DP + jc + 2 * kPer * i) = ov[i];
            __threadfence();
            __syncthreads();
            const int first = static_cast<int>(item_start / per);
            const int last = static_cast<int>((item_start + c.tiles - 1) / per);
            int* counter = p.counters + first * p.Hk + hk;
            if (threadIdx.x == 0) last_flag = atomicAdd(counter, 1) == last - first;
            __syncthreads();
            if (last_flag) {
                __threadfence();
                clear();
#pragma unroll (R == 16 ? 4 : 1)
                for (int x = first; x <= last; ++x) {
                    // the first piece starts at the item's tile 0
                    const float* src = p.partial + (2 * (static_cast<int64_t>(x) * p.Hk + hk) + (x == first)) * kPart;
                    float2 v[kPairs];
#pragma unroll
                    for (int i = 0; i < kPairs; ++i)
                        v[i] = __ldcg(reinterpret_cast<const float2*>(src + 2 * R + jr * DP + jc + 2 * kPer * i));
                    join_into(__ldcg(src + jr), __ldcg(src + R + jr), v);
                }
                store();
                if (threadIdx.x == 0) *counter = 0;  // ready for the next call
            }
        }

        // ---- next row block
        w += t_end - t_begin;
        c.tile = 0;
        if (++c.block >= c.blocks) {
            c.block = 0;
            do {
                if (++c.b >= p.batch) return;
                c.s = sequence(p, c.b);
                c.blocks = blocks_of<R>(p, c.s);
                c.tiles = tiles_of(c.s);
            } while (c.blocks == 0);
        }
    }
}

template <typename T, int DP, int R>
cudaError_t launch_split_rows(const AttentionArgs& a, int ctas, cudaStream_t st) {
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(attention_split_kernel<T, DP, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SplitSmem<DP, R>::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    attention_split_kernel<T, DP, R><<<ctas, kWarps * 32, SplitSmem<DP, R>::kTotal, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int DP>
cudaError_t launch_split(const AttentionArgs& a, int ctas, cudaStream_t st) {
    // two MMA tiles of rows where a sequence has more than 16: its keys are read half as often
    return static_cast<int64_t>(a.Tq) * a.group > 16 * static_cast<int64_t>(a.batch)
               ? launch_split_rows<T, DP, 32>(a, ctas, st)
               : launch_split_rows<T, DP, 16>(a, ctas, st);
}

// Two CTAs per SM, a whole number of key ranges (one at least) for all KV heads.
int split_ctas(int num_sms, int Hk) { return 2 * num_sms / Hk > 0 ? 2 * num_sms / Hk * Hk : Hk; }

}  // namespace

size_t attention_counter_bytes(int num_sms) { return (static_cast<size_t>(2 * num_sms) * 4 + 255) / 256 * 256; }

size_t attention_workspace_bytes(int num_sms) {
    return attention_counter_bytes(num_sms) + static_cast<size_t>(2 * num_sms) * 2 * kPartFloats<128, 32> * 4;
}

cudaError_t launch_attention(const AttentionArgs& args, int dtype, int num_sms, void* workspace, cudaStream_t st) {
    AttentionArgs a = args;
    a.counters = static_cast<int*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attention_counter_bytes(num_sms));
    a.min_tiles = 2;
    // (with more KV heads than CTAs there is one range: no piece, no partial result)
    const int ctas = split_ctas(num_sms, a.Hk);
    if (dtype == kBf16)
        return a.D <= 64 ? launch_split<__nv_bfloat16, 64>(a, ctas, st) : launch_split<__nv_bfloat16, 128>(a, ctas, st);
    return a.D <= 64 ? launch_split<__half, 64>(a, ctas, st) : launch_split<__half, 128>(a, ctas, st);
}

}  // namespace w8a8

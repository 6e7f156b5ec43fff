// Attention of a few queries per sequence over long caches (and, slowly, any
// other): o_i = sum_j softmax_j(scale q_i k_j) v_j with grouped heads.
//
// One query of a group of G heads reads each K and V value once for G
// multiply-adds, so the keys' bytes bound it: the G heads (and the n queries)
// that share a KV head form the rows of one warp MMA tile (16 x 16 x 8), and
// the keys stream through shared memory once.
//
// The keys of all sequences, KV heads and 16-row blocks are laid end to end
// in tiles of 64 and cut into equal ranges, one per CTA, whatever the lengths
// are; the lengths stay on the device.  Within a CTA each warp runs its own
// online softmax over its own 16 keys of every tile (no barrier while keys
// stream), and the four are joined at the end of an item.  An item that spans
// CTAs leaves (max, sum, unnormalized output) per piece in the workspace; the
// CTA that arrives last joins the pieces in key order, so the result does not
// depend on the order of arrival.
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
constexpr int kRows = 16;      // packed (query, head) rows of an item
constexpr int kKeys = 16;      // keys of a warp per tile
constexpr int kTile = kWarps * kKeys;
constexpr int kStages = 3;

template <int DP>
struct SplitSmem {
    static constexpr int kStageBytes = 2 * kKeys * DP * 2;  // K and V of one warp
    static constexpr int kPipe = kWarps * kStages * kStageBytes;
    static constexpr int kQ = kRows * DP * 2;
    static constexpr int kJoin = kWarps * kRows * (DP + 2) * 4;  // reuses the pipe
    static constexpr int kTotal = (kPipe > kJoin ? kPipe : kJoin) + kQ;
};

// Byte offset of 16-byte chunk c of row r in a [rows][DP] tile: chunks
// permuted by the row, so that eight rows of one chunk column fall into
// different banks.
template <int DP>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return static_cast<uint32_t>(r * DP * 2 + ((c ^ (r & 7)) << 4));
}

// Partial result of one piece of an item: [kRows] maxima, [kRows] sums,
// [kRows][DP] outputs.
template <int DP>
constexpr int kPartFloats = kRows * (DP + 2);

// Where a linear tile index lies: sequence, item, tile of the item.
struct Cursor {
    int b;
    Sequence s;
    int blocks;    // 16-row blocks of the sequence
    int tiles;     // tiles of one item
    int item;      // kv_head * blocks + block
    int tile;
};

struct Shape {
    int64_t items;  // per sequence
    int blocks, tiles;
};

__device__ __forceinline__ Shape shape_of(const AttentionArgs& p, const Sequence& s) {
    Shape r;
    r.blocks = (s.n * p.group + kRows - 1) / kRows;
    r.tiles = max(1, (s.m + kTile - 1) / kTile);
    r.items = static_cast<int64_t>(r.blocks) * p.Hk;
    return r;
}

// Sum of all tiles, by every warp on its own.
__device__ __forceinline__ int64_t total_tiles(const AttentionArgs& p) {
    int64_t w = 0;
    for (int b = threadIdx.x & 31; b < p.batch; b += 32) {
        const Shape s = shape_of(p, sequence(p, b));
        w += s.items * s.tiles;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w;
}

// The cursor of linear tile w < total.
__device__ __forceinline__ Cursor locate(const AttentionArgs& p, int64_t w) {
    const int lane = threadIdx.x & 31;
    int64_t before = 0;
    Cursor c{};
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
        int64_t mine = 0;
        if (b0 + lane < p.batch) {
            const Shape s = shape_of(p, sequence(p, b0 + lane));
            mine = s.items * s.tiles;
        }
        int64_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += t;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, before + incl > w);
        if (hit) {
            const int l = __ffs(hit) - 1;
            const int64_t start = before + __shfl_sync(0xffffffffu, incl - mine, l);
            c.b = b0 + l;
            c.s = sequence(p, c.b);
            const Shape s = shape_of(p, c.s);
            c.blocks = s.blocks;
            c.tiles = s.tiles;
            c.item = static_cast<int>((w - start) / s.tiles);
            c.tile = static_cast<int>((w - start) - static_cast<int64_t>(c.item) * s.tiles);
            return c;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
    }
    c.b = -1;
    return c;
}

template <typename T, int DP>
__global__ void __launch_bounds__(kWarps * 32, 2) attention_split_kernel(const AttentionArgs p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int last_flag;
    using L = SplitSmem<DP>;
    constexpr int kChunks = DP / 8;   // 16-byte chunks of a row
    constexpr int kDT = DP / 8;       // 8-wide output column tiles
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int dchunks = p.D >> 3;
    uint8_t* q_smem = smem + L::kTotal - L::kQ;
    uint8_t* pipe = smem + warp * kStages * L::kStageBytes;
    float* join = reinterpret_cast<float*>(smem);

    const int64_t total = total_tiles(p);
    const int64_t per = max(static_cast<int64_t>(p.min_tiles), (total + gridDim.x - 1) / gridDim.x);
    int64_t w = per * blockIdx.x;
    const int64_t w_end = min(total, w + per);
    if (w >= w_end) return;
    Cursor c = locate(p, w);

    while (w < w_end && c.b >= 0) {
        // ---- one piece: tiles [c.tile, t_end) of item c.item of sequence c.b
        const int t_begin = c.tile;
        const int t_end = static_cast<int>(min(static_cast<int64_t>(c.tiles), t_begin + (w_end - w)));
        const int64_t item_start = w - t_begin;
        const int hk = c.item / c.blocks, rb = c.item - hk * c.blocks;
        const Sequence s = c.s;
        const int rows = min(kRows, s.n * p.group - rb * kRows);
        const T* kbase = static_cast<const T*>(p.k) + static_cast<int64_t>(hk) * p.k_head;
        const T* vbase = static_cast<const T*>(p.v) + static_cast<int64_t>(hk) * p.v_head;

        // keys a packed row may see: [0, lim)
        auto limit = [&](int r) {
            if (r >= rows) return 0;
            const int i = (rb * kRows + r) / p.group;
            return p.causal ? clampi(i + s.m - s.n + 1, 0, s.m) : s.m;
        };
        const int lim_top = limit(rows - 1), lim_low = limit(0);

        // Q rows to shared memory
        __syncthreads();  // the previous piece's join is done
        for (int u = threadIdx.x; u < kRows * kChunks; u += kWarps * 32) {
            const int r = u / kChunks, ch = u % kChunks;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < rows && ch < dchunks) {
                const int pr = rb * kRows + r, i = pr / p.group, g = pr - i * p.group;
                v = *reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                    static_cast<int64_t>(s.q0 + i) * p.q_token +
                                                    static_cast<int64_t>(hk * p.group + g) * p.q_head + 8 * ch);
            }
            *reinterpret_cast<uint4*>(q_smem + swz<DP>(r, ch)) = v;
        }
        __syncthreads();
        uint32_t qf[DP / 16][4];
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
            ldmatrix4(qf[kk], smem_u32(q_smem) + swz<DP>(lane & 15, 2 * kk + (lane >> 4)));

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

        float o[kDT][4];
#pragma unroll
        for (int j = 0; j < kDT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.0f, 0.0f};
        const int lim[2] = {limit(lane >> 2), limit((lane >> 2) + 8)};

#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) issue(t_begin + i);
        for (int t = t_begin; t < t_end; ++t) {
            __syncwarp();  // every lane is done with the stage that issue() refills
            issue(t + kStages - 1);
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const int key0 = t * kTile + warp * kKeys;
            if (key0 >= lim_top) continue;
            const uint32_t ks = smem_u32(pipe + ((t - t_begin) % kStages) * L::kStageBytes);
            const uint32_t vs = ks + kKeys * DP * 2;
            float sc[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
                uint32_t kf[4];
                ldmatrix4(kf, ks + swz<DP>((lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
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
            if (!apart) {
                const uint32_t pf[4] = {Pair16<T>::pack(sc[0][0], sc[0][1]), Pair16<T>::pack(sc[0][2], sc[0][3]),
                                        Pair16<T>::pack(sc[1][0], sc[1][1]), Pair16<T>::pack(sc[1][2], sc[1][3])};
#pragma unroll
                for (int j = 0; j < kDT; j += 2) {
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, vs + swz<DP>((lane & 7) + ((lane >> 3) & 1) * 8, j + (lane >> 4)));
                    mma16816<T>(o[j], pf, vf[0], vf[1]);
                    mma16816<T>(o[j + 1], pf, vf[2], vf[3]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kKeys; ++k) {
                    // p of rows lane/4 and lane/4 + 8 at key k
                    const int from = (lane & ~3) | ((k & 7) >> 1);
                    const float p0 = __shfl_sync(0xffffffffu, sc[k >> 3][k & 1], from);
                    const float p1 = __shfl_sync(0xffffffffu, sc[k >> 3][2 + (k & 1)], from);
                    const bool s0 = key0 + k < lim[0], s1 = key0 + k < lim[1];
#pragma unroll
                    for (int j = 0; j < kDT; ++j) {
                        uint32_t w32;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w32) : "r"(vs + swz<DP>(k, j) + 4 * (lane & 3)));
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
        cp_async_wait<0>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 1);
            sum[h] += __shfl_xor_sync(0xffffffffu, sum[h], 2);
        }

        // ---- join the four warps: thread (row, column) pairs
        __syncthreads();
        float* jm = join + warp * kRows * (DP + 2);
        float* jl = jm + kRows;
        float* jo = jl + kRows;
        const int r0 = lane >> 2;
        if ((lane & 3) == 0) {
            jm[r0] = mx[0];
            jm[r0 + 8] = mx[1];
            jl[r0] = sum[0];
            jl[r0 + 8] = sum[1];
        }
#pragma unroll
        for (int j = 0; j < kDT; ++j) {
            const int cc = 8 * j + 2 * (lane & 3);
            *reinterpret_cast<float2*>(jo + r0 * DP + cc) = make_float2(o[j][0], o[j][1]);
            *reinterpret_cast<float2*>(jo + (r0 + 8) * DP + cc) = make_float2(o[j][2], o[j][3]);
        }
        __syncthreads();

        // rows [threadIdx.x / 8], columns in 8 interleaved groups of DP / 8
        const int jr = threadIdx.x >> 3, jc = threadIdx.x & 7;
        const bool whole = t_begin == 0 && t_end == c.tiles;
        float om = -INFINITY, ol = 0.0f, ov[DP / 8];
        auto join_into = [&](float m, float l, auto load) {
            const float nm = fmaxf(om, m);
            const float f0 = om == nm ? 1.0f : exp2_approx(om - nm);
            const float f1 = m == nm ? 1.0f : exp2_approx(m - nm);
            ol = ol * f0 + l * f1;
#pragma unroll
            for (int i = 0; i < DP / 8; i += 2) {
                const float2 v = load(jc * 2 + i * 8);
                ov[i] = ov[i] * f0 + v.x * f1;
                ov[i + 1] = ov[i + 1] * f0 + v.y * f1;
            }
            om = nm;
        };
#pragma unroll
        for (int i = 0; i < DP / 8; ++i) ov[i] = 0.0f;
#pragma unroll
        for (int x = 0; x < kWarps; ++x) {
            const float* pm = join + x * kRows * (DP + 2);
            const float* po = pm + 2 * kRows + jr * DP;
            join_into(pm[jr], pm[kRows + jr], [&](int i) { return *reinterpret_cast<const float2*>(po + i); });
        }

        auto store = [&]() {
            if (jr >= rows) return;
            const int pr = rb * kRows + jr, i = pr / p.group, g = pr - i * p.group, head = hk * p.group + g;
            const bool sees = limit(jr) > 0;
            const float inv = sees ? __frcp_rn(ol) : 0.0f;  // a row that sees keys of no weight is 0 / 0
            T* dst = static_cast<T*>(p.o) + static_cast<int64_t>(s.q0 + i) * p.o_token +
                     static_cast<int64_t>(head) * p.o_head;
#pragma unroll
            for (int x = 0; x < DP / 8; x += 2) {
                const int cc = jc * 2 + x * 8;
                if (cc < p.D)
                    *reinterpret_cast<uint32_t*>(dst + cc) =
                        sees ? Pair16<T>::pack(ov[x] * inv, ov[x + 1] * inv) : 0u;
            }
            if (p.lse && jc == 0)
                p.lse[static_cast<int64_t>(s.q0 + i) * p.Hq + head] = sees ? (om + log2f(ol)) * kLn2 : -INFINITY;
        };

        if (whole) {
            store();
        } else {
            // this piece's partial result, then the last piece to arrive joins all
            float* part = p.partial + (2 * static_cast<int64_t>(blockIdx.x) + (t_begin == 0 ? 1 : 0)) * kPartFloats<DP>;
            if (jc == 0) {
                part[jr] = om;
                part[kRows + jr] = ol;
            }
#pragma unroll
            for (int i = 0; i < DP / 8; i += 2)
                *reinterpret_cast<float2*>(part + 2 * kRows + jr * DP + jc * 2 + i * 8) = make_float2(ov[i], ov[i + 1]);
            __threadfence();
            __syncthreads();
            const int first = static_cast<int>(item_start / per);
            const int last = static_cast<int>((item_start + c.tiles - 1) / per);
            if (threadIdx.x == 0)
                last_flag = atomicAdd(p.counters + first, 1) == last - first;
            __syncthreads();
            if (last_flag) {
                __threadfence();
                om = -INFINITY;
                ol = 0.0f;
#pragma unroll
                for (int i = 0; i < DP / 8; ++i) ov[i] = 0.0f;
                for (int x = first; x <= last; ++x) {
                    // the first piece starts at the item's tile 0
                    const float* src = p.partial + (2 * static_cast<int64_t>(x) + (x == first ? 1 : 0)) * kPartFloats<DP>;
                    const float* so = src + 2 * kRows + jr * DP;
                    join_into(__ldcg(src + jr), __ldcg(src + kRows + jr),
                              [&](int i) { return __ldcg(reinterpret_cast<const float2*>(so + i)); });
                }
                store();
                if (threadIdx.x == 0) p.counters[first] = 0;  // ready for the next call
            }
        }

        // ---- next item
        w += t_end - t_begin;
        c.tile = 0;
        if (++c.item >= c.blocks * p.Hk) {
            c.item = 0;
            do {
                if (++c.b >= p.batch) {
                    c.b = -1;
                    break;
                }
                c.s = sequence(p, c.b);
                const Shape sh = shape_of(p, c.s);
                c.blocks = sh.blocks;
                c.tiles = sh.tiles;
            } while (c.blocks == 0);
        }
    }
}

template <typename T, int DP>
cudaError_t launch_split(const AttentionArgs& a, int ctas, cudaStream_t st) {
    static bool set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev]) {
        e = cudaFuncSetAttribute(attention_split_kernel<T, DP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SplitSmem<DP>::kTotal);
        if (e != cudaSuccess) return e;
        if (dev < 64) set[dev] = true;
    }
    attention_split_kernel<T, DP><<<ctas, kWarps * 32, SplitSmem<DP>::kTotal, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t attention_counter_bytes(int num_sms) { return (static_cast<size_t>(2 * num_sms) * 4 + 255) / 256 * 256; }

size_t attention_workspace_bytes(int num_sms) {
    return attention_counter_bytes(num_sms) + static_cast<size_t>(2 * num_sms) * 2 * kPartFloats<128> * 4;
}

cudaError_t launch_attention(const AttentionArgs& args, int dtype, int num_sms, void* workspace, cudaStream_t st) {
    AttentionArgs a = args;
    a.counters = static_cast<int*>(workspace);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + attention_counter_bytes(num_sms));
    a.min_tiles = 4;
    const int ctas = 2 * num_sms;
    if (dtype == kBf16)
        return a.D <= 64 ? launch_split<__nv_bfloat16, 64>(a, ctas, st) : launch_split<__nv_bfloat16, 128>(a, ctas, st);
    return a.D <= 64 ? launch_split<__half, 64>(a, ctas, st) : launch_split<__half, 128>(a, ctas, st);
}

}  // namespace w8a8

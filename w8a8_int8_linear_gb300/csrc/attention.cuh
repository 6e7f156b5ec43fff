// What the attention kernels share: the sequences' bounds as the device holds
// them, and warp-level tensor-core building blocks.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "operators.h"
#include "ptx.cuh"

namespace w8a8 {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Sequence b: queries [q0, q0 + n) and keys [k0, k0 + m) of the packed rows.
// Offsets and lengths come from device memory and are clamped to the tensors'
// rows, so that no value in them can make a kernel read or write out of range.
struct Sequence {
    int q0, n, k0, m;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// a / b for positive a and b, in 32 bits where a allows.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if ((a | b) >> 32 == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

template <bool kPaged = false>
__device__ __forceinline__ Sequence sequence(const AttentionArgs& p, int b) {
    Sequence s;
    if (p.cu_q) {
        s.q0 = clampi(p.cu_q[b], 0, p.Tq);
        s.n = clampi(p.cu_q[b + 1], s.q0, p.Tq) - s.q0;
    } else {
        s.n = p.Tq / p.batch;
        s.q0 = b * s.n;
    }
    if (kPaged) {
        s.k0 = 0;
        s.m = clampi(p.k_lens[b], 0, p.max_pages * p.page_size);
        return s;
    }
    if (p.cu_k) {
        s.k0 = clampi(p.cu_k[b], 0, p.Tk);
        s.m = clampi(p.cu_k[b + 1], s.k0, p.Tk) - s.k0;
    } else {
        s.m = p.Tk / p.batch;
        s.k0 = b * s.m;
    }
    if (p.k_lens) s.m = clampi(p.k_lens[b], 0, s.m);
    return s;
}

// 3-D tiled load into this CTA's shared memory (`smem_dst` a shared address).
__device__ __forceinline__ void tma_load_3d(uint32_t smem_dst, const void* tmap, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// Page `index` of sequence b, for an index of one of its keys; one that is not in the
// cache comes as `pages`, where copies read zeros.
__device__ __forceinline__ unsigned entry_of(const AttentionArgs& p, int b, unsigned index) {
    return static_cast<unsigned>(__ldg(p.page_table + static_cast<int64_t>(b) * p.table_stride + index));
}
__device__ __forceinline__ int page_of(const AttentionArgs& p, unsigned entry) {
    return static_cast<int>(min(entry, static_cast<unsigned>(p.pages)));
}

// Copy of a box of one page into this CTA's shared memory.
__device__ __forceinline__ void tma_load_page(uint32_t smem_dst, const void* tmap, uint64_t* bar, int32_t c0,
                                              int32_t head, int32_t row, int32_t page) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(head), "r"(row), "r"(page)
        : "memory");
}

// Where the boxes of a sequence's key tiles (of kTile keys) lie, by a warp: lane i has
// box i of a tile.  The entry of a box is on its way for a tile's time before it is
// used, and there are no divisions.
template <int kTile>
struct Boxes {
    int boxes;            // of a tile
    int key, index, row;  // of this lane's box of the next tile
    int pages, rest;      // a tile's keys by the page, and what is left of them
    int m, b;
    int left, first_key, first_index, first_row;  // tiles up to the last; the box of the first
    unsigned entry;       // of the next tile's box
    int page, at_row;     // of the present one's

    __device__ __forceinline__ void look_up(const AttentionArgs& p) {
        entry = ~0u;  // past the keys: no page
        if (threadIdx.x % 32 < boxes && key < m) entry = entry_of(p, b, index);
    }
    __device__ __forceinline__ void place(const AttentionArgs& p) {
        index = static_cast<unsigned>(key) / static_cast<unsigned>(p.page_size);
        row = key - index * p.page_size;
    }
    // for `count` tiles of sequence `seq` with `keys` keys: tiles first + turn, ... to the
    // last, then from `first` on
    __device__ __forceinline__ void start(const AttentionArgs& p, int seq, int keys, int first, int count, int turn) {
        boxes = kTile / p.box;
        b = seq;
        m = keys;
        first_key = key = first * kTile + static_cast<int>(threadIdx.x % 32) * p.box;
        place(p);
        first_index = index;
        first_row = row;
        if (turn > 0) {
            key += turn * kTile;
            place(p);
        }
        left = count - turn;
        pages = kTile / p.page_size;
        rest = kTile - pages * p.page_size;
        look_up(p);
    }
    // on to the next tile
    __device__ __forceinline__ void step(const AttentionArgs& p) {
        page = page_of(p, entry);
        at_row = row;
        key += kTile;
        row += rest;
        index += pages;
        if (row >= p.page_size) {
            row -= p.page_size;
            ++index;
        }
        if (--left == 0) {
            key = first_key;
            index = first_index;
            row = first_row;
        }
        look_up(p);
    }
    // copy(i, row, page) for every box i, by one thread (the copies of several threads
    // go one by one, and slowly)
    template <typename F>
    __device__ __forceinline__ void each(F copy) const {
        constexpr int kAtOnce = 4;
        for (int i0 = 0; i0 < boxes; i0 += kAtOnce) {
            int pg[kAtOnce], rw[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                pg[i] = __shfl_sync(0xffffffffu, page, i0 + i);
                rw[i] = __shfl_sync(0xffffffffu, at_row, i0 + i);
            }
            if (elect_one_sync()) {
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i)
                    if (i == 0 || i0 + i < boxes) copy(i0 + i, rw[i], pg[i]);
            }
        }
    }
};

// 32 lanes x 16 consecutive 32-bit columns from registers.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// d (16 x 8, binary32) += a (16 x 16) b (16 x 8).
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether any of the eight 16-bit floats in w is infinite or NaN: the
// magnitude plus one in the exponent's last place carries into the sign bit.
template <typename T>
__device__ __forceinline__ bool any_non_finite(const uint4& w) {
    constexpr uint32_t one = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    const uint32_t m = 0x7FFF7FFFu;
    return ((((w.x & m) + one) | ((w.y & m) + one) | ((w.z & m) + one) | ((w.w & m) + one)) & 0x80008000u) != 0;
}

}  // namespace
}  // namespace w8a8

// fp8bs_mx_tile.h -- what the two matrix kernels share: copies into LDS, the barrier, the
// tiles of a launch and their order.  Device code, included by fp8bs_mx_gemm.hip and
// fp8bs_mx_grad.hip only.
#pragma once
#include "fp8bs_mx.h"

namespace fp8bs {
namespace mx {
namespace {

#define LDS_AS __attribute__((address_space(3)))

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(LDS_AS const void*)p;
}

// 16 bytes per lane from buffer offset voff + soff to LDS bytes lds + 16 * lane.  The five
// wait states cover a scalar register written by the vector unit just before, and M0 (a
// reserved register that nothing else here uses: LDS instructions do not need it).
template <bool ONCE = false>
__device__ __forceinline__ void copy16(const i32x4& buffer, uint32_t voff, uint32_t soff,
                                       uint32_t lds) {
    // (uniform values all, which not every control flow lets the compiler see)
    const i32x4 b = {__builtin_amdgcn_readfirstlane(buffer[0]), __builtin_amdgcn_readfirstlane(buffer[1]),
                     __builtin_amdgcn_readfirstlane(buffer[2]), __builtin_amdgcn_readfirstlane(buffer[3])};
    const uint32_t at = __builtin_amdgcn_readfirstlane(soff), to = __builtin_amdgcn_readfirstlane(lds);
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen nt lds"
                     :: "v"(voff), "s"(b), "s"(at), "s"(to));
    else
        asm volatile("s_mov_b32 m0, %3\n\ts_nop 4\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                     :: "v"(voff), "s"(b), "s"(at), "s"(to));
}
// every copy, load and store of this wavefront done, then the workgroup meets
__device__ __forceinline__ void wait_and_meet() {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

struct Tile {
    int g;              // expert (weight group)
    int slot;           // masked: slot of A and D; else 0
    int m0, n0;         // first row (of the slot) and first output column
    int rows;           // rows of the slot that may be read, from m0
    int c0, c1;         // steps along the contraction
};

__device__ __forceinline__ int expert_of(const MxParams& p, int block) {
    const int e = p.group_data[block * 128];
    return e >= 0 && e < p.num_groups ? e : -1;
}

// Masked: whether a slot holds more rows than the few-rows kernel takes (all slots then go to the
// tiled kernels; asked by whole wavefronts).
__device__ __forceinline__ bool any_slot_over(const MxParams& p) {
    bool over = false;
    for (int w = 0; w < p.num_groups; w += 64) {
        const int g = w + (int)(threadIdx.x & 63);
        over = over || __any(g < p.num_groups && min(p.group_data[g], p.m) > p.few);
    }
    return over;
}

// The tiles along M that hold a valid row, listed in LDS by one wavefront; returns how many.
// Contiguous: block number * 2 + whether the next 128-row block, of the same expert, belongs
// to the tile (256-row tiles pair the blocks of a run of one expert).  Masked: slot *
// m_tiles + tile.
template <int BM, int LAYOUT>
__device__ int list_tiles(const MxParams& p, uint32_t* list) {
    const int lane = threadIdx.x & 63;
    int count = 0;
    if constexpr (LAYOUT == kContiguous) {
        int run = p.first, before = -2;               // start and expert of the run so far
        for (int w = p.first; w < p.last; w += 64) {
            const int b = w + lane;
            const int e = b < p.last ? expert_of(p, b) : -1;
            const int after = b + 1 < p.last ? expert_of(p, b + 1) : -1;
            const int prev = __shfl_up(e, 1, 64);
            const uint64_t starts = __ballot(e != (lane ? prev : before));
            const uint64_t upto = starts & (lane == 63 ? ~0ull : (2ull << lane) - 1ull);
            const int first = upto ? w + 63 - __clzll(upto) : run;
            const bool head = e >= 0 && (BM < 256 || ((b - first) & 1) == 0);
            const uint64_t heads = __ballot(head);
            if (head)
                list[count + __popcll(heads & ((1ull << lane) - 1ull))] =
                    (uint32_t)(2 * b + (BM >= 256 && after == e ? 1 : 0));
            count += __popcll(heads);
            run = starts ? w + 63 - __clzll(starts) : run;
            before = __shfl(e, 63, 64);
        }
    } else {
        for (int w = p.first; w < p.last; w += 64) {
            const int i = w + lane;
            const int g = min(i, p.last - 1) / p.m_tiles;
            const bool in = i < p.last && (i - g * p.m_tiles) * BM < min(p.group_data[g], p.m);
            const uint64_t heads = __ballot(in);
            if (in) list[count + __popcll(heads & ((1ull << lane) - 1ull))] = (uint32_t)i;
            count += __popcll(heads);
        }
    }
    return count;
}

// Unit u of a launch: a tile of BM rows and COLS output columns.
template <int BM, int COLS, int LAYOUT>
__device__ __forceinline__ void tile_at(const MxParams& p, const uint32_t* list, int m_tiles,
                                        int u, Tile& t) {
    int g = 0;
    if constexpr (LAYOUT == kBlocks) {
        g = u / (m_tiles * p.n_tiles);
        u -= g * (m_tiles * p.n_tiles);
    }
    // groups of `raster` tiles along M sweep the columns
    const int band = u / (p.raster * p.n_tiles);
    const int in_band = u - band * p.raster * p.n_tiles;
    const int first = band * p.raster;
    const int tall = min(p.raster, m_tiles - first);
    const int mt = first + in_band % tall;
    t.n0 = in_band / tall * COLS;
    t.g = g;
    t.slot = 0;
    t.c0 = 0;
    t.c1 = p.chunks;
    if constexpr (LAYOUT == kContiguous) {
        const uint32_t e = __builtin_amdgcn_readfirstlane(list[mt]);
        t.m0 = (int)(e >> 1) * 128;
        t.rows = BM < 256 ? min(BM, 128) : (e & 1) ? 256 : 128;
        t.g = __builtin_amdgcn_readfirstlane(p.group_data[t.m0]);
    } else if constexpr (LAYOUT == kMasked) {
        const int e = (int)__builtin_amdgcn_readfirstlane(list[mt]);
        t.g = t.slot = e / p.m_tiles;
        t.m0 = (e - t.g * p.m_tiles) * BM;
        t.rows = __builtin_amdgcn_readfirstlane(min(p.group_data[t.g], p.m)) - t.m0;
    } else {
        t.m0 = mt * BM;
        t.rows = p.m - t.m0;
        if constexpr (LAYOUT == kBlocks) {
            t.c0 = 2 * __builtin_amdgcn_readfirstlane(p.blocks[g]);
            t.c1 = 2 * __builtin_amdgcn_readfirstlane(p.blocks[g + 1]);
        }
    }
}

}  // namespace
}  // namespace mx
}  // namespace fp8bs

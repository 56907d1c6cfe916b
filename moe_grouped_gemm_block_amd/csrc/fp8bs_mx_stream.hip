// fp8bs_mx_stream.hip -- the MXFP4 product and gated block for few rows (single tokens,
// decode batches, a few slots) on gfx950.
//
// With few rows the weights' bytes are the work, and what bounds it is how fast each CU draws
// its tiles' rows and columns.  A workgroup takes a small tile (16 TM x 16 TN) and its
// wavefronts share the contraction: each multiplies its own run of 256-value steps, brought
// into a ring of its own in LDS by direct-to-LDS copies that read whole 128-byte lines (eight
// rows a copy; fragments loaded straight into registers touch 16 half lines a load and drew
// 27 GB/s per CU against 56: 128 x 4096 x 7168 took 16.9 us instead of 10.5).  Nothing is shared
// until the end, so a wavefront waits for its own copies only; the FP32 partial tiles then
// meet in LDS and are added in a fixed order -- one launch, no workspace, no atomics.  Dense, a
// wavefront takes one run of K; the tile shape, and with it their number, follows from sizes.  The
// tile shape of slots follows from the caller's hint too, so there K is cut into eight runs whatever
// the tile (each of four wavefronts takes two) and their sums are added in the same pairs: every
// shape gives the same bits (0.1 to 1 us a launch slower than four runs).
//
// 1 x 4096 x 7168: 5.7 us, of which 3.7 are there at K = 128 too (launch, sum, store);
// 128 x 2112 x 7168: 10 us (132 tiles of 64 x 32: half of the CUs draw nothing, and K is not split
// over workgroups); 64 x 2048 x 7168 gated, output quantised: 10 us (a quantised output fixes four
// column blocks, so 16-row tiles draw every weight row four times).
//
// Tile row TM * j + i is row j of block i (columns likewise), as in fp8bs_mx_gemm.hip: a lane
// owns 4 TN neighbouring columns and reads its scale words as vectors.  A gated tile has TN / 2
// blocks of the gate and as many of the up projection.
#include <math.h>

#include "fp8bs_mx_tile.h"

namespace fp8bs {
namespace mx {
namespace {

// 16 bytes per lane from each lane's address to LDS bytes lds + 16 * lane
__device__ __forceinline__ void copy16_from(const void* at, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %0, off"
                 :: "v"(at), "s"(__builtin_amdgcn_readfirstlane(lds)));
}
// at most N of this wavefront's copies outstanding
template <int N>
__device__ __forceinline__ void wait_copies() {
    asm volatile("s_waitcnt vmcnt(%0)" :: "n"(N) : "memory");
}

template <int TM, int TN>
struct Ring {
    static constexpr int kWaves = TM + TN <= 4 ? 8 : 4;
    static constexpr int kStep = (TM + TN) * 2048 + 1024;      // bytes: rows, then scale words
    // steps in flight: as many as 160 KB hold, at most three (the waits below tell apart zero, one
    // and two steps behind the one awaited; 16x16 tiles would have room for a fourth)
    static constexpr int kDepth = TM + TN <= 2 ? 3 : TM + TN <= 4 ? 2 : TM + TN <= 6 ? 3 : 2;
    static_assert(kWaves * kStep * kDepth <= 160 * 1024, "LDS of a CU");
};

template <int TM, int TN, int LAYOUT, int EPI>
__global__ void __launch_bounds__((64 * Ring<TM, TN>::kWaves), 1) mx_stream_kernel(const MxParams p) {
    constexpr bool GATED = gated(EPI);
    constexpr int BM = 16 * TM, COLS = GATED ? 8 * TN : 16 * TN;
    constexpr int WAVES = Ring<TM, TN>::kWaves, DEPTH = Ring<TM, TN>::kDepth, STEP = Ring<TM, TN>::kStep;
    constexpr int HALF = TN / 2 > 0 ? TN / 2 : 1;
    constexpr int B_OFF = TM * 2048, S_OFF = (TM + TN) * 2048;
    constexpr int COPIES = 2 * (TM + TN) + 1;                  // of a step
    constexpr int RING_BYTES = WAVES * STEP * DEPTH, PART_BYTES = WAVES * TM * TN * 1024;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[RING_BYTES > PART_BYTES ? RING_BYTES : PART_BYTES];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, q = lane >> 4;

    if (LAYOUT == kMasked && p.few < p.m && any_slot_over(p)) return;

    // ---- the tile: tiles along M of one weight strip are neighbours on one XCD ----
    // (a workgroup for each, unless a launch may not have so many)
    const uint32_t units = (uint32_t)p.m_tiles * p.n_tiles * (LAYOUT == kMasked ? p.num_groups : 1);
    for (uint32_t id = logical_block(); id < units; id += gridDim.x) {
    int mt = id % p.m_tiles;
    const int rest = id / p.m_tiles;
    const int n0 = rest % p.n_tiles * COLS;
    const int g = LAYOUT == kMasked ? rest / p.n_tiles : 0;
    // (kGatedGrad stores zeros in the rows from m to the next multiple of 64)
    const int limit = LAYOUT == kMasked ? min(p.group_data[g], p.m)
                      : EPI == kGatedGrad ? (p.m + 63) & -64 : p.m;
    // (masked: the grid has tiles for the expected rows; a slot with more is walked through)
    for (; mt * BM < limit; mt += p.m_tiles) {
        const int m0 = mt * BM, slot = g;
        const int from = EPI == kGatedGrad ? min(m0, p.m - 1) : m0;    // first row read
        const int rows = (EPI == kGatedGrad ? p.m : limit) - from;

    // ---- operands; rows and columns past the last one repeat it (never stored) ----
    const int64_t group = (int64_t)g * (GATED ? 2 * p.n : p.n);
    const i32x4 a = descriptor(p.a + ((int64_t)slot * p.m + from) * p.a_row, rows * p.a_row);
    const i32x4 b = descriptor(p.b + (group + n0) * p.b_row, (int64_t)(p.n - n0) * p.b_row);
    const i32x4 up = GATED ? descriptor(p.b + (group + n0 + p.n) * p.b_row, (int64_t)(p.n - n0) * p.b_row) : b;
    // copy k of an operand fills LDS rows 8 k .. 8 k + 7: rows 8 (k % 2) .. of block k / 2; the
    // lane's 16-byte unit is permuted by its row as in fp8bs_mx_gemm.hip
    const uint32_t unit = (uint32_t)((lane & 7) ^ (lane >> 3));
    const uint32_t tail_unit = unit >= 4 ? 64u : 0u;           // (see there: half a last step)
    uint32_t a_at[2 * TM], b_at[2 * TN];
#pragma unroll
    for (int k = 0; k < 2 * TM; ++k) {
        const int r = min(TM * (8 * (k & 1) + (lane >> 3)) + k / 2, rows - 1);
        a_at[k] = (uint32_t)r * (uint32_t)p.a_row + 16u * unit;
    }
#pragma unroll
    for (int k = 0; k < 2 * TN; ++k) {
        const int n = k / 2, r = 8 * (k & 1) + (lane >> 3);
        b_at[k] = (uint32_t)min(GATED ? HALF * r + n % HALF : TN * r + n, p.n - 1 - n0) * (uint32_t)p.b_row +
                  16u * unit;
    }
    // scale words: lanes 0 .. 8 TM - 1 bring A's (two word rows of 16 TM), the next 8 TN B's,
    // the rest repeat the first lane's; four words each
    const int32_t* s_from;
    int64_t s_ld;                                              // words from one word row to the next
    bool s_second;
    {
        const bool mine_a = lane < 8 * TM || lane >= 8 * (TM + TN);
        const int l = lane >= 8 * (TM + TN) ? 0 : mine_a ? lane : lane - 8 * TM;
        const int per_row = mine_a ? 4 * TM : 4 * TN;          // lanes of a word row
        s_second = l >= per_row;
        int w = 4 * (l % per_row);
        if (mine_a) {
            s_ld = p.sfa_ld;
            s_from = p.sfa + (int64_t)slot * p.kwords * p.sfa_ld + min(m0 + w, p.sfa_ld - 4);
        } else {
            // a gated tile's words: 8 TN of the gate, then of the up projection
            if (GATED) w = w < COLS ? n0 + w : p.n + n0 + w - COLS;
            else w += n0;
            s_ld = p.sfb_ld;
            s_from = p.sfb + (int64_t)g * p.kwords * p.sfb_ld + min(w, p.sfb_ld - 4);
        }
    }
    const uint32_t lds0 = lds_offset(smem) + (uint32_t)(wave * STEP * DEPTH);
    auto copy_step = [&](int c, int buf) {
        const uint32_t to = lds0 + (uint32_t)(buf * STEP), at = 128u * (uint32_t)c;
        const bool half = 2 * c + 1 >= p.kwords;
        const uint32_t back = half ? tail_unit : 0u;
#pragma unroll
        for (int k = 0; k < 2 * TN; ++k)
            copy16<true>(GATED && k >= TN ? up : b, b_at[k] - back, at, to + (uint32_t)(B_OFF + k * 1024));
        copy16_from(s_from + (2 * c + (s_second && !half ? 1 : 0)) * s_ld, to + (uint32_t)S_OFF);
#pragma unroll
        for (int k = 0; k < 2 * TM; ++k)
            copy16(a, a_at[k] - back, at, to + (uint32_t)(k * 1024));
    };

    constexpr int RUNS = LAYOUT == kMasked ? 8 / WAVES : 1;    // of a wavefront
    auto run_at = [&](int r) { return (int)((int64_t)r * p.chunks / (WAVES * RUNS)); };
    // (accumulators for each: moved aside after the first run, they cost 0.4 us at 64 x 64)
    f32x4 run_sum[RUNS][TM][TN];
#pragma unroll
    for (int run = 0; run < RUNS; ++run)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int n = 0; n < TN; ++n) run_sum[run][i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int c0 = run_at(wave * RUNS), c1 = run_at((wave + 1) * RUNS);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (c0 + d < c1) copy_step(c0 + d, d);
    int buf = 0;
    auto multiply = [&](int c, f32x4 (&acc)[TM][TN]) {
        // the copies of the steps after this one stay in flight
        const int after = min(c1 - 1 - c, DEPTH - 1);
        if (after == 0) wait_copies<0>();
        else if (after == 1) wait_copies<COPIES>();
        else wait_copies<2 * COPIES>();
        const uint8_t* st = smem + (wave * DEPTH + buf) * STEP;
        i32x4 fa[2][TM], fb[2][TN];
        int ea[2][TM], eb[2][TN];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int at = j * 128 + (((4 * h + q) ^ (j & 7)) << 4);
#pragma unroll
            for (int i = 0; i < TM; ++i) fa[h][i] = *(const i32x4*)(st + at + 2048 * i);
#pragma unroll
            for (int n = 0; n < TN; ++n) fb[h][n] = *(const i32x4*)(st + B_OFF + at + 2048 * n);
            const int* sa = (const int*)(st + S_OFF) + h * 16 * TM + TM * j;
            const int* sb = (const int*)(st + S_OFF) + 32 * TM + h * 16 * TN + (GATED ? HALF * j : TN * j);
#pragma unroll
            for (int i = 0; i < TM; ++i) ea[h][i] = sa[i];
#pragma unroll
            for (int n = 0; n < TN; ++n) eb[h][n] = sb[GATED ? n % HALF + n / HALF * COLS : n];
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // read out before it is refilled
        if (c + DEPTH < c1) copy_step(c + DEPTH, buf);
        // (the second round of a row's last step does not exist when K / 128 is odd)
        const int keep = 2 * c + 1 < p.kwords ? 255 : 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    const i32x4 x = fb[h][n], y = fa[h][i];
                    acc[i][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0},
                        i32x8{y[0], y[1], y[2], y[3], 0, 0, 0, 0}, acc[i][n], 4, 4, 0,
                        (eb[h][n] >> (8 * q)) & (h ? keep : 255), 0,
                        (ea[h][i] >> (8 * q)) & (h ? keep : 255));
                }
        buf = buf + 1 == DEPTH ? 0 : buf + 1;
    };
    int c = c0;
    if constexpr (RUNS == 2)
        for (const int end = run_at(wave * 2 + 1); c < end; ++c) multiply(c, run_sum[1]);
    for (; c < c1; ++c) multiply(c, run_sum[0]);

    // ---- the partial tiles, in the rings' place, added in order by the first TM wavefronts (slots:
    // the runs' sums in pairs, (0 + 1) + (2 + 3) + ...) ----
    f32x4* part = (f32x4*)smem;                                // [wave][block][lane]
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int n = 0; n < TN; ++n)
            part[(wave * TM * TN + i * TN + n) * 64 + lane] =
                RUNS == 2 ? run_sum[RUNS - 1][i][n] + run_sum[0][i][n] : run_sum[0][i][n];
    __syncthreads();
    if (wave < TM) {
    constexpr bool PAIRED = LAYOUT == kMasked && RUNS == 1;
    const int i = wave;
    f32x4 sum[TN];
#pragma unroll
    for (int n = 0; n < TN; ++n) {
        auto of = [&](int w) { return part[(w * TM * TN + i * TN + n) * 64 + lane]; };
#pragma unroll
        for (int w = 0; w < WAVES; w += PAIRED ? 2 : 1) {
            const f32x4 next = PAIRED ? of(w) + of(w + 1) : of(w);
            sum[n] = w ? sum[n] + next : next;
        }
    }
    const int r = TM * j + i;
    const bool ok = EPI == kGatedGrad ? m0 + r < p.m : r < rows;
    const int64_t row = (int64_t)slot * p.m + m0 + r;
    if constexpr (!GATED) {
        // columns n0 + TN (4 q + v) + n: 4 TN neighbours
        const int col = n0 + 4 * TN * q;
        uint16_t* d = (uint16_t*)p.d + row * p.d_ld + col;
        if (ok && col + 4 * TN <= p.n && (p.d_ld & (TN == 1 ? 3 : 7)) == 0) {
            uint32_t w[2 * TN];
#pragma unroll
            for (int e = 0; e < 4 * TN; e += 2)
                w[e / 2] = pack_bf16(sum[e % TN][e / TN], sum[(e + 1) % TN][(e + 1) / TN]);
            if constexpr (TN == 1) {
                *(uint2*)d = uint2{w[0], w[1]};
            } else {
#pragma unroll
                for (int e = 0; e < 2 * TN; e += 4)
                    *(u32x4*)(d + 2 * e) = u32x4{w[e], w[e + 1], w[e + 2], w[e + 3]};
            }
        } else if (ok) {
#pragma unroll
            for (int e = 0; e < 4 * TN; ++e)
                if (col + e < p.n) d[e] = to_bf16(sum[e % TN][e / TN]);
        }
    } else {
        // columns n0 + HALF (4 q + v) + n of the gate (blocks below HALF) and the up projection
        constexpr int MINE = 4 * HALF;
        const int col = n0 + MINE * q;
        if constexpr (EPI == kGatedGrad) {
            if (m0 + r < limit && col < p.n) {
                uint32_t dh[MINE / 2] = {}, dg[MINE / 2], du[MINE / 2];
                if (ok) __builtin_memcpy(dh, p.dh + (int64_t)(m0 + r) * p.n + col, 2 * MINE);
#pragma unroll
                for (int e = 0; e < MINE; e += 2) {
                    float gr[2], ur[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int n = (e + x) % HALF, v = (e + x) / HALF;
                        const uint32_t w = dh[e / 2];
                        const float d = __builtin_bit_cast(float, x ? w & 0xFFFF0000u : w << 16);
                        float slope;
                        const float value = activate<true>(p.act, sum[n][v], slope);
                        gr[x] = d * sum[HALF + n][v] * slope;
                        ur[x] = d * value;
                    }
                    dg[e / 2] = ok ? pack_bf16(gr[0], gr[1]) : 0u;
                    du[e / 2] = ok ? pack_bf16(ur[0], ur[1]) : 0u;
                }
                uint16_t* to = (uint16_t*)p.d + (int64_t)(m0 + r) * p.d_ld + col;
                __builtin_memcpy(to, dg, 2 * MINE);
                __builtin_memcpy(to + (int64_t)p.n, du, 2 * MINE);
            }
        } else {
        float h[MINE];
#pragma unroll
        for (int e = 0; e < MINE; ++e) {
            float slope;
            h[e] = activate<false>(p.act, sum[e % HALF][e / HALF], slope) * sum[HALF + e % HALF][e / HALF];
        }
        if constexpr (EPI == kGated) {
            uint16_t* d = (uint16_t*)p.d + row * p.d_ld + col;
            if (ok && col < p.n) {
                if constexpr (HALF == 1)
                    *(uint2*)d = uint2{pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3])};
                else
                    *(u32x4*)d = u32x4{pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]),
                                       pack_bf16(h[4], h[5]), pack_bf16(h[6], h[7])};
            }
        } else {
            static_assert(EPI == kGated || TN == 4, "a 32-value block lies in one wavefront");
            uint32_t ex;
            const uint32_t codes = quantise_row_block(h, ex);
            if (ok) {
                *(uint32_t*)((uint8_t*)p.d + row * p.d_ld + col / 2) = codes;
                if (q == 0) {
                    uint8_t* sf = (uint8_t*)p.d2 +
                        (((int64_t)slot * (p.n / 128) + col / 128) * p.d2_ld + m0 + r) * 4;
                    sf[col / 32 & 3] = (uint8_t)ex;
                }
            }
        }
        }
    }
    }
    if constexpr (LAYOUT == kMasked) __syncthreads();      // before the partials are replaced
    }
    if (LAYOUT != kMasked && id + gridDim.x < units) __syncthreads();
    }
}

typedef void (*KernelFn)(MxParams);

}  // namespace

int launch_stream(int layout, int epilogue, int tm, int tn, const MxParams& params, int groups,
                  int expected_rows, int most, hipStream_t stream) {
    MxParams p = params;
    KernelFn fn = nullptr;
    int threads = 0;
#define MX_CASE(TM, TN, L, E)                                       \
    if (tm == TM && tn == TN && layout == L && epilogue == E)       \
        fn = mx_stream_kernel<TM, TN, L, E>, threads = 64 * Ring<TM, TN>::kWaves;
#define MX_LAYOUTS(TM, TN, E)     \
    MX_CASE(TM, TN, kDense, E)    \
    MX_CASE(TM, TN, kMasked, E)
#define MX_ROWS(TN, E)   \
    MX_LAYOUTS(1, TN, E) \
    MX_LAYOUTS(2, TN, E) \
    MX_LAYOUTS(4, TN, E)
    MX_ROWS(1, kStore)
    MX_ROWS(2, kStore)
    MX_ROWS(4, kStore)
    MX_ROWS(2, kGated)
    MX_ROWS(4, kGated)
    MX_ROWS(4, kGatedQuant)
    MX_CASE(1, 2, kDense, kGatedGrad)
    MX_CASE(2, 2, kDense, kGatedGrad)
    MX_CASE(4, 2, kDense, kGatedGrad)
    MX_CASE(1, 4, kDense, kGatedGrad)
    MX_CASE(2, 4, kDense, kGatedGrad)
    MX_CASE(4, 4, kDense, kGatedGrad)
#undef MX_ROWS
#undef MX_LAYOUTS
#undef MX_CASE
    if (!fn) return (int)hipErrorInvalidValue;
    const int cols = gated(epilogue) ? 8 * tn : 16 * tn;
    p.m_tiles = (expected_rows + 16 * tm - 1) / (16 * tm);
    p.n_tiles = (p.n + cols - 1) / cols;
    int64_t grid = (int64_t)p.m_tiles * p.n_tiles * (layout == kMasked ? groups : 1);
    if (grid > 0x7fffffff) return (int)hipErrorInvalidValue;
    if (grid > most_workgroups(1)) grid = most_workgroups(1);  // (one fits a CU's LDS)
    if (grid > most) grid = most;
    void* argv[] = {&p};
    return (int)hipLaunchKernel((const void*)fn, dim3((unsigned)grid), dim3(threads), argv, 0,
                                stream);
}

}  // namespace mx
}  // namespace fp8bs

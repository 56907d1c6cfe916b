// fp8bs_mx_stream.hip -- the MXFP4 product and gated block for few rows (single tokens,
// decode batches, sparsely filled slots) on gfx950.
//
// With few rows the weights' bytes are the work: they are read once, from HBM, and each is
// used by one 16-row block or a few.  A workgroup takes a small tile (16 TM x 16 TN) and its
// eight wavefronts share the contraction: wavefront w multiplies the 128-value steps of the
// w-th eighth of K with operands loaded straight into registers, several steps ahead, so a
// tile's whole weight strip is in flight at once and the grid has as many workgroups as the
// columns allow.  The eight FP32 partial tiles meet in LDS and are added in a fixed order --
// one launch, no workspace, no atomics.
//
// Fragments: lane (j, q) = (l % 16, l / 16) holds the 16 bytes (one scale block) 16 q of row
// j's step.  B row TN * r + n is row r of block n, so a lane owns 4 TN neighbouring columns;
// a gated tile has TN / 2 blocks of the gate and as many of the up projection.
#include "fp8bs_mx.h"

namespace fp8bs {
namespace mx {
namespace {

constexpr int kWaves = 8;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : bytes > 0xFFFFFFFFll ? 0xFFFFFFFFll : bytes;
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)(uint32_t)n, 0x00020000);
}

template <int TM, int TN, int LAYOUT, int EPI>
__global__ void __launch_bounds__(64 * kWaves, TM + TN <= 5 ? 4 : 2)
mx_stream_kernel(const MxParams p) {
    constexpr bool GATED = gated(EPI);
    constexpr int BM = 16 * TM, COLS = GATED ? 8 * TN : 16 * TN;
    // steps in flight: about 100 registers of operands (twice as many, with one workgroup per
    // CU, measured 0-10% slower)
    constexpr int RING = TM + TN <= 2 ? 8 : TM + TN <= 3 ? 6 : TM + TN <= 4 ? 4 : 3;
    __shared__ f32x4 part[kWaves][TM * TN][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int j = lane & 15, q = lane >> 4;

    // ---- the tile: tiles along M of one weight strip are neighbours on one XCD ----
    const int id = logical_block();
    int mt = id % p.m_tiles;
    const int rest = id / p.m_tiles;
    const int n0 = rest % p.n_tiles * COLS;
    const int g = LAYOUT == kMasked ? rest / p.n_tiles : 0;
    const int limit = LAYOUT == kMasked ? min(p.group_data[g], p.m) : p.m;
    // (masked: the grid has tiles for the expected rows; a slot with more is walked through)
    for (; mt * BM < limit; mt += p.m_tiles) {
        const int m0 = mt * BM, rows = limit - m0, slot = g;

    // ---- operands ----
    const int64_t group = (int64_t)g * (GATED ? 2 * p.n : p.n);
    const auto a = buffer(p.a + ((int64_t)slot * p.m + m0) * p.a_row, rows * p.a_row);
    const auto b = buffer(p.b + (group + n0) * p.b_row, (int64_t)(p.n - n0) * p.b_row);
    const auto up = buffer(p.b + (group + n0 + (GATED ? p.n : 0)) * p.b_row,
                           (int64_t)(p.n - n0) * p.b_row);
    const auto sa = buffer(p.sfa + (int64_t)slot * p.kwords * p.sfa_ld + m0,
                           ((int64_t)p.kwords * p.sfa_ld - m0) * 4);
    const auto sb = buffer(p.sfb + (int64_t)g * p.kwords * p.sfb_ld + n0,
                           ((int64_t)p.kwords * p.sfb_ld - n0) * 4);
    // A row past the last one is the last one again (its results are not stored), a column
    // past the last one the last column: every read stays inside its operand.
    uint32_t a_at[TM], b_at[TN], sa_at[TM], sb_at[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int r = min(16 * i + j, rows - 1);
        a_at[i] = (uint32_t)r * (uint32_t)p.a_row + 16u * q;
        sa_at[i] = 4u * r;
    }
#pragma unroll
    for (int n = 0; n < TN; ++n) {
        constexpr int HALF = TN / 2 > 0 ? TN / 2 : 1;
        const int r = min(GATED ? HALF * j + n % HALF : TN * j + n, p.n - 1 - n0);
        b_at[n] = (uint32_t)r * (uint32_t)p.b_row + 16u * q;
        sb_at[n] = 4u * (uint32_t)(GATED && n >= HALF ? r + p.n : r);
    }
    struct Step {
        i32x4 a[TM], b[TN];
        int sa[TM], sb[TN];
    };
    auto load = [&](int c, Step& s) {
        const uint32_t at = 64u * (uint32_t)c;
        const uint32_t sa_row = 4u * (uint32_t)p.sfa_ld * (uint32_t)c;
        const uint32_t sb_row = 4u * (uint32_t)p.sfb_ld * (uint32_t)c;
#pragma unroll
        for (int n = 0; n < TN; ++n)
            s.b[n] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                GATED && n >= TN / 2 ? up : b, b_at[n], at, 2));      // 2: non-temporal
#pragma unroll
        for (int n = 0; n < TN; ++n)
            s.sb[n] = __builtin_amdgcn_raw_buffer_load_b32(sb, sb_at[n], sb_row, 0);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            s.a[i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                a, a_at[i], at, 0));
            s.sa[i] = __builtin_amdgcn_raw_buffer_load_b32(sa, sa_at[i], sa_row, 0);
        }
    };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int n = 0; n < TN; ++n) acc[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};

    const int c0 = (int)((int64_t)wave * p.kwords / kWaves);
    const int c1 = (int)((int64_t)(wave + 1) * p.kwords / kWaves);
    Step ring[RING];
#pragma unroll
    for (int s = 0; s < RING - 1; ++s)
        if (c0 + s < c1) load(c0 + s, ring[s]);
    for (int c = c0; c < c1; c += RING) {
#pragma unroll
        for (int s = 0; s < RING; ++s) {
            if (c + s < c1) {
                if (c + s + RING - 1 < c1) load(c + s + RING - 1, ring[(s + RING - 1) % RING]);
                int ea[TM], eb[TN];
#pragma unroll
                for (int i = 0; i < TM; ++i) ea[i] = (ring[s].sa[i] >> (8 * q)) & 255;
#pragma unroll
                for (int n = 0; n < TN; ++n) eb[n] = (ring[s].sb[n] >> (8 * q)) & 255;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int n = 0; n < TN; ++n) {
                        const i32x4 x = ring[s].b[n], y = ring[s].a[i];
                        acc[i][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                            i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0},
                            i32x8{y[0], y[1], y[2], y[3], 0, 0, 0, 0}, acc[i][n], 4, 4, 0, eb[n],
                            0, ea[i]);
                    }
            }
        }
    }

    // ---- the eight partial tiles, added in order by the first TM wavefronts ----
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int n = 0; n < TN; ++n) part[wave][i * TN + n][lane] = acc[i][n];
    __syncthreads();
    if (wave < TM) {
    const int i = wave;
    f32x4 sum[TN];
#pragma unroll
    for (int n = 0; n < TN; ++n) {
        sum[n] = part[0][i * TN + n][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum[n] += part[w][i * TN + n][lane];
    }
    const int r = 16 * i + j;
    const bool ok = r < rows;
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
        constexpr int HALF = TN / 2, MINE = 4 * HALF;
        const int col = n0 + MINE * q;
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
    if constexpr (LAYOUT == kMasked) __syncthreads();      // before the partials are replaced
    }
}

typedef void (*KernelFn)(MxParams);

}  // namespace

int launch_stream(int layout, int epilogue, int tm, int tn, const MxParams& params, int groups,
                  int expected_rows, hipStream_t stream) {
    MxParams p = params;
    KernelFn fn = nullptr;
#define MX_CASE(TM, TN, L, E)                                       \
    if (tm == TM && tn == TN && layout == L && epilogue == E)       \
        fn = mx_stream_kernel<TM, TN, L, E>;
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
#undef MX_ROWS
#undef MX_LAYOUTS
#undef MX_CASE
    if (!fn) return (int)hipErrorInvalidValue;
    const int cols = gated(epilogue) ? 8 * tn : 16 * tn;
    p.m_tiles = (expected_rows + 16 * tm - 1) / (16 * tm);
    p.n_tiles = (p.n + cols - 1) / cols;
    const int64_t grid = (int64_t)p.m_tiles * p.n_tiles * (layout == kMasked ? groups : 1);
    if (grid > 0x7fffffff) return (int)hipErrorInvalidValue;
    void* argv[] = {&p};
    return (int)hipLaunchKernel((const void*)fn, dim3((unsigned)grid), dim3(64 * kWaves), argv, 0,
                                stream);
}

}  // namespace mx
}  // namespace fp8bs

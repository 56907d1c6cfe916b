// fp8bs_gated.hip -- gated activation with e4m3 output and an e4m3 checkpoint, its backward pass
// from the checkpoint, and the quantiser along tokens, on gfx950.
//
//   h = act(gate) up, quantised 1x128 for the product that follows; gate and up are kept 1x128
//   backward: dgate = dh up act'(gate), dup = dh act(gate), 1x128 for the product with the weight
//   and 128x1 (a scale for each column and 128 rows) for the weight gradient, with h 128x1
//
// Values stay FP32 from the activation to each rounding; an input byte is read once, an output
// byte written once.
#include "fp8bs_layer.h"

namespace fp8bs {
namespace layer {
namespace {

// exp(-x) of x >= 0, within an ulp or so: v_exp_f32 of the product with log2 e and what that
// product rounds away (104 is past the last result above 0).
__device__ __forceinline__ float exp_minus(float x) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float a = -__builtin_fminf(x, 104.0f);
    const float hi = a * kHi;
    const float lo = __builtin_fmaf(a, kLo, __builtin_fmaf(a, kHi, -hi));
    const float e = __builtin_amdgcn_exp2f(hi);
    return __builtin_fmaf(e, lo * kLn2, e);
}

// The logistic function s of v and 1 - s, neither by a difference.
__device__ __forceinline__ void logistic(float v, float& s, float& rest) {
    const float e = exp_minus(__builtin_fabsf(v));
    const float d = 1.0f + e;
    float r = __builtin_amdgcn_rcpf(d);
    r = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);     // one step of Newton's
    const float small = e * r;
    s = v < 0.0f ? small : r;
    rest = v < 0.0f ? r : small;
}

// act(v), and its derivative.
template <bool GRAD>
__device__ __forceinline__ float activate(int act, float v, float& slope) {
    float s, rest;
    if (act == FP8BS_ACT_SILU) {
        logistic(v, s, rest);
        if (GRAD) slope = s * (1.0f + v * rest);
        return v * s;
    }
    // (1 + tanh(y)) / 2 is the logistic function of 2 y,  y = sqrt(2/pi) (v + 0.044715 v^3)
    constexpr float c = 0.7978845608028654f;
    const float v2 = v * v;
    logistic(2.0f * c * v * (1.0f + 0.044715f * v2), s, rest);
    // (beyond |v| = 1e15, where s (1 - s) is 0, the square stays finite: 0 times it is 0)
    if (GRAD)
        slope = s + 2.0f * v * s * rest * c * (1.0f + 0.134145f * __builtin_fminf(v2, 1e30f));
    return v * s;
}

struct GatedParams {
    const uint16_t* g;          // bf16 [slots][m][2f]
    uint8_t* hq;
    float* sfh;
    uint8_t* gq;                // or nullptr
    float* sfg;
    const int32_t* group_data;
    int layout, m, f, ld, act;
    int row_tiles;
    uint32_t tiles;
};

constexpr int kTileRows = 64;

// Workgroup: 64 rows x a group of 128 columns, of gate and up; a lane eight columns of each, of
// four rows, all loads issued before any arithmetic.
__global__ void __launch_bounds__(256) gated_quant_kernel(GatedParams p) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int seg = lane & 15, sub = lane >> 4;
    const int fb = p.f >> 7;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int c = (int)(tile % fb);
        const int rt = (int)(tile / fb % p.row_tiles);
        const int slot = (int)(tile / fb / p.row_tiles);
        const int held = p.layout == FP8BS_LAYOUT_MASKED && p.group_data[slot] < p.m
                             ? p.group_data[slot] : p.m;
        if (rt * kTileRows >= held) continue;
        const int64_t slot_row = (int64_t)slot * p.m;
        const int col = 128 * c + 8 * seg;
        Eight<true> gate[4], up[4];
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rt * kTileRows + wave * 16 + 4 * i + sub;
            in[i] = r < held && (p.layout != FP8BS_LAYOUT_CONTIGUOUS || p.group_data[r] >= 0);
            gate[i].zero();
            up[i].zero();
            if (in[i]) {
                const int64_t at = (slot_row + r) * 2 * p.f + col;
                gate[i].stream(p.g, at);
                up[i].stream(p.g, at + p.f);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rt * kTileRows + wave * 16 + 4 * i + sub;
            float h[8], unused;
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = activate<false>(p.act, gate[i][e], unused) * up[i][e];
            float inv;
            float s = block_scale(max16(max8(h)), inv);
            if (in[i]) {
                *(u32x2*)(p.hq + (slot_row + r) * p.f + col) = codes8(h, inv);
                if (seg == 0) p.sfh[((int64_t)slot * fb + c) * p.ld + r] = s;
            }
            if (!p.gq) continue;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = half ? up[i][e] : gate[i][e];
                s = block_scale(max16(max8(v)), inv);
                if (in[i]) {
                    *(u32x2*)(p.gq + (slot_row + r) * 2 * p.f + half * p.f + col) = codes8(v, inv);
                    if (seg == 0)
                        p.sfg[((int64_t)slot * 2 * fb + half * fb + c) * p.ld + r] = s;
                }
            }
        }
    }
}

// ---- 128 rows x 128 columns: blocks both ways -----------------------------------

// A tile's workgroup: eight wavefronts of 16 rows, a lane eight columns (8 (lane % 16) ..) of the
// rows 16 wave + 4 i + lane / 16, i = 0 .. 3.
constexpr int kBlock = 128;

// Scales of the tile's 128-row blocks, and what their columns are multiplied by.  top: largest
// magnitudes of the lane's columns over its four rows.  N arrays at a time.
template <int N>
struct ColumnScales {
    float most[N][8][kBlock];   // the wavefronts' largest magnitudes
    float inv[N][kBlock];
};
template <int N>
__device__ __forceinline__ void column_scales(ColumnScales<N>& lds, float (&top)[N][8],
                                              float* const (&to)[N], const int (&cols)[N]) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, seg = lane & 15;
#pragma unroll
    for (int n = 0; n < N; ++n)
        *(f32x2*)&lds.most[n][wave][8 * seg + first_of(lane)] = max_rows(top[n]);
    __syncthreads();
    if (t < N * kBlock) {
        const int n = t >> 7, col = t & 127;
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = __builtin_fmaxf(m, lds.most[n][w][col]);
        float inv;
        const float s = block_scale(m, inv);
        lds.inv[n][col] = inv;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i == n && to[i] && col < cols[i]) to[i][col] = s;
    }
    __syncthreads();
}

// e4m3 codes of a lane's values, a factor for each column
__device__ __forceinline__ u32x2 column_codes(const float (&v)[8], const float* inv) {
    const f32x4 a = *(const f32x4*)inv, b = *(const f32x4*)(inv + 4);
    u32x2 out;
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * a[0], v[1] * a[1], 0, false);
    out[0] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * a[2], v[3] * a[3], w, true);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * b[0], v[5] * b[1], 0, false);
    out[1] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[6] * b[2], v[7] * b[3], w, true);
    return out;
}

struct GatedBackwardParams {
    const void* g;              // e4m3 or bf16 [m][2f]
    const float* sfg;
    const uint16_t* dh;         // bf16 [m][f]
    uint16_t* d;                // bf16 [m][2f], or nullptr
    uint8_t* dq;                // 1x128, or nullptr
    float* sfd;
    uint8_t* dqt;               // 128x1, or nullptr
    float* sfdt;
    uint8_t* hqt;               // 128x1, or nullptr
    float* sfht;
    const int32_t* grouped_layout;
    int m, f, ld, act;
    uint32_t tiles;
};

template <bool KEPT>
__global__ void __launch_bounds__(512) gated_backward_kernel(GatedBackwardParams p) {
    __shared__ ColumnScales<3> lds;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int seg = lane & 15, sub = lane >> 4;
    const int fb = p.f >> 7;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int c = (int)(tile % fb), rt = (int)(tile / fb);
        const int col = kBlock * c + 8 * seg;
        float dg[4][8], du[4][8], h[4][8];
        float top[3][8] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = (int64_t)rt * kBlock + wave * 16 + 4 * i + sub;
            const bool in = r < p.m && (!p.grouped_layout || p.grouped_layout[r] >= 0);
            const int64_t at = r * 2 * p.f + col;
            float gate[8] = {}, up[8] = {};
            Eight<true> dh;
            dh.zero();
            if (in) {
                dh.stream(p.dh, r * p.f + col);
                if constexpr (KEPT) {
                    widen_e4m3(__builtin_nontemporal_load((const u32x2*)((const uint8_t*)p.g + at)),
                               gate);
                    widen_e4m3(__builtin_nontemporal_load(
                                   (const u32x2*)((const uint8_t*)p.g + at + p.f)), up);
                    const float sg = p.sfg[(int64_t)c * p.ld + r];
                    const float su = p.sfg[(int64_t)(fb + c) * p.ld + r];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        gate[e] *= sg;
                        up[e] *= su;
                    }
                } else {
                    Eight<true> a, b;
                    a.stream(p.g, at);
                    b.stream(p.g, at + p.f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        gate[e] = a[e];
                        up[e] = b[e];
                    }
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float slope;
                const float act = activate<true>(p.act, gate[e], slope);
                // (zeros in a row that holds no token)
                dg[i][e] = dh[e] * up[e] * slope;
                du[i][e] = dh[e] * act;
                h[i][e] = act * up[e];
                top[0][e] = __builtin_fmaxf(top[0][e], __builtin_fabsf(dg[i][e]));
                top[1][e] = __builtin_fmaxf(top[1][e], __builtin_fabsf(du[i][e]));
                top[2][e] = __builtin_fmaxf(top[2][e], __builtin_fabsf(h[i][e]));
            }
            if (p.d && in) {
                store8(p.d, true, at, dg[i]);
                store8(p.d, true, at + p.f, du[i]);
            }
            if (p.dq) {
                float inv_g, inv_u;
                const float sg = block_scale(max16(max8(dg[i])), inv_g);
                const float su = block_scale(max16(max8(du[i])), inv_u);
                if (in) {
                    *(u32x2*)(p.dq + at) = codes8(dg[i], inv_g);
                    *(u32x2*)(p.dq + at + p.f) = codes8(du[i], inv_u);
                    if (seg == 0) {
                        p.sfd[(int64_t)c * p.ld + r] = sg;
                        p.sfd[(int64_t)(fb + c) * p.ld + r] = su;
                    }
                }
            }
        }
        if (!p.dqt && !p.hqt) continue;
        float* const to[3] = {
            p.dqt ? p.sfdt + (int64_t)rt * 2 * p.f + kBlock * c : nullptr,
            p.dqt ? p.sfdt + (int64_t)rt * 2 * p.f + p.f + kBlock * c : nullptr,
            p.hqt ? p.sfht + (int64_t)rt * p.f + kBlock * c : nullptr};
        const int cols[3] = {kBlock, kBlock, kBlock};
        column_scales<3>(lds, top, to, cols);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = (int64_t)rt * kBlock + wave * 16 + 4 * i + sub;
            if (p.dqt) {
                *(u32x2*)(p.dqt + r * 2 * p.f + col) = column_codes(dg[i], &lds.inv[0][8 * seg]);
                *(u32x2*)(p.dqt + r * 2 * p.f + p.f + col) =
                    column_codes(du[i], &lds.inv[1][8 * seg]);
            }
            if (p.hqt) *(u32x2*)(p.hqt + r * p.f + col) = column_codes(h[i], &lds.inv[2][8 * seg]);
        }
        __syncthreads();                       // before lds is written again
    }
}

struct ColumnParams {
    const void* x;
    const float* sfx;
    uint8_t* q;
    float* sf;
    const int32_t* grouped_layout;
    int rows, n, ldx, ld, col_tiles;
    uint32_t tiles;
};

// Tile of 128 x 128 as above; n need not be a multiple of 128.
template <int DTYPE>
__global__ void __launch_bounds__(512) quant_128x1_kernel(ColumnParams p) {
    __shared__ ColumnScales<1> lds;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int seg = lane & 15, sub = lane >> 4;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int c = (int)(tile % p.col_tiles), rt = (int)(tile / p.col_tiles);
        const int col = kBlock * c + 8 * seg;
        float v[4][8] = {};
        float top[1][8] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = (int64_t)rt * kBlock + wave * 16 + 4 * i + sub;
            const bool in = r < p.rows && col < p.n &&
                            (!p.grouped_layout || p.grouped_layout[r] >= 0);
            if (in) {
                const int64_t at = r * p.n + col;
                if constexpr (DTYPE == FP8BS_DTYPE_E4M3) {
                    widen_e4m3(__builtin_nontemporal_load((const u32x2*)((const uint8_t*)p.x + at)),
                               v[i]);
                    const float s = p.sfx[(int64_t)c * p.ldx + r];
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] *= s;
                } else {
                    Eight<DTYPE == FP8BS_DTYPE_BF16> x;
                    x.stream(p.x, at);
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = x[e];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top[0][e] = __builtin_fmaxf(top[0][e], __builtin_fabsf(v[i][e]));
        float* const to[1] = {p.sf + (int64_t)rt * p.ld + kBlock * c};
        const int cols[1] = {p.n - kBlock * c};
        column_scales<1>(lds, top, to, cols);
        if (col < p.n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = (int64_t)rt * kBlock + wave * 16 + 4 * i + sub;
                *(u32x2*)(p.q + r * p.n + col) = column_codes(v[i], &lds.inv[0][8 * seg]);
            }
        __syncthreads();                       // before lds is written again
    }
}

bool activation_known(int act) { return act == FP8BS_ACT_SILU || act == FP8BS_ACT_GELU_TANH; }

}  // namespace
}  // namespace layer
}  // namespace fp8bs

extern "C" int fp8bs_gated_quantize(int layout, const void* g, void* hq, float* sfh, void* gq,
                                    float* sfg, const int32_t* group_data, int m, int f,
                                    int num_groups, int activation, hipStream_t stream) {
    using namespace fp8bs::layer;
    if (layout != FP8BS_LAYOUT_DENSE && layout != FP8BS_LAYOUT_CONTIGUOUS &&
        layout != FP8BS_LAYOUT_MASKED)
        return FP8BS_ERR_UNSUPPORTED;
    const int slots = layout == FP8BS_LAYOUT_MASKED ? num_groups : 1;
    if (m < 0 || m > kMaxRows || f < 128 || f % 128 != 0 || f > kMaxK / 2 || slots < 1 ||
        (layout == FP8BS_LAYOUT_CONTIGUOUS && m % 128 != 0))
        return FP8BS_ERR_SHAPE;
    if (!activation_known(activation)) return FP8BS_ERR_UNSUPPORTED;
    const int row_tiles = (int)(((int64_t)m + kTileRows - 1) / kTileRows);
    const double tiles = (double)slots * row_tiles * (f / 128);
    if (tiles > 0x7fffffff) return FP8BS_ERR_UNSUPPORTED;
    if (m == 0) return FP8BS_OK;
    if (!aligned(g) || !aligned(hq) || !aligned(sfh) || !aligned_or_null(gq) ||
        (gq && !aligned(sfg)) || (layout != FP8BS_LAYOUT_DENSE && !aligned(group_data, 4)))
        return FP8BS_ERR_POINTER;
    GatedParams p = {(const uint16_t*)g, (uint8_t*)hq, sfh, (uint8_t*)gq, sfg, group_data, layout,
                     m, f, (int)fp8bs_get_sfa_ld(m), activation, row_tiles, (uint32_t)tiles};
    return launch((const void*)gated_quant_kernel, workgroups(p.tiles, 8), 256, p, stream);
}

extern "C" int fp8bs_gated_quantize_backward(const void* g, int g_dtype, const float* sfg,
                                             const void* dh, void* d, void* dq, float* sfd,
                                             void* dqt, float* sfdt, void* hqt, float* sfht,
                                             const int32_t* grouped_layout, int m, int f,
                                             int activation, hipStream_t stream) {
    using namespace fp8bs::layer;
    if (m < 0 || m > kMaxRows || f < 128 || f % 128 != 0 || f > kMaxK / 2 ||
        (grouped_layout && m % 128 != 0))
        return FP8BS_ERR_SHAPE;
    if ((g_dtype != FP8BS_DTYPE_E4M3 && g_dtype != FP8BS_DTYPE_BF16) || !activation_known(activation))
        return FP8BS_ERR_UNSUPPORTED;
    const double tiles = (double)(((int64_t)m + 127) / 128) * (f / 128);
    if (tiles > 0x7fffffff) return FP8BS_ERR_UNSUPPORTED;
    if (m == 0) return FP8BS_OK;
    const bool kept = g_dtype == FP8BS_DTYPE_E4M3;
    if (!aligned(g) || (kept && !aligned(sfg)) || !aligned(dh) || !aligned_or_null(d) ||
        !aligned_or_null(dq) || (dq && !aligned(sfd)) || !aligned_or_null(dqt) ||
        (dqt && !aligned(sfdt)) || !aligned_or_null(hqt) || (hqt && !aligned(sfht)) ||
        !aligned_or_null(grouped_layout, 4) || !(d || dq || dqt || hqt))
        return FP8BS_ERR_POINTER;
    GatedBackwardParams p = {g, sfg, (const uint16_t*)dh, (uint16_t*)d, (uint8_t*)dq, sfd,
                             (uint8_t*)dqt, sfdt, (uint8_t*)hqt, sfht, grouped_layout, m, f,
                             (int)fp8bs_get_sfa_ld(m), activation, (uint32_t)tiles};
    return launch(kept ? (const void*)gated_backward_kernel<true>
                       : (const void*)gated_backward_kernel<false>,
                  workgroups(p.tiles, 2), 512, p, stream);
}

extern "C" int fp8bs_quantize_128x1(const void* x, int x_dtype, const float* sfx, void* q,
                                    float* sf, const int32_t* grouped_layout, int rows, int n,
                                    hipStream_t stream) {
    using namespace fp8bs::layer;
    const bool kept = x_dtype == FP8BS_DTYPE_E4M3;
    if (!kept && !value_type(x_dtype)) return FP8BS_ERR_UNSUPPORTED;
    if (rows < 0 || rows > kMaxRows || n < 16 || n > kMaxK || n % (kept ? 128 : 16) != 0 ||
        (grouped_layout && rows % 128 != 0))
        return FP8BS_ERR_SHAPE;
    const int col_tiles = (n + 127) / 128;
    const double tiles = (double)(((int64_t)rows + 127) / 128) * col_tiles;
    if (tiles > 0x7fffffff) return FP8BS_ERR_UNSUPPORTED;
    if (rows == 0) return FP8BS_OK;
    if (!aligned(x) || (kept && !aligned(sfx)) || !aligned(q) || !aligned(sf) ||
        !aligned_or_null(grouped_layout, 4))
        return FP8BS_ERR_POINTER;
    ColumnParams p = {x, sfx, (uint8_t*)q, sf, grouped_layout, rows, n, (int)fp8bs_get_sfa_ld(rows),
                      (int)fp8bs_get_sfa_ld(n), col_tiles, (uint32_t)tiles};
    const void* fn = kept ? (const void*)quant_128x1_kernel<FP8BS_DTYPE_E4M3>
                     : x_dtype == FP8BS_DTYPE_BF16 ? (const void*)quant_128x1_kernel<FP8BS_DTYPE_BF16>
                                                   : (const void*)quant_128x1_kernel<FP8BS_DTYPE_F32>;
    return launch(fn, workgroups(p.tiles, 4), 512, p, stream);
}

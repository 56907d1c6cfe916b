// fp8bs_norm.hip -- root-mean-square norm with the residual's addition and e4m3 output, and its
// backward pass, on gfx950.
//
//   s = x + residual,  rstd = 1 / sqrt(mean(s^2) + eps),  y = s rstd w
//   backward: g = w dy, h = s rstd:  dx = dresidual + rstd (g - h mean(g h)),  dw = sum of dy h
//
// Every sum is FP32; s stays in registers between the sum of its squares and its use, so each
// input byte is read once and each output byte written once, and y is quantised from FP32.
#include "fp8bs_layer.h"

namespace fp8bs {
namespace layer {
namespace {

constexpr int kMostCols = 32768;               // 16 wavefronts of four eights a lane

struct NormParams {
    const void* x;
    const void* res;            // nullptr: none
    void* out;                  // s in res's type, or nullptr
    const void* w;
    void* y;                    // or nullptr
    uint8_t* q;                 // or nullptr
    float* sfa;
    float* rstd;                // or nullptr
    int rows, k, ld;
    float eps;
    int w_bf16, y_bf16;
    int tile_rows;              // rows of a unit (their scales leave together)
    uint32_t tiles;
};

__device__ __forceinline__ void load_weights(const void* w, int bf16, int col, float (&v)[8]) {
    if (bf16) {
        Eight<true> t;
        t.load(w, col);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = t[e];
    } else {
        Eight<false> t;
        t.load(w, col);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = t[e];
    }
}

// Sum over the lanes of a row: W wavefronts.  `part` alternates between two buffers, so one
// barrier a sum is enough.
template <int W>
__device__ __forceinline__ float row_sum(float v, float (*part)[16], int& turn) {
    v = sum_wave(v);
    if constexpr (W > 1) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) part[turn][wave] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < W; ++i) v += part[turn][i];
        turn ^= 1;
    }
    return v;
}

// Workgroup = one row at a time on W = 4 or 16 wavefronts, or four rows (W = 1, a wavefront
// each); a lane holds NV runs of eight columns, 512 W apart, 16 lanes a 128-column group.  A unit
// is tile_rows rows, one after another, the next one's loads issued before this one's sum; their
// scales meet in LDS and leave as runs of tile_rows floats (they lie K-group-major).
template <int W, int NV, bool XB, bool RB>
__global__ void __launch_bounds__(W == 16 ? 1024 : 256) rms_norm_kernel(NormParams p) {
    extern __shared__ float scales[];          // [k/128][tile_rows]
    __shared__ float part[2][16];
    constexpr int kThreads = W == 16 ? 1024 : 256, kAtOnce = kThreads / 64 / W;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wr = wave % W, sub = wave / W;
    const float over_k = 1.0f / (float)p.k;
    int turn = 0;
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = ((i * W + wr) * 64 + lane) * 8;

    for (uint32_t unit = blockIdx.x; unit < p.tiles; unit += gridDim.x) {
        const uint32_t tile = xcd_order(unit, p.tiles);
        const int64_t row0 = (int64_t)tile * p.tile_rows;
        Eight<XB> x[NV];
        Eight<RB> r[NV];
        auto fetch = [&](int64_t row) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                x[i].zero();
                r[i].zero();
                if (row < p.rows && col[i] < p.k) {
                    x[i].load(p.x, row * p.k + col[i]);
                    if (p.res) r[i].load(p.res, row * p.k + col[i]);
                }
            }
        };
        fetch(row0 + sub);
        for (int rr = sub; rr < p.tile_rows; rr += kAtOnce) {
            const int64_t row = row0 + rr;
            float s[NV][8];
            float sq = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[i][e] = x[i][e] + r[i][e];
                    sq += s[i][e] * s[i][e];
                }
            if (rr + kAtOnce < p.tile_rows) fetch(row + kAtOnce);
            const bool in = row < p.rows;
            if (p.out && in)
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (col[i] < p.k) store8(p.out, RB, row * p.k + col[i], s[i]);
            float ms = row_sum<W>(sq, part, turn) * over_k;
            float rstd = 1.0f / sqrtf(ms + p.eps), told = rstd;
            if (ms > 3.0e38f) {                // the squares overflow: of s 2^-96 they do not
                sq = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s[i][e] *= 0x1p-96f;
                        sq += s[i][e] * s[i][e];
                    }
                rstd = 1.0f / sqrtf(row_sum<W>(sq, part, turn) * over_k);
                told = rstd * 0x1p-96f;
            }
            if (p.rstd && in && wr == 0 && lane == 0) p.rstd[row] = told;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (col[i] >= p.k) continue;
                float y[8], w[8];
                load_weights(p.w, p.w_bf16, col[i], w);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = s[i][e] * rstd * w[e];
                if (p.y && in) store8(p.y, p.y_bf16, row * p.k + col[i], y);
                if (p.q) {
                    float inv;
                    const float sc = block_scale(max16(max8(y)), inv);
                    if (in) *(u32x2*)(p.q + row * p.k + col[i]) = codes8(y, inv);
                    if ((lane & 15) == 0) scales[(col[i] >> 7) * p.tile_rows + rr] = sc;
                }
            }
        }
        if (p.q) {
            __syncthreads();
            const int n = (p.k >> 7) * p.tile_rows;
            for (int i = threadIdx.x; i < n; i += kThreads) {
                const int c = i / p.tile_rows, rr = i - c * p.tile_rows;
                if (row0 + rr < p.rows) p.sfa[(int64_t)c * p.ld + row0 + rr] = scales[i];
            }
            __syncthreads();
        }
    }
}

struct BackwardParams {
    const void* s;
    const float* rstd;
    const void* w;
    const void* dy;
    const void* dres;           // nullptr: none
    void* dx;
    float* part;                // [units x rows at once][k] sums of dy h, or nullptr
    int rows, k;
    int w_bf16;
    uint32_t units;             // unit u takes the rows u, u + units, ... (times rows at once)
};

template <int W, int NV, bool SB, bool GB, bool DB>
__global__ void __launch_bounds__(W == 16 ? 1024 : 256) rms_norm_backward_kernel(BackwardParams p) {
    __shared__ float part[2][16];
    constexpr int kThreads = W == 16 ? 1024 : 256, kAtOnce = kThreads / 64 / W;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wr = wave % W, sub = wave / W;
    const float over_k = 1.0f / (float)p.k;
    int turn = 0;
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = ((i * W + wr) * 64 + lane) * 8;
    float w[NV][8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (col[i] < p.k) load_weights(p.w, p.w_bf16, col[i], w[i]);

    for (uint32_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        float acc[NV][8] = {};
        const int64_t step = (int64_t)p.units * kAtOnce;
        int64_t row = (int64_t)unit * kAtOnce + sub;
        // (every wavefront of a workgroup makes the same number of turns)
        for (int64_t first = (int64_t)unit * kAtOnce; first < p.rows; first += step, row += step) {
            const bool in = row < p.rows;
            Eight<SB> s[NV];
            Eight<GB> g[NV];
            Eight<DB> d[NV];
            const float r = in ? p.rstd[row] : 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                s[i].zero();
                g[i].zero();
                d[i].zero();
                if (in && col[i] < p.k) {
                    s[i].load(p.s, row * p.k + col[i]);
                    g[i].load(p.dy, row * p.k + col[i]);
                    if (p.dres) d[i].load(p.dres, row * p.k + col[i]);
                }
            }
            float dot = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float h = s[i][e] * r;
                    dot += g[i][e] * w[i][e] * h;
                    acc[i][e] += g[i][e] * h;
                }
            const float mean = row_sum<W>(dot, part, turn) * over_k;
            if (in)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (col[i] >= p.k) continue;
                    float dx[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dx[e] = d[i][e] + r * (g[i][e] * w[i][e] - s[i][e] * r * mean);
                    store8(p.dx, DB, row * p.k + col[i], dx);
                }
        }
        if (p.part)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (col[i] < p.k)
                    store8(p.part, false, ((int64_t)unit * kAtOnce + sub) * p.k + col[i], acc[i]);
    }
}

struct SumParams {
    const float* part;
    float* dw;
    int parts, k, accumulate;
    uint32_t tiles;
};

// dw = the parts' sum: a workgroup 64 columns, 16 wavefronts every 16th part each, then those
// sixteen in order.
__global__ void __launch_bounds__(1024) rms_norm_sum_kernel(SumParams p) {
    __shared__ float sums[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int col = (int)tile * 64 + lane;
        float v = 0.0f;
        if (col < p.k)
#pragma unroll 8
            for (int i = wave; i < p.parts; i += 16) v += p.part[(int64_t)i * p.k + col];
        sums[wave][lane] = v;
        __syncthreads();
        if (wave == 0 && col < p.k) {
            v = p.accumulate ? p.dw[col] : 0.0f;
            float all = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) all += sums[i][lane];
            p.dw[col] = v + all;
        }
        __syncthreads();
    }
}

// ---- launches -----------------------------------------------------------------

// How a row is laid over a workgroup: wavefronts and eights a lane.
struct Shape {
    int waves, eights;
};
Shape shape_of(int k, bool few_rows) {
    // A row of up to 512 columns is one eight a lane of one wavefront; longer ones take up to four
    // eights a lane.  Few rows leave CUs idle, so there a row takes as many wavefronts as it fills.
    for (int waves : {1, 4, 16})
        for (int eights : {1, 2, 4})
            if (k <= 512 * waves * eights && (!few_rows || eights == 1 || waves == 16))
                return {waves, eights};
    return {0, 0};
}

template <int W, int NV>
const void* norm_kernel(bool xb, bool rb) {
    if (xb) return rb ? (const void*)rms_norm_kernel<W, NV, true, true>
                      : (const void*)rms_norm_kernel<W, NV, true, false>;
    return rb ? (const void*)rms_norm_kernel<W, NV, false, true>
              : (const void*)rms_norm_kernel<W, NV, false, false>;
}
template <int W, int NV>
const void* backward_kernel(bool sb, bool gb, bool db) {
    if (sb) {
        if (gb) return db ? (const void*)rms_norm_backward_kernel<W, NV, true, true, true>
                          : (const void*)rms_norm_backward_kernel<W, NV, true, true, false>;
        return db ? (const void*)rms_norm_backward_kernel<W, NV, true, false, true>
                  : (const void*)rms_norm_backward_kernel<W, NV, true, false, false>;
    }
    if (gb) return db ? (const void*)rms_norm_backward_kernel<W, NV, false, true, true>
                      : (const void*)rms_norm_backward_kernel<W, NV, false, true, false>;
    return db ? (const void*)rms_norm_backward_kernel<W, NV, false, false, true>
              : (const void*)rms_norm_backward_kernel<W, NV, false, false, false>;
}

#define FP8BS_BY_SHAPE(call, s, ...)                                                             \
    ((s).waves == 1   ? (s).eights == 1   ? call<1, 1>(__VA_ARGS__)                              \
                        : (s).eights == 2 ? call<1, 2>(__VA_ARGS__) : call<1, 4>(__VA_ARGS__)    \
     : (s).waves == 4 ? (s).eights == 1   ? call<4, 1>(__VA_ARGS__)                              \
                        : (s).eights == 2 ? call<4, 2>(__VA_ARGS__) : call<4, 4>(__VA_ARGS__)    \
     : (s).eights == 1 ? call<16, 1>(__VA_ARGS__)                                                \
     : (s).eights == 2 ? call<16, 2>(__VA_ARGS__) : call<16, 4>(__VA_ARGS__))

int threads_of(Shape s) { return s.waves == 16 ? 1024 : 256; }
int at_once(Shape s) { return s.waves == 1 ? 4 : 1; }

constexpr int kFewRows = 512;
constexpr int kMostUnits = 1024;               // of the backward pass: parts of dw

Shape backward_shape(int64_t rows, int k) { return shape_of(k, rows < kFewRows); }
// By sizes alone, not by the device or the cap on CUs: the units' sums are added in order.
int64_t backward_units(int64_t rows, Shape s) {
    const int64_t n = (rows + at_once(s) - 1) / at_once(s);
    return n < kMostUnits ? n : kMostUnits;
}

}  // namespace
}  // namespace layer
}  // namespace fp8bs

extern "C" int fp8bs_rms_norm(const void* x, int x_dtype, const void* residual, void* residual_out,
                              int residual_dtype, const void* weight, int weight_dtype, void* y,
                              int y_dtype, void* q, float* sfa, float* rstd, int rows, int k,
                              float eps, hipStream_t stream) {
    using namespace fp8bs::layer;
    if (rows < 0 || rows > kMaxRows || k < 8 || k % 8 != 0 || k > kMostCols || (q && k % 128 != 0))
        return FP8BS_ERR_SHAPE;
    if (!(eps > 0.0f) || eps > 3.0e38f) return FP8BS_ERR_SHAPE;
    if (!value_type(x_dtype) || !value_type(residual_dtype) || !value_type(weight_dtype) ||
        !value_type(y_dtype))
        return FP8BS_ERR_UNSUPPORTED;
    if (rows == 0) return FP8BS_OK;
    if (!aligned(x) || !aligned_or_null(residual) || !aligned_or_null(residual_out) ||
        !aligned(weight) || !aligned_or_null(y) || !aligned_or_null(q) || (q && !aligned(sfa)) ||
        !aligned_or_null(rstd, 4) || !(y || q || residual_out))
        return FP8BS_ERR_POINTER;
    const Shape s = shape_of(k, rows < kFewRows);
    NormParams p = {x, residual, residual_out, weight, y, (uint8_t*)q, sfa, rstd, rows, k,
                    (int)fp8bs_get_sfa_ld(rows), eps, weight_dtype == FP8BS_DTYPE_BF16,
                    y_dtype == FP8BS_DTYPE_BF16, 0, 0};
    p.tile_rows = rows >= 8192 ? 8 : 4;
    if (rows < kFewRows) p.tile_rows = at_once(s);
    p.tiles = (uint32_t)((rows + p.tile_rows - 1) / p.tile_rows);
    const bool xb = x_dtype == FP8BS_DTYPE_BF16, rb = residual_dtype == FP8BS_DTYPE_BF16;
    return launch(FP8BS_BY_SHAPE(norm_kernel, s, xb, rb), workgroups(p.tiles, s.waves == 16 ? 2 : 8),
                  threads_of(s), p, stream, q ? (size_t)(k / 128) * p.tile_rows * 4 : 0);
}

extern "C" int64_t fp8bs_rms_norm_backward_workspace_size(int64_t rows, int k) {
    using namespace fp8bs::layer;
    if (rows < 0 || rows > kMaxRows || k < 8 || k % 8 != 0 || k > kMostCols) return -FP8BS_ERR_SHAPE;
    const Shape s = backward_shape(rows, k);
    return backward_units(rows, s) * at_once(s) * k * 4;
}

extern "C" int fp8bs_rms_norm_backward(const void* s, int s_dtype, const float* rstd,
                                       const void* weight, int weight_dtype, const void* dy,
                                       int dy_dtype, const void* dresidual, void* dx, int dx_dtype,
                                       float* dweight, int accumulate, int rows, int k,
                                       void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
    using namespace fp8bs::layer;
    const int64_t need = fp8bs_rms_norm_backward_workspace_size(rows, k);
    if (need < 0) return FP8BS_ERR_SHAPE;
    if (!value_type(s_dtype) || !value_type(weight_dtype) || !value_type(dy_dtype) ||
        !value_type(dx_dtype))
        return FP8BS_ERR_UNSUPPORTED;
    if (!aligned_or_null(dweight)) return FP8BS_ERR_POINTER;
    const Shape shape = backward_shape(rows, k);
    if (rows > 0) {
        if (!aligned(s) || !aligned(rstd, 4) || !aligned(weight) || !aligned(dy) ||
            !aligned_or_null(dresidual) || !aligned(dx) || (dweight && !aligned(workspace)))
            return FP8BS_ERR_POINTER;
        if (dweight && workspace_bytes < (size_t)need) return FP8BS_ERR_UNSUPPORTED;
        BackwardParams p = {s, rstd, weight, dy, dresidual, dx, dweight ? (float*)workspace : nullptr,
                            rows, k, weight_dtype == FP8BS_DTYPE_BF16,
                            (uint32_t)backward_units(rows, shape)};
        const int st = launch(FP8BS_BY_SHAPE(backward_kernel, shape, s_dtype == FP8BS_DTYPE_BF16,
                                             dy_dtype == FP8BS_DTYPE_BF16,
                                             dx_dtype == FP8BS_DTYPE_BF16),
                              workgroups(p.units, shape.waves == 16 ? 1 : 4), threads_of(shape), p,
                              stream);
        if (st != FP8BS_OK) return st;
    }
    if (!dweight) return FP8BS_OK;
    SumParams p = {(const float*)workspace, dweight,
                   rows > 0 ? (int)(backward_units(rows, shape) * at_once(shape)) : 0, k,
                   accumulate != 0, (uint32_t)((k + 63) / 64)};
    return launch((const void*)rms_norm_sum_kernel, workgroups(p.tiles, 2), 1024, p, stream);
}

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
    int out_bf16, y_bf16, far;
    uint32_t units;
};

// N numbers' sum, by halves: log2 N roundings on each number's way.
template <int N>
__device__ __forceinline__ float sum_of(const float (&v)[N]) {
    if constexpr (N == 1) {
        return v[0];
    } else {
        float half[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) half[i] = v[2 * i] + v[2 * i + 1];
        return sum_of<N / 2>(half);
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
        float all[W];
#pragma unroll
        for (int i = 0; i < W; ++i) all[i] = part[turn][i];
        turn ^= 1;
        return sum_of<W>(all);
    }
    return v;
}

// Workgroup = one row on W = 4 or 16 wavefronts, or four rows (W = 1, a wavefront each).  A lane
// holds NV runs of eight columns, 512 W apart, 16 lanes a 128-column group.  RES: type of residual
// (0 none, 1 bf16, 2 FP32).  16384 x 7168 in bf16 takes 138 us (6.0 TB/s; a copy past the caches
// runs at 6.4): loads issued together, the weight's before the sum, a division for NV groups.  Eight rows
// a workgroup, the next one's loads before this one's sum and scales written together, took 150.  One
// row of 7168: 2.9 us, a launch and three latencies.
template <int W, int NV, bool XB, int RES, bool WB>
__global__ void __launch_bounds__(W == 16 ? 1024 : 256) rms_norm_kernel(NormParams p) {
    __shared__ float part[2][16];
    constexpr int kThreads = W == 16 ? 1024 : 256, kAtOnce = kThreads / 64 / W;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, seg = lane & 15;
    const int wr = wave % W;
    int turn = 0;
    int col[NV], from[NV];                     // (past the last column: the last ones again)
    Eight<WB> w[NV];                           // as they come, for all rows
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = ((i * W + wr) * 64 + lane) * 8;
        from[i] = col[i] < p.k ? +col[i] : p.k - 8;
        w[i].load(p.w, from[i]);
    }
    for (uint32_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        // (workgroups go round the 8 XCDs: each XCD takes eight units in a row, as far as 64 are left, so
        // that the scales of neighbouring rows meet in one L2: 1 to 7% of the time)
        const uint32_t place = (unit | 63) < p.units ? (unit & ~63u) | (unit & 7) << 3 | (unit >> 3 & 7) : unit;
        const int64_t row = (int64_t)place * kAtOnce + wave / W;
        const bool in = row < p.rows;
        const int64_t at = (in ? +row : (int64_t)p.rows - 1) * p.k;
        Eight<XB> x[NV];
        Eight<RES != 2> r[RES ? NV : 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            x[i].stream(p.x, at + from[i]);
            if constexpr (RES) r[i].stream(p.res, at + from[i]);
        }
        float s[NV][8], sq[NV] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[i][e] = x[i][e];
                if constexpr (RES) s[i][e] += r[i][e];
                if (col[i] >= p.k) s[i][e] = 0.0f;
                sq[i] += s[i][e] * s[i][e];
            }
        if (p.out && in)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (col[i] < p.k) put_values(p.out, p.out_bf16, at + col[i], s[i], p.far);
        const float ms = row_sum<W>(sum_of<NV>(sq), part, turn) / (float)p.k + p.eps;
        float rstd = 1.0f / sqrtf(ms), told = rstd;
        // The sums overflow: those of s 2^-72 do not (32768 squares of at most 2^112), and values of which that
        // is no normal number are below 2^-110 of the root.  Or the squares and eps may be no normal numbers
        // themselves, which keep fewer bits: those of s 2^72 are.
        if (ms > 3.0e38f || ms < 0x1p-120f) {
            const float by = ms > 1.0f ? 0x1p-72f : 0x1p72f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                sq[i] = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s[i][e] *= by;
                    sq[i] += s[i][e] * s[i][e];
                }
            }
            rstd = 1.0f / sqrtf(row_sum<W>(sum_of<NV>(sq), part, turn) / (float)p.k + p.eps * by * by);
            told = rstd * by;
        }
        if (p.rstd && in && wr == 0 && lane == 0) p.rstd[row] = told;
        float top[NV], inv[NV], y[NV][8];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[i][e] = s[i][e] * rstd * w[i][e];
            top[i] = max8(y[i]);
        }
        if (p.y && in)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (col[i] < p.k) put_values(p.y, p.y_bf16, at + col[i], y[i], p.far);
        if (p.q) {
            const float scale = block_scales(top, seg, inv);
            const int group = (block_of<NV>(seg) * W + wr) * 4 + (lane >> 4);
            if (in && seg < NV && group < (p.k >> 7)) p.sfa[(int64_t)group * p.ld + row] = scale;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in && col[i] < p.k) put_codes(p.q + at + col[i], codes8(y[i], inv[i]), p.far);
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
    float* part;                // [units][k] sums of dy h, or nullptr
    float* dw;                  // of few rows
    int rows, k, far, accumulate;
    uint32_t units;             // unit u takes the rows u, u + units, ... (times rows at once)
    uint32_t tiles;             // units behind those: 64 columns of dweight each, of few rows
};

// dweight of few rows, straight from the inputs: a workgroup 64 columns, eight lanes a row, in chains of
// every (THREADS / 8)-th row, then those by halves.
template <int THREADS, bool SB, bool GB>
__device__ __forceinline__ void dweight_columns(const BackwardParams& p, uint32_t tile,
                                                float (*sums)[64]) {
    constexpr int kChains = THREADS / 8;
    const int t = threadIdx.x, c = t % 8 * 8, chain = t / 8;
    const int col = (int)tile * 64 + c;
    float acc[8] = {};
    if (col < p.k)
#pragma unroll 4
        for (int row = chain; row < p.rows; row += kChains) {
            Eight<SB> s;
            Eight<GB> g;
            s.load(p.s, (int64_t)row * p.k + col);
            g.load(p.dy, (int64_t)row * p.k + col);
            const float rstd = p.rstd[row];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] += g[e] * (s[e] * rstd);
        }
    store8(sums[chain], false, c, acc);
    __syncthreads();
    if (t < 64 && (int)tile * 64 + t < p.k) {
        float each[kChains / 32];
#pragma unroll
        for (int j = 0; j < kChains / 32; ++j) {
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = sums[32 * j + i][t];
            each[j] = sum_of<32>(v);
        }
        float* const to = p.dw + (int64_t)tile * 64 + t;
        const float all = sum_of<kChains / 32>(each);
        *to = p.accumulate ? *to + all : all;
    }
    __syncthreads();
}

// A workgroup goes through rows and keeps its part of dweight in registers; the parts are written
// once and added by the kernel below (few rows: workgroups of their own, above).  16384 x 7168 in bf16 takes 156 + 5 us (940 MB: 5.9 TB/s, HBM).
template <int W, int NV, bool SB, bool GB, bool WB>
__global__ void __launch_bounds__(W == 16 ? 1024 : 256) rms_norm_backward_kernel(BackwardParams p) {
    __shared__ float part[2][16];
    constexpr int kThreads = W == 16 ? 1024 : 256, kAtOnce = kThreads / 64 / W;
    constexpr bool kFew = W != 4 || NV != 4;   // (few rows of no length take that layout)
    __shared__ __attribute__((aligned(16))) float columns[kFew ? kThreads / 8 : 1][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wr = wave % W, sub = wave / W;
    int turn = 0;
    int col[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) col[i] = ((i * W + wr) * 64 + lane) * 8;
    Eight<WB> w[NV];                           // (as they come, for all rows)
#pragma unroll
    for (int i = 0; i < NV; ++i) w[i].load(p.w, col[i] < p.k ? +col[i] : p.k - 8);

    for (uint32_t unit = blockIdx.x; unit < p.units + p.tiles; unit += gridDim.x) {
        if constexpr (kFew)
            if (unit >= p.units) {
                dweight_columns<kThreads, SB, GB>(p, unit - p.units, columns);
                continue;
            }
        float acc[NV][8] = {};
        const int64_t step = (int64_t)p.units * kAtOnce;
        int64_t row = (int64_t)unit * kAtOnce + sub;
        // (every wavefront of a workgroup makes the same number of turns)
        for (int64_t first = (int64_t)unit * kAtOnce; first < p.rows; first += step, row += step) {
            const bool in = row < p.rows;
            const int64_t from = in ? +row : (int64_t)p.rows - 1;
            Eight<SB> s[NV];
            Eight<GB> g[NV];
            Eight<SB> d[NV];
            const float r = p.rstd[from];
#pragma unroll
            for (int i = 0; i < NV; ++i) {     // (past the last row or column: that one again)
                const int64_t at = from * p.k + (col[i] < p.k ? +col[i] : p.k - 8);
                s[i].stream(p.s, at);
                g[i].stream(p.dy, at);
                if (p.dres) d[i].stream(p.dres, at);
            }
            float dot[NV] = {};
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float t = g[i][e] * (s[i][e] * r);
                    const float own = in ? +t : 0.0f;
                    dot[i] += own * w[i][e];
                    acc[i][e] += own;          // (past the last column: nobody reads it)
                }
                if (col[i] >= p.k) dot[i] = 0.0f;      // (not by a factor: a weight may be infinite)
            }
            const float mean = row_sum<W>(sum_of<NV>(dot), part, turn) / (float)p.k;
            if (in)
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    if (col[i] >= p.k) continue;
                    float dx[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        dx[e] = (p.dres ? d[i][e] : 0.0f) +
                                r * (g[i][e] * w[i][e] - s[i][e] * r * mean);
                    put_values(p.dx, SB, row * p.k + col[i], dx, p.far);
                }
        }
        if (!p.part) continue;
        if constexpr (W == 1) {                // the four rows' sums: one part
            __shared__ float sums[kAtOnce][NV * 512];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                store8(sums[sub], false, col[i], acc[i]);
            }
            __syncthreads();
            for (int c = threadIdx.x; c < p.k; c += kThreads)
                p.part[(int64_t)unit * p.k + c] =
                    (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
            __syncthreads();
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (col[i] < p.k) store8(p.part, false, (int64_t)unit * p.k + col[i], acc[i]);
        }
    }
}

struct SumParams {
    const float* part;
    float* dw;
    int parts, k, accumulate;
    uint32_t tiles;
};

// dw = the parts' sum: a workgroup 32 columns, in 32 chains of every 32nd part each, then those by
// halves.  (Of 512 parts x 7168, with the kernel before it: 32 columns 45.7 us for 4096 rows, 16
// columns, reads of half a line, 48.3.)
constexpr int kSumCols = 32;
__global__ void __launch_bounds__(1024) rms_norm_sum_kernel(SumParams p) {
    constexpr int kCols = kSumCols, kChains = 1024 / kCols;
    __shared__ float sums[kChains][kCols];
    const int t = threadIdx.x, c = t % kCols, chain = t / kCols;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int col = (int)tile * kCols + c;
        float v = 0.0f;
        if (col < p.k)
#pragma unroll 8
            for (int i = chain; i < p.parts; i += kChains) v += p.part[(int64_t)i * p.k + col];
        sums[chain][c] = v;
        __syncthreads();
        if (chain == 0 && col < p.k) {
            float each[kChains];
#pragma unroll
            for (int i = 0; i < kChains; ++i) each[i] = sums[i][c];
            const float all = sum_of<kChains>(each);
            p.dw[col] = p.accumulate ? p.dw[col] + all : all;
        }
        __syncthreads();
    }
}

// ---- launches -----------------------------------------------------------------

// How a row is laid over a workgroup: wavefronts and eights a lane.  A short row is one wavefront's,
// four rows a workgroup; longer ones take 4 wavefronts, then 16.  Few rows leave CUs idle, so there
// a row takes more wavefronts instead of more eights a lane (bf16, both layouts measured):
//   2048 columns, 4 x 1 against 1 x 4: 64 rows 2.8 us against 3.5, 512 rows 3.2 and 3.8, 2048 rows
//   6.2 and 5.8; the gradients 4096 rows 18.5 and 27
//   7168 columns, 16 x 1 against 4 x 4: 64 rows 3.5 us against 3.9, 256 rows 4.1 and 4.4, 512 rows 6.3
//   and 6.2, 1024 rows 12.2 and 11.1; the gradients 600 rows 15.4 and 17.4, 1024 rows 19.1 and 22.2, 2048
//   rows 32.9 and 28.4 (between those two only 4 x 4 was measured: 1025 rows 22.7, 1280 24.0, 1536 25.1)
// Past 16384 columns, 16 x 4, the gradients' values do not fit the 128 registers that 1024 threads leave each: some
// 100 of a lane (bf16; FP32 115) go through scratch.  4096 x 32768 takes 576 us (1.07 GB: 1.9 TB/s), FP32 819, 100 rows
// 57; of 16384 columns 104, 219 and 6.7.
struct Shape {
    int waves, eights;
};
constexpr int kFewRows = 512, kFewBackward = 1025;
Shape shape_of(int64_t rows, int k, bool backward) {
    const bool few = rows < kFewRows;
    if (k <= 512) return {1, 1};
    if (k <= 2048 && !few && !backward) return {1, k <= 1024 ? 2 : 4};
    if (k <= 2048) return {4, 1};
    if (k <= 4096) return {4, 2};
    if (k <= 8192) return rows < (backward ? kFewBackward : kFewRows) ? Shape{16, 1} : Shape{4, 4};
    return {16, k <= 16384 ? 2 : 4};
}

#define FP8BS_BY_SHAPE(call, s, ...)                                                             \
    ((s).waves == 4 ? (s).eights == 1   ? call<4, 1>(__VA_ARGS__)                              \
                        : (s).eights == 2 ? call<4, 2>(__VA_ARGS__) : call<4, 4>(__VA_ARGS__)    \
     : (s).eights == 1 ? call<16, 1>(__VA_ARGS__)                                                \
     : (s).eights == 2 ? call<16, 2>(__VA_ARGS__) : call<16, 4>(__VA_ARGS__))

template <int W, int NV, bool XB, bool WB>
const void* norm_kernel(int res) {
    return res == 0   ? (const void*)rms_norm_kernel<W, NV, XB, 0, WB>
           : res == 1 ? (const void*)rms_norm_kernel<W, NV, XB, 1, WB>
                      : (const void*)rms_norm_kernel<W, NV, XB, 2, WB>;
}
template <int W, int NV>
const void* norm_kernel(bool xb, int res, bool wb) {
    if (xb) return wb ? norm_kernel<W, NV, true, true>(res) : norm_kernel<W, NV, true, false>(res);
    return wb ? norm_kernel<W, NV, false, true>(res) : norm_kernel<W, NV, false, false>(res);
}
template <int W, int NV, bool SB>
const void* backward_kernel(bool gb, bool wb) {
    if (gb) return wb ? (const void*)rms_norm_backward_kernel<W, NV, SB, true, true>
                      : (const void*)rms_norm_backward_kernel<W, NV, SB, true, false>;
    return wb ? (const void*)rms_norm_backward_kernel<W, NV, SB, false, true>
              : (const void*)rms_norm_backward_kernel<W, NV, SB, false, false>;
}
template <int W, int NV>
const void* backward_kernel(bool sb, bool gb, bool wb) {
    return sb ? backward_kernel<W, NV, true>(gb, wb) : backward_kernel<W, NV, false>(gb, wb);
}
const void* norm_kernel(Shape s, bool xb, int res, bool wb) {
    if (s.waves == 1)
        return s.eights == 1   ? norm_kernel<1, 1>(xb, res, wb)
               : s.eights == 2 ? norm_kernel<1, 2>(xb, res, wb) : norm_kernel<1, 4>(xb, res, wb);
    return FP8BS_BY_SHAPE(norm_kernel, s, xb, res, wb);
}
const void* backward_kernel(Shape s, bool sb, bool gb, bool wb) {
    return s.waves == 1 ? backward_kernel<1, 1>(sb, gb, wb)
                        : FP8BS_BY_SHAPE(backward_kernel, s, sb, gb, wb);
}

int threads_of(Shape s) { return s.waves == 16 ? 1024 : 256; }
int at_once(Shape s) { return s.waves == 1 ? 4 : 1; }

// Few rows: dweight in the same launch, from the inputs again, which are in the caches then (so, and in
// parts with a second launch: 7168 columns, 64 rows 3.4 us and 6.6, 256 rows 8.1 and 11.5, 384 rows 10.9
// and 13.2, 511 rows 15.8 and 14.1; 4096 columns, 384 rows 6.0 and 9.8, 511 rows 10.1 and 10.6).
constexpr int kDirectRows = 384;
static_assert(kDirectRows < kFewBackward, "no such row is four wavefronts' of four eights");
bool direct(int64_t rows) { return rows > 0 && rows <= kDirectRows; }

// Units of the backward pass: parts of dweight.  By sizes alone, not by the device or the cap on CUs:
// the units' sums are added in order.  512 at most: 16384 x 7168 takes 160 us, with 256 185 (too
// few loads in flight), with 1024 165 (twice the parts).  256 up to 1024 turns: 512 x 7168 takes
// 13.6 us, with a unit a row 16.3.
int64_t backward_units(int64_t rows, Shape s) {
    const int64_t turns = (rows + at_once(s) - 1) / at_once(s);
    if (direct(rows)) return turns;
    return turns < 256 ? turns : turns < 1024 ? 256 : turns < 2048 ? turns / 4 : 512;
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
    const Shape s = shape_of(rows, k, false);
    NormParams p = {x, residual, residual_out, weight, y, (uint8_t*)q, sfa, rstd, rows, k,
                    (int)fp8bs_get_sfa_ld(rows), eps, residual_dtype == FP8BS_DTYPE_BF16,
                    y_dtype == FP8BS_DTYPE_BF16, far_outputs((double)rows * k * (q ? 1 : 2)),
                    (uint32_t)(((int64_t)rows + at_once(s) - 1) / at_once(s))};
    const int res = !residual ? 0 : residual_dtype == FP8BS_DTYPE_BF16 ? 1 : 2;
    return launch(norm_kernel(s, x_dtype == FP8BS_DTYPE_BF16, res, weight_dtype == FP8BS_DTYPE_BF16),
                  workgroups(p.units, s.waves == 16 ? 2 : 8), threads_of(s), p, stream);
}

extern "C" int64_t fp8bs_rms_norm_backward_workspace_size(int64_t rows, int k) {
    using namespace fp8bs::layer;
    if (rows < 0 || rows > kMaxRows || k < 8 || k % 8 != 0 || k > kMostCols) return -FP8BS_ERR_SHAPE;
    return direct(rows) ? 0 : backward_units(rows, shape_of(rows, k, true)) * k * 4;
}

extern "C" int fp8bs_rms_norm_backward(const void* s, int s_dtype, const float* rstd,
                                       const void* weight, int weight_dtype, const void* dy,
                                       int dy_dtype, const void* dresidual, void* dx, float* dweight,
                                       int accumulate, int rows, int k,
                                       void* workspace, size_t workspace_bytes,
                                       hipStream_t stream) {
    using namespace fp8bs::layer;
    const int64_t need = fp8bs_rms_norm_backward_workspace_size(rows, k);
    if (need < 0) return FP8BS_ERR_SHAPE;
    if (!value_type(s_dtype) || !value_type(weight_dtype) || !value_type(dy_dtype))
        return FP8BS_ERR_UNSUPPORTED;
    if (!aligned_or_null(dweight)) return FP8BS_ERR_POINTER;
    const Shape shape = shape_of(rows, k, true);
    if (rows > 0) {
        if (!aligned(s) || !aligned(rstd, 4) || !aligned(weight) || !aligned(dy) ||
            !aligned_or_null(dresidual) || !aligned(dx) || (dweight && need > 0 && !aligned(workspace)))
            return FP8BS_ERR_POINTER;
        if (dweight && workspace_bytes < (size_t)need) return FP8BS_ERR_UNSUPPORTED;
        const bool few = direct(rows);
        BackwardParams p = {s, rstd, weight, dy, dresidual, dx,
                            dweight && !few ? (float*)workspace : nullptr, dweight, rows, k,
                            far_outputs((double)rows * k * 2), accumulate != 0,
                            (uint32_t)backward_units(rows, shape),
                            dweight && few ? (uint32_t)((k + 63) / 64) : 0};
        const void* fn = backward_kernel(shape, s_dtype == FP8BS_DTYPE_BF16,
                                         dy_dtype == FP8BS_DTYPE_BF16,
                                         weight_dtype == FP8BS_DTYPE_BF16);
        const auto run = [&](uint32_t units, uint32_t tiles) {
            p.units = units;
            p.tiles = tiles;
            return launch(fn, workgroups((int64_t)units + tiles, shape.waves == 16 ? 1 : 4),
                          threads_of(shape), p, stream);
        };
        const uint32_t units = p.units, tiles = p.tiles;
        // (in place: the columns are added before the rows are written over)
        const bool first = tiles && (dx == s || dx == dy);
        int st = first ? run(0, tiles) : FP8BS_OK;
        if (st == FP8BS_OK) st = run(units, first ? 0 : tiles);
        if (st != FP8BS_OK || few) return st;
    }
    if (!dweight) return FP8BS_OK;
    SumParams p = {(const float*)workspace, dweight,
                   rows > 0 ? (int)backward_units(rows, shape) : 0, k,
                   accumulate != 0, (uint32_t)((k + kSumCols - 1) / kSumCols)};
    return launch((const void*)rms_norm_sum_kernel, workgroups(p.tiles, 2), 1024, p, stream);
}

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

// The logistic function s of v and, where asked for, 1 - s.  With e = exp(-v): v_exp_f32 of the
// product h with log2 e, and what that product's rounding leaves out of -v by the first term of its
// own exponential (ln 2's rounding is h 1.9e-9: 4 2^-24 at the most); v_rcp_f32 of 1 + e.  s and
// 1 - s are within 10 2^-24, below |v| = 20 within 7 2^-24.  (-v is cut off at 88, where e is finite
// and the reciprocal 0 already, and where e is 0, before its products overflow.)
template <bool GRAD>
__device__ __forceinline__ float logistic(float v, float& rest) {
    constexpr float kLog2 = 1.44269502f, kLn2 = 0.693147182f;
    const float a = __builtin_amdgcn_fmed3f(-v, -200.0f, 88.0f);
    const float h = a * kLog2;
    const float power = __builtin_amdgcn_exp2f(h);
    const float e = __builtin_fmaf(power, __builtin_fmaf(h, -kLn2, a), power);
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    if (GRAD) rest = e * s;
    return s;
}

// act(v), and its derivative.
template <int ACT, bool GRAD>
__device__ __forceinline__ float activate(float v, float& slope) {
    float rest;
    if constexpr (ACT == FP8BS_ACT_SILU) {
        const float s = logistic<GRAD>(v, rest), a = v * s;
        if (GRAD) slope = __builtin_fmaf(a, rest, s);      // s (1 + v (1 - s))
        return a;
    } else {
        // (1 + tanh(y)) / 2 is the logistic function of 2 y,  y = sqrt(2/pi) (v + 0.044715 v^3)
        constexpr float c = 0.7978845608028654f;
        const float v2 = v * v;
        const float s = logistic<GRAD>(2.0f * c * v * __builtin_fmaf(0.044715f, v2, 1.0f), rest);
        // (where s (1 - s) is 0, far out, its factors stay finite: 0 times them is 0)
        if (GRAD)
            slope = __builtin_fmaf(s * rest * v * (2.0f * c),
                                   __builtin_fmaf(0.134145f, __builtin_fminf(v2, 1e30f), 1.0f), s);
        return v * s;
    }
}

template <bool FAR>
__device__ __forceinline__ u32x2 take8(const uint8_t* base, uint32_t at) {
    const u32x2* from = (const u32x2*)(base + at);
    return FAR ? __builtin_nontemporal_load(from) : *from;
}
// Eight bf16 or FP32 values.  (FP32 past the caches as well, unlike Eight::stream: columns from FP32, so and through them:
// 4096 x 4096 17.1 us and 14.5, 8192 rows 32.2 and 33.2, 16384 rows 61.5 and 61.2, 33280 x 7168 226 and 213.)
template <bool FAR, bool BF16>
__device__ __forceinline__ void take(const void* base, uint32_t at, Eight<BF16>& v) {
    const u32x4* from = (const u32x4*)((const uint8_t*)base + at);
#pragma unroll
    for (int i = 0; i < (BF16 ? 1 : 2); ++i)
        v.w[i] = FAR ? __builtin_nontemporal_load(from + i) : from[i];
}
// Byte offset in a tile: row r (at most 127) of rows of `bytes` (less than 2^24), and on.
__device__ __forceinline__ uint32_t place(int r, int bytes, int on) {
    return __umul24((uint32_t)r, (uint32_t)bytes) + (uint32_t)on;
}

// Entries of grouped_layout for a lane's rows r0, r0 + 4, ...  Kept as they come (held() looks at
// them when they are needed): a test here would wait for each before the loads behind it.
__device__ __forceinline__ int clipped(int r, int last) { return r < last ? +r : +last; }
template <int ROWS>
struct Held {
    int32_t entry[ROWS];
    __device__ __forceinline__ void load(const int32_t* layout, int r0, int last) {
        if (layout) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) entry[i] = layout[clipped(r0 + 4 * i, last)];
        } else {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) entry[i] = 0;
        }
    }
    // bit i: the i-th row holds a token
    __device__ __forceinline__ uint32_t held(int r0, int last) const {
        uint32_t in = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) in |= (r0 + 4 * i <= last && entry[i] >= 0 ? 1u : 0u) << i;
        return in;
    }
};

struct GatedParams {
    const uint16_t* g;          // bf16 [slots][m][2f]
    uint8_t* hq;
    float* sfh;
    uint8_t* gq;                // or nullptr
    float* sfg;
    const int32_t* group_data;
    int layout, m, f, ld;
    int row_tiles, far;
    uint32_t tiles;
};

constexpr int kLaneRows = 2, kTileRows = 16 * kLaneRows;

// Workgroup: 32 rows x a group of 128 columns, of gate and up; a lane eight columns of each, of
// two rows, all loads issued before any arithmetic.  The lane divides for one of its group's
// blocks (block_scales): h, gate and up of each of the two rows.  33280 x 2048 with the checkpoint
// takes 83 us (476 MB: 5.7 TB/s), without 58; some 500 rows in 16 slots, without, 4.1 us.  HBM bounds
// it, the vector units are busy for two thirds of the time.  One row a lane: 4% slower.
template <int ACT, bool KEEP, bool FAR>
__global__ void __launch_bounds__(256) gated_quant_kernel(GatedParams p) {
    constexpr int kBlocks = KEEP ? 3 * kLaneRows : kLaneRows;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int seg = lane & 15, lane_row = wave * 4 * kLaneRows + (lane >> 4);
    const int fb = p.f >> 7;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const int c = (int)(tile % fb);
        const int rt = (int)(tile / fb % p.row_tiles);
        const int slot = (int)(tile / fb / p.row_tiles);
        const int held = p.layout == FP8BS_LAYOUT_MASKED && p.group_data[slot] < p.m
                             ? p.group_data[slot] : p.m;
        if (rt * kTileRows >= held) continue;
        const int64_t row0 = (int64_t)slot * p.m + rt * kTileRows;
        const int last = held - 1 - rt * kTileRows;
        const int32_t* layout =
            p.layout == FP8BS_LAYOUT_CONTIGUOUS ? p.group_data + rt * kTileRows : nullptr;
        const uint16_t* from = p.g + row0 * 2 * p.f + 128 * c;
        Eight<true> gate[kLaneRows], up[kLaneRows];
        Held<kLaneRows> rows;
        rows.load(layout, lane_row, last);
        // (no row of the wavefront holds a token, as past the last expert's: nothing to read)
        if (layout && !__ballot(rows.held(lane_row, last))) continue;
#pragma unroll
        for (int i = 0; i < kLaneRows; ++i) {          // (rows past the last: that one again)
            const int r = clipped(lane_row + 4 * i, last);
            take<FAR>(from, place(r, 4 * p.f, 16 * seg), gate[i]);
            take<FAR>(from + p.f, place(r, 4 * p.f, 16 * seg), up[i]);
        }
        float h[kLaneRows][8], top[kBlocks], inv[kBlocks], unused;
#pragma unroll
        for (int i = 0; i < kLaneRows; ++i) {
            float g[8], u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[e] = gate[i][e];
                u[e] = up[i][e];
                h[i][e] = activate<ACT, false>(g[e], unused) * u[e];
            }
            top[i] = max8(h[i]);
            if constexpr (KEEP) {
                top[kLaneRows + i] = max8(g);
                top[2 * kLaneRows + i] = max8(u);
            }
            // (widened again below: held as they came, they take half of the registers)
            asm("" : "+v"(gate[i].w[0]), "+v"(up[i].w[0]));
        }
        const float scale = block_scales(top, seg, inv);
        const uint32_t in = rows.held(lane_row, last);
        const int block = block_of<kBlocks>(seg), of = block % kLaneRows;
        if (seg < kBlocks && (in >> of & 1)) {
            const int which = block / kLaneRows;
            float* to = which == 0 ? p.sfh + ((int64_t)slot * fb + c) * p.ld
                                   : p.sfg + ((int64_t)(slot * 2 + which - 1) * fb + c) * p.ld;
            to[rt * kTileRows + lane_row + 4 * of] = scale;
        }
        uint8_t* const hq = p.hq + row0 * p.f + 128 * c;
        uint8_t* const gq = p.gq + row0 * 2 * p.f + 128 * c;
#pragma unroll
        for (int i = 0; i < kLaneRows; ++i) {
            if (!(in >> i & 1)) continue;
            const int r = lane_row + 4 * i;
            put_codes(hq + place(r, p.f, 8 * seg), codes8(h[i], inv[i]), p.far);
            if constexpr (KEEP) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = gate[i][e];
                put_codes(gq + place(r, 2 * p.f, 8 * seg), codes8(v, inv[kLaneRows + i]), p.far);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = up[i][e];
                put_codes(gq + p.f + place(r, 2 * p.f, 8 * seg), codes8(v, inv[2 * kLaneRows + i]),
                          p.far);
            }
        }
    }
}

// ---- 128 rows x 128 columns: blocks both ways -----------------------------------

// A tile's workgroup: kWaves wavefronts of 128 / kWaves rows, a lane eight columns
// (8 (lane % 16) ..) of the rows first_row(wave) + 4 i + lane / 16.
constexpr int kBlock = 128;

template <int N, int WAVES>
struct ColumnScales {
    float most[N][WAVES][kBlock];   // the wavefronts' largest magnitudes
    float inv[N][kBlock];
};
// Scales of the tile's 128-row blocks, and what their columns are multiplied by, of N arrays.
// top: largest magnitudes of the lane's columns over its rows.  (The first barrier also keeps
// inv until every wavefront has read the tile's before.)
template <int N, int WAVES>
__device__ __forceinline__ void column_scales(ColumnScales<N, WAVES>& lds, float (&top)[N][8],
                                              float* const (&to)[N], int cols) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6, seg = lane & 15;
#pragma unroll
    for (int n = 0; n < N; ++n)
        *(f32x2*)&lds.most[n][wave][8 * seg + first_of(lane)] = max_rows(top[n]);
    __syncthreads();
    if (t < N * kBlock) {
        const int n = t >> 7, col = t & 127;
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) m = larger(m, lds.most[n][w][col]);
        float inv;
        const float s = block_scale(m, inv);
        lds.inv[n][col] = inv;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i == n && to[i] && col < cols) to[i][col] = s;
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
    int m, f, ld, far;
    uint32_t tiles;
};

constexpr int kGradWaves = 16, kGradRows = 32 / kGradWaves;   // rows of a lane

// A lane's inputs as they lie.
template <bool KEPT>
struct GradInputs {
    Eight<true> dh[kGradRows];
    u32x2 gate_q[KEPT ? kGradRows : 1], up_q[KEPT ? kGradRows : 1];
    float gate_s[KEPT ? kGradRows : 1], up_s[KEPT ? kGradRows : 1];
    Eight<true> gate[KEPT ? 1 : kGradRows], up[KEPT ? 1 : kGradRows];
    Held<kGradRows> rows;
};

template <bool KEPT>
__device__ __forceinline__ void fetch(const GatedBackwardParams& p, uint32_t tile, int lane_row,
                                      int seg, GradInputs<KEPT>& v) {
    const int fb = p.f >> 7;
    const int c = (int)(tile % fb), rt = (int)(tile / fb);
    const int64_t row0 = (int64_t)rt * kBlock;
    const int last = p.m - 1 - row0 < kBlock - 1 ? (int)(p.m - 1 - row0) : kBlock - 1;
    const int32_t* layout = p.grouped_layout ? p.grouped_layout + row0 : nullptr;
    const uint16_t* dh = p.dh + row0 * p.f + kBlock * c;
    const int64_t at = row0 * 2 * p.f + kBlock * c;
    v.rows.load(layout, lane_row, last);
#pragma unroll
    for (int i = 0; i < kGradRows; ++i) {      // (rows past the last: that one again)
        const int r = clipped(lane_row + 4 * i, last);
        take<false>(dh, place(r, 2 * p.f, 16 * seg), v.dh[i]);
        if constexpr (KEPT) {
            const uint8_t* g = (const uint8_t*)p.g + at;
            v.gate_q[i] = take8<false>(g, place(r, 2 * p.f, 8 * seg));
            v.up_q[i] = take8<false>(g + p.f, place(r, 2 * p.f, 8 * seg));
            v.gate_s[i] = (p.sfg + (int64_t)c * p.ld + row0)[r];
            v.up_s[i] = (p.sfg + (int64_t)(fb + c) * p.ld + row0)[r];
        } else {
            const uint16_t* g = (const uint16_t*)p.g + at;
            take<false>(g, place(r, 4 * p.f, 16 * seg), v.gate[i]);
            take<false>(g + p.f, place(r, 4 * p.f, 16 * seg), v.up[i]);
        }
    }
}

// What a workgroup makes of a tile: everything, or of few tiles one of two the gate's gradient, the
// other up's and the activation.
enum : int { kWhole, kGate, kUp };

template <int ACT, bool KEPT, int PART>
__device__ __forceinline__ void gradients(const GatedBackwardParams& p, uint32_t first, uint32_t step,
                                          ColumnScales<3, kGradWaves>& shared) {
    // numbers of the outputs among those that are made: dgate, dup, h
    constexpr int kDup = PART == kWhole ? 1 : 0, kH = kDup + 1;
    constexpr int kOuts = PART == kWhole ? 3 : PART == kGate ? 1 : 2;
    constexpr int kRowBlocks = (PART == kWhole ? 2 : 1) * kGradRows;       // 1x128: dgate's, dup's
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int seg = lane & 15, lane_row = wave * 4 * kGradRows + (lane >> 4);
    const int fb = p.f >> 7;
    ColumnScales<kOuts, kGradWaves>& lds = (ColumnScales<kOuts, kGradWaves>&)shared;
    GradInputs<KEPT> v;
    fetch<KEPT>(p, first, lane_row, seg, v);
    for (uint32_t tile = first; tile < p.tiles; tile += step) {
        const int c = (int)(tile % fb), rt = (int)(tile / fb);
        const int64_t row0 = (int64_t)rt * kBlock;
        const int last = p.m - 1 - row0 < kBlock - 1 ? (int)(p.m - 1 - row0) : kBlock - 1;
        const uint32_t held = v.rows.held(lane_row, last);
        float out[kOuts][kGradRows][8];
        float top[kOuts][8] = {};
        // a row that holds no token is zeros
        if (__ballot(held != (1u << kGradRows) - 1)) {
#pragma unroll
            for (int i = 0; i < kGradRows; ++i) {
                if ((held >> i) & 1) continue;
                v.dh[i].zero();
                if constexpr (KEPT) {
                    v.gate_q[i] = v.up_q[i] = u32x2{0, 0};
                    v.gate_s[i] = v.up_s[i] = 0.0f;
                } else {
                    v.gate[i].zero();
                    v.up[i].zero();
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            float gate[8], up[8];
            if constexpr (KEPT) {
                widen_e4m3(v.gate_q[i], gate);
                widen_e4m3(v.up_q[i], up);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (KEPT) {
                    gate[e] *= v.gate_s[i];
                    up[e] *= v.up_s[i];
                } else {
                    gate[e] = v.gate[i][e];
                    up[e] = v.up[i][e];
                }
                const float dh = v.dh[i][e];
                float slope;
                const float act = activate<ACT, PART != kUp>(gate[e], slope);
                if constexpr (PART != kUp) out[0][i][e] = dh * up[e] * slope;
                if constexpr (PART != kGate) {
                    out[kDup][i][e] = dh * act;
                    out[kH][i][e] = act * up[e];
                }
#pragma unroll
                for (int n = 0; n < kOuts; ++n)
                    top[n][e] = __builtin_fmaxf(top[n][e], __builtin_fabsf(out[n][i][e]));
            }
        }
        // columns of [dgate dup] that are made here
        const int64_t half = PART == kUp ? p.f : 0;
        if (p.dq) {
            float most[kRowBlocks], inv[kRowBlocks];
#pragma unroll
            for (int j = 0; j < kRowBlocks; ++j) most[j] = max8(out[j / kGradRows][j % kGradRows]);
            const float scale = block_scales(most, seg, inv);
            if (seg < kRowBlocks && (held >> (seg % kGradRows) & 1))
                p.sfd[(int64_t)((PART == kUp ? fb : 0) + seg / kGradRows * fb + c) * p.ld + row0 +
                      lane_row + 4 * (seg % kGradRows)] = scale;
            uint8_t* const to = p.dq + row0 * 2 * p.f + half + kBlock * c;
#pragma unroll
            for (int i = 0; i < kGradRows; ++i)
                if (held >> i & 1) {
                    const uint32_t at = place(lane_row + 4 * i, 2 * p.f, 8 * seg);
                    put_codes(to + at, codes8(out[0][i], inv[i]), p.far);
                    if constexpr (PART == kWhole)
                        put_codes(to + p.f + at, codes8(out[1][i], inv[kGradRows + i]), p.far);
                }
        }
        if (p.d)
#pragma unroll
            for (int i = 0; i < kGradRows; ++i)
                if (held >> i & 1) {
                    const int64_t at =
                        (row0 + lane_row + 4 * i) * 2 * p.f + half + kBlock * c + 8 * seg;
                    store8(p.d, true, at, out[0][i]);
                    if constexpr (PART == kWhole) store8(p.d, true, at + p.f, out[1][i]);
                }
        if (tile + step < p.tiles) fetch<KEPT>(p, tile + step, lane_row, seg, v);
        if (!p.dqt && !p.hqt) continue;
        float* to[kOuts];
        to[0] = p.dqt ? p.sfdt + (int64_t)rt * 2 * p.f + half + kBlock * c : nullptr;
        if constexpr (PART == kWhole)
            to[1] = p.dqt ? p.sfdt + (int64_t)rt * 2 * p.f + p.f + kBlock * c : nullptr;
        if constexpr (PART != kGate)
            to[kH] = p.hqt ? p.sfht + (int64_t)rt * p.f + kBlock * c : nullptr;
        column_scales(lds, top, to, kBlock);
        uint8_t* const dqt = p.dqt + row0 * 2 * p.f + half + kBlock * c;
        uint8_t* const hqt = p.hqt + row0 * p.f + kBlock * c;
#pragma unroll
        for (int i = 0; i < kGradRows; ++i) {
            const int r = lane_row + 4 * i;
            if (p.dqt) {
                const uint32_t at = place(r, 2 * p.f, 8 * seg);
                put_codes(dqt + at, column_codes(out[0][i], &lds.inv[0][8 * seg]), p.far);
                if constexpr (PART == kWhole)
                    put_codes(dqt + p.f + at, column_codes(out[1][i], &lds.inv[1][8 * seg]), p.far);
            }
            if constexpr (PART != kGate)
                if (p.hqt)
                    put_codes(hqt + place(r, p.f, 8 * seg),
                              column_codes(out[kH][i], &lds.inv[kH][8 * seg]), p.far);
        }
    }
}

// A workgroup a CU, which goes from tile to tile: the next tile's inputs are on their way while this
// one's scales are exchanged, which is what two barriers a tile cost most.  Gradients are FP32 until
// their codes; each is quantised both ways from the registers, so that nothing is read twice.  33280 x
// 2048 from the checkpoint takes 129 us (622 MB: 4.8 TB/s); the vector units are busy for two thirds of
// that, some 40 instructions a value.  Inputs are read through the caches at every size: 129 us against
// 127 past them, 8192 x 2048 29.7 against 35.4.  Without the inputs ahead it took 164 when it took 133 with
// them, two workgroups of 8 wavefronts a CU 148 (there are no registers to keep inputs ahead).  SPLIT:
// two workgroups a tile where that leaves none waiting: a tile is 6 us of one CU's vector units (silu,
// gelu: 128 x 2048 7.0 and 7.3 us against 8.0 and 8.8 whole, 1024 x 2048 8.9 and 9.2 against 9.8 and 10.6).
template <int ACT, bool KEPT, bool SPLIT>
__global__ void __launch_bounds__(64 * kGradWaves)
    gated_backward_kernel(GatedBackwardParams p) {
    __shared__ ColumnScales<3, kGradWaves> lds;
    if constexpr (!SPLIT)
        gradients<ACT, KEPT, kWhole>(p, blockIdx.x, gridDim.x, lds);
    else if (blockIdx.x % 2 == 0)
        gradients<ACT, KEPT, kGate>(p, blockIdx.x / 2, gridDim.x / 2, lds);
    else
        gradients<ACT, KEPT, kUp>(p, blockIdx.x / 2, gridDim.x / 2, lds);
}

struct ColumnParams {
    const void* x;
    const float* sfx;
    uint8_t* q;
    float* sf;
    const int32_t* grouped_layout;
    int rows, n, ldx, ld, col_tiles, far;
    uint32_t tiles;
};

constexpr int kColumnWaves = 8, kColumnRows = 32 / kColumnWaves;

template <int DTYPE>
struct ColumnInputs {
    static constexpr bool kKept = DTYPE == FP8BS_DTYPE_E4M3;
    u32x2 q[kKept ? kColumnRows : 1];
    float s[kKept ? kColumnRows : 1];
    Eight<DTYPE == FP8BS_DTYPE_BF16> x[kKept ? 1 : kColumnRows];
    Held<kColumnRows> rows;
};
template <int DTYPE, bool FAR>
__device__ __forceinline__ void fetch(const ColumnParams& p, uint32_t tile, int lane_row, int seg,
                                      ColumnInputs<DTYPE>& v) {
    const int c = (int)(tile % p.col_tiles), rt = (int)(tile / p.col_tiles);
    const int64_t row0 = (int64_t)rt * kBlock;
    const int last = p.rows - 1 - row0 < kBlock - 1 ? (int)(p.rows - 1 - row0) : kBlock - 1;
    const int32_t* layout = p.grouped_layout ? p.grouped_layout + row0 : nullptr;
    const int64_t at = row0 * p.n + kBlock * c;
    const int col = clipped(8 * seg, p.n - kBlock * c - 8);
    v.rows.load(layout, lane_row, last);
#pragma unroll
    for (int i = 0; i < kColumnRows; ++i) {    // (rows past the last: that one again; columns alike)
        const int r = clipped(lane_row + 4 * i, last);
        if constexpr (DTYPE == FP8BS_DTYPE_E4M3) {
            v.q[i] = take8<FAR>((const uint8_t*)p.x + at, place(r, p.n, col));
            v.s[i] = (p.sfx + (int64_t)c * p.ldx + row0)[r];
        } else if constexpr (DTYPE == FP8BS_DTYPE_BF16) {
            take<FAR>((const uint16_t*)p.x + at, place(r, 2 * p.n, 2 * col), v.x[i]);
        } else {
            take<FAR>((const float*)p.x + at, place(r, 4 * p.n, 4 * col), v.x[i]);
        }
    }
}

// Tile of 128 x 128 as above; n need not be a multiple of 128.  33280 x 7168 from e4m3 takes 90 us
// (488 MB: 5.4 TB/s; a copy of the same tiles, whose rows are single lines, 84 to 93), bf16 16384 x 7168
// 64, FP32 16384 x 4096 63.  A workgroup a tile, three a CU, hide its barriers better than one that goes
// on with the next tile's inputs ahead (101 to 106).  Neighbouring tiles on one XCD, as the scales of
// four tiles lie in one line: 3% of the time.
template <int DTYPE, bool FAR>
__global__ void __launch_bounds__(64 * kColumnWaves) quant_128x1_kernel(ColumnParams p) {
    __shared__ ColumnScales<1, kColumnWaves> lds;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int seg = lane & 15, lane_row = wave * 4 * kColumnRows + (lane >> 4);
    for (uint32_t unit = blockIdx.x; unit < p.tiles; unit += gridDim.x) {
        const uint32_t tile = xcd_order(unit, p.tiles);
        const int c = (int)(tile % p.col_tiles), rt = (int)(tile / p.col_tiles);
        const int64_t row0 = (int64_t)rt * kBlock;
        ColumnInputs<DTYPE> x;
        fetch<DTYPE, FAR>(p, tile, lane_row, seg, x);
        const uint32_t held = x.rows.held(
            lane_row, p.rows - 1 - row0 < kBlock - 1 ? (int)(p.rows - 1 - row0) : kBlock - 1);
        float v[kColumnRows][8];
        float top[1][8] = {};
#pragma unroll
        for (int i = 0; i < kColumnRows; ++i) {
            const bool in = (held >> i) & 1;
            if constexpr (DTYPE == FP8BS_DTYPE_E4M3) {
                widen_e4m3(in ? x.q[i] : u32x2{0, 0}, v[i]);
                const float s = in ? x.s[i] : 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] *= s;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = in ? x.x[i][e] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < kColumnRows; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top[0][e] = __builtin_fmaxf(top[0][e], __builtin_fabsf(v[i][e]));
        float* const to[1] = {p.sf + (int64_t)rt * p.ld + kBlock * c};
        column_scales(lds, top, to, p.n - kBlock * c);
        uint8_t* const q = p.q + (int64_t)rt * kBlock * p.n + kBlock * c;
        if (kBlock * c + 8 * seg < p.n)
#pragma unroll
            for (int i = 0; i < kColumnRows; ++i)
                put_codes(q + place(lane_row + 4 * i, p.n, 8 * seg),
                     column_codes(v[i], &lds.inv[0][8 * seg]), p.far);
    }
}

template <int ACT, bool KEEP>
const void* quant_kernel(bool far) {
    return far ? (const void*)gated_quant_kernel<ACT, KEEP, true>
               : (const void*)gated_quant_kernel<ACT, KEEP, false>;
}
template <int ACT, bool KEPT>
const void* backward_kernel(bool split) {
    return split ? (const void*)gated_backward_kernel<ACT, KEPT, true>
                 : (const void*)gated_backward_kernel<ACT, KEPT, false>;
}
template <int DTYPE>
const void* columns_kernel(bool far) {
    return far ? (const void*)quant_128x1_kernel<DTYPE, true>
               : (const void*)quant_128x1_kernel<DTYPE, false>;
}

constexpr int kMostColumns = 1 << 20;
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
    if (m < 0 || m > kMaxRows || f < 128 || f % 128 != 0 || f > kMostColumns || slots < 1 ||
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
                     m, f, (int)fp8bs_get_sfa_ld(m), row_tiles,
                     far_outputs((double)slots * m * f * (gq ? 3 : 1)), (uint32_t)tiles};
    const bool far = far_inputs((double)slots * m * f * (gq ? 7 : 5));
    const void* fn = activation == FP8BS_ACT_SILU
                         ? gq ? quant_kernel<FP8BS_ACT_SILU, true>(far)
                              : quant_kernel<FP8BS_ACT_SILU, false>(far)
                         : gq ? quant_kernel<FP8BS_ACT_GELU_TANH, true>(far)
                              : quant_kernel<FP8BS_ACT_GELU_TANH, false>(far);
    return launch(fn, workgroups(p.tiles, 8), 256, p, stream);
}

extern "C" int fp8bs_gated_quantize_backward(const void* g, int g_dtype, const float* sfg,
                                             const void* dh, void* d, void* dq, float* sfd,
                                             void* dqt, float* sfdt, void* hqt, float* sfht,
                                             const int32_t* grouped_layout, int m, int f,
                                             int activation, hipStream_t stream) {
    using namespace fp8bs::layer;
    if (m < 0 || m > kMaxRows || f < 128 || f % 128 != 0 || f > kMostColumns ||
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
                             (int)fp8bs_get_sfa_ld(m),
                             far_outputs((double)m * f * ((d ? 4 : 0) + (dq ? 2 : 0) +
                                                          (dqt ? 2 : 0) + (hqt ? 1 : 0))),
                             (uint32_t)tiles};
    const int cus = compute_units();
    if (cus <= 0) return FP8BS_ERR_HIP;
    const bool split = 2 * tiles <= cus;
    const void* fn = activation == FP8BS_ACT_SILU
                         ? kept ? backward_kernel<FP8BS_ACT_SILU, true>(split)
                                : backward_kernel<FP8BS_ACT_SILU, false>(split)
                         : kept ? backward_kernel<FP8BS_ACT_GELU_TANH, true>(split)
                                : backward_kernel<FP8BS_ACT_GELU_TANH, false>(split);
    const uint32_t most = split ? 2 * p.tiles : p.tiles;
    return launch(fn, most < (uint32_t)cus ? most : (unsigned)cus, 64 * kGradWaves, p, stream);
}

extern "C" int fp8bs_quantize_128x1(const void* x, int x_dtype, const float* sfx, void* q,
                                    float* sf, const int32_t* grouped_layout, int rows, int n,
                                    hipStream_t stream) {
    using namespace fp8bs::layer;
    const bool kept = x_dtype == FP8BS_DTYPE_E4M3;
    if (!kept && !value_type(x_dtype)) return FP8BS_ERR_UNSUPPORTED;
    if (rows < 0 || rows > kMaxRows || n < 16 || n > kMostColumns || n % (kept ? 128 : 16) != 0 ||
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
                      (int)fp8bs_get_sfa_ld(n), col_tiles, far_outputs((double)rows * n),
                      (uint32_t)tiles};
    const bool bf16 = x_dtype == FP8BS_DTYPE_BF16;
    const bool far = far_inputs((double)rows * n * (kept ? 2 : bf16 ? 3 : 5));
    const void* fn = kept   ? columns_kernel<FP8BS_DTYPE_E4M3>(far)
                     : bf16 ? columns_kernel<FP8BS_DTYPE_BF16>(far)
                            : columns_kernel<FP8BS_DTYPE_F32>(far);
    return launch(fn, workgroups(p.tiles, 4), 64 * kColumnWaves, p, stream);
}

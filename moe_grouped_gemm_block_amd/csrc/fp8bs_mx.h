// fp8bs_mx.h -- device helpers and host types shared by the MXFP4 translation units
// (fp8bs_mx_quant.hip, fp8bs_mx_gemm.hip, fp8bs_mx_stream.hip, fp8bs_mx_grad.hip,
// fp8bs_mx_api.cpp; fp8bs_mx_tile.h holds what the matrix kernels alone share).
// Not part of the public interface.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8bs.h"

namespace fp8bs {
namespace mx {

// Row layouts, as the FP8 entry points have them.  kBlocks: the contraction runs over the
// token blocks of one expert (the weight gradient of the contiguous layout).
enum Layout : int { kDense = 0, kContiguous = 1, kMasked = 2, kBlocks = 3 };

// What is done with the accumulators.
//   kStore      D = bf16(acc)
//   kStoreF32   D = acc, or D + acc when MxParams::accumulate is set
//   kGated      h = act(gate) * up, rounded to bf16
//   kGatedQuant the same h quantised to MXFP4
//   kGatedGrad  dg = dh * up * act'(gate), du = dh * act(gate), rounded to bf16
enum Epilogue : int { kStore = 0, kStoreF32 = 1, kGated = 2, kGatedQuant = 3, kGatedGrad = 4 };
constexpr bool gated(int epi) { return epi == kGated || epi == kGatedQuant || epi == kGatedGrad; }

// Tiles along M that one launch lists in LDS (contiguous, masked); the host cuts longer
// problems into several launches.
constexpr int kMaxListed = 2048;

// Largest K and most rows of an operand: copy offsets within a 256-row tile, and row and
// column numbers of the last, partial tile, are 32-bit.
constexpr int kMaxK = 1 << 24, kMaxRows = 0x7ffffe00;

struct MxParams {
    const uint8_t* a;           // codes [rows] of a_row bytes; fp8bs_mx_grad.hip: bf16
    const uint8_t* b;           // codes [groups][B rows] of b_row bytes
    const int32_t* sfa;         // [kwords][sfa_ld] (masked: per slot)
    const int32_t* sfb;         // [groups][kwords][sfb_ld]
    void* d;                    // output; kGatedQuant: codes; kGatedGrad: bf16 [rows][2f]
    void* d2;                   // kGatedQuant: exponents
    const uint16_t* dh;         // kGatedGrad: bf16 [rows][f]
    const int32_t* group_data;  // contiguous: grouped_layout; masked: masked_m
    const int32_t* blocks;      // kBlocks: [groups + 1] offsets, then block numbers
    int64_t a_row, b_row;       // row strides in bytes
    int64_t d_ld, d2_ld;        // elements (kGatedQuant: d_ld bytes of codes, d2_ld words)
    int m;                      // dense: M; contiguous: m_total; masked: rows of a slot
    int n;                      // output columns (gated: f)
    int depth;                  // fp8bs_mx_grad.hip: rows of the contraction
    int kwords;                 // words of a row's exponents (its values / 128)
    int chunks;                 // steps of the contraction
    int sfa_ld, sfb_ld;
    int num_groups;
    int m_tiles, n_tiles;       // m_tiles: dense, and per slot for masked
    int few;                    // masked: slots of at most so many rows each are the few-rows kernel's
    int first, last;            // contiguous: blocks, masked: tiles, that this launch covers
    int raster;
    int act;
    int accumulate;
    int splits;                 // fp8bs_mx_grad.hip: parts of the contraction, 1 where whole
    float* part;                // splits > 1: [splits][rows of d][n]
};

#ifdef __HIPCC__

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}
__device__ __forceinline__ uint16_t to_bf16(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
}
__device__ __forceinline__ float from_bf16(uint32_t h) {
    return __builtin_bit_cast(float, h << 16);
}

// E8M0 exponent of a 32-value block from the largest magnitude's FP32 bits: its exponent
// less 2 (6 = 1.5 * 2^2 is the largest e2m1 value), at least 0; 255 (not a number) when the
// block holds an infinity or a NaN.  Magnitudes below 2^-124, zero among them, give 0.
__device__ __forceinline__ uint32_t block_exponent(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}
// 2^(e - 127) as the conversion instructions take it: e = 0 is a subnormal, e = 255 not a number
// (checked on MI355X: v_cvt_scalef32_pk_bf16_fp4 gives the exact value for every code and
// exponent, in subnormals too, NaN for e = 255).
__device__ __forceinline__ float scale_value(uint32_t e) {
    return __builtin_bit_cast(float, e == 0u ? 0x00400000u : e == 255u ? 0x7FC00000u : e << 23);
}

// Activation of the gate and its derivative.  One exponential and one reciprocal each
// (v_exp_f32, v_rcp_f32: about one unit in the last place, far below the bf16 rounding of
// what they end in).
template <bool GRAD>
__device__ __forceinline__ float activate(int act, float v, float& slope) {
    if (act == FP8BS_ACT_SILU) {
        const float sig = __builtin_amdgcn_rcpf(1.0f + __expf(-v));
        if (GRAD) slope = sig * (1.0f + v * (1.0f - sig));
        return v * sig;
    }
    // 0.5 v (1 + tanh(y)) = v / (1 + exp(-2y)),  y = sqrt(2/pi) (v + 0.044715 v^3)
    constexpr float c = 0.7978845608028654f;
    const float y = c * (v + 0.044715f * v * v * v);
    const float sig = __builtin_amdgcn_rcpf(1.0f + __expf(-2.0f * y));
    // (beyond |v| = 1e15, where sig (1 - sig) is 0, the square stays finite: 0 times it is 0)
    if (GRAD)
        slope = sig + 2.0f * v * sig * (1.0f - sig) * c * (1.0f + 0.134145f * fminf(v * v, 1e30f));
    return v * sig;
}

// Quantises a row's 32 values, eight in each of the lanes l, l + 16, l + 32, l + 48: this
// lane's eight codes, and the block's exponent.
__device__ __forceinline__ uint32_t quantise_row_block(const float (&h)[8], uint32_t& exponent) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __builtin_bit_cast(uint32_t, h[e]) & 0x7FFFFFFFu;
        top = b > top ? b : top;
    }
#pragma unroll
    for (int w = 16; w <= 32; w <<= 1) {
        const uint32_t o = __shfl_xor(top, w, 64);
        top = o > top ? o : top;
    }
    exponent = block_exponent(top);
    if (exponent == 255u) return 0u;
    const float scale = scale_value(exponent);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, h[0], h[1], scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, h[2], h[3], scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, h[4], h[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, h[6], h[7], scale, 3);
    return c;
}

// Buffer descriptor of `bytes` bytes at base.  A read whose lane offset lies past the end
// gives zeros and touches no memory.  Only the lane offset is relied on for that (whether the
// scalar offset counts in the check differs between descriptions of it): callers keep lane
// offset + scalar offset inside the buffer for every lane offset inside it.
__device__ __forceinline__ i32x4 descriptor(const void* base, int64_t bytes) {
    const uint64_t at = (uint64_t)base;
    const int64_t n = bytes < 0 ? 0 : bytes > 0xFFFFFFFFll ? 0xFFFFFFFFll : bytes;
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
                 __builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xFFFFu)),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)n), 0x00020000};
}

// Workgroup b runs on XCD b % 8: XCD x takes the contiguous range [x, x + 1) * grid / 8.
__device__ __forceinline__ int logical_block() {
    const int n = gridDim.x, b = blockIdx.x;
    return (n & 7) ? b : (b & 7) * (n >> 3) + (b >> 3);
}

#endif  // __HIPCC__

// Most workgroups of a launch of which per_cu share a CU: those of the process's cap on CUs;
// without one, so many that their threads (at most 512 each) are a 32-bit number.
inline int64_t most_workgroups(int per_cu) {
    const int cap = fp8bs_get_num_cus();
    return cap > 0 ? (int64_t)cap * per_cu : 1 << 22;
}

// Launchers; return a hipError_t value.
// Contiguous layout: out = [num_groups + 1] offsets, then each expert's 128-row blocks in
// order (a block belongs to the expert of its first row).
int launch_block_order(const int32_t* grouped_layout, int blocks, int num_groups, int32_t* out,
                       hipStream_t stream);
// (num_cus: under the process's cap, which changes tiles and grids, never results)
int launch_gemm(int layout, int epilogue, const MxParams& p, int groups, int expected_rows,
                int num_cus, int device_cus, hipStream_t stream);
// Products of bf16 rows with widened codes (fp8bs_mx_grad.hip): D = A W, or with a_t
// D = A^T X, the contraction running over the rows of the second operand.
int launch_grad(int layout, bool a_t, int epilogue, const MxParams& p, int groups, int num_cus,
                hipStream_t stream);
// Into how many parts the contraction of a product is split (sizes only: the workspace holds
// the parts).
int grad_splits(int layout, const MxParams& p, int groups);
// da (layout dense or contiguous, parameters a) and db (b) in one launch, where that takes less
// time than one after the other; either may be null.  Adds the parts of split products.
bool grad_pair_pays(int layout, const MxParams& a, const MxParams& b, int groups, int num_cus);
int launch_grad_pair(int layout, int epilogue, const MxParams* a, const MxParams* b, int groups,
                     hipStream_t stream);
// Few rows, dense and masked layouts: tiles of 16 tm x 16 tn on at most `most` workgroups
// (fp8bs_mx_stream.hip).
int launch_stream(int layout, int epilogue, int tm, int tn, const MxParams& p, int groups,
                  int expected_rows, int most, hipStream_t stream);

}  // namespace mx
}  // namespace fp8bs

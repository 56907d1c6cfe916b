// fp8bs_mx_quant.hip -- MXFP4 quantiser and its inverse on gfx950.
//
// 32 consecutive values of a row share the scale 2^(e - 127), e - 127 =
// floor(log2(max |x|)) - 2; each becomes e2m1(x * 2^(127 - e)), nearest with ties to the
// even code, magnitudes above 6 saturating.  Scaling by a power of two is exact, so a value
// is rounded once and the result does not depend on how the work is laid out.
//
// Both kernels read every input byte once and write every output byte once; HBM bounds
// them: 33152 x 7168 in bf16 takes 92 us to codes and 86 us back (6.5 and 7.0 TB/s; plain
// arithmetic and cached accesses took 134 and 140), in FP32 200 and 379 (5.4 and 2.8 TB/s: a lane's
// two loads or stores each touch 16 of every 32 bytes).  A workgroup takes 32 rows x 256 columns:
// a row's codes are one 128-byte line, the 32 exponent words of a 128-column group (exponents
// lie K-group-major, rows consecutive) another, so no line is written in two pieces by
// different workgroups.
#include "fp8bs_mx.h"

namespace fp8bs {
namespace mx {
namespace {

constexpr int kRows = 32, kCols = 256;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// 8 consecutive inputs as they lie: FP32 (two pieces of 16 bytes) or bf16 (one).  They are
// read once, past the caches.
template <bool BF16>
struct Piece {
    u32x4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const void* x, int64_t at) {
        const u32x4* from = (const u32x4*)((const uint8_t*)x + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = __builtin_nontemporal_load(from + i);
    }
    // FP32 bits of the largest magnitude (bf16: their upper half, compared two at a time)
    __device__ __forceinline__ uint32_t top() const {
        if constexpr (BF16) {
            u16x2 t = {0, 0};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t = __builtin_elementwise_max(t, __builtin_bit_cast(u16x2, w[0][i] & 0x7FFF7FFFu));
            return (uint32_t)(t[0] > t[1] ? t[0] : t[1]) << 16;
        } else {
            uint32_t t = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t b = w[i >> 2][i & 3] & 0x7FFFFFFFu;
                t = b > t ? b : t;
            }
            return t;
        }
    }
    // e2m1 codes of the values divided by scale (a power of two: exact before the rounding)
    __device__ __forceinline__ uint32_t codes(float scale) const {
        uint32_t c = 0;
        if constexpr (BF16) {
            const bf16x8 x = __builtin_bit_cast(bf16x8, w[0]);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2{x[0], x[1]}, scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2{x[2], x[3]}, scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2{x[4], x[5]}, scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16x2{x[6], x[7]}, scale, 3);
        } else {
            const f32x4 a = __builtin_bit_cast(f32x4, w[0]), b = __builtin_bit_cast(f32x4, w[1]);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[0], b[1], scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[2], b[3], scale, 3);
        }
        return c;
    }
};

// Thread t of a workgroup: columns 8 * (t % 32) .. + 7 of rows t / 32 + 8 i.  Four
// neighbouring lanes hold a 32-value block.
template <bool BF16>
__global__ void __launch_bounds__(256) mx_quant_kernel(const void* __restrict__ x,
                                                       uint8_t* __restrict__ q,
                                                       uint32_t* __restrict__ sf, int rows, int k,
                                                       int ld, int row_tiles, int col_tiles,
                                                       uint32_t tiles) {
    __shared__ uint32_t words[2][kRows];
    const int t = threadIdx.x, seg = t & 31;
    // (a workgroup for each tile, unless a launch may not have so many)
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        if (tile != blockIdx.x) __syncthreads();           // before the words are replaced
        const int ct = tile % col_tiles;
        const int rt = tile / col_tiles % row_tiles;
        const int slot = tile / col_tiles / row_tiles;
        const int col = ct * kCols + 8 * seg;
        const int64_t row0 = (int64_t)slot * rows;
        Piece<BF16> v[4] = {};
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rt * kRows + (t >> 5) + 8 * i;
            in[i] = r < rows && col < k;
            if (in[i]) v[i].load(x, (row0 + r) * k + col);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = (t >> 5) + 8 * i;
            // over the block's four lanes, then the four exponents of a 128-column group into one
            // word: exchanges within 4 and 16 lanes (quad permutations, row rotations)
            uint32_t top = v[i].top();
            top = umax(top, __builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));   // lane ^ 1
            top = umax(top, __builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));   // lane ^ 2
            const uint32_t e = block_exponent(top);
            // A block that holds an infinity or a NaN is not a number as a whole (e2m1 has
            // neither); its codes are zeros.
            if (in[i])
                *(uint32_t*)(q + ((row0 + rt * kRows + rr) * k + col) / 2) =
                    e == 255u ? 0u : v[i].codes(scale_value(e));
            uint32_t word = e << (8 * ((seg >> 2) & 3));
            word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x124, 0xF, 0xF, true);   // rotate 4
            word |= (uint32_t)__builtin_amdgcn_update_dpp(0, (int)word, 0x128, 0xF, 0xF, true);   // rotate 8
            if ((seg & 15) == 0) words[seg >> 4][rr] = word;
        }
        __syncthreads();
        if (t < 2 * kRows) {
            const int c = ct * 2 + (t >> 5), r = rt * kRows + (t & 31);
            if (r < rows && c < k / 128)
                sf[((int64_t)slot * (k / 128) + c) * ld + r] = words[t >> 5][t & 31];
        }
    }
}

template <bool BF16>
__global__ void __launch_bounds__(256) mx_dequant_kernel(const uint8_t* __restrict__ q,
                                                         const uint32_t* __restrict__ sf,
                                                         void* __restrict__ x, int rows, int k,
                                                         int ld, int row_tiles, int col_tiles,
                                                         uint32_t tiles) {
    __shared__ uint32_t words[2][kRows];
    const int t = threadIdx.x, seg = t & 31;
    // (a workgroup for each tile, unless a launch may not have so many)
    for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        if (tile != blockIdx.x) __syncthreads();           // before the words are replaced
        const int ct = tile % col_tiles;
        const int rt = tile / col_tiles % row_tiles;
        const int slot = tile / col_tiles / row_tiles;
        const int col = ct * kCols + 8 * seg;
        const int64_t row0 = (int64_t)slot * rows;
        if (t < 2 * kRows) {
            const int c = ct * 2 + (t >> 5), r = rt * kRows + (t & 31);
            words[t >> 5][t & 31] =
                (r < rows && c < k / 128) ? sf[((int64_t)slot * (k / 128) + c) * ld + r] : 0u;
        }
        uint32_t codes[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = rt * kRows + (t >> 5) + 8 * i;
            codes[i] = (r < rows && col < k) ? *(const uint32_t*)(q + ((row0 + r) * k + col) / 2) : 0u;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = (t >> 5) + 8 * i, r = rt * kRows + rr;
            if (r >= rows || col >= k) continue;
            const uint32_t e = (words[seg >> 4][rr] >> (8 * ((seg >> 2) & 3))) & 255u;
            // bf16 holds every value exactly; FP32 values are those, widened
            const float scale = scale_value(e);
            u32x4 w;
            w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 0));
            w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 1));
            w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 2));
            w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[i], scale, 3));
            const int64_t at = (row0 + r) * k + col;
            if constexpr (BF16) {
                __builtin_nontemporal_store(w, (u32x4*)((uint16_t*)x + at));
            } else {
                const u32x4 lo = {w[0] << 16, w[0] & 0xFFFF0000u, w[1] << 16, w[1] & 0xFFFF0000u};
                const u32x4 hi = {w[2] << 16, w[2] & 0xFFFF0000u, w[3] << 16, w[3] & 0xFFFF0000u};
                __builtin_nontemporal_store(lo, (u32x4*)((float*)x + at));
                __builtin_nontemporal_store(hi, (u32x4*)((float*)x + at) + 1);
            }
        }
    }
}

// One workgroup; wavefront w takes the experts w, w + 16, ...: it counts their blocks 64 at a
// time, then writes them in order behind the blocks of the experts before.
__global__ void __launch_bounds__(1024) mx_block_order_kernel(const int32_t* __restrict__ layout,
                                                              int blocks, int groups,
                                                              int32_t* __restrict__ out) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto owned = [&](int b, int e) { return b < blocks && layout[(int64_t)b * 128] == e; };
    for (int e = wave; e < groups; e += 16) {
        int n = 0;
        for (int w = 0; w < blocks; w += 64) n += __popcll(__ballot(owned(w + lane, e)));
        if (lane == 0) out[e + 1] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = 0;
        out[0] = 0;
        for (int e = 0; e < groups; ++e) out[e + 1] = at += out[e + 1];
    }
    __syncthreads();
    int32_t* order = out + groups + 1;
    for (int e = wave; e < groups; e += 16) {
        int at = out[e];
        for (int w = 0; w < blocks; w += 64) {
            const bool mine = owned(w + lane, e);
            const uint64_t all = __ballot(mine);
            if (mine) order[at + __popcll(all & ((1ull << lane) - 1ull))] = w + lane;
            at += __popcll(all);
        }
    }
}

bool aligned(const void* p, uintptr_t to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

// Checks shared by both directions; *grid = workgroups.
int check(const void* x, int dtype, const void* q, const void* sf, int groups, int rows, int k,
          int64_t* grid) {
    if (k < 128 || k % 128 != 0 || rows < 0 || groups < 1 || k > kMaxK || rows > kMaxRows)
        return FP8BS_ERR_SHAPE;
    if (dtype != FP8BS_DTYPE_F32 && dtype != FP8BS_DTYPE_BF16) return FP8BS_ERR_UNSUPPORTED;
    if ((double)groups * rows * k >= 9.0e15) return FP8BS_ERR_SHAPE;
    *grid = (int64_t)groups * ((rows + kRows - 1) / kRows) * ((k + kCols - 1) / kCols);
    if (*grid > 0x7fffffff) return FP8BS_ERR_SHAPE;
    if (rows == 0) return FP8BS_OK;
    if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 16)) return FP8BS_ERR_POINTER;
    return FP8BS_OK;
}

}  // namespace

int launch_block_order(const int32_t* grouped_layout, int blocks, int num_groups, int32_t* out,
                       hipStream_t stream) {
    void* args[] = {&grouped_layout, &blocks, &num_groups, &out};
    return (int)hipLaunchKernel((const void*)mx_block_order_kernel, dim3(1), dim3(1024), args, 0,
                                stream);
}

}  // namespace mx
}  // namespace fp8bs

extern "C" int fp8bs_quantize_mxfp4(const void* x, int x_dtype, void* q, int32_t* sf, int groups,
                                    int rows, int k, hipStream_t stream) {
    using namespace fp8bs::mx;
    int64_t grid = 0;
    const int st = check(x, x_dtype, q, sf, groups, rows, k, &grid);
    if (st != FP8BS_OK || rows == 0) return st;
    int ld = (int)fp8bs_get_sfa_ld(rows), rt = (rows + kRows - 1) / kRows,
        ct = (k + kCols - 1) / kCols;
    uint32_t tiles = (uint32_t)grid;
    if (grid > most_workgroups(8)) grid = most_workgroups(8);
    void* args[] = {(void*)&x, (void*)&q, (void*)&sf, &rows, &k, &ld, &rt, &ct, &tiles};
    const void* fn = x_dtype == FP8BS_DTYPE_BF16 ? (const void*)mx_quant_kernel<true>
                                                 : (const void*)mx_quant_kernel<false>;
    return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), args, 0, stream) == hipSuccess
               ? FP8BS_OK : FP8BS_ERR_HIP;
}

extern "C" int fp8bs_dequantize_mxfp4(const void* q, const int32_t* sf, void* x, int x_dtype,
                                      int groups, int rows, int k, hipStream_t stream) {
    using namespace fp8bs::mx;
    int64_t grid = 0;
    const int st = check(x, x_dtype, q, sf, groups, rows, k, &grid);
    if (st != FP8BS_OK || rows == 0) return st;
    int ld = (int)fp8bs_get_sfa_ld(rows), rt = (rows + kRows - 1) / kRows,
        ct = (k + kCols - 1) / kCols;
    uint32_t tiles = (uint32_t)grid;
    if (grid > most_workgroups(8)) grid = most_workgroups(8);
    void* args[] = {(void*)&q, (void*)&sf, (void*)&x, &rows, &k, &ld, &rt, &ct, &tiles};
    const void* fn = x_dtype == FP8BS_DTYPE_BF16 ? (const void*)mx_dequant_kernel<true>
                                                 : (const void*)mx_dequant_kernel<false>;
    return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(256), args, 0, stream) == hipSuccess
               ? FP8BS_OK : FP8BS_ERR_HIP;
}

// fp8bs_layer.h -- what the operators between the FP8 products share (norm, dispatch and
// combine, gated activation, quantiser along tokens): checks, launches, and the device code of
// loads, exchanges between lanes and e4m3 quantisation.
#ifndef FP8BS_LAYER_H
#define FP8BS_LAYER_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "fp8bs.h"

namespace fp8bs {
namespace layer {

constexpr int kMaxK = 1 << 24;                 // columns of an operand
constexpr int kMaxRows = 0x7fffff00;           // rows, with room to round up

inline bool aligned(const void* p, uintptr_t to = 16) { return p && ((uintptr_t)p & (to - 1)) == 0; }
// an optional buffer
inline bool aligned_or_null(const void* p, uintptr_t to = 16) { return ((uintptr_t)p & (to - 1)) == 0; }
inline bool value_type(int dtype) { return dtype == FP8BS_DTYPE_F32 || dtype == FP8BS_DTYPE_BF16; }

// Workgroups for `units` units of work when `per_cu` workgroups share a CU: one a unit, within
// the process's cap on CUs and so few that their threads (at most 1024 each) are a 32-bit number.
// Kernels go on to further units.
inline unsigned workgroups(int64_t units, int per_cu) {
    const int cap = fp8bs_get_num_cus();
    const int64_t most = cap > 0 ? (int64_t)cap * per_cu : 1 << 21;
    return (unsigned)(units < most ? units : most);
}

// Compute units of the current device under the process's cap; 0 on error.
inline int compute_units() {
    static std::atomic<int> known[64];             // 0: not asked yet
    int dev = 0, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    const bool kept = dev >= 0 && dev < 64;
    if (kept) cus = known[dev].load(std::memory_order_relaxed);
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            return 0;
        if (kept) known[dev].store(cus, std::memory_order_relaxed);
    }
    const int cap = fp8bs_get_num_cus();
    return cap > 0 && cap < cus ? cap : cus;
}

// Whether outputs of so many bytes are written past the caches: they would not stay there for the
// next kernel, and streaming runs 5-10% faster past them (through them and past them: norm of
// 16384 x 7168 148 us and 141, its gradients 174 and 161, gated 33280 x 2048 92 and 87).
inline int far_outputs(double bytes) { return bytes > 64e6; }

// Whether inputs are read past the caches, from the bytes that a call reads and writes: of few the
// kernel before has left them there, and many are gone (through the caches and past them: gated 4096 x
// 2048, 59 MB, 11.6 us and 13.4, 8192 x 2048 24.7 and 22.8; columns of 4096 x 7168 12.4 and 15.2, 8192
// rows 27.9 and 24.0; combine of 1024 tokens, eight choices, 2048 columns, 38 MB, 8.1 and 10.8).
inline bool far_inputs(double bytes) { return bytes > 80e6; }

template <class P>
int launch(const void* kernel, unsigned grid, int threads, P& params, hipStream_t stream,
           size_t lds = 0) {
    void* args[] = {(void*)&params};
    return hipLaunchKernel(kernel, dim3(grid), dim3(threads), args, lds, stream) == hipSuccess
               ? FP8BS_OK : FP8BS_ERR_HIP;
}

#ifdef __HIPCC__

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// (by value: a bit cast of a vector's element in place takes element 0)
__device__ __forceinline__ float as_float(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ uint32_t as_bits(float x) { return __builtin_bit_cast(uint32_t, x); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const f32x2 v = {lo, hi};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
}

// Eight consecutive values as they lie: bf16 in 16 bytes, FP32 in 32.
template <bool BF16>
struct Eight {
    u32x4 w[BF16 ? 1 : 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = u32x4{0, 0, 0, 0};
    }
    __device__ __forceinline__ void load(const void* x, int64_t at) {
        const u32x4* from = (const u32x4*)((const uint8_t*)x + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = from[i];
    }
    // past the caches.  FP32 is not here, nor is it stored so: its two pieces are half of every 32 bytes each,
    // which only a cache makes whole (norm of 8192 x 7168 in FP32 142 us, past them 156; gradients 182, 217).
    __device__ __forceinline__ void stream(const void* x, int64_t at) {
        const u32x4* from = (const u32x4*)((const uint8_t*)x + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) w[i] = BF16 ? __builtin_nontemporal_load(from + i) : from[i];
    }
    template <bool FAR>
    __device__ __forceinline__ void take(const void* x, int64_t at) {
        if constexpr (FAR) stream(x, at);
        else load(x, at);
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (BF16) {
            const uint32_t u = w[0][i >> 1];
            return as_float((i & 1) ? u & 0xFFFF0000u : u << 16);
        } else {
            return as_float(w[i >> 2][i & 3]);
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[0][i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i >> 2][i & 3] = as_bits(v[i]);
        }
    }
    __device__ __forceinline__ void store(void* x, int64_t at) const {
        u32x4* to = (u32x4*)((uint8_t*)x + at * (BF16 ? 2 : 4));
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) to[i] = w[i];
    }
};

__device__ __forceinline__ void store8(void* x, bool bf16, int64_t at, const float (&v)[8]) {
    if (bf16) {
        Eight<true> p;
        p.set(v);
        p.store(x, at);
    } else {
        Eight<false> p;
        p.set(v);
        p.store(x, at);
    }
}

// Stores past the caches (far) or through them: outputs that are too large to stay there.  The
// empty asm on both sides keeps the compiler from making one ordinary store of the branches.
__device__ __forceinline__ void put16(void* to, u32x4 v, bool far) {
    if (far) {
        asm volatile("");
        __builtin_nontemporal_store(v, (u32x4*)to);
        asm volatile("");
    } else {
        *(u32x4*)to = v;
    }
}
__device__ __forceinline__ void put_values(void* x, bool bf16, int64_t at, const float (&v)[8],
                                           bool far) {
    if (bf16) {
        Eight<true> p;
        p.set(v);
        put16((uint8_t*)x + at * 2, p.w[0], far);
    } else {
        store8(x, false, at, v);
    }
}
__device__ __forceinline__ void put_codes(uint8_t* to, u32x2 codes, bool far) {
    if (far) {
        asm volatile("");
        __builtin_nontemporal_store(codes, (u32x2*)to);
        asm volatile("");
    } else {
        *(u32x2*)to = codes;
    }
}

// Eight e4m3 codes, widened.
__device__ __forceinline__ void widen_e4m3(u32x2 w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false);
        const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
        v[4 * i] = lo[0];
        v[4 * i + 1] = lo[1];
        v[4 * i + 2] = hi[0];
        v[4 * i + 3] = hi[1];
    }
}

// ---- exchanges ----------------------------------------------------------------

template <int CTRL>
__device__ __forceinline__ float moved(float x) {
    return as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_bits(x), CTRL, 0xF, 0xF, true));
}
// Largest of two numbers >= 0, by their bits: for floats from exchanges the compiler would make
// sure first that they are no signalling NaN.
__device__ __forceinline__ float larger(float a, float b) {
    const uint32_t x = as_bits(a), y = as_bits(b);
    return as_float(x > y ? x : y);
}
// (magnitudes) over 16 neighbouring lanes: quad permutations, then mirrors of 8 and 16 lanes
__device__ __forceinline__ float max16(float x) {
    x = larger(x, moved<0xB1>(x));
    x = larger(x, moved<0x4E>(x));
    x = larger(x, moved<0x141>(x));
    return larger(x, moved<0x140>(x));
}
__device__ __forceinline__ float sum16(float x) {
    x += moved<0xB1>(x);
    x += moved<0x4E>(x);
    x += moved<0x141>(x);
    return x + moved<0x140>(x);
}
// v_permlane16_swap exchanges the odd rows (of 16 lanes) of its first operand with the even rows
// of its second, v_permlane32_swap the upper half of the first with the lower half of the second.
__device__ __forceinline__ void swap_rows(float& x, float& y) {
    const auto a = __builtin_amdgcn_permlane16_swap(as_bits(x), as_bits(y), false, false);
    x = as_float(a[0]);
    y = as_float(a[1]);
}
__device__ __forceinline__ void swap_halves(float& x, float& y) {
    const auto a = __builtin_amdgcn_permlane32_swap(as_bits(x), as_bits(y), false, false);
    x = as_float(a[0]);
    y = as_float(a[1]);
}
__device__ __forceinline__ float sum_wave(float x) {
    x = sum16(x);
    float y = x;
    swap_rows(x, y);
    x += y;
    y = x;
    swap_halves(x, y);
    return x + y;
}
// Largest of eight magnitudes each over the lanes l, l + 16, l + 32, l + 48, two values an exchange:
// lane l is left with those numbered first_of(l) and the one after.
__device__ __forceinline__ f32x2 max_rows(float (&v)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        swap_rows(v[e], v[e + 4]);
        v[e] = larger(v[e], v[e + 4]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        swap_halves(v[e], v[e + 2]);
        v[e] = larger(v[e], v[e + 2]);
    }
    return f32x2{v[0], v[1]};
}
__device__ __forceinline__ int first_of(int lane) {
    return ((lane >> 4) & 1) * 4 + (lane >> 5) * 2;
}

// ---- quantisation ---------------------------------------------------------------

// Scale of a block whose largest magnitude is amax, and what its values are multiplied by; each
// step one IEEE operation, as for fp8bs_quantize_1x128.
__device__ __forceinline__ float block_scale(float amax, float& inv) {
    const float a = amax < 1e-4f ? 1e-4f : amax;
    inv = 448.0f / a;
    return a / 448.0f;
}
// Two blocks' maxima over a pair of lanes: the lane whose bit is set goes on with b, the other
// with a.  (Unary plus: a conditional of two variables would be one of their addresses.)
template <int CTRL>
__device__ __forceinline__ float join(float a, float b, bool bit) {
    const float own = bit ? +b : +a, other = bit ? +a : +b;
    return larger(own, moved<CTRL>(other));
}
// Largest magnitudes of N blocks that 16 neighbouring lanes share, from the lanes' own: lane seg is
// left with block_of<N>(seg)'s.  Neighbours 1 and 2 away by quad permutations, 4 and 8 by
// rotations, which keep the lower bits.
template <int N>
__device__ __forceinline__ float block_max(const float (&m)[N], int seg) {
    static_assert(N == 1 || N == 2 || N == 4 || N == 6, "");
    float z;
    if constexpr (N == 1) {
        z = larger(m[0], moved<0xB1>(m[0]));
        z = larger(z, moved<0x4E>(z));
    } else if constexpr (N == 2) {
        z = join<0xB1>(m[0], m[1], seg & 1);
        z = larger(z, moved<0x4E>(z));
    } else {
        z = join<0x4E>(join<0xB1>(m[0], m[1], seg & 1), join<0xB1>(m[2], m[3], seg & 1), seg & 2);
    }
    if constexpr (N == 6) {
        float y = join<0xB1>(m[4], m[5], seg & 1);
        y = larger(y, moved<0x4E>(y));
        z = join<0x124>(z, y, seg & 4);
    } else {
        z = larger(z, moved<0x124>(z));
    }
    return larger(z, moved<0x128>(z));
}
// The block of which lane seg holds the maximum above; each is in one lane below N.
template <int N>
__device__ __forceinline__ int block_of(int seg) {
    return N == 6 ? ((seg & 4) ? 4 + (seg & 1) : seg & 3) : seg & (N - 1);
}

template <int N, int J = 0>
__device__ __forceinline__ void factors(float inv, float (&all)[N]) {
    if constexpr (J < N) {
        all[J] = moved<0x150 + J>(inv);        // lane J's, to all 16
        factors<N, J + 1>(inv, all);
    }
}
// Scales of N blocks that 16 neighbouring lanes share, top[j] the lane's own largest magnitude in
// block j.  A lane divides for its block_of() alone, so that a division is made once and not N
// times.  Gives that block's scale, and all blocks' factors.
template <int N>
__device__ __forceinline__ float block_scales(const float (&top)[N], int seg, float (&inv)[N]) {
    float f;
    const float s = block_scale(block_max(top, seg), f);
    factors<N>(f, inv);
    return s;
}
// A NaN leaves the maximum as it is: the operand that is a number wins.
__device__ __forceinline__ float max8(const float (&v)[8]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
    return m;
}
// e4m3 codes of v * inv.  No clamp: |v| is at most the block's maximum, so the product passes
// 448 by a rounding of FP32 at most, and the conversion gives 448 up to 464 (checked on MI355X;
// it gives 0xFF for every NaN).
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], float inv) {
    u32x2 out;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
        out[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv,
                                                           w, true);
    }
    return out;
}

// Workgroup b runs on XCD b % 8, each with an L2 of its own: XCD x takes a contiguous eighth of
// the units, so that neighbouring units' parts of a cache line meet in one L2.
__device__ __forceinline__ uint32_t xcd_order(uint32_t unit, uint32_t units) {
    const uint32_t each = units >> 3;
    return unit < each * 8 ? (unit & 7) * each + (unit >> 3) : unit;
}

#endif  // __HIPCC__

}  // namespace layer
}  // namespace fp8bs

#endif  // FP8BS_LAYER_H

// fp8bs_mx_grad.hip -- the two products of the gated block's backward pass on gfx950:
//
//     da = [dg | du] W        contraction over W's rows (2f), A as it lies
//     db = [dg | du]^T X      contraction over the tokens, A transposed (a_t)
//
// [dg | du] in bf16, W and X in MXFP4 with their 4-bit blocks along the output columns, where
// no matrix instruction can apply the scales: the values are widened to bf16 (exactly) on
// their way into LDS, so the second operand is read from memory at 4.25 bits a value and no
// widened or transposed copy of it exists.  FP32 accumulation, v_mfma_f32_16x16x32_bf16.
//
// A step is 64 rows of the contraction.  The second operand (and a transposed A) lies in LDS
// as [64 rows][columns], and its fragments are read with the transpose load ds_read_b64_tr_b16
// (lane s of 16 points at 8 bytes of row s / 4, piece s % 4; lane t gets column t of four
// rows).  The units of an LDS row are permuted by a key of the row so that what one read or
// store touches falls into different banks.
//
// Widening: a thread loads 16 bytes of codes (one row, one 32-value block) and their exponent
// a step ahead, turns them into pairs with v_cvt_scalef32_pk_bf16_fp4 and stores the 64 bytes.
// Tiles, stages, barrier and copy schedule are those of fp8bs_mx_gemm.hip.  Problems of few tiles
// run both products in one launch, and split a long contraction into parts, FP32, that a second
// launch adds in their order (no atomics; the split depends on sizes only).
//
// Bound by the matrix cores at the clock that power allows (2.1-2.2 GHz; busy 53-57% of the CUs'
// busy time in da, 45-58% in db), by the widening (a tenth of a step) and by filling and storing a
// tile (8 us at 256x256).  8192 rows, f = 2048, k = 7168: da 399-445 us, db 363-450, by card
// (1.1-1.2 and 1.1-1.3 PFLOP/s; the matrix cores fed from registers alone, random operands: 2.15).
#include <math.h>

#include <type_traits>

#include "fp8bs_mx_tile.h"

namespace fp8bs {
namespace mx {
namespace {

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Permutation of a row's 16-byte units, 16 of which span the LDS banks: unit x of row k lies at
// x ^ unit_key(k), with bit 0 turned by bit 4 of x.  A transpose read takes 32 lanes at a time:
// 8 rows (k % 4, and k / 8 even or odd) by two units, 16 places; a store of widened values 16
// lanes: every fourth unit of two rows, 16 places too (without the turn of bit 0, two lanes to
// a place: 43% of the LDS's busy cycles were conflicts).
__device__ __forceinline__ int unit_key(int k) { return ((k & 3) << 1) | (((k >> 3) & 1) << 3); }
__device__ __forceinline__ int unit_at(int x, int key) {
    const int high = x >> 4;
    return high * 16 + ((x & 15) ^ key ^ (high & 1));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : bytes > 0xFFFFFFFFll ? 0xFFFFFFFFll : bytes;
    return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)(uint32_t)n, 0x00020000);
}

// LDS of a workgroup with b x b tiles: two stages of both operands, the list of tiles.
constexpr int grad_lds(int b, int layout) {
    return 2 * 2 * b * 128 + (layout == kContiguous ? (kMaxListed + 1) * 4 : 0);
}

// One workgroup's work, `first` of `grid` persistent ones.
template <int BM, int BN, int WM, int WN, bool AT, int LAYOUT, int EPI, bool SPLIT>
__device__ __forceinline__ void grad_units(const MxParams& p, uint8_t* smem, int first, int grid) {
    constexpr int NW = WM * WN, TM = BM / WM / 16, TN = 4;
    static_assert(BN / WN == 64 && BN / 32 == NW, "one 16-byte piece of codes per thread");
    constexpr int A_COPIES = BM / 8 / NW;
    constexpr int B_OFF = BM * 128, STAGE = B_OFF + BN * 128;
    uint32_t* list = (uint32_t*)(smem + 2 * STAGE);            // (contiguous only)

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int j = lane & 15, q = lane >> 4;

    int m_tiles = p.m_tiles;
    if constexpr (LAYOUT == kContiguous) {
        if (wave == 0) {
            const int n = list_tiles<BM, LAYOUT>(p, list);
            if (lane == 0) list[kMaxListed] = (uint32_t)n;
        }
        __syncthreads();
        m_tiles = __builtin_amdgcn_readfirstlane(list[kMaxListed]);
    }
    const int splits = SPLIT ? p.splits : 1;
    const int units = m_tiles * p.n_tiles * (LAYOUT == kBlocks ? p.num_groups : 1) * splits;
    // unit u: a tile, or part u % splits of its steps (which may be none)
    auto work_at = [&](int u, Tile& t) {
        tile_at<BM, BN, LAYOUT>(p, list, m_tiles, SPLIT ? u / splits : u, t);
        if constexpr (SPLIT) {
            const int part = u % splits, from = t.c0;
            const int64_t steps = t.c1 - t.c0;
            t.c0 = from + (int)(steps * part / splits);
            t.c1 = from + (int)(steps * (part + 1) / splits);
        }
    };
    int u = first;
    if (u >= units) return;

    // ---- A's copies: rows as in fp8bs_mx_gemm.hip, or 64 rows of BM columns (AT) ----
    uint32_t a_row_at[A_COPIES];
    int a_col[A_COPIES];
#pragma unroll
    for (int k = 0; k < A_COPIES; ++k) {
        const int ins = wave * A_COPIES + k;
        if constexpr (AT) {
            const int pos = ins * 1024 + 16 * lane, row = pos / (2 * BM), in_row = pos % (2 * BM);
            // (unit_at is its own inverse)
            a_col[k] = unit_at(in_row >> 4, unit_key(row)) * 8;
            a_row_at[k] = (uint32_t)row * (uint32_t)p.a_row;
        } else {
            const int at = ins * 8 + (lane >> 3);
            const int strip = at / (16 * TM), i = at / 16 % TM, r = at % 16;
            a_col[k] = 8 * ((lane & 7) ^ (lane >> 3));
            a_row_at[k] = (uint32_t)(strip * 16 * TM + TM * r + i) * (uint32_t)p.a_row;
        }
    }
    // ---- the second operand: this thread's row and 32-value block of a step ----
    const int b_row = (int)threadIdx.x / NW, b_block = (int)threadIdx.x % NW;
    int b_to[4];                               // LDS offsets of its values, eight by eight
#pragma unroll
    for (int h = 0; h < 4; ++h)
        b_to[h] = B_OFF + b_row * 2 * BN + unit_at(4 * b_block + h, unit_key(b_row)) * 16;

    const uint32_t lds0 = lds_offset(smem);
    // A step: where its rows start, and this lane's offsets in the operands.
    struct Step {
        i32x4 a;
        uint32_t a_at;                         // scalar offset of A's copies
        int row0, rows;                        // first row of the contraction, rows that exist
    };
    Tile cur, nxt;
    Step next = {};
    uint32_t a_off[A_COPIES];
    uint32_t b_off = 0;                        // byte of the codes within a row
    int b_word = 0;                            // word row of the exponents
    int nu = u, nc = 0;
    int block = 0;                             // kBlocks: the block of step nc (read a step early)
    auto open = [&] {
        const int b = nxt.n0 + 32 * b_block < p.n ? b_block : 0;   // (past the last column: unused)
        b_off = (uint32_t)(nxt.n0 / 2 + 16 * b);
        b_word = nxt.n0 / 128 + b / 4;
#pragma unroll
        for (int k = 0; k < A_COPIES; ++k) {
            if constexpr (AT)
                a_off[k] = a_row_at[k] + 2u * (uint32_t)(nxt.m0 + a_col[k] < p.m ? a_col[k] : 0);
            else
                a_off[k] = a_row_at[k] + 2u * (uint32_t)a_col[k];
        }
    };
    auto locate = [&] {
        // (kBlocks: step nc of an expert is half nc % 2 of its 128-token block nc / 2)
        if constexpr (LAYOUT == kBlocks) {
            next.row0 = block * 128 + (nc & 1) * 64;
            block = p.blocks[p.num_groups + 1 + ((nc + 1) >> 1)];      // for the step after
        } else {
            next.row0 = nc * 64;
        }
        next.rows = p.depth - next.row0;
        if constexpr (AT) {
            next.a = descriptor(p.a + (int64_t)next.row0 * p.a_row + 2 * (int64_t)nxt.m0,
                                64 * p.a_row - 2 * (int64_t)nxt.m0);
            next.a_at = 0;
        } else {
            next.a = descriptor(p.a + (int64_t)nxt.m0 * p.a_row, nxt.rows * p.a_row);
            next.a_at = (uint32_t)nc * 128u;
        }
    };
    auto seek = [&](int from) {
        for (nu = from; nu < units; nu += grid) {
            work_at(nu, nxt);
            if (nxt.c0 < nxt.c1) {
                open();
                nc = nxt.c0;
                if constexpr (LAYOUT == kBlocks) block = p.blocks[p.num_groups + 1 + (nc >> 1)];
                return true;
            }
        }
        return false;
    };
    auto advance = [&] {
        if (nu >= units || (++nc >= nxt.c1 && !seek(nu + grid))) return;
        locate();
    };
    auto copy_part = [&](const Step& x, const uint32_t (&off)[A_COPIES], int stage, int k) {
        copy16(x.a, off[k], x.a_at, lds0 + (uint32_t)(stage * STAGE + (wave * A_COPIES + k) * 1024));
    };
    int codes_g = 0;                           // the expert that the loaded codes serve
    struct Codes {
        u32x4 w;
        uint32_t exponents;
        int expert;                            // kBlocks: of the row; else whether it exists
    };
    auto live = [&](const Codes& x) { return LAYOUT == kBlocks ? x.expert == codes_g : x.expert != 0; };
    // The codes of the next step.  Rows past the contraction's end, and rows that hold no token,
    // meet rows of zeros in A: whatever they read as, they only have to be finite.
    auto load_codes = [&](Codes& x) {
        const int64_t group = AT ? 0 : nxt.g;
        const int k = min(b_row, next.rows - 1);
        const auto codes = buffer(p.b + (group * p.depth + next.row0) * p.b_row, 64 * p.b_row);
        const auto words = buffer(p.sfb + group * p.kwords * p.sfb_ld + next.row0,
                                  ((int64_t)p.kwords * p.sfb_ld - next.row0) * 4);
        x.w = __builtin_amdgcn_raw_buffer_load_b128(codes, (uint32_t)k * (uint32_t)p.b_row + b_off, 0, 0);
        x.exponents = __builtin_amdgcn_raw_buffer_load_b32(
            words, ((uint32_t)b_word * (uint32_t)p.sfb_ld + (uint32_t)k) * 4u, 0, 0);
        x.expert = LAYOUT == kBlocks ? p.group_data[next.row0 + k] : b_row < next.rows;
        codes_g = nxt.g;
    };
    const int b_shift = 8 * (b_block & 3);
    auto scale_of = [&](const Codes& x) {
        return live(x) ? scale_value((x.exponents >> b_shift) & 255u) : 1.0f;
    };
    // 16 of this thread's 32 values into LDS
    auto widen_half = [&](const Codes& x, float scale, int stage, auto half_const) {
        constexpr int HALF = decltype(half_const)::value;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = x.w[2 * HALF + i];
            u32x4 v;
            v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
            v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
            v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
            v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
            *(u32x4*)(smem + stage * STAGE + b_to[2 * HALF + i]) = v;
        }
    };
    constexpr std::integral_constant<int, 0> kFirst{};
    constexpr std::integral_constant<int, 1> kSecond{};

    // ---- fragments: 8 values 32 h + 8 q .. + 7 of the contraction ----
    const int read_key = ((j >> 2) << 1) | ((q & 1) << 3); // unit_key of every row a lane points at
    const int piece = (j & 3) >> 1;                        // unit of a block's two that it points at
    const int read_row = 8 * q + (j >> 2);
    int a_rd[AT ? TM : 2], b_rd[TN];
    if constexpr (AT) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
            a_rd[i] = read_row * 2 * BM + unit_at(2 * (wm * TM + i) + piece, read_key) * 16 + (j & 1) * 8;
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            a_rd[h] = (wm * 16 * TM + j) * 128 + (((4 * h + q) ^ (j & 7)) << 4);
    }
#pragma unroll
    for (int n = 0; n < TN; ++n)
        b_rd[n] = B_OFF + read_row * 2 * BN + unit_at(2 * (wn * 4 + n) + piece, read_key) * 16 + (j & 1) * 8;
    auto read_columns = [&](int at, int width) {           // rows at .. at + 3 and at + 4 .. at + 7
        const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (LDS_AS i16x4*)(LDS_AS void*)(smem + at)));
        const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (LDS_AS i16x4*)(LDS_AS void*)(smem + at + 4 * width)));
        return u32x4{lo[0], lo[1], hi[0], hi[1]};
    };
    auto read_a = [&](int base, int h, int i) {
        if constexpr (AT) return read_columns(base + a_rd[i] + h * 64 * BM, 2 * BM);
        else return *(const u32x4*)(smem + base + a_rd[h] + 2048 * i);
    };
    auto read_b = [&](int base, int h, int n) {
        return read_columns(base + b_rd[n] + h * 64 * BN, 2 * BN);
    };

    f32x4 acc[TM][TN];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int n = 0; n < TN; ++n) acc[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    };
    // Lane (j, q) holds rows m0 + 16 TM wm + (AT: 16 i + j, else TM j + i) and, in block n,
    // columns n0 + 64 wn + 16 n + 4 q .. + 3.
    auto store = [&](const Tile& t, int part) {
        const int64_t row0 = LAYOUT == kBlocks ? (int64_t)t.g * p.m : (int64_t)0;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = t.m0 + wm * 16 * TM + (AT ? 16 * i + j : TM * j + i);
            bool ok = r - t.m0 < t.rows;
            if constexpr (LAYOUT == kContiguous) ok = ok && p.group_data[r] == t.g;
            if (SPLIT && splits > 1) {
                if (!ok) continue;
                const int64_t all = (LAYOUT == kBlocks ? p.num_groups : 1) * (int64_t)p.m;
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    const int col = t.n0 + wn * 64 + 16 * n + 4 * q;
                    if (col < p.n) *(f32x4*)(p.part + (part * all + row0 + r) * p.n + col) = acc[i][n];
                }
            } else if constexpr (EPI == kStore) {
                // Lanes q and q + 1 exchange pieces of two blocks, so that a lane holds 16
                // consecutive bytes and a store writes 64 of every row (with 32 a store, 16384
                // rows of eight experts took 2200 us instead of 2115, all kernels together).
#pragma unroll
                for (int n = 0; n < TN; n += 2) {
                    u32x4 w;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const f32x4 v = acc[i][n], x = acc[i][n + 1];
                        const auto both = __builtin_amdgcn_permlane16_swap(
                            pack_bf16(v[2 * h], v[2 * h + 1]), pack_bf16(x[2 * h], x[2 * h + 1]), false, false);
                        w[h] = both[0];
                        w[2 + h] = both[1];
                    }
                    const int col = t.n0 + wn * 64 + 16 * (n + (q & 1)) + 8 * (q >> 1);
                    if (ok && col < p.n)                   // (k is a multiple of 128)
                        *(u32x4*)((uint16_t*)p.d + (row0 + r) * p.d_ld + col) = w;
                }
            } else {
                if (!ok) continue;
#pragma unroll
                for (int n = 0; n < TN; ++n) {
                    const int col = t.n0 + wn * 64 + 16 * n + 4 * q;
                    if (col >= p.n) continue;
                    float* d = (float*)p.d + (row0 + r) * p.d_ld + col;
                    f32x4 v = acc[i][n];
                    if (p.accumulate) v += *(const f32x4*)d;
                    *(f32x4*)d = v;
                }
            }
        }
    };

    constexpr int GROUPS = 2 * TM, AHEAD = 3, LAST = GROUPS - AHEAD;
    constexpr int PER = (A_COPIES + GROUPS / 2) / (GROUPS / 2 + 1);
    clear();
    const bool any = seek(u);                  // (no step at all: only zeros to store)
    Codes codes = {};
    if (any) {
        locate();
        load_codes(codes);
#pragma unroll
        for (int k = 0; k < A_COPIES; ++k) copy_part(next, a_off, 0, k);
        const float scale = scale_of(codes);
        widen_half(codes, scale, 0, kFirst);
        widen_half(codes, scale, 0, kSecond);
        advance();
        load_codes(codes);
    }
    wait_and_meet();
    float scale = 0.0f;
    if (any) {
#pragma unroll
        for (int k = 0; k < PER * AHEAD && k < A_COPIES; ++k) copy_part(next, a_off, 1, k);
        scale = scale_of(codes);
        widen_half(codes, scale, 1, kFirst);
        widen_half(codes, scale, 1, kSecond);
    }
    u32x4 fa[4], fb[2][TN];
    int base = 0;
#pragma unroll
    for (int n = 0; n < TN; ++n) fb[0][n] = read_b(0, 0, n);
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) fa[g] = read_a(0, 0, g);

    for (; u < units; u += grid) {
        work_at(u, cur);
        for (int c = cur.c0; c < cur.c1; ++c) {
            const int other = base ? 0 : STAGE;
            const Step started = next;                     // its first copies are out
            uint32_t started_off[A_COPIES];
#pragma unroll
            for (int k = 0; k < A_COPIES; ++k) started_off[k] = a_off[k];
            advance();
            load_codes(codes);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int h = g / TM, i = g % TM;
                if (g == LAST) {
                    wait_and_meet();
                    // (the codes have landed with the copies; used any earlier, as the compiler
                    // would have it, they stalled the step for their latency)
                    asm volatile("" : "+v"(codes.w), "+v"(codes.exponents), "+v"(codes.expert));
                }
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    if (g >= LAST) {
                        if ((g - LAST) * PER + k < A_COPIES)
                            copy_part(next, a_off, base ? 1 : 0, (g - LAST) * PER + k);
                    } else if ((g + AHEAD) * PER + k < A_COPIES) {
                        copy_part(started, started_off, base ? 0 : 1, (g + AHEAD) * PER + k);
                    }
                }
                const int ahead = g + AHEAD;
                fa[ahead % 4] = ahead < GROUPS ? read_a(base, ahead / TM, ahead % TM)
                                               : read_a(other, 0, ahead - GROUPS);
                if (g < TN) fb[1][g] = read_b(base, 1, g);
                if (g == LAST) {
#pragma unroll
                    for (int n = 0; n < TN; ++n) fb[0][n] = read_b(other, 0, n);
                    scale = scale_of(codes);
                    widen_half(codes, scale, base ? 1 : 0, kFirst);
                }
                if (g == LAST + 1) widen_half(codes, scale, base ? 1 : 0, kSecond);
#pragma unroll
                for (int n = 0; n < TN; ++n)
                    acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, fb[h][n]), __builtin_bit_cast(bf16x8, fa[g % 4]),
                        acc[i][n], 0, 0, 0);
                __builtin_amdgcn_sched_barrier(0);
            }
            base = other;
        }
        store(cur, u % splits);
        clear();
    }
}

template <int B, int WM, int WN, bool AT, int LAYOUT, int EPI>
__global__ void __launch_bounds__(64 * WM * WN, 2) mx_grad_kernel(const MxParams p) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[grad_lds(B, LAYOUT)];
    grad_units<B, B, WM, WN, AT, LAYOUT, EPI, false>(p, smem, logical_block(), gridDim.x);
}

// Both products of a small or medium problem side by side: workgroups below `split` work on da, the
// others on db.  (Without SPLIT both are whole: the arithmetic of parts costs 0.6 to 2.5 us.)
template <int LAYOUT, int EPI, bool SPLIT>
__global__ void __launch_bounds__(256, 2) mx_grad_pair_kernel(const MxParams a, const MxParams b,
                                                              int split) {
    __shared__ __attribute__((aligned(1024))) uint8_t smem[grad_lds(128, LAYOUT)];
    const int id = blockIdx.x;
    if (id < split)
        grad_units<128, 128, 2, 2, false, LAYOUT, kStore, SPLIT>(a, smem, id, split);
    else
        grad_units<128, 128, 2, 2, true, LAYOUT == kContiguous ? kBlocks : kDense, EPI, SPLIT>(
            b, smem, id - split, gridDim.x - split);
}

// The parts of split products added in their order: four values a thread, the first `split`
// workgroups those of a (bf16; contiguous: valid rows only), the others b's.
template <int LAYOUT, int EPI>
__global__ void __launch_bounds__(256) mx_grad_sum_kernel(const MxParams a, const MxParams b, int split) {
    const bool first = (int)blockIdx.x < split;
    const MxParams& p = first ? a : b;
    const int64_t rows = (!first && LAYOUT == kContiguous ? p.num_groups : 1) * (int64_t)p.m;
    const int64_t all = rows * p.n;
    const int64_t stride = (int64_t)(first ? split : gridDim.x - split) * 1024;
    int64_t at = ((int64_t)(first ? blockIdx.x : blockIdx.x - split) * 256 + threadIdx.x) * 4;
    for (; at < all; at += stride) {
        if (LAYOUT == kContiguous && first) {
            const int64_t r = at / p.n;
            const int e = expert_of(p, (int)(r >> 7));
            if (e < 0 || p.group_data[r] != e) continue;
        }
        f32x4 sum = *(const f32x4*)(p.part + at);
        for (int s = 1; s < p.splits; ++s) sum += *(const f32x4*)(p.part + s * all + at);
        if (EPI == kStoreF32 && !first) {
            float* d = (float*)p.d + at;
            if (p.accumulate) sum += *(const f32x4*)d;
            *(f32x4*)d = sum;
        } else {
            *(u32x2*)((uint16_t*)p.d + at) = u32x2{pack_bf16(sum[0], sum[1]), pack_bf16(sum[2], sum[3])};
        }
    }
}

typedef void (*KernelFn)(MxParams);

// Workgroups of two jobs that share a launch, at most `most` (two or more; a job keeps one).
void share(int64_t& a, int64_t& b, int64_t most) {
    if (a + b <= most) return;
    const int64_t part = (int64_t)(most * (double)a / (double)(a + b));
    a = b == 0 ? most : a == 0 ? 0 : part < 1 ? 1 : part < most ? part : most - 1;
    b = most - a;
}

// 128x128 tiles of a product's grid (an upper bound for the contiguous layout)
int64_t small_tiles(const MxParams& p, int layout, int groups) {
    return (int64_t)(layout == kBlocks ? groups : 1) * ((p.m + 127) / 128) * ((p.n + 127) / 128);
}
void small_grid(MxParams& p, int layout) {
    p.m_tiles = (p.m + 127) / 128;
    p.n_tiles = (p.n + 127) / 128;
    p.raster = 8;
    p.first = 0;
    p.last = layout == kContiguous ? p.m / 128 : p.m_tiles;
}

// Steps of a tile (kBlocks: of an expert, on average).
double mean_steps(const MxParams& p, int layout, int groups) {
    return layout == kBlocks ? (double)p.chunks / groups : p.chunks;
}

// 256x256 tiles, one workgroup per CU: 1.5 us a step of 64 rows and 8 to fill and store.
// 128x128, two per CU: 1.1 and 8; 0.9 and 3 while every workgroup has a CU for itself.
// Measured, 256x256 against 128x128 (one of the slower cards), 64 steps: 32 large tiles 98
// against 59 us, 128: 107 against 79, 256: 121 against 159, 448: 224 against 301, 896: 438
// against 536; 32 steps, 128 tiles: 57 against 46, 224: 57 against 77; 16 steps, 128: 32
// against 26; 128 steps, 448: 446 against 597.
struct Cost {
    double large, small;                       // us
    bool large_pays() const { return large <= small; }
    double least() const { return large_pays() ? large : small; }
};
Cost cost(const MxParams& p, int layout, int groups, int num_cus) {
    auto tiles = [&](int b) {
        return (layout == kBlocks ? groups : 1.0) * ((p.m + b - 1) / b) * ((p.n + b - 1) / b);
    };
    const double steps = mean_steps(p, layout, groups);
    if (p.splits > 1) return {1e30, 0.9 * steps / p.splits + 3 + 6};
    return {ceil(tiles(256) / num_cus) * (1.5 * steps + 8),
            tiles(128) <= num_cus ? 0.9 * steps + 3
                                  : ceil(tiles(128) / (2 * num_cus)) * (1.1 * steps + 8)};
}

}  // namespace

// Few tiles of a long contraction: as many parts as 256 workgroups take, of 8 steps at least,
// where the steps saved are worth more than the second launch and the parts' bytes.  The whole
// backward pass with and without: 16384 x 128 x 256 38 against 235 us, 8192 x 512 x 1024 77 against
// 149, 128 x 4096 x 4096 63 against 175, 64 x 2048 x 2048 24 against 71, 1024 x 128 x 1024 21 against 24.
int grad_splits(int layout, const MxParams& p, int groups) {
    const int64_t tiles = small_tiles(p, layout, groups);
    const double steps = mean_steps(p, layout, groups);
    if (tiles < 1 || tiles > 128) return 1;
    int n = (int)(256 / tiles);
    if (n > steps / 8) n = (int)(steps / 8);
    return n >= 2 && 0.9 * (steps - steps / n) > 6 + 0.03 * n * tiles ? n : 1;
}

// Side by side against one after the other, the whole backward pass: 300 x 704 x 1664 31 against
// 40 us, 1024 x 2048 x 2048 78 against 102, 2048 x 1024 x 2048 57 against 80, eight experts 2048 x
// 512 x 1024 38 against 50; 1024 x 2048 x 7168 172 against 164, 4096 x 2048 x 4096 355 against 280.
bool grad_pair_pays(int layout, const MxParams& a, const MxParams& b, int groups, int num_cus) {
    const int layout_b = layout == kContiguous ? kBlocks : kDense;
    const double ta = (double)small_tiles(a, layout, groups) * a.splits;
    const double tb = (double)small_tiles(b, layout_b, groups) * b.splits;
    if (ta + tb > 0x7fffffff || (layout == kContiguous && a.m / 128 > kMaxListed)) return false;
    const double sa = (double)a.chunks / a.splits, sb = mean_steps(b, layout_b, groups) / b.splits;
    // the slots of 2 num_cus workgroups share all steps, but no tile ends before its own
    const double all = (ta * sa + tb * sb) / (2 * num_cus) * 1.1 + 8 * ceil((ta + tb) / (2 * num_cus));
    const double longest = (ta + tb <= num_cus ? 0.9 : 1.1) * (sa > sb ? sa : sb) + 8 +
                           (a.splits > 1 || b.splits > 1 ? 6 : 0);
    return (all > longest ? all : longest) <
           cost(a, layout, groups, num_cus).least() + cost(b, layout_b, groups, num_cus).least() + 3;
}

int launch_grad_pair(int layout, int epilogue, const MxParams* pa, const MxParams* pb, int groups,
                     hipStream_t stream) {
    const int layout_b = layout == kContiguous ? kBlocks : kDense;
    MxParams a = {}, b = {};
    int64_t na = 0, nb = 0, sum_a = 0, sum_b = 0;              // workgroups of both launches
    if (pa) {
        a = *pa;
        small_grid(a, layout);
        na = small_tiles(a, layout, groups) * a.splits;
        if (a.splits > 1) sum_a = ((int64_t)a.m * a.n + 1023) / 1024;
    }
    if (pb) {
        b = *pb;
        small_grid(b, layout_b);
        nb = small_tiles(b, layout_b, groups) * b.splits;
        if (b.splits > 1) sum_b = ((layout_b == kBlocks ? groups : 1) * (int64_t)b.m * b.n + 1023) / 1024;
    }
    if (na + nb == 0) return (int)hipSuccess;
    if (na + nb > 0x7fffffff) return (int)hipErrorInvalidValue;
    const void *fn = nullptr, *add = nullptr;
#define MX_CASE(L, E)                                                            \
    if (layout == L && epilogue == E) {                                          \
        fn = sum_a + sum_b > 0 ? (const void*)mx_grad_pair_kernel<L, E, true>    \
                               : (const void*)mx_grad_pair_kernel<L, E, false>;  \
        add = (const void*)mx_grad_sum_kernel<L, E>;                             \
    }
    MX_CASE(kDense, kStore)
    MX_CASE(kDense, kStoreF32)
    MX_CASE(kContiguous, kStore)
    MX_CASE(kContiguous, kStoreF32)
#undef MX_CASE
    if (!fn) return (int)hipErrorInvalidValue;
    share(na, nb, most_workgroups(2));
    int split = (int)na;
    void* argv[] = {&a, &b, &split};
    const hipError_t err = hipLaunchKernel(fn, dim3((unsigned)(na + nb)), dim3(256), argv, 0, stream);
    if (err != hipSuccess || sum_a + sum_b == 0) return (int)err;
    share(sum_a, sum_b, most_workgroups(8));
    split = (int)sum_a;
    return (int)hipLaunchKernel(add, dim3((unsigned)(sum_a + sum_b)), dim3(256), argv, 0, stream);
}

int launch_grad(int layout, bool a_t, int epilogue, const MxParams& params, int groups,
                int num_cus, hipStream_t stream) {
    MxParams p = params;
    const bool large = cost(p, layout, groups, num_cus).large_pays();
    const int64_t slots = layout == kBlocks ? groups : 1;
    KernelFn fn = nullptr;
#define MX_CASE(AT, L, E)                                                       \
    if (a_t == AT && layout == L && epilogue == E)                              \
        fn = large ? (KernelFn)mx_grad_kernel<256, 2, 4, AT, L, E>              \
                   : (KernelFn)mx_grad_kernel<128, 2, 2, AT, L, E>;
    MX_CASE(false, kDense, kStore)
    MX_CASE(false, kContiguous, kStore)
    MX_CASE(true, kDense, kStore)
    MX_CASE(true, kDense, kStoreF32)
    MX_CASE(true, kBlocks, kStore)
    MX_CASE(true, kBlocks, kStoreF32)
#undef MX_CASE
    if (!fn) return (int)hipErrorInvalidValue;
    const int side = large ? 256 : 128;
    p.m_tiles = (p.m + side - 1) / side;
    p.n_tiles = (p.n + side - 1) / side;
    p.raster = 8;
    const bool listed = layout == kContiguous;
    const int64_t all = listed ? p.m / 128 : slots * p.m_tiles;
    if (all * p.n_tiles > 0x7fffffff) return (int)hipErrorInvalidValue;
    // a launch lists at most kMaxListed tiles along M
    for (int64_t first = 0; first < all; first += kMaxListed) {
        p.first = (int)first;
        p.last = (int)(listed && first + kMaxListed < all ? first + kMaxListed : all);
        int64_t grid = (int64_t)num_cus * (large ? 1 : 2);
        const int64_t most = (p.last - p.first) * (int64_t)p.n_tiles;
        if (grid > most) grid = most;
        void* argv[] = {&p};
        const hipError_t err = hipLaunchKernel((const void*)fn, dim3((unsigned)grid),
                                               dim3(large ? 512 : 256), argv, 0, stream);
        if (err != hipSuccess || !listed) return (int)err;
    }
    return (int)hipSuccess;
}

}  // namespace mx
}  // namespace fp8bs

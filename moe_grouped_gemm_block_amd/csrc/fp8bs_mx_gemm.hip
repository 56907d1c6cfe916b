// fp8bs_mx_gemm.hip -- the matrix kernel of the MXFP4 operators on gfx950: D = A B^T with
// 4-bit operands (32-value blocks along K, power-of-two scales applied by the matrix core)
// and what the operators do with the accumulators (fp8bs_mx.h, Epilogue).
//
// Operands move in steps of 128 bytes -- 256 values -- per row; a step feeds two rounds of
// v_mfma_scale_f32_16x16x128_f8f6f4 (16 cycles each), lane (j, q) = (l % 16, l / 16) holding
// the 16 bytes, one scale block, at byte 16 q of row j's round.
//
// Tile: BM x BN by WM x WN wavefronts, each 16 TM x 64.  B rows are the instruction's first
// operand and A rows its second, so a lane's results belong to one A row.  Rows are dealt to
// the 16-row blocks with strides (A row TM * j + i is row j of block i; B row 4 r + jn is row
// r of block jn): a lane then owns TM neighbouring rows and 16 neighbouring columns, stores
// whole 16-byte pieces and reads its scale words as vectors.  The copies into LDS do the
// dealing: a direct-to-LDS copy writes 1024 consecutive bytes but reads from any address per
// lane.  A gated tile takes half its B rows from the gate and half from the up projection,
// blocks 0-1 and 2-3 of every wavefront, so a lane holds both of each output element.
//
// Pipeline: two stages in LDS.  A step is 2 TM groups of 4 products, one A fragment each;
// fragments are read three groups ahead, into the next step's stage at the end.  Between
// the last read of a stage and the first of the next stands the only barrier of the step:
// past it the stage read out is refilled with the step after next, so a copy has a whole
// step's products (2048 cycles of 256x256) to land.  Copies are inline assembly: the
// compiler knows of no LDS write in flight and adds no waits of its own to the fragment
// reads; the waits for copies are the ones written here.  They write LDS only, no register.
//
// The grid is persistent: workgroup w takes units w, w + grid, ... in an order in which the
// workgroups of an XCD (dealt round-robin) run neighbouring tiles, and copies the next
// unit's first steps while it finishes and stores the present one.
//
// Bound by the clock that power allows (1.9-1.95 GHz; with zero operands everything runs 25%
// faster) and by the products with their fragment reads: the barrier taken out is worth 2-3%,
// the copies 2%, the stores 5% (15% with 8 steps a tile), the activation 1%.
// 4096 x 7168 x 16384: 247 us, 3.9 PFLOP/s (the matrix cores fed from registers alone, random
// operands: 7.0); gated, 33280 rows of eight experts, f = 2048, k = 7168: 500 us, 3.8;
// 16 slots of up to 256 rows, 7168 x 2048: 45 us.
#include <math.h>

#include "fp8bs_mx_tile.h"

namespace fp8bs {
namespace mx {
namespace {

__device__ __forceinline__ i32x8 widen(const i32x4& v) {
    return i32x8{v[0], v[1], v[2], v[3], 0, 0, 0, 0};
}

template <int BM, int BN, int WM, int WN, int LAYOUT, int EPI>
__global__ void __launch_bounds__(64 * WM * WN, 2) mx_gemm_kernel(const MxParams p) {
    constexpr int NW = WM * WN, TM = BM / WM / 16, TN = 4;
    static_assert(BN / WN == 64, "a wavefront has four column blocks");
    constexpr bool GATED = gated(EPI);
    constexpr int COLS = GATED ? BN / 2 : BN;              // output columns of a tile
    constexpr int A_COPIES = BM / 8 / NW, B_COPIES = BN / 8 / NW;
    static_assert(A_COPIES * NW * 8 == BM && B_COPIES * NW * 8 == BN, "whole copies");
    // scale words of a step: two (128 values each) per row, [2][rows], at least one copy
    constexpr int SA_COPIES = (BM * 8 + 1023) / 1024;
    constexpr int SB_COPIES = (BN * 8 + 1023) / 1024;
    static_assert(SA_COPIES + SB_COPIES <= NW, "one scale copy per wavefront");
    constexpr int B_OFF = BM * 128, SA_OFF = B_OFF + BN * 128, SB_OFF = SA_OFF + SA_COPIES * 1024;
    // (the other wavefronts copy nothing into a spare kilobyte, which keeps a step branch-free)
    constexpr int SPARE_OFF = SB_OFF + SB_COPIES * 1024;
    constexpr int STAGE = SPARE_OFF + 1024;
    constexpr bool LISTED = LAYOUT == kContiguous || LAYOUT == kMasked;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE];
    __shared__ uint32_t list[LISTED ? kMaxListed + 1 : 1];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / WN, wn = wave % WN;
    const int j = lane & 15, q = lane >> 4;

    int m_tiles = p.m_tiles;
    if constexpr (LISTED) {
        if (wave == 0) {
            const bool none = LAYOUT == kMasked && p.few > 0 && !any_slot_over(p);
            const int n = none ? 0 : list_tiles<BM, LAYOUT>(p, list);
            if (lane == 0) list[kMaxListed] = (uint32_t)n;
        }
        __syncthreads();
        m_tiles = __builtin_amdgcn_readfirstlane(list[kMaxListed]);
    }
    const int units = m_tiles * p.n_tiles;
    int u = logical_block();
    if (u >= units) return;

    // ---- copies ----
    // Copy `ins` of an operand fills LDS rows 8 ins .. 8 ins + 7 of its tile; lane L fills
    // 16-byte slot L % 8 of row 8 ins + L / 8 with unit slot ^ (row % 8), which spreads the
    // fragment reads over the LDS banks: a 16-byte read takes the lanes in four groups of 16
    // that are not consecutive, and within each no bank comes twice (keys that also use bit
    // 3 of the row, conflict-free for consecutive lanes, measured 58% of the LDS's busy
    // cycles in conflicts).
    // (Where K / 128 is odd the upper half of a row's last step does not exist: lanes that
    // would read it read the lower half again, tail_a, tail_s bytes before.)
    uint32_t a_at[A_COPIES], b_at[B_COPIES];
    const uint32_t tail_a = ((lane & 7) ^ (lane >> 3)) >= 4 ? 64u : 0u;
    static_assert(!GATED || B_COPIES == 4, "a wavefront's B copies: two blocks, gate or up");
    const bool b_up = GATED && (wave & 1);
#pragma unroll
    for (int k = 0; k < A_COPIES; ++k) {
        const int ins = wave * A_COPIES + k;
        const int unit = (lane & 7) ^ (lane >> 3);
        const int at = ins * 8 + (lane >> 3);              // LDS row
        const int strip = at / (16 * TM), i = at / 16 % TM, r = at % 16;
        a_at[k] = (uint32_t)(strip * 16 * TM + TM * r + i) * (uint32_t)p.a_row + 16u * unit;
    }
#pragma unroll
    for (int k = 0; k < B_COPIES; ++k) {
        const int ins = wave * B_COPIES + k;
        const int unit = (lane & 7) ^ (lane >> 3);
        const int at = ins * 8 + (lane >> 3);
        const int strip = at / 64, jn = at / 16 % 4, r = at % 16;
        const int row = GATED ? strip * 32 + 2 * r + (jn & 1) : strip * 64 + 4 * r + jn;
        b_at[k] = (uint32_t)row * (uint32_t)p.b_row + 16u * unit;
    }
    // scale copies, one per wavefront: waves 0 .. SA_COPIES-1 bring A's, the next B's
    const bool sa_mine = wave < SA_COPIES;
    const bool sb_mine = !sa_mine && wave < SA_COPIES + SB_COPIES;
    uint32_t s_row = 0, s_word = 0, s_lds = 0;             // row of the tile, word row (0, 1)
    {
        const int rows = sa_mine ? BM : BN;
        const int ins = sa_mine ? wave : wave - SA_COPIES;
        const int word = ins * 256 + lane * 4;             // of the [2][rows] words
        const int h = word / rows, r = word % rows;
        s_word = h < 2 ? (uint32_t)h : 0u;
        s_row = (uint32_t)(GATED && !sa_mine && r >= COLS ? r - COLS + p.n : r);
        if (h > 1) s_row = 0;                              // past the words: a harmless read
        s_lds = (uint32_t)(sa_mine ? SA_OFF + ins * 1024 : sb_mine ? SB_OFF + ins * 1024 : SPARE_OFF);
    }

    const uint32_t lds0 = lds_offset(smem);
    struct Source {
        i32x4 a, b, s;
        uint32_t s_at;                                     // this lane's offset in the scale words
        uint32_t s_ld;                                     // bytes of a word row
    };
    auto open = [&](const Tile& t, Source& s) {
        const int64_t group = (int64_t)t.g * (GATED ? 2 * p.n : p.n);
        s.a = descriptor(p.a + ((int64_t)t.slot * p.m + t.m0) * p.a_row, t.rows * p.a_row);
        s.b = descriptor(p.b + (group + t.n0 + (b_up ? p.n : 0)) * p.b_row,
                         (int64_t)(p.n - t.n0) * p.b_row);
        const int64_t words = p.kwords;
        const int ld = sa_mine ? p.sfa_ld : p.sfb_ld, at = sa_mine ? t.m0 : t.n0;
        const int32_t* base = sa_mine ? p.sfa + (int64_t)t.slot * words * ld
                                      : p.sfb + (int64_t)t.g * words * ld;
        s.s = descriptor(base + at, (words * ld - at) * 4);
        s.s_ld = 4u * (uint32_t)ld;
        // rows past the padded end read its last four words (they belong to no result)
        s.s_at = 4u * min(s_row, (uint32_t)(ld - at - 4)) + s_word * s.s_ld;
    };
    // A wavefront's copies of a step, numbered: A's, B's, its part of the scale words.  Past the
    // stream's end they repeat the last step.
    constexpr int COPIES = A_COPIES + B_COPIES + 1;
    struct Step {
        Source s;
        uint32_t at;                                       // byte offset within a row
        uint32_t s_at;                                     // ... within the scale words
        uint32_t tail;                                     // all ones in a half step, else 0
    };
    auto copy_part = [&](const Step& x, int stage, int k) {
        const uint32_t to = lds0 + (uint32_t)(stage * STAGE);
        if (k < A_COPIES)
            copy16(x.s.a, a_at[k] - (tail_a & x.tail), x.at,
                   to + (uint32_t)(wave * A_COPIES + k) * 1024u);
        else if (k < A_COPIES + B_COPIES)
            copy16<LAYOUT == kMasked>(x.s.b, b_at[k - A_COPIES] - (tail_a & x.tail), x.at,
                   to + (uint32_t)(B_OFF + (wave * B_COPIES + k - A_COPIES) * 1024));
        else
            copy16(x.s.s, x.s.s_at - (s_word * x.s.s_ld & x.tail), x.s_at, to + s_lds);
    };

    // ---- fragment and scale reads ----
    const int key = j & 7;
    int a_rd[2], b_rd[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        a_rd[h] = (wm * 16 * TM + j) * 128 + (((4 * h + q) ^ key) << 4);
        b_rd[h] = B_OFF + (wn * 64 + j) * 128 + (((4 * h + q) ^ key) << 4);
    }
    const int sa_rd = SA_OFF + (wm * 16 * TM + TM * j) * 4;
    const int sb_rd = SB_OFF + (GATED ? wn * 32 + 2 * j : wn * 64 + 4 * j) * 4;
    auto read_a = [&](int base, int h, int i) {
        return *(const i32x4*)(smem + base + a_rd[h] + 2048 * i);
    };
    auto read_b = [&](int base, int h, int n) {
        return *(const i32x4*)(smem + base + b_rd[h] + 2048 * n);
    };
    // Words of the 128 values of round h; the lane's block is their byte q, shifted down when
    // the word is used (the matrix instruction takes a scale register's low byte).  The second
    // round of a row's last step does not exist when K / 128 is odd: its exponents become
    // 2^-127, whose products with any 4-bit values vanish.
    const int shift = 8 * q;
    auto read_sa = [&](int base, int h, int i) {
        return *(const int*)(smem + base + sa_rd + h * BM * 4 + 4 * i);
    };
    auto read_sb = [&](int base, int h, int (&s)[TN]) {
#pragma unroll
        for (int n = 0; n < TN; ++n) {
            const int word = GATED ? (n & 1) + (n >> 1) * COLS : n;
            s[n] = *(const int*)(smem + base + sb_rd + h * BN * 4 + 4 * word);
        }
    };

    f32x4 acc[TM][TN];
    auto clear = [&] {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int n = 0; n < TN; ++n) acc[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
    };

    // ---- the stream of (unit, step): what is multiplied, and what is copied next ----
    Tile cur, nxt;
    Step next = {};                            // the next step to copy: step nc of unit nu
    int nu = u, nc = 0;
    auto locate = [&] {
        next.at = (uint32_t)nc * 128u;
        next.s_at = (uint32_t)nc * 2u * next.s.s_ld;
        next.tail = 2 * nc + 1 < p.kwords ? 0u : ~0u;
    };
    auto advance = [&] {
        if (nu >= units) return;               // past the last unit
        if (++nc >= p.chunks) {
            nu += gridDim.x;
            if (nu >= units) return;
            tile_at<BM, COLS, LAYOUT>(p, list, m_tiles, nu, nxt);
            open(nxt, next.s);
            nc = 0;
        }
        locate();
    };
    // Lane (j, q) holds rows m0 + 16 TM wm + TM j + i, i < TM, and columns n0 + 64 wn + 16 q +
    // 4 v + n (element v of block n); gated: n0 + 32 wn + 8 q + 2 v + n of the gate (blocks 0,
    // 1) and of the up projection (blocks 2, 3).
    auto store = [&](const Tile& t) {
        const int r0 = t.m0 + wm * 16 * TM + TM * j;       // this lane's first row
        bool ok[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int r = r0 + i;
            ok[i] = r - t.m0 < t.rows;
            if constexpr (LAYOUT == kContiguous) ok[i] = ok[i] && p.group_data[r] == t.g;
        }
        if constexpr (EPI == kStore) {
            const int col = t.n0 + wn * 64 + 16 * q;
            const int64_t first = LAYOUT == kMasked ? (int64_t)t.slot * p.m : (int64_t)0;
            const bool whole = col + 16 <= p.n && (p.d_ld & 7) == 0;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                if (!ok[i]) continue;
                uint16_t* d = (uint16_t*)p.d + (first + r0 + i) * p.d_ld + col;
                if (whole) {
                    uint32_t w[8];
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        w[2 * v] = pack_bf16(acc[i][0][v], acc[i][1][v]);
                        w[2 * v + 1] = pack_bf16(acc[i][2][v], acc[i][3][v]);
                    }
                    *(u32x4*)d = u32x4{w[0], w[1], w[2], w[3]};
                    *(u32x4*)(d + 8) = u32x4{w[4], w[5], w[6], w[7]};
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (col + e < p.n) d[e] = to_bf16(acc[i][e & 3][e >> 2]);
                }
            }
        } else {
            // f is a multiple of 32 (of 128 for kGatedQuant): a wavefront's 32 columns exist
            // or do not exist together
            const int col = t.n0 + wn * 32 + 8 * q;
            if (t.n0 + wn * 32 >= p.n) return;
            const int64_t first = LAYOUT == kMasked ? (int64_t)t.slot * p.m : (int64_t)0;
            if constexpr (EPI == kGatedGrad) {
                // dense: rows past the last one, up to a multiple of 64, are written as zeros
                // (the weight's gradient runs over them), and so are rows that hold no token,
                // which may read as anything.  Half of the rows' dh at a time: all at once do
                // not fit the registers beside the accumulators and the next tile's fragments.
                const int last = LAYOUT == kContiguous ? t.m0 + t.rows : (p.m + 63) & -64;
                constexpr int PART = TM / 2;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    u32x4 dh[PART];
#pragma unroll
                    for (int i = 0; i < PART; ++i) {
                        dh[i] = u32x4{0u, 0u, 0u, 0u};
                        if (ok[part * PART + i])
                            dh[i] = *(const u32x4*)(p.dh + (int64_t)(r0 + part * PART + i) * p.n + col);
                    }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < PART; ++i) {
                        const int a = part * PART + i, r = r0 + a;
                        u32x4 dg, du;
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            float g[2], u[2];
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                const uint32_t w = dh[i][v];
                                const float x = __builtin_bit_cast(float, n ? w & 0xFFFF0000u : w << 16);
                                float slope;
                                const float value = activate<true>(p.act, acc[a][n][v], slope);
                                g[n] = x * acc[a][2 + n][v] * slope;
                                u[n] = x * value;
                            }
                            dg[v] = ok[a] ? pack_bf16(g[0], g[1]) : 0u;
                            du[v] = ok[a] ? pack_bf16(u[0], u[1]) : 0u;
                        }
                        if (r < last) {
                            uint16_t* at = (uint16_t*)p.d + (int64_t)r * p.d_ld + col;
                            *(u32x4*)at = dg;
                            *(u32x4*)(at + (int64_t)p.n) = du;
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    float h[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float slope;
                        h[e] = activate<false>(p.act, acc[i][e & 1][e >> 1], slope) *
                               acc[i][2 + (e & 1)][e >> 1];
                    }
                    const int64_t row = first + r0 + i;
                    if constexpr (EPI == kGated) {
                        if (ok[i])
                            *(u32x4*)((uint16_t*)p.d + row * p.d_ld + col) =
                                u32x4{pack_bf16(h[0], h[1]), pack_bf16(h[2], h[3]),
                                      pack_bf16(h[4], h[5]), pack_bf16(h[6], h[7])};
                    } else {
                        uint32_t ex;
                        const uint32_t codes = quantise_row_block(h, ex);
                        if (ok[i]) {
                            *(uint32_t*)((uint8_t*)p.d + row * p.d_ld + col / 2) = codes;
                            if (q == 0) {
                                const int block = col / 32;
                                uint8_t* sf = (uint8_t*)p.d2 +
                                    (((int64_t)t.slot * (p.n / 128) + block / 4) * p.d2_ld + r0 + i) * 4;
                                sf[block & 3] = (uint8_t)ex;
                            }
                        }
                    }
                }
            }
        }
    };

    // Groups of a step; fragments are read AHEAD groups early.  At group LAST the present
    // stage has been read out: the barrier stands there, and from there on, PER a group, go
    // the copies that refill it, the rest of them early in the next step.  (All of them at
    // once kept every wavefront from its products until the eight had pushed 72 kilobyte-wide
    // copies through one address unit.)
    constexpr int GROUPS = 2 * TM, AHEAD = 3, LAST = GROUPS - AHEAD;
    constexpr int PER = (COPIES + GROUPS / 2) / (GROUPS / 2 + 1);
    static_assert(PER * (GROUPS - 1) >= COPIES, "a step's copies fit between two barriers");
    clear();
    tile_at<BM, COLS, LAYOUT>(p, list, m_tiles, u, nxt);
    open(nxt, next.s);
    locate();
#pragma unroll
    for (int k = 0; k < COPIES; ++k) copy_part(next, 0, k);
    advance();
    wait_and_meet();
#pragma unroll
    for (int k = 0; k < PER * AHEAD && k < COPIES; ++k) copy_part(next, 1, k);
    i32x4 fa[4], fb[2][TN];
    int sa[4], sb[2][TN];                      // scale words as read
    int eb[TN];                                // this round's B exponents
    int base = 0;
    auto read_first = [&] {                    // the fragments that a step finds read
#pragma unroll
        for (int n = 0; n < TN; ++n) fb[0][n] = read_b(base, 0, n);
        read_sb(base, 0, sb[0]);
#pragma unroll
        for (int g = 0; g < AHEAD; ++g) {
            fa[g] = read_a(base, 0, g);
            sa[g] = read_sa(base, 0, g);
        }
    };
    read_first();

    for (; u < units; u += gridDim.x) {
        tile_at<BM, COLS, LAYOUT>(p, list, m_tiles, u, cur);
        // A wavefront whose rows all lie past the tile's last one only copies and meets the
        // others, which have the matrix cores to themselves (16 slots of up to 256 rows: 3-4%
        // faster; the dense layout has at most one such row of tiles).
        if (LAYOUT != kDense && wm * 16 * TM >= cur.rows) {
            for (int c = 0; c < p.chunks; ++c) {
                const Step started = next;
                advance();
#pragma unroll
                for (int k = PER * AHEAD; k < COPIES; ++k) copy_part(started, base ? 0 : 1, k);
                wait_and_meet();
#pragma unroll
                for (int k = 0; k < PER * AHEAD && k < COPIES; ++k) copy_part(next, base ? 1 : 0, k);
                base = base ? 0 : STAGE;
            }
            read_first();
            continue;
        }
        for (int c = 0; c < p.chunks; ++c) {
            const int other = base ? 0 : STAGE;
            const int keep = 2 * c + 1 < p.kwords ? 255 : 0;
            const Step started = next;                     // its first copies are out
            advance();
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int h = g / TM, i = g % TM;
                if (g == LAST) {
                    wait_and_meet();
                }
#pragma unroll
                for (int k = 0; k < PER; ++k) {
                    if (g >= LAST) {
                        if ((g - LAST) * PER + k < COPIES) copy_part(next, base ? 1 : 0, (g - LAST) * PER + k);
                    } else if ((g + AHEAD) * PER + k < COPIES) {
                        copy_part(started, base ? 0 : 1, (g + AHEAD) * PER + k);
                    }
                }
                const int ahead = g + AHEAD;
                if (ahead < GROUPS) {
                    fa[ahead % 4] = read_a(base, ahead / TM, ahead % TM);
                    sa[ahead % 4] = read_sa(base, ahead / TM, ahead % TM);
                } else {
                    fa[ahead % 4] = read_a(other, 0, ahead - GROUPS);
                    sa[ahead % 4] = read_sa(other, 0, ahead - GROUPS);
                }
                if (g < TN) fb[1][g] = read_b(base, 1, g);
                if (g == 0) read_sb(base, 1, sb[1]);
                if (g == LAST) {
                    read_sb(other, 0, sb[0]);
#pragma unroll
                    for (int n = 0; n < TN; ++n) fb[0][n] = read_b(other, 0, n);
                }
                const int mask = h ? keep : 255;
                const int ea = (sa[g % 4] >> shift) & mask;
                if (i == 0) {
#pragma unroll
                    for (int n = 0; n < TN; ++n) eb[n] = (sb[h][n] >> shift) & mask;
                }
#pragma unroll
                for (int n = 0; n < TN; ++n)
                    acc[i][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        widen(fb[h][n]), widen(fa[g % 4]), acc[i][n], 4, 4, 0, eb[n], 0, ea);
                __builtin_amdgcn_sched_barrier(0);
            }
            base = other;
        }
        store(cur);
        clear();
    }
}

typedef void (*KernelFn)(MxParams);

struct Shape {
    int bm, bn;
};

template <int LAYOUT, int EPI>
void pick(bool large, KernelFn* fn, Shape* shape, int* threads, int* per_cu) {
    if (large) {
        *fn = mx_gemm_kernel<256, 256, 2, 4, LAYOUT, EPI>;
        *shape = {256, 256};
        *threads = 512;
        *per_cu = 1;
    } else {
        *fn = mx_gemm_kernel<128, 128, 2, 2, LAYOUT, EPI>;
        *shape = {128, 128};
        *threads = 256;
        *per_cu = 2;
    }
}

// What each kernel would take for `rows` rows (masked: of every slot) on `cus` CUs, in
// microseconds; few: the few-rows kernel with its best tile, tm x tn blocks.
struct Times {
    double large, small, few;
    double drawn;                          // the tiled kernels' time to draw the slots' weights
    int tm, tn;
    double tiled() const {
        const double us = large < small ? large : small;
        return us > drawn ? us : drawn;
    }
};

// MI355X, weights not in cache:
// - 256x256 tiles, one workgroup per CU: 1.4 a step of 128 bytes, 5 to fill and store.
// - 128x128, two per CU: 1.0 a step and 5 to fill and store; 0.77 and 2 while every
//   workgroup has a CU for itself.  28 steps, up to 256 tiles: 26 against 43 with 256x256;
//   256 x 7168 x 2048: 11.5 against 19.6; 2048 x 7168 x 2048: 30 against 26; 16 slots of up
//   to 256 rows, gated, f = 2048, k = 7168, all full: 97 against 73, of 32 rows: 52 against 57.
// - few rows, dense: 1.3 a tile, and its rows' and columns' bytes at the 56 GB/s that a CU
//   draws.  1 x 4096 x 7168: 5.9 (16x16 tiles) against 25; 48: 8.1 (32x32) against 26; 128:
//   10.5 (64x32) against 26; 256: 13 (64x64) against 29; 512: 23 against 31; 256 x 7168 x
//   2048: 12.2 against 11.3.
// - slots: tiles follow one another on a CU, which costs the few-rows kernel 3.3 a tile; the
//   others take 1.2 times as long as dense and 2.5.  All CUs draw weights at once, at 6 TB/s (few
//   rows, whose rows come on top) or 4.9.
//   Few-rows against 128x128 tiles, 16 rows a slot, 7168 x 2048: 2 slots 6 against 12, 4: 11
//   against 13-16, 8: 21 against 18, 16: 36 against 33, 32: 68 against 61; gated, f = 2048, k =
//   7168: 2 slots 9 against 33, 8: 26 against 37-46, 16: 48 against 52; 64 rows: 8: 30 against
//   37-49, 16: 59 against 54; 128 rows: 4: 26 against 36, 8: 51 against 50, 16: 96 against 58.
// A masked slot's row count is spread around the expected one; exact: all have just `rows`.
Times times(int layout, int epilogue, const MxParams& p, int groups, int rows, int cus,
            bool exact = false) {
    const double cols = gated(epilogue) ? 2.0 * p.n : p.n, slots = layout == kMasked ? groups : 1;
    auto tiles = [&](int bm, int bn) {                     // tiles that hold rows
        double tall = ceil(rows / (double)bm);
        if (layout == kMasked && !exact) {
            tall = rows / (double)bm + 0.5;
            const double most = ceil(p.m / (double)bm);
            tall = tall < 1 ? 1 : tall > most ? most : tall;
        }
        return slots * tall * ceil(cols / bn);
    };
    const double steps = p.chunks, factor = layout == kMasked ? 1.2 : 1.0;
    const double start = layout == kMasked ? 2.5 : 0;
    const double row_bytes = (double)p.a_row * 1.0625;     // with its exponents
    const double weights = layout == kMasked ? slots * cols * row_bytes : 0;
    const double big = tiles(256, 256), small = tiles(128, 128);
    Times t;
    t.large = start + factor * ceil(big / cus) * (1.4 * steps + 5);
    t.small = start + factor * (small <= cus ? 0.77 * steps + 2
                                             : ceil(small / (2.0 * cus)) * (1.0 * steps + 5));
    t.drawn = weights / 4.9e6;
    t.few = 1e30;
    t.tm = t.tn = 0;
    if (layout == kContiguous) return t;
    for (int tm = 4; tm >= 1; tm /= 2) {                   // (of equals the tallest: reads B least)
        for (int tn = epilogue == kGatedQuant ? 4 : gated(epilogue) ? 2 : 1; tn <= 4; tn *= 2) {
            const double rounds = ceil(tiles(16 * tm, 16 * tn) / cus), block = 16 * row_bytes / 56e3;
            double us = rounds * ((layout == kMasked ? 3.3 : 1.3) + (tm + tn) * block);
            const double drawn = weights / 6e6 + rounds * tm * block;
            if (us < drawn) us = drawn;
            if (us < t.few) {
                t.few = us;
                t.tm = tm;
                t.tn = tn;
            }
        }
    }
    return t;
}

// Up to how many rows the few-rows kernel takes: none or all (dense); masked, slots of which none
// holds more.  The two kernels add along K in different orders, so this follows from sizes and
// the device alone, and where the limit lies below max_m from the counts themselves: both
// kernels are launched and one of them finds that the slots are the other's, which costs it 1.6 to
// 2.6 us.  No result depends on the hint or on the cap on CUs.  (Slot by slot, the two
// kernels' times add: 16 slots of 0 to 256 rows, layer, took 139 us instead of 129.)
int few_rows_limit(int layout, int epilogue, const MxParams& p, int groups, int device_cus) {
    auto gain = [&](int64_t rows) {
        const Times t = times(layout, epilogue, p, groups, (int)(rows < p.m ? rows : p.m),
                              device_cus, true);
        return t.tiled() - t.few;
    };
    if (layout != kMasked) return gain(p.m) > 0 ? p.m : 0;
    if (groups > 4096) return gain(p.m) > 0 ? p.m : 0;     // (every workgroup reads all counts)
    int64_t limit = 0;
    for (int64_t rows = 16; limit < p.m && gain(rows) > 0; rows *= 2) limit = rows;
    if (limit >= p.m) return p.m;
    return limit > 0 && gain(16) > 2 ? (int)limit : 0;
}

}  // namespace

int launch_gemm(int layout, int epilogue, const MxParams& params, int groups,
                int expected_rows, int num_cus, int device_cus, hipStream_t stream) {
    MxParams p = params;
    const int64_t slots = layout == kMasked ? groups : 1;
    p.few = few_rows_limit(layout, epilogue, p, groups, device_cus);
    if (p.few > 0) {
        const int rows = expected_rows < p.few ? expected_rows : p.few;
        // (dense: the tile decides how many parts of K are added)
        const Times t = times(layout, epilogue, p, groups, rows, layout == kDense ? device_cus : num_cus);
        // (slots expected not to be its: a workgroup a CU looks; 16 slots of 128 rows, gated, with one
        // for each of 1024 tiles 67.5 us, so 65.4)
        const int err = launch_stream(layout, epilogue, t.tm, t.tn, p, groups,
                                      epilogue == kGatedGrad ? (rows + 63) & -64 : rows,
                                      expected_rows > p.few ? num_cus : 0x7fffffff, stream);
        if (err != (int)hipSuccess || p.few >= p.m) return err;
        if (expected_rows <= p.few) expected_rows = p.few + 1;
    }
    const Times t = times(layout, epilogue, p, groups, expected_rows, num_cus);
    const bool large = t.large <= t.small;
    KernelFn fn = nullptr;
    Shape s{0, 0};
    int threads = 0, per_cu = 1;
#define MX_CASE(L, E) \
    if (layout == L && epilogue == E) pick<L, E>(large, &fn, &s, &threads, &per_cu);
    MX_CASE(kDense, kStore)
    MX_CASE(kContiguous, kStore)
    MX_CASE(kMasked, kStore)
    MX_CASE(kDense, kGated)
    MX_CASE(kContiguous, kGated)
    MX_CASE(kMasked, kGated)
    MX_CASE(kDense, kGatedQuant)
    MX_CASE(kContiguous, kGatedQuant)
    MX_CASE(kMasked, kGatedQuant)
    MX_CASE(kDense, kGatedGrad)
    MX_CASE(kContiguous, kGatedGrad)
#undef MX_CASE
    if (!fn) return (int)hipErrorInvalidValue;
    const int bn_cols = gated(epilogue) ? s.bn / 2 : s.bn;
    p.m_tiles = (p.m + s.bm - 1) / s.bm;
    p.n_tiles = (p.n + bn_cols - 1) / bn_cols;
    p.raster = 8;
    const bool listed = layout == kContiguous || layout == kMasked;
    const int64_t all = layout == kContiguous ? p.m / 128 : slots * p.m_tiles;
    if (all * p.n_tiles > 0x7fffffff) return (int)hipErrorInvalidValue;
    // a launch lists at most kMaxListed tiles along M
    for (int64_t first = 0; first < all; first += kMaxListed) {
        p.first = (int)first;
        p.last = (int)(listed && first + kMaxListed < all ? first + kMaxListed : all);
        int64_t grid = (int64_t)num_cus * per_cu;
        const int64_t most = (p.last - p.first) * (int64_t)p.n_tiles;
        if (grid > most) grid = most;
        void* argv[] = {&p};
        const hipError_t err = hipLaunchKernel((const void*)fn, dim3((unsigned)grid),
                                               dim3(threads), argv, 0, stream);
        if (err != hipSuccess || !listed) return (int)err;
    }
    return (int)hipSuccess;
}

}  // namespace mx
}  // namespace fp8bs

// fp8bs_dispatch.hip -- tokens to their experts' rows and back, on gfx950.
//
// Assignment i = (token i / topk, choice i % topk) of expert e = ids[i] gets the rank r = number
// of earlier assignments of e.  Its row: contiguous start[e] + r, start[e + 1] = start[e] +
// roundup128(count[e]); masked e m + r, dropped if r >= m.  Ranks come from counts and ballots
// alone, so they do not depend on scheduling.
//
//   dispatch  a[row] = x[token]                      (e4m3 rows with their scales, or values)
//   combine   y[token] = sum_j w[j] d[row_j]         (FP32, j ascending)
//   combine's backward  dd[row_j] = w[j] dy[token],  dw[j] = <dy[token], d[row_j]>
//
// All are bound by HBM: a token's row is read once and written topk times, or the other way.
#include "fp8bs_layer.h"

namespace fp8bs {
namespace layer {
namespace {

constexpr int kMostGroups = 1024;
constexpr int kMostTopk = 64;
constexpr int kMostAssignments = 1 << 30;
constexpr int kMostChunks = 256;

struct DispatchParams {
    const void* ids;            // int32 or int64 [tokens * topk]
    const uint8_t* x;           // rows of row_bytes
    const float* sfx;           // e4m3: [groups of columns][sfx_ld], else nullptr
    uint8_t* a;
    float* sfa;
    int32_t* group_data;        // contiguous: the rows' experts; masked: the slots' rows
    int32_t* positions;
    int32_t* counts;
    int32_t* chunk_counts;      // workspace [chunks][groups]
    int32_t* source;            // workspace [rows]: the row's token
    int ids64, masked;
    int n, topk, tokens;        // n = tokens * topk
    int groups, m;              // m: rows (contiguous) or rows of a slot
    int vectors;                // 16-byte pieces of a row
    int kb;                     // scales of a row (0: none)
    int sfx_ld, sfa_ld;
    int chunk, chunks;          // assignments of a chunk (a multiple of 256)
    int rank_units;             // at least the chunks
    int far;
    uint32_t units;
};

// N choices of a lane, every `step`-th, as they lie: all loads issued before any is looked at.
template <int N>
struct Choices {
    uint32_t lo[N], hi[N];
    // (past the last: that one again)
    __device__ __forceinline__ void load(const DispatchParams& p, int64_t first, int step) {
        const u32x2* wide = (const u32x2*)p.ids;
        const uint32_t* narrow = (const uint32_t*)p.ids;
        if (p.ids64) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t at = first + (int64_t)step * i;
                const u32x2 w = wide[at < p.n ? at : p.n - 1];
                lo[i] = w[0];
                hi[i] = w[1];
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t at = first + (int64_t)step * i;
                lo[i] = narrow[at < p.n ? at : p.n - 1];
                hi[i] = 0;                     // (a negative number is above all experts)
            }
        }
    }
    __device__ __forceinline__ int expert(int i, int groups) const {
        return hi[i] == 0 && lo[i] < (uint32_t)groups ? (int)lo[i] : -1;
    }
};

// Lanes whose expert is this lane's (bits of the group number one by one).
__device__ __forceinline__ uint64_t same_expert(int e, int groups) {
    uint64_t same = ~0ull;
    for (int b = 1; b < groups; b <<= 1) {
        const uint64_t set = __ballot(e & b);
        same &= (e & b) ? set : ~set;
    }
    return same & __ballot(e >= 0);
}

// start[0 .. groups]: first rows of the experts' segments from their counts (contiguous), by
// 256 threads.
__device__ __forceinline__ void segment_starts(const int* counts, int groups, int* start,
                                               int* wave_sums) {
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int each = (groups + 255) / 256;     // at most 4
    int own = 0;
    for (int i = 0; i < each; ++i) {
        const int e = t * each + i;
        if (e < groups) own += (counts[e] + 127) & ~127;
    }
    int before = own;
#pragma unroll
    for (int w = 1; w < 64; w <<= 1) {
        const int o = __shfl_up(before, w, 64);
        if (lane >= w) before += o;
    }
    if (lane == 63) wave_sums[wave] = before;
    __syncthreads();
    before -= own;
    for (int w = 0; w < wave; ++w) before += wave_sums[w];
    for (int i = 0; i < each; ++i) {
        const int e = t * each + i;
        if (e < groups) {
            start[e] = before;
            before += (counts[e] + 127) & ~127;
            if (e == groups - 1) start[groups] = before;
        }
    }
    __syncthreads();
}

// Outputs that follow from the counts: this workgroup's share of the rows' experts, and by
// workgroup 0 the counts.  256 threads.
__device__ __forceinline__ void write_group_data(const DispatchParams& p, const int* counts,
                                                 const int* start, int block, int blocks) {
    if (block == 0)
        for (int e = threadIdx.x; e < p.groups; e += 256) {
            p.counts[e] = counts[e];
            if (p.masked) p.group_data[e] = counts[e] < p.m ? counts[e] : p.m;
        }
    if (p.masked) return;
    for (int64_t r = (int64_t)block * 256 + threadIdx.x; r < p.m; r += (int64_t)blocks * 256) {
        int lo = 0, hi = p.groups;             // the last segment that starts at or before r
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= r) lo = mid; else hi = mid;
        }
        p.group_data[r] = r - start[lo] < counts[lo] ? lo : -1;
    }
}

__device__ __forceinline__ int row_of(const DispatchParams& p, const int* start, int e, int rank) {
    if (e < 0) return -1;
    if (p.masked) return rank < p.m ? e * p.m + rank : -1;
    return start[e] + rank;
}

// ---- many assignments: counts of chunks, ranks, rows -----------------------------

constexpr int kBatch = 8;                      // loads on their way (scales: 16 and more no faster)

// BATCH: choices of a lane at a time (1 where a chunk has no more).
template <int BATCH>
__global__ void __launch_bounds__(256) dispatch_count_kernel(DispatchParams p) {
    __shared__ int hist[kMostGroups];
    for (int c = blockIdx.x; c < p.chunks; c += gridDim.x) {
        for (int e = threadIdx.x; e < p.groups; e += 256) hist[e] = 0;
        __syncthreads();
        const int64_t end = (int64_t)(c + 1) * p.chunk < p.n ? (int64_t)(c + 1) * p.chunk : p.n;
        for (int64_t i = (int64_t)c * p.chunk; i < end; i += 256 * BATCH) {
            Choices<BATCH> ids;
            ids.load(p, i + threadIdx.x, 256);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int e = ids.expert(j, p.groups);
                if (i + 256 * j + threadIdx.x < end && e >= 0) atomicAdd(&hist[e], 1);
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < p.groups; e += 256)
            p.chunk_counts[(int64_t)c * p.groups + e] = hist[e];
        __syncthreads();
    }
}

// A chunk's four wavefronts take a quarter each, in order.  (More workgroups than chunks: the
// others write their share of the rows' experts alone.)  16384 tokens of two choices, eight experts:
// 5 us, like the counts before it bound by latency; of eight choices, 1024 experts, 51 together,
// with every load waited for by itself 118.
template <int BATCH>
__global__ void __launch_bounds__(256) dispatch_rank_kernel(DispatchParams p) {
    __shared__ int total[kMostGroups], start[kMostGroups + 1], wave_sums[4];
    __shared__ int next[4][kMostGroups];       // the wavefront's next rank of each expert
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    for (int c = blockIdx.x; c < p.rank_units; c += gridDim.x) {
        for (int e = t; e < p.groups; e += 256) {
            total[e] = 0;
            for (int w = 0; w < 4; ++w) next[w][e] = 0;
        }
        const int quarter = p.chunk / 4;
        const int64_t first = (int64_t)c * p.chunk + (int64_t)wave * quarter;
        const int64_t end =
            c >= p.chunks ? first : first + quarter < p.n ? first + quarter : (int64_t)p.n;
        // (the first choices are on their way while the counts are added)
        Choices<BATCH> ids;
        ids.load(p, first + lane, 64);
        __syncthreads();
        // (assignments of earlier chunks go into next[0], those of the chunk's earlier
        // wavefronts below)
        const int all = p.chunks * p.groups;
        for (int i0 = t; i0 < all; i0 += 256 * kBatch) {
            int v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = i0 + 256 * i;   // (past the last: that one again)
                v[i] = p.chunk_counts[at < all ? at : all - 1];
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int at = i0 + 256 * i, of = (int)((uint32_t)at / (uint32_t)p.groups);
                const int e = at - of * p.groups;
                if (at >= all || v[i] == 0) continue;
                atomicAdd(&total[e], v[i]);
                if (of < c) atomicAdd(&next[0][e], v[i]);
            }
        }
        if (wave < 3)
            for (int64_t base = first; base < end; base += 64 * BATCH) {
                Choices<BATCH> own = ids;
                if (base != first) own.load(p, base + lane, 64);
#pragma unroll
                for (int j = 0; j < BATCH; ++j) {
                    const int e = own.expert(j, p.groups);
                    if (base + 64 * j + lane < end && e >= 0) atomicAdd(&next[wave + 1][e], 1);
                }
            }
        __syncthreads();
        for (int e = t; e < p.groups; e += 256)
            for (int w = 1; w < 4; ++w) next[w][e] += next[w - 1][e];
        segment_starts(total, p.groups, start, wave_sums);
        write_group_data(p, total, start, c, p.rank_units);
        for (int64_t base = first; base < end; base += 64 * BATCH) {
            if (base != first) ids.load(p, base + lane, 64);
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int64_t i = base + 64 * j + lane;
                if (base + 64 * j >= end) break;
                const int e = i < end ? ids.expert(j, p.groups) : -1;
                const uint64_t same = same_expert(e, p.groups);
                const uint64_t below = same & ((1ull << lane) - 1ull);
                const int rank = e < 0 ? 0 : next[wave][e] + __popcll(below);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (e >= 0 && below == 0) next[wave][e] += __popcll(same);
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                if (i < end) {
                    const int row = row_of(p, start, e, rank);
                    p.positions[i] = row;
                    if (row >= 0 && p.kb) p.source[row] = (int)(i / p.topk);
                }
            }
        }
        __syncthreads();
    }
}

// A wavefront copies 1 KB of a token's row to the rows of its assignments (2 KB: 4% slower, 4 KB 6%).  The load
// does not wait for the positions, so tokens without a row here are read too: 16384 tokens of one choice among 64
// experts, eight of them here, take 35 us, of eight experts 51.
__device__ __forceinline__ void copy_row(const DispatchParams& p, int token, int at,
                                         const int32_t* rows) {
    if (at >= p.vectors) return;
    const u32x4 v = __builtin_nontemporal_load((const u32x4*)p.x + (int64_t)token * p.vectors + at);
    for (int j = 0; j < p.topk; ++j)
        if (rows[j] >= 0) put16((u32x4*)p.a + (int64_t)rows[j] * p.vectors + at, v, p.far);
}

// Scales lie column-group-major, so they go by rows: a wavefront 64 neighbouring rows of the
// output, whose scales it writes in runs of 256 bytes, reading where the rows' tokens are.
__device__ __forceinline__ void copy_scales(const DispatchParams& p, uint32_t block, int lane) {
    const uint32_t blocks = (uint32_t)((p.m + 63) / 64);
    const int slot = (int)(block / blocks);
    const int r = (int)(block - slot * blocks) * 64 + lane;
    if (r >= p.m) return;
    const bool held = p.masked ? r < p.group_data[slot] : p.group_data[r] >= 0;
    if (!held) return;
    const int token = p.source[(int64_t)slot * p.m + r];
    float* to = p.sfa + (int64_t)slot * p.kb * p.sfa_ld + r;
    for (int c0 = 0; c0 < p.kb; c0 += kBatch) {
        float v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {     // (past the last: that one again)
            const int c = c0 + i < p.kb ? c0 + i : p.kb - 1;
            v[i] = p.sfx[(int64_t)c * p.sfx_ld + token];
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (c0 + i < p.kb) to[(int64_t)(c0 + i) * p.sfa_ld] = v[i];
    }
}

// Scales first, as their units are the longer ones (last: 13% slower).  16384 tokens of two choices,
// e4m3 rows of 7168: 62 us (364 MB: 5.9 TB/s); a row is read once, its copies written past the caches.
__global__ void __launch_bounds__(256) dispatch_rows_kernel(DispatchParams p, int pieces,
                                                            uint32_t scale_units) {
    const int lane = threadIdx.x & 63;
    // (uniform over the wavefront)
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    for (uint32_t unit = wave; unit < p.units; unit += gridDim.x * 4) {
        if (unit < scale_units) {
            copy_scales(p, unit, lane);
            continue;
        }
        const uint32_t u = unit - scale_units;
        const int token = (int)(u / pieces), piece = (int)(u - (uint32_t)token * pieces);
        copy_row(p, token, piece * 64 + lane, p.positions + (int64_t)token * p.topk);
    }
}

// ---- few assignments: one launch ---------------------------------------------------

constexpr int kFewAssignments = 4096;
// Up to so many assignments: the time grows with their square (every workgroup goes through them),
// that of the three launches with the groups.  e4m3 rows of 2048 and 7168, eight choices: 8 groups, 2048
// assignments 8.3 and 10.2 us against 9.7 and 13.1, 4096 12.3 and 14.5 against 10.6 and 15.4; 256 groups,
// 4096 assignments 12.9 and 14.7 against 14.9 and 20.1.
constexpr int few_assignments(int groups) { return groups < 64 ? 2048 : kFewAssignments; }

// Workgroup = one token at a time.  Each ranks its own choices by going through all earlier ones, 512
// at a time; the token's row and scales are on their way meanwhile.  64 tokens, eight choices each,
// e4m3 rows of 7168 into slots: 4.7 us replayed in a graph; a load of each kind after the other took
// 5.8.  Three sizes of the choices' registers: 8 choices take 4.4 us with two a thread, 4.6 with eight.  The
// workgroups share grouped_layout's rows behind their tokens: far more rows than choices cost a single token 10 us
// of 1024, 28 of 16384, 157 of 131072 (64 tokens 12).
template <int MOST>
__global__ void __launch_bounds__(256) dispatch_few_kernel(DispatchParams p) {
    constexpr int kIds = MOST / 256;               // of a thread
    __shared__ __attribute__((aligned(16))) int16_t ids[MOST];
    __shared__ int total[kMostGroups], start[kMostGroups + 1], wave_sums[4];
    __shared__ int32_t rows[kMostTopk];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    // (slots start at their number: the counts are outputs alone, of workgroup 0)
    const bool count = !p.masked || blockIdx.x == 0;
    // (all loads issued before any is looked at, the choices' first)
    Choices<kIds> choices;
    if (p.n > 0) choices.load(p, t, 256);
    u32x4 v[4];
    float scale = 0.0f;
    const auto fetch = [&](int token) {
        const u32x4* from = (const u32x4*)p.x + (int64_t)token * p.vectors;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = t + 256 * i;
            v[i] = __builtin_nontemporal_load(from + (at < p.vectors ? +at : p.vectors - 1));
        }
        if (t < p.kb) scale = p.sfx[(int64_t)t * p.sfx_ld + token];
    };
    int token = blockIdx.x;
    if (token < p.tokens) fetch(token);
    if (count) {
        for (int e = t; e < p.groups; e += 256) total[e] = 0;
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
        if (t + 256 * i >= p.n) continue;
        const int e = choices.expert(i, p.groups);
        ids[t + 256 * i] = (int16_t)e;
        if (count && e >= 0) atomicAdd(&total[e], 1);
    }
    __syncthreads();
    if (!p.masked) segment_starts(total, p.groups, start, wave_sums);
    while (token < p.tokens) {
        for (int j = wave; j < p.topk; j += 4) {
            const int i = token * p.topk + j, e = ids[i];
            int rank = 0;
            for (int base = 0; base < i; base += 512) {
                const u32x4 w = *(const u32x4*)&ids[base + 8 * lane];
                const int before = i - base - 8 * lane;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int other = (int16_t)(w[k / 2] >> (k % 2 * 16));
                    rank += __popcll(__ballot(k < before && other == e));
                }
            }
            const int row = row_of(p, start, e, rank);
            if (lane == 0) {
                rows[j] = row;
                p.positions[i] = row;
            }
        }
        __syncthreads();
        const u32x4* from = (const u32x4*)p.x + (int64_t)token * p.vectors;
        for (int j = 0; j < p.topk; ++j) {
            const int row = rows[j];
            if (row < 0) continue;
            u32x4* to = (u32x4*)p.a + (int64_t)row * p.vectors;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + 256 * i < p.vectors) put16(to + t + 256 * i, v[i], p.far);
            for (int at = t + 1024; at < p.vectors; at += 256) put16(to + at, from[at], p.far);
            const int slot = p.masked ? row / p.m : 0;
            float* sf = p.sfa + (int64_t)slot * p.kb * p.sfa_ld + row - slot * p.m;
            if (t < p.kb) sf[(int64_t)t * p.sfa_ld] = scale;
            for (int c = t + 256; c < p.kb; c += 256)
                sf[(int64_t)c * p.sfa_ld] = p.sfx[(int64_t)c * p.sfx_ld + token];
        }
        token += gridDim.x;
        if (token >= p.tokens) break;
        fetch(token);
        __syncthreads();
    }
    if (count) write_group_data(p, total, start, blockIdx.x, gridDim.x);
}

// ---- the way back ------------------------------------------------------------------

struct CombineParams {
    const uint16_t* d;
    const int32_t* positions;
    const float* weights;       // nullptr: ones
    void* y;
    int64_t rows;
    int tokens, topk, k, pieces, far;
    uint32_t units;
};

// A wavefront: 512 columns of a token, four choices' rows on their way at a time.  16384 tokens of two
// choices, 7168 columns: 117 us (705 MB: 6 TB/s, HBM); 64 tokens of eight choices 3.8.
template <bool YB, bool FAR>
__global__ void __launch_bounds__(256) combine_kernel(CombineParams p) {
    const int lane = threadIdx.x & 63;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
    for (uint32_t unit = wave; unit < p.units; unit += gridDim.x * 4) {
        const int token = (int)(unit / p.pieces);
        const int col = (int)(unit - (uint32_t)token * p.pieces) * 512 + lane * 8;
        if (col >= p.k) continue;
        const int32_t* at = p.positions + (int64_t)token * p.topk;
        const float* w = p.weights ? p.weights + (int64_t)token * p.topk : nullptr;
        float y[8] = {};
        for (int j0 = 0; j0 < p.topk; j0 += 4) {
            Eight<true> v[4];
            float f[4];
            bool in[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int row = j0 + j < p.topk ? at[j0 + j] : -1;
                in[j] = row >= 0 && row < p.rows;
                f[j] = in[j] && w ? w[j0 + j] : 1.0f;
                if (in[j]) v[j].take<FAR>(p.d, (int64_t)row * p.k + col);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (in[j])
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] += f[j] * v[j][e];
        }
        put_values(p.y, YB, (int64_t)token * p.k + col, y, p.far);
    }
}

struct CombineBackwardParams {
    const void* dy;
    const uint16_t* d;
    const int32_t* positions;
    const float* weights;
    uint16_t* dd;
    uint8_t* q;
    float* sfa;
    float* dw;
    int64_t rows;
    int m, ld, tokens, topk, k, far;
    uint32_t units;
};

// Workgroup = two choices of a token; a lane eight columns of each 2048, 16 lanes a group of 128.  A
// group's largest |w dy| is |w| times that of |dy| (rounding keeps the order).  Workgroups go round
// the 8 XCDs: eight tokens' first pairs are followed by their second ones, so that a token's pairs
// find its dy in one L2.  16384 tokens of two choices, 7168 columns: 166 us (947 MB: 5.7 TB/s; reads
// alone run at 6.9); 512 threads take the same.  Tokens without a row here are read too: one choice among 64 experts,
// eight of them here, 70 us, of eight experts 110.
template <bool GB, bool FAR>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineBackwardParams p) {
    __shared__ float dots[2][2][4];
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    int turn = 0;
    const uint32_t pairs = (uint32_t)(p.topk + 1) / 2;
    for (uint32_t unit = blockIdx.x; unit < p.units; unit += gridDim.x) {
        const int token = (int)(unit / (8 * pairs) * 8 + unit % 8);
        const int j0 = (int)(unit / 8 % pairs) * 2;
        if (token >= p.tokens) continue;
        const int32_t* at = p.positions + (int64_t)token * p.topk;
        const float* w = p.weights ? p.weights + (int64_t)token * p.topk : nullptr;
        int row[2];
        bool in[2];
        const uint16_t* from[2];
        float f[2], dot[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            row[j] = j0 + j < p.topk ? at[j0 + j] : -1;
            in[j] = row[j] >= 0 && row[j] < p.rows;
            f[j] = in[j] && w ? w[j0 + j] : 1.0f;
            // (a choice without a row reads dy in its place)
            from[j] = in[j] ? p.d + (int64_t)row[j] * p.k
                            : (const uint16_t*)p.dy + (int64_t)token * p.k;
        }
        for (int col = t * 8; col < p.k; col += 2048) {
            Eight<GB> g;
            Eight<true> d[2];
            // (past the caches only where no other pair reads it: eight choices 244 us, so 228)
            if (FAR && pairs == 1) {
                asm volatile("");
                g.stream(p.dy, (int64_t)token * p.k + col);
                asm volatile("");
            } else {
                g.load(p.dy, (int64_t)token * p.k + col);
            }
            if (p.dw)
#pragma unroll
                for (int j = 0; j < 2; ++j) d[j].take<FAR>(from[j], col);
            float dy[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] = g[e];
            const float top = p.q ? max16(max8(dy)) : 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (!in[j]) continue;
                if (p.dw)
#pragma unroll
                    for (int e = 0; e < 8; ++e) dot[j] += dy[e] * d[j][e];
                float dd[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) dd[e] = f[j] * dy[e];
                const int64_t to = (int64_t)row[j] * p.k + col;
                if (p.dd) put_values(p.dd, true, to, dd, p.far);
                if (p.q) {
                    float inv;             // (a NaN product is no maximum)
                    const float sc =
                        block_scale(__builtin_fmaxf(__builtin_fabsf(f[j]) * top, 0.0f), inv);
                    put_codes(p.q + to, codes8(dd, inv), p.far);
                    if ((lane & 15) == 0) {
                        const int slot = row[j] / p.m;
                        p.sfa[((int64_t)slot * (p.k >> 7) + (col >> 7)) * p.ld + row[j] -
                              slot * p.m] = sc;
                    }
                }
            }
        }
        if (p.dw) {                        // (two buffers: one barrier a unit)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float sum = sum_wave(dot[j]);
                if (lane == 0) dots[turn][j][wave] = sum;
            }
            __syncthreads();
            if (t < 2 && j0 + t < p.topk)
                p.dw[(int64_t)token * p.topk + j0 + t] =
                    (dots[turn][t][0] + dots[turn][t][1]) + (dots[turn][t][2] + dots[turn][t][3]);
            turn ^= 1;
        }
    }
}

// ---- launches -----------------------------------------------------------------

bool counts_fit(int64_t tokens, int topk, int num_groups) {
    return tokens >= 0 && topk >= 1 && topk <= kMostTopk && num_groups >= 1 &&
           num_groups <= kMostGroups && tokens <= kMostAssignments / topk;
}
int64_t capacity_of(int64_t n, int num_groups) {
    return (n + 127 * (n < num_groups ? n : (int64_t)num_groups)) / 128 * 128;
}
// Assignments of a chunk, a multiple of 256.  A workgroup of the ranks' launch goes through all
// chunks' counts and its own chunk's choices, eight loads on their way in both: about as many steps
// of the one as of the other (1024 experts, 8192 choices in 8 chunks 20 us, 131072 in 32 51, in 8 84).
int chunk_of(int64_t n, int num_groups) {
    int64_t chunks = (int64_t)__builtin_sqrt(8.0 * (double)n / num_groups);
    chunks = chunks < 1 ? 1 : chunks < kMostChunks ? chunks : kMostChunks;
    return (int)(((n + chunks - 1) / chunks + 255) / 256 * 256);
}
bool few(int64_t n, int groups) { return n <= few_assignments(groups); }

}  // namespace
}  // namespace layer
}  // namespace fp8bs

extern "C" int64_t fp8bs_moe_capacity(int64_t tokens, int topk, int num_groups) {
    using namespace fp8bs::layer;
    if (!counts_fit(tokens, topk, num_groups)) return -FP8BS_ERR_SHAPE;
    return capacity_of(tokens * topk, num_groups);
}

extern "C" int64_t fp8bs_moe_dispatch_workspace_size(int layout, int64_t tokens, int topk,
                                                     int num_groups, int64_t m) {
    using namespace fp8bs::layer;
    if (layout != FP8BS_LAYOUT_CONTIGUOUS && layout != FP8BS_LAYOUT_MASKED)
        return -FP8BS_ERR_UNSUPPORTED;
    if (!counts_fit(tokens, topk, num_groups) || m < 0 || m > kMaxRows) return -FP8BS_ERR_SHAPE;
    const int64_t n = tokens * topk;
    if (few(n, num_groups)) return 0;
    const int64_t rows = layout == FP8BS_LAYOUT_MASKED ? m * num_groups : m;
    return (int64_t)kMostChunks * num_groups * 4 + (rows + 3) / 4 * 16;
}

extern "C" int fp8bs_moe_dispatch(int layout, const void* ids, int id_bytes, const void* x,
                                  int x_dtype, const float* sfx, void* a, float* sfa,
                                  int32_t* group_data, int32_t* positions, int32_t* counts,
                                  int tokens, int topk, int num_groups, int m, int k,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
    using namespace fp8bs::layer;
    const int64_t need = fp8bs_moe_dispatch_workspace_size(layout, tokens, topk, num_groups, m);
    if (need < 0) return (int)-need;
    const bool masked = layout == FP8BS_LAYOUT_MASKED, e4m3 = x_dtype == FP8BS_DTYPE_E4M3;
    if (!e4m3 && !value_type(x_dtype)) return FP8BS_ERR_UNSUPPORTED;
    if (id_bytes != 4 && id_bytes != 8) return FP8BS_ERR_UNSUPPORTED;
    if (k < 8 || k > kMaxK || k % (e4m3 ? 128 : 8) != 0) return FP8BS_ERR_SHAPE;
    const int64_t n = (int64_t)tokens * topk;
    if (masked ? (int64_t)m * num_groups > kMaxRows
               : m % 128 != 0 || m < capacity_of(n, num_groups))
        return FP8BS_ERR_SHAPE;
    const int64_t rows = masked ? (int64_t)m * num_groups : m;
    if (!aligned(counts, 4) || ((masked || m > 0) && !aligned(group_data, 4)))
        return FP8BS_ERR_POINTER;
    // (tokens' rows and scales are fetched before it is known whether their choices have a row)
    if (n > 0 && (!aligned(ids, (uintptr_t)id_bytes) || !aligned(positions, 4) || !aligned(x) ||
                  (e4m3 && !aligned(sfx))))
        return FP8BS_ERR_POINTER;
    if (n > 0 && rows > 0 && (!aligned(a) || (e4m3 && !aligned(sfa)))) return FP8BS_ERR_POINTER;
    if (need > 0 && !aligned(workspace)) return FP8BS_ERR_POINTER;
    if (workspace_bytes < (size_t)need) return FP8BS_ERR_UNSUPPORTED;
    DispatchParams p = {};
    p.ids = ids;
    p.x = (const uint8_t*)x;
    p.sfx = sfx;
    p.a = (uint8_t*)a;
    p.sfa = sfa;
    p.group_data = group_data;
    p.positions = positions;
    p.counts = counts;
    p.ids64 = id_bytes == 8;
    p.masked = masked;
    p.n = (int)n;
    p.topk = topk;
    p.tokens = tokens;
    p.groups = num_groups;
    p.m = m;
    p.vectors = k / (e4m3 ? 16 : x_dtype == FP8BS_DTYPE_BF16 ? 8 : 4);
    p.kb = e4m3 ? k / 128 : 0;
    p.sfx_ld = (int)fp8bs_get_sfa_ld(tokens);
    p.sfa_ld = (int)fp8bs_get_sfa_ld(m);
    p.far = far_outputs((double)n * p.vectors * 16);
    if (few(n, num_groups)) {
        // (without tokens: the group data alone)
        const int64_t units = tokens > 0 ? tokens : m / 1024 + 1;
        return launch(n <= 512    ? (const void*)dispatch_few_kernel<512>
                      : n <= 2048 ? (const void*)dispatch_few_kernel<2048>
                                  : (const void*)dispatch_few_kernel<kFewAssignments>,
                      workgroups(units, 4), 256, p, stream);
    }
    p.chunk_counts = (int32_t*)workspace;
    p.source = p.chunk_counts + (int64_t)kMostChunks * num_groups;
    p.chunk = chunk_of(n, num_groups);
    p.chunks = (int)((n + p.chunk - 1) / p.chunk);
    p.rank_units = p.chunks;
    if (!masked && m / 512 > p.chunks) p.rank_units = m / 512 < 256 ? m / 512 : 256;
    if (p.rank_units < p.chunks) p.rank_units = p.chunks;
    const int pieces = (p.vectors + 63) / 64;
    const int64_t scale_units = e4m3 ? (int64_t)((m + 63) / 64) * (masked ? num_groups : 1) : 0;
    const int64_t units = scale_units + (int64_t)tokens * pieces;
    if (units > 0x7fffffff) return FP8BS_ERR_UNSUPPORTED;
    p.units = (uint32_t)units;
    const bool one = p.chunk == 256;
    int st = launch(one ? (const void*)dispatch_count_kernel<1>
                        : (const void*)dispatch_count_kernel<kBatch>,
                    workgroups(p.chunks, 4), 256, p, stream);
    if (st != FP8BS_OK) return st;
    st = launch(one ? (const void*)dispatch_rank_kernel<1> : (const void*)dispatch_rank_kernel<kBatch>,
                workgroups(p.rank_units, 4), 256, p, stream);
    if (st != FP8BS_OK || rows == 0) return st;
    uint32_t su = (uint32_t)scale_units;
    int pc = pieces;
    void* args[] = {(void*)&p, (void*)&pc, (void*)&su};
    return hipLaunchKernel((const void*)dispatch_rows_kernel, dim3(workgroups((units + 3) / 4, 8)),
                           dim3(256), args, 0, stream) == hipSuccess ? FP8BS_OK : FP8BS_ERR_HIP;
}

extern "C" int fp8bs_moe_combine(const void* d, const int32_t* positions, const float* weights,
                                 void* y, int y_dtype, int64_t rows, int tokens, int topk, int k,
                                 hipStream_t stream) {
    using namespace fp8bs::layer;
    if (!counts_fit(tokens, topk, 1) || rows < 0 || rows > 0x7fffffff || k < 8 || k % 8 != 0 ||
        k > kMaxK)
        return FP8BS_ERR_SHAPE;
    if (!value_type(y_dtype)) return FP8BS_ERR_UNSUPPORTED;
    if (tokens == 0) return FP8BS_OK;
    if ((rows > 0 ? !aligned(d) : false) || !aligned(positions, 4) || !aligned_or_null(weights, 4) ||
        !aligned(y))
        return FP8BS_ERR_POINTER;
    const bool bf16 = y_dtype == FP8BS_DTYPE_BF16;
    const int pieces = (k + 511) / 512;
    const int64_t units = (int64_t)tokens * pieces;
    if (units > 0x7fffffff) return FP8BS_ERR_UNSUPPORTED;
    CombineParams p = {(const uint16_t*)d, positions, weights, y, rows, tokens, topk, k, pieces,
                       far_outputs((double)tokens * k * (bf16 ? 2 : 4)), (uint32_t)units};
    const bool far = far_inputs((double)tokens * k * (topk * 2 + (bf16 ? 2 : 4)));
    return launch(bf16  ? far ? (const void*)combine_kernel<true, true>
                              : (const void*)combine_kernel<true, false>
                  : far ? (const void*)combine_kernel<false, true>
                        : (const void*)combine_kernel<false, false>,
                  workgroups((units + 3) / 4, 8), 256, p, stream);
}

extern "C" int fp8bs_moe_combine_backward(const void* dy, int dy_dtype, const void* d,
                                          const int32_t* positions, const float* weights, void* dd,
                                          void* q, float* sfa, float* dweights, int slots, int m,
                                          int tokens, int topk, int k, hipStream_t stream) {
    using namespace fp8bs::layer;
    if (!counts_fit(tokens, topk, 1) || slots < 1 || m < 0 || (int64_t)slots * m > kMaxRows ||
        k < 8 || k > kMaxK || k % (q ? 128 : 8) != 0)
        return FP8BS_ERR_SHAPE;
    if (!value_type(dy_dtype)) return FP8BS_ERR_UNSUPPORTED;
    if (tokens == 0) return FP8BS_OK;
    const int64_t rows = (int64_t)slots * m;
    if (!aligned(dy) || !aligned(positions, 4) || !aligned_or_null(weights, 4) ||
        !aligned_or_null(dd) || !aligned_or_null(q) || !aligned_or_null(dweights, 4) ||
        (rows > 0 && ((dweights && !aligned(d)) || (q && !aligned(sfa)))) || !(dd || q || dweights))
        return FP8BS_ERR_POINTER;
    const int64_t units = ((int64_t)tokens + 7) / 8 * 8 * ((topk + 1) / 2);
    if (units > 0x7fffffff) return FP8BS_ERR_UNSUPPORTED;
    CombineBackwardParams p = {dy, (const uint16_t*)d, positions, weights, (uint16_t*)dd,
                               (uint8_t*)q, sfa, dweights, rows, m > 0 ? m : 1,
                               (int)fp8bs_get_sfa_ld(m), tokens, topk, k,
                               far_outputs((double)tokens * topk * k * ((dd ? 2 : 0) + (q ? 1 : 0))),
                               (uint32_t)units};
    const bool bf16 = dy_dtype == FP8BS_DTYPE_BF16;
    const bool far = far_inputs(
        (double)tokens * k * ((bf16 ? 2 : 4) + topk * ((dd ? 2 : 0) + (q ? 1 : 0) + (dweights ? 2 : 0))));
    return launch(bf16  ? far ? (const void*)combine_backward_kernel<true, true>
                              : (const void*)combine_backward_kernel<true, false>
                  : far ? (const void*)combine_backward_kernel<false, true>
                        : (const void*)combine_backward_kernel<false, false>,
                  workgroups(units, 8), 256, p, stream);
}

// fp8bs_mx_api.cpp -- C entry points of the MXFP4 products and of the gated feed-forward
// block (declared in include/fp8bs.h): checks of sizes and pointers, the kernels' parameters
// and the launches.  No allocation, no synchronisation, no host read of device data.
#include <hip/hip_runtime.h>
#include <string.h>

#include <atomic>

#include "fp8bs_mx.h"

namespace {

using namespace fp8bs::mx;

constexpr int kMaxDevices = 64;
std::atomic<int> g_cus[kMaxDevices];           // 0: not asked yet

// Compute units of the current device (0 on error), and those under the process's cap.
struct Cus {
    int device, capped;
};
Cus compute_units() {
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return {0, 0};
    int cus = dev >= 0 && dev < kMaxDevices ? g_cus[dev].load(std::memory_order_relaxed) : 0;
    if (cus == 0) {
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            return {0, 0};
        if (dev >= 0 && dev < kMaxDevices) g_cus[dev].store(cus, std::memory_order_relaxed);
    }
    const int cap = fp8bs_get_num_cus();
    return {cus, cap > 0 && cap < cus ? cap : cus};
}

bool aligned(const void* p, uintptr_t to) { return p && ((uintptr_t)p & (to - 1)) == 0; }

// Sizes of one call: rows (dense M, contiguous m_total, masked max_m), columns of the
// weight (product n, gated 2f), k, groups.
int check_sizes(int layout, int64_t m, int64_t cols, int k, int groups) {
    if (k < 128 || k % 128 != 0 || m < 0 || cols < 1 || groups < 1) return FP8BS_ERR_SHAPE;
    if (layout == kContiguous && m % 128 != 0) return FP8BS_ERR_SHAPE;
    if (k > kMaxK || m > kMaxRows || cols > kMaxRows) return FP8BS_ERR_SHAPE;
    const double words = k / 128.0;                // an operand's exponents: 32-bit byte offsets
    if ((m + 3) * words * 4 >= 4294967296.0 || (cols + 3) * words * 4 >= 4294967296.0)
        return FP8BS_ERR_SHAPE;
    return FP8BS_OK;
}

// Whether the 128x128 tiles of m x n in each of `slots` have 32-bit numbers: asked before a call
// that launches several kernels launches the first.
bool tiles_fit(int64_t m, int64_t n, int64_t slots) {
    return (double)((m + 127) / 128) * ((n + 127) / 128) * slots <= 0x7fffffff;
}

// The parameters that every call shares.
MxParams base_params(const void* a, const int32_t* sfa, const void* b, const int32_t* sfb,
                     const int32_t* group_data, int m, int64_t cols, int k, int groups) {
    MxParams p;
    memset(&p, 0, sizeof p);
    p.a = (const uint8_t*)a;
    p.b = (const uint8_t*)b;
    p.sfa = sfa;
    p.sfb = sfb;
    p.group_data = group_data;
    p.a_row = p.b_row = k / 2;
    p.m = m;
    p.kwords = k / 128;
    p.chunks = (k + 255) / 256;
    p.sfa_ld = (int)fp8bs_get_sfa_ld(m);
    p.sfb_ld = (int)fp8bs_get_sfa_ld(cols);
    p.num_groups = groups;
    return p;
}

bool pointers_ok(const void* a, const void* sfa, const void* b, const void* sfb, int layout,
                 const int32_t* group_data) {
    return aligned(a, 16) && aligned(sfa, 16) && aligned(b, 16) && aligned(sfb, 16) &&
           (layout == kDense || aligned(group_data, 4));
}

int status(int hip) {
    return hip == (int)hipSuccess ? FP8BS_OK
           : hip == (int)hipErrorInvalidValue ? FP8BS_ERR_UNSUPPORTED : FP8BS_ERR_HIP;
}

int product(int layout, const void* a, const int32_t* sfa, const void* b, const int32_t* sfb,
            void* d, const int32_t* group_data, int m, int expected_m, int n, int k, int groups,
            hipStream_t stream) {
    const int st = check_sizes(layout, m, n, k, groups);
    if (st != FP8BS_OK || m == 0) return st;
    if (!pointers_ok(a, sfa, b, sfb, layout, group_data) || !aligned(d, 16))
        return FP8BS_ERR_POINTER;
    if (!tiles_fit(m, n, layout == kMasked ? groups : 1)) return FP8BS_ERR_UNSUPPORTED;
    const Cus cus = compute_units();
    if (cus.capped <= 0) return FP8BS_ERR_HIP;
    MxParams p = base_params(a, sfa, b, sfb, group_data, m, n, k, groups);
    p.d = d;
    p.d_ld = n;
    p.n = n;
    const int rows = layout == kMasked && expected_m > 0 && expected_m < m ? expected_m : m;
    return status(launch_gemm(layout, kStore, p, groups, rows, cus.capped,
                              cus.device, stream));
}

int gated_forward(int layout, const void* a, const int32_t* sfa, const void* b,
                  const int32_t* sfb, void* h, int32_t* sfh, bool quantise,
                  const int32_t* group_data, int m, int expected_m, int f, int k, int groups,
                  int activation, hipStream_t stream) {
    if (f < 1 || f % (quantise ? 128 : 32) != 0) return FP8BS_ERR_SHAPE;
    const int st = check_sizes(layout, m, 2 * (int64_t)f, k, groups);
    if (st != FP8BS_OK) return st;
    if (activation != FP8BS_ACT_SILU && activation != FP8BS_ACT_GELU_TANH)
        return FP8BS_ERR_UNSUPPORTED;
    if (m == 0) return FP8BS_OK;
    if (!pointers_ok(a, sfa, b, sfb, layout, group_data) || !aligned(h, 16) ||
        (quantise && !aligned(sfh, 16)))
        return FP8BS_ERR_POINTER;
    if (!tiles_fit(m, 2 * (int64_t)f, layout == kMasked ? groups : 1)) return FP8BS_ERR_UNSUPPORTED;
    const Cus cus = compute_units();
    if (cus.capped <= 0) return FP8BS_ERR_HIP;
    MxParams p = base_params(a, sfa, b, sfb, group_data, m, 2 * (int64_t)f, k, groups);
    p.d = h;
    p.d2 = sfh;
    p.d_ld = quantise ? f / 2 : f;
    p.d2_ld = quantise ? p.sfa_ld : 0;
    p.n = f;
    p.act = activation;
    const int rows = layout == kMasked && expected_m > 0 && expected_m < m ? expected_m : m;
    return status(launch_gemm(layout, quantise ? kGatedQuant : kGated, p, groups, rows,
                              cus.capped, cus.device, stream));
}

// The backward pass's two products, sizes only: da over W's rows, db over the tokens.
void gradient_sizes(MxParams& a, MxParams& b, int layout, int64_t m, int f, int k, int groups) {
    a.m = (int)m;
    a.depth = 2 * f;
    a.chunks = f / 32;
    b.m = 2 * f;
    b.depth = (int)m;
    b.chunks = (int)((m + 63) / 64);
    a.n = b.n = k;
    a.splits = grad_splits(layout, a, groups);
    b.splits = grad_splits(layout == kContiguous ? kBlocks : kDense, b, groups);
}

// Workspace of the backward pass: dg | du, [rows up to a multiple of 64][2f]; for db of the
// contiguous layout the blocks by expert; the parts of split products.  Each starts at a multiple
// of 256 bytes.
struct Parts {
    int64_t order, part_a, part_b, total;
};
Parts parts(int layout, int64_t m, int f, int k, int groups, bool want_da, bool want_db) {
    auto whole = [](int64_t bytes) { return (bytes + 255) / 256 * 256; };
    Parts w;
    w.order = whole((m + 63) / 64 * 64 * 2 * f * 2);
    // (four entries to spare: the copies look up to two steps past the last block)
    w.total = w.order + (want_db && layout == kContiguous ? (groups + 1 + m / 128 + 4) * 4 : 0);
    MxParams a, b;
    memset(&a, 0, sizeof a);
    memset(&b, 0, sizeof b);
    gradient_sizes(a, b, layout, m, f, k, groups);
    w.part_a = w.part_b = whole(w.total);
    if (want_da && a.splits > 1) w.total = w.part_b = w.part_a + whole(a.splits * m * k * 4);
    if (want_db && b.splits > 1)
        w.total = w.part_b + b.splits * (int64_t)(layout == kContiguous ? groups : 1) * 2 * f * k * 4;
    return w;
}

int check_backward(int layout, int64_t m, int f, int k, int groups) {
    if (layout != kDense && layout != kContiguous) return FP8BS_ERR_SHAPE;
    if (f < 1 || f % 32 != 0) return FP8BS_ERR_SHAPE;
    const int st = check_sizes(layout, m, 2 * (int64_t)f, k, groups);
    if (st != FP8BS_OK) return st;
    // 256 rows of dg | du within 32-bit copy offsets
    if (f > (1 << 21)) return FP8BS_ERR_SHAPE;
    return FP8BS_OK;
}

int gated_backward(int layout, const void* a, const int32_t* sfa, const void* b,
                   const int32_t* sfb, const void* dh, void* da, void* db, int db_dtype,
                   int accumulate, const int32_t* group_data, int m, int f, int k, int groups,
                   int activation, void* workspace, size_t workspace_bytes, hipStream_t stream) {
    int st = check_backward(layout, m, f, k, groups);
    if (st != FP8BS_OK) return st;
    if (activation != FP8BS_ACT_SILU && activation != FP8BS_ACT_GELU_TANH)
        return FP8BS_ERR_UNSUPPORTED;
    const bool f32 = db_dtype == FP8BS_DTYPE_F32;
    if (!f32 && db_dtype != FP8BS_DTYPE_BF16) return FP8BS_ERR_UNSUPPORTED;
    if (accumulate && !f32) return FP8BS_ERR_UNSUPPORTED;
    if (!da && !db) return FP8BS_OK;
    if ((da && !aligned(da, 16)) || (db && !aligned(db, 16))) return FP8BS_ERR_POINTER;
    if (m > 0 && (!pointers_ok(a, sfa, b, sfb, layout, group_data) || !aligned(dh, 16)))
        return FP8BS_ERR_POINTER;
    if (m == 0 && (!db || accumulate)) return FP8BS_OK;
    const Parts w = parts(layout, m, f, k, groups, da != nullptr, db != nullptr);
    if (w.total > 0 && workspace_bytes < (size_t)w.total) return FP8BS_ERR_UNSUPPORTED;
    if (w.total > 0 && !aligned(workspace, 16)) return FP8BS_ERR_POINTER;
    if (!tiles_fit(m, 2 * (int64_t)f, 1) || (da && !tiles_fit(m, k, 1)) ||
        (db && !tiles_fit(2 * (int64_t)f, k, layout == kContiguous ? groups : 1)))
        return FP8BS_ERR_UNSUPPORTED;
    const Cus cus = compute_units();
    if (cus.capped <= 0) return FP8BS_ERR_HIP;
    uint8_t* grad = (uint8_t*)workspace;
    int32_t* order = (int32_t*)(grad + w.order);

    MxParams p = base_params(a, sfa, b, sfb, group_data, m, 2 * (int64_t)f, k, groups);
    if (m > 0) {
        p.n = f;
        p.act = activation;
        p.dh = (const uint16_t*)dh;
        p.d = grad;
        p.d_ld = 2 * (int64_t)f;
        st = status(launch_gemm(layout, kGatedGrad, p, groups, m, cus.capped, cus.device,
                                stream));
        if (st != FP8BS_OK) return st;
    }
    // both products: bf16 dg | du, 4-bit second operand with k columns
    p.a = grad;
    p.a_row = 4 * (int64_t)f;
    p.d_ld = k;
    MxParams xa = p, xb = p;
    gradient_sizes(xa, xb, layout, m, f, k, groups);
    xa.d = da;
    xa.part = (float*)(grad + w.part_a);
    xb.b = (const uint8_t*)a;
    xb.sfb = sfa;
    xb.sfb_ld = p.sfa_ld;
    xb.blocks = order;
    xb.d = db;
    xb.part = (float*)(grad + w.part_b);
    xb.accumulate = accumulate;
    const int layout_b = layout == kContiguous ? kBlocks : kDense, epilogue_b = f32 ? kStoreF32 : kStore;
    const bool want_da = da && m > 0;
    if (db && layout == kContiguous) {
        st = status(launch_block_order(group_data, m / 128, groups, order, stream));
        if (st != FP8BS_OK) return st;
    }
    if (want_da && db && grad_pair_pays(layout, xa, xb, groups, cus.capped))
        return status(launch_grad_pair(layout, epilogue_b, &xa, &xb, groups, stream));
    if (want_da)
        st = status(xa.splits > 1 ? launch_grad_pair(layout, kStore, &xa, nullptr, groups, stream)
                                  : launch_grad(layout, false, kStore, xa, groups, cus.capped, stream));
    if (st == FP8BS_OK && db)
        st = status(xb.splits > 1 ? launch_grad_pair(layout, epilogue_b, nullptr, &xb, groups, stream)
                                  : launch_grad(layout_b, true, epilogue_b, xb, groups, cus.capped, stream));
    return st;
}

// Workspace of the feed-forward layer: x's codes and exponents, h's.
struct LayerParts {
    int64_t q, sf, hq, sfh, total;
};
LayerParts layer_parts(int64_t slots, int64_t m, int f, int k) {
    LayerParts w;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    const int64_t ld = fp8bs_get_sfa_ld(m);
    w.q = take(slots * m * (k / 2));
    w.sf = take(slots * (k / 128) * ld * 4);
    w.hq = take(slots * m * (f / 2));
    w.sfh = take(slots * (f / 128) * ld * 4);
    w.total = at;
    return w;
}

int check_layer(int layout, int64_t m, int f, int k, int groups) {
    if (layout != kDense && layout != kContiguous && layout != kMasked) return FP8BS_ERR_SHAPE;
    if (f < 128 || f % 128 != 0) return FP8BS_ERR_SHAPE;
    const int st = check_sizes(layout, m, 2 * (int64_t)f, k, groups);
    // (as for the quantiser: sizes in bytes stay within 64 bits)
    if ((layout == kMasked ? groups : 1.0) * m * (k > f ? k : f) >= 9.0e15) return FP8BS_ERR_SHAPE;
    return st != FP8BS_OK ? st : check_sizes(layout, m, 1, f, groups);
}

int feed_forward(int layout, const void* x, int x_dtype, const void* b, const int32_t* sfb,
                 const void* b2, const int32_t* sfb2, void* d, const int32_t* group_data, int m,
                 int expected_m, int f, int k, int n, int groups, int activation, void* workspace,
                 size_t workspace_bytes, hipStream_t stream) {
    int st = check_layer(layout, m, f, k, groups);
    if (st == FP8BS_OK) st = check_sizes(layout, m, n, f, groups);
    if (st != FP8BS_OK) return st;
    if (x_dtype != FP8BS_DTYPE_F32 && x_dtype != FP8BS_DTYPE_BF16) return FP8BS_ERR_UNSUPPORTED;
    if (activation != FP8BS_ACT_SILU && activation != FP8BS_ACT_GELU_TANH)
        return FP8BS_ERR_UNSUPPORTED;
    if (m == 0) return FP8BS_OK;
    if (!pointers_ok(x, b, sfb, b2, layout, group_data) || !aligned(sfb2, 16) || !aligned(d, 16))
        return FP8BS_ERR_POINTER;
    const int64_t slots = layout == kMasked ? groups : 1;
    const LayerParts w = layer_parts(slots, m, f, k);
    if (workspace_bytes < (size_t)w.total) return FP8BS_ERR_UNSUPPORTED;
    if (!aligned(workspace, 16)) return FP8BS_ERR_POINTER;
    if (!tiles_fit(m, 2 * (int64_t)f, slots) || !tiles_fit(m, n, slots)) return FP8BS_ERR_UNSUPPORTED;
    uint8_t* ws = (uint8_t*)workspace;
    int32_t* sf = (int32_t*)(ws + w.sf);
    int32_t* sfh = (int32_t*)(ws + w.sfh);
    st = fp8bs_quantize_mxfp4(x, x_dtype, ws + w.q, sf, (int)slots, m, k, stream);
    if (st == FP8BS_OK)
        st = gated_forward(layout, ws + w.q, sf, b, sfb, ws + w.hq, sfh, true, group_data, m,
                           expected_m, f, k, groups, activation, stream);
    if (st == FP8BS_OK)
        st = product(layout, ws + w.hq, sfh, b2, sfb2, d, group_data, m, expected_m, n, f, groups,
                     stream);
    return st;
}

}  // namespace

extern "C" {

int64_t fp8bs_feed_forward_workspace_size(int layout, int64_t m, int f, int k, int num_groups) {
    const int groups = layout == kDense ? 1 : num_groups;
    const int st = check_layer(layout, m, f, k, groups);
    if (st != FP8BS_OK) return -(int64_t)st;
    return layer_parts(layout == kMasked ? groups : 1, m, f, k).total;
}

int fp8bs_feed_forward_mxfp4(int layout, const void* x, int x_dtype, const void* b,
                             const int32_t* sfb, const void* b2, const int32_t* sfb2, void* d,
                             const int32_t* group_data, int m, int expected_m, int f, int k,
                             int n, int num_groups, int activation, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    return feed_forward(layout, x, x_dtype, b, sfb, b2, sfb2, d, group_data, m, expected_m, f, k,
                        n, layout == kDense ? 1 : num_groups, activation, workspace,
                        workspace_bytes, stream);
}

int fp8bs_dense_nt_mxfp4(const void* a, const int32_t* sfa, const void* b, const int32_t* sfb,
                         void* d, int m, int n, int k, hipStream_t stream) {
    return product(kDense, a, sfa, b, sfb, d, nullptr, m, 0, n, k, 1, stream);
}

int fp8bs_grouped_contiguous_nt_mxfp4(const void* a, const int32_t* sfa, const void* b,
                                      const int32_t* sfb, void* d, const int32_t* grouped_layout,
                                      int m_total, int n, int k, int num_groups,
                                      hipStream_t stream) {
    return product(kContiguous, a, sfa, b, sfb, d, grouped_layout, m_total, 0, n, k, num_groups,
                   stream);
}

int fp8bs_grouped_masked_nt_mxfp4(const void* a, const int32_t* sfa, const void* b,
                                  const int32_t* sfb, void* d, const int32_t* masked_m,
                                  int num_groups, int max_m, int expected_m, int n, int k,
                                  hipStream_t stream) {
    return product(kMasked, a, sfa, b, sfb, d, masked_m, max_m, expected_m, n, k, num_groups,
                   stream);
}

int fp8bs_gated_dense_mxfp4(const void* a, const int32_t* sfa, const void* b, const int32_t* sfb,
                            void* h, int m, int f, int k, int activation, hipStream_t stream) {
    return gated_forward(kDense, a, sfa, b, sfb, h, nullptr, false, nullptr, m, 0, f, k, 1,
                         activation, stream);
}

int fp8bs_gated_contiguous_mxfp4(const void* a, const int32_t* sfa, const void* b,
                                 const int32_t* sfb, void* h, const int32_t* grouped_layout,
                                 int m_total, int f, int k, int num_groups, int activation,
                                 hipStream_t stream) {
    return gated_forward(kContiguous, a, sfa, b, sfb, h, nullptr, false, grouped_layout, m_total,
                         0, f, k, num_groups, activation, stream);
}

int fp8bs_gated_masked_mxfp4(const void* a, const int32_t* sfa, const void* b,
                             const int32_t* sfb, void* h, const int32_t* masked_m,
                             int num_groups, int max_m, int expected_m, int f, int k,
                             int activation, hipStream_t stream) {
    return gated_forward(kMasked, a, sfa, b, sfb, h, nullptr, false, masked_m, max_m, expected_m,
                         f, k, num_groups, activation, stream);
}

int fp8bs_gated_dense_mxfp4_q(const void* a, const int32_t* sfa, const void* b,
                              const int32_t* sfb, void* hq, int32_t* sfh, int m, int f, int k,
                              int activation, hipStream_t stream) {
    return gated_forward(kDense, a, sfa, b, sfb, hq, sfh, true, nullptr, m, 0, f, k, 1,
                         activation, stream);
}

int fp8bs_gated_contiguous_mxfp4_q(const void* a, const int32_t* sfa, const void* b,
                                   const int32_t* sfb, void* hq, int32_t* sfh,
                                   const int32_t* grouped_layout, int m_total, int f, int k,
                                   int num_groups, int activation, hipStream_t stream) {
    return gated_forward(kContiguous, a, sfa, b, sfb, hq, sfh, true, grouped_layout, m_total, 0,
                         f, k, num_groups, activation, stream);
}

int fp8bs_gated_masked_mxfp4_q(const void* a, const int32_t* sfa, const void* b,
                               const int32_t* sfb, void* hq, int32_t* sfh,
                               const int32_t* masked_m, int num_groups, int max_m,
                               int expected_m, int f, int k, int activation,
                               hipStream_t stream) {
    return gated_forward(kMasked, a, sfa, b, sfb, hq, sfh, true, masked_m, max_m, expected_m, f,
                         k, num_groups, activation, stream);
}

int64_t fp8bs_gated_backward_workspace_size(int layout, int64_t m, int f, int k, int num_groups,
                                            int want_da, int want_db) {
    const int st = check_backward(layout, m, f, k, layout == kDense ? 1 : num_groups);
    if (st != FP8BS_OK) return -(int64_t)st;
    if (!want_da && !want_db) return 0;
    return parts(layout, m, f, k, layout == kDense ? 1 : num_groups, want_da != 0, want_db != 0).total;
}

int fp8bs_gated_dense_mxfp4_backward(const void* a, const int32_t* sfa, const void* b,
                                     const int32_t* sfb, const void* dh, void* da, void* db,
                                     int db_dtype, int accumulate, int m, int f, int k,
                                     int activation, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream) {
    return gated_backward(kDense, a, sfa, b, sfb, dh, da, db, db_dtype, accumulate, nullptr, m, f,
                          k, 1, activation, workspace, workspace_bytes, stream);
}

int fp8bs_gated_contiguous_mxfp4_backward(const void* a, const int32_t* sfa, const void* b,
                                          const int32_t* sfb, const void* dh, void* da, void* db,
                                          int db_dtype, int accumulate,
                                          const int32_t* grouped_layout, int m_total, int f,
                                          int k, int num_groups, int activation, void* workspace,
                                          size_t workspace_bytes, hipStream_t stream) {
    return gated_backward(kContiguous, a, sfa, b, sfb, dh, da, db, db_dtype, accumulate,
                          grouped_layout, m_total, f, k, num_groups, activation, workspace,
                          workspace_bytes, stream);
}

}  // extern "C"

// What the MXFP4 entry points launch, asked without a GPU: their host code, built with
// AddressSanitizer and UndefinedBehaviorSanitizer, against stand-ins for the HIP calls that
// it makes (a device of 256 compute units; a launch is recorded, nothing runs).
// tests/_mx_launches.py builds and feeds it.
//
// A line of input: cap op layout m expected n k groups flag.  op: quantise dequantise product
// gated gated_q layer (n: f; flag: n of the layer, columns of its output) backward (n: f; flag:
// 1 da + 2 db, 4 added for an f32 db, 8 for accumulation) size (backward, of the same) and
// layer_size.  A line of output: status or size, then "name grid threads" of every launch,
// separated by ';'.  With an argument it prints the names of all kernels instead.
#include <cxxabi.h>
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <string>

#include "fp8bs.h"

static int g_cap = 0;
static std::string g_seen;
static std::map<const void*, std::string>& names() {
    static std::map<const void*, std::string> m;
    return m;
}

extern "C" {
int fp8bs_get_num_cus(void) { return g_cap; }
int64_t fp8bs_get_sfa_ld(int64_t rows) { return rows < 0 ? -1 : (rows + 3) / 4 * 4; }

void** __hipRegisterFatBinary(const void*) {
    static void* handle;
    return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void* host, char*, const char* device, unsigned, void*,
                           void*, void*, void*, int*) {
    int bad = 0;
    char* plain = abi::__cxa_demangle(device, nullptr, nullptr, &bad);
    std::string s = plain ? plain : device;
    free(plain);
    const size_t at = s.find("mx_");
    s = s.substr(at == std::string::npos ? 0 : at);
    const size_t end = s.rfind('(');
    names()[host] = s.substr(0, end);
}
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
    *d = 0;
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
    *v = 256;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void**, size_t, hipStream_t) {
    const auto it = names().find(fn);
    g_seen += "; " + (it == names().end() ? std::string("unknown") : it->second) + " " +
              std::to_string(grid.x) + " " + std::to_string(block.x);
    // a launch's threads along a dimension are a 32-bit number
    if (grid.x < 1 || (uint64_t)grid.x * block.x > 0xFFFFFFFFull) return hipErrorInvalidConfiguration;
    return hipSuccess;
}
}  // extern "C"

int main(int argc, char**) {
    if (argc > 1) {
        for (const auto& it : names()) printf("%s\n", it.second.c_str());
        return 0;
    }
    // addresses of the right alignment that nothing may read
    void* p = (void*)(uintptr_t)4096;
    int32_t* ip = (int32_t*)p;
    char op[32];
    long long cap, layout, m, expected, n, k, g, flag;
    while (scanf("%lld %31s %lld %lld %lld %lld %lld %lld %lld", &cap, op, &layout, &m, &expected, &n,
                 &k, &g, &flag) == 9) {
        g_cap = (int)cap;
        g_seen.clear();
        const std::string o = op;
        const size_t all = (size_t)1 << 62;
        const int M = (int)m, E = (int)expected, N = (int)n, K = (int)k, G = (int)g;
        long long st = -100;
        if (o == "quantise") st = fp8bs_quantize_mxfp4(p, (int)flag, p, ip, G, M, K, nullptr);
        if (o == "dequantise") st = fp8bs_dequantize_mxfp4(p, ip, p, (int)flag, G, M, K, nullptr);
        if (o == "product")
            st = layout == 0   ? fp8bs_dense_nt_mxfp4(p, ip, p, ip, p, M, N, K, nullptr)
                 : layout == 1 ? fp8bs_grouped_contiguous_nt_mxfp4(p, ip, p, ip, p, ip, M, N, K, G, nullptr)
                               : fp8bs_grouped_masked_nt_mxfp4(p, ip, p, ip, p, ip, G, M, E, N, K, nullptr);
        if (o == "gated")
            st = layout == 0   ? fp8bs_gated_dense_mxfp4(p, ip, p, ip, p, M, N, K, 0, nullptr)
                 : layout == 1 ? fp8bs_gated_contiguous_mxfp4(p, ip, p, ip, p, ip, M, N, K, G, 0, nullptr)
                               : fp8bs_gated_masked_mxfp4(p, ip, p, ip, p, ip, G, M, E, N, K, 0, nullptr);
        if (o == "gated_q")
            st = layout == 0   ? fp8bs_gated_dense_mxfp4_q(p, ip, p, ip, p, ip, M, N, K, 0, nullptr)
                 : layout == 1 ? fp8bs_gated_contiguous_mxfp4_q(p, ip, p, ip, p, ip, ip, M, N, K, G, 0, nullptr)
                               : fp8bs_gated_masked_mxfp4_q(p, ip, p, ip, p, ip, ip, G, M, E, N, K, 0, nullptr);
        if (o == "layer")
            st = fp8bs_feed_forward_mxfp4((int)layout, p, 1, p, ip, p, ip, p, ip, M, E, N, K, (int)flag, G,
                                          0, p, all, nullptr);
        if (o == "backward") {
            void* da = flag & 1 ? p : nullptr;
            void* db = flag & 2 ? p : nullptr;
            const int dt = flag & 4 ? 0 : 1, add = flag & 8 ? 1 : 0;
            st = layout == 0 ? fp8bs_gated_dense_mxfp4_backward(p, ip, p, ip, p, da, db, dt, add, M, N, K,
                                                                0, p, all, nullptr)
                             : fp8bs_gated_contiguous_mxfp4_backward(p, ip, p, ip, p, da, db, dt, add, ip,
                                                                     M, N, K, G, 0, p, all, nullptr);
        }
        if (o == "size")
            st = fp8bs_gated_backward_workspace_size((int)layout, m, N, K, G, (int)(flag & 1), (int)(flag & 2));
        if (o == "layer_size") st = fp8bs_feed_forward_workspace_size((int)layout, m, N, K, G);
        printf("%lld%s\n", st, g_seen.c_str());
    }
    return 0;
}

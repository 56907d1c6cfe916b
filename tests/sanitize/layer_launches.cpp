// What the operators between the FP8 products launch, asked without a GPU: their host code, built
// with AddressSanitizer and UndefinedBehaviorSanitizer, against stand-ins for the HIP calls that it
// makes (a device of 256 compute units; a launch is recorded, nothing runs).
// tests/test_layer_launches.py builds and feeds it.
//
// A line of input: cap op a b c d e.  norm: rows k types(x + 4 res + 16 weight; 2: no residual) outputs(1 y,
// 2 q); norm_back: rows k types dweight; dispatch: layout tokens topk groups m (k 256, e4m3);
// combine: tokens topk k; combine_back: tokens topk k; gated: layout m f slots keep; gated_back:
// m f kept act; columns: rows n type.  A line of output: status, then "name grid threads" of every launch,
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
    const size_t at = s.find("namespace)::");
    s = s.substr(at == std::string::npos ? 0 : at + 12);
    names()[host] = s.substr(0, s.find('('));
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
    float* fp = (float*)p;
    const size_t all = (size_t)1 << 62;
    char op[32];
    long long cap, a, b, c, d, e;
    while (scanf("%lld %31s %lld %lld %lld %lld %lld", &cap, op, &a, &b, &c, &d, &e) == 7) {
        g_cap = (int)cap;
        g_seen.clear();
        const std::string o = op;
        const int A = (int)a, B = (int)b, C = (int)c, D = (int)d, E = (int)e;
        long long st = -100;
        if (o == "norm")
            st = fp8bs_rms_norm(p, C & 3, (C >> 2 & 3) == 2 ? nullptr : p, p, (C >> 2 & 3) & 1, p,
                                C >> 4 & 1, D & 1 ? p : nullptr, 1, D & 2 ? p : nullptr, fp, fp, A, B,
                                1e-6f, nullptr);
        if (o == "norm_back")
            st = fp8bs_rms_norm_backward(p, C & 3, fp, p, C >> 4 & 1, p, C >> 2 & 3, p, p,
                                         D ? fp : nullptr, 0, A, B, p, all, nullptr);
        if (o == "dispatch")
            st = fp8bs_moe_dispatch(A, p, 4, p, FP8BS_DTYPE_E4M3, fp, p, fp, ip, ip, ip, B, C, D, E, 256,
                                    p, all, nullptr);
        if (o == "dispatch_size") st = fp8bs_moe_dispatch_workspace_size(A, b, C, D, e);
        if (o == "combine") st = fp8bs_moe_combine(p, ip, fp, p, D, 1000, A, B, C, nullptr);
        if (o == "combine_back")
            st = fp8bs_moe_combine_backward(p, D, p, ip, fp, p, C % 128 ? nullptr : p, fp, fp, 1, 1000, A,
                                            B, C, nullptr);
        if (o == "gated")
            st = fp8bs_gated_quantize(A, p, p, fp, E & 1 ? p : nullptr, fp, ip, B, C, D, E >> 1, nullptr);
        if (o == "gated_back")
            st = fp8bs_gated_quantize_backward(p, C ? FP8BS_DTYPE_E4M3 : FP8BS_DTYPE_BF16, fp, p, p, p,
                                               fp, p, fp, p, fp, E ? ip : nullptr, A, B, D, nullptr);
        if (o == "columns") st = fp8bs_quantize_128x1(p, C, fp, p, fp, D ? ip : nullptr, A, B, nullptr);
        printf("%lld%s\n", st, g_seen.c_str());
    }
    return 0;
}

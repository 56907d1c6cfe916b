// In which parts the norm's backward pass adds dweight, asked without a GPU: its host code, built with
// AddressSanitizer and UndefinedBehaviorSanitizer around stand-ins for the HIP calls that it makes, which
// look at what a launch would give its kernel.  tests/test_layer_sums.py builds and feeds it.
//
// A line of input: cap cus rows k in_place.  A line of output: status, then for every launch its grid, and
// "rows" units tiles direct (no parts), or "sum" parts tiles.
#include "fp8bs_norm.hip"

#include <stdio.h>

#include <string>

static int g_cap = 0, g_cus = 256;
static std::string g_seen;

extern "C" {
int fp8bs_get_num_cus(void) { return g_cap; }
int64_t fp8bs_get_sfa_ld(int64_t rows) { return rows < 0 ? -1 : (rows + 3) / 4 * 4; }
void** __hipRegisterFatBinary(const void*) {
    static void* handle;
    return &handle;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipSuccess; }
hipError_t hipGetDevice(int* d) {
    *d = 0;
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t, int) {
    *v = g_cus;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3, void** args, size_t, hipStream_t) {
    using namespace fp8bs::layer;
    g_seen += "; " + std::to_string(grid.x);
    if (fn == (const void*)rms_norm_sum_kernel) {
        const SumParams& p = *(const SumParams*)args[0];
        g_seen += " sum " + std::to_string(p.parts) + " " + std::to_string(p.tiles);
    } else {
        const BackwardParams& p = *(const BackwardParams*)args[0];
        g_seen += " rows " + std::to_string(p.units) + " " + std::to_string(p.tiles) + " " + (p.part ? "0" : "1");
    }
    return hipSuccess;
}
}  // extern "C"

int main() {
    // addresses of the right alignment that nothing may read
    void *p = (void*)(uintptr_t)4096, *other = (void*)(uintptr_t)8192;
    int rows, k, in_place;
    while (scanf("%d %d %d %d %d", &g_cap, &g_cus, &rows, &k, &in_place) == 5) {
        g_seen.clear();
        const int st = fp8bs_rms_norm_backward(p, FP8BS_DTYPE_BF16, (const float*)p, p, FP8BS_DTYPE_BF16, p, FP8BS_DTYPE_BF16, p,
                                               in_place ? p : other, (float*)p, 0, rows, k, p, (size_t)1 << 62, nullptr);
        printf("%d%s\n", st, g_seen.c_str());
    }
    return 0;
}

// The 8-bit layer's calls with their arguments in one array, for the Python
// binding: ctypes takes 0.2 us to convert an argument (3.8 us for the norm's
// nineteen), struct.pack all of them in 0.4 us.  Not part of the C ABI.
#include <string.h>

#include "gemm_scaled.h"

namespace {

template <typename T>
T* ptr(int64_t v) { return reinterpret_cast<T*>(static_cast<uintptr_t>(v)); }

float real(int64_t v) {  // a double's bits
    double d;
    memcpy(&d, &v, sizeof d);
    return (float)d;
}

}  // namespace

extern "C" int psm_packed_call(int op, const int64_t* a) {
    switch (op) {
        case 0:
            return gemm_scaled_quantize((gemm_quantize_t)a[0], ptr<void>(a[1]), a[2], a[3], a[4], (gemm_dtype_t)a[5], (gemm_fp8_t)a[6],
                                        ptr<void>(a[7]), a[8], ptr<float>(a[9]), ptr<CUstream_st>(a[10]));
        case 1:
            return gemm_scaled_quantize_both(ptr<void>(a[0]), a[1], a[2], a[3], (gemm_dtype_t)a[4], (gemm_fp8_t)a[5], ptr<void>(a[6]), a[7],
                                             ptr<float>(a[8]), ptr<void>(a[9]), a[10], ptr<float>(a[11]), ptr<CUstream_st>(a[12]));
        case 2:
            return gemm_rms_norm(ptr<void>(a[0]), a[1], ptr<void>(a[2]), a[3], ptr<void>(a[4]), real(a[5]), a[6], a[7], (gemm_dtype_t)a[8],
                                 ptr<void>(a[9]), a[10], ptr<void>(a[11]), a[12], ptr<void>(a[13]), a[14], (gemm_fp8_t)a[15],
                                 ptr<float>(a[16]), ptr<float>(a[17]), ptr<CUstream_st>(a[18]));
        case 3:
            return gemm_rms_norm_grad(ptr<void>(a[0]), a[1], ptr<void>(a[2]), a[3], ptr<void>(a[4]), ptr<float>(a[5]), ptr<void>(a[6]), a[7],
                                      a[8], a[9], (gemm_dtype_t)a[10], ptr<void>(a[11]), a[12], ptr<float>(a[13]), ptr<void>(a[14]),
                                      ptr<CUstream_st>(a[15]));
        case 4:
            return gemm_scaled_run(ptr<gemm_scaled_plan>(a[0]), ptr<void>(a[1]), ptr<float>(a[2]), ptr<void>(a[3]), ptr<float>(a[4]),
                                   ptr<void>(a[5]), ptr<void>(a[6]), ptr<CUstream_st>(a[7]));
        default: return GEMM_ERR_INVALID_ARG;
    }
}

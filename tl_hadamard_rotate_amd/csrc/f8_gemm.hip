#include "tl_internal.h"

namespace tl {

int64_t f8_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k) { return 0; }

hipError_t launch_f8_gemm(const uint8_t* codes, const uint8_t* scales, const uint8_t* x, const uint8_t* x_scales,
                          int64_t m, int64_t n, int64_t k, void* y, int y_dtype, void* ws, hipStream_t stream) {
    return launch_f8_gemv(codes, scales, x, x_scales, m, n, k, y, y_dtype, stream);
}

}  // namespace tl

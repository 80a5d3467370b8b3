// C ABI of the microscaled 8-bit rows: argument checks, the choice of a kernel
// and the launches.  Declarations and contracts are in include/sgemm.h.
#include "sgemm.h"

#include <hip/hip_runtime.h>

#include "mx_host.hpp"

using namespace sgemm;

extern "C" {

int sgemm_mx_byte_quantize(sgemm_handle_t h, int dtype, int trans, int R, int K, const void* X,
                       int ldx, void* codes, int ldc, void* scales, int lds,
                       hipStream_t stream) {
  return quantize_entry<Mx8Format>(h, dtype, trans, R, K, X, ldx, codes, ldc, scales, lds, stream);
}

int sgemm_mx_byte_dequantize(sgemm_handle_t h, int dtype, int R, int K, const void* codes, int ldc,
                         const void* scales, int lds, void* Y, int ldy, hipStream_t stream) {
  return dequantize_entry<Mx8Format>(h, dtype, R, K, codes, ldc, scales, lds, Y, ldy, stream);
}

}  // extern "C"

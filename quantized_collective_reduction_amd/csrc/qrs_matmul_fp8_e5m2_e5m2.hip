// The 8-bit floating-point product of E5M2 a and E5M2 b.

#include "qrs_matmul_fp8.h"

namespace qrs {

hipError_t launch_fp8_e5m2_e5m2(const MatmulFp8Launch& l, hipStream_t stream) {
  return launch_formats<kXE5M2, kXE5M2>(l, stream);
}

}  // namespace qrs

// The 8-bit floating-point product of E4M3 a and E4M3 b, and the choice between
// the formats.

#include "qrs_matmul_fp8.h"

namespace qrs {

hipError_t launch_fp8_e4m3_e4m3(const MatmulFp8Launch& l, hipStream_t stream) {
  return launch_formats<kXE4M3FN, kXE4M3FN>(l, stream);
}

hipError_t launch_matmul_fp8(const MatmulFp8Launch& l, hipStream_t stream) {
  if (l.a_format == kXE4M3FN)
    return l.b_format == kXE4M3FN ? launch_fp8_e4m3_e4m3(l, stream) : launch_fp8_e4m3_e5m2(l, stream);
  return l.b_format == kXE4M3FN ? launch_fp8_e5m2_e4m3(l, stream) : launch_fp8_e5m2_e5m2(l, stream);
}

// The choice does not go by the formats.
MatmulShape matmul_fp8_shape(const MatmulFp8Launch& l) {
  const Choice c = choose<kXE4M3FN, kXE4M3FN>(l);
  return {c.id, c.blocks, c.threads};
}

}  // namespace qrs

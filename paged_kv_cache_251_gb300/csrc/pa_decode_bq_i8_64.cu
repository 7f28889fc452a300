// Block-scaled decode kernels: INT8 codes, head_dim 64.
#include "pa_decode_bq.cuh"

namespace pa {

const void *decode_bq_kernel_i8_64(bool wide, bool f32, bool b8) { return decode_bq_kernel<64, kFmtI8>(wide, f32, b8); }

}  // namespace pa

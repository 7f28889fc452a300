// Block-scaled decode kernels: E4M3 codes, head_dim 128.
#include "pa_decode_bq.cuh"

namespace pa {

const void *decode_bq_kernel_e4m3_128(bool wide, bool f32, bool b8) { return decode_bq_kernel<128, kFmtE4M3>(wide, f32, b8); }

}  // namespace pa

// decode_fp4_d128_g8.cu -- decode_fp4_kernel at head_dim 128 for groups of up to 8 query heads.
#include "decode_fp4_kernel.cuh"

namespace minisgl {

template cudaError_t launch_decode_fp4_as<128, 1>(const DecodeFp4Args &, cudaStream_t);
template cudaError_t read_fp4_timeouts_as<128, 1>(unsigned int *);

}  // namespace minisgl

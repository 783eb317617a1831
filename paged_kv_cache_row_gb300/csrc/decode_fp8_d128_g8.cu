// decode_fp8_d128_g8.cu -- decode_fp8_kernel at head_dim 128 for groups of up to 8 query heads.
#include "decode_fp8_kernel.cuh"

namespace minisgl {

template cudaError_t launch_decode_fp8_as<128, 1>(const DecodeFp8Args &, cudaStream_t);
template cudaError_t read_fp8_timeouts_as<128, 1>(unsigned int *);

}  // namespace minisgl

// decode_fp8_d64_g8.cu -- decode_fp8_kernel at head_dim 64 for groups of up to 8 query heads.
#include "decode_fp8_kernel.cuh"

namespace minisgl {

template cudaError_t launch_decode_fp8_as<64, 1>(const DecodeFp8Args &, cudaStream_t);
template cudaError_t read_fp8_timeouts_as<64, 1>(unsigned int *);

}  // namespace minisgl

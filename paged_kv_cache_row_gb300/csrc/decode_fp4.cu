// decode_fp4.cu -- decode attention over the 4-bit pool: the choice of kernel.
//
// The kernels (decode_fp4_kernel.cuh) are compiled in one file per head_dim
// and number of 8-head query tiles, each for 1 to 8 KV heads.
#include "kernels.h"

namespace minisgl {

template <int D, int NG>
cudaError_t launch_decode_fp4_as(const DecodeFp4Args &a, cudaStream_t s);
template <int D, int NG>
cudaError_t read_fp4_timeouts_as(unsigned int *count);

cudaError_t launch_decode_fp4(const DecodeFp4Args &a, cudaStream_t s) {
    if (a.d.batch == 0) return cudaSuccess;
    const int G = a.d.num_q_heads / a.d.num_kv_heads;
    if (a.d.head_dim == 128)
        return G <= 8 ? launch_decode_fp4_as<128, 1>(a, s) : launch_decode_fp4_as<128, 2>(a, s);
    return G <= 8 ? launch_decode_fp4_as<64, 1>(a, s) : launch_decode_fp4_as<64, 2>(a, s);
}

cudaError_t read_fp4_timeouts(unsigned int *count) {
    *count = 0;
    for (auto read : {read_fp4_timeouts_as<128, 1>, read_fp4_timeouts_as<128, 2>, read_fp4_timeouts_as<64, 1>,
                      read_fp4_timeouts_as<64, 2>}) {
        unsigned int n = 0;
        const cudaError_t e = read(&n);
        if (e != cudaSuccess) return e;
        *count += n;
    }
    return cudaSuccess;
}

}  // namespace minisgl

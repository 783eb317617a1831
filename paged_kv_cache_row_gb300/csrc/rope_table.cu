// rope_table.cu -- rows [m cos(p theta_j) | m sin(p theta_j)] of the cos/sin
// table that the rotary stores read, for given positions p.
//
// An angle matters modulo one turn, and fp32 loses it: at p = 10^6 a product
// p * theta is off by up to 0.03.  So a frequency is a 64-bit fixed-point
// number of turns, theta / 2 pi * 2^64, whose product with p modulo 2^64 is the
// angle in turns modulo 1, exactly (the frequency's own rounding, in double,
// moves the angle by at most p * 2^-53 of theta).  The two highest bits of the
// phase (rounded) are the quarter turn; cos and sin of the rest, at most pi/4,
// are their Taylor polynomials up to x^10 and x^9, whose first terms left out
// are below 2^-32 and 2^-29.
//
// Bound by writes, 4 rotary_dim bytes a position, if a pair takes few
// instructions: a thread keeps four frequencies in registers and goes over
// positions.  131072 positions of 128 channels: 14.1 us, 4.8 TB/s of writes (a
// copy moves 6.8 TB/s, half of them reads; a fill of more than L2 writes 3.8).
// With the frequencies read from the parameters by every thread 15.3.
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int THREADS = 256;
constexpr int RESIDENT = 8;  // blocks per SM

// cos and sin of phase / 2^64 turns
__device__ __forceinline__ void cos_sin_of(uint64_t phase, float &c, float &s) {
    const uint32_t quarter = (uint32_t)((phase + (1ull << 61)) >> 62);
    const int64_t rest = (int64_t)(phase - ((uint64_t)quarter << 62));  // within 1/8 turn
    // the high word as a float, and the low one where it still counts
    const float turns = fmaf((float)(uint32_t)rest, 0x1p-32f, (float)(int32_t)(rest >> 32));
    const float x = turns * (float)(6.283185307179586 * 0x1p-32), z = x * x;
    const float sn = fmaf(x * z, fmaf(z, fmaf(z, fmaf(z, 1.f / 362880.f, -1.f / 5040.f), 1.f / 120.f), -1.f / 6.f), x);
    const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -1.f / 3628800.f, 1.f / 40320.f), -1.f / 720.f), 1.f / 24.f),
                                  -0.5f), 1.f);
    c = quarter & 1 ? sn : cs;
    s = quarter & 1 ? cs : sn;
    if (quarter == 1 || quarter == 2) c = -c;
    if (quarter >= 2) s = -s;
}

}  // namespace

// h / 4 threads a position (h = rotary_dim / 2), `rows` positions a block at a time.
__global__ void __launch_bounds__(THREADS, RESIDENT) rope_table_kernel(const __grid_constant__ RopeTableArgs a, int rows) {
    // through shared memory: lanes that read parameters at different places do so one after the other
    __shared__ uint64_t s_turns[ROPE_MAX_DIM / 2];
    const int h = a.rotary_dim / 2, per_row = h / 4;
    if ((int)threadIdx.x < h) s_turns[threadIdx.x] = a.turns[threadIdx.x];
    __syncthreads();
    pdl_wait();  // no early start for the next kernel: rope_store_kv reads the table with non-coherent loads
    const int sub = threadIdx.x / per_row, j = (threadIdx.x - sub * per_row) * 4;
    if (sub >= rows) return;
    uint64_t f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = s_turns[j + k];
    for (int64_t i = (int64_t)blockIdx.x * rows + sub; i < a.n; i += (int64_t)gridDim.x * rows) {
        const uint64_t p = (uint64_t)(int64_t)a.positions[i];
        float c[4], s[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            cos_sin_of(f[k] * p, c[k], s[k]);
            c[k] *= a.attention;
            s[k] *= a.attention;
        }
        float *row = a.out + i * a.rotary_dim + j;
        *reinterpret_cast<float4 *>(row) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4 *>(row + h) = make_float4(s[0], s[1], s[2], s[3]);
    }
}

cudaError_t launch_rope_table(const RopeTableArgs &a, cudaStream_t s) {
    if (a.n == 0) return cudaSuccess;
    const int rows = THREADS / (a.rotary_dim / 8);
    const int64_t blocks = std::min<int64_t>(((int64_t)a.n + rows - 1) / rows, (int64_t)device_sm_count() * RESIDENT);
    return launch_pdl(rope_table_kernel, dim3((unsigned)blocks), dim3(THREADS), 0, s, a, rows);
}

}  // namespace minisgl

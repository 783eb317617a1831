// rope_table.cu -- rows [m cos(p theta_j) | m sin(p theta_j)] of the cos/sin
// table that the rotary stores read, for given positions p.
//
// An angle matters modulo one turn, and fp32 loses it: at p = 10^6 a product
// p * theta is off by up to 0.03.  So a frequency is a 64-bit fixed-point
// number of turns, theta / 2 pi * 2^64, whose product with p modulo 2^64 is the
// angle in turns modulo 1, exactly (what the frequency itself is off by, computed
// in double, moves the angle by at most p * 2^-50 radians, for frequencies in bands
// by a small multiple).  The two highest bits of the
// phase (rounded) are the quarter turn; cos and sin of the rest, at most pi/4,
// are their Taylor polynomials up to x^10 and x^9, whose first terms left out
// are below 2^-32 and 2^-29.  From the reduced angle on everything is fp32, for
// the call is bound by issue slots: rows are off by 2.9e-8 and 3.9e-8 (of the
// norm) where a 64-bit result rounded once is off by 2.1e-8 and 2.7e-8.
//
// Bound by writes, 4 rotary_dim bytes a position, and nearly as much by issue
// slots: a thread keeps four frequencies in registers and goes over positions,
// two frequencies at a time (the polynomials in packed pairs).  131072 positions
// of 128 channels: 11.9 us, 5.7 TB/s of writes; a fill of the same 67 MB, which
// stay in L2, takes 9.3.  Steps: 15.3 - 14.1 (the frequencies through shared
// memory) - 12.8 (the quarter turn in 32-bit words, signs on the factor) - 11.9.
#include <algorithm>

#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int THREADS = 256;
constexpr int RESIDENT = 5;  // blocks per SM (8 leave 32 registers: 12.3 us instead of 11.9)

// Two floats in a 64-bit register: one multiply-add for both.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};\n" : "=l"(v) : "f"(a), "f"(b));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t v;
    asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(v) : "l"(a), "l"(b), "l"(c));
    return v;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t v;
    asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(v) : "l"(a), "l"(b));
    return v;
}
__device__ __forceinline__ uint64_t both(float a) { return pair_of(a, a); }

// The quarter turn that position p is in under frequency f, and the rest of the
// angle in turns * 2^32, within 1/8 turn.  (All in 32-bit words: the quarter is
// decided by the phase's high word, and only that changes when it is taken off.)
__device__ __forceinline__ float rest_of(uint64_t f, int p, uint32_t &quarter) {
    const uint64_t phase = f * (uint64_t)(int64_t)p;
    const uint32_t high = (uint32_t)(phase >> 32) + (1u << 29);
    quarter = high >> 30;
    const int rest = (int)(high & 0x3fffffffu) - (1 << 29);
    // the high word as a float, and the low one where it still counts
    return fmaf((float)(uint32_t)phase, 0x1p-32f, (float)rest);
}

// m cos and m sin of position p under two frequencies.
__device__ __forceinline__ void cos_sin_of(const uint64_t *f, int p, float m, float *c, float *s) {
    uint32_t quarter[2];
    const float r0 = rest_of(f[0], p, quarter[0]), r1 = rest_of(f[1], p, quarter[1]);
    const uint64_t x = mul2(pair_of(r0, r1), both((float)(6.283185307179586 * 0x1p-32))), z = mul2(x, x);
    const uint64_t sn = fma2(mul2(x, z), fma2(z, fma2(z, fma2(z, both(1.f / 362880.f), both(-1.f / 5040.f)),
                                                      both(1.f / 120.f)), both(-1.f / 6.f)), x);
    const uint64_t cs = fma2(z, fma2(z, fma2(z, fma2(z, fma2(z, both(-1.f / 3628800.f), both(1.f / 40320.f)),
                                                     both(-1.f / 720.f)), both(1.f / 24.f)), both(-0.5f)), both(1.f));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float sk = __uint_as_float((uint32_t)(sn >> (32 * k))), ck = __uint_as_float((uint32_t)(cs >> (32 * k)));
        // quarters 0 to 3: (ck, sk), (-sk, ck), (-ck, -sk), (sk, -ck)
        const uint32_t q = quarter[k], sign_c = (q + 1u) << 30 & 0x80000000u, sign_s = q << 30 & 0x80000000u;
        c[k] = (q & 1u ? sk : ck) * __uint_as_float(__float_as_uint(m) ^ sign_c);
        s[k] = (q & 1u ? ck : sk) * __uint_as_float(__float_as_uint(m) ^ sign_s);
    }
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
        const int p = a.positions[i];
        float c[4], s[4];
#pragma unroll
        for (int k = 0; k < 4; k += 2) cos_sin_of(f + k, p, a.attention, c + k, s + k);
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

// store_kv_fp4.cu -- new K/V rows into the 4-bit pool, and cached rows out of it.
//
// Store: a thread quantises one block of 16 channels: 32 bytes of bf16 in,
// 8 bytes of e2m1 pairs and one e4m3 scale out.
//     a = max|x| * 2^-exp,  s = e4m3(a / 6),  c = e2m1(x * 2^-exp / s)
// Every rounding is decided exactly.  x has 8 significant bits and 2^-exp
// moves only its exponent.  A border between two e4m3 values has at most 5
// bits, six times it 7, so a is either exactly on it or at least a relative
// 2^-8 away: a / 6 rounded to fp32 falls on the same side.  A border between
// two e2m1 values has at most 3 bits, times s 7, so x * 2^-exp / s too is
// either exactly on a border or 2^-8 away from all of them.  x times the
// rounded 1/s is within 2^-22 of the quotient; rounded once more, to 12
// significant bits, it is exactly on the border in the first case and on the
// right side of it in the second.
// Load: the reverse, bf16(c * s * 2^exp), which is exact.
#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {
constexpr int FP4_THREADS = 256;

// x to 12 significant bits, nearest; keeps signs and infinities
__device__ __forceinline__ float round12(float x) {
    return __uint_as_float((__float_as_uint(x) + 0x800u) & 0xfffff000u);
}
}  // namespace

// blocks16: blocks of 16 per K (or V) row.  Item w: token, then K or V, then
// the block, so neighbouring threads take neighbouring blocks of one row.
__global__ void __launch_bounds__(FP4_THREADS) store_kv_fp4_kernel(StoreFp4Args a, uint32_t blocks16,
                                                                   int log2_per_tok) {
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t per_tok = 2u * blocks16;
    const uint32_t total = (uint32_t)a.n_tokens * per_tok;
    for (uint32_t w = blockIdx.x * FP4_THREADS + threadIdx.x; w < total; w += gridDim.x * FP4_THREADS) {
        const uint32_t i = log2_per_tok >= 0 ? w >> log2_per_tok : w / per_tok;
        const uint32_t rem = w - i * per_tok;
        const bool is_v = rem >= blocks16;
        const uint32_t blk = is_v ? rem - blocks16 : rem;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(is_v ? a.v : a.k) +
                                   (int64_t)i * (is_v ? a.v_tok_stride : a.k_tok_stride) + blk * FP4_BLOCK;
        const uint4 x0 = ld_nc_v4(src), x1 = ld_nc_v4(src + 8);
        const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        // max|x| on the bit patterns: infinity above every number, NaN above infinity
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = __vmaxu2(m, x[j] & 0x7fff7fffu);
        m = max(m & 0xffffu, m >> 16);
        const float unit = pow2i(-(is_v ? a.pool.v_exp : a.pool.k_exp));
        const uint32_t sb = f32_to_e4m3(__fdiv_rn(__uint_as_float(m << 16) * unit, 6.f));
        const float s = f16x2_to_f32(e4m3x2_to_f16x2(sb)).x;
        const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
        float y[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            y[2 * j] = round12(__uint_as_float(x[j] << 16) * unit * inv);
            y[2 * j + 1] = round12(__uint_as_float(x[j] & 0xffff0000u) * unit * inv);
        }
        int row = __ldg(a.out_loc + i);
        // out-of-range rows are a caller error; clamp so the write stays in the pool
        row = min(max(row, 0), a.pool.num_rows - 1);
        *reinterpret_cast<uint2 *>((is_v ? a.pool.v_data : a.pool.k_data) + (int64_t)row * a.pool.data_stride +
                                   blk * (FP4_BLOCK / 2)) = make_uint2(f32_to_e2m1x8(y), f32_to_e2m1x8(y + 8));
        ((is_v ? a.pool.v_scale : a.pool.k_scale) + (int64_t)row * a.pool.scale_stride)[blk] = (uint8_t)sb;
    }
}

namespace {

// Tokens a block of the load kernel takes at a time.
constexpr int LOAD_TOKENS = 32;

}  // namespace

__global__ void __launch_bounds__(FP4_THREADS) load_kv_fp4_kernel(LoadFp4Args a, uint32_t blocks16) {
    __shared__ int s_row[LOAD_TOKENS];  // pool row of each token, or -1
    pdl_wait();
    pdl_launch_dependents();
    const float k_unit = pow2i(a.pool.k_exp), v_unit = pow2i(a.pool.v_exp);
    const uint32_t per_tok = 2u * blocks16;
    const int64_t tiles = ((int64_t)a.total_tokens + LOAD_TOKENS - 1) / LOAD_TOKENS;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int64_t t0 = tile * LOAD_TOKENS;
        if (threadIdx.x < LOAD_TOKENS) {
            const int64_t t = t0 + threadIdx.x;
            int row = -1;
            if (t < a.total_tokens) {
                int lo = 0, hi = a.batch;  // the last request with offsets[r] <= t
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (__ldg(a.offsets + mid) <= t) lo = mid; else hi = mid;
                }
                const int64_t j = t - __ldg(a.offsets + lo);
                const int n = min(max(__ldg(a.lens + lo), 0), a.pt_width);
                if (j >= 0 && j < n && t < __ldg(a.offsets + lo + 1))
                    row = min(max(__ldg(a.page_table + lo * a.pt_stride + j), 0), a.pool.num_rows - 1);
            }
            s_row[threadIdx.x] = row;
        }
        __syncthreads();
        for (uint32_t w = threadIdx.x; w < LOAD_TOKENS * per_tok; w += FP4_THREADS) {
            const uint32_t i = w / per_tok, rem = w - i * per_tok;
            const int row = s_row[i];
            if (row < 0) continue;
            const bool is_v = rem >= blocks16;
            const uint32_t blk = is_v ? rem - blocks16 : rem;
            const uint2 c = *reinterpret_cast<const uint2 *>((is_v ? a.pool.v_data : a.pool.k_data) +
                                                             (int64_t)row * a.pool.data_stride + blk * (FP4_BLOCK / 2));
            const uint32_t sb = ((is_v ? a.pool.v_scale : a.pool.k_scale) + (int64_t)row * a.pool.scale_stride)[blk];
            const uint32_t s = e4m3x2_to_f16x2(sb | (sb << 8));
            const float unit = is_v ? v_unit : k_unit;
            uint32_t h[2][4], o[8];
            e2m1x8_to_f16x2(c.x, h[0]);
            e2m1x8_to_f16x2(c.y, h[1]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = f16x2_to_f32(mul_f16x2(h[j >> 2][j & 3], s));
                o[j] = pack_bf16x2(f.x * unit, f.y * unit);
            }
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_v ? a.v_out : a.k_out) +
                                 (t0 + i) * (is_v ? a.v_tok_stride : a.k_tok_stride) + blk * FP4_BLOCK;
            st_v4(dst, make_uint4(o[0], o[1], o[2], o[3]));
            st_v4(dst + 8, make_uint4(o[4], o[5], o[6], o[7]));
        }
        __syncthreads();
    }
}

cudaError_t launch_store_kv_fp4(const StoreFp4Args &a, cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    const int64_t blocks16 = (int64_t)a.pool.num_kv_heads * a.pool.head_dim / FP4_BLOCK;
    const int64_t per_tok = 2 * blocks16, total = a.n_tokens * per_tok;
    if (total >= (int64_t(1) << 31)) return cudaErrorInvalidValue;  // the host refuses this first
    int log2_per_tok = -1;
    if ((per_tok & (per_tok - 1)) == 0)
        for (log2_per_tok = 0; (int64_t(1) << log2_per_tok) < per_tok; ++log2_per_tok) {
        }
    int64_t blocks = (total + FP4_THREADS - 1) / FP4_THREADS;
    const int64_t cap = (int64_t)device_sm_count() * 8;
    if (blocks > cap) blocks = cap;
    return launch_pdl(store_kv_fp4_kernel, dim3((unsigned)blocks), dim3(FP4_THREADS), 0, s, a, (uint32_t)blocks16,
                      log2_per_tok);
}

cudaError_t launch_load_kv_fp4(const LoadFp4Args &a, cudaStream_t s) {
    if (a.batch == 0 || a.total_tokens == 0) return cudaSuccess;
    const int64_t blocks16 = (int64_t)a.pool.num_kv_heads * a.pool.head_dim / FP4_BLOCK;
    int64_t blocks = ((int64_t)a.total_tokens + LOAD_TOKENS - 1) / LOAD_TOKENS;
    const int64_t cap = (int64_t)device_sm_count() * 8;
    if (blocks > cap) blocks = cap;
    return launch_pdl(load_kv_fp4_kernel, dim3((unsigned)blocks), dim3(FP4_THREADS), 0, s, a, (uint32_t)blocks16);
}

}  // namespace minisgl

// store_kv_fp4.cu -- new K/V rows into the 4-bit pool, and cached rows out of it.
//
// Store: a thread quantises one block of 16 channels: 32 bytes of bf16 in,
// 8 bytes of e2m1 pairs and one e4m3 scale out.
//     a = max|x| * 2^-exp,  s = e4m3(a / 6),  c = e2m1(x * 2^-exp / s)
// Every rounding is decided exactly.  x has 8 significant bits and 2^-exp
// moves only its exponent.  A border between two e4m3 values has at most 5
// bits, six times it 7, so a / 6 is either exactly on it or at least a
// relative 2^-8 away; a border between two e2m1 values has at most 3 bits,
// times s 7, so the same holds for x * 2^-exp / s.  The quotient x / s is
// formed from 1/s = r + t with r a little below 1/s and t = (1 - r s) r, the
// first step of Newton's iteration: fma(x, r, x t) is within 2^-40 of it
// before its one rounding, so a quotient that lies on a border comes out
// exactly there, and every other on its own side.  r, t > 0 keep the sign of
// a zero and let an infinity through (it saturates).
// Load: the reverse, bf16(c * s * 2^exp), which is exact.
//
// Both are bound by HBM (2.56 bytes a channel) only if the arithmetic stays
// near 8 instructions a channel.  So a thread keeps one column (K or V, and
// the block) for all its tokens: the division of the index and the choice of
// pointers happen once, not once per block, which took half of all issue
// slots.
#include <algorithm>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {
constexpr int MAX_THREADS = 512;
constexpr int STORE_RESIDENT = 1536;  // threads per SM: 40 registers, one block of 16 per thread in
                                      // flight (two took 64 registers and the same time)
constexpr int LOAD_RESIDENT = 1024;   // threads per SM of the load kernel
constexpr int LOAD_U = 4;             // blocks of 16 that a thread of it has in flight
constexpr int LOAD_TOKENS = 128; // most tokens of a load tile

}  // namespace

// Every load here is a coherent one: the kernel is resident while the one
// before it may still write the slots, the new rows or the pool.
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// 32 bytes from 32-byte (WIDE) or 16-byte aligned memory
template <bool WIDE>
__device__ __forceinline__ void ld_32(const void *p, uint32_t (&x)[8]) {
    if constexpr (WIDE) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                     : "l"(p));
    } else {
        const uint4 a = ld_v4(p), b = ld_v4(static_cast<const char *>(p) + 16);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}
template <bool WIDE>
__device__ __forceinline__ void st_32(void *p, const uint32_t (&x)[8]) {
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                     "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
    } else {
        st_v4(p, make_uint4(x[0], x[1], x[2], x[3]));
        st_v4(static_cast<char *>(p) + 16, make_uint4(x[4], x[5], x[6], x[7]));
    }
}

// 1/s = r + t to about 2^-40, for 2^-9 <= s <= 448
__device__ __forceinline__ void split_reciprocal(float s, float &r, float &t) {
    r = __fdividef(1.f, s) * (1.f - 0x1p-21f);  // below 1/s: the approximation is within 2 ulp
    t = fmaf(-r, s, 1.f) * r;
}

// One block of 16: x (bf16) to e2m1 pairs c and the scale's byte.
__device__ __forceinline__ void quantise16(const uint32_t (&x)[8], float unit, uint2 &c, uint32_t &sb) {
    // max|x| (its sign comes out as the exclusive or); a NaN wins
    uint32_t m = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;\n" : "+r"(m) : "r"(x[j]));
    m &= 0x7fff7fffu;
    m = max(m & 0xffffu, m >> 16);  // bit patterns order like the values, NaN above infinity
    float r, t;
    split_reciprocal(6.f, r, t);
    const float a = __uint_as_float(m << 16) * unit;
    sb = f32_to_e4m3(fmaf(a, r, a * t));
    const float s = f16x2_to_f32(e4m3x2_to_f16x2(sb)).x;
    split_reciprocal(s, r, t);
    r = s > 0.f ? r * unit : 0.f;
    t = s > 0.f ? t * unit : 0.f;
    float y[16];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float lo = __uint_as_float(x[j] << 16), hi = __uint_as_float(x[j] & 0xffff0000u);
        y[2 * j] = fmaf(lo, r, lo * t);
        y[2 * j + 1] = fmaf(hi, r, hi * t);
    }
    c = make_uint2(f32_to_e2m1x8(y), f32_to_e2m1x8(y + 8));
}

// A block of threads has one thread per column (K blocks of 16, then V blocks)
// of `toks` tokens; with more columns than threads (toks = 1) it goes over
// them in steps.  A thread takes every (grid * toks)-th token.
template <bool WIDE>
__global__ void __launch_bounds__(MAX_THREADS, STORE_RESIDENT / MAX_THREADS) store_kv_fp4_kernel(StoreFp4Args a, int blocks16, int toks) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = threadIdx.x / (2 * blocks16);
    if (sub >= toks) return;
    const int64_t step = (int64_t)gridDim.x * toks;
    for (int col = threadIdx.x - sub * 2 * blocks16; col < 2 * blocks16; col += blockDim.x) {
        const bool is_v = col >= blocks16;
        const int blk = is_v ? col - blocks16 : col;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(is_v ? a.v : a.k) + blk * FP4_BLOCK;
        const int64_t tok_stride = is_v ? a.v_tok_stride : a.k_tok_stride;
        uint8_t *data = (is_v ? a.pool.v_data : a.pool.k_data) + blk * (FP4_BLOCK / 2);
        uint8_t *scale = (is_v ? a.pool.v_scale : a.pool.k_scale) + blk;
        const float unit = pow2i(-(is_v ? a.pool.v_exp : a.pool.k_exp));
        for (int64_t i = blockIdx.x * toks + sub; i < a.n_tokens; i += step) {
            uint32_t x[8], sb;
            uint2 c;
            ld_32<WIDE>(src + i * tok_stride, x);
            const int row = a.out_loc[i];
            quantise16(x, unit, c, sb);
            // out-of-range rows are a caller error; clamp so the write stays in the pool
            const uint32_t r = (uint32_t)min(max(row, 0), a.pool.num_rows - 1);
            *reinterpret_cast<uint2 *>(data + (uint64_t)r * (uint32_t)a.pool.data_stride) = c;
            scale[(uint64_t)r * (uint32_t)a.pool.scale_stride] = (uint8_t)sb;
        }
    }
}

// A block of the load kernel takes a run of tiles of tile_toks tokens, one
// thread per column of `toks` tokens at a time.  Its first tile_toks threads
// look up the pool rows of a tile before the block converts the one before
// it: the request of a run's first tokens by binary search, the later ones by
// walking on.
template <bool WIDE>
__global__ void __launch_bounds__(MAX_THREADS, LOAD_RESIDENT / MAX_THREADS)
    load_kv_fp4_kernel(LoadFp4Args a, int blocks16, int toks, int tile_toks) {
    __shared__ int s_row[2][LOAD_TOKENS];  // pool row of each token, or -1
    pdl_wait();  // no early start for the next kernel: store_kv may read the rows with non-coherent loads
    const int64_t tiles = ((int64_t)a.total_tokens + tile_toks - 1) / tile_toks;
    const int64_t first = blockIdx.x * tiles / gridDim.x, last = (blockIdx.x + 1) * tiles / gridDim.x;
    int req = -1;  // lane's request
    auto look_up = [&](int64_t tile, int *rows) {
        const int64_t t = tile * tile_toks + threadIdx.x;
        int row = -1;
        if (t < a.total_tokens) {
            if (req < 0) {
                int lo = 0, hi = a.batch;  // the last request with offsets[r] <= t
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (a.offsets[mid] <= t) lo = mid; else hi = mid;
                }
                req = lo;
            }
            int end = a.offsets[req + 1];
            while (req + 1 < a.batch && end <= t) end = a.offsets[++req + 1];
            const int64_t j = t - a.offsets[req];
            const int n = min(max(a.lens[req], 0), a.pt_width);
            if (j >= 0 && j < n && t < end)
                row = min(max(a.page_table[req * a.pt_stride + j], 0), a.pool.num_rows - 1);
        }
        rows[threadIdx.x] = row;
    };
    const int sub = threadIdx.x / (2 * blocks16);
    if ((int)threadIdx.x < tile_toks && first < last) look_up(first, s_row[0]);
    for (int64_t tile = first; tile < last; ++tile) {
        const int *rows = s_row[(tile - first) & 1];
        __syncthreads();
        if ((int)threadIdx.x < tile_toks && tile + 1 < last) look_up(tile + 1, s_row[(tile + 1 - first) & 1]);
        if (sub >= toks) continue;
        for (int col = threadIdx.x - sub * 2 * blocks16; col < 2 * blocks16; col += blockDim.x) {
            const bool is_v = col >= blocks16;
            const int blk = is_v ? col - blocks16 : col;
            const uint8_t *data = (is_v ? a.pool.v_data : a.pool.k_data) + blk * (FP4_BLOCK / 2);
            const uint8_t *scale = (is_v ? a.pool.v_scale : a.pool.k_scale) + blk;
            const float unit = pow2i(is_v ? a.pool.v_exp : a.pool.k_exp);
            const int64_t tok_stride = is_v ? a.v_tok_stride : a.k_tok_stride;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_v ? a.v_out : a.k_out) +
                                 tile * tile_toks * tok_stride + blk * FP4_BLOCK;
            for (int i0 = sub; i0 < tile_toks; i0 += LOAD_U * toks) {
                uint2 c[LOAD_U];
                uint32_t sb[LOAD_U];
                int row[LOAD_U];
#pragma unroll
                for (int u = 0; u < LOAD_U; ++u) {
                    const int i = i0 + u * toks;
                    row[u] = i < tile_toks ? rows[i] : -1;
                    if (row[u] >= 0) {
                        const uint32_t r = (uint32_t)row[u];
                        c[u] = *reinterpret_cast<const uint2 *>(data + (uint64_t)r * (uint32_t)a.pool.data_stride);
                        sb[u] = scale[(uint64_t)r * (uint32_t)a.pool.scale_stride];
                    }
                }
#pragma unroll
                for (int u = 0; u < LOAD_U; ++u) {
                    if (row[u] < 0) continue;
                    const uint32_t s = e4m3x2_to_f16x2(sb[u] | (sb[u] << 8));
                    uint32_t h[2][4], o[8];
                    e2m1x8_to_f16x2(c[u].x, h[0]);
                    e2m1x8_to_f16x2(c[u].y, h[1]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 f = f16x2_to_f32(mul_f16x2(h[j >> 2][j & 3], s));
                        o[j] = pack_bf16x2(f.x * unit, f.y * unit);
                    }
                    st_32<WIDE>(dst + (i0 + u * toks) * tok_stride, o);
                }
            }
        }
    }
}

namespace {

// Threads per block and tokens per block-wide step for this many columns.
void block_shape(int columns, int &threads, int &toks) {
    toks = columns < 256 ? 256 / columns : 1;
    threads = (int)std::min<int64_t>(((int64_t)toks * columns + 31) / 32 * 32, MAX_THREADS);
}

bool aligned32(const void *p, int64_t tok_stride) {
    return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && tok_stride % 16 == 0;
}

}  // namespace

cudaError_t launch_store_kv_fp4(const StoreFp4Args &a, cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    const int blocks16 = a.pool.num_kv_heads * a.pool.head_dim / FP4_BLOCK;
    int threads, toks;
    block_shape(2 * blocks16, threads, toks);
    int64_t blocks = ((int64_t)a.n_tokens + toks - 1) / toks;
    const int64_t cap = (int64_t)device_sm_count() * (STORE_RESIDENT / threads);
    if (blocks > cap) blocks = cap;
    const bool wide = aligned32(a.k, a.k_tok_stride) && aligned32(a.v, a.v_tok_stride);
    return launch_pdl(wide ? store_kv_fp4_kernel<true> : store_kv_fp4_kernel<false>, dim3((unsigned)blocks),
                      dim3(threads), 0, s, a, blocks16, toks);
}

cudaError_t launch_load_kv_fp4(const LoadFp4Args &a, cudaStream_t s) {
    if (a.batch == 0 || a.total_tokens == 0) return cudaSuccess;
    const int blocks16 = a.pool.num_kv_heads * a.pool.head_dim / FP4_BLOCK;
    int threads, toks;
    block_shape(2 * blocks16, threads, toks);
    // tiles as large as still give every resident block one; at least a step of the block
    const int64_t cap = (int64_t)device_sm_count() * (LOAD_RESIDENT / threads);
    const int tile = (int)std::min<int64_t>(LOAD_TOKENS, std::max<int64_t>(toks, (a.total_tokens + cap - 1) / cap));
    const int64_t blocks = std::min(cap, ((int64_t)a.total_tokens + tile - 1) / tile);
    const bool wide = aligned32(a.k_out, a.k_tok_stride) && aligned32(a.v_out, a.v_tok_stride);
    return launch_pdl(wide ? load_kv_fp4_kernel<true> : load_kv_fp4_kernel<false>, dim3((unsigned)blocks),
                      dim3(threads), 0, s, a, blocks16, toks, tile);
}

}  // namespace minisgl

// load_kv_fp8.cu -- cached rows of the 8-bit pool as packed bf16 rows:
//     out[offsets[r] + j] = c * 2^e of row page_table[r, j],  j < lens[r],
// exact in bf16: an element has 4 significant bits, and the smallest one, 2^-9,
// times the smallest scale that a store gives, 2^-120, is above bf16's 2^-133.
//
// Bound by HBM: 16 bytes in and 32 out for 16 channels, so writes are two
// thirds of it.  A thread keeps one column (K or V, and 16 channels) for all
// its tokens and asks for its next pieces before it converts those it has; a
// block looks up the pool rows of a tile of tokens while it converts the one
// before.  328k tokens of 8 heads of 128: 326 us, 6.2 TB/s (a copy of as many bytes
// runs at 6.9); 31k tokens 33.4 us (5.6).  With a run of tiles to each block 328 and
// 35.2, without asking ahead 331 and 35.4; half the threads with 8 pieces in
// flight 322 and 34.4, but 60 instead of 44 us for 41k tokens in 40 requests.
#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int MAX_THREADS = 512;
constexpr int RESIDENT = 1024;   // threads per SM
constexpr int IN_FLIGHT = 4;     // pieces of 16 channels that a thread has under way
constexpr int MOST_TOKENS = 128; // of a tile

__device__ __forceinline__ uint4 ld_v4(const void *p) {  // coherent, as in the store
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// 32 bytes to 32-byte (WIDE) or 16-byte aligned memory
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

}  // namespace

// A block takes every gridDim.x-th tile of tile_toks tokens (so that the blocks
// together write one place at a time), one thread per column of `toks` tokens at a
// time (with more columns than threads it goes over them in steps).
template <bool WIDE>
__global__ void __launch_bounds__(MAX_THREADS, RESIDENT / MAX_THREADS)
    load_kv_fp8_kernel(const LoadFp8Args a, int pieces, int toks, int tile_toks) {
    __shared__ int s_row[2][MOST_TOKENS];  // pool row of each token, or -1
    pdl_wait();  // no early start for the next kernel: store_kv may read the rows with non-coherent loads
    const int64_t tiles = ((int64_t)a.total_tokens + tile_toks - 1) / tile_toks;
    auto look_up = [&](int64_t tile, int *rows) {
        const int64_t t = tile * tile_toks + threadIdx.x;
        int row = -1;
        if (t < a.total_tokens) {
            int req = 0, hi = a.batch;  // the last request with offsets[r] <= t
            while (hi - req > 1) {
                const int mid = (req + hi) >> 1;
                if (a.offsets[mid] <= t) req = mid; else hi = mid;
            }
            const int64_t j = t - a.offsets[req];
            const int n = min(max(a.lens[req], 0), a.pt_width);
            if (j >= 0 && j < n && t < a.offsets[req + 1])
                row = min(max(a.page_table[req * a.pt_stride + j], 0), a.pool.num_rows - 1);
        }
        rows[threadIdx.x] = row;
    };
    const int per_head = a.pool.head_dim / 16;
    const int sub = threadIdx.x / (2 * pieces);
    if ((int)threadIdx.x < tile_toks && blockIdx.x < tiles) look_up(blockIdx.x, s_row[0]);
    int at = 0;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, at ^= 1) {
        const int *rows = s_row[at];
        __syncthreads();
        if ((int)threadIdx.x < tile_toks && tile + gridDim.x < tiles) look_up(tile + gridDim.x, s_row[at ^ 1]);
        if (sub >= toks) continue;
        for (int col = threadIdx.x - sub * 2 * pieces; col < 2 * pieces; col += blockDim.x) {
            const bool is_v = col >= pieces;
            const int piece = is_v ? col - pieces : col;
            const uint8_t *data = (is_v ? a.pool.v_data : a.pool.k_data) + piece * 16;
            const uint8_t *scale = (is_v ? a.pool.v_scale : a.pool.k_scale) + piece / per_head;
            const int64_t tok_stride = is_v ? a.v_tok_stride : a.k_tok_stride;
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(is_v ? a.v_out : a.k_out) +
                                 tile * tile_toks * tok_stride + piece * 16;
            // the next pieces are asked for before these are converted and stored
            uint4 c[IN_FLIGHT], next[IN_FLIGHT];
            uint32_t e[IN_FLIGHT], next_e[IN_FLIGHT];
            auto ask = [&](int i0, uint4 (&x)[IN_FLIGHT], uint32_t (&scale_of)[IN_FLIGHT]) {
#pragma unroll
                for (int u = 0; u < IN_FLIGHT; ++u) {
                    const int i = i0 + u * toks, row = i < tile_toks ? rows[i] : -1;
                    scale_of[u] = ~0u;  // none
                    if (row >= 0) {
                        const uint32_t r = (uint32_t)row;
                        x[u] = ld_v4(data + (uint64_t)r * (uint32_t)a.pool.data_stride);
                        scale_of[u] = scale[(uint64_t)(r >> a.pool.block_log2) * (uint32_t)a.pool.scale_stride];
                    }
                }
            };
            ask(sub, next, next_e);
            for (int i0 = sub; i0 < tile_toks; i0 += IN_FLIGHT * toks) {
#pragma unroll
                for (int u = 0; u < IN_FLIGHT; ++u) {
                    c[u] = next[u];
                    e[u] = next_e[u];
                }
                if (i0 + IN_FLIGHT * toks < tile_toks) ask(i0 + IN_FLIGHT * toks, next, next_e);
#pragma unroll
                for (int u = 0; u < IN_FLIGHT; ++u) {
                    if (e[u] == ~0u) continue;
                    const float unit = __uint_as_float(e[u] << 23);
                    const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
                    uint32_t o[8];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        uint32_t lo, hi;
                        fp8::e4m3x4_to_f16x2(w[j], lo, hi);
                        const float2 f = f16x2_to_f32(lo), g = f16x2_to_f32(hi);
                        o[2 * j] = pack_bf16x2(f.x * unit, f.y * unit);
                        o[2 * j + 1] = pack_bf16x2(g.x * unit, g.y * unit);
                    }
                    st_32<WIDE>(dst + (i0 + u * toks) * tok_stride, o);
                }
            }
        }
    }
}

cudaError_t launch_load_kv_fp8(const LoadFp8Args &a, cudaStream_t s) {
    if (a.batch == 0 || a.total_tokens == 0) return cudaSuccess;
    const int pieces = a.pool.num_kv_heads * a.pool.head_dim / 16, columns = 2 * pieces;
    const int toks = columns < 256 ? 256 / columns : 1;
    const int threads = (int)std::min<int64_t>(((int64_t)toks * columns + 31) / 32 * 32, MAX_THREADS);
    // Tiles of 32 tokens, or of a block's step with all pieces in flight; smaller ones
    // if that leaves resident blocks without one, but at least a step of the block.
    const int64_t cap = (int64_t)device_sm_count() * (RESIDENT / threads);
    const int most = std::max(32, toks * IN_FLIGHT);  // up to MOST_TOKENS: toks is up to 32
    const int tile = (int)std::min<int64_t>(most, std::max<int64_t>(toks, (a.total_tokens + cap - 1) / cap));
    const int64_t blocks = std::min(cap, ((int64_t)a.total_tokens + tile - 1) / tile);
    auto wide = [](const void *p, int64_t tok_stride) {
        return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && tok_stride % 16 == 0;
    };
    return launch_pdl(wide(a.k_out, a.k_tok_stride) && wide(a.v_out, a.v_tok_stride) ? load_kv_fp8_kernel<true>
                                                                                     : load_kv_fp8_kernel<false>,
                      dim3((unsigned)blocks), dim3(threads), 0, s, a, pieces, toks, tile);
}

}  // namespace minisgl

// store_kv_fp8.cu -- new K/V rows into the 8-bit pool, rotated on the way or
// as they are, and q rotated beside them.
//
// For token i with row r = out_loc[i] in block b = r / B (B rows a block):
//     y = R(positions[i]) k[i]   (fp32; the first rotary_dim channels in pairs)
//     e(b, h) = smallest e with |y| <= 448 * 2^e over the new rows of b, and at
//               least the e that b had, if the new rows begin inside the block
//     element = e4m3(y * 2^-e),  the block's older rows: e4m3(c * 2^(e_old - e))
// and the same for v without a rotation.  Multiplying by a power of two is
// exact, so an element is rounded once.  Rows are bf16 or their fp32 rotation;
// an infinity becomes NaN (e4m3 has none), and neither counts for e.
//
// Work: the new rows of one block are consecutive in out_loc and in the pool
// (a run).  A warp takes one run and one column (a K head or a V head): d/16
// lanes hold a token's head, each 16 channels as 8 pairs, so that a rotation,
// the block's maximum (one reduction over the warp) and the quantisation all
// happen in registers.  Runs are found by the warps themselves: a warp looks
// at the rows of a window of tokens and takes the runs that begin in it.
// With single-row blocks d/16 lanes take a head's row by themselves.
#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;

// Coherent loads: the kernel is resident while the one before it may still
// write what is read here.
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A lane's 16 channels of a head: chunks of 8 at a and b.
struct Chunks {
    int a, b;
    bool turned;  // the chunks are the lane's 8 pairs
};

// Lane t of the d/16 lanes of a row: with half-split pairs its 8 pairs are
// channels 8t.. and rotary/2 + 8t.., else 16 neighbours.
__device__ __forceinline__ Chunks chunks_of(int t, int rotary, bool interleaved) {
    Chunks c;
    c.turned = t < rotary / 16;
    const bool split = c.turned && !interleaved;
    c.a = split ? 8 * t : 16 * t;
    c.b = split ? rotary / 2 + 8 * t : 16 * t + 8;
    return c;
}

__device__ __forceinline__ void widen(const uint4 &a, const uint4 &b, float (&x)[16]) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// The lane's 8 pairs turned: (x[e], x[8 + e]), or (x[2e], x[2e + 1]).
// row: the table's row of the token's position, [cos | sin].
__device__ __forceinline__ void turn(float (&x)[16], const float *row, int t, int rotary, bool interleaved) {
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 u = *reinterpret_cast<const float4 *>(row + 8 * t + 4 * i);
        const float4 v = *reinterpret_cast<const float4 *>(row + rotary / 2 + 8 * t + 4 * i);
        c[4 * i] = u.x, c[4 * i + 1] = u.y, c[4 * i + 2] = u.z, c[4 * i + 3] = u.w;
        s[4 * i] = v.x, s[4 * i + 1] = v.y, s[4 * i + 2] = v.z, s[4 * i + 3] = v.w;
    }
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = fmaf(p, c[e], -q * s[e]);
            x[2 * e + 1] = fmaf(q, c[e], p * s[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p = x[e], q = x[8 + e];
            x[e] = fmaf(p, c[e], -q * s[e]);
            x[8 + e] = fmaf(q, c[e], p * s[e]);
        }
    }
}

__device__ __forceinline__ const float *table_row(const StoreFp8Args &a, int64_t i) {
    const int p = min(max(a.positions[i], 0), a.max_positions - 1);  // outside: a caller error
    return a.cos_sin + (int64_t)p * a.rotary_dim;
}

__device__ __forceinline__ int pool_row(const StoreFp8Args &a, int64_t i) {
    return min(max(a.out_loc[i], 0), a.pool.num_rows - 1);  // likewise
}

// The largest |x| as bits (NaN does not count, infinity does).
__device__ __forceinline__ uint32_t top_of(const float (&x)[16]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(x[j]));
    return __float_as_uint(m);
}

// infinities to NaN, the rest as it is
__device__ __forceinline__ void no_infinity(float (&x)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = fmaf(x[j], 0.f, x[j]);
}

__device__ __forceinline__ void put(uint8_t *dst, const Chunks &c, const float (&x)[16], float unit) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = fp8::f32_to_e4m3x4(x[4 * i] * unit, x[4 * i + 1] * unit, x[4 * i + 2] * unit, x[4 * i + 3] * unit);
    if (c.b == c.a + 8) {
        st_v4(dst + c.a, make_uint4(w[0], w[1], w[2], w[3]));
    } else {
        *reinterpret_cast<uint2 *>(dst + c.a) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(dst + c.b) = make_uint2(w[2], w[3]);
    }
}

// q rows turned into q_out: d/16 lanes a row, block `b` of `blocks`.
template <int D>
__device__ __forceinline__ void turn_queries(const StoreFp8Args &a, int b, int blocks) {
    constexpr int TPR = D / 16;
    const int t = threadIdx.x % TPR;
    const Chunks ch = chunks_of(t, a.rotary_dim, a.interleaved);
    const bool in_place = a.q_out == a.q;
    const uint32_t rows = (uint32_t)a.n_tokens * a.num_q_heads;
    for (uint32_t at = b * (THREADS / TPR) + threadIdx.x / TPR; at < rows; at += blocks * (THREADS / TPR)) {
        const uint32_t i = at / a.num_q_heads, h = at - i * a.num_q_heads;
        const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) + i * a.q_tok_stride + h * D;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.q_out) + i * a.q_out_tok_stride + h * D;
        if (in_place && !ch.turned) continue;
        uint4 va = ld_v4(src + ch.a), vb = ld_v4(src + ch.b);
        if (ch.turned) {
            float x[16];
            widen(va, vb, x);
            turn(x, table_row(a, i), t, a.rotary_dim, a.interleaved);
            va = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                            pack_bf16x2(x[6], x[7]));
            vb = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                            pack_bf16x2(x[14], x[15]));
        }
        st_v4(dst + ch.a, va);
        st_v4(dst + ch.b, vb);
    }
}

// One column of the pool: a K head or a V head.
struct Column {
    const __nv_bfloat16 *src;  // of token 0
    int64_t tok_stride;
    uint8_t *data, *scale;     // of row 0, block 0
    bool is_k;
};

__device__ __forceinline__ Column column(const StoreFp8Args &a, int col, int d) {
    Column c;
    c.is_k = col < a.pool.num_kv_heads;
    const int h = c.is_k ? col : col - a.pool.num_kv_heads;
    c.src = static_cast<const __nv_bfloat16 *>(c.is_k ? a.k : a.v) + h * d;
    c.tok_stride = c.is_k ? a.k_tok_stride : a.v_tok_stride;
    c.data = (c.is_k ? a.pool.k_data : a.pool.v_data) + h * d;
    c.scale = (c.is_k ? a.pool.k_scale : a.pool.v_scale) + h;
    return c;
}

// Tokens i0 .. i0 + len - 1 into rows row0 .. of their block, `off` rows of
// which are older, by one warp.
template <int D>
__device__ __forceinline__ void store_run(const StoreFp8Args &a, const Column &col, int64_t i0, int row0, int off,
                                          int len, int lane) {
    constexpr int TPR = D / 16, RPW = 32 / TPR;  // lanes per row, rows per warp
    constexpr int C = 16 / RPW;                  // rows that a lane holds at a time
    const int t = lane % TPR, g = lane / TPR;
    const Chunks ch = chunks_of(t, col.is_k ? a.rotary_dim : 0, a.interleaved);
    const int passes = (len + C * RPW - 1) / (C * RPW);
    uint8_t *scale = col.scale + (int64_t)(row0 >> a.pool.block_log2) * a.pool.scale_stride;
    const int before = off > 0 ? (int)*scale - fp8::EXP_BIAS : fp8::EXP_LOW;
    float x[C][16];
    bool clean = false;
    auto load = [&](int p) {
        uint4 va[C], vb[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int l = (p * C + c) * RPW + g;
            va[c] = vb[c] = make_uint4(0u, 0u, 0u, 0u);
            if (l < len) {
                const __nv_bfloat16 *src = col.src + (i0 + l) * col.tok_stride;
                va[c] = ld_v4(src + ch.a);
                vb[c] = ld_v4(src + ch.b);
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int l = (p * C + c) * RPW + g;
            widen(va[c], vb[c], x[c]);
            if (ch.turned && l < len) turn(x[c], table_row(a, i0 + l), t, a.rotary_dim, a.interleaved);
            if (clean) no_infinity(x[c]);
        }
    };
    uint32_t top;
    for (;;) {
        top = 0;
        for (int p = 0; p < passes; ++p) {
            load(p);
#pragma unroll
            for (int c = 0; c < C; ++c) top = max(top, top_of(x[c]));
        }
        top = __reduce_max_sync(0xffffffffu, top);
        if (top < 0x7f800000u) break;
        clean = true;  // once more without the infinities
    }
    const int need = fp8::exponent_for(top), e = max(need, before);
    if (lane == 0 && (off == 0 || e != before)) *scale = (uint8_t)(e + fp8::EXP_BIAS);
    if (off > 0 && e > before) {  // the older rows under the new scale
        const float down = pow2i(max(before - e, -126));
        for (int r = g; r < off; r += RPW) {
            uint4 *p = reinterpret_cast<uint4 *>(col.data + (int64_t)(row0 - off + r) * a.pool.data_stride) + t;
            uint4 v = ld_v4(p);
            uint32_t *w = &v.x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t lo, hi;
                fp8::e4m3x4_to_f16x2(w[i], lo, hi);
                const float2 f = f16x2_to_f32(lo), s = f16x2_to_f32(hi);
                w[i] = fp8::f32_to_e4m3x4(f.x * down, f.y * down, s.x * down, s.y * down);
            }
            st_v4(p, v);
        }
    }
    const float unit = pow2i(-e);
    for (int p = passes - 1; p >= 0; --p) {
        if (p < passes - 1) load(p);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int l = (p * C + c) * RPW + g;
            if (l < len) put(col.data + (int64_t)(row0 + l) * a.pool.data_stride, ch, x[c], unit);
        }
    }
}

}  // namespace

// Blocks of several rows.  Unit u of the K/V part: window u / columns (of
// 2^win_log2 <= 16 tokens), column u % columns.  Blocks from kv_blocks on turn q.
template <int D>
__global__ void __launch_bounds__(THREADS) store_kv_fp8_kernel(const StoreFp8Args a, int win_log2, int kv_blocks) {
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x >= kv_blocks) {
        turn_queries<D>(a, blockIdx.x - kv_blocks, gridDim.x - kv_blocks);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int n = a.n_tokens, in_block = (1 << a.pool.block_log2) - 1;
    const uint32_t columns = 2 * a.pool.num_kv_heads;
    const uint32_t units = (uint32_t)((n + (1 << win_log2) - 1) >> win_log2) * columns;
    for (uint32_t u = blockIdx.x * WARPS + (threadIdx.x >> 5); u < units; u += kv_blocks * WARPS) {
        const uint32_t win = u / columns;
        const Column col = column(a, (int)(u - win * columns), D);
        const int t0 = (int)win << win_log2;
        // where runs begin among tokens t0 .. t0 + 31: at a block's first row, behind
        // a row that is not the one before, and past the last token
        const int r = t0 + lane < n ? pool_row(a, t0 + lane) : -2;
        int prev = t0 > 0 ? pool_row(a, t0 - 1) : -2;
        const int up = __shfl_up_sync(0xffffffffu, r, 1);
        if (lane > 0) prev = up;
        const uint32_t starts = __ballot_sync(0xffffffffu, r < 0 || r != prev + 1 || (r & in_block) == 0);
        const uint32_t mine = __ballot_sync(0xffffffffu, r >= 0 && lane < (1 << win_log2));
        for (uint32_t todo = starts & mine; todo; todo &= todo - 1) {
            const int s = __ffs(todo) - 1;
            const int row0 = __shfl_sync(0xffffffffu, r, s), off = row0 & in_block;
            const uint32_t later = starts & ~((2u << s) - 1u);
            int len = later ? __ffs(later) - 1 - s : 32 - s;
            while (!later && len <= in_block - off) {  // rows past the 32 looked at
                const int next = t0 + s + len + lane;
                const int q = next < n ? pool_row(a, next) : -2;
                const uint32_t other = __ballot_sync(0xffffffffu, q != row0 + len + lane || off + len + lane > in_block);
                if (other) {
                    len += __ffs(other) - 1;
                    break;
                }
                len += 32;
            }
            store_run<D>(a, col, t0 + s, row0, off, len, lane);
        }
    }
}

// Blocks of one row: d/16 lanes a head's row.
template <int D>
__global__ void __launch_bounds__(THREADS) store_rows_fp8_kernel(const StoreFp8Args a, int kv_blocks) {
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x >= kv_blocks) {
        turn_queries<D>(a, blockIdx.x - kv_blocks, gridDim.x - kv_blocks);
        return;
    }
    constexpr int TPR = D / 16;
    const int t = threadIdx.x % TPR;
    const uint32_t columns = 2 * a.pool.num_kv_heads, rows = (uint32_t)a.n_tokens * columns;
    const uint32_t group = 0xffffffffu >> (32 - TPR) << (threadIdx.x % 32 / TPR * TPR);
    for (uint32_t at = blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR; at < rows; at += kv_blocks * (THREADS / TPR)) {
        const uint32_t i = at / columns;
        const Column col = column(a, (int)(at - i * columns), D);
        const Chunks ch = chunks_of(t, col.is_k ? a.rotary_dim : 0, a.interleaved);
        const __nv_bfloat16 *src = col.src + i * col.tok_stride;
        const uint4 va = ld_v4(src + ch.a), vb = ld_v4(src + ch.b);
        const int row = pool_row(a, i);
        float x[16];
        widen(va, vb, x);
        if (ch.turned) turn(x, table_row(a, i), t, a.rotary_dim, a.interleaved);
        uint32_t top = top_of(x);
#pragma unroll
        for (int o = TPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
        if (top >= 0x7f800000u) {
            no_infinity(x);
            top = top_of(x);
#pragma unroll
            for (int o = TPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(group, top, o));
        }
        const int e = fp8::exponent_for(top);
        if (t == 0) col.scale[(int64_t)row * a.pool.scale_stride] = (uint8_t)(e + fp8::EXP_BIAS);
        put(col.data + (int64_t)row * a.pool.data_stride, ch, x, pow2i(-e));
    }
}

namespace {

template <int D>
cudaError_t launch_as(const StoreFp8Args &a, cudaStream_t s) {
    constexpr int64_t ROWS = THREADS / (D / 16);  // rows that a block takes at a time
    const int64_t sms = device_sm_count(), n = a.n_tokens, columns = 2 * a.pool.num_kv_heads;
    const int64_t q_rows = n * a.num_q_heads;
    const int64_t q_blocks = std::min((q_rows + ROWS - 1) / ROWS, sms * 8);
    if (a.pool.block_log2 == 0) {
        const int64_t kv = std::min((n * columns + ROWS - 1) / ROWS, sms * 8);
        return launch_pdl(store_rows_fp8_kernel<D>, dim3((unsigned)(kv + q_blocks)), dim3(THREADS), 0, s, a, (int)kv);
    }
    // windows as wide as still give every resident warp one
    int win = 0;
    while (win < 4 && (n >> (win + 1)) * columns >= sms * 16) ++win;
    const int64_t units = ((n + (1 << win) - 1) >> win) * columns;
    const int64_t kv = std::min((units + WARPS - 1) / WARPS, sms * 8);
    return launch_pdl(store_kv_fp8_kernel<D>, dim3((unsigned)(kv + q_blocks)), dim3(THREADS), 0, s, a, win, (int)kv);
}

}  // namespace

cudaError_t launch_store_kv_fp8(const StoreFp8Args &a, cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    return a.pool.head_dim == 128 ? launch_as<128>(a, s) : launch_as<64>(a, s);
}

}  // namespace minisgl

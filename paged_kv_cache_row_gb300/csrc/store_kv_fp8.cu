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
// Work: a token's head is d/16 lanes, each with 16 channels as 8 pairs, so that
// the rotation happens in registers.  The new rows of one block are consecutive
// in out_loc and in the pool (a run).  One to four warps (a group) take a run
// and one column (a K head or a V head) and hold all of it: one reduction gives
// the block's maximum, and every row is read once.  Runs are found by the
// groups themselves: a group looks at the rows of a window of tokens and takes
// the runs that begin in it.  Rows that need no common maximum (q, and blocks of
// one row) are taken by tokens: d/16 lanes a token and four of its heads, whose
// loads are under way together and share the token's cos and sin.
//
// What bounds it: HBM, if enough loads are under way.  So a lane has 128 bytes
// asked for: four of its token's heads, or its rows of the next head (in shared
// memory, by cp.async) while it works on one.  Rotated K is then bound by issue
// slots as much: its 64 values a lane stay in registers until the maximum is
// known, which leaves 16 warps an SM.
//
// Measured (device time, in a graph): 133k tokens, 15 query and 5 KV heads of 64,
// blocks of 64, half of the head rotated, 147 us (5.3 TB/s; K and V without a
// rotation 46, 5.5 TB/s, rotated 69); 8.2k tokens, 32 and 8 heads of 128, blocks of
// 16, 34.1 us (5.6 TB/s); K and V of 41k tokens, 8 heads of 128, blocks of one row,
// 41 us (6.2 TB/s).  Steps on the first: 189 (a warp per run, read twice for the
// maximum) - 176 (groups of warps, q by four heads a token) - 166 (fetched a run
// ahead) - 151 (windows of a block's rows, where windows of 32 tokens left half the
// groups with twice the work; the next head of the same run instead of the next
// run) - 147 (half of the blocks begin with q).  Not kept: the rotation in packed
// pairs of fp32 (157, and 44 instead of 41 on the third); the table's rows asked
// for ahead (152); cos and sin kept for all heads of a run and K rotated twice
// instead, for the maximum and again (146 where 151 were taken, but 38 instead of
// 36.4 on the second).
#include <algorithm>

#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int THREADS = 128;
constexpr int WARPS = THREADS / 32;
constexpr int RESIDENT = 4;       // blocks per SM: 128 registers a thread
constexpr int ROWS_RESIDENT = 5;  // of single-row blocks: 96
constexpr int HEADS = 4;          // heads of a token that a lane has under way

// Coherent loads: the kernel is resident while the one before it may still
// write what is read here.
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// A lane's 16 channels of a head: chunks of 8 at a and b.  The lanes' chunks a
// lie side by side, and so do their chunks b, so that an instruction takes whole
// sectors: the rotated channels (half each) and the others (half each).
struct Chunks {
    int a, b, t;  // t: number among the lanes that rotate
    bool turned;
};
template <int D>
__device__ __forceinline__ Chunks chunks_of(int t, int rotary) {
    Chunks c;
    c.turned = t < rotary / 16;
    c.t = c.turned ? t : t - rotary / 16;
    c.a = (c.turned ? 0 : rotary) + 8 * c.t;
    c.b = c.a + (c.turned ? rotary : D - rotary) / 2;
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

// cos and sin of the lane's 8 pairs, from the table's row [cos | sin] of a
// position: half-split, the pairs are (a + e, b + e); interleaved, chunk a has
// four pairs of neighbours and chunk b four.
struct Angles {
    float c[8], s[8];
};
__device__ __forceinline__ void load_angles(Angles &w, const float *row, int t, int rotary, bool interleaved) {
    const int first = interleaved ? 4 * t : 8 * t, second = interleaved ? rotary / 4 + 4 * t : 8 * t + 4;
    const float4 u0 = *reinterpret_cast<const float4 *>(row + first);
    const float4 u1 = *reinterpret_cast<const float4 *>(row + second);
    const float4 v0 = *reinterpret_cast<const float4 *>(row + rotary / 2 + first);
    const float4 v1 = *reinterpret_cast<const float4 *>(row + rotary / 2 + second);
    w.c[0] = u0.x, w.c[1] = u0.y, w.c[2] = u0.z, w.c[3] = u0.w;
    w.c[4] = u1.x, w.c[5] = u1.y, w.c[6] = u1.z, w.c[7] = u1.w;
    w.s[0] = v0.x, w.s[1] = v0.y, w.s[2] = v0.z, w.s[3] = v0.w;
    w.s[4] = v1.x, w.s[5] = v1.y, w.s[6] = v1.z, w.s[7] = v1.w;
}

// The lane's 8 pairs turned: (x[e], x[8 + e]), or (x[2e], x[2e + 1]).
__device__ __forceinline__ void turn(float (&x)[16], const Angles &w, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p = x[2 * e], q = x[2 * e + 1];
            x[2 * e] = fmaf(p, w.c[e], -q * w.s[e]);
            x[2 * e + 1] = fmaf(q, w.c[e], p * w.s[e]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p = x[e], q = x[8 + e];
            x[e] = fmaf(p, w.c[e], -q * w.s[e]);
            x[8 + e] = fmaf(q, w.c[e], p * w.s[e]);
        }
    }
}

__device__ __forceinline__ const float *table_row(const StoreFp8Args &a, int position) {
    const int p = min(max(position, 0), a.max_positions - 1);  // outside: a caller error
    return a.cos_sin + (int64_t)p * a.rotary_dim;
}

__device__ __forceinline__ int pool_row(const StoreFp8Args &a, int64_t i) {
    return min(max(a.out_loc[i], 0), a.pool.num_rows - 1);  // likewise
}

// The largest |x| as bits (NaN does not count, infinity does).
__device__ __forceinline__ float max_of(float m, float a, float b) {
    asm("{\n .reg .f32 x, y;\n abs.f32 x, %1;\n abs.f32 y, %2;\n max.f32 %0, %0, x, y;\n}\n" : "+f"(m) : "f"(a), "f"(b));
    return m;
}
__device__ __forceinline__ uint32_t top_of(const float (&x)[16]) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 2) m = max_of(m, x[j], x[j + 1]);
    return __float_as_uint(m);
}
// The same over bf16 pairs, in place (signs are left in it).
__device__ __forceinline__ void top_of_pairs(uint32_t &m, const uint32_t (&w)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("max.xorsign.abs.bf16x2 %0, %0, %1;\n" : "+r"(m) : "r"(w[j]));
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t c;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(c) : "r"(a), "r"(b));
    return c;
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
    *reinterpret_cast<uint2 *>(dst + c.a) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2 *>(dst + c.b) = make_uint2(w[2], w[3]);
}

// The rows of four heads of each of a warp's tokens, unit u: tokens
// u / chunks * RPW .. and heads u % chunks * 4 ..  KIND: q to q_out, or K or V
// into single-row blocks of the pool.
enum Kind { QUERY, KEY, VALUE };
template <int D, Kind KIND>
__device__ __forceinline__ void by_token(const StoreFp8Args &a, uint32_t u, int chunks, int lane) {
    constexpr int TPR = D / 16, RPW = 32 / TPR;
    const int t = lane % TPR;
    const uint32_t tile = u / chunks, h0 = (u - tile * chunks) * HEADS;
    const int64_t i = (int64_t)tile * RPW + lane / TPR;
    if (i >= a.n_tokens) return;
    const Chunks ch = chunks_of<D>(t, KIND == VALUE ? 0 : a.rotary_dim);
    const bool in_place = KIND == QUERY && a.q_out == a.q;
    if (in_place && !ch.turned) return;
    const int heads = KIND == QUERY ? a.num_q_heads : a.pool.num_kv_heads;
    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(KIND == QUERY ? a.q : KIND == KEY ? a.k : a.v) +
                               i * (KIND == QUERY ? a.q_tok_stride : KIND == KEY ? a.k_tok_stride : a.v_tok_stride) +
                               h0 * D;
    const int position = ch.turned ? a.positions[i] : 0;
    const int row = KIND == QUERY ? 0 : pool_row(a, i);
    uint4 va[HEADS], vb[HEADS];
#pragma unroll
    for (int h = 0; h < HEADS; ++h)
        if ((int)h0 + h < heads) {
            va[h] = ld_v4(src + h * D + ch.a);
            vb[h] = ld_v4(src + h * D + ch.b);
        }
    Angles w;
    if (ch.turned) load_angles(w, table_row(a, position), ch.t, a.rotary_dim, a.interleaved);
    const uint32_t group = 0xffffffffu >> (32 - TPR) << (lane / TPR * TPR);
#pragma unroll
    for (int h = 0; h < HEADS; ++h) {
        if ((int)h0 + h >= heads) continue;
        float x[16];
        if constexpr (KIND == QUERY) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.q_out) + i * a.q_out_tok_stride + (h0 + h) * D;
            if (ch.turned) {
                widen(va[h], vb[h], x);
                turn(x, w, a.interleaved);
                va[h] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                                   pack_bf16x2(x[6], x[7]));
                vb[h] = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]),
                                   pack_bf16x2(x[14], x[15]));
            }
            st_v4(dst + ch.a, va[h]);
            st_v4(dst + ch.b, vb[h]);
        } else {
            widen(va[h], vb[h], x);
            if (ch.turned) turn(x, w, a.interleaved);
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
            uint8_t *data = (KIND == KEY ? a.pool.k_data : a.pool.v_data) + (int64_t)row * a.pool.data_stride;
            uint8_t *scale = (KIND == KEY ? a.pool.k_scale : a.pool.v_scale) + (int64_t)row * a.pool.scale_stride;
            if (t == 0) scale[h0 + h] = (uint8_t)(e + fp8::EXP_BIAS);
            put(data + (h0 + h) * D, ch, x, pow2i(-e));
        }
    }
}

// Units of by_token for this many heads.
__host__ __device__ inline int head_chunks(int heads) { return (heads + HEADS - 1) / HEADS; }

// Tokens i0 .. i0 + len - 1 into rows row0 .. of their block, `off` rows of which
// are older, and the head that is next.
struct Run {
    int i0, row0, off, len, head, last;
};

// The runs that begin in a group's windows, one after the other, each for a
// chunk of heads.  Unit u: window u / chunks (of 2^win_log2 <= 64 tokens) and
// heads u % chunks * heads ..
struct Runs {
    uint32_t u, step, units, chunks;
    uint64_t starts, todo;  // where runs begin among tokens t0 .. t0 + 63; those of the window that are left
    int win_log2, heads, h0, t0;
    int r[2];               // rows of tokens t0 + lane and t0 + 32 + lane, or -2
    int ahead[2], before;   // rows of the next window and of the token before it, asked for a unit ahead

    __device__ __forceinline__ void ask(const StoreFp8Args &a, int lane) {
        if (u >= units) return;
        const int t = (int)(u / chunks) << win_log2;
#pragma unroll
        for (int i = 0; i < 2; ++i) ahead[i] = t + 32 * i + lane < a.n_tokens ? pool_row(a, t + 32 * i + lane) : -2;
        before = t > 0 ? pool_row(a, t - 1) : -2;
    }
    __device__ __forceinline__ void init(const StoreFp8Args &a, int win, int heads_, uint32_t first, uint32_t step_,
                                         int lane) {
        win_log2 = win;
        heads = heads_;
        u = first;
        step = step_;
        chunks = (a.pool.num_kv_heads + heads - 1) / heads;
        units = (uint32_t)((a.n_tokens + (1 << win) - 1) >> win) * chunks;
        todo = 0;
        ask(a, lane);
    }
    __device__ __forceinline__ bool next(const StoreFp8Args &a, Run &run, int lane) {
        const int in_block = (1 << a.pool.block_log2) - 1;
        while (todo == 0) {
            if (u >= units) return false;
            const uint32_t win = u / chunks;
            h0 = (int)(u - win * chunks) * heads;
            t0 = (int)win << win_log2;
            int last = before;
            r[0] = ahead[0];
            r[1] = ahead[1];
            u += step;
            ask(a, lane);
            // a run begins at a block's first row, behind a row that is not the one
            // before, and (the last one's end) past the last token
            starts = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int up = __shfl_up_sync(0xffffffffu, r[i], 1), prev = lane > 0 ? up : last;
                last = __shfl_sync(0xffffffffu, r[i], 31);
                starts |= (uint64_t)__ballot_sync(0xffffffffu, r[i] < 0 || r[i] != prev + 1 || (r[i] & in_block) == 0)
                          << (32 * i);
            }
            const int count = min(1 << win_log2, a.n_tokens - t0);
            todo = starts & (~0ull >> (64 - count));
        }
        const int s = __ffsll(todo) - 1;
        todo &= todo - 1;
        run.head = h0;
        run.last = min(h0 + heads, a.pool.num_kv_heads) - 1;
        run.i0 = t0 + s;
        run.row0 = __shfl_sync(0xffffffffu, s < 32 ? r[0] : r[1], s & 31);
        run.off = run.row0 & in_block;
        const uint64_t later = starts & ~((2ull << s) - 1u);
        run.len = later ? __ffsll(later) - 1 - s : 64 - s;
        while (!later && run.len <= in_block - run.off) {  // rows past the 64 looked at
            const int i = run.i0 + run.len + lane;
            const int q = i < a.n_tokens ? pool_row(a, i) : -2;
            const uint32_t other =
                __ballot_sync(0xffffffffu, q != run.row0 + run.len + lane || run.off + run.len + lane > in_block);
            if (other) {
                run.len += __ffs(other) - 1;
                break;
            }
            run.len += 32;
        }
        return true;
    }
};

// K or V: the new rows and where they go.
struct Side {
    const __nv_bfloat16 *src;  // token 0
    int64_t tok_stride;
    uint8_t *data, *scale;     // row 0, block 0
};
__device__ __forceinline__ Side side_of(const StoreFp8Args &a, bool is_k) {
    Side x;
    x.src = static_cast<const __nv_bfloat16 *>(is_k ? a.k : a.v);
    x.tok_stride = is_k ? a.k_tok_stride : a.v_tok_stride;
    x.data = is_k ? a.pool.k_data : a.pool.v_data;
    x.scale = is_k ? a.pool.k_scale : a.pool.v_scale;
    return x;
}

// A group's share of the work on K or V: W warps, C rows to a lane; row l of a
// run is a lane's if l = g + c * W * RPW.  TURN: the rows are rotated (K), and
// stay in registers in fp32 until the maximum is known; else they stay in shared
// memory, and the maximum and the scaling (exact in bf16) take two at a time.
template <int D, int W, int C, bool TURN>
struct Group {
    static constexpr int TPR = D / 16, RPW = 32 / TPR;  // lanes per row, rows per warp
    int lane, part, group, t, g;
    Chunks ch;
    Side side;

    __device__ __forceinline__ Group(const StoreFp8Args &a, bool is_k) {
        side = side_of(a, is_k);
        lane = threadIdx.x & 31;
        const int warp = threadIdx.x >> 5;
        part = warp % W;
        group = warp / W;
        t = lane % TPR;
        g = part * RPW + lane / TPR;
        ch = chunks_of<D>(t, TURN ? a.rotary_dim : 0);
    }

    __device__ __forceinline__ uint8_t *scale_of(const StoreFp8Args &a, const Run &run) const {
        return side.scale + run.head + (run.row0 >> a.pool.block_log2) * a.pool.scale_stride;
    }

    // The lane's rows of a head on their way to its place in shared memory, and the
    // block's scale so far; with a run's first head the rows' positions.
    __device__ __forceinline__ void fetch(const StoreFp8Args &a, const Run &run, uint32_t to, bool first,
                                          int (&position)[C], int &before) const {
        before = run.off > 0 ? (int)*scale_of(a, run) : fp8::EXP_BIAS + fp8::EXP_LOW;
        const __nv_bfloat16 *src = side.src + run.head * D + run.i0 * side.tok_stride;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int l = g + c * W * RPW;
            const bool live = l < run.len;
            const __nv_bfloat16 *row = src + (live ? l : 0) * side.tok_stride;
            cp_async_16(to + (2 * c) * THREADS * 16, row + ch.a, live ? 16 : 0);
            cp_async_16(to + (2 * c + 1) * THREADS * 16, row + ch.b, live ? 16 : 0);
            if (TURN && first) position[c] = ch.turned && live ? a.positions[run.i0 + l] : 0;
        }
    }

    __device__ __forceinline__ uint32_t over_group(uint32_t top, uint32_t (&s_top)[2][W], int &round) const {
        top = __reduce_max_sync(0xffffffffu, top);
        if constexpr (W > 1) {
            uint32_t(&at)[W] = s_top[round & 1];  // two in turn: a warp may be a round ahead of another's reads
            ++round;
            if (lane == 0) at[part] = top;
            // named by constants: a block that names one by a register reserves all 16, and an SM has 64
            if (W == WARPS || group == 0) asm volatile("bar.sync 1, %0;\n" ::"n"(32 * W) : "memory");
            else asm volatile("bar.sync 2, %0;\n" ::"n"(32 * W) : "memory");
#pragma unroll
            for (int i = 0; i < W; ++i) top = max(top, at[i]);
        }
        return top;
    }

    // Row c of the lane as it was fetched.
    __device__ __forceinline__ void words(uint32_t from, int c, uint32_t (&va)[4], uint32_t (&vb)[4]) const {
        lds_words<4>(from + (2 * c) * THREADS * 16, va);
        lds_words<4>(from + (2 * c + 1) * THREADS * 16, vb);
    }

    __device__ __forceinline__ void store(const StoreFp8Args &a, const Run &run, uint32_t from, const int (&position)[C],
                                          int before, uint32_t (&s_top)[2][W], int &round) const {
        uint8_t *data = side.data + run.head * D + run.row0 * a.pool.data_stride;
        float x[TURN ? C : 1][16];
        uint32_t top = 0;
        if constexpr (TURN) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uint32_t va[4], vb[4];
                words(from, c, va, vb);
                widen(make_uint4(va[0], va[1], va[2], va[3]), make_uint4(vb[0], vb[1], vb[2], vb[3]), x[c]);
                if (ch.turned && g + c * W * RPW < run.len) {
                    Angles w;
                    load_angles(w, table_row(a, position[c]), ch.t, a.rotary_dim, a.interleaved);
                    turn(x[c], w, a.interleaved);
                }
                top = max(top, top_of(x[c]));
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                uint32_t va[4], vb[4];
                words(from, c, va, vb);
                top_of_pairs(top, va);
                top_of_pairs(top, vb);
            }
            top &= 0x7fff7fffu;
            top = max(top << 16, top & 0xffff0000u);
        }
        top = over_group(top, s_top, round);
        const bool infinite = top >= 0x7f800000u;
        if (infinite) {  // once more without the infinities
            top = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float (&y)[16] = x[TURN ? c : 0];
                if constexpr (!TURN) {
                    uint32_t va[4], vb[4];
                    words(from, c, va, vb);
                    widen(make_uint4(va[0], va[1], va[2], va[3]), make_uint4(vb[0], vb[1], vb[2], vb[3]), y);
                }
                no_infinity(y);
                top = max(top, top_of(y));
            }
            top = over_group(top, s_top, round);
        }
        before -= fp8::EXP_BIAS;
        const int e = max(fp8::exponent_for(top), before);
        if (part == 0 && lane == 0 && (run.off == 0 || e != before)) *scale_of(a, run) = (uint8_t)(e + fp8::EXP_BIAS);
        if (run.off > 0 && e > before) {  // the older rows under the new scale
            const float down = pow2i(max(before - e, -126));
            for (int r = g; r < run.off; r += W * RPW) {
                uint4 *p = reinterpret_cast<uint4 *>(data + (r - run.off) * a.pool.data_stride) + t;
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
        const uint32_t unit2 = (uint32_t)(fp8::EXP_BIAS - e) * 0x00800080u;  // 2^-e as two bf16
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int l = g + c * W * RPW;
            if (l >= run.len) continue;
            if constexpr (TURN) {
                put(data + l * a.pool.data_stride, ch, x[c], pow2i(-e));
            } else {  // an exact product in bf16: what it loses to underflow is far below half an element
                uint32_t v[8];
                words(from, c, *reinterpret_cast<uint32_t(*)[4]>(v), *reinterpret_cast<uint32_t(*)[4]>(v + 4));
                float y[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = mul_bf16x2(v[i], unit2);
                widen(make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7]), y);
                if (infinite) no_infinity(y);
                put(data + l * a.pool.data_stride, ch, y, 1.f);
            }
        }
    }
};

// K's or V's units from u on; a group fetches its next head of a run, or its
// next run, while it works on one.  place: the thread's in shared memory.
template <int D, int W, int C, bool TURN>
__device__ __forceinline__ void store_all(const StoreFp8Args &a, bool is_k, uint32_t &u, uint32_t step, int win_log2, int heads,
                                          uint32_t place, uint32_t (&s_top)[2][W], int &round) {
    constexpr uint32_t PLACE = 2 * C * THREADS * 16;
    const Group<D, W, C, TURN> w(a, is_k);
    Runs runs;
    runs.init(a, win_log2, heads, u, step, w.lane);
    Run run, next;
    int position[C], ahead[C], before = 0, before_ahead = 0;
    bool more = runs.next(a, run, w.lane);
    uint32_t at = 0;
    if (more) w.fetch(a, run, place, true, position, before);
    cp_async_commit();
    next = run;
    while (more) {
        const bool fresh = next.head == next.last;
        if (fresh) more = runs.next(a, next, w.lane);
        else ++next.head;
        if (more) w.fetch(a, next, place + (at ^ PLACE), fresh, ahead, before_ahead);
        cp_async_commit();
        cp_async_wait<1>();
        w.store(a, run, place + at, position, before, s_top, round);
        run = next;
        before = before_ahead;
        if (TURN && fresh) {
#pragma unroll
            for (int c = 0; c < C; ++c) position[c] = ahead[c];
        }
        at ^= PLACE;
    }
    u = runs.u - runs.units;
}

}  // namespace

// Blocks of W * C * 512 / d rows.  K's units (TURN: rotated) and V's, and q's.
template <int D, int W, int C, bool TURN>
__global__ void __launch_bounds__(THREADS, RESIDENT) store_kv_fp8_kernel(const StoreFp8Args a, int win_log2, int heads,
                                                                          bool mixed) {
    // two places for a lane's rows: [place][chunk of a row][thread], 16 bytes each
    __shared__ __align__(16) uint8_t s_rows[2][2 * C][THREADS][16];
    __shared__ uint32_t s_top[WARPS / W][2][W];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, group = warp / W;
    const uint32_t step = gridDim.x * (WARPS / W), place = smem_u32(&s_rows[0][0][threadIdx.x][0]);
    uint32_t u = blockIdx.x * (WARPS / W) + group;
    int round = 0;
    // q: one unit of by_token for each warp, the groups' numbers going on behind K's and V's units
    const uint32_t chunks = head_chunks(a.num_q_heads), last = (a.n_tokens + 512 / D - 1) / (512 / D) * chunks;
    auto queries = [&](uint32_t first) {
        for (uint32_t v = first * W + warp % W; v < last; v += step * W)
            by_token<D, QUERY>(a, v, chunks, threadIdx.x & 31);
    };
    // In a full grid half of an SM's blocks begin with q, whose rows are bound by HBM,
    // while the others have K, which is bound by more
    const bool q_first = TURN && mixed && (blockIdx.x * RESIDENT / gridDim.x) % 2;
    if (q_first) {
        const uint32_t kv = 2u * ((a.n_tokens + (1 << win_log2) - 1) >> win_log2) * ((a.pool.num_kv_heads + heads - 1) / heads);
        queries((u + step - kv % step) % step);
    }
    if constexpr (TURN) store_all<D, W, C, true>(a, true, u, step, win_log2, heads, place, s_top[group], round);
#pragma unroll 1
    for (int is_k = TURN ? 0 : 1; is_k >= 0; --is_k)
        store_all<D, W, C, false>(a, is_k, u, step, win_log2, heads, place, s_top[group], round);
    if (TURN && !q_first) queries(u);
}

// Blocks of one row: K's units, then V's, then q's.
template <int D>
__global__ void __launch_bounds__(THREADS, ROWS_RESIDENT) store_rows_fp8_kernel(const StoreFp8Args a) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t tiles = (a.n_tokens + 512 / D - 1) / (512 / D);
    const uint32_t kv_chunks = head_chunks(a.pool.num_kv_heads), q_chunks = head_chunks(a.num_q_heads);
    const uint32_t each = tiles * kv_chunks, step = gridDim.x * WARPS;
    uint32_t u = blockIdx.x * WARPS + (threadIdx.x >> 5);
    for (; u < each; u += step) by_token<D, KEY>(a, u, kv_chunks, lane);
    for (u -= each; u < each; u += step) by_token<D, VALUE>(a, u, kv_chunks, lane);
    for (u -= each; u < tiles * q_chunks; u += step) by_token<D, QUERY>(a, u, q_chunks, lane);
}

namespace {

template <int D, int W, int C>
cudaError_t launch_runs(const StoreFp8Args &a, cudaStream_t s) {
    const int64_t resident = (int64_t)device_sm_count() * RESIDENT, groups = WARPS / W;
    const int64_t n = a.n_tokens, H = a.pool.num_kv_heads;
    // Windows as wide as still give every resident group two units, up to a block's
    // rows (about one run begins in each then), and then as many heads to a unit as
    // leave eight.
    auto units = [&](int win, int64_t chunks) { return 2 * ((n + (1 << win) - 1) >> win) * chunks; };
    int win = 0;
    while (win < a.pool.block_log2 && units(win + 1, H) >= 2 * resident * groups) ++win;
    int64_t chunks = H;
    while (chunks > 1 && units(win, (chunks + 1) / 2) >= 8 * resident * groups) chunks = (chunks + 1) / 2;
    const int64_t heads = (H + chunks - 1) / chunks;
    const int64_t q_units = (n + 512 / D - 1) / (512 / D) * head_chunks(a.num_q_heads);
    const int64_t blocks =
        std::min((units(win, (H + heads - 1) / heads) + (q_units + W - 1) / W + groups - 1) / groups, resident);
    return launch_pdl(a.rotary_dim ? store_kv_fp8_kernel<D, W, C, true> : store_kv_fp8_kernel<D, W, C, false>,
                      dim3((unsigned)blocks), dim3(THREADS), 0, s, a, win, (int)heads, blocks == resident);
}

template <int D>
cudaError_t launch_as(const StoreFp8Args &a, cudaStream_t s) {
    switch (a.pool.block_log2) {
        case 0: {
            const int64_t tiles = ((int64_t)a.n_tokens + 512 / D - 1) / (512 / D);
            const int64_t units = tiles * (2 * head_chunks(a.pool.num_kv_heads) + head_chunks(a.num_q_heads));
            const int64_t blocks = std::min((units + WARPS - 1) / WARPS, (int64_t)device_sm_count() * ROWS_RESIDENT);
            return launch_pdl(store_rows_fp8_kernel<D>, dim3((unsigned)blocks), dim3(THREADS), 0, s, a);
        }
        case 4: return launch_runs<D, 1, D / 32>(a, s);
        case 5: return launch_runs<D, D / 64, 4>(a, s);
        default: return launch_runs<D, D / 32, 4>(a, s);
    }
}

}  // namespace

cudaError_t launch_store_kv_fp8(const StoreFp8Args &a, cudaStream_t s) {
    if (a.n_tokens == 0) return cudaSuccess;
    return a.pool.head_dim == 128 ? launch_as<128>(a, s) : launch_as<64>(a, s);
}

}  // namespace minisgl

// decode_fp4.cuh -- one warp's share of decode attention over the 4-bit pool:
// the running softmax and output of one (request, KV head), fed with tiles of
// tokens in shared memory.
//
//   * An element times its scale is exact in fp16, so the tiles enter fp16
//     MMAs: cvt e2m1x2 -> f16x2 gives two elements, one f16x2 multiplication
//     by the scale gives two values.
//   * S^T = K Q^T (m16n8k16): a lane of the A operand holds whole bytes.  The
//     sum over channels may run in any order, so lane t of a row's four lanes
//     takes channels [t d/4, (t+1) d/4), contiguous in memory (one 16-byte
//     read a row at d 128), and the queries are laid out to match.
//   * O^T += V^T P^T: the A operand pairs two tokens in a register, and the
//     elements of one channel of both tokens are brought into one byte by
//     shifts and masks before the conversion (two instructions for four
//     bytes).  Lane group g takes channels [g d/8, (g+1) d/8).
//   * q enters as fp16 after an exact power-of-two scaling per head (largest
//     |q| below 2^15), undone in the softmax scale; bf16 elements keep all
//     their bits unless 2^32 times smaller than the head's largest.
//   * The softmax weights are 2^(x - ref) with a reference that follows the
//     running maximum lazily: it starts 8 below the maximum and moves only
//     when a weight would pass 2^15, so that the accumulators are rescaled
//     seldom and no shuffle is needed per tile.  Weights below the maximum by
//     up to 2^-22 keep fp16's 11 bits, and are gone below 2^-32.  Sums and
//     accumulators are fp32.
#pragma once
#include <cstdint>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {
namespace fp4 {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float REF_START = -3.402823466e38f;  // no finite score is below: the first tile sets the reference
constexpr float REF_BELOW = 8.f;     // the reference starts this far below the maximum (base 2)
constexpr float REF_ROOM = 15.f;     // and moves when a score passes it by more: 2^15 fits fp16

template <int D>
struct Head {
    static constexpr int RB = D / 2;          // bytes of one head row
    static constexpr int SB = D / FP4_BLOCK;  // scale bytes of one head row
    static constexpr int KS = D / 16;         // k16 steps along head_dim (QK^T)
    static constexpr int MT = D / 16;         // m16 tiles along head_dim (PV)
    static constexpr int QPT = D / 4;         // channels of a lane in QK^T
    static constexpr int OPT = D / 8;         // channels of a lane group in PV
};

__device__ __forceinline__ int clamp_len(int n, int w) { return min(max(n, 0), w); }

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero accumulator.
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                                    uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%10,%10,%10};\n"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Transpose an 8x8 b16 matrix held in the mma fragment layout.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t ad) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];\n" : "=r"(v) : "r"(ad));
    return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t ad) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];\n" : "=h"(v) : "r"(ad));
    return v;
}
template <int WORDS>
__device__ __forceinline__ void lds_words(uint32_t ad, uint32_t (&w)[WORDS]) {
    if constexpr (WORDS == 4)
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                     : "r"(ad));
    else if constexpr (WORDS == 2)
        asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(ad));
    else
        asm volatile("ld.shared.u32 %0, [%1];\n" : "=r"(w[0]) : "r"(ad));
}

// A tile in shared memory: one record per token of 32, [K rows of all heads,
// V rows, K scales, V scales], records `stride` bytes apart with
// stride % 128 == 32 or 96.  Token x lies in slot slot(x).  The lanes' reads
// then spread over all banks: a quarter-warp reads the 64-byte K rows (d 128)
// of tokens 2i and 2i+1, whose slots differ by 2 mod 4, so by 64 bytes; the
// lanes of a V read have tokens 2t (or 2t+1), t = 0..3, in slots that are
// distinct mod 4, 32 bytes apart.
__device__ __forceinline__ int slot(int x) {
    return (x & 24) | ((x & 1) ? 4 | (((x >> 1) & 3) ^ 2) : (x >> 1) & 3);
}

// NG: n8 tiles of query heads (1 when the group has <= 8 heads, else 2).
// Column e of n-tile n is query head n*8 + 2*(lane%4) + e of the group.
template <int D, int NG>
struct Stream {
    using C = Head<D>;
    float ref[NG][2], l[NG][2], sc[NG][2];
    float o[C::MT][NG][4];
    uint32_t qb[NG][C::KS][2];

    // Asks L1 for the queries that open() will load: G rows from row0.
    __device__ __forceinline__ void prefetch(const DecodeArgs &a, int64_t row0, int G, bool live, int lane) const {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int h = n * 8 + (lane >> 2);
            if (h < G && live)
                asm volatile("prefetch.global.L1 [%0];\n" ::"l"(static_cast<const __nv_bfloat16 *>(a.q) + (row0 + h) * D +
                                                                (lane & 3) * C::QPT));
        }
    }

    // Loads the group's queries (q: G rows of D; null leaves zeros) and clears the sums.
    __device__ __forceinline__ void open(const __nv_bfloat16 *q, int G, float scale_log2, int lane) {
        const int lg = lane >> 2, lt = lane & 3;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const int h = n * 8 + lg;
            uint32_t w[C::QPT / 2];  // this lane's channels of head h
#pragma unroll
            for (int i = 0; i < C::QPT / 2; ++i) w[i] = 0u;
            if (h < G && q) {
                const __nv_bfloat16 *src = q + h * D + lt * C::QPT;
#pragma unroll
                for (int i = 0; i < C::QPT / 8; ++i) {
                    const uint4 v = reinterpret_cast<const uint4 *>(src)[i];
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
            }
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < C::QPT / 2; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
            m = max(m & 0xffffu, m >> 16);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            // largest |q| in [2^(b-127), 2^(b-126)): times 2^(141-b) it is below 2^15
            const int b = max((int)(m >> 7), 20);
            const float up = __int_as_float((268 - b) << 23);
            const float down = __int_as_float((b - 14) << 23) * scale_log2;
#pragma unroll
            for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x = w[2 * ks + i];
                    qb[n][ks][i] = f32_to_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sc[n][e] = __shfl_sync(0xffffffffu, down, (2 * lt + e) * 4);
                ref[n][e] = REF_START;
                l[n][e] = 0.f;
            }
        }
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int n = 0; n < NG; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }

    // Where the lane reads in a stage (kp, skp of scores(), vp[2], svp[2] of
    // values()), kept in registers: made again for every tile they took 17 of
    // 634 instructions a tile.  k, sk, v, sv: shared addresses of this head's K row, K
    // scales, V row and V scales in slot 0.
    __device__ __forceinline__ void addresses(uint32_t k, uint32_t sk, uint32_t v, uint32_t sv, int stride, int lane,
                                              uint32_t (&rd)[6]) const {
        const int lg = lane >> 2, lt = lane & 3;
        rd[0] = k + slot(lg) * stride + lt * (C::QPT / 2);
        rd[1] = sk + slot(lg) * stride + (D == 128 ? 2 * lt : lt);
        const uint32_t vo = lg * (C::OPT / 2), so = D == 128 ? lg : lg >> 1;
        rd[2] = v + lt * stride + vo;
        rd[3] = v + (4 + (lt ^ 2)) * stride + vo;
        rd[4] = sv + lt * stride + so;
        rd[5] = sv + (4 + (lt ^ 2)) * stride + so;
#pragma unroll
        for (int i = 0; i < 6; ++i) asm("" : "+r"(rd[i]));
    }

    // The weights of 32 tokens, the first `left` of which count, as the B
    // operand of the product with V.
    __device__ __forceinline__ void scores(uint32_t kp, uint32_t skp, int stride, int left, int lane,
                                           uint32_t (&pb)[2][NG][2]) {
        const int lg = lane >> 2;
        // ---- S^T = K Q^T for two blocks of 16 tokens ----
        float sa[2][NG][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            constexpr int WORDS = C::QPT / 8;  // 32-bit words of a lane's channels
            uint32_t k0[WORDS], k1[WORDS];
            lds_words<WORDS>(kp + (16 * b) * stride, k0);
            lds_words<WORDS>(kp + (16 * b + 8) * stride, k1);
            uint32_t s0, s1;  // the scales of the lane's two blocks, or of its one (twice)
            if constexpr (D == 128) {
                s0 = e4m3x2_to_f16x2(lds_u16(skp + (16 * b) * stride));
                s1 = e4m3x2_to_f16x2(lds_u16(skp + (16 * b + 8) * stride));
            } else {
                s0 = e4m3x2_to_f16x2(lds_u8(skp + (16 * b) * stride));
                s1 = e4m3x2_to_f16x2(lds_u8(skp + (16 * b + 8) * stride));
            }
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                uint32_t e0[4], e1[4];
                e2m1x8_to_f16x2(k0[i], e0);
                e2m1x8_to_f16x2(k1[i], e1);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    e0[u] = i < 2 ? mul_f16x2_half<false>(e0[u], s0) : mul_f16x2_half<true>(e0[u], s0);
                    e1[u] = i < 2 ? mul_f16x2_half<false>(e1[u], s1) : mul_f16x2_half<true>(e1[u], s1);
                }
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    if (i == 0)
                        mma_f16_16816_first(sa[b][n], e0[0], e1[0], e0[1], e1[1], qb[n][0][0], qb[n][0][1]);
                    else
                        mma_f16_16816(sa[b][n], e0[0], e1[0], e0[1], e1[1], qb[n][2 * i][0], qb[n][2 * i][1]);
                    mma_f16_16816(sa[b][n], e0[2], e1[2], e0[3], e1[3], qb[n][2 * i + 1][0], qb[n][2 * i + 1][1]);
                }
            }
        }
        // ---- softmax weights; this lane holds tokens lg + 8*i (i < 4) ----
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            // [e][token]: scores less the reference, then weights.  The scores are
            // rounded before the subtraction: in one fma the largest could come
            // out half a unit of its last place (8 and more from 2^27 on) off
            // the reference that is made of it.
            float x[2][4];
            auto relative = [&]() {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[e][i] = __fsub_rn(__fmul_rn(sa[i >> 1][n][2 * (i & 1) + e], sc[n][e]), ref[n][e]);
                if (left < 32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (lg + 8 * i >= left) x[0][i] = x[1][i] = -INFINITY;
                }
            };
            relative();
            float mx[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) mx[e] = fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3]));
            if (__any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) > REF_ROOM)) {
                const float old[2] = {ref[n][0], ref[n][1]};
                ref[n][0] = ref[n][1] = 0.f;
                relative();  // the scores themselves: the first reference is too far off to add back
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[e] = fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3]));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 4));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 8));
                    mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 16));
                    ref[n][e] = fmaxf(old[e], mx[e] - REF_BELOW);
                    const float al = ex2(old[e] - ref[n][e]);
                    l[n][e] *= al;
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        o[mt][n][e] *= al;
                        o[mt][n][2 + e] *= al;
                    }
                }
                relative();
                // from 2^27 on the reference itself may be rounded to 16 below; a NaN stays
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[e][i] = x[e][i] > REF_ROOM ? REF_ROOM : x[e][i];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[e][i] = ex2(x[e][i]);
                    l[n][e] += x[e][i];
                }
            // P^T as the B operand: transpose the 8x8 token-by-head blocks
#pragma unroll
            for (int i = 0; i < 4; ++i) pb[i >> 1][n][i & 1] = movmatrix_t(f32_to_f16x2(x[0][i], x[1][i]));
        }
    }

    // O^T += V^T P^T for the same tokens.
    __device__ __forceinline__ void values(uint32_t vp0, uint32_t vp1, uint32_t svp0, uint32_t svp1, int stride,
                                           const uint32_t (&pb)[2][NG][2]) {
        // tokens 2lt, 2lt+1, 2lt+8, 2lt+9 of a block: slots lt, 4 + (lt ^ 2), and 8 more
        const uint32_t vp[2] = {vp0, vp1}, svp[2] = {svp0, svp1};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            constexpr int WORDS = C::OPT / 8;
            uint32_t w[4][WORDS], s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                lds_words<WORDS>(vp[i & 1] + (16 * b + 4 * (i & 2)) * stride, w[i]);
                s[i] = lds_u8(svp[i & 1] + (16 * b + 4 * (i & 2)) * stride);
            }
            const uint32_t s01 = e4m3x2_to_f16x2(s[0] | (s[1] << 8));
            const uint32_t s23 = e4m3x2_to_f16x2(s[2] | (s[3] << 8));
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                // bytes of (token, next token) of one channel: even channels, odd channels
                uint32_t f[4][4];
                e2m1x8_to_f16x2((w[0][i] & 0x0f0f0f0fu) | ((w[1][i] << 4) & 0xf0f0f0f0u), f[0]);
                e2m1x8_to_f16x2(((w[0][i] >> 4) & 0x0f0f0f0fu) | (w[1][i] & 0xf0f0f0f0u), f[1]);
                e2m1x8_to_f16x2((w[2][i] & 0x0f0f0f0fu) | ((w[3][i] << 4) & 0xf0f0f0f0u), f[2]);
                e2m1x8_to_f16x2(((w[2][i] >> 4) & 0x0f0f0f0fu) | (w[3][i] & 0xf0f0f0f0u), f[3]);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t a0 = mul_f16x2(f[0][u], s01), a1 = mul_f16x2(f[1][u], s01);
                    const uint32_t a2 = mul_f16x2(f[2][u], s23), a3 = mul_f16x2(f[3][u], s23);
#pragma unroll
                    for (int n = 0; n < NG; ++n)
                        mma_f16_16816(o[4 * i + u][n], a0, a1, a2, a3, pb[b][n][0], pb[b][n][1]);
                }
            }
        }
    }

    // Writes the result: bf16 rows if the stream is whole, else fp32 partial
    // `split` and its natural-log LSE.  row0: index of the group's first
    // (request, query head) row.
    __device__ __forceinline__ void close(const DecodeArgs &a, int64_t row0, int G, bool whole, int split,
                                          float out_scale, int lane) const {
        const int lg = lane >> 2, lt = lane & 3;
#pragma unroll
        for (int n = 0; n < NG; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                const int h = n * 8 + 2 * lt + e;
                if (h >= G) continue;
                const float inv = out_scale / sum;
                const int64_t hh = row0 + h;
                // this lane's channels lg*OPT + 2*mt + {0, 1} are contiguous
                if (whole) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + hh * D + lg * C::OPT;
#pragma unroll
                    for (int mt = 0; mt < C::MT; mt += 4)
                        st_v4(dst + 2 * mt, make_uint4(pack_bf16x2(o[mt][n][e] * inv, o[mt][n][2 + e] * inv),
                                                       pack_bf16x2(o[mt + 1][n][e] * inv, o[mt + 1][n][2 + e] * inv),
                                                       pack_bf16x2(o[mt + 2][n][e] * inv, o[mt + 2][n][2 + e] * inv),
                                                       pack_bf16x2(o[mt + 3][n][e] * inv, o[mt + 3][n][2 + e] * inv)));
                } else {
                    float *dst = a.ws_o + (hh * a.max_splits + split) * D + lg * C::OPT;
#pragma unroll
                    for (int mt = 0; mt < C::MT; mt += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * mt) =
                            make_float4(o[mt][n][e] * inv, o[mt][n][2 + e] * inv, o[mt + 1][n][e] * inv,
                                        o[mt + 1][n][2 + e] * inv);
                    if (lg == 0) a.ws_lse[hh * a.max_splits + split] = (ref[n][e] + __log2f(sum)) * LN2;
                }
            }
    }
};

// ---- the cut of the work into ranges ---------------------------------------
constexpr int TILE = 32;  // tokens of a tile

// A tile: its request and head block, and the tokens from its first one to
// the end of the request's context.
struct Cursor {
    int r, hb, left;
};

// Every CTA derives the same schedule from seq_lens: the tiles of all streams
// (request, head block) in a row, cut into nseg ranges whose lengths differ
// by at most one tile (32-bit arithmetic: all tiles together are below 2^31).  The prefix sums are kept for every CHUNK-th request
// only, so that they leave room for the rings at the largest batch.
constexpr int CHUNK = 4;
__host__ __device__ constexpr int schedule_ints(int batch) { return (batch + CHUNK - 1) / CHUNK + 2; }

struct Schedule {
    const int32_t *prefix;  // shared: tiles before request CHUNK * k, then all tiles
    const int32_t *seq_lens;
    int batch, W, hblocks, chunks, total;
    bool whole;             // range i is stream i
    int nseg, each, more;   // ranges, tiles of each, how many have one more

    // Called by all threads of the CTA (it synchronises them); s_prefix has
    // room for schedule_ints(batch).  With whole there is nothing to sum.
    __device__ __forceinline__ void init(int32_t *s_prefix, const DecodeArgs &a, int hblocks_, int ranges,
                                         bool whole_) {
        whole = whole_;
        prefix = s_prefix;
        seq_lens = a.seq_lens;
        batch = a.batch;
        W = a.pt_width;
        hblocks = hblocks_;
        chunks = (a.batch + CHUNK - 1) / CHUNK;
        if (whole) {
            nseg = a.batch * hblocks;
            total = 1;
            __syncthreads();
            return;
        }
        // every thread sums the tiles of its chunks, then a scan over the CTA
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        __shared__ int s_sum[32], s_max[32];
        const int share = (chunks + blockDim.x - 1) / blockDim.x;
        const int busy = (chunks + 32 * share - 1) / (32 * share);  // warps that have any
        const int k0 = min(tid * share, chunks), k1 = min(k0 + share, chunks);
        int mine = 0, mx = 0;
        for (int k = k0; k < k1; ++k) {
            int nt[CHUNK];
            chunk_tiles(k, nt);
#pragma unroll
            for (int q = 0; q < CHUNK; ++q) {
                mine += nt[q];
                mx = max(mx, nt[q]);
            }
        }
        mine *= hblocks;
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += u;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (chunks <= 32) {  // warp 0 has them all
            if (warp == 0 && lane < chunks) s_prefix[lane] = inc - mine;
            if (tid == 31) {
                s_prefix[chunks] = inc;
                s_prefix[chunks + 1] = mx;
            }
        } else {
            if (lane == 31) {
                s_sum[warp] = inc;
                s_max[warp] = mx;
            }
            __syncthreads();
            int at = inc - mine;  // tiles before this thread's chunks
            for (int w = 0; w < min(warp, busy); ++w) at += s_sum[w];
            for (int k = k0; k < k1; ++k) {
                s_prefix[k] = at;
                if (share == 1) break;
                int nt[CHUNK];
                chunk_tiles(k, nt);
#pragma unroll
                for (int q = 0; q < CHUNK; ++q) at += nt[q] * hblocks;
            }
            if (tid == 0) {
                int all = 0, longest = 0;
                for (int w = 0; w < busy; ++w) {
                    all += s_sum[w];
                    longest = max(longest, s_max[w]);
                }
                s_prefix[chunks] = all;
                s_prefix[chunks + 1] = longest;
            }
        }
        __syncthreads();
        total = s_prefix[chunks];
        // nseg ranges of L = total / nseg >= 1 tiles, the first `more` with one
        // more.  A stream of nt tiles meets at most (nt - 2) / L + 2 of them, and
        // L >= (nt - 1) / (max_splits - 1) keeps that within max_splits.
        const int longest = s_prefix[chunks + 1];
        nseg = ranges;
        each = (uint32_t)total / (uint32_t)ranges;
        if (a.split_tokens > 0 || each == 0 || (int64_t)each * (a.max_splits - 1) < longest) {
            int want = a.split_tokens > 0 ? (int)(((int64_t)a.split_tokens + TILE - 1) / TILE) : 1;
            want = max(want, (longest + a.max_splits - 2) / (a.max_splits - 1));
            const int most = total / want;
            nseg = max(1, a.split_tokens > 0 ? most : min(ranges, most));
            each = total / nseg;
        }
        more = total - each * nseg;
    }
    __device__ __forceinline__ int begin(int seg) const { return seg * each + min(seg, more); }
    // the range that holds tile t
    __device__ __forceinline__ int range_of(int t) const {
        const int longer = more * (each + 1);  // tiles of the longer ranges
        return t < longer ? t / (each + 1) : more + (t - longer) / each;
    }
    __device__ __forceinline__ int len(int r) const { return clamp_len(seq_lens[r], W); }
    __device__ __forceinline__ int tiles(int r) const { return (len(r) + TILE - 1) / TILE; }
    // the same of a chunk's requests, all loads at once
    __device__ __forceinline__ void chunk_tiles(int k, int (&nt)[CHUNK]) const {
#pragma unroll
        for (int q = 0; q < CHUNK; ++q) nt[q] = k * CHUNK + q < batch ? seq_lens[k * CHUNK + q] : 0;
#pragma unroll
        for (int q = 0; q < CHUNK; ++q) nt[q] = (clamp_len(nt[q], W) + TILE - 1) / TILE;
    }
    // tiles before head block hb of request r
    __device__ __forceinline__ int before(int r, int hb) const {
        int nt[CHUNK], t = prefix[r / CHUNK];
        chunk_tiles(r / CHUNK, nt);
#pragma unroll
        for (int q = 0; q < CHUNK; ++q) t += nt[q] * (q < r % CHUNK ? hblocks : q == r % CHUNK ? hb : 0);
        return t;
    }
    __device__ __forceinline__ void locate(Cursor &c, int t) const {
        int lo = 0, hi = chunks;  // largest chunk with prefix <= t: it holds tile t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= t) lo = mid; else hi = mid;
        }
        int off = t - prefix[lo], nt[CHUNK], q = 0;
        chunk_tiles(lo, nt);
        int n = nt[0];
#pragma unroll
        for (int i = 1; i < CHUNK; ++i)
            if (q == i - 1 && off >= n * hblocks) {
                off -= n * hblocks;
                n = nt[i];
                q = i;
            }
        c.r = lo * CHUNK + q;
        c.hb = hblocks == 1 ? 0 : off / n;
        c.left = len(c.r) - (off - c.hb * n) * TILE;
    }
    // Tiles of range seg.
    __device__ __forceinline__ int range_tiles(int seg) const {
        return whole ? tiles(seg / hblocks) : begin(seg + 1) - begin(seg);
    }
    // The same, and its first tile (with no tiles: the stream).
    __device__ __forceinline__ int range(int seg, Cursor &c) const {
        if (whole) {
            c.r = hblocks == 1 ? seg : seg / hblocks;
            c.hb = seg - c.r * hblocks;
            c.left = len(c.r);
            return (c.left + TILE - 1) / TILE;
        }
        const int t = begin(seg);
        locate(c, t);
        return begin(seg + 1) - t;
    }
    // To the first tile of the next stream (there is one).
    __device__ __forceinline__ void next_stream(Cursor &c) const {
        if (++c.hb == hblocks) {
            c.hb = 0;
            do { ++c.r; } while (len(c.r) == 0);
        }
        c.left = len(c.r);
    }
};

}  // namespace fp4
}  // namespace minisgl

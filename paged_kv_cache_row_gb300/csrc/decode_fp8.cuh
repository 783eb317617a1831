// decode_fp8.cuh -- one warp's share of decode attention over the 8-bit pool:
// the running softmax and output of one (request, KV head), fed with tiles of
// tokens in shared memory.
//
//   * e4m3 elements enter fp16 MMAs as they are (cvt e4m3x2 -> f16x2 is exact).
//     The block's power of two is a factor of a whole row, so it is applied to
//     the row's score and weight, not to its channels: per token and query head
//     one multiplication for K and one addition to the exponent for V.
//   * S^T = K Q^T (m16n8k16).  The sum over channels may run in any order, so
//     lane t of a row's four lanes takes channels [t d/4, (t+1) d/4), contiguous
//     in memory, and the queries are laid out to match.
//   * O^T += V^T P^T: the A operand pairs two tokens in a register, so the bytes
//     of two token rows are interleaved before the conversion.  Lane group g
//     takes channels [g d/8, (g+1) d/8).
//   * q enters as fp16 after an exact power-of-two scaling per head, undone in
//     the softmax scale.
//   * With scores s_j (base 2) and V's exponents v_j, the sum is of 2^(x_j), x_j =
//     s_j - a, and the product with V has the weights 2^(x_j + v_j - b), in fp16.
//     The references a and b are whole numbers that follow the running maxima
//     lazily: they leave the largest exponent between 7 and 8 and move when the
//     weights' would pass 15 (or the sum's 60), so that a tile needs no reduction.
//     Weights down to 2^-21 of the largest keep fp16's 11 bits, and may be gone below 2^-32.
//     Why fp16: the product with V is an MMA whose other operand, the elements, is
//     exact in it, and weights in two parts would take twice the MMAs.  bf16's rounding
//     of the output hides it: against 64 bits the outputs of four batches are off by
//     1.6e-3 to 1.7e-3 (of the norm), those of fp32 weights by the same (outputs of the
//     two differ by 0.7e-3 to 1.2e-3, where a bf16 rounding falls the other way).
//     Blocks whose scales are far apart need both references: with one, a zero
//     block's 2^-120 would take its tokens out of the sum.  b is relative to a,
//     for scores past 2^24 would swallow v_j.  Sums and accumulators are fp32.
#pragma once
#include <cstdint>

#include "decode_split.cuh"
#include "fp8.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {
namespace fp8 {

using split::LN2;
using split::movmatrix_t;
constexpr float REF_START = -3.402823466e38f;  // no finite score is below: the first tile sets the references
constexpr float REF_BELOW = 8.f;     // they start this far below the maxima (base 2)
constexpr float REF_ROOM = 15.f;     // largest exponent of a weight before they move: 2^15 fits fp16
constexpr float SUM_ROOM = 60.f;     // and of a term of the sum

template <int D>
struct Head {
    static constexpr int KS = D / 16;   // k16 steps along head_dim (QK^T)
    static constexpr int MT = D / 16;   // m16 tiles along head_dim (PV)
    static constexpr int QPT = D / 4;   // channels of a lane in QK^T
    static constexpr int OPT = D / 8;   // channels of a lane group in PV
};

// A tile in shared memory: one record per token of 32, [K rows of all heads, V
// rows], `stride` bytes apart.  The lanes' 16-byte reads at d 128 spread over
// all banks with stride % 128 == 16: a quarter-warp reads 32-byte pieces of K
// rows 2i and 2i+1, 16 bytes apart, and pieces of V rows 0, 2, 4, 6, 32 bytes
// apart.  At d 64 the stride is 32 % 128 and token x lies in slot slot(x): K
// rows 2i and 2i+1 are 64 bytes apart, V rows 2t (or 2t+1) 32.
template <int D>
__host__ __device__ constexpr int record_stride(int heads) {
    return heads * 2 * D + (D == 128 ? 16 : 32);
}
template <int D>
__device__ __forceinline__ int slot(int x) {
    if constexpr (D == 128) return x;
    return (x & 24) | ((x & 1) ? 4 | (((x >> 1) & 3) ^ 2) : (x >> 1) & 3);
}

// bytes (a0, b0, a1, b1) and (a2, b2, a3, b3) of two words
__device__ __forceinline__ void interleave(uint32_t a, uint32_t b, uint32_t &lo, uint32_t &hi) {
    lo = __byte_perm(a, b, 0x5140);
    hi = __byte_perm(a, b, 0x7362);
}

// NG: n8 tiles of query heads (1 when the group has <= 8 heads, else 2).
// Column e of n-tile n is query head n*8 + 2*(lane%4) + e of the group.
template <int D, int NG>
struct Stream {
    using C = Head<D>;
    float ref_s[NG][2], ref_v[NG][2];  // a, and b relative to a
    float l[NG][2], sc[NG][2];
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
        const int lt = lane & 3;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            const float down = split::load_queries<D>(q, n * 8, G, scale_log2, lane, qb[n]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                sc[n][e] = __shfl_sync(0xffffffffu, down, (2 * lt + e) * 4);
                ref_s[n][e] = REF_START;
                ref_v[n][e] = 0.f;
                l[n][e] = 0.f;
            }
        }
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int n = 0; n < NG; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    }

    // The weights of 32 tokens, the first `left` of which count, as the B
    // operand of the product with V.  kp: where the lane reads K in the tile's
    // first record; sp: the tile's scale words, (K, V) per token, this head's
    // in the byte `shift` bits up.
    __device__ __forceinline__ void scores(uint32_t kp, uint32_t sp, int shift, int stride, int left, int lane,
                                           uint32_t (&pb)[2][NG][2]) {
        const int lg = lane >> 2;
        // ---- the scales of tokens lg + 8*i: 2^eK as a factor, eV as a number ----
        float kf[4], ve[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t w[2];
            lds_words<2>(sp + (lg + 8 * i) * 8, w);
            kf[i] = __uint_as_float(((w[0] >> shift) & 0xffu) << 23);
            // 2^23 + byte less 2^23 + 127
            ve[i] = __uint_as_float(((w[1] >> shift) & 0xffu) | 0x4b000000u) - (8388608.f + EXP_BIAS);
        }
        // ---- S^T = K Q^T for two blocks of 16 tokens ----
        float sa[2][NG][4];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            constexpr int QUADS = C::QPT / 16;  // 16-byte pieces of a lane's channels
            uint32_t k0[QUADS][4], k1[QUADS][4];
#pragma unroll
            for (int i = 0; i < QUADS; ++i) {
                lds_words<4>(kp + (16 * b) * stride + 16 * i, k0[i]);
                lds_words<4>(kp + (16 * b + 8) * stride + 16 * i, k1[i]);
            }
#pragma unroll
            for (int i = 0; i < 4 * QUADS; ++i) {
                uint32_t a0, a1, a2, a3;
                e4m3x4_to_f16x2(k0[i >> 2][i & 3], a0, a2);
                e4m3x4_to_f16x2(k1[i >> 2][i & 3], a1, a3);
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    if (i == 0)
                        mma_f16_16816_first(sa[b][n], a0, a1, a2, a3, qb[n][0][0], qb[n][0][1]);
                    else
                        mma_f16_16816(sa[b][n], a0, a1, a2, a3, qb[n][i][0], qb[n][i][1]);
                }
            }
        }
        // ---- softmax weights; this lane holds tokens lg + 8*i (i < 4) ----
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            // [e][token]: exponents of the sum and of the weights.  A score is
            // rounded before a reference is taken from it: in one fma the largest
            // could come out half a unit of its last place off the reference that
            // is made of it.
            float x[2][4], y[2][4], ms[2], mv[2];
            auto sums = [&](const float (&a)[2]) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        x[e][i] = __fsub_rn(
                            __fmul_rn(sa[i >> 1][n][2 * (i & 1) + e], __fmul_rn(sc[n][e], kf[i])), a[e]);
                if (left < 32) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (lg + 8 * i >= left) x[0][i] = x[1][i] = -INFINITY;
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) ms[e] = fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3]));
            };
            auto weights = [&](const float (&b)[2]) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[e][i] = x[e][i] + (ve[i] - b[e]);
                    mv[e] = fmaxf(fmaxf(y[e][0], y[e][1]), fmaxf(y[e][2], y[e][3]));
                }
            };
            sums(ref_s[n]);
            weights(ref_v[n]);
            if (__any_sync(0xffffffffu, fmaxf(mv[0], mv[1]) > REF_ROOM || fmaxf(ms[0], ms[1]) > SUM_ROOM)) {
                const float zero[2] = {0.f, 0.f};
                auto over_warp = [&](float (&m)[2]) {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], d));
                };
                float moved[2];
                sums(zero);  // the scores themselves: the first reference is too far off to add back
                over_warp(ms);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float old = ref_s[n][e];
                    ref_s[n][e] = fmaxf(old, ceilf(ms[e]) - REF_BELOW);
                    moved[e] = old - ref_s[n][e];
                    l[n][e] *= ex2(moved[e]);
                }
                sums(ref_s[n]);  // (from 2^27 on a itself is rounded, and the largest exponent is 0 or 16)
                weights(zero);
                over_warp(mv);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float old = ref_v[n][e] + moved[e];
                    ref_v[n][e] = fmaxf(old, ceilf(mv[e]) - REF_BELOW);
                    const float al = ex2(old - ref_v[n][e]);
#pragma unroll
                    for (int mt = 0; mt < C::MT; ++mt) {
                        o[mt][n][e] *= al;
                        o[mt][n][2 + e] *= al;
                    }
                }
                weights(ref_v[n]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    l[n][e] += ex2(x[e][i]);
                    y[e][i] = ex2(y[e][i]);
                }
            // P^T as the B operand: transpose the 8x8 token-by-head blocks
#pragma unroll
            for (int i = 0; i < 4; ++i) pb[i >> 1][n][i & 1] = movmatrix_t(f32_to_f16x2(y[0][i], y[1][i]));
        }
    }

    // O^T += V^T P^T for the same tokens.  vp0, vp1: where the lane reads V of
    // tokens 2t and 2t + 1 in the tile.
    __device__ __forceinline__ void values(uint32_t vp0, uint32_t vp1, int stride, const uint32_t (&pb)[2][NG][2]) {
        const uint32_t vp[2] = {vp0, vp1};
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            constexpr int WORDS = C::OPT / 4;
            uint32_t w[4][WORDS];  // tokens 2t, 2t+1, 2t+8, 2t+9 of the block
#pragma unroll
            for (int i = 0; i < 4; ++i) lds_words<WORDS>(vp[i & 1] + (16 * b + 4 * (i & 2)) * stride, w[i]);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                uint32_t p[2], q[2];
                interleave(w[0][i], w[1][i], p[0], p[1]);
                interleave(w[2][i], w[3][i], q[0], q[1]);
#pragma unroll
                for (int u = 0; u < 2; ++u) {  // channels 4i + 2u and the next
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_f16x2(p[u], a0, a1);
                    e4m3x4_to_f16x2(q[u], a2, a3);
#pragma unroll
                    for (int n = 0; n < NG; ++n)
                        mma_f16_16816(o[2 * i + u][n], a0, a1, a2, a3, pb[b][n][0], pb[b][n][1]);
                }
            }
        }
    }

    // Writes the result: bf16 rows if the stream is whole, else fp32 partial
    // `split` and its natural-log LSE.  row0: index of the group's first
    // (request, query head) row.
    __device__ __forceinline__ void close(const DecodeArgs &a, int64_t row0, int G, bool whole, int split,
                                          int lane) const {
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
                // 2^b / sum in two factors: the first may pass fp32's range where the result does not
                const int d = (int)fminf(fmaxf(ref_v[n][e], -252.f), 252.f), d2 = d / 2;
                const float inv = pow2i(d2) / sum, rest = pow2i(d - d2);
                const int64_t hh = row0 + h;
                float r[C::MT][2];  // this lane's channels lg*OPT + 2*mt + {0, 1} are contiguous
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt) {
                    r[mt][0] = o[mt][n][e] * inv * rest;
                    r[mt][1] = o[mt][n][2 + e] * inv * rest;
                }
                if (whole) {
                    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(a.out) + hh * D + lg * C::OPT;
#pragma unroll
                    for (int mt = 0; mt < C::MT; mt += 4)
                        st_v4(dst + 2 * mt, make_uint4(pack_bf16x2(r[mt][0], r[mt][1]), pack_bf16x2(r[mt + 1][0], r[mt + 1][1]),
                                                       pack_bf16x2(r[mt + 2][0], r[mt + 2][1]),
                                                       pack_bf16x2(r[mt + 3][0], r[mt + 3][1])));
                } else {
                    float *dst = a.ws_o + (hh * a.max_splits + split) * D + lg * C::OPT;
#pragma unroll
                    for (int mt = 0; mt < C::MT; mt += 2)
                        *reinterpret_cast<float4 *>(dst + 2 * mt) =
                            make_float4(r[mt][0], r[mt][1], r[mt + 1][0], r[mt + 1][1]);
                    if (lg == 0) a.ws_lse[hh * a.max_splits + split] = (ref_s[n][e] + __log2f(sum)) * LN2;
                }
            }
    }
};

}  // namespace fp8
}  // namespace minisgl

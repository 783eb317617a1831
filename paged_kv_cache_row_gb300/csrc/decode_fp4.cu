// decode_fp4.cu -- split-KV GQA decode attention over the 4-bit paged pool.
//
//     out[r,h] = sum_j softmax_j(sm_scale <q[r,h], K_j>) V_j,   j < seq_len[r],
// K_j and V_j the values c * s * 2^exp of row page_table[r, j] (the pool's
// format is in the public header).  Split partials are merged by
// decode_merge_kernel, as for the bf16 pool.
//
// What bounds it: the K/V bytes, 2 * (d/2 + d/16) a token and KV head, 144 at
// d 128.  At the card's copy rate that is one element every 1/43 of a cycle
// per SM, so the conversion of the elements has to stay near one instruction
// per element:
//   * an element times its scale is exact in fp16, so the tiles enter fp16
//     MMAs: cvt e2m1x2 -> f16x2 gives two elements, one f16x2 multiplication
//     by the scale gives two values;
//   * S^T = K Q^T (m16n8k16): a lane of the A operand holds whole bytes.  The
//     sum over channels may run in any order, so lane t of a row's four lanes
//     takes channels [t d/4, (t+1) d/4), contiguous in memory (one 16-byte
//     read a row at d 128), and the queries are laid out to match;
//   * O^T += V^T P^T: the A operand pairs two tokens in a register, and the
//     elements of one channel of both tokens are brought into one byte by
//     shifts and masks before the conversion (two instructions for four
//     bytes).  Lane group g takes channels [g d/8, (g+1) d/8);
//   * q enters as fp16 after an exact power-of-two scaling per head (largest
//     |q| below 2^15), undone in the softmax scale; bf16 elements keep all
//     their bits unless 2^32 times smaller than the head's largest;
//   * the softmax weights are 2^(x - ref) with a reference that follows the
//     running maximum lazily: it starts 8 below the maximum and moves only
//     when a weight would pass 2^15, so that the accumulators are rescaled
//     seldom and no shuffle is needed per tile.  Weights below the maximum by
//     up to 2^-22 keep fp16's 11 bits, and are gone below 2^-32.  Sums and
//     accumulators are fp32.
//
// Work: tiles of 32 tokens of one request; a CTA's warps take different KV
// heads of the same tiles (a token's row is contiguous over the heads, and
// eight heads' scales share 64 bytes), or different tile ranges where there
// are fewer heads than warps.  The tiles of all requests are cut evenly over
// the CTAs (times the ranges per CTA): contiguous ranges whose lengths
// differ by at most one tile.  Every warp runs its own cp.async ring; only
// the schedule's prefix sum is shared.
#include <cmath>
#include <mutex>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int TILE = 32;       // tokens per warp tile, two MMA row blocks of 16
constexpr int MAX_WARPS = 8;   // per CTA
constexpr int STAGES = 3;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float REF_START = -1e30f;  // below every finite score: the first tile sets the reference
constexpr float REF_BELOW = 8.f;     // the reference starts this far below the maximum (base 2)
constexpr float REF_ROOM = 15.f;     // and moves when a score passes it by more: 2^15 fits fp16

// Bytes of a tile in shared memory: K elements, V elements, K scales, V scales.
template <int D>
struct Fp4Tile {
    static constexpr int RB = D / 2;                // bytes of one head row
    static constexpr int CPR = RB / 16;             // 16-byte chunks per row
    static constexpr int SB = D / FP4_BLOCK;        // scale bytes per row
    static constexpr int V_OFF = TILE * RB;
    static constexpr int KS_OFF = 2 * TILE * RB;
    static constexpr int VS_OFF = KS_OFF + TILE * SB;
    static constexpr int BYTES = VS_OFF + TILE * SB;
    static constexpr int KS = D / 16;               // k16 steps along head_dim (QK^T)
    static constexpr int MT = D / 16;               // m16 tiles along head_dim (PV)
    static constexpr int QPT = D / 4;               // channels of a lane in QK^T
    static constexpr int OPT = D / 8;               // channels of a lane group in PV
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

// 4- or 8-byte cp.async through L1 (the heads of a CTA share the 32-byte
// sectors that hold the scales); src_bytes = 0 fills with zeros.
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;\n" ::"r"(dst), "l"(src), "n"(N), "r"(src_bytes)
                 : "memory");
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

// Where token x (0..31) of a V tile lies: each lane reads tokens 2t, 2t+1,
// 2t+8 and 2t+9 of a row block, and this order puts each of the four reads'
// tokens t = 0..3 next to one another.
__device__ __forceinline__ int v_slot(int x) { return (x & 24) | ((x & 1) << 2) | ((x >> 1) & 3); }

// Byte of 16-byte chunk c of V slot s.  At d 128 four rows of 64 bytes would
// meet in the same banks; slots with bit 1 set have their chunk halves swapped.
template <int D>
__device__ __forceinline__ int v_chunk(int s, int c) {
    return s * Fp4Tile<D>::RB + ((D == 128 ? c ^ (s & 2) : c) << 4);
}

struct Cursor {
    int r, hb, j, nt, n;  // request, head block, tile in stream, tiles in stream, tokens
};

}  // namespace

// NG: n8 tiles of query heads (1 when the group has <= 8 heads, else 2).
// heads: KV heads a CTA works on at a time; subs: tile ranges per CTA, so a
// CTA has heads * subs warps; hblocks: head blocks of `heads` heads.
template <int D, int NG>
__global__ void __launch_bounds__(MAX_WARPS * 32, NG == 1 ? 2 : 1)
    decode_fp4_kernel(const DecodeFp4Args args, const float scale_log2, const float out_scale, const int heads,
                      const int subs, const int hblocks, const int prefix_bytes) {
    using C = Fp4Tile<D>;
    const DecodeArgs &a = args.d;
    const Fp4Layer &pool = args.pool;
    extern __shared__ __align__(128) uint8_t smem[];
    int32_t *s_prefix = reinterpret_cast<int32_t *>(smem);  // [B + 1], then the longest stream
    int32_t &s_maxtiles = s_prefix[a.batch + 1];

    const int B = a.batch, Hkv = a.num_kv_heads, Hq = a.num_q_heads, W = a.pt_width;
    const int G = Hq / Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lg = lane >> 2, lt = lane & 3;
    pdl_wait();
    pdl_launch_dependents();

    // ---- schedule: prefix over requests of (tiles per stream) * hblocks ----
    if (warp == 0) {
        int carry = 0, mx = 0;
        if (lane == 0) s_prefix[0] = 0;
        for (int base = 0; base < B; base += 32) {
            const int r = base + lane;
            int nt = 0;
            if (r < B) nt = (clamp_len(__ldg(a.seq_lens + r), W) + TILE - 1) / TILE;
            mx = max(mx, nt);
            int v = nt * hblocks;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (r < B) s_prefix[r + 1] = carry + v;
            carry += __shfl_sync(0xffffffffu, v, 31);
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (lane == 0) s_maxtiles = mx;
    }
    __syncthreads();
    const int total = s_prefix[B];
    if (total == 0) return;
    // nseg ranges [seg * total / nseg, (seg + 1) * total / nseg), each at least
    // L = total / nseg >= 1 tiles long.  A stream of nt tiles meets at most
    // (nt - 2) / L + 2 of them, and L >= (nt - 1) / (max_splits - 1) keeps that
    // within max_splits.
    int64_t nseg = (int64_t)gridDim.x * subs;
    int want = a.split_tokens > 0 ? (int)(((int64_t)a.split_tokens + TILE - 1) / TILE) : 1;
    want = max(want, (s_maxtiles + a.max_splits - 2) / (a.max_splits - 1));
    if (a.split_tokens > 0) nseg = total / want;
    nseg = max((int64_t)1, min(nseg, (int64_t)(total / want)));

    const int head_in = warp % heads, sub = warp / heads;
    const uint32_t ring = smem_u32(smem + prefix_bytes) + warp * STAGES * C::BYTES;
    const uint32_t data_stride = (uint32_t)pool.data_stride, scale_stride = (uint32_t)pool.scale_stride;

    auto set_request = [&](Cursor &c) {
        c.n = clamp_len(__ldg(a.seq_lens + c.r), W);
        c.nt = (c.n + TILE - 1) / TILE;
    };
    auto locate = [&](Cursor &c, int t) {
        int lo = 0, hi = B;  // largest r with prefix[r] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_prefix[mid] <= t) lo = mid; else hi = mid;
        }
        c.r = lo;
        set_request(c);
        const int off = t - s_prefix[lo];
        c.hb = off / c.nt;
        c.j = off - c.hb * c.nt;
    };
    auto advance = [&](Cursor &c) {  // only called when a next tile exists
        if (++c.j == c.nt) {
            c.j = 0;
            if (++c.hb == hblocks) {
                c.hb = 0;
                do { ++c.r; } while (s_prefix[c.r + 1] == s_prefix[c.r]);
                set_request(c);
            }
        }
    };
    // physical row of token 32*j + lane of the cursor's request, or -1 past its end
    auto load_row = [&](const Cursor &c) -> int {
        const int tok = c.j * TILE + lane;
        if (tok >= c.n) return -1;
        return min(max(__ldg(a.page_table + (int64_t)c.r * a.pt_stride + tok), 0), a.num_rows - 1);
    };
    auto head_of = [&](const Cursor &c) { return c.hb * heads + head_in; };
    // one tile's rows into the ring stage at st
    auto issue = [&](uint32_t st, const Cursor &c, int row) {
        const int head = head_of(c);
        if (head < Hkv) {
            const int cc = lane % C::CPR;  // this lane's 16-byte chunk of every row it copies
            const uint8_t *kd = pool.k_data + head * C::RB + cc * 16, *vd = pool.v_data + head * C::RB + cc * 16;
#pragma unroll
            for (int i = 0; i < TILE * C::CPR / 32; ++i) {
                const int x = lane / C::CPR + i * (32 / C::CPR);
                const int rr = __shfl_sync(0xffffffffu, row, x);
                const uint64_t e = (uint64_t)(uint32_t)max(rr, 0) * data_stride;
                const int bytes = rr >= 0 ? 16 : 0;
                cp_async_16(st + x * C::RB + cc * 16, kd + e, bytes);
                cp_async_16(st + C::V_OFF + v_chunk<D>(v_slot(x), cc), vd + e, bytes);
            }
            const uint64_t e = (uint64_t)(uint32_t)max(row, 0) * scale_stride + head * C::SB;
            const int bytes = row >= 0 ? C::SB : 0;
            cp_async_small<C::SB>(st + C::KS_OFF + lane * C::SB, pool.k_scale + e, bytes);
            cp_async_small<C::SB>(st + C::VS_OFF + v_slot(lane) * C::SB, pool.v_scale + e, bytes);
        }
        cp_async_commit();
    };

    for (int64_t seg = (int64_t)blockIdx.x * subs + sub; seg < nseg; seg += (int64_t)gridDim.x * subs) {
        const int t0 = (int)(seg * total / nseg), t1 = (int)((seg + 1) * total / nseg);

        Cursor pc, cc;
        locate(pc, t0);
        cc = pc;
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            if (t0 + s < t1) {
                issue(ring + s * C::BYTES, pc, load_row(pc));
                if (t0 + s + 1 < t1) advance(pc);
            } else {
                cp_async_commit();
            }
        }
        // the page-table entries of the next tile to issue
        int row_next = -1;
        if (t0 + STAGES - 1 < t1) row_next = load_row(pc);

        // consumer state; column e of n-tile n is query head n*8 + 2*lt + e of the group
        int cur_r = -1, cur_hb = 0, cur_nt = 0, cur_start = 0, first_j = 0, last_j = 0;
        float ref[NG][2], l[NG][2], sc[NG][2];
        float o[C::MT][NG][4];
        uint32_t qb[NG][C::KS][2];

        auto flush = [&]() {
            const int head = cur_hb * heads + head_in;
            if (head >= Hkv) return;
            const bool last = last_j == cur_nt - 1;
            const bool whole = first_j == 0 && last;
            // the range that holds the stream's first tile
            const int64_t seg0 = (((int64_t)cur_start + 1) * nseg - 1) / total;
            const int s = whole ? 0 : (int)(seg - seg0);
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
                    const int64_t hh = (int64_t)cur_r * Hq + head * G + h;
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
                        float *dst = a.ws_o + (hh * a.max_splits + s) * D + lg * C::OPT;
#pragma unroll
                        for (int mt = 0; mt < C::MT; mt += 2)
                            *reinterpret_cast<float4 *>(dst + 2 * mt) =
                                make_float4(o[mt][n][e] * inv, o[mt][n][2 + e] * inv, o[mt + 1][n][e] * inv,
                                            o[mt + 1][n][2 + e] * inv);
                        if (lg == 0) a.ws_lse[hh * a.max_splits + s] = (ref[n][e] + __log2f(sum)) * LN2;
                    }
                }
            if (last && lane == 0) a.split_count[(int64_t)cur_r * Hkv + head] = s + 1;
        };

        auto open_stream = [&]() {
            const int head = head_of(cc);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int h = n * 8 + lg;
                uint32_t w[C::QPT / 2];  // this lane's channels of head h
#pragma unroll
                for (int i = 0; i < C::QPT / 2; ++i) w[i] = 0u;
                if (h < G && head < Hkv) {
                    const __nv_bfloat16 *src = static_cast<const __nv_bfloat16 *>(a.q) +
                                               ((int64_t)cc.r * Hq + head * G + h) * D + lt * C::QPT;
#pragma unroll
                    for (int i = 0; i < C::QPT / 8; ++i) {
                        const uint4 v = ld_nc_v4(src + 8 * i);
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
                        qb[n][ks][i] = f32_to_f16x2(__uint_as_float(x << 16) * up,
                                                    __uint_as_float(x & 0xffff0000u) * up);
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
        };

        uint32_t st = ring, st_in = ring + (STAGES - 1) * C::BYTES;  // stage to use, stage to fill
        for (int t = t0; t < t1; ++t) {
            const int tp = t + STAGES - 1;
            if (tp < t1) {
                issue(st_in, pc, row_next);
                if (tp + 1 < t1) {
                    advance(pc);
                    row_next = load_row(pc);
                }
            } else {
                cp_async_commit();
            }
            if (cc.r != cur_r || cc.hb != cur_hb) {
                if (cur_r >= 0) flush();
                cur_r = cc.r;
                cur_hb = cc.hb;
                cur_nt = cc.nt;
                cur_start = s_prefix[cc.r] + cc.hb * cc.nt;
                first_j = cc.j;
                open_stream();
            }
            cp_async_wait<STAGES - 1>();
            __syncwarp();

            // ---- S^T = K Q^T for two blocks of 16 tokens ----
            float sa[2][NG][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                constexpr int WORDS = C::QPT / 8;  // 32-bit words of a lane's channels
                uint32_t k0[WORDS], k1[WORDS];
                const int x0 = 16 * b + lg, x1 = x0 + 8;
                lds_words<WORDS>(st + x0 * C::RB + lt * (C::QPT / 2), k0);
                lds_words<WORDS>(st + x1 * C::RB + lt * (C::QPT / 2), k1);
                uint32_t s0[2], s1[2];  // the scales of the lane's one or two blocks, in both halves
                if constexpr (D == 128) {
                    const uint32_t h0 = e4m3x2_to_f16x2(lds_u16(st + C::KS_OFF + x0 * C::SB + 2 * lt));
                    const uint32_t h1 = e4m3x2_to_f16x2(lds_u16(st + C::KS_OFF + x1 * C::SB + 2 * lt));
                    s0[0] = __byte_perm(h0, h0, 0x1010);
                    s0[1] = __byte_perm(h0, h0, 0x3232);
                    s1[0] = __byte_perm(h1, h1, 0x1010);
                    s1[1] = __byte_perm(h1, h1, 0x3232);
                } else {
                    const uint32_t h0 = lds_u8(st + C::KS_OFF + x0 * C::SB + lt);
                    const uint32_t h1 = lds_u8(st + C::KS_OFF + x1 * C::SB + lt);
                    s0[0] = s0[1] = e4m3x2_to_f16x2(h0 | (h0 << 8));
                    s1[0] = s1[1] = e4m3x2_to_f16x2(h1 | (h1 << 8));
                }
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    uint32_t e0[4], e1[4];
                    e2m1x8_to_f16x2(k0[i], e0);
                    e2m1x8_to_f16x2(k1[i], e1);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        e0[u] = mul_f16x2(e0[u], s0[i / 2]);
                        e1[u] = mul_f16x2(e1[u], s1[i / 2]);
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
            uint32_t pb[2][NG][2];
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                float x[2][4];  // [e][token]: scores less the reference, then weights
                auto scores = [&]() {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[e][i] = fmaf(sa[i >> 1][n][2 * (i & 1) + e], sc[n][e], -ref[n][e]);
                    if (cc.j == cc.nt - 1) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (cc.j * TILE + lg + 8 * i >= cc.n) x[0][i] = x[1][i] = -INFINITY;
                    }
                };
                scores();
                float mx[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) mx[e] = fmaxf(fmaxf(x[e][0], x[e][1]), fmaxf(x[e][2], x[e][3]));
                if (__any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) > REF_ROOM)) {
                    const float old[2] = {ref[n][0], ref[n][1]};
                    ref[n][0] = ref[n][1] = 0.f;
                    scores();  // the scores themselves: the first reference is too far off to add back
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
                    scores();
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
            // ---- O^T += V^T P^T ----
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                constexpr int WORDS = C::OPT / 8;
                uint32_t v[4][WORDS], sv[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // tokens 2lt, 2lt+1, 2lt+8, 2lt+9 of the block
                    const int s = 16 * b + 4 * i + lt;
                    const uint32_t ad = D == 128 ? v_chunk<D>(s, lg >> 1) + (lg & 1) * 8 : s * C::RB + lg * 4;
                    lds_words<WORDS>(st + C::V_OFF + ad, v[i]);
                    sv[i] = lds_u8(st + C::VS_OFF + s * C::SB + (D == 128 ? lg : lg >> 1));
                }
                const uint32_t sa01 = e4m3x2_to_f16x2(sv[0] | (sv[1] << 8));
                const uint32_t sa23 = e4m3x2_to_f16x2(sv[2] | (sv[3] << 8));
#pragma unroll
                for (int i = 0; i < WORDS; ++i) {
                    // bytes of (token, next token) of one channel: even channels, odd channels
                    uint32_t f[4][4];
                    e2m1x8_to_f16x2((v[0][i] & 0x0f0f0f0fu) | ((v[1][i] << 4) & 0xf0f0f0f0u), f[0]);
                    e2m1x8_to_f16x2(((v[0][i] >> 4) & 0x0f0f0f0fu) | (v[1][i] & 0xf0f0f0f0u), f[1]);
                    e2m1x8_to_f16x2((v[2][i] & 0x0f0f0f0fu) | ((v[3][i] << 4) & 0xf0f0f0f0u), f[2]);
                    e2m1x8_to_f16x2(((v[2][i] >> 4) & 0x0f0f0f0fu) | (v[3][i] & 0xf0f0f0f0u), f[3]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t a0 = mul_f16x2(f[0][u], sa01), a1 = mul_f16x2(f[1][u], sa01);
                        const uint32_t a2 = mul_f16x2(f[2][u], sa23), a3 = mul_f16x2(f[3][u], sa23);
#pragma unroll
                        for (int n = 0; n < NG; ++n)
                            mma_f16_16816(o[4 * i + u][n], a0, a1, a2, a3, pb[b][n][0], pb[b][n][1]);
                    }
                }
            }
            last_j = cc.j;
            if (t + 1 < t1) advance(cc);
            st_in = st;
            st = st == ring + (STAGES - 1) * C::BYTES ? ring : st + C::BYTES;
            __syncwarp();
        }
        if (cur_r >= 0) flush();
        cp_async_wait<0>();
        __syncwarp();
    }
}

namespace {

// CTAs of `kernel` per SM at this block size and dynamic shared memory; the
// kernel's shared-memory limit is raised to the device's.
template <typename K>
cudaError_t blocks_per_sm(K kernel, int threads, size_t smem, int &blocks) {
    struct Entry { const void *fn; int dev, threads; size_t smem; int blocks; };
    static std::mutex mu;
    static Entry cache[64];
    static int used = 0;
    int dev = 0, optin = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].fn == (const void *)kernel && cache[i].dev == dev && cache[i].threads == threads &&
            cache[i].smem == smem) {
            blocks = cache[i].blocks;
            return cudaSuccess;
        }
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem);
    if (e != cudaSuccess) {
        cudaGetLastError();  // do not leave the failure for the next caller to find
        return e;
    }
    if (blocks < 1) return cudaErrorInvalidConfiguration;
    if (used < 64) cache[used++] = {(const void *)kernel, dev, threads, smem, blocks};
    return cudaSuccess;
}

template <int D, int NG>
cudaError_t launch_cfg(const DecodeFp4Args &args, cudaStream_t s) {
    using C = Fp4Tile<D>;
    const DecodeArgs &a = args.d;
    // head blocks of equal size, at most MAX_WARPS heads; tile ranges fill the CTA
    const int hblocks = (a.num_kv_heads + MAX_WARPS - 1) / MAX_WARPS;
    const int heads = (a.num_kv_heads + hblocks - 1) / hblocks;
    const int subs = MAX_WARPS / heads;
    const int warps = heads * subs;
    const int prefix_bytes = (((a.batch + 2) * 4) + 1023) / 1024 * 1024;
    const size_t smem = prefix_bytes + (size_t)warps * STAGES * C::BYTES;
    auto kern = decode_fp4_kernel<D, NG>;
    int nb = 0;
    cudaError_t e = blocks_per_sm(kern, warps * 32, smem, nb);
    if (e != cudaSuccess) return e;
    // never more ranges than tiles could exist
    const int64_t max_tiles = (int64_t)a.batch * hblocks * ((a.pt_width + TILE - 1) / TILE);
    int64_t grid = (int64_t)device_sm_count() * nb;
    const int64_t need = (max_tiles + subs - 1) / subs;
    if (grid > need) grid = need;
    if (grid < 1) grid = 1;
    e = launch_pdl(kern, dim3((unsigned)grid), dim3(warps * 32), smem, s, args,
                   a.sm_scale * LOG2E * ldexpf(1.f, args.pool.k_exp), ldexpf(1.f, args.pool.v_exp), heads, subs,
                   hblocks, prefix_bytes);
    if (e != cudaSuccess) return e;
    return launch_decode_merge(a, s);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeFp4Args &a, cudaStream_t s) {
    if (a.d.batch == 0) return cudaSuccess;
    const int G = a.d.num_q_heads / a.d.num_kv_heads;
    if (a.d.head_dim == 128) return G <= 8 ? launch_cfg<128, 1>(a, s) : launch_cfg<128, 2>(a, s);
    return G <= 8 ? launch_cfg<64, 1>(a, s) : launch_cfg<64, 2>(a, s);
}

}  // namespace minisgl

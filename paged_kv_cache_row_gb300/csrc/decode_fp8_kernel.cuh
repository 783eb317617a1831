// decode_fp8_kernel.cuh -- split-KV GQA decode attention over the 8-bit paged pool.
//
//     out[r,h] = sum_j softmax_j(sm_scale <q[r,h], K_j>) V_j,   j < seq_len[r],
// K_j and V_j the values c * 2^e of row page_table[r, j] (the pool's format is
// in the public header).  Split partials are joined by merge_rows_kernel or merge_row_kernel.
//
// What bounds it: the K/V bytes, 2 d a token and KV head.  256 requests of 1k to
// 8k tokens, 8 KV heads of 128: 219 us for the kernel alone (6.5 TB/s, 0.96 of the
// measured copy rate) and 4.8 for the merge; issue slots are a third busy.
//
// Work: tiles of 32 tokens of one request and a block of KV heads, one warp to a
// head, so that a token's row of these heads (contiguous) is fetched as one
// piece of up to 512 bytes.  A CTA (one per SM) has as many such groups of warps
// as fit 8 warps (16 at d 64), each with a range of tiles of its own; the tiles
// of all requests are cut evenly over the groups of all CTAs (split::Schedule).
// At d 128, 8 heads, blocks of 4 make two groups, which load and compute in turns
// of their own: 256 requests 224 us and 64 requests 58, where one block of 8
// takes 228 and 60.  Other counts of heads: see block_heads.
//
// Loads: each group has a ring of three or more stages with a full and an
// empty mbarrier each.  The group's warps fetch a tile together, each its run
// of the tokens, in 16-byte cp.async pieces; a warp's own head's scales, one
// byte of K and one of V per token, come as the 4-byte words that hold them.
// Page-table entries are read a tile before the rows they name.  Rows past a
// request's end repeat its last row; their weights are zero.
#pragma once
#include <algorithm>
#include <cmath>

#include "decode_fp4_plan.h"
#include "decode_fp8.cuh"

namespace minisgl {
namespace fp8 {

// KV heads of a block, up to 512 bytes of a row; the last block has what is left.
// Times below are us for two batches of as many bytes whatever the heads (floors 45
// and 210 us), with 4 query heads to a KV head.
//
// d 128: the largest of 4, 2 and 1 that leaves at most one warp in eight without a
// head.  All 8 warps have to be in a group (two groups of 3 leave two out), and a warp
// without a head still goes through its group's tiles.
//   KV heads         3       5       6       7       8       9       10      13
//   blocks of 4              70 285  63 249  60 233  58 226          60 237  61 243
//   of 3             64 252          64 252                  63 253
//   of 2             63 247  61 242  58 228  61 240  58 228  60 239  58 228  60 238
//   of 1             61 238  60 239  62 253  62 252  62 252  62      62 252  62
// (5 heads as 3 and 2: 71 294.  With 16 query heads 3, 5 and 6 KV heads take 70, 69 and
// 67 us by the rule, and 80, 91 and 80 in blocks of 3.)
//
// d 64, where a head is 64 bytes of a row: one block of up to 8 heads, above that blocks
// of 4 for an even count (every piece whole 128-byte lines), of one size for an odd one.
//   KV heads         3       5       6       7       8       10      11      12      14      15
//   one size, <= 8   60 234  61 239  62 241  61 237  58 224  63 266  66 267  61 240  61 253  61 251
//   blocks of 4              68 305  66 288  65 279  59 224  60 239  64 276  57 226  60 239  64 278
//   blocks of 2      78 348  74 341  61 240  72 337  59 235  60 240  72      - 252
// (5, 6 and 7 heads as 3 and 2, 3 and 3, 4 and 3 in the second row.  With 16 query heads
// blocks of 4 are better by 3 to 14 % for 12, 14 and 18, and worse by 3 for 10.)
template <int D>
constexpr int MOST_HEADS = 512 / D;
template <int D>
constexpr int block_heads(int num_kv_heads) {
    const auto blocks = [=](int heads) { return (num_kv_heads + heads - 1) / heads; };
    if constexpr (D == 64) {
        if (num_kv_heads > MOST_HEADS<D> && num_kv_heads % 2 == 0) return 4;
        return blocks(blocks(MOST_HEADS<D>));
    } else {
        for (int heads = MOST_HEADS<D>; heads > 1; heads /= 2)
            if ((blocks(heads) * heads - num_kv_heads) * 8 <= blocks(heads) * heads) return heads;
        return 1;
    }
}

}  // namespace fp8

namespace {

__device__ unsigned int fp8_timeouts = 0;  // one per translation unit

using split::align_up;
using split::cp_async_arrive;
using split::Cursor;
using split::guarded_wait;
using split::ld_s32;
using split::log2_up;
using split::raise_limit;
using split::row_at;
using split::Schedule;
using split::TILE;

template <int D>
constexpr int MAX_WARPS = D == 128 ? 8 : 16;
constexpr int MAX_STAGES = 8;

// How a CTA's warps and shared memory are laid out (set by the host).
struct Layout {
    int subs, hblocks;          // groups of HEADS warps, head blocks
    int stages;                 // of a ring
    int whole;                  // a group takes whole streams, at most one each: no schedule, no merge
    int off_bars, off_ring;
};

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(src) : "memory");
}

template <int D>
constexpr int stage_bytes_of(int heads) {  // the tile's records, and 32 scale words of K and V for each head
    return TILE * fp8::record_stride<D>(heads) + heads * TILE * 8;
}

}  // namespace

// HEADS: KV heads of a head block, one warp each (the last block may have fewer).
template <int D, int NG, int HEADS>
__global__ void __launch_bounds__(MAX_WARPS<D> * 32, 1)
    decode_fp8_kernel(const DecodeFp8Args args, const float scale_log2, const Layout lay) {
    using C = fp8::Head<D>;
    const DecodeArgs &a = args.d;
    const Fp8Layer &pool = args.pool;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_abort;
    constexpr int stride = fp8::record_stride<D>(HEADS);
    constexpr uint32_t stage_bytes = stage_bytes_of<D>(HEADS);
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads, G = Hq / Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = lay.stages;
    const uint32_t data_stride = (uint32_t)pool.data_stride, scale_stride = (uint32_t)pool.scale_stride;

    if ((int)threadIdx.x < lay.subs * stages) {  // full, empty of (ring, stage)
        const uint32_t b = smem_u32(smem + lay.off_bars) + threadIdx.x * 16u;
        mbar_init(b, 32u * HEADS);
        mbar_init(b + 8u, HEADS);
    }
    if (threadIdx.x == 0) s_abort = 0;
    fence_mbar_init();
    pdl_wait();
    pdl_launch_dependents();
    Schedule sch;
    sch.init(reinterpret_cast<int32_t *>(smem), a, lay.hblocks, (int)gridDim.x * lay.subs, lay.whole);
    if (sch.total == 0) return;

    // warp (sub, head): the ring of its group
    const int head_in = warp % HEADS, sub = warp / HEADS;
    const uint32_t bars = smem_u32(smem + lay.off_bars) + (uint32_t)(sub * stages) * 16u;
    const uint32_t ring = smem_u32(smem + lay.off_ring) + (uint32_t)(sub * stages) * stage_bytes;
    constexpr int v_off = HEADS * D, s_off = TILE * stride;

    // This warp fetches tokens head_in * MINE .. of a tile (the last warp
    // what is left); lane i holds the page-table entry of the tile's token i (past the end:
    // the last one's).
    constexpr int MINE = (TILE + HEADS - 1) / HEADS;
    const int32_t *table = nullptr;  // entry of the first token of the tile to fetch
    auto load_row = [&](int left) -> int { return ld_s32(table + min(lane, left - 1)); };
    // A token's K (or V) row of HEADS heads is up to 32 pieces of 16 bytes: one
    // instruction copies them, or those of several tokens.
    constexpr int LANES = 1 << log2_up(HEADS * D / 16), TOKS = 32 / LANES;
    const int piece = lane % LANES, sub_tok = lane / LANES;
    uint32_t in_at = 0, in_parity = 1;  // stage to fill; the first round finds every stage empty
    auto issue = [&](int hb, int raw) {
        const int row = min(max(raw, 0), a.num_rows - 1);
        const uint32_t bar = bars + in_at * 16u, to = ring + in_at * stage_bytes;
        const int h0 = hb * HEADS, nh = min(HEADS, Hkv - h0);
        guarded_wait(bar + 8u, in_parity, &s_abort, &fp8_timeouts);
        const uint8_t *ksrc = pool.k_data + h0 * D + piece * 16, *vsrc = pool.v_data + h0 * D + piece * 16;
#pragma unroll
        for (int i0 = 0; i0 < MINE; i0 += TOKS) {
            const int i = i0 + sub_tok, tok = head_in * MINE + i;
            const uint32_t e = __shfl_sync(0xffffffffu, row, tok & 31);
            const uint32_t dst = to + fp8::slot<D>(tok) * stride + piece * 16;
            if (piece * 16 < nh * D && (TILE % HEADS == 0 || (i < MINE && tok < TILE))) {
                cp_async_16(dst, row_at(ksrc, e, data_stride), 16);
                cp_async_16(dst + v_off, row_at(vsrc, e, data_stride), 16);
            }
        }
        if (head_in < nh) {
            const uint32_t blk = (uint32_t)row >> pool.block_log2, word = (uint32_t)(h0 + head_in) & ~3u;
            const uint32_t dst = to + s_off + head_in * (TILE * 8) + lane * 8;
            cp_async_4(dst, row_at(pool.k_scale + word, blk, scale_stride));
            cp_async_4(dst + 4, row_at(pool.v_scale + word, blk, scale_stride));
        }
        cp_async_arrive(bar);
        if (++in_at == (uint32_t)stages) {
            in_at = 0;
            in_parity ^= 1;
        }
    };

    fp8::Stream<D, NG> w;
    uint32_t at = 0, parity = 0;  // stage to use
    // where the lane reads in the first stage: K of token lane / 4, the scale
    // words, V of tokens 2 (lane % 4) and the next
    const int lg = lane >> 2, lt = lane & 3;
    const uint32_t rd_k = ring + head_in * D + fp8::slot<D>(lg) * stride + lt * C::QPT;
    const uint32_t rd_s = ring + s_off + head_in * (TILE * 8);
    const uint32_t rd_v0 = ring + v_off + head_in * D + fp8::slot<D>(2 * lt) * stride + lg * C::OPT;
    const uint32_t rd_v1 = ring + v_off + head_in * D + fp8::slot<D>(2 * lt + 1) * stride + lg * C::OPT;
    const int seg_step = (int)gridDim.x * lay.subs;
    // neighbouring ranges on different SMs: few ranges spread over all of them
    for (int seg = blockIdx.x + sub * (int)gridDim.x; seg < sch.nseg; seg += seg_step) {
        Cursor c, pc;  // the tile to use, the tile to fetch
        int use = sch.range(seg, c);  // tiles not used yet
        if (use == 0) {  // a whole stream without context: zeros
            const int head = c.hb * HEADS + head_in;
            if (head < Hkv)
                for (int i = lane; i < G * D / 8; i += 32)
                    st_v4(static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)c.r * Hq + head * G) * D + i * 8,
                          make_uint4(0u, 0u, 0u, 0u));
            continue;
        }
        // The tiles to fetch are those of pc until left reaches `stop`, then
        // `later` more of the streams behind it.
        pc = c;
        int stop, later = use;
        auto enter = [&]() {
            table = a.page_table + (int64_t)pc.r * a.pt_stride + (sch.len(pc.r) - pc.left);
            const int n = min(later, (pc.left + TILE - 1) / TILE);
            stop = pc.left - n * TILE;
            later -= n;
        };
        auto advance = [&]() -> int {  // the next tile to fetch; its page-table entry
            pc.left -= TILE;
            table += TILE;
            if (pc.left <= stop && later > 0) {
                sch.next_stream(pc);
                enter();
                // its queries, wanted when this tile is used
                const int head = pc.hb * HEADS + head_in;
                w.prefetch(a, (int64_t)pc.r * Hq + head * G, G, head < Hkv, lane);
            }
            return pc.left > stop ? load_row(pc.left) : 0;
        };
        enter();
        // the first two tiles' page-table entries at once, then one tile ahead
        int row = load_row(pc.left);
        for (int i = 0; i < stages - 1 && pc.left > stop; ++i) {
            const int now = row, now_hb = pc.hb;
            row = advance();
            issue(now_hb, now);
        }
        bool from_start = c.left == sch.len(c.r);
        // which of its stream's partials the range begins with (later streams begin here)
        int split = from_start ? 0 : seg - sch.range_of(sch.before(c.r, c.hb));
        while (use > 0) {  // a stream, or the range's part of it
            const int head = c.hb * HEADS + head_in;
            const bool live = head < Hkv;
            const int shift = (head & 3) * 8;
            w.open(live ? static_cast<const __nv_bfloat16 *>(a.q) + ((int64_t)c.r * Hq + head * G) * D : nullptr, G,
                   scale_log2, lane);
            const int n = min(use, (c.left + TILE - 1) / TILE), end = c.left - n * TILE;
            use -= n;
            for (; c.left > end; c.left -= TILE) {
                guarded_wait(bars + at * 16u, parity, &s_abort, &fp8_timeouts);
                const uint32_t st = at * stage_bytes;
                uint32_t pb[2][NG][2];
                if (live) {
                    w.scores(rd_k + st, rd_s + st, shift, stride, c.left, lane, pb);
                    w.values(rd_v0 + st, rd_v1 + st, stride, pb);
                }
                if (pc.left > stop) {  // into the stage of the tile before this one
                    issue(pc.hb, row);
                    row = advance();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bars + at * 16u + 8u);
                if (++at == (uint32_t)stages) {
                    at = 0;
                    parity ^= 1;
                }
            }
            const bool last = c.left <= 0;
            if (live) {
                w.close(a, (int64_t)c.r * Hq + head * G, G, from_start && last, split, lane);
                if (last && lane == 0 && !sch.whole) a.split_count[(int64_t)c.r * Hkv + head] = split + 1;
            }
            if (use > 0) sch.next_stream(c);
            from_start = true;
            split = 0;
        }
    }
    cp_async_wait<0>();  // nothing in flight when the CTA ends, even after a wait that ran out
}

namespace {

// The partials of the streams that were cut, joined: out = sum_k w_k O_k / sum_k
// w_k, w_k = e^(LSE_k - max LSE).  Rows that are whole hold their output already;
// empty requests get zeros.  Two kernels for the two ways a call is cut.  What
// bounds both are rounds of dependent loads, about 1 us each behind the launch:
// there are two, the counts with the first LSEs (read before it is known how many
// count) and the partials.
template <int D>
struct Acc {
    static constexpr int CPL = D / 32;  // channels per lane
    float c[CPL];
    __device__ __forceinline__ void load(const float *row, int lane) {
        if constexpr (CPL == 4) {
            const float4 v = *reinterpret_cast<const float4 *>(row + lane * 4);
            c[0] = v.x, c[1] = v.y, c[2] = v.z, c[3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2 *>(row + lane * 2);
            c[0] = v.x, c[1] = v.y;
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < CPL; ++i) c[i] = 0.f;
    }
    __device__ __forceinline__ void add(const Acc &x, float w) {
#pragma unroll
        for (int i = 0; i < CPL; ++i) c[i] += w * x.c[i];
    }
    __device__ __forceinline__ void write(void *out, int64_t row, int lane, float scale) const {
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(out) + row * D + lane * CPL;
#pragma unroll
        for (int i = 0; i < CPL; i += 2)
            *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16x2(c[i] * scale, c[i + 1] * scale);
    }
};

__device__ __forceinline__ int partials_of(const DecodeArgs &a, int row) {
    const int r = row / a.num_q_heads, g = (row - r * a.num_q_heads) / (a.num_q_heads / a.num_kv_heads);
    const int len = a.seq_lens[r], cnt = a.split_count[(int64_t)r * a.num_kv_heads + g];
    return split::clamp_len(len, a.pt_width) == 0 ? 0 : min(cnt, a.max_splits);  // no count without context
}

// Many rows of a few partials: a warp takes 2 rows, all their loads under way
// together (lane 16 i + k has the LSE of partial k of row i).  1024 rows in 3
// partials take 2.9 us behind the kernel before, 4 rows to a warp 5.7; 8192 rows
// 4.8 either way.
constexpr int MERGE_THREADS = 128, MERGE_ROWS = 2;
constexpr int MERGE_MANY = 4;  // ranges to a stream from which on a block takes a row
template <int D>
__global__ void __launch_bounds__(MERGE_THREADS) merge_rows_kernel(const DecodeArgs a) {
    constexpr int ROWS = MERGE_ROWS, MOST = 8, LANES = 32 / ROWS;  // rows, partials of one in flight, lanes of a row's LSEs
    const int rows = a.batch * a.num_q_heads, lane = threadIdx.x & 31, k = lane % LANES;
    const int row0 = (blockIdx.x * (MERGE_THREADS / 32) + (threadIdx.x >> 5)) * ROWS;
    pdl_wait();
    pdl_launch_dependents();
    if (row0 >= rows) return;
    const int mine = min(row0 + lane / LANES, rows - 1);
    const float *lse = a.ws_lse + (int64_t)mine * a.max_splits;
    const float l0 = k < a.max_splits ? lse[k] : 0.f;
    const int n = partials_of(a, mine);
    if (__all_sync(0xffffffffu, n == 1)) return;
    float top = k < n ? l0 : -INFINITY;
    for (int s = k + LANES; s < n; s += LANES) top = fmaxf(top, lse[s]);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float w0 = k < n ? __expf(l0 - top) : 0.f;
    int cnt[ROWS];
    Acc<D> x[ROWS][MOST];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        cnt[i] = row0 + i < rows ? __shfl_sync(0xffffffffu, n, LANES * i) : 1;
        const float *o = a.ws_o + (int64_t)(row0 + i) * a.max_splits * D;
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (cnt[i] > 1 && j < cnt[i]) x[i][j].load(o + j * D, lane);
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        Acc<D> acc;
        acc.clear();
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < MOST; ++j) {
            const float w = __shfl_sync(0xffffffffu, w0, LANES * i + j);
            if (j < cnt[i]) {
                sum += w;
                acc.add(x[i][j], w);
            }
        }
        const float peak = __shfl_sync(0xffffffffu, top, LANES * i);
        if (cnt[i] > MOST) {  // a long request among short ones
            const float *o = a.ws_o + (int64_t)(row0 + i) * a.max_splits * D;
            const float *l = a.ws_lse + (int64_t)(row0 + i) * a.max_splits;
            for (int j0 = MOST; j0 < cnt[i]; j0 += MOST) {
                Acc<D> y[MOST];
                float w[MOST];
#pragma unroll
                for (int j = 0; j < MOST; ++j)
                    if (j0 + j < cnt[i]) {
                        y[j].load(o + (j0 + j) * D, lane);
                        w[j] = l[j0 + j];
                    }
#pragma unroll
                for (int j = 0; j < MOST; ++j)
                    if (j0 + j < cnt[i]) {
                        const float e = __expf(w[j] - peak);
                        sum += e;
                        acc.add(y[j], e);
                    }
            }
        }
        if (cnt[i] != 1) acc.write(a.out, row0 + i, lane, cnt[i] == 0 ? 1.f : 1.f / sum);
    }
}

// A few rows of many partials: a block of 8 warps takes one row, a warp every
// 8th partial (one request of 32768 tokens, 152 partials a row: 20 us for the
// call, 28 with a warp a row).
template <int D>
__global__ void __launch_bounds__(256) merge_row_kernel(const DecodeArgs a) {
    constexpr int WARPS = 8, MOST = 8;
    __shared__ float s_acc[WARPS][D], s_sum[WARPS];
    const int row = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const float *lse = a.ws_lse + (int64_t)row * a.max_splits, *o = a.ws_o + (int64_t)row * a.max_splits * D;
    const float l0 = lane < a.max_splits ? lse[lane] : 0.f;
    const int n = partials_of(a, row);
    if (n == 1) return;
    float top = lane < n ? l0 : -INFINITY;
    for (int s = lane + 32; s < n; s += 32) top = fmaxf(top, lse[s]);
#pragma unroll
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    Acc<D> acc;
    acc.clear();
    float sum = 0.f;
    for (int j0 = warp; j0 < n; j0 += WARPS * MOST) {
        Acc<D> y[MOST];
        float w[MOST];
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (j0 + j * WARPS < n) {
                y[j].load(o + (j0 + j * WARPS) * D, lane);
                w[j] = lse[j0 + j * WARPS];
            }
#pragma unroll
        for (int j = 0; j < MOST; ++j)
            if (j0 + j * WARPS < n) {
                const float e = __expf(w[j] - top);
                sum += e;
                acc.add(y[j], e);
            }
    }
#pragma unroll
    for (int i = 0; i < Acc<D>::CPL; ++i) s_acc[warp][lane * Acc<D>::CPL + i] = acc.c[i];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (threadIdx.x < D / 2) {
        float lo = 0.f, hi = 0.f, all = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            lo += s_acc[w][2 * threadIdx.x];
            hi += s_acc[w][2 * threadIdx.x + 1];
            all += s_sum[w];
        }
        const float scale = n == 0 ? 1.f : 1.f / all;
        reinterpret_cast<uint32_t *>(a.out)[(int64_t)row * (D / 2) + threadIdx.x] = pack_bf16x2(lo * scale, hi * scale);
    }
}

template <int D, int NG, int HEADS>
cudaError_t launch_cfg(const DecodeFp8Args &args, cudaStream_t s) {
    const DecodeArgs &a = args.d;
    Layout lay;
    lay.hblocks = (a.num_kv_heads + HEADS - 1) / HEADS;
    auto kern = decode_fp8_kernel<D, NG, HEADS>;
    int optin = 0;
    cudaError_t e = raise_limit(kern, optin);
    if (e != cudaSuccess) return e;
    // as many groups as leave three stages to each
    constexpr int stage = stage_bytes_of<D>(HEADS);
    lay.subs = MAX_WARPS<D> / HEADS;
    lay.off_bars = align_up(split::schedule_ints(a.batch) * 4, 16);
    lay.off_ring = align_up(lay.off_bars + MAX_STAGES * lay.subs * 16, 128);
    lay.subs = std::min(lay.subs, (optin - lay.off_ring) / (3 * stage));
    if (lay.subs < 1) return cudaErrorInvalidConfiguration;
    lay.stages = std::min((optin - lay.off_ring) / (lay.subs * stage), MAX_STAGES);
    const size_t smem = (size_t)lay.off_ring + (size_t)lay.stages * lay.subs * stage;
    const int64_t sms = device_sm_count(), streams = (int64_t)a.batch * lay.hblocks;
    const int64_t wide = (a.pt_width + TILE - 1) / TILE;
    // The 4-bit decode's rule for leaving streams whole holds here too.  Whole / split in
    // a graph, 8 KV heads, d 128, 64 and 152 requests, in tables of 5, 8 and 12 tiles (us):
    //   all as long as the table       8.7/13.1 11.9/14.1 15.8/16.6   11.1/14.3 15.0/18.0 24.1/27.0
    //   one of them, the others 1 tile 8.4/7.9  11.0/8.3  14.7/9.6     8.8/10.8 11.4/10.8 14.9/11.9
    lay.whole = fp4::leave_whole(streams, sms * lay.subs, wide) && a.split_tokens == 0;
    // never more ranges than tiles could exist
    const int64_t max_tiles = streams * wide;
    const int64_t grid = std::max<int64_t>(1, std::min(sms, lay.whole ? streams : max_tiles));
    e = launch_pdl(kern, dim3((unsigned)grid), dim3(HEADS * lay.subs * 32), smem, s, args,
                   a.sm_scale * split::LOG2E, lay);
    if (e != cudaSuccess || lay.whole) return e;
    const int64_t rows = (int64_t)a.batch * a.num_q_heads;
    if (streams * MERGE_MANY < sms * lay.subs)
        return launch_pdl(merge_row_kernel<D>, dim3((unsigned)rows), dim3(256), 0, s, a);
    constexpr int per_cta = MERGE_THREADS / 32 * MERGE_ROWS;
    return launch_pdl(merge_rows_kernel<D>, dim3((unsigned)((rows + per_cta - 1) / per_cta)), dim3(MERGE_THREADS), 0, s, a);
}

}  // namespace

template <int D, int NG>
cudaError_t launch_decode_fp8_as(const DecodeFp8Args &a, cudaStream_t s) {
    switch (fp8::block_heads<D>(a.d.num_kv_heads)) {
        case 1: return launch_cfg<D, NG, 1>(a, s);
        case 2: return launch_cfg<D, NG, 2>(a, s);
        case 4: return launch_cfg<D, NG, 4>(a, s);
        default: break;
    }
    if constexpr (D == 64) {
        switch (fp8::block_heads<D>(a.d.num_kv_heads)) {
            case 3: return launch_cfg<D, NG, 3>(a, s);
            case 5: return launch_cfg<D, NG, 5>(a, s);
            case 6: return launch_cfg<D, NG, 6>(a, s);
            case 7: return launch_cfg<D, NG, 7>(a, s);
            case 8: return launch_cfg<D, NG, 8>(a, s);
            default: break;
        }
    }
    return cudaErrorInvalidValue;
}

template <int D, int NG>
cudaError_t read_fp8_timeouts_as(unsigned int *count) {
    return cudaMemcpyFromSymbol(count, fp8_timeouts, sizeof(unsigned int));
}

}  // namespace minisgl

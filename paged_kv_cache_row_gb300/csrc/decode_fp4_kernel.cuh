// decode_fp4_kernel.cuh -- split-KV GQA decode attention over the 4-bit paged pool.
//
//     out[r,h] = sum_j softmax_j(sm_scale <q[r,h], K_j>) V_j,   j < seq_len[r],
// K_j and V_j the values c * s * 2^exp of row page_table[r, j] (the pool's
// format is in the public header).  Split partials are merged by
// decode_fp4_merge_kernel.
//
// What bounds it: the K/V bytes, 2 * (d/2 + d/16) a token and KV head, 144 at
// d 128.  At the card's copy rate that is 43 elements a cycle and SM, so the
// arithmetic (decode_fp4.cuh) has to stay near one instruction per element,
// and the rows have to arrive without many requests: a head's row is only 64
// + 8 bytes, in two places each for K and V.
//
// Work: tiles of 32 tokens of one request and a block of up to 8 KV heads, one
// warp to a head, so a token's row of these heads (contiguous) is fetched as
// one piece.  A CTA (one per SM) has as many such groups of warps as fit 16
// warps, each with a range of tiles of its own.  The tiles of all requests are
// cut evenly over the groups of all CTAs: contiguous ranges whose lengths
// differ by at most one (in narrow tables a group may take a request whole:
// decode_fp4_plan.h).  The workspace's splits bound the ranges of a request and
// block of heads, which one request of 32768 tokens (64 query heads) shows: 96 us
// with 16, 53 with 32, 47 with 256.
//
// Loads: each group has a ring of three or more stages with a full and an
// empty mbarrier each.  The group's warps fetch a tile together, each its
// share of the tokens, in 16-byte cp.async pieces: a warp instruction covers a
// token's K row of eight heads (512 bytes at d 128), so few rows and lines are
// touched at a time.  Page-table entries are read a tile before the rows they
// name, and not looked at until then (a clamp right behind the load held its
// warp for the load's latency once per tile: 174 us where 156 were taken then).
// Rows past a request's end repeat its last row; their weights are zero.
//
// Measured (8 KV heads, d 128, warm): 256 requests of 1k to 8k tokens in
// single-row pages 148 us, 5.4 TB/s of algorithmic bytes; 32 of 8k to 32k in
// 64-row pages 136 us.  With the arithmetic left out 144 and 127, with the
// loads left out 137 and 129: the two nearly balance, so that every instruction
// of a tile counts (634 to 588 a warp took 152 and 143.5 us to these), and about
// 10 us are the start of the pipeline, the last ranges and the merge.
//
// Arrangements timed and not kept, on the first of these: every warp fetching
// its own head's 64- and 8-byte pieces 241 us; one CTA barrier per tile for
// the mbarriers 204 (174 then); one bulk copy (TMA) per row 396, about 41
// cycles a copy and SM, whatever its size; four producer warps with eight
// consumers and six stages 164, with sixteen consumers and registers shared
// out 151, but 1.5 to 2.5 times slower at 1 and 2 heads.  At 149: rows marked to
// be evicted first 153, two accumulators for Q K^T 150, its two blocks of 16
// tokens interleaved 152, the mbarriers inside the stages 151.
#pragma once
#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "decode_fp4.cuh"
#include "decode_fp4_plan.h"
#include "tcgen05.cuh"

namespace minisgl {

namespace {

__device__ unsigned int fp4_timeouts = 0;  // one per translation unit

using fp4::Cursor;
using fp4::Head;
using fp4::Schedule;
using fp4::TILE;

// Warps per CTA (one CTA per SM): 16 at up to 128 registers each; the 16-head
// form at d 128 needs more.
template <int D, int NG>
constexpr int MAX_WARPS = D == 128 && NG == 2 ? 8 : 16;
constexpr int MAX_STAGES = 8;
constexpr long long WAIT_LIMIT = 1000000000LL;  // SM cycles (about 0.5 s)

// How a CTA's warps and shared memory are laid out (set by the host).
struct Layout {
    int subs, hblocks;          // groups of HEADS warps, head blocks
    int stages;                 // of a ring
    int wide_scales;            // scale rows are 16-byte aligned
    int whole;                  // a group takes whole streams, at most one each: no schedule, no merge
    int off_bars, off_ring;
};

constexpr int log2_up(int x) { return x <= 1 ? 0 : 1 + log2_up((x + 1) / 2); }

// Bytes between the token records of `heads` heads.
template <int D>
__host__ __device__ constexpr int record_stride(int heads) {
    int s = (heads * 2 * (Head<D>::RB + Head<D>::SB) + 15) / 16 * 16;
    while (s % 128 != 32 && s % 128 != 96) s += 16;
    return s;
}

// Bounded wait: once one wait has run out, the CTA stops waiting altogether,
// so every warp reaches the end (the output is then garbage and counted).
__device__ __forceinline__ void guarded_wait(uint32_t b, uint32_t parity, volatile int *abort_flag) {
    if (mbar_try_wait(b, parity)) return;
    if (*abort_flag) return;
    if (!mbar_wait(b, parity, WAIT_LIMIT)) {
        *abort_flag = 1;
        atomicAdd(&fp4_timeouts, 1u);
    }
}

template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// base + row * stride, one multiply-add for each of K and V instead of a product and two sums
__device__ __forceinline__ const uint8_t *row_at(const uint8_t *base, uint32_t row, uint32_t stride) {
    const uint8_t *p;
    asm("mad.wide.u32 %0, %1, %2, %3;\n" : "=l"(p) : "r"(row), "r"(stride), "l"(base));
    return p;
}
// A coherent load (the step's slots may still be written when this kernel
// starts), and one that stays behind the copies it follows in the source: left
// to the compiler's order it took 148 us where 136 are taken.
__device__ __forceinline__ int ld_s32(const int32_t *p) {
    int v;
    asm volatile("ld.global.s32 %0, [%1];\n" : "=r"(v) : "l"(p));
    return v;
}
// One arrival on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

}  // namespace

// HEADS: KV heads of a head block, one warp each (the record stride and the
// copies' offsets are constants then; with them in registers 4 heads took 156
// us where 8 took 88 for the same bytes).  MULTI: there are several head
// blocks (the sources move with them and the last may have fewer heads).
template <int D, int NG, int HEADS, bool MULTI>
__global__ void __launch_bounds__(MAX_WARPS<D, NG> * 32, 1)
    decode_fp4_kernel(const DecodeFp4Args args, const float scale_log2, const float out_scale, const Layout lay) {
    using C = Head<D>;
    const DecodeArgs &a = args.d;
    const Fp4Layer &pool = args.pool;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_abort;
    constexpr int stride = record_stride<D>(HEADS);
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads, G = Hq / Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = lay.stages;
    constexpr uint32_t stage_bytes = TILE * stride;
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
    sch.init(reinterpret_cast<int32_t *>(smem), a, MULTI ? lay.hblocks : 1, (int)gridDim.x * lay.subs, lay.whole);
    if (sch.total == 0) return;

    // warp (sub, head): the ring of its group
    const int head_in = warp % HEADS, sub = warp / HEADS;
    const uint32_t bars = smem_u32(smem + lay.off_bars) + (uint32_t)(sub * stages) * 16u;
    const uint32_t ring = smem_u32(smem + lay.off_ring) + (uint32_t)(sub * stages) * stage_bytes;
    constexpr int v_off = HEADS * C::RB, sk_off = 2 * v_off, sv_off = sk_off + HEADS * C::SB;

    // This warp fetches `mine` tokens of a tile: a run of them where that is a
    // multiple of 8 tokens, else every HEADS-th.  Lane i holds the i-th one's
    // page-table entry (past the end: the last token's).
    constexpr bool RUN = HEADS <= 4 && TILE % HEADS == 0;
    constexpr int MOST = (TILE + HEADS - 1) / HEADS;
    const int mine = TILE % HEADS == 0 ? MOST : (TILE - head_in + HEADS - 1) / HEADS;
    const int my_tok = min(RUN ? head_in * MOST + lane : head_in + HEADS * lane, TILE - 1);
    auto slot_of = [&](int i) {  // of this warp's i-th token
        return RUN ? head_in * MOST + fp4::slot(i)
                   : HEADS == 8 ? fp4::slot(head_in) + 8 * i : fp4::slot(head_in + HEADS * i);
    };
    const int32_t *table = nullptr;  // entry of the first token of the tile to fetch
    auto load_row = [&](int left) -> int { return ld_s32(table + min(my_tok, left - 1)); };
    // The 16-byte pieces of a token's K and V rows are dealt to 2^LP lanes (K
    // and V in one instruction, or one each), so a lane's piece is the same for
    // every token; the same for the scales.
    constexpr int HALF = HEADS * C::RB / 16, PIECES = 2 * HALF;
    constexpr bool TWO = PIECES > 32;
    constexpr int LP = TWO ? 5 : log2_up(PIECES), TOKS = 32 >> LP;
    const int piece = lane & ((1 << LP) - 1), sub_tok = lane >> LP;
    const bool is_v = !TWO && piece >= HALF;
    const int off = !TWO && piece >= PIECES ? 1 << 30 : (is_v ? piece - HALF : piece) * 16;
    const uint8_t *ksrc = (is_v ? pool.v_data : pool.k_data) + off, *vsrc = pool.v_data + off;
    constexpr int WIDE = fp4::scale_piece(HEADS, C::SB);  // bytes of a scale piece
    const bool narrow = WIDE == 16 && !lay.wide_scales;
    constexpr int SHALF = HEADS * C::SB / WIDE, SPIECES = 2 * SHALF, SLP = log2_up(SPIECES), STOKS = 32 >> SLP;
    const int sp = lane & ((1 << SLP) - 1), ssub_tok = lane >> SLP;
    const bool s_is_v = sp >= SHALF;
    const int soff = sp >= SPIECES ? 1 << 30 : (s_is_v ? sp - SHALF : sp) * WIDE;
    const uint8_t *ssrc = (s_is_v ? pool.v_scale : pool.k_scale) + soff;
    // the head block that the sources above belong to, whether it has the lane's
    // data piece, and the bytes of the lane's scale piece in it (fewer than WIDE
    // only in a short last block; the first block is full)
    int in_hb = 0;
    bool have = off < HEADS * C::RB;
    int sbytes = fp4::piece_bytes(HEADS * C::SB, soff, WIDE);

    // the lane's first destinations in stage 0, kept in registers as the sources are
    uint32_t to_data = ring + slot_of(sub_tok) * stride + piece * 16;
    uint32_t to_scale = ring + slot_of(ssub_tok) * stride + sk_off + sp * WIDE;
    asm("" : "+r"(to_data), "+r"(to_scale));
    asm("" : "+l"(ksrc), "+l"(vsrc), "+l"(ssrc));
    uint32_t in_at = 0, in_parity = 1;  // stage to fill; the first round finds every stage empty
    auto issue = [&](int hb, int raw) {
        const int row = min(max(raw, 0), a.num_rows - 1);
        const uint32_t bar = bars + in_at * 16u, at_stage = in_at * stage_bytes;
        if (MULTI && hb != in_hb) {
            const int d = (hb - in_hb) * HEADS, nh = fp4::heads_of_block(Hkv, HEADS, hb);
            ksrc += d * C::RB;
            vsrc += d * C::RB;
            ssrc += d * C::SB;
            have = off < nh * C::RB;
            sbytes = fp4::piece_bytes(nh * C::SB, soff, WIDE);
            in_hb = hb;
        }
        guarded_wait(bar + 8u, in_parity, &s_abort);
#pragma unroll
        for (int i0 = 0; i0 < MOST; i0 += TOKS) {
            const int i = i0 + sub_tok;
            const uint32_t e = __shfl_sync(0xffffffffu, row, i & 31);
            // (8 heads: slot_of() is linear in i)
            const uint32_t to = to_data + at_stage +
                                (HEADS == 8 ? slot_of(i0) - slot_of(0) : slot_of(i) - slot_of(sub_tok)) * stride;
            if (i < mine && have) {
                cp_async_16(to, row_at(ksrc, e, data_stride), 16);
                if constexpr (TWO) cp_async_16(to + HALF * 16, row_at(vsrc, e, data_stride), 16);
            }
        }
#pragma unroll
        for (int i0 = 0; i0 < MOST; i0 += STOKS) {
            const int i = i0 + ssub_tok;
            const uint8_t *from = row_at(ssrc, __shfl_sync(0xffffffffu, row, i & 31), scale_stride);
            const uint32_t to = to_scale + at_stage + (slot_of(i) - slot_of(ssub_tok)) * stride;
            if (i < mine && sbytes > 0) {
                if constexpr (WIDE == 16) {
                    const int n = MULTI ? sbytes : 16;
                    if (narrow) {  // rows that do not start on 16 bytes: d/16 bytes at a time
                        for (int k = 0; k < n; k += C::SB) cp_async_small<C::SB>(to + k, from + k);
                    } else {
                        cp_async_16(to, from, n);  // reads n bytes
                    }
                } else {
                    cp_async_small<WIDE>(to, from);
                }
            }
        }
        cp_async_arrive(bar);
        if (++in_at == (uint32_t)stages) {
            in_at = 0;
            in_parity ^= 1;
        }
    };

    fp4::Stream<D, NG> w;
    uint32_t at = 0, parity = 0;  // stage to use
    const uint32_t my_k = ring + head_in * C::RB, my_s = ring + sk_off + head_in * C::SB;
    uint32_t rd[6];  // where the lane reads in the first stage
    w.addresses(my_k, my_s, my_k + v_off, my_s + (sv_off - sk_off), stride, lane, rd);
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
                // its queries, wanted when this tile is used (67 -> 64 us at 1000 requests of 17 to 300 tokens)
                w.prefetch(a, (int64_t)pc.r * Hq + (MULTI ? pc.hb * HEADS + head_in : head_in) * G, G,
                           !MULTI || pc.hb * HEADS + head_in < Hkv, lane);
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
            const int head = MULTI ? c.hb * HEADS + head_in : head_in;
            const bool live = !MULTI || head < Hkv;
            w.open(live ? static_cast<const __nv_bfloat16 *>(a.q) + ((int64_t)c.r * Hq + head * G) * D : nullptr, G,
                   scale_log2, lane);
            const int n = min(use, (c.left + TILE - 1) / TILE), end = c.left - n * TILE;
            use -= n;
            for (; c.left > end; c.left -= TILE) {
                guarded_wait(bars + at * 16u, parity, &s_abort);
                const uint32_t st = at * stage_bytes;
                uint32_t pb[2][NG][2];
                if (live) {
                    w.scores(rd[0] + st, rd[1] + st, stride, c.left, lane, pb);
                    w.values(rd[2] + st, rd[3] + st, rd[4] + st, rd[5] + st, stride, pb);
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
                w.close(a, (int64_t)c.r * Hq + head * G, G, from_start && last, split, out_scale, lane);
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

// Joins the partials of the streams that were cut, one warp per (request, query
// head) row: out = sum_k w_k O_k / sum_k w_k, w_k = e^(LSE_k - max LSE).  Rows
// that are whole hold their output already; empty requests get zeros.
//
// What bounds it are rounds of dependent loads, about 1 us each behind the
// launch, and how many rows are under way.  There are two rounds: the length
// and the count, then the LSEs and MOST partials.  MOST 16 takes 96 registers
// and so 2432 rows at once, MOST 4 takes 40 and three times as many: 16 takes
// 0.9 us less for 1024 rows in 2-3 partials, 1.5 less for 2048 rows in about 10,
// 2.7 more for 8192 rows in 2-3.
template <int D, int MOST>
__global__ void __launch_bounds__(128, MOST > 8 ? 4 : 12) decode_fp4_merge_kernel(const DecodeArgs a) {
    constexpr int CPL = D / 32;  // channels per lane
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    if (row >= a.batch * Hq) return;
    const int r = row / Hq, g = (row - r * Hq) / (Hq / Hkv);
    const int len = a.seq_lens[r], cnt = a.split_count[(int64_t)r * Hkv + g];
    const int n = fp4::clamp_len(len, a.pt_width) == 0 ? 0 : min(cnt, a.max_splits);  // no count without context
    if (n == 1) return;
    const int64_t base = (int64_t)row * a.max_splits;
    const float l0 = lane < n ? a.ws_lse[base + lane] : -INFINITY;
    float M = l0;
    for (int s = 32 + lane; s < n; s += 32) M = fmaxf(M, a.ws_lse[base + s]);
    const float *src = a.ws_o + base * D + lane * CPL;  // of partial k at src + k * D
    float acc[CPL], tot = n == 0 ? 1.f : 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) acc[c] = 0.f;
    for (int k0 = 0; k0 < n; k0 += MOST) {
        float x[MOST][CPL];
#pragma unroll
        for (int k = 0; k < MOST; ++k)
            if (k0 + k < n) {
                if constexpr (CPL == 4) {
                    const float4 v = *reinterpret_cast<const float4 *>(src + (k0 + k) * D);
                    x[k][0] = v.x, x[k][1] = v.y, x[k][2] = v.z, x[k][3] = v.w;
                } else {
                    const float2 v = *reinterpret_cast<const float2 *>(src + (k0 + k) * D);
                    x[k][0] = v.x, x[k][1] = v.y;
                }
            }
        if (k0 == 0) {  // while the first rows come
#pragma unroll
            for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        }
        // the weights, in the first MOST lanes
        const float w = lane < MOST && k0 + lane < n ? __expf((k0 ? a.ws_lse[base + k0 + lane] : l0) - M) : 0.f;
#pragma unroll
        for (int k = 0; k < MOST; ++k)
            if (k0 + k < n) {
                const float wk = __shfl_sync(0xffffffffu, w, k);
                tot += wk;
#pragma unroll
                for (int c = 0; c < CPL; ++c) acc[c] += wk * x[k][c];
            }
    }
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (int64_t)row * D + lane * CPL;
    const float inv = 1.f / tot;
#pragma unroll
    for (int c = 0; c < CPL; c += 2)
        *reinterpret_cast<uint32_t *>(out + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
}

// The kernel's shared-memory limit raised to the device's, once per device.
template <typename K>
cudaError_t raise_limit(K kernel, int &optin) {
    struct Entry { const void *fn; int dev, optin; };
    static std::mutex mu;
    static Entry cache[64];
    static int used = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < used; ++i)
        if (cache[i].fn == (const void *)kernel && cache[i].dev == dev) {
            optin = cache[i].optin;
            return cudaSuccess;
        }
    cudaFuncAttributes fa;
    e = cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, kernel);
    if (e == cudaSuccess) {
        optin -= (int)fa.sharedSizeBytes;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, optin);
    }
    if (e != cudaSuccess) {
        cudaGetLastError();  // do not leave the failure for the next caller to find
        return e;
    }
    if (used < 64) cache[used++] = {(const void *)kernel, dev, optin};
    return cudaSuccess;
}

int align_up(int x, int a) { return (x + a - 1) / a * a; }

template <int D, int NG, int HEADS>
cudaError_t launch_cfg(const DecodeFp4Args &args, cudaStream_t s) {
    const DecodeArgs &a = args.d;
    const Fp4Layer &p = args.pool;
    Layout lay;
    lay.hblocks = (a.num_kv_heads + HEADS - 1) / HEADS;
    lay.wide_scales = p.scale_stride % 16 == 0 &&
                      ((reinterpret_cast<uintptr_t>(p.k_scale) | reinterpret_cast<uintptr_t>(p.v_scale)) & 15u) == 0;
    // more than 8 heads come in blocks of 5 to 8
    auto kern = HEADS > 4 && lay.hblocks > 1 ? decode_fp4_kernel<D, NG, HEADS, (HEADS > 4)>
                                             : decode_fp4_kernel<D, NG, HEADS, false>;
    int optin = 0;
    cudaError_t e = raise_limit(kern, optin);
    if (e != cudaSuccess) return e;
    // as many groups as leave three stages to each
    constexpr int stage = TILE * record_stride<D>(HEADS);
    lay.subs = MAX_WARPS<D, NG> / HEADS;
    lay.off_bars = align_up(fp4::schedule_ints(a.batch) * 4, 16);
    lay.off_ring = align_up(lay.off_bars + MAX_STAGES * lay.subs * 16, 128);
    lay.subs = std::min(lay.subs, (optin - lay.off_ring) / (3 * stage));
    if (lay.subs < 1) return cudaErrorInvalidConfiguration;
    lay.stages = std::min((optin - lay.off_ring) / (lay.subs * stage), MAX_STAGES);
    const size_t smem = (size_t)lay.off_ring + (size_t)lay.stages * lay.subs * stage;
    const int64_t sms = device_sm_count(), streams = (int64_t)a.batch * lay.hblocks;
    const int64_t wide = (a.pt_width + TILE - 1) / TILE;
    lay.whole = fp4::leave_whole(streams, sms * lay.subs, wide) && a.split_tokens == 0;
    // never more ranges than tiles could exist
    const int64_t max_tiles = streams * wide;
    const int64_t grid = std::max<int64_t>(1, std::min(sms, lay.whole ? streams : max_tiles));
    e = launch_pdl(kern, dim3((unsigned)grid), dim3(HEADS * lay.subs * 32), smem, s, args,
                   a.sm_scale * fp4::LOG2E * ldexpf(1.f, p.k_exp), ldexpf(1.f, p.v_exp), lay);
    if (e != cudaSuccess || lay.whole) return e;
    const int64_t rows = (int64_t)a.batch * a.num_q_heads;  // up to 4 CTAs of 4 an SM: the wide form
    return launch_pdl(rows <= 16 * sms ? decode_fp4_merge_kernel<D, 16> : decode_fp4_merge_kernel<D, 4>,
                      dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, s, a);
}

}  // namespace

template <int D, int NG>
cudaError_t launch_decode_fp4_as(const DecodeFp4Args &a, cudaStream_t s) {
    switch (fp4::block_heads(a.d.num_kv_heads)) {
        case 1: return launch_cfg<D, NG, 1>(a, s);
        case 2: return launch_cfg<D, NG, 2>(a, s);
        case 3: return launch_cfg<D, NG, 3>(a, s);
        case 4: return launch_cfg<D, NG, 4>(a, s);
        case 5: return launch_cfg<D, NG, 5>(a, s);
        case 6: return launch_cfg<D, NG, 6>(a, s);
        case 7: return launch_cfg<D, NG, 7>(a, s);
        default: return launch_cfg<D, NG, 8>(a, s);
    }
}

template <int D, int NG>
cudaError_t read_fp4_timeouts_as(unsigned int *count) {
    return cudaMemcpyFromSymbol(count, fp4_timeouts, sizeof(unsigned int));
}

}  // namespace minisgl

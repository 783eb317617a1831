// decode_fp4.cu -- split-KV GQA decode attention over the 4-bit paged pool.
//
//     out[r,h] = sum_j softmax_j(sm_scale <q[r,h], K_j>) V_j,   j < seq_len[r],
// K_j and V_j the values c * s * 2^exp of row page_table[r, j] (the pool's
// format is in the public header).  Split partials are merged by
// decode_merge_kernel, as for the bf16 pool.
//
// What bounds it: the K/V bytes, 2 * (d/2 + d/16) a token and KV head, 144 at
// d 128.  At the card's copy rate that is 43 elements a cycle and SM, so the
// arithmetic (decode_fp4.cuh) has to stay near one instruction per element,
// and the rows have to arrive without many requests: a head's row is only 64
// + 8 bytes, in two places each for K and V.
//
// Work: tiles of 32 tokens of one request and up to 16 KV heads, one warp to
// a head, so a token's row of all heads (contiguous) is fetched as one piece.
// With fewer heads a CTA has several such groups of warps, each with a range
// of tiles of its own.  The tiles of all requests are cut evenly over the
// groups of all CTAs: contiguous ranges whose lengths differ by at most one.
//
// Loads: each group has a ring of stages with a full and an empty mbarrier
// each.  The group's warps fetch a tile together, each its share of the
// tokens, in 16-byte cp.async pieces: a warp instruction covers a token's K
// row of eight heads (512 bytes at d 128), so few rows and lines are touched
// at a time.  Page-table entries are read a tile before the rows they name.
// Rows past a request's end repeat its last row; their weights are zero.
//
// Arrangements timed and not kept, 256 requests of 1k to 8k tokens (8 KV
// heads, d 128; this one takes 156 us): every warp fetching its own head's
// 64- and 8-byte pieces 241; one barrier per tile instead of the mbarriers
// 204 (174 then); one bulk copy (TMA) per row 396, about 41 cycles a copy and
// SM, whatever its size; four producer warps, eight consumers and six stages
// 164.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "decode_fp4.cuh"
#include "tcgen05.cuh"

namespace minisgl {

__device__ unsigned int g_fp4_timeouts = 0;

namespace {

using fp4::Cursor;
using fp4::Head;
using fp4::Schedule;
using fp4::TILE;

// Warps per CTA (one CTA per SM): 16 at up to 128 registers each; the 16-head
// form at d 128 needs more.
template <int D, int NG>
constexpr int MAX_WARPS = D == 128 && NG == 2 ? 8 : 16;
constexpr int MAX_STAGES = 8;
#ifndef WW
#define WW 256
#endif
constexpr int WHOLE_WIDTH = WW;  // widest page table whose streams may be left whole
constexpr long long WAIT_LIMIT = 1000000000LL;  // SM cycles (about 0.5 s)

// How a CTA's warps and shared memory are laid out (set by the host).
struct Layout {
    int heads, subs, hblocks;   // KV heads at a time, groups of warps, head blocks
    int stages, stride;         // stages of a ring, bytes between token records
    int scale_bytes;            // piece of a scale row that one copy takes: 16, or d/16
    int whole;                  // a group takes whole streams, at most one each: no schedule, no merge
    int off_bars, off_ring;
};

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
        atomicAdd(&g_fp4_timeouts, 1u);
    }
}

template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
// One arrival on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

}  // namespace

// HEADS: 8 when there are 8 KV heads and their scales are 16-byte pieces (the
// record stride is a constant then, and a warp's share of a tile 4 tokens in
// 9 copies at d 128), else 0.
template <int D, int NG, int HEADS>
__global__ void __launch_bounds__(MAX_WARPS<D, NG> * 32, 1)
    decode_fp4_kernel(const DecodeFp4Args args, const float scale_log2, const float out_scale, const Layout lay) {
    using C = Head<D>;
    const DecodeArgs &a = args.d;
    const Fp4Layer &pool = args.pool;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int s_abort;
    const int heads = HEADS ? HEADS : lay.heads, stride = HEADS ? record_stride<D>(HEADS) : lay.stride;
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads, G = Hq / Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stages = lay.stages;
    const uint32_t stage_bytes = TILE * stride;
    const uint32_t data_stride = (uint32_t)pool.data_stride, scale_stride = (uint32_t)pool.scale_stride;

    if ((int)threadIdx.x < lay.subs * stages) {  // full, empty of (ring, stage)
        const uint32_t b = smem_u32(smem + lay.off_bars) + threadIdx.x * 16u;
        mbar_init(b, 32u * (uint32_t)heads);
        mbar_init(b + 8u, (uint32_t)heads);
    }
    if (threadIdx.x == 0) s_abort = 0;
    fence_mbar_init();
    pdl_wait();
    pdl_launch_dependents();
    Schedule sch;
    sch.init(reinterpret_cast<int32_t *>(smem), a, lay.hblocks, (int64_t)gridDim.x * lay.subs,
             lay.whole);
    if (sch.total == 0) return;

    // warp (sub, head): the ring of its group
    const int head_in = warp % heads, sub = warp / heads;
    const uint32_t bars = smem_u32(smem + lay.off_bars) + (uint32_t)(sub * stages) * 16u;
    const uint32_t ring = smem_u32(smem + lay.off_ring) + (uint32_t)(sub * stages) * stage_bytes;
    const int v_off = heads * C::RB, sk_off = 2 * heads * C::RB, sv_off = sk_off + heads * C::SB;

    // This warp fetches tokens head_in + heads * i of a tile, i < mine; lane i
    // holds the i-th one's physical row (past the end: the last token's).
    const int mine = HEADS ? TILE / 8 : (TILE - head_in + heads - 1) / heads;
    const int my_tok = min(head_in + heads * lane, TILE - 1);
    const int32_t *table = nullptr;  // entry of the first token of the tile to fetch
    auto load_row = [&](int left) -> int {
        return __ldg(table + min(my_tok, left - 1));
    };
    // The pieces of a token's K and V rows are dealt to lanes in powers of two:
    // 2^lp >= pieces lanes to a token (or all 32, several times), and the same
    // for the scales.  A lane's piece is the same for every token.
    const int pieces = 2 * heads * C::RB / 16, half = pieces / 2;
    const int lp = pieces >= 32 ? 5 : 32 - __clz(pieces - 1), times = (pieces + 31) / 32;
    const int spieces = 2 * heads * C::SB / lay.scale_bytes, shalf = spieces / 2;
    const int slp = HEADS ? (D == 128 ? 3 : 2) : 32 - __clz(spieces - 1);
    const int sub_tok = lane >> lp, piece0 = lane & ((1 << lp) - 1);
    const int ssub_tok = lane >> slp, spiece = lane & ((1 << slp) - 1);
    const bool s_isv = spiece >= shalf;
    const int soff = (s_isv ? spiece - shalf : spiece) * lay.scale_bytes;
    const uint8_t *const ssrc = (s_isv ? pool.v_scale : pool.k_scale) + soff;
    const uint32_t sdst = sk_off + spiece * lay.scale_bytes;
    // 8 heads: this lane's piece of K (or, at d 64, of K or V), and where its pieces go
    const uint8_t *const ksrc = (D == 64 && lane >= 16 ? pool.v_data - 256 : pool.k_data) + lane * 16;
    const uint8_t *const vsrc = pool.v_data + lane * 16;
    const uint32_t kto = fp4::slot(head_in) * stride + lane * 16;
    const uint32_t sto = fp4::slot(head_in + 8 * ssub_tok) * stride + sdst;

    uint32_t in_at = 0, in_parity = 1;  // stage to fill; the first round finds every stage empty
    auto issue = [&](int hb, int raw) {
        const int row = min(max(raw, 0), a.num_rows - 1);
        const uint32_t bar = bars + in_at * 16u, dst = ring + in_at * stage_bytes;
        guarded_wait(bar + 8u, in_parity, &s_abort);
        if constexpr (HEADS == 8) {
#pragma unroll
            for (int i = 0; i < TILE / 8; ++i) {
                const uint64_t e = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, row, i) * data_stride;
                cp_async_16(dst + kto + 8 * i * stride, ksrc + e, 16);
                if constexpr (D == 128) cp_async_16(dst + kto + 8 * i * stride + 8 * C::RB, vsrc + e, 16);
            }
            const uint64_t e = (uint64_t)(uint32_t)__shfl_sync(0xffffffffu, row, ssub_tok) * scale_stride;
            if (D == 128 || lane < 16) cp_async_16(dst + sto, ssrc + e, 16);
        } else {
            const int h0 = hb * heads, nh = min(heads, Hkv - h0);
            for (int i0 = 0; i0 < mine; i0 += 1 << (5 - lp)) {
                const int i = i0 + sub_tok;
                const int rr = __shfl_sync(0xffffffffu, row, i);
                const uint64_t e = (uint64_t)(uint32_t)rr * data_stride + h0 * C::RB;
                const uint32_t to = dst + fp4::slot(head_in + heads * i) * stride;
                for (int k = 0; k < times; ++k) {
                    const int piece = piece0 + 32 * k;
                    const bool isv = piece >= half;
                    const int off = (isv ? piece - half : piece) * 16;
                    if (i < mine && piece < pieces && off < nh * C::RB)
                        cp_async_16(to + piece * 16, (isv ? pool.v_data : pool.k_data) + e + off, 16);
                }
            }
            for (int i0 = 0; i0 < mine; i0 += 1 << (5 - slp)) {
                const int i = i0 + ssub_tok;
                const int rr = __shfl_sync(0xffffffffu, row, i);
                const uint8_t *src = ssrc + (uint64_t)(uint32_t)rr * scale_stride + h0 * C::SB;
                const uint32_t to = dst + fp4::slot(head_in + heads * i) * stride + sdst;
                if (i < mine && spiece < spieces && soff < nh * C::SB) {
                    if (lay.scale_bytes == 16) cp_async_16(to, src, 16);
                    else cp_async_small<C::SB>(to, src);
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
    const int64_t seg_step = (int64_t)gridDim.x * lay.subs;
    // neighbouring ranges on different SMs: few ranges spread over all of them
    for (int64_t seg = blockIdx.x + (int64_t)sub * gridDim.x; seg < sch.nseg; seg += seg_step) {
        int t0, t1;
        Cursor c, pc;  // the tile to use, the tile to fetch
        if (lay.whole) {
            c.r = (int)(seg / lay.hblocks);
            c.hb = (int)(seg - (int64_t)c.r * lay.hblocks);
            c.left = sch.len(c.r);
            t0 = 0;
            t1 = (c.left + TILE - 1) / TILE;
            if (t1 == 0) {  // no context: zeros
                const int head = c.hb * heads + head_in;
                if (head < Hkv)
                    for (int i = lane; i < G * D / 8; i += 32)
                        st_v4(static_cast<__nv_bfloat16 *>(a.out) + ((int64_t)c.r * Hq + head * G) * D + i * 8,
                              make_uint4(0u, 0u, 0u, 0u));
                continue;
            }
        } else {
            t0 = sch.begin(seg);
            t1 = sch.begin(seg + 1);
            sch.locate(c, t0);
        }
        pc = c;
        auto set_table = [&]() { table = a.page_table + (int64_t)pc.r * a.pt_stride + (sch.len(pc.r) - pc.left); };
        auto fetch_next = [&]() {  // only called when a next tile exists
            pc.left -= TILE;
            table += TILE;
            if (pc.left <= 0) {
                sch.next_stream(pc);
                set_table();
            }
        };
        set_table();
        int todo = t1 - t0;  // tiles not asked for yet
        // the first two tiles' page-table entries at once, then one tile ahead
        int row = load_row(pc.left), hb = pc.hb;
        for (int i = 0; i < stages - 1 && todo > 0; ++i) {
            const int now = row, now_hb = hb;
            if (--todo > 0) {
                fetch_next();
                row = load_row(pc.left);
                hb = pc.hb;
            }
            issue(now_hb, now);
        }
        bool open = true, from_start = c.left == sch.len(c.r);
        for (int t = t0; t < t1; ++t) {
            const int head = HEADS ? head_in : c.hb * heads + head_in;
            const bool live = HEADS || head < Hkv;
            if (open) {
                open = false;
                w.open(live ? static_cast<const __nv_bfloat16 *>(a.q) + ((int64_t)c.r * Hq + head * G) * D : nullptr, G,
                       scale_log2, lane);
            }
            guarded_wait(bars + at * 16u, parity, &s_abort);
            const uint32_t st = at * stage_bytes;
            uint32_t pb[2][NG][2];
            if (live) {
                w.scores(my_k + st, my_s + st, stride, c.left, lane, pb);
                w.values(my_k + st + v_off, my_s + st + (sv_off - sk_off), stride, lane, pb);
            }
            if (todo > 0) {
                issue(hb, row);  // into the stage of the tile before this one
                if (--todo > 0) {
                    fetch_next();
                    row = load_row(pc.left);  // for the next iteration
                    hb = pc.hb;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bars + at * 16u + 8u);
            if (++at == (uint32_t)stages) {
                at = 0;
                parity ^= 1;
            }
            c.left -= TILE;
            if (c.left <= 0 || t + 1 == t1) {  // end of the stream or of the range
                const bool last = c.left <= 0;
                if (live) {
                    const bool whole = from_start && last;
                    const int split = whole ? 0 : (int)(seg - sch.range_of(sch.before(c.r, c.hb)));
                    w.close(a, (int64_t)c.r * Hq + head * G, G, whole, split, out_scale, lane);
                    if (last && lane == 0 && !lay.whole) a.split_count[(int64_t)c.r * Hkv + head] = split + 1;
                }
                if (t + 1 < t1) sch.next_stream(c);
                open = from_start = true;
            }
        }
    }
    cp_async_wait<0>();  // nothing in flight when the CTA ends, even after a wait that ran out
}

namespace {

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
cudaError_t launch_cfg(const DecodeFp4Args &args, Layout lay, cudaStream_t s) {
    using C = Head<D>;
    const DecodeArgs &a = args.d;
    const Fp4Layer &p = args.pool;
    lay.subs = MAX_WARPS<D, NG> / lay.heads;
    lay.stride = record_stride<D>(lay.heads);
    const int sb = lay.heads * C::SB, sb_last = (a.num_kv_heads - (lay.hblocks - 1) * lay.heads) * C::SB;
    const bool wide = sb % 16 == 0 && sb_last % 16 == 0 && p.scale_stride % 16 == 0 &&
                      ((reinterpret_cast<uintptr_t>(p.k_scale) | reinterpret_cast<uintptr_t>(p.v_scale)) & 15u) == 0;
    lay.scale_bytes = wide ? 16 : C::SB;
    lay.off_bars = align_up(fp4::schedule_ints(a.batch) * 4, 16);
    lay.off_ring = align_up(lay.off_bars + MAX_STAGES * lay.subs * 16, 128);
    auto kern = decode_fp4_kernel<D, NG, HEADS>;
    int optin = 0;
    cudaError_t e = raise_limit(kern, optin);
    if (e != cudaSuccess) return e;
    lay.stages = (optin - lay.off_ring) / (lay.subs * TILE * lay.stride);
    if (lay.stages > MAX_STAGES) lay.stages = MAX_STAGES;
    if (lay.stages < 2) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)lay.off_ring + (size_t)lay.stages * lay.subs * TILE * lay.stride;
    // Where every stream can have a group of its own and is short, it is left
    // whole: no schedule to sum, no partials and no merge launch.
    const int64_t sms = device_sm_count(), streams = (int64_t)a.batch * lay.hblocks;
    lay.whole = a.pt_width <= WHOLE_WIDTH && streams <= sms * lay.subs && a.split_tokens == 0;
    // never more ranges than tiles could exist
    const int64_t max_tiles = streams * ((a.pt_width + TILE - 1) / TILE);
    const int64_t grid = std::max<int64_t>(1, std::min(sms, lay.whole ? streams : max_tiles));
    e = launch_pdl(kern, dim3((unsigned)grid), dim3(lay.heads * lay.subs * 32), smem, s, args,
                   a.sm_scale * fp4::LOG2E * ldexpf(1.f, p.k_exp), ldexpf(1.f, p.v_exp), lay);
    if (e != cudaSuccess || lay.whole) return e;
    return launch_decode_merge(a, s);
}

template <int D, int NG>
cudaError_t launch_heads(const DecodeFp4Args &a, cudaStream_t s) {
    Layout lay{};
    constexpr int most = MAX_WARPS<D, NG>;
    lay.hblocks = (a.d.num_kv_heads + most - 1) / most;
    lay.heads = (a.d.num_kv_heads + lay.hblocks - 1) / lay.hblocks;
    const Fp4Layer &p = a.pool;
    const bool wide = p.scale_stride % 16 == 0 &&
                      ((reinterpret_cast<uintptr_t>(p.k_scale) | reinterpret_cast<uintptr_t>(p.v_scale)) & 15u) == 0;
    return p.num_kv_heads == 8 && wide ? launch_cfg<D, NG, 8>(a, lay, s) : launch_cfg<D, NG, 0>(a, lay, s);
}

}  // namespace

cudaError_t launch_decode_fp4(const DecodeFp4Args &a, cudaStream_t s) {
    if (a.d.batch == 0) return cudaSuccess;
    const int G = a.d.num_q_heads / a.d.num_kv_heads;
    if (a.d.head_dim == 128) return G <= 8 ? launch_heads<128, 1>(a, s) : launch_heads<128, 2>(a, s);
    return G <= 8 ? launch_heads<64, 1>(a, s) : launch_heads<64, 2>(a, s);
}

cudaError_t read_fp4_timeouts(unsigned int *count) {
    return cudaMemcpyFromSymbol(count, g_fp4_timeouts, sizeof(unsigned int));
}

}  // namespace minisgl

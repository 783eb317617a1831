// decode_split.cuh -- what the decode kernels of the quantised pools (4 and 8
// bits) share: the cut of a batch's tiles into ranges, the queries' layout and
// bounded waits on their rings; and the kernel that joins the 4-bit decode's split
// partials (the 8-bit one's are beside it).
#pragma once
#include <algorithm>
#include <cstdint>
#include <mutex>

#include "fp4.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace minisgl {
namespace split {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ int clamp_len(int n, int w) { return min(max(n, 0), w); }

// Bounded wait: once one wait has run out, the CTA stops waiting altogether,
// so every warp reaches the end (the output is then garbage and counted).
constexpr long long WAIT_LIMIT = 1000000000LL;  // SM cycles (about 0.5 s)
__device__ __forceinline__ void guarded_wait(uint32_t b, uint32_t parity, volatile int *abort_flag,
                                             unsigned int *timeouts) {
    if (mbar_try_wait(b, parity)) return;
    if (*abort_flag) return;
    if (!mbar_wait(b, parity, WAIT_LIMIT)) {
        *abort_flag = 1;
        atomicAdd(timeouts, 1u);
    }
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
// Transpose an 8x8 b16 matrix held in the mma fragment layout.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
    return y;
}
// One arrival on `bar` when this thread's cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// Queries h0 + lane / 4 of a group (q: G rows of D; null or past G leaves
// zeros) as the B operands of the products with K: lane t of a row's four has
// channels [t d/4, (t+1) d/4), in fp16 after an exact power-of-two scaling of
// the head.  Returns what undoes it, times scale_log2.
template <int D>
__device__ __forceinline__ float load_queries(const __nv_bfloat16 *q, int h0, int G, float scale_log2, int lane,
                                              uint32_t (&qb)[D / 16][2]) {
    constexpr int QPT = D / 4;
    const int h = h0 + (lane >> 2);
    uint32_t w[QPT / 2];  // this lane's channels of head h
#pragma unroll
    for (int i = 0; i < QPT / 2; ++i) w[i] = 0u;
    if (h < G && q) {
        const __nv_bfloat16 *src = q + h * D + (lane & 3) * QPT;
#pragma unroll
        for (int i = 0; i < QPT / 8; ++i) {
            const uint4 v = reinterpret_cast<const uint4 *>(src)[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < QPT / 2; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    m = max(m & 0xffffu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    // largest |q| in [2^(b-127), 2^(b-126)): times 2^(141-b) it is below 2^15
    const int b = max((int)(m >> 7), 20);
    const float up = __int_as_float((268 - b) << 23);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t x = w[2 * ks + i];
            qb[ks][i] = f32_to_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
        }
    return __int_as_float((b - 14) << 23) * scale_log2;
}

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

namespace {  // one kernel per translation unit that launches it

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
__global__ void __launch_bounds__(128, MOST > 8 ? 4 : 12) decode_merge_kernel(const DecodeArgs a) {
    constexpr int CPL = D / 32;  // channels per lane
    const int Hkv = a.num_kv_heads, Hq = a.num_q_heads;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    if (row >= a.batch * Hq) return;
    const int r = row / Hq, g = (row - r * Hq) / (Hq / Hkv);
    const int len = a.seq_lens[r], cnt = a.split_count[(int64_t)r * Hkv + g];
    const int n = clamp_len(len, a.pt_width) == 0 ? 0 : min(cnt, a.max_splits);  // no count without context
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

}  // namespace

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

inline int align_up(int x, int a) { return (x + a - 1) / a * a; }
constexpr int log2_up(int x) { return x <= 1 ? 0 : 1 + log2_up((x + 1) / 2); }

}  // namespace split
}  // namespace minisgl

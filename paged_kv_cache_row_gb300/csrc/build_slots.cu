// build_slots.cu -- page-table rows, out_loc, positions, offsets and lengths
// of one step, from the requests' lengths.
//
// Mathematics (mini-sglang-learn, paged KV pool chapter: the pages of
// [cached_len, device_len) are allocated and written into the page table;
// sglang guide: out_cache_loc, positions): two exclusive prefix sums over the
// requests, of the new tokens (q_offsets) and of the new pages (the place in
// the free list where a request's pages begin), and then one row per token.
//
// One launch and no wait between its blocks: every block sums all lengths
// itself (8 bytes a request, at most 32 KB, which come from L2), and the
// tokens are spread over the blocks.  A token finds its request by binary
// search in the prefix sums in shared memory.  The sums saturate at 2^30, far
// above what total_tokens and num_free allow, so that no lengths overflow.
#include "kernels.h"
#include "ptx.cuh"

namespace minisgl {

namespace {

constexpr int SLOT_THREADS = 256;
constexpr int SLOT_U = 4;  // tokens per thread
constexpr int SLOT_MAX_BATCH = 4096;
constexpr int32_t SLOT_SAT = 1 << 30;

// 0 <= a, b <= 2^30: the sum needs 32 bits without a sign
__device__ __forceinline__ int sat_add(int a, int b) {
    return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)SLOT_SAT);
}

}  // namespace

// shift >= 0: page_size is 1 << shift
__global__ void __launch_bounds__(SLOT_THREADS) build_slots_kernel(SlotArgs a, int shift) {
    __shared__ int s_off[SLOT_MAX_BATCH + 1], s_page[SLOT_MAX_BATCH + 1];
    __shared__ int s_warp[2][SLOT_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int B = a.batch, W = a.pt_width;
    auto page_of = [&](int p) { return shift >= 0 ? p >> shift : p / a.page_size; };
    // pages that cover the first p positions
    auto pages_for = [&](int p) { return page_of(p) + (p - page_of(p) * a.page_size ? 1 : 0); };
    // No early start for the next kernel: the library's other kernels read the
    // page table, out_loc, positions and lengths with non-coherent loads, whose
    // memory must not change while they are resident.
    pdl_wait();

    // each thread sums `per` consecutive requests, then a block-wide scan
    const int per = (B + SLOT_THREADS - 1) / SLOT_THREADS;
    const int r0 = min(tid * per, B), r1 = min(r0 + per, B);
    int sum_e = 0, sum_p = 0;
    for (int r = r0; r < r1; ++r) {
        const int c = min(a.cached_lens[r], SLOT_SAT), e = min(max(a.extend_lens[r], 0), SLOT_SAT);
        const int start = max(c, 0), end = min(sat_add(start, e), W);
        const int need = c < 0 ? 0 : max(pages_for(end) - pages_for(start), 0);
        // s_off, s_page hold each request's own numbers until the scan is known
        s_off[r] = e;
        s_page[r] = need;
        sum_e = sat_add(sum_e, e);
        sum_p = sat_add(sum_p, need);
        if (blockIdx.x == 0) a.seq_lens[r] = end;
    }
    int inc_e = sum_e, inc_p = sum_p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int ue = __shfl_up_sync(0xffffffffu, inc_e, o), up = __shfl_up_sync(0xffffffffu, inc_p, o);
        if (lane >= o) {
            inc_e = sat_add(inc_e, ue);
            inc_p = sat_add(inc_p, up);
        }
    }
    if (lane == 31) {
        s_warp[0][warp] = inc_e;
        s_warp[1][warp] = inc_p;
    }
    // what the warp's earlier lanes sum to
    int ex_e = __shfl_up_sync(0xffffffffu, inc_e, 1), ex_p = __shfl_up_sync(0xffffffffu, inc_p, 1);
    if (lane == 0) ex_e = ex_p = 0;
    __syncthreads();
    for (int w = 0; w < warp; ++w) {
        ex_e = sat_add(ex_e, s_warp[0][w]);
        ex_p = sat_add(ex_p, s_warp[1][w]);
    }
    for (int r = r0; r < r1; ++r) {
        const int e = s_off[r], need = s_page[r];
        s_off[r] = ex_e;
        s_page[r] = ex_p;
        if (blockIdx.x == 0) a.q_offsets[r] = ex_e;
        ex_e = sat_add(ex_e, e);
        ex_p = sat_add(ex_p, need);
    }
    if (tid == SLOT_THREADS - 1) {  // r1 == B here
        s_off[B] = ex_e;
        if (blockIdx.x == 0) {
            a.q_offsets[B] = ex_e;
            a.pages_used[0] = ex_p;
        }
    }
    __syncthreads();

    // SLOT_U consecutive tokens per thread: the request of the first by search, of the next by walking on
    const int all = s_off[B];
    const int64_t step = (int64_t)gridDim.x * SLOT_THREADS * SLOT_U;
    for (int64_t base = ((int64_t)blockIdx.x * SLOT_THREADS + tid) * SLOT_U; base < a.total_tokens; base += step) {
        int r = 0;
        if (base < all) {
            int hi = B;  // the last request that starts at or before the token: s_off[r] <= i < s_off[r + 1]
            while (hi - r > 1) {
                const int mid = (r + hi) >> 1;
                if (s_off[mid] <= base) r = mid; else hi = mid;
            }
        }
        int row[SLOT_U], pos[SLOT_U];  // row: what is known of it before the loads below
        const int32_t *from[SLOT_U];   // where the rest of it comes from, or null
        int32_t *to[SLOT_U];
        bool fresh[SLOT_U];            // *from is a page number
#pragma unroll
        for (int u = 0; u < SLOT_U; ++u) {
            row[u] = a.dummy_row;
            pos[u] = 0;
            from[u] = nullptr;
            to[u] = nullptr;
            fresh[u] = false;
            const int64_t i64 = base + u;
            if (i64 >= min(all, a.total_tokens)) continue;
            const int i = (int)i64;
            while (s_off[r + 1] <= i) ++r;
            const int c = min(a.cached_lens[r], SLOT_SAT), start = max(c, 0);
            const int p = sat_add(start, i - s_off[r]);
            pos[u] = p;
            if (p >= W) continue;
            int32_t *table = a.page_table + (int64_t)r * a.pt_stride;
            to[u] = table + p;
            if (c < 0) continue;
            const int pg = page_of(p);
            if (c > 0 && pg == page_of(c - 1)) {
                row[u] = p - (c - 1);
                from[u] = table + (c - 1);
            } else {
                const int k = s_page[r] + (pg - pages_for(c));
                if (k < a.num_free) {
                    row[u] = p - pg * a.page_size;
                    from[u] = a.free_pages + k;
                    fresh[u] = true;
                }
            }
        }
        int got[SLOT_U];
#pragma unroll
        for (int u = 0; u < SLOT_U; ++u) got[u] = from[u] ? *from[u] : 0;
#pragma unroll
        for (int u = 0; u < SLOT_U; ++u) {
            // a last row on dummy_row had no page: the rows behind dummy_row are not this request's
            if (from[u] && !fresh[u] && got[u] == a.dummy_row) row[u] = 0;
            row[u] += fresh[u] ? (int)((uint32_t)got[u] * (uint32_t)a.page_size) : got[u];
            if (to[u]) *to[u] = row[u];
            if (base + u < a.total_tokens) {
                a.out_loc[base + u] = row[u];
                a.positions[base + u] = pos[u];
            }
        }
    }
}

cudaError_t launch_build_slots(const SlotArgs &a, cudaStream_t s) {
    int shift = -1;
    if ((a.page_size & (a.page_size - 1)) == 0)
        for (shift = 0; (1 << shift) < a.page_size; ++shift) {
        }
    constexpr int SPAN = SLOT_THREADS * SLOT_U;
    int64_t blocks = ((int64_t)a.total_tokens + SPAN - 1) / SPAN;
    const int64_t cap = 4LL * max(device_sm_count(), 1);
    if (blocks > cap) blocks = cap;
    if (blocks < 1) blocks = 1;
    return launch_pdl(build_slots_kernel, dim3((unsigned)blocks), dim3(SLOT_THREADS), 0, s, a, shift);
}

}  // namespace minisgl

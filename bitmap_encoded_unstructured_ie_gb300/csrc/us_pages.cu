// us_pages.cu -- page tables and slots worked out on the GPU from request lengths.
//
// Reserve: request b holds ceil(len / page_size) pages afterwards.  With rel_b and
// tak_b the pages that it gives back and wants, R_b and T_b their sums over the
// requests before it, and c the free pages before the call, page i of request b
//   given back  goes to   free[c + R_b + i]
//   taken       is        free[c + R - 1 - (T_b + i)],  R = sum of rel_b
// so every page's place follows from two prefix sums, and the pages move in any order:
// those given back first, a barrier, then those taken.
//
// Nothing here computes: it is latency (lengths, sums, entries, one after the other).
// One launch of one thread-block cluster does it, its barrier between the two moves:
// each CTA makes the prefix sums for itself (B <= 1024), then the cluster's threads
// share the pages, finding a page's request by bisection of the sums, so that one long
// request is spread like many short ones.
#include "us_internal.h"
#include "us_kv.cuh"
#include "us_launch.cuh"

namespace {

constexpr int kCtas = 8, kThreads = 1024, kMaxB = 1024, kAll = kCtas * kThreads;
constexpr int kAtOnce = 4;                        // pages of a thread on their way at once

struct Sums {
    int rel[kMaxB], tak[kMaxB];                   // pages of the requests up to this one, itself among them
    int from[kMaxB], have[kMaxB];                 // pages kept (the first one given back), pages held
    int64_t wsum[2][32];
    int all_rel, all_tak;
    int bad;
};

// Inclusive sums of a and b over the block's threads.
US_DEV void scan2(int64_t& a, int64_t& b, int64_t (&w)[2][32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
        if (lane >= d) a += x, b += y;
    }
    if (lane == 31) w[0][warp] = a, w[1][warp] = b;
    __syncthreads();
    if (warp < 2) {
        int64_t v = w[warp][lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += x;
        }
        w[warp][lane] = v;
    }
    __syncthreads();
    if (warp) a += w[0][warp - 1], b += w[1][warp - 1];
}

// First request whose sum is above x.
US_DEV int owner(const int* sum, int B, int x) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
reserve_kernel(const us_kv_pool P, int page_shift, const int32_t* len, unsigned* status) {
    __shared__ Sums S;
    us::pdl_wait();
    const int b = threadIdx.x, at = blockIdx.x * kThreads + threadIdx.x;
    unsigned* says = blockIdx.x == 0 ? status : nullptr;
    const int count = *P.free_count;
    if (b == 0) S.bad = count < 0 || count > P.num_pages;
    __syncthreads();
    int64_t rel = 0, tak = 0;
    int want = 0, have = 0;
    if (b < P.B) {
        have = P.held[b];
        const int n = len[b];
        if (have < 0 || have > P.max_pages) S.bad = 1;
        want = (int)(((int64_t)n + (1 << page_shift) - 1) >> page_shift);
        if (n < 0 || want > P.max_pages) want = have, us::set_status(says, US_ERR_INVALID_ARG);
        rel = want < have ? have - want : 0;
        tak = want > have ? want - have : 0;
    }
    int64_t rel_to = rel, tak_to = tak;
    scan2(rel_to, tak_to, S.wsum);
    const int64_t all = S.wsum[0][31];
    if (S.bad || all > P.num_pages - count) {              // (the same in every CTA)
        if (b == 0) us::set_status(says, US_ERR_CORRUPT);
        us::pdl_launch_dependents();
        return;
    }
    const int R = (int)all, room = count + R;
    const bool served = tak_to <= room;
    if (b < P.B) {
        S.rel[b] = (int)rel_to;
        S.tak[b] = served ? (int)tak_to : 0x7FFFFFFF;
        S.from[b] = want;
        S.have[b] = have;
        if (!served && tak) us::set_status(says, US_ERR_WORKSPACE);
    }
    if (b == 0) S.all_tak = 0;
    __syncthreads();
    if (b < P.B && served) atomicMax(&S.all_tak, (int)tak_to);
    for (int x0 = at; x0 < R; x0 += kAtOnce * kAll) {
        int32_t* from[kAtOnce];
        int page[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int x = x0 + u * kAll;
            from[u] = nullptr;
            if (x >= R) continue;
            const int o = owner(S.rel, P.B, x), i = x - (o ? S.rel[o - 1] : 0);
            from[u] = P.page_table + (int64_t)o * P.max_pages + S.from[o] + i;
            page[u] = *from[u];
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (from[u]) P.free_pages[count + x0 + u * kAll] = page[u], *from[u] = -1;
    }
    us::cluster_sync();                                    // (everyone has read held and the count, too)
    const int taken = S.all_tak;
    for (int x0 = at; x0 < taken; x0 += kAtOnce * kAll) {
        int page[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int x = x0 + u * kAll;
            if (x < taken) page[u] = __ldcg(P.free_pages + room - 1 - x);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int x = x0 + u * kAll;
            if (x >= taken) continue;
            const int o = owner(S.tak, P.B, x), i = x - (o ? S.tak[o - 1] : 0);
            P.page_table[(int64_t)o * P.max_pages + S.have[o] + i] = page[u];
        }
    }
    if (blockIdx.x == 0) {
        if (b < P.B && (served || !tak)) P.held[b] = want;
        if (b == 0) *P.free_count = room - taken;
    }
    us::pdl_launch_dependents();
}

__global__ void __launch_bounds__(256)
slots_kernel(const UsKvCache c, const UsKvCall a, int64_t* slots) {
    us::pdl_wait();
    const int b = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x, pos = a.pos[b];
    int row0;
    const int n = us::kv_rows(a, b, row0, c.status);
    if (i < n) {
        const int p = us::kv_pos(pos, i), id = us::kv_page(c, b, p);
        slots[row0 + i] = id < 0 ? -1 : ((int64_t)id << c.page_shift) + (p & ((1 << c.page_shift) - 1));
    }
    us::pdl_launch_dependents();
}

}  // namespace

namespace us {

us_status launch_reserve(const us_kv_pool& P, const int32_t* len, unsigned* status, cudaStream_t st) {
    return launch_pdl(reserve_kernel, dim3(kCtas), kThreads, 0, st, P, __builtin_ctz((unsigned)P.page_size), len, status);
}

us_status launch_slots(const UsKvCache& c, const UsKvCall& a, int64_t* slots, cudaStream_t st) {
    return launch_pdl(slots_kernel, dim3((unsigned)((a.max_n + 255) / 256), (unsigned)c.B), 256, 0, st, c, a, slots);
}

}  // namespace us

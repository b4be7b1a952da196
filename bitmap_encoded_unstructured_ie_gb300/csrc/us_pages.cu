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
// each CTA makes the prefix sums for itself (B <= 1024), then the cluster's warps share
// the pages in runs of up to 128 of one request, so that one long request is spread like
// many short ones.  A warp finds a run's request in two steps, each lane looking at
// another sum (by bisection for each page: 512 requests that give and take 280000 pages
// 25 us, 11 us so).  48 requests that grow by up to four positions take 2.6 us a call.
#include "us_internal.h"
#include "us_kv.cuh"
#include "us_launch.cuh"

namespace {

constexpr int kCtas = 8, kThreads = 1024, kMaxB = 1024, kAll = kCtas * kThreads;
constexpr int kAtOnce = 4;                        // pages of a thread on their way at once

constexpr int kRun = 32 * kAtOnce;

struct Sums {
    int rel[kMaxB], tak[kMaxB];                   // pages of the requests before this one
    int rel_run[kMaxB], tak_run[kMaxB];           // runs of the requests up to this one, itself among them; behind the last one 2^31 - 1
    int from[kMaxB], have[kMaxB];                 // pages kept (the first one given back), pages held
    bool served[kMaxB];
    int64_t wsum[3][32];
    int all_tak;
    int bad;
};

// Inclusive sums of a, b and c over the block's threads.
US_DEV void scan3(int64_t& a, int64_t& b, int64_t& c, int64_t (&w)[3][32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d), z = __shfl_up_sync(0xffffffffu, c, d);
        if (lane >= d) a += x, b += y, c += z;
    }
    if (lane == 31) w[0][warp] = a, w[1][warp] = b, w[2][warp] = c;
    __syncthreads();
    if (warp < 3) {
        int64_t v = w[warp][lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, v, d);
            if (lane >= d) v += x;
        }
        w[warp][lane] = v;
    }
    __syncthreads();
    if (warp) a += w[0][warp - 1], b += w[1][warp - 1], c += w[2][warp - 1];
}

// The request of run x of the warp's (the first one whose sum is above x), and which of
// its runs it is.
US_DEV int owner(const int* sum, int x, int& run) {
    const int lane = threadIdx.x & 31;
    const int row = 32 * (__ffs(__ballot_sync(0xffffffffu, sum[32 * lane + 31] > x)) - 1);
    const int v = sum[row + lane], at = __ffs(__ballot_sync(0xffffffffu, v > x)) - 1, o = row + at;
    run = x - (o ? sum[o - 1] : 0);
    return o;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
reserve_kernel(const us_kv_pool P, int page_shift, const int32_t* len, unsigned* status) {
    __shared__ Sums S;
    us::pdl_wait();
    const int b = threadIdx.x, lane = b & 31;
    const int warp = ((int)blockIdx.x * kThreads + b) / 32;    // of the cluster's
    constexpr int kWarps = kAll / 32;
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
    int64_t rel_to = rel, tak_to = tak, run_to = (rel + kRun - 1) / kRun << 32 | (tak + kRun - 1) / kRun;
    scan3(rel_to, tak_to, run_to, S.wsum);
    const int64_t all = S.wsum[0][31];
    if (S.bad || all > P.num_pages - count) {              // (the same in every CTA)
        if (b == 0) us::set_status(says, US_ERR_CORRUPT);
        us::pdl_launch_dependents();
        return;
    }
    const int R = (int)all, room = count + R;
    const bool served = tak_to <= room;
    S.rel[b] = (int)(rel_to - rel);
    S.tak[b] = served ? (int)(tak_to - tak) : 0;
    S.rel_run[b] = b < P.B ? (int)(run_to >> 32) : 0x7FFFFFFF;
    S.tak_run[b] = b < P.B ? (int)run_to : 0x7FFFFFFF;
    S.from[b] = want;
    S.have[b] = have;
    S.served[b] = served;
    if (!served && tak) us::set_status(says, US_ERR_WORKSPACE);
    if (b == 0) S.all_tak = 0;
    __syncthreads();
    if (b < P.B && served) atomicMax(&S.all_tak, (int)tak_to);
    const int rel_runs = (int)(S.wsum[2][31] >> 32), tak_runs = (int)S.wsum[2][31];
    for (int x = warp; x < rel_runs; x += kWarps) {
        int run, page[kAtOnce];
        const int o = owner(S.rel_run, x, run), i0 = run * kRun + lane, n = S.have[o] - S.from[o];
        int32_t* from = P.page_table + (int64_t)o * P.max_pages + S.from[o] + i0;
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (i0 + 32 * u < n) page[u] = from[32 * u];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (i0 + 32 * u < n) P.free_pages[count + S.rel[o] + i0 + 32 * u] = page[u], from[32 * u] = -1;
    }
    us::cluster_sync();                                    // (everyone has read held and the count, too)
    const int taken = S.all_tak;
    for (int x = warp; x < tak_runs; x += kWarps) {
        int run, page[kAtOnce];
        const int o = owner(S.tak_run, x, run), i0 = run * kRun + lane, n = S.from[o] - S.have[o];
        if (!S.served[o]) break;                           // nor is one behind it
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (i0 + 32 * u < n) page[u] = __ldcg(P.free_pages + room - 1 - (S.tak[o] + i0 + 32 * u));
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u)
            if (i0 + 32 * u < n) P.page_table[(int64_t)o * P.max_pages + S.have[o] + i0 + 32 * u] = page[u];
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

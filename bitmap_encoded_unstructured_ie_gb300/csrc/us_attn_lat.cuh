// us_attn_lat.cuh -- what the attention over latent rows and over expanded rows share:
// parameters, and the join of the states that several CTAs hold of one segment.
#pragma once

#include "us_attn.cuh"
#include "us_lat.cuh"
#include "us_launch.cuh"

// Of the base: c has the pages and one key head, G = Hq.
struct UsAttnLatParams : UsAttnParams {
    const uint16_t* rows;
    int Dc, W;
};

// Of the base: c has H key heads and limits that no request meets, G = 1, no mask.
struct UsAttnRowsParams : UsAttnParams {
    us_attn_kv_rows k;
    const int32_t* kv_off;           // request b's key rows; its tokens are the last of them

    // (a template's call finds these by the parameters' own type)
    static constexpr bool kOffsets = true;
    US_DEV int context(int b, int o0, int o1) const {
        const int k0 = kv_off[b], k1 = kv_off[b + 1];
        return k0 >= 0 && k1 >= k0 && k1 <= k.S && o1 >= o0 && k1 - k0 >= o1 - o0 ? (k1 - k0) - (o1 - o0) : -1;
    }
};

namespace us {

int num_sms();

namespace attn {

// Waits for phase `parity` of `bar`, at most kWaitLimitNs (then US_ERR_TIMEOUT is
// recorded).  Without a pause between tries: these kernels' few warps leave the issue
// slots to it.
US_DEV bool spin(uint64_t* bar, uint32_t parity, unsigned* status) {
    if (us::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = us::globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int n = 0; n < 1024; ++n)
            if (us::mbar_try_wait(bar, parity)) return true;
        if (us::globaltimer_ns() - t0 > us::kWaitLimitNs) break;
    }
    us::set_status(status, US_ERR_TIMEOUT);
    return false;
}

// A row's reference for scores up to `top`: R, or a new one less than the largest by
// kTop, log2 of its weight, once that is beyond kRoom (scores from kFine on: by nothing).
US_DEV float reference(float R, float top) {
    constexpr float kTop = 11.f, kRoom = 15.9f;
    return top > R + (fabsf(R) < kFine ? kRoom : 0.f) ? top - (fabsf(top) < kFine ? kTop : 0.f) : R;
}

// fp16 pairs with infinities and NaN as 0.  A value that a row does not see has weight
// 0 in it, and 0 times what is not finite would be NaN.  What a row that sees it gets:
// over latent rows its key has made NaN of the weight, over expanded rows it is added
// at the segment's end.
US_DEV uint32_t not_finite(uint32_t x) { return __vcmpeq2(x & 0x7C007C00u, 0x7C007C00u); }
US_DEV bool all_finite(uint4 x) { return (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) == 0; }
US_DEV uint4 finite(uint4 x) {
    return make_uint4(x.x & ~not_finite(x.x), x.y & ~not_finite(x.y), x.z & ~not_finite(x.z), x.w & ~not_finite(x.w));
}

// us::tmem_ld32 in two parts: its values are there after us::tmem_ld_frag32_end
US_DEV void tmem_ld32_begin(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

// A partial state of ROWS rows of D columns in the workspace: the rows' references, their
// sums, then the outputs in fours of columns, rows side by side.
constexpr int slot_floats(int rows, int d) { return 2 * rows + rows * d; }
constexpr int kMaxCtas = 512, kPartBytes = kMaxCtas * 32, kJoinThreads = 256;
static_assert(sizeof(Part) <= 32, "parts");

// Joins the partial states of shared segments.  A thread adds up kVec times four
// columns of a row, kAtOnce states at once; its group of threads takes every
// GROUPS-th state of the segment, and the groups' sums are added in shared memory.
// Few segments have many sharers each and are given 8 groups; many have about two, and
// one group does: up to an eighth as many segments as CTAs (19), and there both take about
// as long (one token of B requests of 60000 / B positions, 8 groups / 1: B = 1 30.8 / 138 us,
// 8 27.1 / 43.4, 19 29.7 / 33.4, 32 33.4 / 30.3, 76 48.9 / 30.9; 16 expanded rows behind 8000:
// 1 head 13.5 / 25.6, 19 heads 29.1 / 29.7, 64 heads 63.7 / 60.7).
// blockIdx.x: a shared segment and 16 of its rows (of `blocks` such), blockIdx.y: which
// columns; segments by the CTA that shares one first, or, where they are few, counted.
template <int ROWS, int D, int GROUPS, class P>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const P p, int blocks, int ctas) {
    constexpr int kVec = GROUPS > 1 ? 1 : D >= 256 ? 4 : D / 64, kAtOnce = GROUPS > 1 ? 4 : 8 / kVec, kLanes = kJoinThreads / GROUPS;
    __shared__ float held[GROUPS == 1 ? 1 : 6][kJoinThreads];
    us::pdl_wait();
    us::pdl_launch_dependents();
    int which = (int)blockIdx.x / blocks;
    if constexpr (GROUPS > 1) {
        const int lane = threadIdx.x & 31;
        int at = -1;
        for (int c0 = 0; c0 < ctas && at < 0; c0 += 32) {
            unsigned who = __ballot_sync(0xffffffffu, c0 + lane < ctas && p.ws_parts[c0 + lane].rows > 0);
            for (; who; who &= who - 1)
                if (which-- == 0) {
                    at = c0 + __ffs(who) - 1;
                    break;
                }
        }
        which = at;
        if (at < 0) return;
    }
    Part a = p.ws_parts[which];
    // (a workspace that two calls share at once may hold anything: nothing outside it and O is touched)
    if (a.rows > 0 && (a.first < 0 || a.last >= ctas || a.rows > ROWS || a.h < 0 || a.h >= p.c.Hkv || a.row0 < 0 || a.rb < 0 ||
                       (int64_t)a.row0 + ((int64_t)a.rb * ROWS + a.rows - 1) / p.G >= p.a.T)) {
        us::set_status(p.c.status, US_ERR_CORRUPT);
        a.rows = 0;
    }
    const int group = threadIdx.x / kLanes, t = threadIdx.x % kLanes;
    const int row = (int)blockIdx.x % blocks * 16 + (t & 15), col = ((int)blockIdx.y * (kLanes / 16 * kVec) + (t >> 4)) * 4;
    if (row - (t & 15) < a.rows) {                         // (uniform; 0 rows: no shared segment)
        float top = -INFINITY, sum = 0.f, y[kVec][4] = {};
        for (int c = a.first + group; c <= a.last; c += GROUPS * kAtOnce) {
            float4 v[kAtOnce][kVec];
            float r[kAtOnce], l[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int cta = c + u * GROUPS;
                const bool there = cta <= a.last && row < a.rows;
                const float* sl = p.ws_slots + a.slot(there ? cta : a.first) * slot_floats(ROWS, D);
                r[u] = there ? __ldcg(sl + row) : -INFINITY, l[u] = there ? __ldcg(sl + ROWS + row) : 0.f;
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                    v[u][k] = there ? __ldcg(reinterpret_cast<const float4*>(sl + 2 * ROWS) + (col / 4 + k * (kLanes / 16)) * ROWS + row)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float m = top;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) m = fmaxf(m, r[u]);
            // (a state without a reference has weights 0, or NaN, which stays)
            const float at = m == -INFINITY ? 0.f : m, f0 = ex2(top - at);
            sum *= f0;
#pragma unroll
            for (int k = 0; k < kVec; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) y[k][i] *= f0;
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const float f = ex2(r[u] - at);
                sum += l[u] * f;
#pragma unroll
                for (int k = 0; k < kVec; ++k)
                    y[k][0] += v[u][k].x * f, y[k][1] += v[u][k].y * f, y[k][2] += v[u][k].z * f, y[k][3] += v[u][k].w * f;
            }
            top = m;
        }
        if constexpr (GROUPS > 1) {
            held[0][threadIdx.x] = top, held[1][threadIdx.x] = sum;
#pragma unroll
            for (int i = 0; i < 4; ++i) held[2 + i][threadIdx.x] = y[0][i];
            __syncthreads();
            float m = -INFINITY;
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) m = fmaxf(m, held[0][kLanes * u + t]);
            const float at = m == -INFINITY ? 0.f : m;
            sum = 0.f, y[0][0] = y[0][1] = y[0][2] = y[0][3] = 0.f;
#pragma unroll
            for (int u = 0; u < GROUPS; ++u) {
                const float f = ex2(held[0][kLanes * u + t] - at);
                sum += held[1][kLanes * u + t] * f;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[0][i] += held[2 + i][kLanes * u + t] * f;
            }
        }
        if (group == 0 && row < a.rows) {
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            uint16_t* out = out_row<ROWS>(p, a.row0, a.h, a.rb, row, D) + col;
#pragma unroll
            for (int k = 0; k < kVec; ++k)
                *reinterpret_cast<uint2*>(out + k * (kLanes / 4)) =
                    make_uint2(pack_out(y[k][0] * inv, y[k][1] * inv), pack_out(y[k][2] * inv, y[k][3] * inv));
        }
    }
}

inline int attn_ctas() { return us::num_sms() < kMaxCtas ? us::num_sms() : kMaxCtas; }
inline size_t join_ws(int ctas, int rows, int d) { return kPartBytes + (size_t)2 * ctas * slot_floats(rows, d) * 4; }

template <int ROWS, int D, class P>
us_status launch_join(const P& p, int ctas, cudaStream_t st) {
    const int64_t rows = (int64_t)p.a.max_n * p.G, segments = (rows + ROWS - 1) / ROWS * p.c.Hkv * p.c.B;      // at most
    const int blocks = rows < ROWS ? ((int)rows + 15) / 16 : ROWS / 16;
    if (8 * segments <= ctas)
        return us::launch_pdl(join_kernel<ROWS, D, 8, P>, dim3((unsigned)(segments * blocks), D / 8), kJoinThreads, 0, st, p, blocks, ctas);
    return us::launch_pdl(join_kernel<ROWS, D, 1, P>, dim3((unsigned)(ctas * blocks), D < 256 ? 1 : D / 256), kJoinThreads, 0, st, p, blocks, ctas);
}

}  // namespace attn
}  // namespace us

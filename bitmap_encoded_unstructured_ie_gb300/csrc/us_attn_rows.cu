// us_attn_rows.cu -- attention over expanded rows: one CTA a query
// row and head, its warps taking the positions in turn, with a running maximum and sum
// each, joined at the end.
#include "us_attn_lat.cuh"
#include "us_internal.h"
#include "us_launch.cuh"

namespace {

constexpr int kWarps = 4;

US_DEV float2 two(const uint16_t* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }

// KW, VW: values of a key and of a value; key(p, j), value(p, j): two values from the
// 2j-th on; seen(p)
template <int KW, int VW, class Key, class Value, class Seen>
US_DEV void attend(const uint16_t* q, uint16_t* out, int positions, float scale, Key key, Value value, Seen seen) {
    __shared__ float part[kWarps][VW + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float m = -INFINITY, l = 0.f, o[VW / 32] = {};
    for (int p = warp; p < positions; p += kWarps) {
        if (!seen(p)) continue;
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < KW / 64; ++j) {
            const float2 a = two(q + 2 * (lane + 32 * j)), b = key(p, lane + 32 * j);
            s = fmaf(a.x, b.x, fmaf(a.y, b.y, s));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= scale;
        const float t = fmaxf(m, s), f = m == -INFINITY ? 0.f : expf(m - t), w = expf(s - t);
        l = l * f + w;
        m = t;
#pragma unroll
        for (int j = 0; j < VW / 64; ++j) {
            const float2 v = value(p, lane + 32 * j);
            o[2 * j] = o[2 * j] * f + w * v.x;
            o[2 * j + 1] = o[2 * j + 1] * f + w * v.y;
        }
    }
#pragma unroll
    for (int j = 0; j < VW / 64; ++j)
        part[warp][2 * (lane + 32 * j)] = o[2 * j], part[warp][2 * (lane + 32 * j) + 1] = o[2 * j + 1];
    if (lane == 0) part[warp][VW] = m, part[warp][VW + 1] = l;
    __syncthreads();
    float top = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part[w][VW]);
    for (int w = 0; w < kWarps; ++w) sum += part[w][VW] == -INFINITY ? 0.f : part[w][VW + 1] * expf(part[w][VW] - top);
    for (int d = threadIdx.x; d < VW; d += 32 * kWarps) {
        float y = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (part[w][VW] != -INFINITY) y += part[w][d] * expf(part[w][VW] - top);
        y = sum == 0.f ? 0.f : y / sum;
        out[d] = us::float_to_half_bits(y != y ? y : fminf(fmaxf(y, -65504.f), 65504.f));
    }
}

template <int DN, int DV>
__global__ void __launch_bounds__(32 * kWarps) attn_rows_kernel(const UsAttnRowsParams p) {
    us::pdl_wait();
    const int b = blockIdx.y, i = blockIdx.x / p.k.H, h = blockIdx.x % p.k.H;
    const int row0 = p.off[b], n = p.off[b + 1] - row0, k0 = p.kv_off[b], kn = p.kv_off[b + 1] - k0;
    const bool ok = row0 >= 0 && n >= 0 && row0 + n <= p.T && n <= p.max_n && k0 >= 0 && kn >= n && k0 + (int64_t)kn <= p.k.S;
    if (!ok) us::set_status(p.status, US_ERR_INVALID_ARG);
    if (ok && i < n) {
        attend<DN + 64, DV>(
            p.Q + (int64_t)(row0 + i) * p.ldq + (int64_t)h * (DN + 64), p.O + (int64_t)(row0 + i) * p.ldo + (int64_t)h * DV,
            kn - n + i + 1, p.scale,
            [&](int pos, int j) {
                return 2 * j < DN ? two(p.k.K + (k0 + pos) * p.k.ldk + h * p.k.hsk + 2 * j)
                                  : two(p.k.KR + (k0 + pos) * p.k.ldkr + 2 * j - DN);
            },
            [&](int pos, int j) { return two(p.k.V + (k0 + pos) * p.k.ldv + h * p.k.hsv + 2 * j); },
            [](int) { return true; });
    }
    us::pdl_launch_dependents();
}

}  // namespace

namespace us {

size_t attn_rows_ws(const UsAttnRowsParams&) { return 0; }
us_status launch_attn_rows(const UsAttnRowsParams& p, cudaStream_t st) {
    return launch_pdl(p.k.Dn == 128 ? attn_rows_kernel<128, 128> : attn_rows_kernel<64, 64>,
                      dim3((unsigned)(p.max_n * p.k.H), (unsigned)p.B), 32 * kWarps, 0, st, p);
}

}  // namespace us

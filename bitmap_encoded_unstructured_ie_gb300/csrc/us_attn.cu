// us_attn.cu -- attention of new tokens over the quantised K/V cache.
//
// Query row (token i of request b, head hq) sees the positions p < ctx, and of
// the call's own tokens j = p - ctx those whose bit is set in the token's mask
// (no mask: j <= i).  o = sum_p w_p v_p / sum_p w_p, w_p = exp(scale q.k_p), 0
// for a row that sees nothing.
//
// One CTA per query row; each warp walks every fourth position with a running
// maximum and sum, its lanes holding D/32 dimensions; the four states are
// joined at the end.
#include "us_internal.h"
#include "us_kv.cuh"

namespace {

constexpr int kWarps = 4;

// D/32 neighbouring codes of a row, from dimension lane * D/32
template <int ELEM, int DL>
US_DEV void codes(const uint8_t* row, int lane, float (&x)[DL]) {
#pragma unroll
    for (int i = 0; i < DL; ++i) {
        const int d = lane * DL + i;
        x[i] = ELEM == US_I8 ? (float)(int8_t)row[d] : (float)us::sext4((uint32_t)row[d >> 1] >> (4 * (d & 1)));
    }
}

template <int ELEM, int D>
__global__ void __launch_bounds__(32 * kWarps)
attn_row_kernel(const UsAttnParams p) {
    constexpr int DL = D / 32;
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    us::pdl_wait();
    const UsKvCache& c = p.c;
    const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int row0;
    const int n = us::kv_rows(c, p.a, b, row0);
    if (i >= n) return;
    const int64_t t = row0 + i;
    const int ctx = us::kv_context(c, p.a, b, n);
    if (ctx < 0) return;
    const int G = p.Hq / c.Hkv, h = hq / G;
    const uint64_t mask = p.mask ? p.mask[t] : 0;
    const float sc = p.scale * 1.4426950408889634f;           // exp2 domain
    float q[DL], o[DL] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int d = 0; d < DL; ++d) q[d] = us::half_bits_to_float(p.Q[t * p.ldq + hq * D + lane * DL + d]) * sc;
    for (int pos = warp; pos < ctx + n; pos += kWarps) {
        const int j = pos - ctx;
        if (j >= 0 && !(p.mask ? (mask >> j) & 1 : j <= i)) continue;
        const int id = us::kv_page(c, b, pos);
        if (id < 0) continue;
        const int64_t e = us::kv_entry(c, id, h, pos);
        const uint32_t s2 = reinterpret_cast<const uint32_t*>(c.scale)[e];
        float x[DL], s = 0.f;
        codes<ELEM, DL>(c.k + e * c.row_bytes, lane, x);
#pragma unroll
        for (int d = 0; d < DL; ++d) s += q[d] * x[d];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= us::half_bits_to_float((uint16_t)s2);
        const float mn = fmaxf(m, s), f = exp2f(m - mn), w = exp2f(s - mn);
        const float wv = w * us::half_bits_to_float((uint16_t)(s2 >> 16));
        codes<ELEM, DL>(c.v + e * c.row_bytes, lane, x);
#pragma unroll
        for (int d = 0; d < DL; ++d) o[d] = o[d] * f + wv * x[d];
        l = l * f + w;
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int d = 0; d < DL; ++d) so[warp][lane * DL + d] = o[d];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 32 * kWarps) {
        float top = -INFINITY, sum = 0.f, y = 0.f;
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
        for (int w = 0; w < kWarps; ++w) {
            const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - top);
            sum += sl[w] * f;
            y += so[w][d] * f;
        }
        p.O[t * p.ldo + hq * D + d] = us::float_to_half_bits(sum == 0.f ? 0.f : y / sum);
    }
    us::pdl_launch_dependents();
}

}  // namespace

namespace us {

size_t attn_ws(const UsAttnParams&) { return 0; }

us_status launch_attn(const UsAttnParams& p, cudaStream_t st) {
    auto kern = p.c.elem == US_I8 ? (p.c.D == 64 ? attn_row_kernel<US_I8, 64> : attn_row_kernel<US_I8, 128>)
                                  : (p.c.D == 64 ? attn_row_kernel<US_I4, 64> : attn_row_kernel<US_I4, 128>);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.a.max_n, (unsigned)p.Hq, (unsigned)p.c.B);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? US_OK : US_ERR_CUDA;
}

}  // namespace us

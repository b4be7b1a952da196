// us_rope.cu -- norm and position rotation of queries and keys for each head, and the
// same with keys and values quantised into the cache (us_kv_append).
//
// A row x of D values becomes y = x rsqrt(mean(x^2) + eps) w, and its first R values
// are turned in pairs by A = 2 pi (p turns[j] mod 2^64) / 2^64: the product of a
// position and a frequency held as a 64-bit fraction of a turn wraps where the angle
// does, so the angle is off by 2^-33 turns at any position, where p * freq in fp32
// would be off by p * 2^-24 radians.  cos and sin are made once a token and CTA, in
// shared memory, and serve all of its heads.
//
// D / 8 lanes (of 8, 16 or 32) hold a row, 16 bytes each; the pairs (j, j + R/2) lie
// R / 16 lanes apart and are exchanged by shuffles.  Four rows a thread are on their
// way at once.  What bounds it: bytes (each row read and written once) for prompts,
// latency for single tokens: offsets, rows, the sum's shuffles, one after the other.
#include "us_internal.h"
#include "us_kv_quant.cuh"
#include "us_launch.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;                       // of a CTA, at most
constexpr int kAtOnce = 4;                        // rows of a thread on their way at once
constexpr int kNone = -1;                         // no cache

struct Call {
    us_rope rope;
    us_heads q, k;                                // H = 0: none
    UsKvCall a;
    const int32_t* depth;
    int D;
    UsKvCache c;                                  // us_kv_append: the cache, and V's rows
    const uint16_t* V;
    int64_t ldv;
};

// Lanes: of a row.  ELEM: the cache's, or kNone.
template <int LANES, int ELEM>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(const Call p, int tokens) {
    constexpr int kRows = kThreads / LANES;
    __shared__ float cs[kTokens][2][128];
    __shared__ int64_t place[kTokens];
    us::pdl_wait();
    const int b = blockIdx.y, pos = p.a.pos[b];
    int row0;
    const int n = us::kv_rows(p.a, b, row0, p.c.status), i0 = blockIdx.x * tokens, count = min(tokens, n - i0);
    if (count <= 0) {
        us::pdl_launch_dependents();
        return;
    }
    const int l = threadIdx.x % LANES, heads = p.q.H + p.k.H + (ELEM == kNone ? 0 : p.c.Hkv), rows = count * heads;
    const bool here = 8 * l < p.D;
    // the lane's weights; 0x3C00 is 1.0
    uint4 wq = make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u), wk = wq;
    if (p.q.H && p.q.w && here) wq = reinterpret_cast<const uint4*>(p.q.w)[l];
    if (p.k.H && p.k.w && here) wk = reinterpret_cast<const uint4*>(p.k.w)[l];
    const int R = p.rope.R, half = R / 16;
    const bool pairs = p.rope.style == US_ROPE_PAIRS;
    const bool turned = 8 * l < R;
    // halves: the lane with the other ones of its pairs, and its angles' first index
    const int other = pairs || !turned ? l : l < half ? l + half : l - half;
    const int first = pairs ? 4 * l : 8 * (l < half ? l : l - half);
    bool ready = false;
    for (int r0 = threadIdx.x / LANES; r0 - (int)threadIdx.x / LANES < rows; r0 += kAtOnce * kRows) {
        uint4 in[kAtOnce];
        int tok[kAtOnce], h[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = r0 + u * kRows;
            in[u] = make_uint4(0, 0, 0, 0);
            tok[u] = (int)((unsigned)r / (unsigned)heads), h[u] = r - tok[u] * heads;
            if (r < rows && here) {
                const int64_t t = row0 + i0 + tok[u];
                const uint16_t* x = h[u] < p.q.H ? p.q.x + t * p.q.ld + h[u] * p.q.hs
                                    : ELEM == kNone || h[u] < p.q.H + p.k.H
                                        ? p.k.x + t * p.k.ld + (h[u] - p.q.H) * p.k.hs
                                        : p.V + t * p.ldv + (int64_t)(h[u] - p.q.H - p.k.H) * p.D;
                in[u] = *reinterpret_cast<const uint4*>(x + 8 * l);
            }
        }
        if (!ready) {                                      // while the rows are on their way
            for (int x = threadIdx.x; x < count * (R / 2); x += kThreads) {
                const int i = x / (R / 2), j = x - i * (R / 2);
                const int at = us::kv_pos(pos, p.depth ? p.depth[row0 + i0 + i] : i0 + i);
                const int32_t turn = (int32_t)(((uint64_t)(int64_t)at * p.rope.turns[j]) >> 32);
                sincospif((float)turn * 0x1p-31f, &cs[i][1][j], &cs[i][0][j]);
            }
            if (ELEM != kNone && (int)threadIdx.x < count) {
                const int at = us::kv_pos(pos, i0 + threadIdx.x), id = us::kv_page(p.c, b, at);
                place[threadIdx.x] = id < 0 ? -1 : us::kv_entry(p.c, id, 0, at);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = r0 + u * kRows;
            if (u && r - (int)threadIdx.x / LANES >= rows) break;
            const bool is_q = h[u] < p.q.H, is_v = ELEM != kNone && h[u] >= p.q.H + p.k.H, ok = r < rows;
            const us_heads& g = is_q ? p.q : p.k;
            uint4 out = in[u];
            {
                float y[8];
                const uint32_t x4[4] = {in[u].x, in[u].y, in[u].z, in[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x4[i]));
                    y[2 * i] = f.x, y[2 * i + 1] = f.y;
                }
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) ss = fmaf(y[i], y[i], ss);
#pragma unroll
                for (int d = LANES / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
                if (g.w) {
                    const float f = rsqrtf(ss / (float)p.D + p.rope.eps);
                    const uint4 w = is_q ? wq : wk;
                    const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 wf = __half22float2(*reinterpret_cast<const __half2*>(&w4[i]));
                        y[2 * i] = y[2 * i] * f * wf.x, y[2 * i + 1] = y[2 * i + 1] * f * wf.y;
                    }
                }
                if (R) {
                    const float* c = cs[ok ? tok[u] : 0][0] + (turned ? first : 0);
                    const float* s = c + 128;
                    if (pairs) {
                        if (turned) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float a = y[2 * i], d = y[2 * i + 1];
                                y[2 * i] = a * c[i] - d * s[i];
                                y[2 * i + 1] = d * c[i] + a * s[i];
                            }
                        }
                    } else {
                        float z[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) z[i] = __shfl_sync(0xffffffffu, y[i], other, LANES);
                        if (turned) {
                            const float sign = l < half ? -1.f : 1.f;
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = y[i] * c[i] + sign * s[i] * z[i];
                        }
                    }
                }
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = (uint32_t)us::float_to_half_bits(y[2 * i]) | ((uint32_t)us::float_to_half_bits(y[2 * i + 1]) << 16);
                if (!is_v) out = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (ok && here && !is_v && g.y)
                *reinterpret_cast<uint4*>(g.y + (int64_t)(row0 + i0 + tok[u]) * g.ldy + (h[u] - (is_q ? 0 : p.q.H)) * g.hsy + 8 * l) = out;
            if constexpr (ELEM != kNone) {
                constexpr int kBytes = ELEM == US_I8 ? 8 : 4;     // of a lane's codes
                if (__any_sync(0xffffffffu, ok && !is_q)) {
                    uint2 codes;
                    const uint16_t s = us::quantise_row<ELEM, 8 * LANES>(out, codes);
                    if (ok && !is_q && place[tok[u]] >= 0) {
                        const int kh = h[u] - p.q.H - (is_v ? p.k.H : 0);
                        const int64_t e = place[tok[u]] + ((int64_t)kh << p.c.page_shift);
                        us::store_codes<ELEM>((is_v ? p.c.v : p.c.k) + (e * LANES + l) * kBytes, codes);
                        if (l == 0) p.c.scale[2 * e + is_v] = s;
                    }
                }
            }
        }
    }
    us::pdl_launch_dependents();
}

// Tokens of a CTA: four rows a thread, or fewer where that leaves SMs without a CTA.
int cta_tokens(int heads, int lanes, int64_t tokens) {
    const int per = kThreads / lanes;
    int t = (kAtOnce * per + heads - 1) / heads;
    if (t > kTokens) t = kTokens;
    while (t > 1 && tokens < (int64_t)t * 2 * us::num_sms()) t /= 2;
    return t;
}

template <int ELEM>
us_status launch(const Call& p, cudaStream_t st) {
    const int lanes = p.D <= 64 ? 8 : p.D <= 128 ? 16 : 32;
    const int heads = p.q.H + p.k.H + (ELEM == kNone ? 0 : p.c.Hkv);
    const int t = cta_tokens(heads, lanes, (int64_t)p.a.max_n * p.c.B);
    const dim3 grid((unsigned)((p.a.max_n + t - 1) / t), (unsigned)p.c.B);
    if (lanes == 8) return us::launch_pdl(norm_rope_kernel<8, ELEM>, grid, kThreads, 0, st, p, t);
    if (lanes == 16) return us::launch_pdl(norm_rope_kernel<16, ELEM>, grid, kThreads, 0, st, p, t);
    if constexpr (ELEM == kNone) return us::launch_pdl(norm_rope_kernel<32, ELEM>, grid, kThreads, 0, st, p, t);
    return US_ERR_UNSUPPORTED;
}

}  // namespace

namespace us {

us_status launch_norm_rope(const us_rope& rope, int D, const us_heads& q, const us_heads& k, const UsKvCache& c, const UsKvCall& a,
                           const int32_t* depth, const uint16_t* V, int64_t ldv, cudaStream_t st) {
    const Call p = {rope, q, k, a, depth, D, c, V, ldv};
    if (!V) return launch<kNone>(p, st);
    return c.elem == US_I8 ? launch<US_I8>(p, st) : launch<US_I4>(p, st);
}

}  // namespace us

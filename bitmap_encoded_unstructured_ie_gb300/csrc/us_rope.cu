// us_rope.cu -- norm and position rotation of queries and keys for each head, and the
// same with keys and values quantised into the cache (us_kv_append).
//
// A row x of D values becomes y = x rsqrt(mean(x^2) + eps) w, and its first R values
// are turned in pairs by A = 2 pi (p turns[j] mod 2^64) / 2^64: the product of a
// position and a frequency held as a 64-bit fraction of a turn wraps where the angle
// does.  Its upper 32 bits, as a signed fraction of a turn, are rounded to fp32: the angle
// is off by at most 2^-26 + 2^-32 turns (1e-7 radians, and sincospi's 2 ulp) at any
// position, where p * freq in fp32 would be off by p * 2^-24 radians.  cos and sin are made
// once a token and CTA, in shared memory, and serve all of its heads.
//
// D / 16 lanes (of 4, 8 or 16) hold a row, each two pieces of eight values: of the first
// R those whose values are turned with one another, (8 l .., R/2 + 8 l ..) or 16 values
// side by side, so that a rotation stays in its lane (with eight values a lane and the
// pairs exchanged by shuffles, prompts took 200 instructions a warp for four rows of
// 128, 79 us where this takes 53).  Such a group of lanes takes HEADS heads of one
// token at a time (a chunk: of queries, keys or values), with weights, cos and sin in
// registers.  Prompts of 252 MB of queries and keys of 128 pass at 4.8 TB/s (37 us at a copy's
// rate), between bytes and issue: 43 % of the slots, four CTAs of 128 registers an SM.
#include "us_attn.cuh"
#include "us_internal.h"
#include "us_kv_quant.cuh"
#include "us_launch.cuh"

namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 16;                       // of a CTA, at most
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

using us::attn::add2;
using us::attn::fma2;
using us::attn::mul2;
using us::attn::pack_half2;
using us::attn::pair;
using us::attn::unpair;

// Eight fp16 values as four pairs of fp32
US_DEV void unpack(uint4 in, uint64_t (&y)[4]) {
    const uint32_t u[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        y[i] = pair(f.x, f.y);
    }
}
US_DEV uint32_t pack(uint64_t y) {
    float a, b;
    unpair(y, a, b);
    return pack_half2(a, b);
}

// LANES: of a row.  HEADS: of a chunk.  ELEM: the cache's, or kNone.  A CTA takes `chunks`
// chunks of a request's, which belong to kTokens tokens at most.
template <int LANES, int HEADS, int ELEM>
__global__ void __launch_bounds__(kThreads, HEADS == 1 ? 6 : 4)
norm_rope_kernel(const Call p, int chunks) {
    constexpr int kGroups = kThreads / LANES;
    __shared__ __align__(16) float cs[kTokens][2][128];
    __shared__ int64_t place[kTokens];
    us::pdl_wait();
    const int b = blockIdx.y, pos = p.a.pos[b];
    int row0;
    // chunks of a token: queries, keys, values
    const int nq = (p.q.H + HEADS - 1) / HEADS, nk = (p.k.H + HEADS - 1) / HEADS, per = nq + nk + (ELEM == kNone ? 0 : nk);
    const int64_t x0 = (int64_t)blockIdx.x * chunks, x1 = (int64_t)us::kv_rows(p.a, b, row0, p.c.status) * per;
    const int mine = (int)min(x1 - x0, (int64_t)chunks);
    if (mine <= 0) {
        us::pdl_launch_dependents();
        return;
    }
    const int i0 = (int)(x0 / per), skip = (int)(x0 - (int64_t)i0 * per);              // the first chunk's token, and its place there
    const int count = (skip + mine - 1) / per + 1;
    const int l = threadIdx.x % LANES, R = p.rope.R, turning = R / 16;
    const bool pairs = p.rope.style == US_ROPE_PAIRS, turned = l < turning;
    // the lane's pieces, and whether a row has them
    const int piece[2] = {turned && !pairs ? l : 2 * l, turned && !pairs ? l + turning : 2 * l + 1};
    const bool has[2] = {8 * piece[0] < p.D, 8 * piece[1] < p.D};
    const float inv_d = 1.f / (float)p.D;
    bool ready = false;
    for (int x = threadIdx.x / LANES; x - (int)threadIdx.x / LANES < mine; x += kGroups) {       // (as many rounds for all threads)
        const bool some = x < mine;
        const int tok = some ? (int)((unsigned)(x + skip) / (unsigned)per) : 0, q = some ? x + skip - tok * per : 0;
        const int kind = q < nq ? 0 : ELEM == kNone || q < nq + nk ? 1 : 2;            // queries, keys, values
        const us_heads& g = kind == 0 ? p.q : p.k;
        const int h0 = (q - (kind == 0 ? 0 : kind == 1 ? nq : nq + nk)) * HEADS, heads = some ? min(HEADS, g.H - h0) : 0;
        const int64_t t = row0 + i0 + tok, hs = kind == 2 ? p.D : g.hs;
        const uint16_t* src = (kind == 2 ? p.V + t * p.ldv : g.x + t * g.ld) + h0 * hs;
        uint4 in[HEADS][2];
#pragma unroll
        for (int u = 0; u < HEADS; ++u)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                in[u][k] = u < heads && has[k] ? *reinterpret_cast<const uint4*>(src + u * hs + 8 * piece[k]) : make_uint4(0, 0, 0, 0);
        if (!ready) {                                      // while the first rows are on their way
            for (int y = threadIdx.x; y < count * (R / 2); y += kThreads) {
                const int i = y / (R / 2), j = y - i * (R / 2);
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
        const bool normed = kind < 2 && g.w != nullptr;
        uint64_t w[2][4], co[4], si[4], ns[4];             // weights, cos, sin, -sin, two in each
#pragma unroll
        for (int k = 0; k < 2; ++k)
            unpack(normed && has[k] ? reinterpret_cast<const uint4*>(g.w)[piece[k]] : make_uint4(0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u), w[k]);
        if (turned) {
            const ulonglong2* c2 = reinterpret_cast<const ulonglong2*>(&cs[tok][0][8 * l]);
            const ulonglong2 a = c2[0], d = c2[1], e = c2[32], f = c2[33];
            co[0] = a.x, co[1] = a.y, co[2] = d.x, co[3] = d.y, si[0] = e.x, si[1] = e.y, si[2] = f.x, si[3] = f.y;
#pragma unroll
            for (int i = 0; i < 4; ++i) ns[i] = si[i] ^ 0x8000000080000000ull;
        }
        uint16_t* dst = kind < 2 && g.y ? g.y + t * g.ldy + h0 * g.hsy : nullptr;
#pragma unroll
        for (int u = 0; u < HEADS; ++u) {
            uint64_t y[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) unpack(in[u][k], y[k]);
            uint64_t s2 = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = fma2(y[k][i], y[k][i], s2);
            float ss, sb;
            unpair(s2, ss, sb);
            ss += sb;
#pragma unroll
            for (int d = LANES / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            if (normed) {
                const float f = rsqrtf(ss * inv_d + p.rope.eps);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[k][i] = mul2(mul2(y[k][i], pair(f, f)), w[k][i]);
            }
            if (turned && kind < 2) {
                if (pairs) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float a, d, c[2], s[2];
                            unpair(y[k][i], a, d);
                            unpair(co[2 * k + (i >> 1)], c[0], c[1]);
                            unpair(si[2 * k + (i >> 1)], s[0], s[1]);
                            y[k][i] = pair(a * c[i & 1] - d * s[i & 1], d * c[i & 1] + a * s[i & 1]);
                        }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint64_t a = y[0][i], d = y[1][i];
                        y[0][i] = fma2(d, ns[i], mul2(a, co[i]));
                        y[1][i] = fma2(a, si[i], mul2(d, co[i]));
                    }
                }
            }
            if (kind < 2) {
#pragma unroll
                for (int k = 0; k < 2; ++k) in[u][k] = make_uint4(pack(y[k][0]), pack(y[k][1]), pack(y[k][2]), pack(y[k][3]));
            }
            if (u < heads && dst) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (has[k]) *reinterpret_cast<uint4*>(dst + u * g.hsy + 8 * piece[k]) = in[u][k];
            }
            if constexpr (ELEM != kNone) {
                constexpr int kBytes = ELEM == US_I8 ? 8 : 4;     // of a piece's codes
                const bool kept = u < heads && kind > 0;
                if (__any_sync(0xffffffffu, kept)) {
                    uint2 codes[2];
                    const uint16_t s = us::quantise_row<ELEM, 16 * LANES, 2>(in[u], codes);
                    if (kept && place[tok] >= 0) {
                        const int64_t e = place[tok] + ((int64_t)(h0 + u) << p.c.page_shift);
                        uint8_t* to = (kind == 2 ? p.c.v : p.c.k) + e * (2 * LANES * kBytes);
#pragma unroll
                        for (int k = 0; k < 2; ++k) us::store_codes<ELEM>(to + piece[k] * kBytes, codes[k]);
                        if (l == 0) p.c.scale[2 * e + (kind == 2)] = s;
                    }
                }
            }
        }
    }
    us::pdl_launch_dependents();
}

template <int LANES, int HEADS, int ELEM>
us_status launch_as(const Call& p, cudaStream_t st) {
    constexpr int kGroups = kThreads / LANES;
    const int nq = (p.q.H + HEADS - 1) / HEADS, nk = (p.k.H + HEADS - 1) / HEADS, per = nq + nk + (ELEM == kNone ? 0 : nk);
    // four rounds a CTA, or one where that leaves SMs without work (16384 tokens of 40 heads of 128, four heads a
    // chunk: 65.5 / 68.1 us, quantised into the cache 98.6 / 112.8; 16 tokens, one head a chunk: 4.1 / 2.25)
    const int64_t all = (int64_t)p.a.max_n * per;
    int chunks = all * p.c.B >= (int64_t)8 * kGroups * us::num_sms() ? 4 * kGroups : kGroups;
    if (chunks > (kTokens - 1) * per) chunks = (kTokens - 1) * per;
    return us::launch_pdl(norm_rope_kernel<LANES, HEADS, ELEM>, dim3((unsigned)((all + chunks - 1) / chunks), (unsigned)p.c.B), kThreads, 0, st, p,
                          chunks);
}

// Four heads a chunk where that leaves work for every SM, else one: a step of 16 tokens
// is latency, which four heads one after the other lengthen (written and read back in 5.2 us,
// 7.1 with four), prompts are bytes and instructions, which four heads share (52.6 us, 60.5 with one).
// Near the border, 40 heads of 128: 256 tokens 3.1 with one, 3.5 with four (one round a CTA, as
// above); 768 5.8 / 4.6; 1024 6.7 / 6.5; 2048 11.1 / 10.0, where four rounds take 11.2; 8192 40.8 /
// 36.2, 38.0.  Heads that four does not divide are worse off: 8192 tokens of 5 and 5 heads 13.7, one 12.1.
template <int LANES, int ELEM>
us_status launch_heads(const Call& p, cudaStream_t st) {
    const int64_t rows = (int64_t)p.a.max_n * p.c.B * (p.q.H + p.k.H + (ELEM == kNone ? 0 : p.c.Hkv));
    return rows * LANES >= (int64_t)16 * kThreads * us::num_sms() ? launch_as<LANES, 4, ELEM>(p, st) : launch_as<LANES, 1, ELEM>(p, st);
}

template <int ELEM>
us_status launch(const Call& p, cudaStream_t st) {
    if (p.D <= 64) return launch_heads<4, ELEM>(p, st);
    if (p.D <= 128) return launch_heads<8, ELEM>(p, st);
    if constexpr (ELEM == kNone) return launch_heads<16, ELEM>(p, st);
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

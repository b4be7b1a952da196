// us_kv.cu -- writing, reading back and committing the quantised K/V cache.
//
// Write: per token and head, s = fp16_rn(max|x| / q), 1 if that is 0, with
// q = 127 (int8) or 7 (int4), and code = clamp(rint(x / s), -q-1, q): the rule
// of us_quantize_x on one head's row.  Infinities count as +-65504 and NaN as
// 0, so that every stored entry is finite.  Read: y = fp16_rn(code * s), at most 65504
// (the scale of a row of 65504 is rounded up: 127 * 516 = 65532 and 7 * 9360 = 65520).
// Commit: entries of listed tokens move to consecutive positions, all of one
// request's reads before its writes.
//
// Bytes bound the long calls: four prompts of up to 4096 tokens written and read back
// (152 MB) in 32 us, of which the write takes 21; 253 MB of a prefix read in 42.3 (6.0
// TB/s, 90 % of a plain copy).  Short calls are latency: offsets, page table, rows, one
// after the other, 2.5 to 3 us each in a replayed graph (launched one by one, the host's
// 5 to 6 us a call bound them).
#include "us_internal.h"
#include "us_kv.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 64;                       // of a CTA of write and read, at most
constexpr int kAtOnce = 4;                        // (token, head) rows of a thread on their way at once

// x as eight fp32 values, infinities at the largest fp16 value, NaN as 0
US_DEV void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = us::half_bits_to_float((uint16_t)(u[i >> 1] >> (16 * (i & 1))));
        x[i] = f == f ? fminf(fmaxf(f, -65504.f), 65504.f) : 0.f;
    }
}

// Eight codes (as fp32 whole numbers plus 1.5 2^23, whose low bits they are) -> bytes or nibbles.
template <int ELEM>
US_DEV uint2 pack_codes(const float (&v)[8]) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(v[i]);
    if constexpr (ELEM == US_I8) {
        return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (b[i] & 0xFu) << (4 * i);
        return make_uint2(w, 0u);
    }
}

// Quantises one row held eight values a lane by D/8 neighbouring lanes (all
// 32 lanes of the warp take part); returns the scale.
//
// rint(x / s) without a division: q = x (1/s), corrected once by its exact
// remainder.  x and s have 11 bits, so x / s is either exactly a half-way point
// k + 1/2, which has few bits and is what the correction then arrives at, or at
// least 2^-20 of itself away from one, where an error of 2^-22 does not matter.
// Rows with infinities, NaN or a subnormal scale (whose codes may need the clamp)
// take the plain way.
template <int ELEM, int D>
US_DEV uint16_t quantise_row(uint4 in, uint2& codes) {
    constexpr float q = ELEM == US_I8 ? 127.f : 7.f, kRound = 12582912.f;
    const uint32_t u[4] = {in.x, in.y, in.z, in.w};
    auto h2 = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
    __half2 m2 = h2(u[0] & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i) m2 = __hmax2_nan(m2, h2(u[i] & 0x7FFF7FFFu));
#pragma unroll
    for (int d = D / 16; d > 0; d >>= 1) m2 = __hmax2_nan(m2, __shfl_xor_sync(0xffffffffu, m2, d));
    const __half m = __hmax_nan(__low2half(m2), __high2half(m2));
    float amax = __half2float(m);
    uint16_t s16 = us::float_to_half_bits(amax / q);
    float v[8];
    if (__any_sync(0xffffffffu, !(amax <= 65504.f) || (s16 < 0x0400u && s16 != 0u))) {
        unpack8(in, v);
        amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
        for (int d = D / 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        s16 = us::float_to_half_bits(amax / q);
        if (s16 == 0) s16 = 0x3C00u;                          // 1.0
        const float s = us::half_bits_to_float(s16);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(rintf(v[i] / s), -q - 1.f), q) + kRound;
    } else {
        if (s16 == 0) s16 = 0x3C00u;
        const float s = us::half_bits_to_float(s16), inv = 1.f / s;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = __half22float2(h2(u[i]));
            const float a = x.x * inv, b = x.y * inv;
            v[2 * i] = fmaf(fmaf(-a, s, x.x), inv, a) + kRound;
            v[2 * i + 1] = fmaf(fmaf(-b, s, x.y), inv, b) + kRound;
        }
    }
    codes = pack_codes<ELEM>(v);
    return s16;
}

template <int ELEM>
US_DEV void store_codes(uint8_t* dst, uint2 w) {
    if constexpr (ELEM == US_I8) *reinterpret_cast<uint2*>(dst) = w;
    else *reinterpret_cast<uint32_t*>(dst) = w.x;
}

// The tokens of one CTA of write and read, [i0, i1) of request b, and their first
// row.
struct Tokens {
    int i0, i1, row0, pos;
};
US_DEV Tokens find_tokens(const UsKvCache& c, const UsKvCall& a, int tokens) {
    Tokens t;
    const int b = blockIdx.y;
    t.pos = a.pos[b];
    const int n = us::kv_rows(a, b, t.row0, c.status);
    t.i0 = blockIdx.x * tokens, t.i1 = min(n, t.i0 + tokens);
    return t;
}
// Their entries' page and slot (head 0), -1 where there is none; ends with a barrier.
US_DEV void find_places(const UsKvCache& c, const Tokens& t, int64_t* place) {
    const int i = t.i0 + (int)threadIdx.x;
    if (i < t.i1) {
        const int p = us::kv_pos(t.pos, i), id = us::kv_page(c, blockIdx.y, p);
        place[threadIdx.x] = id < 0 ? -1 : us::kv_entry(c, id, 0, p);
    }
    __syncthreads();
}

// D/8 lanes per (token, head), 16 bytes of K and of V each; heads run fastest, so
// a warp reads contiguous parts of a token's row.  Four rows a thread at a time:
// enough bytes on their way to run at HBM's rate.
template <int ELEM, int D>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const UsKvCache c, const UsKvCall a, int tokens, const uint16_t* __restrict__ K, int64_t ldk,
                const uint16_t* __restrict__ V, int64_t ldv) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes, kBytes = D * (ELEM == US_I8 ? 8 : 4) / 8;
    __shared__ int64_t place[kTokens];
    us::pdl_wait();
    const Tokens tk = find_tokens(c, a, tokens);
    const int j = threadIdx.x % kLanes, rows = (tk.i1 - tk.i0) * c.Hkv;
    bool first = true;
    for (int r0 = threadIdx.x / kLanes; r0 - (int)threadIdx.x / kLanes < rows; r0 += kAtOnce * kRows) {
        uint4 k[kAtOnce], v[kAtOnce];
        int tok[kAtOnce], h[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = r0 + u * kRows;
            k[u] = v[u] = make_uint4(0, 0, 0, 0);
            tok[u] = (int)((unsigned)r / (unsigned)c.Hkv), h[u] = r - tok[u] * c.Hkv;
            if (r < rows) {
                const int64_t t = tk.row0 + tk.i0 + tok[u];
                k[u] = __ldcs(reinterpret_cast<const uint4*>(K + t * ldk + h[u] * D + 8 * j));
                v[u] = __ldcs(reinterpret_cast<const uint4*>(V + t * ldv + h[u] * D + 8 * j));
            }
        }
        if (first) find_places(c, tk, place), first = false;   // while the rows are on their way
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (u && r0 - (int)threadIdx.x / kLanes + u * kRows >= rows) break;
            const int64_t e0 = r0 + u * kRows < rows ? place[tok[u]] : -1, e = e0 + ((int64_t)h[u] << c.page_shift);
            uint2 ck, cv;
            const uint16_t sk = quantise_row<ELEM, D>(k[u], ck), sv = quantise_row<ELEM, D>(v[u], cv);
            if (e0 < 0) continue;
            store_codes<ELEM>(c.k + e * kBytes + j * (kBytes / kLanes), ck);
            store_codes<ELEM>(c.v + e * kBytes + j * (kBytes / kLanes), cv);
            if (j == 0) reinterpret_cast<uint32_t*>(c.scale)[e] = (uint32_t)sk | ((uint32_t)sv << 16);
        }
    }
    us::pdl_launch_dependents();
}

// eight codes and a scale -> eight fp16 values
template <int ELEM>
US_DEV uint4 dequantise8(uint2 w, float s) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = 2 * i + k;
            const int code = ELEM == US_I8 ? (int)(int8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3))) : us::sext4(w.x >> (4 * e));
            y[k] = (float)code * s;
        }
        o[i] = (uint32_t)us::float_to_half_bits(y[0]) | ((uint32_t)us::float_to_half_bits(y[1]) << 16);
    }
    // (only a large scale's: on every value it took a long prefix from 43.6 to 48.1 us)
    if (fabsf(s) >= (ELEM == US_I8 ? 511.f : 8188.f)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = us::saturate_half2(o[i]);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int ELEM>
US_DEV uint2 load_codes(const uint8_t* src) {
    if constexpr (ELEM == US_I8) return __ldcg(reinterpret_cast<const uint2*>(src));
    else return make_uint2(__ldcg(reinterpret_cast<const uint32_t*>(src)), 0u);
}

template <int ELEM, int D>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const UsKvCache c, const UsKvCall a, int tokens, uint16_t* __restrict__ K, int64_t ldk,
               uint16_t* __restrict__ V, int64_t ldv) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes, kBytes = D * (ELEM == US_I8 ? 8 : 4) / 8;
    __shared__ int64_t place[kTokens];
    us::pdl_wait();
    const Tokens tk = find_tokens(c, a, tokens);
    find_places(c, tk, place);
    const int j = threadIdx.x % kLanes, rows = (tk.i1 - tk.i0) * c.Hkv;
    for (int r0 = threadIdx.x / kLanes; r0 < rows; r0 += kAtOnce * kRows) {
        uint2 k[kAtOnce], v[kAtOnce];
        uint32_t s[kAtOnce];
        int tok[kAtOnce], h[kAtOnce];
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            const int r = r0 + u * kRows;
            tok[u] = (int)((unsigned)r / (unsigned)c.Hkv), h[u] = r - tok[u] * c.Hkv;
            const int64_t e0 = r < rows ? place[tok[u]] : -1, e = e0 + ((int64_t)h[u] << c.page_shift);
            if (e0 < 0) {
                tok[u] = -1;
                continue;
            }
            k[u] = load_codes<ELEM>(c.k + e * kBytes + j * (kBytes / kLanes));
            v[u] = load_codes<ELEM>(c.v + e * kBytes + j * (kBytes / kLanes));
            s[u] = __ldcg(reinterpret_cast<const uint32_t*>(c.scale) + e);
        }
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            if (tok[u] < 0) continue;
            const int64_t t = tk.row0 + tk.i0 + tok[u];
            *reinterpret_cast<uint4*>(K + t * ldk + h[u] * D + 8 * j) =
                dequantise8<ELEM>(k[u], us::half_bits_to_float((uint16_t)s[u]));
            *reinterpret_cast<uint4*>(V + t * ldv + h[u] * D + 8 * j) =
                dequantise8<ELEM>(v[u], us::half_bits_to_float((uint16_t)(s[u] >> 16)));
        }
    }
    us::pdl_launch_dependents();
}

// One CTA per (head, request): the listed entries of K, of V and the scales are
// read into shared memory, then written, so that a path may overlap itself.  As many
// threads as there are 16-byte pieces of K, so that more CTAs wait side by side.
__global__ void __launch_bounds__(kThreads)
kv_commit_kernel(const UsKvCache c, const UsKvCall a, const int32_t* acc) {
    extern __shared__ __align__(16) uint8_t held[];
    __shared__ int64_t from[US_KV_MAX_COMMIT], to[US_KV_MAX_COMMIT];
    us::pdl_wait();
    const int h = blockIdx.x, b = blockIdx.y;
    int row0;
    const int n = us::kv_rows(a, b, row0, c.status), chunks = c.row_bytes / 16;
    uint32_t* held_s = reinterpret_cast<uint32_t*>(held + (size_t)a.max_n * 2 * c.row_bytes);
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int p0 = a.pos[b], d = acc[row0 + i];
        const int sp = d >= 0 ? us::kv_pos(p0, d) : -1, dp = us::kv_pos(p0, i);
        const int si = us::kv_page(c, b, sp), di = us::kv_page(c, b, dp);
        const bool ok = si >= 0 && di >= 0;
        from[i] = ok ? us::kv_entry(c, si, h, sp) : -1;
        to[i] = ok ? us::kv_entry(c, di, h, dp) : -1;
    }
    __syncthreads();
    uint4* hv = reinterpret_cast<uint4*>(held);
    const uint4* k4 = reinterpret_cast<const uint4*>(c.k);
    const uint4* v4 = reinterpret_cast<const uint4*>(c.v);
    for (int x = threadIdx.x; x < n * chunks; x += blockDim.x) {
        const int i = x / chunks, j = x - i * chunks;
        if (from[i] < 0) continue;
        hv[2 * x] = k4[from[i] * chunks + j];
        hv[2 * x + 1] = v4[from[i] * chunks + j];
        if (j == 0) held_s[i] = reinterpret_cast<const uint32_t*>(c.scale)[from[i]];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < n * chunks; x += blockDim.x) {
        const int i = x / chunks, j = x - i * chunks;
        if (from[i] < 0) continue;
        reinterpret_cast<uint4*>(c.k)[to[i] * chunks + j] = hv[2 * x];
        reinterpret_cast<uint4*>(c.v)[to[i] * chunks + j] = hv[2 * x + 1];
        if (j == 0) reinterpret_cast<uint32_t*>(c.scale)[to[i]] = held_s[i];
    }
    us::pdl_launch_dependents();
}

template <class Kern, class... Args>
us_status launch(Kern kern, dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? US_OK : US_ERR_CUDA;
}

// Tokens of a CTA: four (token, head) rows a thread, or one where that leaves
// SMs without a CTA.
int cta_tokens(const UsKvCache& c, const UsKvCall& a) {
    const int64_t per = kThreads / (c.D / 8), rows = (int64_t)a.max_n * c.B * c.Hkv;
    const int64_t want = rows >= 2 * kAtOnce * per * us::num_sms() ? kAtOnce * per : per;
    const int64_t t = want / c.Hkv;
    return (int)(t < 1 ? 1 : t > kTokens ? kTokens : t);
}
dim3 row_grid(const UsKvCache& c, const UsKvCall& a) {
    const int t = cta_tokens(c, a);
    return dim3((unsigned)((a.max_n + t - 1) / t), (unsigned)c.B);
}

}  // namespace

namespace us {

us_status launch_kv_write(const UsKvCache& c, const UsKvCall& a, const uint16_t* K, int64_t ldk, const uint16_t* V,
                          int64_t ldv, cudaStream_t st) {
    auto kern = c.elem == US_I8 ? (c.D == 64 ? kv_write_kernel<US_I8, 64> : kv_write_kernel<US_I8, 128>)
                                : (c.D == 64 ? kv_write_kernel<US_I4, 64> : kv_write_kernel<US_I4, 128>);
    return launch(kern, row_grid(c, a), kThreads, 0, st, c, a, cta_tokens(c, a), K, ldk, V, ldv);
}

us_status launch_kv_read(const UsKvCache& c, const UsKvCall& a, uint16_t* K, int64_t ldk, uint16_t* V, int64_t ldv,
                         cudaStream_t st) {
    auto kern = c.elem == US_I8 ? (c.D == 64 ? kv_read_kernel<US_I8, 64> : kv_read_kernel<US_I8, 128>)
                                : (c.D == 64 ? kv_read_kernel<US_I4, 64> : kv_read_kernel<US_I4, 128>);
    return launch(kern, row_grid(c, a), kThreads, 0, st, c, a, cta_tokens(c, a), K, ldk, V, ldv);
}

us_status launch_kv_commit(const UsKvCache& c, const UsKvCall& a, const int32_t* acc, cudaStream_t st) {
    const size_t smem = (size_t)a.max_n * (2 * c.row_bytes + 4);
    const int pieces = (a.max_n * (c.row_bytes / 16) + 31) / 32 * 32, threads = pieces < 64 ? 64 : pieces > kThreads ? kThreads : pieces;
    return launch(kv_commit_kernel, dim3((unsigned)c.Hkv, (unsigned)c.B), threads, smem, st, c, a, acc);
}

}  // namespace us

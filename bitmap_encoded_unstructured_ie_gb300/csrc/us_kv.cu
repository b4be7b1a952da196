// us_kv.cu -- writing, reading back and committing the quantised K/V cache.
//
// Write: per token and head, s = fp16_rn(max|x| / q), 1 if that is 0, with
// q = 127 (int8) or 7 (int4), and code = clamp(rint(x / s), -q-1, q): the rule
// of us_quantize_x on one head's row.  Infinities count as +-65504 and NaN as
// 0, so that every stored entry is finite.  Read: y = fp16_rn(code * s).
// Commit: entries of listed tokens move to consecutive positions, all of one
// request's reads before its writes.
#include "us_internal.h"
#include "us_kv.cuh"

namespace {

constexpr int kThreads = 256;

// x as eight fp32 values, infinities at the largest fp16 value, NaN as 0
US_DEV void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = us::half_bits_to_float((uint16_t)(u[i >> 1] >> (16 * (i & 1))));
        x[i] = f == f ? fminf(fmaxf(f, -65504.f), 65504.f) : 0.f;
    }
}

// Quantises one row held eight values a lane by D/8 neighbouring lanes (all
// 32 lanes of the warp take part); stores the lane's codes, returns the scale.
template <int ELEM, int D>
US_DEV uint16_t quantise_row(const float (&x)[8], uint8_t* dst, bool store) {
    constexpr float q = ELEM == US_I8 ? 127.f : 7.f;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
    for (int d = D / 16; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
    uint16_t s16 = us::float_to_half_bits(amax / q);
    if (s16 == 0) s16 = 0x3C00u;                              // 1.0
    const float s = us::half_bits_to_float(s16);
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int c = (int)fminf(fmaxf(rintf(x[i] / s), -q - 1.f), q);
        if constexpr (ELEM == US_I8) w[i >> 2] |= ((uint32_t)c & 0xFFu) << (8 * (i & 3));
        else w[0] |= ((uint32_t)c & 0xFu) << (4 * i);
    }
    if (store) {
        if constexpr (ELEM == US_I8) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(dst) = w[0];
    }
    return s16;
}

// D/8 lanes per (token, head): one 16-byte load of K and of V each, one scale
// pair.  Heads run fastest, so a warp reads contiguous parts of a token's row.
template <int ELEM, int D>
__global__ void __launch_bounds__(kThreads)
kv_write_kernel(const UsKvCache c, const UsKvCall a, const uint16_t* __restrict__ K, int64_t ldk,
                const uint16_t* __restrict__ V, int64_t ldv) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
    us::pdl_wait();
    const int b = blockIdx.y;
    int row0;
    const int n = us::kv_rows(a, b, row0, c.status);
    const int r = blockIdx.x * kRows + threadIdx.x / kLanes, j = threadIdx.x % kLanes;
    const int i = r / c.Hkv, h = r - i * c.Hkv;
    const bool in = i < n;
    const int id = in ? us::kv_page(c, b, us::kv_pos(a.pos[b], i)) : -1;
    float xk[8] = {}, xv[8] = {};
    if (in) {
        const int64_t t = row0 + i;
        unpack8(*reinterpret_cast<const uint4*>(K + t * ldk + h * D + 8 * j), xk);
        unpack8(*reinterpret_cast<const uint4*>(V + t * ldv + h * D + 8 * j), xv);
    }
    const int64_t e = id >= 0 ? us::kv_entry(c, id, h, a.pos[b] + i) : 0;
    const uint16_t sk = quantise_row<ELEM, D>(xk, c.k + e * c.row_bytes + j * (c.row_bytes / kLanes), id >= 0);
    const uint16_t sv = quantise_row<ELEM, D>(xv, c.v + e * c.row_bytes + j * (c.row_bytes / kLanes), id >= 0);
    if (id >= 0 && j == 0) reinterpret_cast<uint32_t*>(c.scale)[e] = (uint32_t)sk | ((uint32_t)sv << 16);
    us::pdl_launch_dependents();
}

// eight codes and a scale -> eight fp16 values
template <int ELEM>
US_DEV uint4 dequantise8(const uint8_t* src, uint16_t s16) {
    const float s = us::half_bits_to_float(s16);
    uint32_t w[2], o[4];
    if constexpr (ELEM == US_I8) {
        const uint2 u = *reinterpret_cast<const uint2*>(src);
        w[0] = u.x, w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(src);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int e = 2 * i + k;
            const int code = ELEM == US_I8 ? (int)(int8_t)(w[e >> 2] >> (8 * (e & 3))) : us::sext4(w[0] >> (4 * e));
            y[k] = (float)code * s;
        }
        o[i] = (uint32_t)us::float_to_half_bits(y[0]) | ((uint32_t)us::float_to_half_bits(y[1]) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int ELEM, int D>
__global__ void __launch_bounds__(kThreads)
kv_read_kernel(const UsKvCache c, const UsKvCall a, uint16_t* __restrict__ K, int64_t ldk,
               uint16_t* __restrict__ V, int64_t ldv) {
    constexpr int kLanes = D / 8, kRows = kThreads / kLanes;
    us::pdl_wait();
    const int b = blockIdx.y;
    int row0;
    const int n = us::kv_rows(a, b, row0, c.status);
    const int r = blockIdx.x * kRows + threadIdx.x / kLanes, j = threadIdx.x % kLanes;
    const int i = r / c.Hkv, h = r - i * c.Hkv;
    if (i < n) {
        const int p = us::kv_pos(a.pos[b], i), id = us::kv_page(c, b, p);
        if (id >= 0) {
            const int64_t e = us::kv_entry(c, id, h, p), t = row0 + i;
            const uint32_t s = reinterpret_cast<const uint32_t*>(c.scale)[e];
            const int64_t at = e * c.row_bytes + j * (c.row_bytes / kLanes);
            *reinterpret_cast<uint4*>(K + t * ldk + h * D + 8 * j) = dequantise8<ELEM>(c.k + at, (uint16_t)s);
            *reinterpret_cast<uint4*>(V + t * ldv + h * D + 8 * j) = dequantise8<ELEM>(c.v + at, (uint16_t)(s >> 16));
        }
    }
    us::pdl_launch_dependents();
}

// One CTA per (head, request): the listed entries of K, of V and the scales are
// read into shared memory, then written, so that a path may overlap itself.
__global__ void __launch_bounds__(kThreads)
kv_commit_kernel(const UsKvCache c, const UsKvCall a, const int32_t* __restrict__ acc) {
    extern __shared__ __align__(16) uint8_t held[];
    __shared__ int64_t from[US_KV_MAX_COMMIT], to[US_KV_MAX_COMMIT];
    us::pdl_wait();
    const int h = blockIdx.x, b = blockIdx.y;
    int row0;
    const int n = us::kv_rows(a, b, row0, c.status), chunks = c.row_bytes / 16;
    uint32_t* held_s = reinterpret_cast<uint32_t*>(held + (size_t)a.max_n * 2 * c.row_bytes);
    for (int i = threadIdx.x; i < n; i += kThreads) {
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
    for (int x = threadIdx.x; x < n * chunks; x += kThreads) {
        const int i = x / chunks, j = x - i * chunks;
        if (from[i] < 0) continue;
        hv[2 * x] = k4[from[i] * chunks + j];
        hv[2 * x + 1] = v4[from[i] * chunks + j];
        if (j == 0) held_s[i] = reinterpret_cast<const uint32_t*>(c.scale)[from[i]];
    }
    __syncthreads();
    for (int x = threadIdx.x; x < n * chunks; x += kThreads) {
        const int i = x / chunks, j = x - i * chunks;
        if (from[i] < 0) continue;
        reinterpret_cast<uint4*>(c.k)[to[i] * chunks + j] = hv[2 * x];
        reinterpret_cast<uint4*>(c.v)[to[i] * chunks + j] = hv[2 * x + 1];
        if (j == 0) reinterpret_cast<uint32_t*>(c.scale)[to[i]] = held_s[i];
    }
    us::pdl_launch_dependents();
}

template <class Kern, class... Args>
us_status launch(Kern kern, dim3 grid, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? US_OK : US_ERR_CUDA;
}

dim3 row_grid(const UsKvCache& c, const UsKvCall& a) {
    const int64_t rows = (int64_t)a.max_n * c.Hkv, per = kThreads / (c.D / 8);
    return dim3((unsigned)((rows + per - 1) / per), (unsigned)c.B);
}

}  // namespace

namespace us {

us_status launch_kv_write(const UsKvCache& c, const UsKvCall& a, const uint16_t* K, int64_t ldk, const uint16_t* V,
                          int64_t ldv, cudaStream_t st) {
    auto kern = c.elem == US_I8 ? (c.D == 64 ? kv_write_kernel<US_I8, 64> : kv_write_kernel<US_I8, 128>)
                                : (c.D == 64 ? kv_write_kernel<US_I4, 64> : kv_write_kernel<US_I4, 128>);
    return launch(kern, row_grid(c, a), 0, st, c, a, K, ldk, V, ldv);
}

us_status launch_kv_read(const UsKvCache& c, const UsKvCall& a, uint16_t* K, int64_t ldk, uint16_t* V, int64_t ldv,
                         cudaStream_t st) {
    auto kern = c.elem == US_I8 ? (c.D == 64 ? kv_read_kernel<US_I8, 64> : kv_read_kernel<US_I8, 128>)
                                : (c.D == 64 ? kv_read_kernel<US_I4, 64> : kv_read_kernel<US_I4, 128>);
    return launch(kern, row_grid(c, a), 0, st, c, a, K, ldk, V, ldv);
}

us_status launch_kv_commit(const UsKvCache& c, const UsKvCall& a, const int32_t* acc, cudaStream_t st) {
    const size_t smem = (size_t)a.max_n * (2 * c.row_bytes + 4);
    return launch(kv_commit_kernel, dim3((unsigned)c.Hkv, (unsigned)c.B), smem, st, c, a, acc);
}

}  // namespace us

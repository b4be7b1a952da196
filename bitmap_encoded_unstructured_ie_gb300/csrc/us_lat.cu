// us_lat.cu -- writing, reading back and committing the cache of latent rows.
//
// Write: the Dc latent values are normed (y = x rsqrt(mean(x^2) + eps) w), the 64
// values of the shared key turned by their position as in us_rope.cu, all in fp32,
// rounded once to fp16, kept finite.  A warp has a token: 16 bytes a lane of each 256
// latent values, and one pair of the key, whose angle is its own.  Eight tokens a CTA.
// Commit: entries of listed tokens move to consecutive positions, all of a request's
// reads before its writes; 128 bytes of every row a CTA.
//
// Bytes bound the long calls (three prompts of up to 8192 tokens written and read back, 85 MB:
// 16.4 us, 5.2 TB/s; 12.5 us at a copy's rate), latency the short ones (offsets and table, rows,
// the sum's shuffles: a token each of 24 requests written and read back 3.6 us).
#include "us_internal.h"
#include "us_lat.cuh"
#include "us_launch.cuh"

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

US_DEV float finite(float x) { return x == x ? fminf(fmaxf(x, -65504.f), 65504.f) : 0.f; }
US_DEV uint32_t pack(float a, float b) {
    return (uint32_t)us::float_to_half_bits(finite(a)) | ((uint32_t)us::float_to_half_bits(finite(b)) << 16);
}

template <int DC>
__global__ void __launch_bounds__(kThreads)
lat_write_kernel(const UsLatCache L, const UsKvCall a, const us_rope rope, const uint16_t* X, int64_t ldx,
                 const uint16_t* w, const int32_t* depth) {
    constexpr int kV = DC / 256;
    us::pdl_wait();
    const int b = blockIdx.y, lane = threadIdx.x & 31, i = blockIdx.x * kWarps + (threadIdx.x >> 5), pos = a.pos[b];
    int row0;
    const int n = us::kv_rows(a, b, row0, L.c.status);
    if (i < n) {
        const uint16_t* x = X + (int64_t)(row0 + i) * ldx;
        uint4 in[kV], wv[kV];
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            in[v] = __ldcs(reinterpret_cast<const uint4*>(x) + 32 * v + lane);
            if (w) wv[v] = reinterpret_cast<const uint4*>(w)[32 * v + lane];
        }
        // the lane's pair of the key
        const bool pairs = rope.style == US_ROPE_PAIRS || !rope.R;
        const uint16_t* xr = x + DC;
        float ka, kb;
        if (pairs) {
            const uint32_t u = reinterpret_cast<const uint32_t*>(xr)[lane];
            ka = us::half_bits_to_float((uint16_t)u), kb = us::half_bits_to_float((uint16_t)(u >> 16));
        } else {
            ka = us::half_bits_to_float(xr[lane]), kb = us::half_bits_to_float(xr[lane + 32]);
        }
        const int64_t to = us::lat_row(L, b, us::kv_pos(pos, i));
        float c = 1.f, s = 0.f;
        if (rope.R) {
            const int at = us::kv_pos(pos, depth ? depth[row0 + i] : i);
            const int32_t turn = (int32_t)(((uint64_t)(int64_t)at * rope.turns[lane]) >> 32);
            sincospif((float)turn * 0x1p-31f, &s, &c);
        }
        float y[kV][8], ss = 0.f;
#pragma unroll
        for (int v = 0; v < kV; ++v) {
            const uint32_t u[4] = {in[v].x, in[v].y, in[v].z, in[v].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
                y[v][2 * j] = f.x, y[v][2 * j + 1] = f.y;
                ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
            }
        }
        if (w) {
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
            const float f = rsqrtf(ss / (float)DC + rope.eps);
#pragma unroll
            for (int v = 0; v < kV; ++v) {
                const uint32_t u[4] = {wv[v].x, wv[v].y, wv[v].z, wv[v].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
                    y[v][2 * j] = y[v][2 * j] * f * g.x, y[v][2 * j + 1] = y[v][2 * j + 1] * f * g.y;
                }
            }
        }
        if (to >= 0) {
            uint16_t* row = L.rows + to;
#pragma unroll
            for (int v = 0; v < kV; ++v)
                reinterpret_cast<uint4*>(row)[32 * v + lane] = make_uint4(pack(y[v][0], y[v][1]), pack(y[v][2], y[v][3]),
                                                                          pack(y[v][4], y[v][5]), pack(y[v][6], y[v][7]));
            // (without a rotation a value does not meet its neighbour, which may not be finite)
            const uint32_t k2 = rope.R ? pack(ka * c - kb * s, kb * c + ka * s) : pack(ka, kb);
            if (pairs) {
                reinterpret_cast<uint32_t*>(row + DC)[lane] = k2;
            } else {
                row[DC + lane] = (uint16_t)k2, row[DC + 32 + lane] = (uint16_t)(k2 >> 16);
            }
        }
    }
    us::pdl_launch_dependents();
}

__global__ void __launch_bounds__(kThreads)
lat_read_kernel(const UsLatCache L, const UsKvCall a, uint16_t* X, int64_t ldx) {
    us::pdl_wait();
    const int b = blockIdx.y, lane = threadIdx.x & 31, i = blockIdx.x * kWarps + (threadIdx.x >> 5), pos = a.pos[b];
    int row0;
    const int n = us::kv_rows(a, b, row0, L.c.status);
    if (i < n) {
        const int64_t from = us::lat_row(L, b, us::kv_pos(pos, i));
        if (from >= 0) {
            const uint4* src = reinterpret_cast<const uint4*>(L.rows + from);
            uint4* dst = reinterpret_cast<uint4*>(X + (int64_t)(row0 + i) * ldx);
            uint4 v[3];
#pragma unroll
            for (int u = 0; u < 3; ++u)
                if (32 * u + lane < L.W / 8) v[u] = __ldcg(src + 32 * u + lane);
#pragma unroll
            for (int u = 0; u < 3; ++u)
                if (32 * u + lane < L.W / 8) dst[32 * u + lane] = v[u];
        }
    }
    us::pdl_launch_dependents();
}

// blockIdx.x: which 128 bytes of the rows
__global__ void __launch_bounds__(kThreads)
lat_commit_kernel(const UsLatCache L, const UsKvCall a, const int32_t* acc) {
    __shared__ uint4 held[US_KV_MAX_COMMIT * 8];
    __shared__ int64_t from[US_KV_MAX_COMMIT], to[US_KV_MAX_COMMIT];
    us::pdl_wait();
    const int b = blockIdx.y;
    int row0;
    const int n = us::kv_rows(a, b, row0, L.c.status);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int p0 = a.pos[b], d = acc[row0 + i];
        const int64_t s = us::lat_row(L, b, d >= 0 ? us::kv_pos(p0, d) : -1), t = us::lat_row(L, b, us::kv_pos(p0, i));
        from[i] = t < 0 ? -1 : s;
        to[i] = t;
    }
    __syncthreads();
    const int at = blockIdx.x * 64;
    for (int x = threadIdx.x; x < n * 8; x += kThreads)
        if (from[x / 8] >= 0) held[x] = reinterpret_cast<const uint4*>(L.rows + from[x / 8] + at)[x % 8];
    __syncthreads();
    for (int x = threadIdx.x; x < n * 8; x += kThreads)
        if (from[x / 8] >= 0) reinterpret_cast<uint4*>(L.rows + to[x / 8] + at)[x % 8] = held[x];
    us::pdl_launch_dependents();
}

dim3 token_grid(const UsKvCall& a, int B) { return dim3((unsigned)((a.max_n + kWarps - 1) / kWarps), (unsigned)B); }

}  // namespace

namespace us {

us_status launch_lat_write(const UsLatCache& L, const UsKvCall& a, const us_rope& rope, const uint16_t* X, int64_t ldx,
                           const uint16_t* w, const int32_t* depth, cudaStream_t st) {
    auto kern = L.Dc == 512 ? lat_write_kernel<512> : lat_write_kernel<256>;
    return launch_pdl(kern, token_grid(a, L.c.B), kThreads, 0, st, L, a, rope, X, ldx, w, depth);
}

us_status launch_lat_read(const UsLatCache& L, const UsKvCall& a, uint16_t* X, int64_t ldx, cudaStream_t st) {
    return launch_pdl(lat_read_kernel, token_grid(a, L.c.B), kThreads, 0, st, L, a, X, ldx);
}

us_status launch_lat_commit(const UsLatCache& L, const UsKvCall& a, const int32_t* acc, cudaStream_t st) {
    return launch_pdl(lat_commit_kernel, dim3((unsigned)(L.W / 64), (unsigned)L.c.B), kThreads, 0, st, L, a, acc);
}

}  // namespace us

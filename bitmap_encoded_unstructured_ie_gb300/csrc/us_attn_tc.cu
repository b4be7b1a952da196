// us_attn_tc.cu -- attention of many query rows per key head over the quantised
// K/V cache (drafted trees, chunks of a prompt), on the tensor cores (tcgen05).
//
// Same function as us_attn.cu.  A segment is (request, key head, block of 128 NQ
// query rows); its positions come in tiles of 128, and the tiles of all segments
// are spread evenly over the CTAs (one an SM):
//   S = Q Ck^T    A = Q (shared memory), B = the tile's K codes as fp16
//   O += P Cv     A = P (TMEM, fp16), B = the tile's V codes as fp16, MN-major
// K enters as its codes, its scale on the scores in fp32.  V enters as fp16(code *
// scale), the values that us_kv_read returns: one more rounding of 2^-11 of a value,
// against a register's worth of shared memory traffic per score for a scale in the
// weights.  The dimensions stand in shared memory in the order in which the codes
// leave their words (within each eight), the same for Q, K and V; only the outputs
// are put back.
//
// Two streams, each with its own scores, outputs, row references and softmax
// warps, so that the tensor cores work on one while the other's weights are made.
// With more than 128 rows (NQ = 2) a stream is a half of the rows and takes every
// tile: each tile's codes are converted once for 256 rows.  Else (NQ = 1) the tiles
// alternate between the streams, which are joined at the segment's end.
//   warps 0-3, 4-7: softmax of stream 0 / 1, 32 rows each, 16 at a time, in the
//               fragment order of 16-lane TMEM loads: a lane has a quarter of the
//               columns, so it reads a quarter of the scales (what bounds these warps
//               is the load / store pipe: every register that comes from TMEM or
//               shared memory takes a cycle of it a warp)
//   warp 8: one thread issues the MMAs: PV of a tile, then QK of the stream's next
//               (it is held up at the rate of their execution, 64 cycles each)
//   warps 9-15: codes -> fp16, in items of 16 positions of K or of V; the codes of
//               a warp's next two items are on their way to its registers
// 16 warps: a thread may have 128 registers (17 would leave 96).
// Weights are 2^(s - R); a row's reference R is its maximum less 11 when it is set,
// and moves only when a weight could pass 2^15 (fp16 keeps 2^-14 of them exactly as
// it does the largest).  R, sums and outputs of a segment shared by several CTAs are
// joined by the last of them to arrive.
#include "us_attn.cuh"
#include "us_internal.h"
#include "us_tcgen05.cuh"

namespace {

using namespace us::attn;

constexpr int kM = 128, kTile = 128;              // query rows of a stream, positions of a tile
constexpr int kSoftWarps = 8, kMmaWarp = 8, kConvWarps = 7;
constexpr int kThreads = 32 * (kSoftWarps + 1 + kConvWarps);
constexpr int kItems = 16;                        // of a tile: 8 of K, then 8 of V
constexpr int kKS = 2, kSS = 4;                   // stages: K, scales (V: Shape::kVS)
constexpr float kTop = 11.f, kLag = 4.f;          // a row's largest weight is 2^11 at first, 2^15 at most

struct Header {
    uint64_t k_full[kKS], k_free[kKS], v_full[3], v_free[3], s_full[kSS];
    uint64_t qk_done[2], p_full[2], pv_done[2];   // by stream
    uint64_t q_full;
    alignas(16) float ks[kSS][kTile];                         // K's scales times scale log2(e) of the tiles on their way
    alignas(16) uint16_t valid[kSS][8];                       // which of 16 positions exist
    float xr[2][kM], xl[2][kM];                   // the streams' references and sums
    uint32_t tmem;
    unsigned last;
    int parts;
    Part part[2];
    Work work;
};

static_assert(offsetof(Header, ks) % 16 == 0 && offsetof(Header, valid) % 16 == 0, "read 8 and 16 bytes at a time");
constexpr int kNoPage = -0x7fffffff - 1;          // nothing to read (any other bad number is recorded)

template <int ELEM, int D, int NQ>
struct Shape {
    static constexpr int kRow = D * (ELEM == US_I8 ? 8 : 4) / 8;    // bytes of a row of codes
    static constexpr int kC = kRow / 16;                            // 16-byte chunks of it
    static constexpr int kLoads = kC / 2;                           // chunks a lane converts of 16 rows
    static constexpr int kOut = ELEM == US_I8 ? 2 : 4;              // 16-byte chunks of fp16 a chunk becomes
    static constexpr int kOperand = 128 * D * 2;                    // Q, K tile or V tile as fp16
    static constexpr int kGroup = 128 * 128;                        // one 64-dimension half of it
    static constexpr int kRows = kM * NQ;                           // query rows of a segment
    static constexpr int kVS = NQ == 2 ? 2 : 3;
    static constexpr int kSmem = (NQ + kKS + kVS) * kOperand + (int)sizeof(Header) + 1024;
    static constexpr int kSlotFloats = 2 * kRows + kRows * D;
};

// Column j of eight -> its dimension of eight: the order in which codes leave a word.
template <int ELEM>
US_DEV constexpr int dim_of(int j) {
    return ELEM == US_I8 ? (j & 4) | ((j & 1) << 1) | ((j >> 1) & 1) : ((j & 1) << 2) | (j >> 1);
}

// 16 bytes of codes -> kOut chunks of eight fp16 values
template <int ELEM>
US_DEV void convert(uint4 u, uint4 (&out)[ELEM == US_I8 ? 2 : 4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (ELEM == US_I8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t a[2], b[2];
            decode_i8(w[2 * i], a);
            decode_i8(w[2 * i + 1], b);
            out[i] = make_uint4(a[0], a[1], b[0], b[1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[4];
            decode_i4(w[i], a);
            out[i] = make_uint4(a[0], a[1], a[2], a[3]);
        }
    }
}

// Eight fp16 values in the order of dim_of
template <int ELEM>
US_DEV uint4 reorder(uint4 u) {
    if constexpr (ELEM == US_I8)
        return make_uint4(__byte_perm(u.x, u.y, 0x5410), __byte_perm(u.x, u.y, 0x7632), __byte_perm(u.z, u.w, 0x5410),
                          __byte_perm(u.z, u.w, 0x7632));
    else
        return make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632), __byte_perm(u.y, u.w, 0x5410),
                          __byte_perm(u.y, u.w, 0x7632));
}

// 16-byte chunk `chunk` of row `row` of an operand (64-dimension halves, 128-byte swizzle)
US_DEV uint8_t* operand_at(uint8_t* base, int row, int chunk) {
    return base + (chunk >> 3) * (128 * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// Eight outputs in the order of dim_of -> fp16 in the order of the dimensions
template <int ELEM>
US_DEV void store8(uint16_t* out, const float* y, float f) {
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[dim_of<ELEM>(j)] = y[j] * f;
    *reinterpret_cast<uint4*>(out) =
        make_uint4(pack_half2(d[0], d[1]), pack_half2(d[2], d[3]), pack_half2(d[4], d[5]), pack_half2(d[6], d[7]));
}

// The last CTA of a shared segment joins the partial states: 4 / NQ threads take a
// row's columns, O stands as float4 of four columns, row after row.
template <int ELEM, int D, int NQ>
US_DEV void join_states(const UsAttnParams& p, const Part& a) {
    using Sh = Shape<ELEM, D, NQ>;
    constexpr int kRows = Sh::kRows, kCols = D * NQ / 4, kN = kCols / 4;
    static_assert(kThreads == 4 * kM, "threads of a row");
    const int row = threadIdx.x & (kRows - 1), part = threadIdx.x / kRows;
    if (row >= a.rows) return;
    float top = -INFINITY, sum = 0.f, y[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) y[i] = 0.f;
#pragma unroll 4
    for (int c = a.first; c <= a.last; ++c) top = fmaxf(top, __ldcg(p.ws_slots + a.slot(c) * Sh::kSlotFloats + row));
    for (int c = a.first; c <= a.last; ++c) {
        const float* sl = p.ws_slots + a.slot(c) * Sh::kSlotFloats;
        const float r = __ldcg(sl + row), f = r == -INFINITY ? 0.f : ex2(r - top);
        sum += __ldcg(sl + kRows + row) * f;
        const float4* o = reinterpret_cast<const float4*>(sl + 2 * kRows) + part * kN * kRows + row;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            const float4 v = __ldcg(o + i * kRows);
            y[4 * i] += v.x * f, y[4 * i + 1] += v.y * f, y[4 * i + 2] += v.z * f, y[4 * i + 3] += v.w * f;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* out = out_row<kRows>(p, a.row0, a.h, a.rb, row, D) + part * kCols;
#pragma unroll
    for (int i = 0; i < kCols / 8; ++i) store8<ELEM>(out + 8 * i, y + 8 * i, inv);
}

template <int ELEM, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const UsAttnParams p) {
    using Sh = Shape<ELEM, D, NQ>;
    constexpr int kRows = Sh::kRows, kVS = Sh::kVS;
    using Cur = Cursor<kRows, kTile>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* q_sm = smem;
    uint8_t* k_sm = q_sm + NQ * Sh::kOperand;
    uint8_t* v_sm = k_sm + kKS * Sh::kOperand;
    Header& H = *reinterpret_cast<Header*>(v_sm + kVS * Sh::kOperand);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKS; ++i) us::mbar_init(&H.k_full[i], 8), us::mbar_init(&H.k_free[i], 1);
        for (int i = 0; i < kVS; ++i) us::mbar_init(&H.v_full[i], 8), us::mbar_init(&H.v_free[i], 1);
        for (int i = 0; i < kSS; ++i) us::mbar_init(&H.s_full[i], 8);
        for (int i = 0; i < 2; ++i)
            us::mbar_init(&H.qk_done[i], 1), us::mbar_init(&H.p_full[i], 4), us::mbar_init(&H.pv_done[i], 1);
        us::mbar_init(&H.q_full, kSoftWarps);
        us::fence_mbar_init();
    }
    if (warp == kSoftWarps) us::tmem_alloc(&H.tmem, 512);
    us::pdl_wait();

    Work wk;
    Cur cur;
    const bool any = find_work<kRows, kTile, kThreads>(p, wk, cur);       // its barrier covers the set-up above
    if (threadIdx.x == 0) H.work = wk;                     // the softmax warps need it at a segment's end
    us::tc_fence_after();
    const uint32_t tmem = H.tmem;                          // S0, S1, O0, O1: 128 columns each
    const int count = any ? (int)(wk.t1 - wk.t0) : 0, G = p.G;
    bool failed = false;
    auto wait = [&](uint64_t* bar, int use) {              // for the use-th completion of bar
        if (!failed && !us::mbar_wait(bar, (uint32_t)use & 1u, p.c.status)) failed = true;
    };

    if (warp < kSoftWarps) {
        // ----------------------------------------------------------- softmax
        const int st = warp >> 2, g = lane >> 2, c2 = 2 * (lane & 3);
        const int wrow = (warp & 3) * 32 + (NQ == 2 ? kM * st : 0);           // the warp's first row of the segment
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t s_tm = tmem + lanes + st * 128, o_tm = tmem + lanes + 256 + st * 128;
        int parts = 0;
        for (int it = 0; it < count;) {
            // ---- a segment, or this CTA's part of it: tiles it .. end - 1
            const int end = min(count, it + cur.tiles - cur.tile), tile0 = cur.tile;
            const int rows = min(kRows, cur.r.n * G - cur.rb * kRows);
#pragma unroll
            for (int x = threadIdx.x; x < kRows * (D / 8); x += 32 * kSoftWarps) {
                const int r = x / (D / 8), chunk = x % (D / 8), rr = cur.rb * kRows + r, i = rr / G;
                uint4 u = make_uint4(0, 0, 0, 0);
                if (r < rows)
                    u = *reinterpret_cast<const uint4*>(p.Q + (int64_t)(cur.r.row0 + i) * p.ldq + (int64_t)(cur.h * G + rr - i * G) * D + 8 * chunk);
                *reinterpret_cast<uint4*>(operand_at(q_sm + (r / kM) * Sh::kOperand, r % kM, chunk)) = reorder<ELEM>(u);
            }
            us::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) us::mbar_arrive(&H.q_full);
            // positions that a row sees among 32 from `base` behind the context
            auto seen32 = [&](int base, uint64_t tree, int chain) {
                if (base <= -32) return 0xFFFFFFFFu;
                const int lo = base < 0 ? -base : 0;       // context positions among them
                uint32_t own;
                if (p.mask) {
                    own = base < 64 ? (uint32_t)(tree >> (base > 0 ? base : 0)) : 0u;
                } else {
                    const int k = chain - (base > 0 ? base : 0);
                    own = k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
                }
                return (own << lo) | (lo ? 0xFFFFFFFFu >> (32 - lo) : 0u);
            };
            float R[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
            uint64_t l2[2][2] = {};                        // two partial sums each
            constexpr int kStep = NQ == 2 ? 1 : 2;         // a stream's tiles: every one, or every other
            const int i0 = NQ == 2 ? it : it + ((it ^ st) & 1);
            for (int i = i0; i < end; i += kStep) {
                const int ss = i % kSS;
                wait(&H.s_full[ss], i / kSS);
                wait(&H.qk_done[st], i / kStep);
                us::tc_fence_after();
                const float2* ks2 = reinterpret_cast<const float2*>(H.ks[ss]) + (lane & 3);
                const uint4 ok = *reinterpret_cast<const uint4*>(H.valid[ss]);
                const int base = (tile0 + i - it) * kTile - cur.r.ctx;
                const bool edge = base + kTile > 0 || (ok.x & ok.y & ok.z & ok.w) != 0xFFFFFFFFu;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (wrow + 16 * h >= rows) continue;
                    const uint32_t half = (uint32_t)(16 * h) << 16;
                    float v[64];
                    us::tmem_ld_frag128(s_tm + half, v);
                    // scores and their maxima
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 sk = ks2[4 * k];
                        const uint64_t s = pair(sk.x, sk.y);
                        unpair(mul2(pair(v[4 * k], v[4 * k + 1]), s), v[4 * k], v[4 * k + 1]);
                        unpair(mul2(pair(v[4 * k + 2], v[4 * k + 3]), s), v[4 * k + 2], v[4 * k + 3]);
                    }
                    if (edge) {
                        const uint32_t okw[4] = {ok.x, ok.y, ok.z, ok.w};
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const int r = wrow + 16 * h + 8 * u + g, tok = (cur.rb * kRows + r) / G;
                            const uint64_t mask = p.mask && r < rows ? p.mask[cur.r.row0 + tok] & (~0ull >> (64 - cur.r.n)) : 0ull;
                            const int own = r < rows ? tok + 1 : 0;        // a chain's row sees so many of the call
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const uint32_t seen = (seen32(base + 32 * c, mask, own) & okw[c]) >> c2;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (!((seen >> (8 * k + e)) & 1u)) v[4 * (4 * c + k) + 2 * u + e] = -INFINITY;
                            }
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        mx[0] = max3(mx[0], v[4 * k], v[4 * k + 1]);
                        mx[1] = max3(mx[1], v[4 * k + 2], v[4 * k + 3]);
                    }
                    if (__any_sync(0xffffffffu, mx[0] > R[h][0] + (kTop + kLag) || mx[1] > R[h][1] + (kTop + kLag))) {
                        float f[2];
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float x = mx[u];
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                            const float to = x > R[h][u] + (kTop + kLag) ? x - kTop : R[h][u];
                            f[u] = to == R[h][u] ? 1.f : ex2(R[h][u] - to);
                            R[h][u] = to;
                            l2[h][u] = mul2(l2[h][u], pair(f[u], f[u]));
                        }
                        if (i - it >= kStep) {             // the stream has outputs: PV of its last tile first
                            wait(&H.pv_done[st], i / kStep - 1);
                            us::tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 32) {
                                uint32_t w[16];
                                us::tmem_ld_frag32(o_tm + half + c, w);
#pragma unroll
                                for (int j = 0; j < 16; ++j) w[j] = __float_as_uint(__uint_as_float(w[j]) * f[(j >> 1) & 1]);
                                us::tmem_st_frag32(o_tm + half + c, w);
                            }
                            us::tmem_wait_st();
                        }
                    }
                    // weights, as fp16 over the scores
                    uint32_t w[32];
                    uint64_t neg[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float ref = R[h][u] == -INFINITY ? 0.f : R[h][u];
                        neg[u] = pair(-ref, -ref);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            float a, b;
                            unpair(add2(pair(v[4 * k + 2 * u], v[4 * k + 2 * u + 1]), neg[u]), a, b);
                            a = ex2(a), b = ex2(b);
                            l2[h][u] = add2(l2[h][u], pair(a, b));
                            w[2 * k + u] = pack_half2(a, b);
                        }
                    us::tmem_st_pairs64(s_tm + half, w);
                }
                us::tmem_wait_st();
                us::tc_fence_before();
                __syncwarp();
                if (lane == 0) us::mbar_arrive(&H.p_full[st]);
            }
            // ---- the segment's end: the streams' sums and outputs
            const int srow = (warp & 3) * 32;              // the warp's first row of its stream
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float a, b;
                    unpair(l2[h][u], a, b);
                    a += b;
                    a += __shfl_xor_sync(0xffffffffu, a, 1);
                    a += __shfl_xor_sync(0xffffffffu, a, 2);
                    if (c2 == 0) H.xr[st][srow + 16 * h + 8 * u + g] = R[h][u], H.xl[st][srow + 16 * h + 8 * u + g] = a;
                }
            // the streams whose outputs the warp reads, and whether they had a tile
            bool has[2];
            if constexpr (NQ == 2) {
                has[0] = true, has[1] = false;
                wait(&H.pv_done[st], end - 1);
                __syncwarp();
            } else {
                has[0] = end - it >= 2 || !(it & 1), has[1] = end - it >= 2 || (it & 1);
                wait(&H.pv_done[(end - 1) & 1], (end - 1) / 2);
                if (end - it >= 2) wait(&H.pv_done[end & 1], (end - 2) / 2);
                us::named_bar_sync(1, 32 * kSoftWarps);
            }
            us::tc_fence_after();
            const int64_t s0 = H.work.t0 + it - tile0;
            const Part part = H.work.sharers(s0, s0 + cur.tiles, cur, rows);
            const bool whole = part.first == part.last;
            if (wrow < rows) {
                const int row = wrow + lane, sr = srow + lane, s1 = NQ == 2 ? st : 0;
                const float r0 = H.xr[s1][sr], r1 = NQ == 2 ? -INFINITY : H.xr[1][sr], top = fmaxf(r0, r1);
                const float f0 = r0 == -INFINITY ? 0.f : ex2(r0 - top), f1 = r1 == -INFINITY ? 0.f : ex2(r1 - top);
                const float sum = H.xl[s1][sr] * f0 + (NQ == 2 ? 0.f : H.xl[1][sr] * f1), inv = sum == 0.f ? 0.f : 1.f / sum;
                float* slot = p.ws_slots + part.slot(blockIdx.x) * Sh::kSlotFloats;
                if (!whole && (NQ == 2 || st == 0)) {
                    __stcg(slot + row, top);
                    __stcg(slot + kRows + row, sum);
                }
                uint16_t* out = row < rows ? out_row<kRows>(p, cur.r.row0, cur.h, cur.rb, row, D) : nullptr;
                // NQ = 1: each stream's warps put out half of the columns
                const int c0 = NQ == 2 ? 0 : st * (D / 2), c1 = NQ == 2 ? D : c0 + D / 2;
#pragma unroll 1
                for (int c = c0; c < c1; c += 16) {
                    float a[16], b[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) a[j] = b[j] = 0.f;
                    if (has[0]) us::tmem_ld16(tmem + lanes + 256 + s1 * 128 + c, a);
                    if (NQ == 1 && has[1]) us::tmem_ld16(tmem + lanes + 384 + c, b);
#pragma unroll
                    for (int j = 0; j < 16; ++j) a[j] = (f0 == 0.f ? 0.f : a[j] * f0) + (f1 == 0.f ? 0.f : b[j] * f1);
                    if (whole) {
                        if (row < rows) {
                            store8<ELEM>(out + c, a, inv);
                            store8<ELEM>(out + c + 8, a + 8, inv);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            __stcg(reinterpret_cast<float4*>(slot + 2 * kRows) + (c + j) / 4 * kRows + row,
                                   make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]));
                    }
                }
            }
            if (!whole) {
                if (threadIdx.x == 0) H.part[parts] = part;
                ++parts;
            }
            us::tc_fence_before();
            us::named_bar_sync(1, 32 * kSoftWarps);        // Q, the streams' TMEM and sums are free
            us::tc_fence_after();
            it = end;
            if (it < count) cur.next_segment(p);
        }
        if (threadIdx.x == 0) H.parts = parts;
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------------- MMA
        if (lane == 0) {
            int segment = 0;
            for (int it = 0; it < count; ++segment) {
                const int end = min(count, it + cur.tiles - cur.tile);
                // scores of tile i for stream st, and whether they are the last that read its K
                auto qk = [&](int i, int st, bool last) {
                    constexpr uint32_t id = us::umma_idesc_f16(kM, kTile);
                    wait(&H.k_full[i % kKS], i / kKS);
                    us::tc_fence_after();
                    const uint64_t qd = us::umma_smem_desc_sw128(q_sm + (NQ == 2 ? st * Sh::kOperand : 0));
                    const uint64_t kd = us::umma_smem_desc_sw128(k_sm + (i % kKS) * Sh::kOperand);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t at = (uint64_t)(((kk >> 2) * Sh::kGroup + (kk & 3) * 32) >> 4);
                        us::umma_f16(tmem + st * 128, qd + at, kd + at, id, kk > 0);
                    }
                    us::umma_commit(&H.qk_done[st]);
                    if (last) us::umma_commit(&H.k_free[i % kKS]);
                };
                // outputs of tile i for stream st; its weights are the stream's use-th
                auto pv = [&](int i, int st, int use, bool first, bool last) {
                    constexpr uint32_t id = us::umma_idesc_f16(kM, D) | us::kUmmaBMajorMN;
                    wait(&H.v_full[i % kVS], i / kVS);
                    wait(&H.p_full[st], use);
                    us::tc_fence_after();
                    const uint64_t vd = us::umma_smem_desc_mn_sw128(v_sm + (i % kVS) * Sh::kOperand, Sh::kGroup);
#pragma unroll
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        us::umma_f16_ta(tmem + 256 + st * 128, tmem + st * 128 + 8 * kk, vd + (uint64_t)(kk * 2048 >> 4), id,
                                        !first || kk > 0);
                    us::umma_commit(&H.pv_done[st]);
                    if (last) us::umma_commit(&H.v_free[i % kVS]);
                };
                wait(&H.q_full, segment);
                if constexpr (NQ == 2) {
                    qk(it, 0, false);
                    qk(it, 1, true);
                    for (int i = it; i < end; ++i)
#pragma unroll
                        for (int st = 0; st < 2; ++st) {
                            pv(i, st, i, i == it, st == 1);
                            if (i + 1 < end) qk(i + 1, st, st == 1);
                        }
                } else {
                    qk(it, it & 1, true);
                    if (it + 1 < end) qk(it + 1, (it + 1) & 1, true);
                    for (int i = it; i < end; ++i) {
                        pv(i, i & 1, i / 2, i - it < 2, true);
                        if (i + 2 < end) qk(i + 2, i & 1, true);
                    }
                }
                it = end;
                if (it < count) cur.next_segment(p);
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- conversion
        // Items in their order, tile after tile across segments: item x of the CTA is
        // block x % 16 of tile x / 16, every seventh is this warp's.  Three are under
        // way: the page number of one, the codes of one, the conversion of one.
        struct Where {
            int item, page, pos, h, left;                  // left: positions up to the last of the request
        };
        int next_item = warp - kSoftWarps - 1, tile = 0;   // the cursor's tile
        auto locate = [&]() {
            Where w = {next_item, kNoPage, 0, 0, 0};
            next_item += kConvWarps;
            const int i = w.item / kItems;
            if (i < count) {
                if (i > tile) cur.next(p), ++tile;
                w.pos = cur.tile * kTile + (w.item & 7) * 16;
                w.h = cur.h;
                w.left = cur.r.ctx + cur.r.n - w.pos;
                if (w.left > 0) w.page = p.c.table[(int64_t)cur.b * p.c.max_pages + (w.pos >> p.c.page_shift)];
            }
            return w;
        };
        struct Codes {
            uint4 c[Sh::kLoads];
            uint32_t scale;                                // (K, V) scales of position `lane`
        };
        auto row_chunk = [&](int u, int& r, int& chunk) {  // eight lanes on eight rows: no bank conflicts
            if constexpr (Sh::kC == 2) r = lane & 15, chunk = lane >> 4;
            else r = 8 * (u / (Sh::kC / 4)) + (lane & 7), chunk = 4 * (u % (Sh::kC / 4)) + (lane >> 3);
        };
        // where a lane's first chunk of an item goes (operand_at, with what depends on
        // the lane alone): its row, its 64 dimensions, and the swizzled chunk
        uint32_t put_base, put_chunk;
        {
            int r, chunk;
            row_chunk(0, r, chunk);
            put_base = (uint32_t)(r * 128 + (chunk * Sh::kOut >> 3) * Sh::kGroup);
            put_chunk = (uint32_t)(((chunk * Sh::kOut & 7) ^ (r & 7)) << 4);
        }
        auto exists = [&](const Where& w) { return w.page >= 0 && w.page < p.c.num_pages; };
        auto fetch = [&](const Where& w, Codes& f) {
            const bool ok = exists(w);
            if (w.page != kNoPage && !ok) us::set_status(p.c.status, US_ERR_CORRUPT);
            const int64_t e = us::kv_entry(p.c, w.page, w.h, w.pos);
            const uint8_t* src = (w.item & 8 ? p.c.v : p.c.k) + e * Sh::kRow;
#pragma unroll
            for (int u = 0; u < Sh::kLoads; ++u) {
                int r, chunk;
                row_chunk(u, r, chunk);
                f.c[u] = ok ? __ldcg(reinterpret_cast<const uint4*>(src + r * Sh::kRow) + chunk) : make_uint4(0, 0, 0, 0);
            }
            f.scale = ok && lane < 16 ? __ldcg(reinterpret_cast<const uint32_t*>(p.c.scale) + e + lane) : 0u;
        };
        // one item: its place in the ring, the conversion, the sign that it is there
        auto convert_item = [&](const Where& w, const Codes& f) {
            const int i = w.item / kItems, block = w.item & 7, ss = i % kSS;
            const bool is_v = (w.item & 8) != 0;
            // Entries that no row sees may hold any scale: behind the request's last
            // position V's counts as 0, and one that is not finite is left to those
            // who see its entry, through K's.
            float sk = us::half_bits_to_float((uint16_t)f.scale) * (p.scale * 1.4426950408889634f);
            uint32_t sv = f.scale >> 16;
            if ((sv & 0x7C00u) == 0x7C00u) sv = 0, sk = __uint_as_float(0x7FC00000u);
            if (lane >= w.left) sv = 0;
            sv |= sv << 16;
            uint8_t* operand;
            if (is_v) {
                if (i >= kVS) wait(&H.v_free[i % kVS], i / kVS - 1);
                operand = v_sm + (i % kVS) * Sh::kOperand;
            } else {
                if (i >= kKS) wait(&H.k_free[i % kKS], i / kKS - 1);
                operand = k_sm + (i % kKS) * Sh::kOperand;
                if (lane < 16) H.ks[ss][16 * block + lane] = sk;
                if (lane == 0) H.valid[ss][block] = exists(w) ? 0xFFFFu : 0u;
            }
            uint8_t* at = operand + block * 16 * 128 + put_base;
#pragma unroll
            for (int u = 0; u < Sh::kLoads; ++u) {
                uint4 out[Sh::kOut];
                convert<ELEM>(f.c[u], out);
                if (is_v) {
                    const uint32_t s = __shfl_sync(0xffffffffu, sv, Sh::kC == 2 ? lane & 15 : 8 * (u / (Sh::kC / 4)) + (lane & 7));
#pragma unroll
                    for (int k = 0; k < Sh::kOut; ++k)
                        out[k] = make_uint4(hmul2(out[k].x, s), hmul2(out[k].y, s), hmul2(out[k].z, s), hmul2(out[k].w, s));
                }
                // eight rows further, or the other 64 dimensions
                uint8_t* to = at + (Sh::kC == 8 ? (u >> 1) * 1024 + (u & 1) * Sh::kGroup : u * 1024);
#pragma unroll
                for (int k = 0; k < Sh::kOut; ++k) *reinterpret_cast<uint4*>(to + (put_chunk ^ (k << 4))) = out[k];
            }
            us::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                us::mbar_arrive(is_v ? &H.v_full[i % kVS] : &H.k_full[i % kKS]);
                if (!is_v) us::mbar_arrive(&H.s_full[ss]);
            }
        };
        Codes fa, fb;
        Where wa = locate(), wb = locate();
        fetch(wa, fa);
        fetch(wb, fb);
        Where wc = locate(), wd = locate();                // two behind them, page numbers on their way
        for (; wa.item < kItems * count; wa = wc, wb = wd, wc = locate(), wd = locate()) {
            convert_item(wa, fa);
            fetch(wc, fa);
            if (wb.item < kItems * count) convert_item(wb, fb);
            fetch(wd, fb);
        }
    }
    __syncthreads();
    const int parts = any ? H.parts : 0;

    // ---- shared segments (at most two a CTA): the last CTA to arrive joins them
    for (int i = 0; i < parts; ++i) {
        __syncthreads();
        const Part a = H.part[i];
        if (threadIdx.x == 0) {                            // one thread's fences order the whole CTA's accesses
            __threadfence();
            H.last = atomicAdd(p.ws_count + a.first, 1u) == (unsigned)(a.last - a.first);
            __threadfence();
        }
        __syncthreads();
        if (!H.last) continue;
        if (threadIdx.x == 0) p.ws_count[a.first] = 0;
        join_states<ELEM, D, NQ>(p, a);
    }
    us::tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps) us::tmem_dealloc(tmem, 512);
    us::pdl_launch_dependents();
}

template <int ELEM, int D, int NQ>
us_status launch(UsAttnParams p, cudaStream_t st) {
    using Sh = Shape<ELEM, D, NQ>;
    static_assert(Sh::kSmem <= 232448, "shared memory");
    p.ws_count = static_cast<unsigned*>(p.ws);
    p.ws_slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + 4096);
    auto kern = attn_tc_kernel<ELEM, D, NQ>;
    static bool ready[64] = {};                            // the attribute is set once a device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return US_ERR_CUDA;
    if (!ready[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess)
            return US_ERR_CUDA;
        ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)us::num_sms());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? US_OK : US_ERR_CUDA;
}

}  // namespace

namespace us {

bool attn_tc_serves(const UsAttnParams& p) { return (int64_t)p.a.max_n * p.G > 16; }

size_t attn_tc_ws(const UsAttnParams& p) {
    const size_t rows = (int64_t)p.a.max_n * p.G > kM ? 2 * kM : kM;
    return 4096 + (size_t)2 * num_sms() * (2 * rows + rows * p.c.D) * 4;
}

us_status launch_attn_tc(const UsAttnParams& p, cudaStream_t st) {
    const bool two = (int64_t)p.a.max_n * p.G > kM;
#define US_ATTN_PICK(E, D) (two ? launch<E, D, 2>(p, st) : launch<E, D, 1>(p, st))
    if (p.c.elem == US_I8) return p.c.D == 64 ? US_ATTN_PICK(US_I8, 64) : US_ATTN_PICK(US_I8, 128);
    return p.c.D == 64 ? US_ATTN_PICK(US_I4, 64) : US_ATTN_PICK(US_I4, 128);
#undef US_ATTN_PICK
}

}  // namespace us

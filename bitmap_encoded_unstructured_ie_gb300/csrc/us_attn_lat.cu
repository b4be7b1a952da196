// us_attn_lat.cu -- attention over the paged cache of latent rows, on the tensor cores
// (tcgen05).
//
// All heads of a token share one key row of W = Dc + 64 values, whose first Dc are the
// value row too: the n Hq query rows of a request are the rows of one product,
//   S = Q X^T     A = Q (shared memory), B = 64 positions' rows X, K-major
//   O += P X_c    A = P (shared memory, fp16), B = the same X in shared memory,
//                 its first Dc columns, MN-major
// so a position's row is read once and used twice, for 64 query rows.
//
// A segment is (request, block of 64 query rows); its positions come in tiles of 64,
// and the tiles of all segments are spread evenly over the CTAs (one an SM).  64 rows
// a block, not 128: O's 512 columns of 128 rows would take all of TMEM.  A product of
// 64 rows takes 16 lanes of each warp's 32 in TMEM; O's columns 256 .. 511 lie in the
// other 16 lanes, so O takes 256 columns and two tiles' scores 128 more.
//   warps 0-3: softmax of 16 rows each, the first segment's Q, the outputs
//   warps 4-7: find pages and copy the tiles' rows and further Q, 16 bytes a lane, to their places of
//           the 128-byte swizzle.  (By tensor copies, a box a page: 152 requests of 2000 positions
//           in pages of 16 took 83 us, 65 so; pages of 64 the same, trees 3 % less.)
//   warp 8: one thread issues the MMAs, whichever of the next tile's scores (its rows
//           have landed) and the last one's outputs (its weights are there) can go
// Weights are 2^(s - R); a row's reference R is its maximum less 11 when it is set, and
// moves when a score passes R + 15.9 (fp16 holds 2^15.9 and keeps all bits of weights
// down to 2^-25 of the largest).  R, sums and outputs of a segment shared by several CTAs
// are joined by a second kernel.
//
// What bounds it (clock stamps of the slowest SM, in us).  Long caches: bytes, a tile every
// 1.9 on each of 152 SMs, 5.9 TB/s, as both stages, 147 KB, are held while their products
// run.  48 requests of up to 8192 positions, 343 MB, take 79 (50.5 at a copy's rate): 59 are
// its 31 tiles, 3 pass until its share is found, 5 until first scores, 5 are the ends of two
// segments' parts, 4.5 the join.  Trees: 320 rows of each of 8 requests behind up to 4095
// positions take 44: 20 are 13 tiles (1.55 each, of which 2270 cycles are the tensor cores', as a
// product of 64 rows takes as long as one of 128), 7 the ends of two parts, 3 the first
// scores, 2 the share, 9 the join: 40 segments are shared out as 180 parts.  Short ones: a
// launch and its join, 11, and 6 a further segment on an SM (its scores, weights and product one
// after the other, outputs out of TMEM in 4000 cycles).
#include <atomic>

#include "us_attn_lat.cuh"
#include "us_internal.h"
#include "us_launch.cuh"
#include "us_tcgen05.cuh"

namespace {

using namespace us::attn;

constexpr int kM = 64, kTile = 64;                // query rows of a segment, positions of a tile
constexpr int kSoftWarps = 4, kLoadWarps = 4, kMmaWarp = kSoftWarps + kLoadWarps, kThreads = 32 * (kMmaWarp + 1);
constexpr int kBlock = 64 * 128;                  // bytes of 64 rows of 64 values
constexpr int kMaxStages = 4;

struct Header {
    uint64_t full[kMaxStages][3], free[kMaxStages][3], s_full[2], p_full, pv_done, q_full, q_free, over;
    uint64_t valid[kMaxStages];                   // which of the tile's positions exist
    uint32_t tmem;
};

template <int DC>
struct Shape {
    static constexpr int kW = DC + us::kLatDr, kC = kW / 64;        // blocks of 64 values of a row
    static constexpr int kOperand = kC * kBlock;                    // Q, or a tile's rows
    static constexpr int kStages = DC == 512 ? 2 : 4;
    static constexpr int kHalves = DC / 256;                        // products of 256 columns of O
    // A tile's parts land and are freed by themselves: those of each half's columns,
    // and the key's 64 values (part kHalves), which the scores alone read.
    static constexpr int kParts = kHalves + 1;
    static constexpr int kSmem = (1 + kStages) * kOperand + kBlock + (int)sizeof(Header) + 1024;
    static constexpr int kSlotFloats = us::attn::slot_floats(kM, DC);
    static_assert(kSmem <= 232448, "shared memory");
};

// This thread's copies so far arrive at `bar` when they have landed (one of the arrivals
// that it was set up for).
US_DEV void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(us::smem_addr(bar)) : "memory");
}

// 16 bytes of global memory, or of zeros, to shared memory
US_DEV void cp_async16_if(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// 16 lanes x 64 columns in fragment order: lane (g, c) gets rows g (v[4k], v[4k + 1])
// and g + 8 (v[4k + 2], v[4k + 3]) of columns 8k + 2c, 8k + 2c + 1
US_DEV void tmem_ld_frag64(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
    us::tmem_ld_frag32_end(r, v);
}
US_DEV void tmem_st32(uint32_t taddr, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
        "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]),
        "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]),
        "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31]),
        "r"(taddr)
        : "memory");
}

template <int DC>
__global__ void __launch_bounds__(kThreads, 1)
attn_lat_kernel(const UsAttnLatParams p) {
    using Sh = Shape<DC>;
    constexpr int kStages = Sh::kStages;
    using Cur = Cursor<kM, kTile>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((0u - us::smem_addr(smem_raw)) & 1023u);
    uint8_t* q_sm = smem;
    uint8_t* x_sm = q_sm + Sh::kOperand;
    uint8_t* p_sm = x_sm + kStages * Sh::kOperand;
    Header& H = *reinterpret_cast<Header*>(p_sm + kBlock);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i)
            for (int j = 0; j < Sh::kParts; ++j)               // (part 0: `valid`, too)
                us::mbar_init(&H.full[i][j], 32 * kLoadWarps + (j == 0)), us::mbar_init(&H.free[i][j], 1);
        for (int i = 0; i < 2; ++i) us::mbar_init(&H.s_full[i], 1);
        us::mbar_init(&H.p_full, kSoftWarps), us::mbar_init(&H.pv_done, 1), us::mbar_init(&H.q_full, 32 * kLoadWarps), us::mbar_init(&H.q_free, 1), us::mbar_init(&H.over, 1);
        us::fence_mbar_init();
    }
    if (warp == kMmaWarp) us::tmem_alloc(&H.tmem, 512);
    us::tc_fence_before();
    __syncthreads();
    us::tc_fence_after();
    us::pdl_wait();
    us::pdl_launch_dependents();                           // (the join's CTAs come now, and wait for this kernel's end)

    Work wk;
    Cur cur;
    const bool any = find_work<kM, kTile>(p, wk, cur);
    const uint32_t tmem = H.tmem;                          // O: 256 columns; scores: 2 x 64
    const int count = any ? (int)(wk.t1 - wk.t0) : 0, G = p.G;
    bool failed = false;
    auto wait = [&](uint64_t* bar, int use) {              // for the use-th completion of bar
        if (!failed && !spin(bar, (uint32_t)use & 1u, p.c.status)) failed = true;
    };

    // A segment's Q on its way to shared memory, by 128 threads: eight have 128 bytes of a row, rows
    // 16 k + t / 8.  The first segment's by the softmax warps, the others' by the copying ones.
    auto q_row = [&](const Cur& at, int r) {
        const int rr = at.rb * kM + r, i = (int)((unsigned)rr / (unsigned)G), h = rr - i * G;
        return rr < at.r.n * G ? p.Q + (int64_t)(at.r.row0 + i) * p.ldq + (int64_t)h * Sh::kW : nullptr;
    };
    auto request_q = [&](const Cur& at, int t) {
        const int r0 = t >> 3, chunk = t & 7;
        const uint32_t to = us::smem_addr(q_sm) + r0 * 128 + ((chunk ^ (r0 & 7)) << 4);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint16_t* src = q_row(at, 16 * k + r0);
            if (!src) break;
#pragma unroll
            for (int c = 0; c < Sh::kC; ++c) cp_async16(to + c * kBlock + k * 2048, src + 64 * c + 8 * chunk);
        }
        cp_async_arrive(&H.q_full);
    };

    if (warp < kSoftWarps) {
        // ----------------------------------------------------------- softmax
        const int g = lane >> 2, c2 = 2 * (lane & 3), wrow = 16 * warp;
        const uint32_t lanes = (uint32_t)warp * 32u << 16;
        const float scale = p.scale * 1.4426950408889634f;
        const uint64_t s2 = pair(scale, scale);
        if (threadIdx.x == 0) p.ws_parts[blockIdx.x].rows = 0;     // until a shared segment begins here
        // what the lane's rows see of the call's own positions: their masks, or in a chain how many
        auto seen_of = [&](const Cur& at, uint64_t (&seen)[2]) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const int rr = at.rb * kM + wrow + 8 * q + g, tok = (int)((unsigned)rr / (unsigned)G);
                seen[q] = rr >= at.r.n * G ? 0 : p.mask ? p.mask[at.r.row0 + tok] & (~0ull >> (64 - at.r.n)) : (uint64_t)(tok + 1);
            }
        };
        uint64_t own_seen[2] = {};
        if (count) {
            request_q(cur, threadIdx.x);
            seen_of(cur, own_seen);
        }
        for (int it = 0; it < count;) {
            // ---- a segment, or this CTA's part of it: tiles it .. end - 1
            const int end = min(count, it + cur.tiles - cur.tile), tile0 = cur.tile;
            const int rows = min(kM, cur.r.n * G - cur.rb * kM);
            // positions that a row sees among 64 from `base` behind the context
            auto seen64 = [&](int base, uint64_t row) {
                if (base <= -64) return ~0ull;
                const int lo = base < 0 ? -base : 0;       // context positions among them
                uint64_t own;
                if (p.mask) {
                    own = base < 64 ? row >> (base > 0 ? base : 0) : 0ull;
                } else {
                    const int k = (int)row - (base > 0 ? base : 0);
                    own = k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1ull;
                }
                return (own << lo) | (lo ? ~0ull >> (64 - lo) : 0ull);
            };
            float R[2] = {-INFINITY, -INFINITY};           // of the lane's rows wrow + 8 q + g
            uint64_t l2[2] = {};                           // their sums, two partial ones each
            for (int i = it; i < end; ++i) {
                const int st = i % kStages;
                wait(&H.full[st][0], i / kStages);         // (the scores came from it: for its positions)
                wait(&H.s_full[i & 1], i >> 1);
                us::tc_fence_after();
                const uint64_t ok = H.valid[st];
                const int base = (tile0 + i - it) * kTile - cur.r.ctx;
                if (wrow < rows) {
                    float v[32];
                    tmem_ld_frag64(tmem + lanes + 256 + 64 * (i & 1), v);
                    // s + 0 s: an infinite score becomes NaN, so that an entry which is not finite makes NaN of the
                    // rows that see it whichever sign it has there (a weight of 0 would lose it)
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const uint64_t x = mul2(pair(v[j], v[j + 1]), s2);
                        unpair(fma2(x, 0ull, x), v[j], v[j + 1]);
                    }
                    if (base + 64 > 0 || ok != ~0ull) {
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const uint64_t seen = (seen64(base, own_seen[q]) & ok) >> c2;
#pragma unroll
                            for (int k = 0; k < 8; ++k)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    if (!((seen >> (8 * k + e)) & 1ull)) v[4 * k + 2 * q + e] = -INFINITY;
                        }
                    }
                    uint64_t neg[2];
                    float f[2];
                    bool moved = false;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        float top = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 8; ++k) top = max3(top, v[4 * k + 2 * q], v[4 * k + 2 * q + 1]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        const float to = reference(R[q], top);
                        f[q] = to == R[q] ? 1.f : ex2(R[q] - to);
                        moved |= to != R[q];
                        R[q] = to;
                        l2[q] = mul2(l2[q], pair(f[q], f[q]));
                        const float ref = to == -INFINITY ? 0.f : to;
                        neg[q] = pair(-ref, -ref);
                    }
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float x, y;
                            unpair(add2(pair(v[4 * k + 2 * q], v[4 * k + 2 * q + 1]), neg[q]), x, y);
                            const uint64_t e = pair(ex2(x), ex2(y));
                            l2[q] = add2(l2[q], e);
                            unpair(e, x, y);
                            w[2 * k + q] = pack_half2(x, y);
                        }
                    if (i > it) {                          // the tile before: its weights are read, the outputs so far there
                        wait(&H.pv_done, i - 1);
                        us::tc_fence_after();
                        if (__any_sync(0xffffffffu, moved)) {
                            // lane: row lane & 15, of which row g = lane & 7 of the quads' first or second ones
                            const float f0 = __shfl_sync(0xffffffffu, f[0], 4 * (lane & 7)), f1 = __shfl_sync(0xffffffffu, f[1], 4 * (lane & 7));
                            const float fr = lane & 8 ? f1 : f0;
#pragma unroll 1
                            for (int c = 0; c < 256; c += 32) {
                                float y[32];
                                us::tmem_ld32(tmem + lanes + c, y);
#pragma unroll
                                for (int j = 0; j < 32; ++j) y[j] *= fr;
                                tmem_st32(tmem + lanes + c, y);
                            }
                            us::tmem_wait_st();
                        }
                    }
                    uint8_t* to = p_sm + (wrow + g) * 128 + 2 * c2;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        *reinterpret_cast<uint32_t*>(to + ((k ^ g) << 4)) = w[2 * k];
                        *reinterpret_cast<uint32_t*>(to + 1024 + ((k ^ g) << 4)) = w[2 * k + 1];
                    }
                }
                // (a warp without rows must not arrive for this tile while the last one's phase is open)
                if (wrow >= rows && i > it) wait(&H.pv_done, i - 1);
                // What some rows do not see is made finite (drafts, or in a chain what is behind the
                // segment's first token); what is not there was copied as zeros.
                const int behind = cur.r.n - base, all_see = max(0, (p.mask ? 0 : cur.rb * kM / G + 1) - base);
                if (all_see < min(kTile, behind)) {
                    // eight threads have 128 bytes of a row, each row's blocks at once
                    uint8_t* x = x_sm + st * Sh::kOperand + (threadIdx.x & 7) * 16;
#pragma unroll 1
                    for (int r = all_see + (threadIdx.x >> 3); r < min(kTile, behind); r += 16) {
                        uint4 y[DC / 64];
#pragma unroll
                        for (int c = 0; c < DC / 64; ++c) y[c] = *reinterpret_cast<const uint4*>(x + c * kBlock + r * 128);
#pragma unroll
                        for (int c = 0; c < DC / 64; ++c)
                            if (!all_finite(y[c])) *reinterpret_cast<uint4*>(x + c * kBlock + r * 128) = finite(y[c]);
                    }
                }
                us::fence_proxy_async_smem();
                us::tc_fence_before();
                __syncwarp();
                if (lane == 0) us::mbar_arrive(&H.p_full);
            }
            // ---- the segment's end: what is to be known for it while the last product runs
            const bool whole = tile0 == 0 && end - it == cur.tiles;
            Part part = {};
            if (!whole) part = wk.sharers(wk.t0 + it - tile0, wk.t0 + it - tile0 + cur.tiles, cur, rows);
            float l[2];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float a, b;
                unpair(l2[q], a, b);
                a += b;
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                l[q] = a + __shfl_xor_sync(0xffffffffu, a, 2);
            }
            const int src = 4 * (lane & 7), row = wrow + (lane & 15);
            const float l0 = __shfl_sync(0xffffffffu, l[0], src), l1 = __shfl_sync(0xffffffffu, l[1], src);
            const float ref0 = __shfl_sync(0xffffffffu, R[0], src), ref1 = __shfl_sync(0xffffffffu, R[1], src);
            const float sum = lane & 8 ? l1 : l0, ref = lane & 8 ? ref1 : ref0, inv = sum == 0.f ? 0.f : 1.f / sum;
            const int chunk = lane & 7, half = chunk >> 2;
            uint16_t* to[4];                               // of the rows that the lane writes
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = wrow + 4 * k + (lane >> 3);
                to[k] = whole && r < rows && half < Sh::kHalves ? out_row<kM>(p, cur.r.row0, 0, cur.rb, r, DC) + 256 * half + 8 * (chunk & 3) : nullptr;
            }
            float* slot = p.ws_slots + part.slot(blockIdx.x) * Sh::kSlotFloats;
            if (!whole && wrow < rows && lane < 16) {
                __stcg(slot + row, ref);
                __stcg(slot + kM + row, sum);
            }
            if (!whole && part.first == (int)blockIdx.x && threadIdx.x == 0) p.ws_parts[blockIdx.x] = part;
            if (end < count) {
                cur.next_segment(p);
                seen_of(cur, own_seen);
            }
            wait(&H.pv_done, end - 1);
            us::tc_fence_after();
            if (wrow < rows) {
                const bool mine = row < rows && (Sh::kHalves == 2 || lane < 16);
                const int col0 = lane & 16 ? 256 : 0;
                auto load_outputs = [&](int c, float (&a)[4][32]) {        // (one wait for 128 columns)
                    uint32_t r[4][32];
#pragma unroll
                    for (int u = 0; u < 4; ++u) tmem_ld32_begin(tmem + lanes + c + 32 * u, r[u]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) us::tmem_ld_frag32_end(r[u], a[u]);
                };
                if (whole) {
                    // Through the weights' place (the warp's 16 rows of 128 bytes, which no product
                    // reads any more), so that 64 bytes of a row are written at once: 32 columns of
                    // each half, which the row's two lanes hold.
                    const int at = lane & 15;
                    uint8_t* st = p_sm + wrow * 128;
#pragma unroll 1
                    for (int c0 = 0; c0 < 256; c0 += 128) {
                        float a[4][32];
                        load_outputs(c0, a);
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            const float (&v)[32] = a[u];
#pragma unroll
                            for (int j = 0; j < 32; j += 8)
                                *reinterpret_cast<uint4*>(st + at * 128 + ((((lane >> 4) * 4 + j / 8) ^ (at & 7)) << 4)) =
                                    make_uint4(pack_out(v[j] * inv, v[j + 1] * inv), pack_out(v[j + 2] * inv, v[j + 3] * inv),
                                               pack_out(v[j + 4] * inv, v[j + 5] * inv), pack_out(v[j + 6] * inv, v[j + 7] * inv));
                            __syncwarp();
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int r = 4 * k + (lane >> 3);
                                const uint4 y = *reinterpret_cast<const uint4*>(st + r * 128 + ((chunk ^ (r & 7)) << 4));
                                if (to[k]) *reinterpret_cast<uint4*>(to[k] + c0 + 32 * u) = y;
                            }
                            __syncwarp();
                        }
                    }
                } else {
#pragma unroll 1
                    for (int c0 = 0; c0 < 256; c0 += 128) {
                        float a[4][32];
                        load_outputs(c0, a);
                        if (mine) {
#pragma unroll
                            for (int j = 0; j < 128; j += 4)
                                __stcg(reinterpret_cast<float4*>(slot + 2 * kM) + (col0 + c0 + j) / 4 * kM + row,
                                       make_float4(a[j / 32][j % 32], a[j / 32][j % 32 + 1], a[j / 32][j % 32 + 2], a[j / 32][j % 32 + 3]));
                        }
                        __syncwarp();
                    }
                }
            }
            it = end;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < kMmaWarp) {
        // ------------------------------------------------------------- copies
        // Eight lanes have 128 bytes of a row; the warp's rows are 16 k + 4 w + lane / 8, k < 4.
        const int w = warp - kSoftWarps, row0 = 4 * w + (lane >> 3), chunk = lane & 7;
        const uint32_t to0 = us::smem_addr(x_sm) + row0 * 128 + ((chunk ^ (row0 & 7)) << 4);
        // The page of each piece of page_size positions (64 at most), a lane each: of the 32 from piece
        // `first` of a segment's part on
        const int piece = min(kTile, 1 << p.c.page_shift), pieces = kTile / piece, shift = __ffs(piece) - 1;
        auto page_of = [&](const Cur& c, int first) {
            const int pos = c.tile * kTile + ((first + lane) << shift);
            return pos < c.r.ctx + c.r.n ? p.c.table[(int64_t)c.b * p.c.max_pages + (pos >> p.c.page_shift)] : -1;
        };
        int ids = count ? page_of(cur, 0) : -1, segment = 0;
        for (int it = 0; it < count;) {
            const int end = min(count, it + cur.tiles - cur.tile), last = cur.r.ctx + cur.r.n;
            Cur next = cur;
            int ahead = page_of(cur, 32), after = -1, at = 0;              // the pages behind these, on their way
            for (int i = it; i < end; ++i, at += pieces) {
                if (at && (at & 31) == 0) ids = ahead, ahead = page_of(cur, at + 32);
                const int st = i % kStages, pos0 = (cur.tile + i - it) * kTile;
                uint64_t ok = 0;
                const uint16_t* src[4];                    // of the lane's rows
                bool has[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int id = __shfl_sync(0xffffffffu, ids, (at + ((16 * k) >> shift)) & 31), pos = pos0 + 16 * k + row0;
                    const int here = min(16, last - pos0 - 16 * k);        // of the sixteen rows
                    const bool good = id >= 0 && id < p.c.num_pages;
                    if (here > 0 && !good) us::set_status(p.c.status, US_ERR_CORRUPT);
                    if (here > 0 && good) ok |= ((1ull << here) - 1ull) << (16 * k);
                    has[k] = (ok >> (16 * k + row0)) & 1ull;
                    // (a row that is not there is copied as zeros: its weight is 0, which times anything stale might be NaN)
                    src[k] = p.rows + (has[k] ? (((int64_t)id << p.c.page_shift) + (pos & ((1 << p.c.page_shift) - 1))) * Sh::kW : 0) + 8 * chunk;
                }
                const uint32_t to = to0 + st * Sh::kOperand;
#pragma unroll
                for (int j = 0; j < Sh::kParts; ++j) {
                    const int part = j ? j - 1 : Sh::kHalves;              // the key's part first
                    if (i >= kStages) wait(&H.free[st][part], i / kStages - 1);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int c = 0; c < (j ? 4 : 1); ++c)
                            cp_async16_if(to + (4 * part + c) * kBlock + k * 2048, src[k] + (4 * part + c) * 64, has[k]);
                    cp_async_arrive(&H.full[st][part]);
                    if (j == 1 && w == 0 && lane == 0) {   // (part 0 was freed by those who read it)
                        H.valid[st] = ok;
                        us::mbar_arrive(&H.full[st][0]);
                    }
                }
                if (i > it) continue;
                if (segment) {                             // Q when the last segment's scores are made
                    wait(&H.q_free, segment - 1);
                    request_q(cur, threadIdx.x - 32 * kSoftWarps);
                }
                ++segment;
                if (end < count) {                         // the next segment's first pages, and its Q to L2
                    next.next_segment(p);
                    after = page_of(next, 0);
                    if (const uint16_t* q = q_row(next, 16 * w + (lane >> 1)))
#pragma unroll
                        for (int c = lane & 1; c < Sh::kC; c += 2) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + 64 * c));
                }
            }
            it = end;
            cur = next, ids = after;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
        // --------------------------------------------------------------- MMA
        if (us::elect_one()) {
            int segment = 0;
            for (int it = 0; it < count && !failed; ++segment) {
                const int end = min(count, it + cur.tiles - cur.tile);
                wait(&H.q_full, segment);
                us::fence_proxy_async_smem();              // (written by plain copies, as the tiles' rows)
                const uint64_t qd = us::umma_smem_desc_sw128(q_sm), pd = us::umma_smem_desc_sw128(p_sm);
                int s = it, sp = 0, o = it;                // the next tile's scores (from part sp on), the next one's outputs
                uint64_t since = 0;
                unsigned idle = 0;
                while (o < end && !failed) {
                    const int st = s % kStages, part = sp ? sp - 1 : Sh::kHalves;
                    if (s < end && s - o < 2 && us::mbar_test(&H.full[st][part], (uint32_t)(s / kStages) & 1u)) {
                        constexpr uint32_t id = us::umma_idesc_f16(kM, kTile);
                        us::fence_proxy_async_smem();      // (the rows were written by plain copies)
                        us::tc_fence_after();
                        const uint64_t from = (uint64_t)(4 * part * kBlock >> 4);
                        const uint64_t q = qd + from, xd = us::umma_smem_desc_sw128(x_sm + st * Sh::kOperand) + from;
                        const uint32_t to = tmem + 256 + 64 * (s & 1);
                        auto block = [&](int k, bool first) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint64_t at = (uint64_t)((k * kBlock + kk * 32) >> 4);
                                us::umma_f16(to, q + at, xd + at, id, !first || kk > 0);
                            }
                        };
                        if (sp == 0) {
                            block(0, true);
                            us::umma_commit(&H.free[st][Sh::kHalves]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) block(k, false);
                        }
                        if (++sp == Sh::kParts) {
                            us::umma_commit(&H.s_full[s & 1]);
                            if (++s == end && end < count) us::umma_commit(&H.q_free);
                            sp = 0;
                        }
                        idle = 0;
                    } else if (o < s && us::mbar_test(&H.p_full, (uint32_t)o & 1u)) {
                        constexpr uint32_t id = us::umma_idesc_f16(kM, 256) | us::kUmmaBMajorMN;
                        us::tc_fence_after();
                        const int os = o % kStages;
#pragma unroll
                        for (int h = 0; h < Sh::kHalves; ++h) {
                            const uint64_t xd = us::umma_smem_desc_mn_sw128(x_sm + os * Sh::kOperand + 4 * h * kBlock, kBlock);
#pragma unroll
                            for (int kk = 0; kk < kTile / 16; ++kk)
                                us::umma_f16(tmem + ((uint32_t)(16 * h) << 16), pd + (uint64_t)(kk * 32 >> 4),
                                             xd + (uint64_t)(kk * 2048 >> 4), id, o > it || kk > 0);
                            us::umma_commit(&H.free[os][h]);
                        }
                        us::umma_commit(&H.pv_done);
                        ++o, idle = 0;
                    } else if ((++idle & 1023u) == 0) {    // bounded, as every wait
                        const uint64_t now = us::globaltimer_ns();
                        if (idle == 1024u) since = now;
                        else if (now - since > us::kWaitLimitNs) us::set_status(p.c.status, US_ERR_TIMEOUT), failed = true;
                    }
                }
                it = end;
                if (it < count) cur.next_segment(p);
            }
            // Arrivals that no other warp waits for: they land while the CTA still has its shared memory
            if (count) {
                for (int i = max(0, count - kStages); i < count; ++i)
                    for (int j = 0; j < Sh::kParts; ++j) wait(&H.free[i % kStages][j], i / kStages);
                wait(&H.pv_done, count - 1);
            }
            if (failed) {                                  // (after a wait that ran out: its products, before TMEM is given back)
                us::umma_commit(&H.over);
                spin(&H.over, 0, p.c.status);
            }
        }
        __syncwarp();
    }
    us::tc_fence_before();
    __syncthreads();
    us::tc_fence_after();
    if (warp == kMmaWarp) us::tmem_dealloc(tmem, 512);
}

template <int DC>
us_status launch(UsAttnLatParams p, cudaStream_t st) {
    using Sh = Shape<DC>;
    p.ws_parts = static_cast<Part*>(p.ws);
    p.ws_slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kPartBytes);
    auto kern = attn_lat_kernel<DC>;
    static std::atomic<bool> ready[64];                // the attribute is set once a device, by whichever thread
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return US_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess)
            return US_ERR_CUDA;
        ready[dev].store(true, std::memory_order_release);
    }
    us_status s = us::launch_pdl(kern, dim3((unsigned)us::attn::attn_ctas()), kThreads, Sh::kSmem, st, p);
    if (s != US_OK) return s;
    return us::attn::launch_join<kM, DC>(p, us::attn::attn_ctas(), st);
}

}  // namespace

namespace us {

size_t attn_lat_ws(const UsAttnLatParams& p) {
    return us::attn::join_ws(attn::attn_ctas(), kM, p.Dc);
}

us_status launch_attn_lat(const UsAttnLatParams& p, cudaStream_t st) { return p.Dc == 512 ? launch<512>(p, st) : launch<256>(p, st); }

}  // namespace us

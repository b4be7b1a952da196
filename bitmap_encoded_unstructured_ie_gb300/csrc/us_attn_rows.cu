// us_attn_rows.cu -- causal attention over expanded rows (a prompt's tokens, their keys
// and values made from latent rows for each head), on the tensor cores (tcgen05).
//
//   S = Q K^T     A = Q (shared memory), B = 128 positions' keys: Dn of the head's own
//                 and 64 that all heads share
//   O += P V      A = P (TMEM, fp16, where S was), B = the positions' values, MN-major
//
// A segment is (request, head, block of 256 query rows); its positions come in tiles of
// 128, and the tiles of all segments are spread evenly over the CTAs (one an SM).  Two
// streams of 128 rows, each with its own scores, outputs and softmax warps: the tensor
// cores work on one while the other's weights are made.  A stream takes the tiles that
// its last row sees.
//   warps 0-7, 8-15: softmax of stream 0 / 1, two threads a row, 64 positions each
//   warps 16, 17: one thread issues the MMAs of stream 0 / 1
//   warp 18: one thread issues the copies (TMA, 128-byte swizzle): Q, then tile after
//           tile, its keys and its values as an item each, in blocks of 128 rows of 64
//           values, into a ring of such blocks
// Weights are 2^(s - R); a row's reference R is its maximum less 11 when it is set, and
// moves when a score passes R + 15.9 (fp16 holds 2^15.9 and keeps all bits of weights
// down to 2^-25 of the largest).  R, sums and outputs of a segment shared by several
// CTAs are joined by a second kernel.
//
// What bounds it: the way round.  Of 3800 cycles for a tile of both streams the tensor
// cores work 2620 (12 steps of 65 cycles a stream for the scores, 8 of 66 for the outputs).
// A tile's keys find their place in the ring when stream 1 is through with the values
// before the last (Q and ring are 224 KB), take 2500 cycles to land (80 KB a tile and SM
// come at 20 of about 33 bytes a cycle), and then stream 0's scores and stream 1's outputs
// follow, which free the next values.  A stream's softmax, 1850 cycles, hides behind that
// (with one thread a row it took 2500, and all 2 to 4 % longer).  512 tokens behind 8192, 32
// heads: 82 us (46.7 at the rate of a large product; 3 % more where a copy brings 128 bytes
// to L2, not 256), of which, by clock stamps, 60 are the slowest SM's 29 tiles, 5 pass until
// first scores, 5 are segments' ends, 2.6 its share, 6 the join.  Three prompts of up to 1777,
// 32 heads: 94 us (30.9): half of a diagonal tile is masked, and an even share of tiles, 24 or
// 25, has 2 to 7 segments in it: the slowest SM's 25 tiles are 58, the ends of six segments 15,
// their first scores 9, its share 3.5; the quickest is through after three quarters of that.
// 64-wide heads: 71 and 78 us.
#include <atomic>

#include "us_attn_lat.cuh"
#include "us_internal.h"
#include "us_launch.cuh"
#include "us_tcgen05.cuh"

namespace {

using namespace us::attn;

constexpr int kM = 128, kRows = 256, kTile = 128; // query rows of a stream, of a segment; positions of a tile
constexpr int kSoftWarps = 16, kMmaWarp = 16, kLoadWarp = 18, kThreads = 608;
constexpr int kBlock = 128 * 128;                 // bytes of 128 rows of 64 values
constexpr int kItems = 4;                         // keys, and values, of tiles that have a barrier each

struct Header {
    uint64_t k_full[kItems], v_full[kItems], k_free[kItems], v_free[kItems];
    uint64_t q_full[2], q_free[2], s_full[2], p_full[2][2], pv_done[2], turn[2], over[2];      // by stream (weights: and half of the positions)
    float row[2][2][kM];                          // by stream and half of the positions: of its rows
    uint32_t tmem, cleared;                       // cleared: some value was not finite, and made 0 in the ring
    int4 part[kSoftWarps];                        // of the warp's segment that ends (registers are short): see there
    int request[kSoftWarps];
};

template <int D>                                  // Dn = Dv
struct Shape {
    static constexpr int kK = D / 64 + 1, kV = D / 64, kT = kK + kV;       // blocks of a tile's keys, values, both
    static constexpr int kSlots = D == 128 ? 8 : 9;                        // blocks of the ring
    static_assert((kSlots + kT - 1) / kT + 1 <= kItems, "tiles that have blocks in the ring");
    static constexpr int kSmem = (2 * kK + kSlots) * kBlock + (int)sizeof(Header);
    static constexpr int kSlotFloats = slot_floats(kRows, D);
    static_assert(kSmem <= 232448, "shared memory");
};

struct Maps {
    CUtensorMap q, k, r, v;
};

US_DEV void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(us::smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(us::smem_addr(bar))
        : "memory");
}

// Of two lanes `apart`, the lower one's b and the upper one's a change places.
US_DEV void swap_quads(uint4& a, uint4& b, int apart) {
    const bool up = threadIdx.x & apart;
    auto move = [&](uint32_t& x, uint32_t& y) {
        const uint32_t z = __shfl_xor_sync(0xffffffffu, up ? x : y, apart);
        if (up) x = z;
        else y = z;
    };
    move(a.x, b.x), move(a.y, b.y), move(a.z, b.z), move(a.w, b.w);
}
US_DEV void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(v[0]),
        "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
        : "memory");
}
// Tiles of the segment that stream st's rows see (none: it has no rows).
US_DEV int stream_tiles(const Request& r, int rb, int st) {
    const int first = rb * kRows + st * kM, end = min(r.n, first + kM);
    return first >= r.n ? 0 : (r.ctx + end + kTile - 1) / kTile;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_rows_kernel(const UsAttnRowsParams p, const __grid_constant__ Maps maps) {
    using Sh = Shape<D>;
    constexpr int kK = Sh::kK, kV = Sh::kV, kT = Sh::kT, kSlots = Sh::kSlots;
    using Cur = Cursor<kRows, kTile>;
    extern __shared__ __align__(1024) uint8_t smem[];      // (there is no room to align it by hand)
    if (us::smem_addr(smem) & 1023u) {
        if (threadIdx.x == 0) us::set_status(p.c.status, US_ERR_CUDA);
        return;
    }
    uint8_t* q_sm = smem;
    uint8_t* ring = q_sm + 2 * kK * kBlock;
    Header& H = *reinterpret_cast<Header*>(ring + kSlots * kBlock);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i)
            us::mbar_init(&H.k_full[i], 1), us::mbar_init(&H.v_full[i], 1), us::mbar_init(&H.k_free[i], 2), us::mbar_init(&H.v_free[i], 2);
        for (int i = 0; i < 2; ++i) {
            us::mbar_init(&H.q_full[i], 1), us::mbar_init(&H.q_free[i], 1), us::mbar_init(&H.s_full[i], 1);
            // (the first half's weights and all of the outputs' columns, the second half's weights)
            us::mbar_init(&H.p_full[i][0], 8), us::mbar_init(&H.p_full[i][1], 4), us::mbar_init(&H.pv_done[i], 1), us::mbar_init(&H.turn[i], 1), us::mbar_init(&H.over[i], 1);
        }
        us::fence_mbar_init();
        H.cleared = 0;
    }
    if (warp == kLoadWarp && lane < 4)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.q + lane)) : "memory");
    if (warp == kMmaWarp) us::tmem_alloc(&H.tmem, 512);
    us::tc_fence_before();
    __syncthreads();
    us::tc_fence_after();
    us::pdl_wait();
    us::pdl_launch_dependents();                           // (the join's CTAs come now, and wait for this kernel's end)

    Work wk;
    Cur cur;
    const bool any = find_work<kRows, kTile>(p, wk, cur);
    const uint32_t tmem = H.tmem;                          // S0, S1, O0, O1: 128 columns each
    const int count = any ? (int)(wk.t1 - wk.t0) : 0;
    bool failed = false;
    auto wait = [&](uint64_t* bar, int use) {              // for the use-th completion of bar
        if (!failed && !spin(bar, (uint32_t)use & 1u, p.c.status)) failed = true;
    };

    if (warp < kSoftWarps) {
        // ----------------------------------------------------------- softmax
        const int st = warp >> 3, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane;      // of the stream
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t s_tm = tmem + lanes + st * 128 + half * 64;
        const uint32_t o_tm = tmem + lanes + 256 + st * 128 + half * (D / 2);      // the thread's columns of its row
        // (a scale of 0 would make NaN of masked scores; this one makes 1 of every weight, too)
        const float scale = p.scale == 0.f ? 1e-37f : p.scale * 1.4426950408889634f;
        const float none = scale < 0.f ? INFINITY : -INFINITY;         // an unseen score: -inf when scaled
        const uint64_t s2 = pair(scale, scale);
        if (threadIdx.x == 0) p.ws_parts[blockIdx.x].rows = 0;     // until a shared segment begins here
        // What the row's other thread has; both warps of the rows take part.  (The next tile's
        // scores, and so its maxima, come after both have arrived with their weights.)
        auto exchange = [&](float x) {
            H.row[st][half][row] = x;
            us::named_bar_sync(1 + 4 * st + (warp & 3), 64);
            return H.row[st][half ^ 1][row];
        };
        int used = 0, segment = 0;                         // tiles and segments of this stream so far
        for (int it = 0; it < count;) {
            // ---- a segment, or this CTA's part of it: tiles it .. end - 1, of which the stream's `mine`
            const int end = min(count, it + cur.tiles - cur.tile), tile0 = cur.tile;
            const int rows = min(kRows, cur.r.n - cur.rb * kRows), tok = min(cur.r.n - 1, cur.rb * kRows + st * kM + row);
            const int mine = min(end - it, max(0, stream_tiles(cur.r, cur.rb, st) - tile0));
            float R = -INFINITY;
            uint64_t l2 = 0;
            for (int j = 0; j < mine; ++j, ++used) {
                const int pos0 = (tile0 + j) * kTile;
                wait(&H.s_full[st], used);
                us::tc_fence_after();
                // The thread's 64 scores of its row are read twice, 32 at a time.
                const int seen = cur.r.ctx + tok + 1 - pos0 - 64 * half;       // positions that the row sees
                const bool edge = __any_sync(0xffffffffu, seen < 64);
                uint32_t r0[32], r1[32];
                auto finish = [&](int c, uint32_t (&r)[32], float (&v)[32]) {
                    us::tmem_ld_frag32_end(r, v);
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (c + k >= seen) v[k] = none;
                    }
                };
                float top = -INFINITY;
                auto largest = [&](const float (&v)[32]) {
                    float t[2] = {top, -INFINITY};
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float x, y;
                        unpair(mul2(pair(v[2 * k], v[2 * k + 1]), s2), x, y);
                        t[k & 1] = max3(t[k & 1], x, y);
                    }
                    top = fmaxf(t[0], t[1]);
                };
                {
                    float v[32];
                    tmem_ld32_begin(s_tm, r0);
                    finish(0, r0, v);
                    tmem_ld32_begin(s_tm + 32, r1);
                    largest(v);
                    finish(32, r1, v);
                    tmem_ld32_begin(s_tm, r0);
                    largest(v);
                }
                top = fmaxf(top, exchange(top));
                const float to = reference(R, top);
                const float f = to == R ? 1.f : ex2(R - to);
                const bool moved = to != R;
                R = to;
                l2 = mul2(l2, pair(f, f));
                const float ref = to == -INFINITY ? 0.f : to;
                const uint64_t neg = pair(-ref, -ref);
                // Large scores are rounded before the reference, which is one of them, is taken off: unrounded,
                // the largest would lie up to half a step, which may be thousands, beside it.
                const bool coarse = __any_sync(0xffffffffu, fabsf(ref) >= kFine);
                if (j && __any_sync(0xffffffffu, moved)) { // the outputs so far first (their product is done: these scores came after)
#pragma unroll 1
                    for (int c = 0; c < D / 2; c += 16) {
                        float y[16];
                        uint32_t o[16];
                        us::tmem_ld16(o_tm + c, y);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(y[k] * f);
                        tmem_st16(o_tm + c, o);
                    }
                    us::tmem_wait_st();
                }
                // The product of the first 64 positions adds to all columns of the outputs, so it waits
                // for this half's columns too, not only for the other half's weights.
                if (half) {
                    us::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) us::mbar_arrive(&H.p_full[st][0]);
                }
                // Values where no position is count as 0, and of those that some rows do not see (positions
                // behind the segment's first one) what is not finite is cleared; the rows that see it get it
                // at the segment's end.  Stream 0 does that for both: its product with a tile goes first.
                // Tiles that it does not read are stream 1's.
                const int there = cur.r.ctx + cur.r.n - pos0, all_see = cur.r.ctx + cur.rb * kRows + 1 - pos0;
                if (min(there, all_see) < 64 * half + 64 && (st == 0 || stream_tiles(cur.r, cur.rb, 0) - tile0 <= j)) {
                    const int x = it + j;
                    wait(&H.v_full[x % kItems], x / kItems);
#pragma unroll 1
                    for (int c = 0; c < 2 * kV; ++c) {
                        uint4* b = reinterpret_cast<uint4*>(ring + (x * kT + kK + c / 2) % kSlots * kBlock) + 512 * half + 256 * (c & 1) + (threadIdx.x & 127);
                        uint4 y[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) y[i] = b[128 * i];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int at = 64 * half + 32 * (c & 1) + (threadIdx.x & 127) / 8 + 16 * i;           // the position
                            if (at >= there) b[128 * i] = make_uint4(0, 0, 0, 0);
                            else if (at >= all_see && !all_finite(y[i]))
                                b[128 * i] = finite(y[i]), *static_cast<volatile uint32_t*>(&H.cleared) = 1;
                        }
                    }
                    us::fence_proxy_async_smem();
                }
                uint64_t sums[2] = {};
                auto weigh = [&](int c, const float (&v)[32]) {
                    uint32_t w[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float x, y;
                        unpair(fma2(pair(v[2 * k], v[2 * k + 1]), s2, neg), x, y);
                        x = ex2(x), y = ex2(y);
                        sums[k & 1] = add2(sums[k & 1], pair(x, y));
                        w[k] = pack_half2(x, y);
                    }
                    tmem_st16(s_tm + c / 2, w);            // over scores that this thread has read
                };
                {
                    float v[32];
                    finish(0, r0, v);
                    if (!coarse) {
                        tmem_ld32_begin(s_tm + 32, r1);
                        weigh(0, v);
                        finish(32, r1, v);
                        weigh(32, v);
                    } else {
#pragma unroll 1
                        for (int c = 0; c < 64; c += 32) {
                            uint32_t w[16];
                            if (c) tmem_ld32_begin(s_tm + 32, r1), finish(32, r1, v);
#pragma unroll
                            for (int k = 0; k < 16; ++k) {
                                const float x = ex2(__fadd_rn(__fmul_rn(v[2 * k], scale), -ref)), y = ex2(__fadd_rn(__fmul_rn(v[2 * k + 1], scale), -ref));
                                sums[k & 1] = add2(sums[k & 1], pair(x, y));
                                w[k] = pack_half2(x, y);
                            }
                            tmem_st16(s_tm + c / 2, w);
                        }
                    }
                }
                us::tmem_wait_st();
                us::tc_fence_before();
                __syncwarp();
                if (lane == 0) us::mbar_arrive(&H.p_full[st][half]);
                l2 = add2(l2, add2(sums[0], sums[1]));
            }
            // ---- the segment's end: what is to be known for it while the last product runs
            const bool whole = tile0 == 0 && end - it == cur.tiles;
            Part part = {};
            if (!whole) part = wk.sharers(wk.t0 + it - tile0, wk.t0 + it - tile0 + cur.tiles, cur, rows);
            const int srow = st * kM + row, wrow = srow & ~31;         // of the segment
            float* slot = p.ws_slots + part.slot(blockIdx.x) * Sh::kSlotFloats;
            if (!whole && part.first == (int)blockIdx.x && threadIdx.x == 0) p.ws_parts[blockIdx.x] = part;
            // (the row that the lane's quad begins with, and the lane's piece of each of the quad's rows)
            uint16_t* out = p.O + (int64_t)(cur.r.row0 + cur.rb * kRows + (srow & ~3)) * p.ldo + (int64_t)cur.h * D + half * (D / 2) + 8 * (lane & 3);
            const int left = rows - (srow & ~3);
            if (lane == 0) {                               // where values may have been cleared: positions between z and w, seen as x says
                H.part[warp] = make_int4(cur.r.ctx + cur.rb * kRows + 1, cur.h, tile0 * kTile, min(cur.r.ctx + cur.r.n, (tile0 + end - it) * kTile));
                H.request[warp] = cur.b;
            }
            if (end < count) cur.next_segment(p);
            if (mine) wait(&H.pv_done[st], segment++);
            us::tc_fence_after();
            // (once set, for good: such inputs are rare; a vote, as the other stream may set it between two lanes' reads)
            if (mine && __any_sync(0xffffffffu, *static_cast<volatile uint32_t*>(&H.cleared) != 0)) {
                const int4 of = H.part[warp];
                const int v0 = max(of.x, of.z), v1 = min(of.x + srow, of.w);
                const uint16_t* v = p.k.V + (int64_t)(p.kv_off[H.request[warp]] + v0) * p.k.ldv + of.y * p.k.hsv + half * (D / 2);
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 16) {
                    float y[16];
                    uint32_t o[16];
                    us::tmem_ld16(o_tm + c, y);
                    // (a weight is positive: what is not finite is the sum)
#pragma unroll 1
                    for (int at = 0; at < v1 - v0; ++at)
#pragma unroll
                        for (int k = 0; k < 16; k += 8) {
                            const uint4 x = *reinterpret_cast<const uint4*>(v + at * p.k.ldv + c + k);
                            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float z = us::half_bits_to_float((uint16_t)(u[e >> 1] >> (16 * (e & 1))));
                                y[k + e] += z - z == 0.f ? 0.f : z;
                            }
                        }
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(y[k]);
                    tmem_st16(o_tm + c, o);
                }
                us::tmem_wait_st();
            }
            float a, b;
            unpair(l2, a, b);
            a += b;
            const float sum = a + exchange(a), inv = sum == 0.f ? 0.f : 1.f / sum;
            us::named_bar_sync(1 + 4 * st + (warp & 3), 64);           // (read, before a maximum of the next segment comes there)
            if (wrow < rows) {
                if (!whole && half == 0) {
                    __stcg(slot + srow, R);
                    __stcg(slot + kRows + srow, sum);
                }
#pragma unroll 1
                for (int c = 0; c < D / 2; c += 32) {
                    float y[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) y[k] = 0.f;
                    if (mine) us::tmem_ld32(o_tm + c, y);
                    if (whole) {
                        // four lanes exchange their 64 bytes each of four rows: 64 bytes of a row are written at once
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            v[k] = make_uint4(pack_out(y[8 * k] * inv, y[8 * k + 1] * inv), pack_out(y[8 * k + 2] * inv, y[8 * k + 3] * inv),
                                              pack_out(y[8 * k + 4] * inv, y[8 * k + 5] * inv), pack_out(y[8 * k + 6] * inv, y[8 * k + 7] * inv));
                        swap_quads(v[0], v[1], 1), swap_quads(v[2], v[3], 1);
                        swap_quads(v[0], v[2], 2), swap_quads(v[1], v[3], 2);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < left) *reinterpret_cast<uint4*>(out + k * p.ldo + c) = v[k];
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 4)
                            __stcg(reinterpret_cast<float4*>(slot + 2 * kRows) + (half * (D / 2) + c + k) / 4 * kRows + srow,
                                   make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]));
                    }
                    __syncwarp();
                }
            }
            it = end;
        }
    } else if (warp == kLoadWarp) {
        // ------------------------------------------------------------- copies
        if (us::elect_one()) {
            int segment[2] = {0, 0}, keys = 0, values = 0; // segments of each stream, and tiles, that copies have been begun for
            for (int it = 0; it < count && !failed;) {
                const int end = min(count, it + cur.tiles - cur.tile), k0 = p.kv_off[cur.b];
                auto queries = [&](int st) {
                    if (stream_tiles(cur.r, cur.rb, st) <= cur.tile) return;
                    if (segment[st]) wait(&H.q_free[st], segment[st] - 1);
                    if (failed) return;
                    ++segment[st];
                    us::mbar_arrive_expect_tx(&H.q_full[st], kK * kBlock);
                    for (int c = 0; c < kK; ++c)
                        tma_load_3d(q_sm + (st * kK + c) * kBlock, &maps.q, 64 * c, cur.h, cur.r.row0 + cur.rb * kRows + st * kM, &H.q_full[st]);
                };
                queries(0);                                // (all in the order in which the MMAs need it)
                for (int i = it; i < end && !failed; ++i) {
                    const int row = k0 + (cur.tile + i - it) * kTile, item = i % kItems;
                    // block c of the tile, when the one whose place it takes is free
                    auto place = [&](int c) {
                        const int x = i * kT + c, old = x - kSlots, t = old / kT;
                        if (old >= 0) wait(old - t * kT < kK ? &H.k_free[t % kItems] : &H.v_free[t % kItems], t / kItems);
                        return ring + x % kSlots * kBlock;
                    };
                    uint64_t* bar = &H.k_full[item];
#pragma unroll 1
                    for (int c = 0; c < kK; ++c) {
                        uint8_t* to = place(c);
                        if (failed) break;
                        if (c == 0) us::mbar_arrive_expect_tx(bar, kK * kBlock), keys = i + 1;
                        if (c < kK - 1) tma_load_3d(to, &maps.k, 64 * c, cur.h, row, bar);
                        else tma_load_3d(to, &maps.r, 0, 0, row, bar);
                    }
                    if (i == it && !failed) queries(1);
                    bar = &H.v_full[item];
#pragma unroll 1
                    for (int c = 0; c < kV; ++c) {
                        uint8_t* to = place(kK + c);
                        if (failed) break;
                        if (c == 0) us::mbar_arrive_expect_tx(bar, kV * kBlock), values = i + 1;
                        tma_load_3d(to, &maps.v, 64 * c, cur.h, row, bar);
                    }
                }
                it = end;
                if (it < count) cur.next_segment(p);
            }
            // nothing of its own is left in flight when the CTA ends, after a wait that ran out neither
            auto landed = [&](uint64_t* bar, int use) { spin(bar, (uint32_t)use & 1u, p.c.status); };
            for (int i = max(0, keys - kItems); i < keys; ++i) landed(&H.k_full[i % kItems], i / kItems);
            for (int i = max(0, values - kItems); i < values; ++i) landed(&H.v_full[i % kItems], i / kItems);
            for (int st = 0; st < 2; ++st)
                if (segment[st]) landed(&H.q_full[st], segment[st] - 1);
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------- MMA
        // A thread for each stream, so that one's waits, commits and arithmetic (six cycles an instruction)
        // do not hold up the other, and they take turns (a tile's outputs and the next one's scores):
        // left to themselves, both streams come to want the tensor cores, then the exponentials, at once.
        if (us::elect_one()) {
            const int st = warp - kMmaWarp;
            int segment = 0, used = 0, it = 0, end = 0, mine = 0;          // segments and tiles of the stream so far
            // What the stream has to do with a tile (they are asked for one after the other): whether it
            // reads it, and whether that is the first or last one of its segment here.
            constexpr unsigned kUse = 1, kFirst = 2, kLast = 4;
            auto todo = [&](int x) -> unsigned {
                if (x >= count) return 0;
                if (x == end) {
                    if (x) cur.next_segment(p);
                    it = end, end = min(count, it + cur.tiles - cur.tile);
                    mine = min(end - it, max(0, stream_tiles(cur.r, cur.rb, st) - cur.tile));
                }
                return (x - it < mine ? kUse : 0) | (x == it ? kFirst : 0) | (x - it == mine - 1 ? kLast : 0);
            };
            auto qk = [&](int x, unsigned what) {
                constexpr uint32_t id = us::umma_idesc_f16(kM, kTile);
                if (what & kFirst) wait(&H.q_full[st], segment++);
                us::tc_fence_after();
                const uint64_t qd = us::umma_smem_desc_sw128(q_sm + st * kK * kBlock);
#pragma unroll
                for (int c = 0; c < kK; ++c) {
                    const uint64_t kd = us::umma_smem_desc_sw128(ring + (x * kT + c) % kSlots * kBlock);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        us::umma_f16(tmem + st * 128, qd + (uint64_t)((c * kBlock + kk * 32) >> 4), kd + (uint64_t)(kk * 32 >> 4), id,
                                     c > 0 || kk > 0);
                }
                us::mbar_arrive(&H.turn[st]);
                us::umma_commit(&H.s_full[st]);
                us::umma_commit(&H.k_free[x % kItems]);
                if (what & kLast) us::umma_commit(&H.q_free[st]);
            };
            auto pv = [&](int x, unsigned what) {
                const uint32_t o = tmem + 256 + st * 128, w = tmem + st * 128;
                const int v0 = (x * kT + kK) % kSlots;
                const uint64_t rd = us::umma_smem_desc_mn_sw128(ring, kBlock), vd = rd + (uint64_t)(v0 * (kBlock >> 4));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    wait(&H.p_full[st][half], used);
                    us::tc_fence_after();
                    if (kV == 1 || v0 + 1 == kSlots) {     // one block of columns, or two that the ring's end parts
#pragma unroll
                        for (int c = 0; c < kV; ++c)
#pragma unroll
                            for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                                us::umma_f16_ta(o + 64 * c, w + 8 * kk + 32 * half, (c ? rd : vd) + (uint64_t)(kk * 2048 >> 4),
                                                us::umma_idesc_f16(kM, 64) | us::kUmmaBMajorMN, !(what & kFirst) || kk > 0);
                    } else {
#pragma unroll
                        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                            us::umma_f16_ta(o, w + 8 * kk + 32 * half, vd + (uint64_t)(kk * 2048 >> 4), us::umma_idesc_f16(kM, 64 * kV) | us::kUmmaBMajorMN,
                                            !(what & kFirst) || kk > 0);
                    }
                }
                ++used;
                us::umma_commit(&H.v_free[x % kItems]);
                if (what & kLast) us::umma_commit(&H.pv_done[st]);         // (within a segment the next scores say it)
            };
            // The stream's outputs of a tile and its scores of the next, be that of the next segment (whose
            // scores are there, then, when the last one's outputs have been written).  A tile that the
            // stream does not read it gives back as it comes: every one is given back by both.
            unsigned now = 0, next = todo(0);
#pragma unroll 1
            for (int x = -1; x < count && !failed; ++x) {
                if (x >= 0) wait(&H.v_full[x % kItems], x / kItems);
                if (st || x >= 0) wait(&H.turn[st ^ 1], x + st);
                if (x >= 0) {
                    if (now & kUse) pv(x, now);
                    else us::mbar_arrive(&H.v_free[x % kItems]);
                }
                if (x + 1 < count) {
                    wait(&H.k_full[(x + 1) % kItems], (x + 1) / kItems);
                    if (next & kUse) qk(x + 1, next);
                    else us::mbar_arrive(&H.turn[st]), us::mbar_arrive(&H.k_free[(x + 1) % kItems]);
                } else {
                    us::mbar_arrive(&H.turn[st]);
                }
                now = next, next = todo(x + 2);
            }
            // Arrivals that no other warp waits for: they land while the CTA still has its shared memory
            for (int i = max(0, count - kItems); i < count; ++i) wait(&H.k_free[i % kItems], i / kItems), wait(&H.v_free[i % kItems], i / kItems);
            if (segment) wait(&H.pv_done[st], segment - 1), wait(&H.q_free[st], segment - 1);
            if (failed) {                                  // (after a wait that ran out: its products, before TMEM is given back)
                us::umma_commit(&H.over[st]);
                spin(&H.over[st], 0, p.c.status);
            }
        }
        __syncwarp();
    }
    us::tc_fence_before();
    __syncthreads();
    us::tc_fence_after();
    if (warp == kMmaWarp) us::tmem_dealloc(tmem, 512);
}

// (64 values, heads, rows) of rows `ld` and heads `hs` elements apart, 128 rows of a head a copy
bool encode_map(CUtensorMap* map, const uint16_t* x, int width, int heads, int64_t hs, int64_t rows, int64_t ld) {
    auto enc = us::tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t stride[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, 1, 128}, estr[3] = {1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<uint16_t*>(x), dim, stride, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
us_status launch(UsAttnRowsParams p, cudaStream_t st) {
    using Sh = Shape<D>;
    p.ws_parts = static_cast<Part*>(p.ws);
    p.ws_slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kPartBytes);
    Maps maps;
    const us_attn_kv_rows& k = p.k;
    if (!encode_map(&maps.q, p.Q, D + us::kLatDr, k.H, D + us::kLatDr, p.a.T, p.ldq) ||
        !encode_map(&maps.k, k.K, D, k.H, k.H > 1 ? k.hsk : D, k.S, k.ldk) ||
        !encode_map(&maps.r, k.KR, us::kLatDr, 1, us::kLatDr, k.S, k.ldkr) ||
        !encode_map(&maps.v, k.V, D, k.H, k.H > 1 ? k.hsv : D, k.S, k.ldv))
        return US_ERR_CUDA;
    auto kern = attn_rows_kernel<D>;
    static std::atomic<bool> ready[64];                // the attribute is set once a device, by whichever thread
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return US_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess)
            return US_ERR_CUDA;
        ready[dev].store(true, std::memory_order_release);
    }
    const us_status s = us::launch_pdl(kern, dim3((unsigned)attn_ctas()), kThreads, Sh::kSmem, st, p, maps);
    return s != US_OK ? s : launch_join<kRows, D>(p, attn_ctas(), st);
}

}  // namespace

namespace us {

size_t attn_rows_ws(const UsAttnRowsParams& p) { return attn::join_ws(attn::attn_ctas(), kRows, p.k.Dv); }

us_status launch_attn_rows(const UsAttnRowsParams& p, cudaStream_t st) { return p.k.Dv == 128 ? launch<128>(p, st) : launch<64>(p, st); }

}  // namespace us

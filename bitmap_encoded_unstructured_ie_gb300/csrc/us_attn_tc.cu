// us_attn_tc.cu -- attention of many query rows per key head over the quantised
// K/V cache (drafted trees, chunks of a prompt), on the tensor cores (tcgen05).
//
// Same function as us_attn.cu.  A segment is (request, key head, block of 128 NQ
// query rows); its positions come in tiles of 128, and the tiles of all segments
// are spread evenly over the CTAs (one an SM):
//   S = Q Ck^T    A = Q (shared memory), B = the tile's K codes as fp16
//   O += P Cv     A = P (TMEM, fp16), B = the tile's V codes as fp16, MN-major
// K enters as its codes, its scale on the scores in fp32.  V enters as code * 2^e,
// exactly; the rest of its scale 2^e m (1 <= m < 2) multiplies the weight in fp32, so
// that a weight's rounding to fp16 is the only one (V as fp16(code * scale) needs no
// multiplication there, but a second rounding of 2^-11: outputs 3.6e-4 of their
// norm off, 2.9e-4 so).  The dimensions stand in shared memory in the order in which
// the codes leave their words (within each eight), the same for Q, K and V; only the
// outputs are put back.
//
// Two streams, each with its own scores, outputs, row references and softmax
// warps, so that the tensor cores work on one while the other's weights are made.
// With more than 128 rows (NQ = 2) a stream is a half of the rows and takes every
// tile: each tile's codes are converted once for 256 rows.  Else (NQ = 1) the tiles
// alternate between the streams, which are joined at the segment's end.
//   warps 0-3, 4-7: softmax of stream 0 / 1, 32 rows each, 64 positions at a time
//               (the scores of the other 64 are made meanwhile), in the fragment
//               order of 16-lane TMEM loads: a lane has a quarter of the columns, so
//               it reads a quarter of the scales (every register that comes from
//               TMEM or shared memory takes a cycle of the load / store pipe a warp)
//   warp 8: one thread issues the MMAs: PV of a half tile, then QK of the next tile's
//               (it is held up at the rate of their execution, 64 cycles each)
//   warps 9-15: codes -> fp16, in items of 16 positions of K or of V; a warp's next
//               items are on their way to its own ring, each lane's to its own place
// 16 warps: 128 registers a thread, of which the softmax takes 160 and leaves 96 to
// the others (at 128 it spilled: chunk of 512 tokens 202 us, 195 so).  The roles' loops
// are kept short (one copy of each body): four warps of a scheduler run three
// different programs, and fetching them was a sixth of its time.
// Weights are 2^(s - R); a row's reference R is its maximum less 11 when it is set,
// and moves when eight weights of a lane sum to more than 2^14.9, which no fp16 weight
// times m < 2 may reach, or a masked tile has a larger maximum (at 2^11 and above,
// fp16 keeps all of its bits down to 2^-25 of a weight).  R, sums and outputs of a
// segment shared by several CTAs are joined by a second kernel.
//
// What bounds it.  A tile of 256 rows takes about 5200 cycles: the tensor pipe is busy
// for 33 % (48 MMAs of 64 cycles; a score MMA of 64 positions reads 6 KB of shared
// memory for its 32 cycles of work), issue slots for 56 %, the exponentials' unit for
// 35 %.  Softmax, MMAs and conversion wait for each other in turn; what would shorten
// the turn (more stages, scores of a whole tile) has no shared memory or TMEM left.
// 512 tokens of 64 query heads on 8, behind 8192 positions, int8: 178 us, 800 TFLOP/s;
// four trees of 64 tokens of 32 heads on 8, behind 4095, int4: 40 us, of which 13 are
// tiles, 5 pass until the first scores, 4 are a CTA's partial state, and the rest is
// the join and two launches.
#include <atomic>

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
constexpr float kTop = 11.f, kMost = 30573.f;     // log2 of a row's largest weight when R is set; 2^14.9

struct Header {
    uint64_t k_full[kKS], k_free[kKS], v_full[3], v_free[3], s_full[kSS];
    uint64_t qk_done[2][2], p_full[2][2], pv_done[2][2];       // by stream and half tile
    uint64_t q_full;
    // by pairs of positions of the tiles on their way: K's scales times scale log2(e), V's m
    float4 scales[kSS][kTile / 2];
    alignas(16) uint16_t valid[kSS][8];                       // which of 16 positions exist
    uint32_t tmem;
    Work work;
};

static_assert(offsetof(Header, scales) % 16 == 0 && offsetof(Header, valid) % 16 == 0, "read 8 and 16 bytes at a time");
struct Ends {                                     // of a stream's rows at a segment's end, where Q was
    float ref[kM], sum[kM];
};

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
    static constexpr int kRaw = 16 * kRow + 64;                     // codes and scales of an item
    static constexpr int kFit = (232448 - 1024 - 512 - (NQ + kKS + kVS) * kOperand - (int)sizeof(Header)) / (kConvWarps * kRaw);
    static constexpr int kRS = kFit > 4 ? 4 : kFit;                 // items of a warp's ring
    static_assert(kRS >= 2, "ring");
    static constexpr int kSmem = (NQ + kKS + kVS) * kOperand + (int)sizeof(Header) + kConvWarps * kRS * kRaw + 1024;
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
        make_uint4(pack_out(d[0], d[1]), pack_out(d[2], d[3]), pack_out(d[4], d[5]), pack_out(d[6], d[7]));
}

template <int ELEM, int D, int NQ>
__global__ void __launch_bounds__(kThreads, 1)
attn_tc_kernel(const UsAttnParams p) {
    using Sh = Shape<ELEM, D, NQ>;
    constexpr int kRows = Sh::kRows, kVS = Sh::kVS;
    using Cur = Cursor<kRows, kTile>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((0u - us::smem_addr(smem_raw)) & 1023u);     // (still known to be shared memory)
    uint8_t* q_sm = smem;
    uint8_t* k_sm = q_sm + NQ * Sh::kOperand;
    uint8_t* v_sm = k_sm + kKS * Sh::kOperand;
    uint8_t* raw_sm = v_sm + kVS * Sh::kOperand;
    Header& H = *reinterpret_cast<Header*>(raw_sm + kConvWarps * Sh::kRS * Sh::kRaw);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kKS; ++i) us::mbar_init(&H.k_full[i], 8), us::mbar_init(&H.k_free[i], 1);
        for (int i = 0; i < kVS; ++i) us::mbar_init(&H.v_full[i], 8), us::mbar_init(&H.v_free[i], 1);
        for (int i = 0; i < kSS; ++i) us::mbar_init(&H.s_full[i], 8);
        for (int i = 0; i < 2; ++i) {
            for (int a = 0; a < 2; ++a)
                us::mbar_init(&H.qk_done[i][a], 1), us::mbar_init(&H.p_full[i][a], 4), us::mbar_init(&H.pv_done[i][a], 1);
        }
        us::mbar_init(&H.q_full, kSoftWarps);
        us::fence_mbar_init();
    }
    if (warp == kSoftWarps) us::tmem_alloc(&H.tmem, 512);
    __syncthreads();
    us::pdl_wait();

    Work wk;
    Cur cur;
    const bool any = find_work<kRows, kTile>(p, wk, cur);
    if (threadIdx.x == 0) H.work = wk;                     // the softmax warps need it at a segment's end
    us::tc_fence_after();
    const uint32_t tmem = H.tmem;                          // S0, S1, O0, O1: 128 columns each
    const int count = any ? (int)(wk.t1 - wk.t0) : 0, G = p.G;
    bool failed = false;
    auto wait = [&](uint64_t* bar, int use) {              // for the use-th completion of bar
        if (!failed && !wait_bar(bar, (uint32_t)use & 1u, p.c.status)) failed = true;
    };

    // 256 threads of each: together the 128 registers a thread of the launch
    if (warp < kSoftWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    if (warp < kSoftWarps) {
        // ----------------------------------------------------------- softmax
        const int st = warp >> 2, g = lane >> 2, c2 = 2 * (lane & 3);
        const int wrow = (warp & 3) * 32 + (NQ == 2 ? kM * st : 0);           // the warp's first row of the segment
        const uint32_t lanes = (uint32_t)(warp & 3) * 32u << 16;
        const uint32_t s_tm = tmem + lanes + st * 128, o_tm = tmem + lanes + 256 + st * 128;
        if (threadIdx.x == 0) p.ws_parts[blockIdx.x].rows = 0;     // until a shared segment begins here
        for (int it = 0; it < count;) {
            // ---- a segment, or this CTA's part of it: tiles it .. end - 1
            const int end = min(count, it + cur.tiles - cur.tile), tile0 = cur.tile;
            const int rows = min(kRows, cur.r.n * G - cur.rb * kRows);
            // Q: a thread takes one 16-byte chunk of every kQR-th row, up to 16 loads at once
            constexpr int kQR = 32 * kSoftWarps / (D / 8), kAtOnce = kRows / kQR < 16 ? kRows / kQR : 16;
            const int q_row = threadIdx.x / (D / 8), q_chunk = threadIdx.x % (D / 8);
            // (row q_row + k kQR: token q_tok, query head q_head of the key head's)
            const int q_dtok = (int)((unsigned)kQR / (unsigned)G), q_dhead = kQR - q_dtok * G, q_first = cur.rb * kRows + q_row;
            int q_tok = (int)((unsigned)q_first / (unsigned)G), q_head = q_first - q_tok * G;
#pragma unroll 1
            for (int r0 = q_row; r0 < kRows; r0 += kAtOnce * kQR) {
                uint4 u[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    u[k] = make_uint4(0, 0, 0, 0);
                    if (r0 + k * kQR < rows)
                        u[k] = reinterpret_cast<const uint4*>(p.Q + (int64_t)(cur.r.row0 + q_tok) * p.ldq + (int64_t)(cur.h * G + q_head) * D)[q_chunk];
                    q_tok += q_dtok, q_head += q_dhead;
                    if (q_head >= G) q_head -= G, ++q_tok;
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int r = r0 + k * kQR;
                    *reinterpret_cast<uint4*>(operand_at(q_sm + (r / kM) * Sh::kOperand, r % kM, q_chunk)) = reorder<ELEM>(u[k]);
                }
            }
            us::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) us::mbar_arrive(&H.q_full);
            // what the lane's rows see of the call's own positions: their masks, or in a chain how many
            uint64_t own_seen[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int r = wrow + 8 * q + g, tok = (int)((unsigned)(cur.rb * kRows + r) / (unsigned)G);
                own_seen[q] = r >= rows ? 0 : p.mask ? p.mask[cur.r.row0 + tok] & (~0ull >> (64 - cur.r.n)) : (uint64_t)(tok + 1);
            }
            // positions that a row sees among 32 from `base` behind the context
            auto seen32 = [&](int base, uint64_t row) {
                if (base <= -32) return 0xFFFFFFFFu;
                const int lo = base < 0 ? -base : 0;       // context positions among them
                uint32_t own;
                if (p.mask) {
                    own = base < 64 ? (uint32_t)(row >> (base > 0 ? base : 0)) : 0u;
                } else {
                    const int k = (int)row - (base > 0 ? base : 0);
                    own = k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
                }
                return (own << lo) | (lo ? 0xFFFFFFFFu >> (32 - lo) : 0u);
            };
            // references and sums (two partial ones each) of the lane's rows wrow + 8 q + g
            float R[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            uint64_t l2[4] = {};
            constexpr int kStep = NQ == 2 ? 1 : 2;         // a stream's tiles: every one, or every other
            const int i0 = NQ == 2 ? it : it + ((it ^ st) & 1);
            for (int i = i0; i < end; i += kStep) {
                const int ss = i % kSS;
                wait(&H.s_full[ss], i / kSS);
#pragma unroll 1
                for (int a = 0; a < 2; ++a) {              // the tile's halves of 64 positions
                    const uint2 ok = *reinterpret_cast<const uint2*>(&H.valid[ss][4 * a]);
                    const int base = (tile0 + i - it) * kTile + 64 * a - cur.r.ctx;
                    const bool edge = base + 64 > 0 || (ok.x & ok.y) != 0xFFFFFFFFu;
                    wait(&H.qk_done[st][a], i / kStep);
                    us::tc_fence_after();
                    if (wrow < rows) {
                        const float4* sc2 = H.scales[ss] + 32 * a + (lane & 3);
                        // Scores mostly stay below R + 14.9: their weights are made at once, and
                        // again if a lane's sum of eight of them passes 2^14.9 (rows of equal
                        // scores reach 2^14), or where some are unseen.
                        uint32_t w[32];                    // the weights as fp16 pairs
                        uint64_t sum[4], neg[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) neg[q] = pair(-R[q], -R[q]);
                        // (a segment's first tile has no reference yet)
                        for (bool fit = edge || (i == i0 && a == 0);; fit = true) {
                            if (fit) {
                                // scaled and masked scores, back in their place, and what they move
                                float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                                for (int c = 0; c < 2; ++c) {
                                    float v[32];
                                    us::tmem_ld_frag32(s_tm + 64 * a + 32 * c, v);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const float4 sc = sc2[16 * c + 4 * k];
#pragma unroll
                                        for (int q = 0; q < 4; ++q) {
                                            const int at = 16 * (q >> 1) + 4 * k + 2 * (q & 1);
                                            v[at] *= sc.x, v[at + 1] *= sc.y;
                                        }
                                    }
                                    if (edge) {
#pragma unroll
                                        for (int q = 0; q < 4; ++q) {
                                            const uint32_t seen = (seen32(base + 32 * c, own_seen[q]) & (c ? ok.y : ok.x)) >> c2;
#pragma unroll
                                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                                for (int e = 0; e < 2; ++e)
                                                    if (!((seen >> (8 * k + e)) & 1u)) v[16 * (q >> 1) + 4 * k + 2 * (q & 1) + e] = -INFINITY;
                                        }
                                    }
#pragma unroll
                                    for (int q = 0; q < 4; ++q)
#pragma unroll
                                        for (int k = 0; k < 4; ++k) {
                                            const int at = 16 * (q >> 1) + 4 * k + 2 * (q & 1);
                                            top[q] = max3(top[q], v[at], v[at + 1]);
                                        }
                                    us::tmem_st_frag32(s_tm + 64 * a + 32 * c, v);
                                }
                                us::tmem_wait_st();
                                float f[4];
                                bool moved = false;
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    float x = top[q];
                                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                                    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                                    const float to = x > R[q] + kTop ? x - kTop : R[q];
                                    f[q] = to == R[q] ? 1.f : ex2(R[q] - to);
                                    moved |= to != R[q];
                                    R[q] = to;
                                    l2[q] = mul2(l2[q], pair(f[q], f[q]));
                                    const float ref = to == -INFINITY ? 0.f : to;
                                    neg[q] = pair(-ref, -ref);
                                }
                                if ((i != i0 || a) && __any_sync(0xffffffffu, moved)) {
                                    wait(&H.pv_done[st][a ^ 1], i / kStep + a - 1);    // the stream's outputs so far first
                                    us::tc_fence_after();
#pragma unroll 1
                                    for (int c = 0; c < D; c += 32) {
                                        float y[32];
                                        us::tmem_ld_frag32(o_tm + c, y);
#pragma unroll
                                        for (int j = 0; j < 32; ++j) y[j] *= f[2 * (j >> 4) + ((j >> 1) & 1)];
                                        us::tmem_st_frag32(o_tm + c, y);
                                    }
                                    us::tmem_wait_st();
                                }
                            }
#pragma unroll
                            for (int q = 0; q < 4; ++q) sum[q] = 0;
                            auto weigh = [&](const float (&v)[32], int c, int k) {     // 8 positions
                                const float4 sc = sc2[16 * c + 4 * k];
                                const uint64_t s = fit ? pair(1.f, 1.f) : pair(sc.x, sc.y), m = pair(sc.z, sc.w);
#pragma unroll
                                for (int q = 0; q < 4; ++q) {
                                    const int at = 16 * (q >> 1) + 4 * k + 2 * (q & 1);
                                    float x, y;
                                    unpair(fma2(pair(v[at], v[at + 1]), s, neg[q]), x, y);
                                    const uint64_t e = pair(ex2(x), ex2(y));
                                    sum[q] = add2(sum[q], e);
                                    unpair(mul2(e, m), x, y);
                                    w[16 * (q >> 1) + 8 * c + 2 * k + (q & 1)] = pack_half2(x, y);
                                }
                            };
                            // 32 positions at a time, the second ones loaded when half of the first are done
                            uint32_t r[32];
                            float v[32];
                            us::tmem_ld_frag32(s_tm + 64 * a, v);
                            weigh(v, 0, 0), weigh(v, 0, 1);
                            us::tmem_ld_frag32_begin(s_tm + 64 * a + 32, r);
                            weigh(v, 0, 2), weigh(v, 0, 3);
                            us::tmem_ld_frag32_end(r, v);
#pragma unroll
                            for (int k = 0; k < 4; ++k) weigh(v, 1, k);
                            if (fit) break;
                            bool far = false;
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                float x, y;
                                unpair(sum[q], x, y);
                                far |= !(fmaxf(x, y) <= kMost) || x != x || y != y;
                            }
                            if (!__any_sync(0xffffffffu, far)) break;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) l2[q] = add2(l2[q], sum[q]);
                        us::tmem_st_pairs32(s_tm + 64 * a, w);     // over scores that were read
                        us::tmem_st_pairs32(s_tm + 64 * a + (16u << 16), w + 16);
                        us::tmem_wait_st();
                    }
                    us::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) us::mbar_arrive(&H.p_full[st][a]);
                }
            }
            // ---- the segment's end: the streams' sums and outputs
            const int srow = (warp & 3) * 32;              // the warp's first row of its stream
            // the streams whose outputs the warp reads, and whether they had a tile
            bool has[2];
            // PV of the last tile of stream x (the tile before it is done: a parity tells
            // only neighbouring phases apart); nothing reads its Q any more
            auto finish = [&](int x, int tile) { wait(&H.pv_done[x][1], tile / kStep); };
            if constexpr (NQ == 2) {
                has[0] = true, has[1] = false;
                finish(st, end - 1);
            } else {
                has[0] = end - it >= 2 || !(it & 1), has[1] = end - it >= 2 || (it & 1);
                // the warp's own stream first: all but the last tile of the other come before it
                const int own = ((end - 1) & 1) == st ? end - 1 : end - 2, other = 2 * end - 3 - own;
                if (has[st]) finish(st, own);
                if (has[st ^ 1]) finish(st ^ 1, other);
            }
            // (NQ = 2: a stream's Q is its own; else both streams are done)
            auto ends = [&](int x) -> Ends& {
                return *reinterpret_cast<Ends*>(NQ == 2 ? q_sm + x * Sh::kOperand : q_sm + x * sizeof(Ends));
            };
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float a, b;
                unpair(l2[q], a, b);
                a += b;
                a += __shfl_xor_sync(0xffffffffu, a, 1);
                a += __shfl_xor_sync(0xffffffffu, a, 2);
                if (c2 == 0) ends(st).ref[srow + 8 * q + g] = R[q], ends(st).sum[srow + 8 * q + g] = a;
            }
            if constexpr (NQ == 2) __syncwarp();
            else us::named_bar_sync(1, 32 * kSoftWarps);
            us::tc_fence_after();
            const int64_t s0 = H.work.t0 + it - tile0;
            const Part part = H.work.sharers(s0, s0 + cur.tiles, cur, rows);
            const bool whole = part.first == part.last;
            if (wrow < rows) {
                const int row = wrow + lane, sr = srow + lane, s1 = NQ == 2 ? st : 0;
                const float r0 = ends(s1).ref[sr], r1 = NQ == 2 ? -INFINITY : ends(1).ref[sr], top = fmaxf(r0, r1);
                const float f0 = r0 == -INFINITY ? 0.f : ex2(r0 - top), f1 = r1 == -INFINITY ? 0.f : ex2(r1 - top);
                const float sum = ends(s1).sum[sr] * f0 + (NQ == 2 ? 0.f : ends(1).sum[sr] * f1), inv = sum == 0.f ? 0.f : 1.f / sum;
                float* slot = p.ws_slots + part.slot(blockIdx.x) * Sh::kSlotFloats;
                if (!whole && (NQ == 2 || st == 0)) {
                    __stcg(slot + row, top);
                    __stcg(slot + kRows + row, sum);
                }
                uint16_t* out = row < rows ? out_row<kRows>(p, cur.r.row0, cur.h, cur.rb, row, D) : nullptr;
                // NQ = 1: each stream's warps put out half of the columns
                const int c0 = NQ == 2 ? 0 : st * (D / 2), c1 = NQ == 2 ? D : c0 + D / 2;
                constexpr int kCols = NQ == 2 ? 32 : 16;
#pragma unroll 1
                for (int c = c0; c < c1; c += kCols) {
                    float a[kCols];
                    if constexpr (NQ == 2) {
                        us::tmem_ld32(tmem + lanes + 256 + st * 128 + c, a);
#pragma unroll
                        for (int j = 0; j < kCols; ++j) a[j] = f0 == 0.f ? 0.f : a[j] * f0;
                    } else {
                        float b[kCols];
#pragma unroll
                        for (int j = 0; j < kCols; ++j) a[j] = b[j] = 0.f;
                        if (has[0]) us::tmem_ld16(tmem + lanes + 256 + c, a);
                        if (has[1]) us::tmem_ld16(tmem + lanes + 384 + c, b);
#pragma unroll
                        for (int j = 0; j < kCols; ++j) a[j] = (f0 == 0.f ? 0.f : a[j] * f0) + (f1 == 0.f ? 0.f : b[j] * f1);
                    }
                    if (whole) {
                        if (row < rows) {
#pragma unroll
                            for (int j = 0; j < kCols; j += 8) store8<ELEM>(out + c + j, a + j, inv);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < kCols; j += 4)
                            __stcg(reinterpret_cast<float4*>(slot + 2 * kRows) + (c + j) / 4 * kRows + row,
                                   make_float4(a[j], a[j + 1], a[j + 2], a[j + 3]));
                    }
                }
            }
            if (!whole && part.first == (int)blockIdx.x && threadIdx.x == 0) p.ws_parts[blockIdx.x] = part;
            us::tc_fence_before();
            us::named_bar_sync(1, 32 * kSoftWarps);        // Q, the streams' TMEM and sums are free
            us::tc_fence_after();
            it = end;
            if (it < count) cur.next_segment(p);
        }
    } else if (warp == kMmaWarp) {
        // --------------------------------------------------------------- MMA
        if (us::elect_one()) {
            int segment = 0;
            for (int it = 0; it < count; ++segment) {
                const int end = min(count, it + cur.tiles - cur.tile);
                // scores of half a of tile i for stream st; last: nothing after them reads the tile's K
                auto qk = [&](int i, int st, int a, bool last) {
                    constexpr uint32_t id = us::umma_idesc_f16(kM, 64);
                    if (a == 0) wait(&H.k_full[i % kKS], i / kKS);
                    us::tc_fence_after();
                    const uint64_t qd = us::umma_smem_desc_sw128(q_sm + (NQ == 2 ? st * Sh::kOperand : 0));
                    const uint64_t kd = us::umma_smem_desc_sw128(k_sm + (i % kKS) * Sh::kOperand) + (uint64_t)(a * 64 * 128 >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint64_t at = (uint64_t)(((kk >> 2) * Sh::kGroup + (kk & 3) * 32) >> 4);
                        us::umma_f16(tmem + st * 128 + a * 64, qd + at, kd + at, id, kk > 0);
                    }
                    us::umma_commit(&H.qk_done[st][a]);
                    if (last) us::umma_commit(&H.k_free[i % kKS]);
                };
                // outputs of half a of tile i for stream st, whose use-th tile it is
                auto pv = [&](int i, int st, int a, int use, bool first, bool last) {
                    constexpr uint32_t id = us::umma_idesc_f16(kM, D) | us::kUmmaBMajorMN;
                    if (a == 0) wait(&H.v_full[i % kVS], i / kVS);
                    wait(&H.p_full[st][a], use);
                    us::tc_fence_after();
                    const uint64_t vd = us::umma_smem_desc_mn_sw128(v_sm + (i % kVS) * Sh::kOperand, Sh::kGroup) + (uint64_t)(a * 64 * 128 >> 4);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        us::umma_f16_ta(tmem + 256 + st * 128, tmem + st * 128 + a * 64 + 8 * kk, vd + (uint64_t)(kk * 2048 >> 4), id,
                                        !first || kk > 0);
                    us::umma_commit(&H.pv_done[st][a]);
                    if (last) us::umma_commit(&H.v_free[i % kVS]);
                };
                wait(&H.q_full, segment);
                if constexpr (NQ == 2) {
#pragma unroll 1
                    for (int x = 0; x < 4; ++x) qk(it, x & 1, x >> 1, x == 3);
                    for (int i = it; i < end; ++i)
#pragma unroll 1
                        for (int x = 0; x < 4; ++x) {
                            const int st = x & 1, a = x >> 1;
                            pv(i, st, a, i, i == it && a == 0, x == 3);
                            if (i + 1 < end) qk(i + 1, st, a, x == 3);
                        }
                } else {
#pragma unroll 1
                    for (int x = 0; x < 4 && it + (x >> 1) < end; ++x) qk(it + (x >> 1), (it + (x >> 1)) & 1, x & 1, x & 1);
                    for (int i = it; i < end; ++i)
#pragma unroll 1
                        for (int a = 0; a < 2; ++a) {
                            pv(i, i & 1, a, i / 2, i - it < 2 && a == 0, a == 1);
                            if (i + 2 < end) qk(i + 2, i & 1, a, a == 1);
                        }
                }
                it = end;
                if (it < count) cur.next_segment(p);
            }
            // Arrivals that no other warp waits for: they land while the CTA still has its shared memory
            for (int i = max(0, count - kKS); i < count; ++i) wait(&H.k_free[i % kKS], i / kKS);
            for (int i = max(0, count - kVS); i < count; ++i) wait(&H.v_free[i % kVS], i / kVS);
            for (int x = 0; x < 2; ++x) {
                const int used = NQ == 2 ? count : (count + 1 - x) / 2;     // tiles of stream x
                if (used) wait(&H.pv_done[x][0], used - 1);
            }
        }
        __syncwarp();
    } else {
        // -------------------------------------------------------- conversion
        // Items in their order, tile after tile across segments: item x of the CTA is
        // block x % 16 of tile x / 16, every seventh is this warp's.  While one is
        // converted, the next kRS - 1 are copied and the page number of the one behind
        // them is loaded.
        constexpr int kRS = Sh::kRS;
        const int items = kItems * count;
        // the lane's chunks: u-th is 8 rows, or 64 bytes, behind the one before (eight
        // lanes on eight rows: no bank conflicts when they are put)
        const int lrow = Sh::kC == 2 ? lane & 15 : lane & 7, lchunk = Sh::kC == 2 ? lane >> 4 : lane >> 3;
        const uint32_t get_at = (uint32_t)(lrow * Sh::kRow + lchunk * 16);
        auto get_u = [](int u) { return Sh::kC == 8 ? (u >> 1) * 8 * Sh::kRow + (u & 1) * 64 : u * 8 * Sh::kRow; };
        // where they go (operand_at, with what depends on the lane alone): row, 64
        // dimensions, swizzled chunk
        const uint32_t put_base = (uint32_t)(lrow * 128 + (lchunk * Sh::kOut >> 3) * Sh::kGroup);
        const uint32_t put_chunk = (uint32_t)(((lchunk * Sh::kOut & 7) ^ (lrow & 7)) << 4);
        auto put_u = [](int u) { return Sh::kC == 8 ? (u >> 1) * 1024 + (u & 1) * Sh::kGroup : u * 1024; };
        uint8_t* raw = raw_sm + (warp - kMmaWarp - 1) * kRS * Sh::kRaw;

        // the item whose page number is on its way
        int nx_item = warp - kMmaWarp - 1, nx_tile = 0, nx_page = -1, nx_pos = 0;
        auto locate = [&]() {                              // (at most one tile further)
            if (nx_item >= items) return;
            if ((nx_item >> 4) > nx_tile) cur.next(p), ++nx_tile;
            nx_pos = cur.tile * kTile + (nx_item & 7) * 16;
            if (nx_pos < cur.r.ctx + cur.r.n) nx_page = p.c.table[(int64_t)cur.b * p.c.max_pages + (nx_pos >> p.c.page_shift)];
        };
        // copies it (key head h, `after` positions of the request from its first on) to
        // ring place `slot`; says how many of its positions are the request's, 0 if it
        // has no entries
        auto copy_item = [&](int slot, int h, int after) {
            int left = 0;
            if (nx_item < items && after > 0) {
                if (nx_page >= 0 && nx_page < p.c.num_pages) {
                    const int64_t e = us::kv_entry(p.c, nx_page, h, nx_pos);
                    const uint8_t* src = (nx_item & 8 ? p.c.v : p.c.k) + e * Sh::kRow + get_at;
                    const uint32_t to = us::smem_addr(raw + slot * Sh::kRaw) + lane * 16;
#pragma unroll
                    for (int u = 0; u < Sh::kLoads; ++u) cp_async16(to + u * 512, src + get_u(u));
                    if (lane < 16)
                        cp_async4(us::smem_addr(raw + slot * Sh::kRaw) + 16 * Sh::kRow + lane * 4, p.c.scale + 2 * (e + lane));
                    left = min(16, after);
                } else {
                    us::set_status(p.c.status, US_ERR_CORRUPT);
                }
            }
            cp_async_commit();
            return left;
        };
        auto fetch = [&](int slot) {
            const int left = copy_item(slot, cur.h, cur.r.ctx + cur.r.n - nx_pos);
            if (nx_item < items) {
                nx_item += kConvWarps;
                locate();
            }
            return left;
        };
        // the first kRS items: their page numbers at once, a lane each
        uint32_t lefts = 0;                                // of the items under way, 8 bits each
        {
            Cur at = cur;
            const int mine = nx_item + kConvWarps * lane, tile = mine >> 4;
            const bool want = lane < kRS && mine < items;
            if (want)
                for (int t = 0; t < tile; ++t) at.next(p);
            const int pos = at.tile * kTile + (mine & 7) * 16, left = want ? at.r.ctx + at.r.n - pos : 0;
            const int page = left > 0 ? p.c.table[(int64_t)at.b * p.c.max_pages + (pos >> p.c.page_shift)] : -1;
#pragma unroll
            for (int s = 0; s < kRS; ++s) {
                nx_page = __shfl_sync(0xffffffffu, page, s);
                nx_pos = __shfl_sync(0xffffffffu, pos, s);
                const int h = __shfl_sync(0xffffffffu, at.h, s), l = __shfl_sync(0xffffffffu, left, s);
                lefts |= (uint32_t)copy_item(s, h, l) << (8 * s);
                if (nx_item < items) nx_item += kConvWarps;
            }
            const int last = nx_item < items ? nx_item >> 4 : 0;
            for (; nx_tile < last; ++nx_tile) cur.next(p);
            locate();
        }
        int slot = 0;
        for (int item = warp - kMmaWarp - 1; item < items; item += kConvWarps) {
            const int i = item >> 4, block = item & 7, left = (int)(lefts & 0xFFu);
            const bool is_v = (item & 8) != 0;
            cp_async_wait<kRS - 1>();                      // a lane reads what it copied
            const uint8_t* r = raw + slot * Sh::kRaw;
            uint4 c[Sh::kLoads];
#pragma unroll
            for (int u = 0; u < Sh::kLoads; ++u)
                c[u] = left ? *reinterpret_cast<const uint4*>(r + u * 512 + lane * 16) : make_uint4(0, 0, 0, 0);
            const uint32_t scale = left && lane < 16 ? reinterpret_cast<const uint32_t*>(r + 16 * Sh::kRow)[lane] : 0u;
            // Entries that no row sees may hold any scale: behind the request's last
            // position V's counts as 0, and one that is not finite is left to those
            // who see its entry, through K's.
            uint32_t sv = scale >> 16;
            const bool bad = (sv & 0x7C00u) == 0x7C00u;
            if (bad || lane >= left) sv = 0;
            const uint32_t vbits = __float_as_uint(us::half_bits_to_float((uint16_t)sv));      // (a subnormal scale too)
            const float vp = __uint_as_float(vbits & 0x7F800000u), vm = __uint_as_float((vbits & 0x807FFFFFu) | 0x3F800000u);
            const uint32_t vp2 = pack_half2(vp, vp);
            // -128 at 2^9 and -8 at 2^13 are beyond fp16: us_kv_write stores no such entry, but
            // 0 times an infinity would be every row's NaN.  Largest codes saturate instead.
            const bool large = __any_sync(0xffffffffu, vp >= (ELEM == US_I8 ? 512.f : 8192.f));
            uint32_t vscale[2];                            // of the lane's rows
#pragma unroll
            for (int u = 0; u < 2; ++u) vscale[u] = __shfl_sync(0xffffffffu, vp2, Sh::kC == 2 ? lane & 15 : 8 * u + (lane & 7));
            lefts = lefts >> 8 | (uint32_t)fetch(slot) << (8 * (kRS - 1));       // its place is free
            slot = slot + 1 == kRS ? 0 : slot + 1;
            uint8_t* operand;
            if (is_v) {
                if (i >= kVS) wait(&H.v_free[i % kVS], i / kVS - 1);
                operand = v_sm + (i % kVS) * Sh::kOperand;
            } else {
                if (i >= kKS) wait(&H.k_free[i % kKS], i / kKS - 1);
                operand = k_sm + (i % kKS) * Sh::kOperand;
                const float sk = us::half_bits_to_float((uint16_t)scale) * (p.scale * 1.4426950408889634f);
                if (lane < 16) {
                    float* at = reinterpret_cast<float*>(H.scales[i % kSS]) + 32 * block + 4 * (lane >> 1) + (lane & 1);
                    at[0] = bad ? __uint_as_float(0x7FC00000u) : sk;
                    at[2] = vm;
                }
                if (lane == 0) H.valid[i % kSS][block] = left ? 0xFFFFu : 0u;
            }
            uint8_t* to = operand + block * 16 * 128 + put_base;
#pragma unroll
            for (int u = 0; u < Sh::kLoads; ++u) {
                uint4 out[Sh::kOut];
                convert<ELEM>(c[u], out);
                if (is_v) {
                    const uint32_t s = vscale[Sh::kC == 2 ? 0 : u / (Sh::kC / 4)];
#pragma unroll
                    for (int k = 0; k < Sh::kOut; ++k)
                        out[k] = make_uint4(hmul2(out[k].x, s), hmul2(out[k].y, s), hmul2(out[k].z, s), hmul2(out[k].w, s));
                    if (large) {
#pragma unroll
                        for (int k = 0; k < Sh::kOut; ++k)
                            out[k] = make_uint4(us::saturate_half2(out[k].x), us::saturate_half2(out[k].y),
                                                us::saturate_half2(out[k].z), us::saturate_half2(out[k].w));
                    }
                }
#pragma unroll
                for (int k = 0; k < Sh::kOut; ++k) *reinterpret_cast<uint4*>(to + put_u(u) + (put_chunk ^ (k << 4))) = out[k];
            }
            us::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                us::mbar_arrive(is_v ? &H.v_full[i % kVS] : &H.k_full[i % kKS]);
                if (!is_v) us::mbar_arrive(&H.s_full[i % kSS]);
            }
        }
        cp_async_wait<0>();
    }
    us::tc_fence_before();
    __syncthreads();
    if (warp == kSoftWarps) us::tmem_dealloc(tmem, 512);
    us::pdl_launch_dependents();
}

// Joins the partial states of shared segments, 16 rows of one at a time: CTAs take
// such pieces in turn from the list of shared segments, which each makes for itself
// (part c: the segment whose first sharer was CTA c, if there is one).  A thread takes
// 8 columns of a row; its loads of AT states are on their way at once.  A launch of
// its own: joined by one of the sharers, a segment's states (131 KB each at 256 rows
// of 128) came at the 76 GB/s that one SM draws from L2.
// Few segments have many sharers each: eight states at once (a tree of 32
// tokens of one request behind 4000 positions: 20 us with the attention, 29 with two
// at once; of 64 tokens 23 and 27).  Many have about two: two at once, and three times
// as many CTAs (chunk of 512: 177 us, 180 with eight).
constexpr int kJoinRows = 16, kMaxCtas = 512;
constexpr int join_ctas(int at, int D) { return (at == 8 ? 256 : 768) / D; }       // an SM
template <int ELEM, int D, int NQ, int AT>
__global__ void __launch_bounds__(kJoinRows * D / 8, join_ctas(AT, D))
attn_tc_join_kernel(const UsAttnParams p, int ctas) {
    using Sh = Shape<ELEM, D, NQ>;
    constexpr int kRows = Sh::kRows, kPieces = kRows / kJoinRows;
    __shared__ uint16_t list[kMaxCtas];
    __shared__ int listed;
    us::pdl_wait();
    if (threadIdx.x < 32) {
        int n = 0;
        for (int c0 = 0; c0 < ctas; c0 += 32) {
            const int c = c0 + (int)threadIdx.x;
            const bool shared = c < ctas && p.ws_parts[c].rows > 0;
            const unsigned who = __ballot_sync(0xffffffffu, shared);
            if (shared) list[n + __popc(who & ((1u << threadIdx.x) - 1u))] = (uint16_t)c;
            n += __popc(who);
        }
        if (threadIdx.x == 0) listed = n;
    }
    __syncthreads();
    for (int x = blockIdx.x; x < listed * kPieces; x += gridDim.x) {
        const Part a = p.ws_parts[list[x / kPieces]];
        const int row = x % kPieces * kJoinRows + threadIdx.x % kJoinRows, col = threadIdx.x / kJoinRows * 8;
        if (row >= a.rows) continue;
        float top = -INFINITY, sum = 0.f, y[8] = {};
        for (int c = a.first; c <= a.last; c += AT) {
            float4 v[AT][2];
            float r[AT], l[AT];
#pragma unroll
            for (int u = 0; u < AT; ++u) {
                const float* sl = p.ws_slots + a.slot(c + u) * Sh::kSlotFloats;
                const float4* o = reinterpret_cast<const float4*>(sl + 2 * kRows) + col / 4 * kRows + row;
                r[u] = -INFINITY, l[u] = 0.f;
                v[u][0] = v[u][1] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c + u <= a.last) {
                    r[u] = __ldcg(sl + row);
                    l[u] = __ldcg(sl + kRows + row);
                    v[u][0] = __ldcg(o), v[u][1] = __ldcg(o + kRows);
                }
            }
            float m = top;
#pragma unroll
            for (int u = 0; u < AT; ++u) m = fmaxf(m, r[u]);
            // (a state without a reference has weights 0, or NaN, which stays)
            const float at = m == -INFINITY ? 0.f : m, f0 = ex2(top - at);
            sum *= f0;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] *= f0;
#pragma unroll
            for (int u = 0; u < AT; ++u) {
                const float f = ex2(r[u] - at);
                sum += l[u] * f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    y[4 * i] += v[u][i].x * f, y[4 * i + 1] += v[u][i].y * f;
                    y[4 * i + 2] += v[u][i].z * f, y[4 * i + 3] += v[u][i].w * f;
                }
            }
            top = m;
        }
        store8<ELEM>(out_row<kRows>(p, a.row0, a.h, a.rb, row, D) + col, y, sum == 0.f ? 0.f : 1.f / sum);
    }
    us::pdl_launch_dependents();
}

int grid() { return us::num_sms() < kMaxCtas ? us::num_sms() : kMaxCtas; }
constexpr int kPartBytes = 4096 + kMaxCtas * 32;       // counters, parts
static_assert(sizeof(Part) <= 32, "parts");

template <int ELEM, int D, int NQ>
us_status launch(UsAttnParams p, cudaStream_t st) {
    using Sh = Shape<ELEM, D, NQ>;
    static_assert(Sh::kSmem <= 232448, "shared memory");
    p.ws_parts = reinterpret_cast<Part*>(static_cast<uint8_t*>(p.ws) + 4096);      // behind the other kernel's counters
    p.ws_slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kPartBytes);
    auto kern = attn_tc_kernel<ELEM, D, NQ>;
    static std::atomic<bool> ready[64];                // the attribute is set once a device, by whichever thread
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return US_ERR_CUDA;
    if (!ready[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess)
            return US_ERR_CUDA;
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Sh::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return US_ERR_CUDA;
    const int64_t segments = (((int64_t)p.a.max_n * p.G + Sh::kRows - 1) / Sh::kRows) * p.c.Hkv * p.c.B;      // at most
    const bool few = 4 * segments <= grid();
    cfg.gridDim = dim3((unsigned)(join_ctas(few ? 8 : 2, D) * us::num_sms()));
    cfg.blockDim = dim3(kJoinRows * D / 8);
    cfg.dynamicSmemBytes = 0;
    auto join = few ? attn_tc_join_kernel<ELEM, D, NQ, 8> : attn_tc_join_kernel<ELEM, D, NQ, 2>;
    return cudaLaunchKernelEx(&cfg, join, p, grid()) == cudaSuccess ? US_OK : US_ERR_CUDA;
}

}  // namespace

namespace us {

// From 33 rows per key head.  Below, the mma.sync kernel is faster, although it reads
// the cache once for every 16 rows of 128 dimensions; it has 32 of 64 at once (32 rows,
// 16 requests of 4000 positions / two of 131000, us there and here; int4, 128: 50, 59 /
// 146, 173; int8, 128: 54, 62 / 159, 184; int4, 64: 32, 52 / 86, 152; int8, 64: 35, 53 /
// 89, 157).  Above, 128 dimensions need a third pass (36 rows; int4: 66, 61 / 205, 181;
// int8: 72, 64 / 224, 193).  64 need a second, and there the two are near each other
// (int4: 50, 53 / 147, 159; int8: 53, 54 / 151, 161): one rule for both widths.
bool attn_tc_serves(const UsAttnParams& p) { return (int64_t)p.a.max_n * p.G > 32; }

size_t attn_tc_ws(const UsAttnParams& p) {
    const size_t rows = (int64_t)p.a.max_n * p.G > kM ? 2 * kM : kM;
    return kPartBytes + (size_t)2 * grid() * (2 * rows + rows * p.c.D) * 4;
}

us_status launch_attn_tc(const UsAttnParams& p, cudaStream_t st) {
    const bool two = (int64_t)p.a.max_n * p.G > kM;
#define US_ATTN_PICK(E, D) (two ? launch<E, D, 2>(p, st) : launch<E, D, 1>(p, st))
    if (p.c.elem == US_I8) return p.c.D == 64 ? US_ATTN_PICK(US_I8, 64) : US_ATTN_PICK(US_I8, 128);
    return p.c.D == 64 ? US_ATTN_PICK(US_I4, 64) : US_ATTN_PICK(US_I4, 128);
#undef US_ATTN_PICK
}

}  // namespace us

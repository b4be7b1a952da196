// us_attn.cu -- attention of few query rows per key head over the quantised
// K/V cache (single tokens and small trees), on mma.sync.
//
// Query row (token i of request b, head hq) sees the positions p < ctx, and of
// the call's own tokens j = p - ctx those whose bit is set in the token's mask
// (no mask: j <= i).  o = sum_p w_p v_p / sum_p w_p, w_p = exp(scale q.k_p), 0
// for a row that sees nothing.  With k_p = s_kp ck_p and v_p = s_vp cv_p the
// scales multiply the score and the weight, so the products take the integer
// codes, which fp16 holds exactly:
//   S^T = Ck Q^T   (tokens x rows),   O^T = Cv^T P^T   (dimensions x rows).
// Both products have the cache as the 16-row A operand and the query rows as
// the 8-column B operand: few rows waste little of an MMA, and each code is
// converted once for all rows.
//
// Which lane holds what.  The contraction of S^T may run over the dimensions
// in any order, and the tokens may enter O^T in any order, so both are chosen
// such that a lane's codes are neighbours in memory: lane (g, c) = (lane / 4,
// lane % 4) takes D/4 codes of K of tokens g' and g' + 8, and of V the D/8
// dimensions from g D/8 of tokens c, c + 4, c + 8, c + 12.
//
// Codes of both become signed fp16 numbers before the product.  K's could enter with
// their offset of 8 (128), taken back from the sum, for one operation a pair less; but
// then rounding goes by 128 sum |q| however small the products are (keys of few large
// channels, one rounding a step: scores of 220 off by 4.7).  So with V's in an output.
//
// Work: the (request, key head, row block) segments are cut into tiles of 64 to 256
// positions, and the tile sequence is spread evenly over the CTAs, whatever the
// lengths (they are read on the device).  A warp takes 16 or 32 positions of each
// tile, copied into the warp's own ring several tiles ahead and across segments (a
// page's entries of one head are contiguous).  A segment shared by several CTAs leaves
// partial states in the workspace; the CTA that arrives last joins them in the order
// of the tiles.
//
// What bounds it: at one token of a long context HBM (two requests of 131000
// positions, int8: 5.3 TB/s of a cache that streams once), with more requests the
// instructions of the codes' conversion (48 requests of 4096 to 8192, int4: ALU pipe
// 45 % and issue slots 56 % busy, 3.8 TB/s), with one short request latency (9 us
// for 777 positions: starting, finding the work, three trips to memory, the join).
#include <atomic>

#include "us_attn.cuh"
#include "us_internal.h"

namespace {

using namespace us::attn;

constexpr int kBlock = 16;                        // positions of one MMA's rows: they lie in one page
// log2 of a row's largest weight with V's scale in it: when its reference is set, and what
// it may grow to after that (2^15 < 65504; small weights keep fp16's bits down to 2^-25 of it)
constexpr float kTop = 11.f, kMost = 15.f;

template <int ELEM, int D, int NT, int W>
struct Shape {
    static constexpr int kWarps = W, kThreads = 32 * W;
    static constexpr int kRows = 8 * NT;
    static constexpr int kRow = D * (ELEM == US_I8 ? 8 : 4) / 8;    // bytes of a row of codes
    static constexpr int kKW = kRow / 16;                           // words a lane holds of a K row
    static constexpr int kVW = kRow / 32;                           // ... of a V row (its D/8 dimensions)
    static constexpr int kKS = D / 16;                              // MMA steps over the dimensions
    static constexpr int kMT = D / 16;                              // 16-dimension blocks of O^T
    // CTAs an SM.  Rows of 128 dimensions, and 17 to 32 rows of 64, need more than the
    // 168 registers that three CTAs of four warps leave (16 trees of 4 tokens, 4 query
    // heads to a key head, behind 4095 positions, int4: 33 us with two CTAs, 35 with
    // three of one block a step; 12 trees of 13 to 25, 64 dimensions, int8: 62 and 96);
    // 9 to 16 rows of 64 do not (trees of up to 12: 46 and 41).
    static constexpr int kMinB = W == 8 || NT == 4 || D == 128 ? 2 : 3;
    // 16-position blocks of a warp's step: with two there are twice as many MMAs that do
    // not wait for each other (4 tokens of two requests of 131000 positions, int8: 90 us
    // against 103), where the registers hold their codes.
    static constexpr int kSub = kRow == 128 && NT == 1 ? 1 : 2;
    static constexpr int kStep = kSub * kBlock;
    static constexpr int kTile = kWarps * kStep;                    // positions of a CTA's step
    static constexpr int kStageBytes = 2 * kStep * kRow + kStep * 4;
    static constexpr int kJoin = kWarps * 32 * 32 * 4;              // O^T of four warps, 32 values a lane at a time
    static constexpr int kFixed = kJoin + kWarps * kRows * 8 + kRows * 20 + 512;
    static constexpr int kFit = (224 * 1024 / kMinB - 2048 - kFixed) / (kWarps * kStageBytes);
    static constexpr int kStages = kFit > 5 ? 5 : kFit;
    static constexpr int kSmem = kFixed + kWarps * kStages * kStageBytes;
    static_assert(kStages >= 2, "ring");
    static constexpr int kSlotFloats = 2 * kRows + kRows * D;       // m, l, O^T of one partial state
};

US_DEV uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

template <int N>
US_DEV void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N >= 4) {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            // 64 bytes apart: K rows of 128 bytes are read as two halves
            const uint4 u = *reinterpret_cast<const uint4*>(p + 64 * i);
            w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
        }
    } else if constexpr (N == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x, w[1] = u.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// Joins the partial states of a shared segment: O^T of eight states at a time
// is on its way while the rows' maxima and the states' factors (kBatch states in
// `buf`) are found.
template <int ELEM, int D, int NT, int W>
US_DEV void join_states(const UsAttnParams& p, float* buf, float* sums, const Part& a) {
    using Sh = Shape<ELEM, D, NT, W>;
    constexpr int kThreads = Sh::kThreads, kRows = Sh::kRows, kQuads = D * kRows / 4;
    constexpr int kMine = (kQuads + kThreads - 1) / kThreads, kPar = kThreads / kRows, kBatch = 8 * kPar;
    constexpr int kLoads = kMine > 2 ? 4 : 8;              // states in flight
    static_assert(kBatch * kRows * 4 <= Sh::kJoin, "factors");
    const int lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
    const int first = a.first, np = a.last - a.first + 1;
    auto slot_of = [&](int j) { return p.ws_slots + a.slot(first + j) * Sh::kSlotFloats; };
    auto row_of = [&](int k) {
        const int x = threadIdx.x + k * kThreads;
        return 8 * ((x >> 6) % NT) + 2 * c4 + ((x >> 5) & 1);
    };
    float4 v[kLoads][kMine];
    auto load = [&](int j) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
#pragma unroll
            for (int k = 0; k < kMine; ++k)
                v[u][k] = j + u < np && row_of(k) < a.rows && threadIdx.x + k * kThreads < kQuads
                              ? __ldcg(reinterpret_cast<const float4*>(slot_of(j + u) + 2 * kRows) + threadIdx.x + k * kThreads)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    load(0);
    const int r = threadIdx.x % kRows, j0 = threadIdx.x / kRows;
    float m0 = -INFINITY, l0 = 0.f;                        // of the thread's first state
    if (j0 < np) m0 = __ldcg(slot_of(j0) + r), l0 = __ldcg(slot_of(j0) + kRows + r);
    float t = m0;
#pragma unroll 4
    for (int j = j0 + kPar; j < np; j += kPar) t = fmaxf(t, __ldcg(slot_of(j) + r));
    buf[threadIdx.x] = t;
    __syncthreads();
    t = buf[r];
#pragma unroll
    for (int j = 1; j < kPar; ++j) t = fmaxf(t, buf[j * kRows + r]);
    __syncthreads();
    float sum = 0.f;                                       // of the thread's states of row r
    float4 y[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < np; base += kBatch) {
        const int nb = min(kBatch, np - base);
        if (base) __syncthreads();
        for (int j = j0; j < nb; j += kPar) {
            const float* sl = slot_of(base + j);
            const bool kept = base + j == j0;
            const float mc = kept ? m0 : __ldcg(sl + r), lc = kept ? l0 : __ldcg(sl + kRows + r);
            const float f = mc == -INFINITY ? 0.f : ex2(mc - t);
            sum += lc * f;
            buf[j * kRows + r] = f;
        }
        __syncthreads();
        for (int j = 0; j < nb; j += kLoads) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u)
#pragma unroll
                for (int k = 0; k < kMine; ++k) {
                    const float f = j + u < nb ? buf[(j + u) * kRows + row_of(k)] : 0.f;
                    y[k].x += v[u][k].x * f, y[k].y += v[u][k].y * f;
                    y[k].z += v[u][k].z * f, y[k].w += v[u][k].w * f;
                }
            load(base + j + kLoads);
        }
    }
    __syncthreads();
    buf[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < kRows) {
        for (int j = 1; j < kPar; ++j) sum += buf[j * kRows + r];
        sums[r] = sum == 0.f ? 0.f : 1.f / sum;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
        const int x = threadIdx.x + k * kThreads, row = row_of(k);
        if (row >= a.rows || x >= kQuads) continue;
        const float inv = sums[row];
        uint16_t* out = out_row<kRows>(p, a.row0, a.h, a.rb, row, D) + g * (D / 8) + 4 * ((x >> 6) / NT);
        *reinterpret_cast<uint2*>(out) = make_uint2(pack_out(y[k].x * inv, y[k].y * inv), pack_out(y[k].z * inv, y[k].w * inv));
    }
}

template <int ELEM, int D, int NT, int W>
__global__ void __launch_bounds__(32 * W, (Shape<ELEM, D, NT, W>::kMinB))
attn_mma_kernel(const UsAttnParams p) {
    using Sh = Shape<ELEM, D, NT, W>;
    constexpr int kRows = Sh::kRows, kStages = Sh::kStages, kKW = Sh::kKW, kVW = Sh::kVW, kMT = Sh::kMT;
    constexpr int kSub = Sh::kSub, kStep = Sh::kStep, kWarps = Sh::kWarps, kThreads = Sh::kThreads;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* ring = smem;
    float* join = reinterpret_cast<float*>(ring + kWarps * kStages * Sh::kStageBytes);
    float* sm_m = join + Sh::kJoin / 4;                    // [kWarps][kRows]
    float* sm_l = sm_m + kWarps * kRows;
    uint64_t* sm_mask = reinterpret_cast<uint64_t*>(sm_l + kWarps * kRows);     // [kRows]
    int* sm_tok = reinterpret_cast<int*>(sm_mask + kRows);                       // [kRows]
    float* sm_inv = reinterpret_cast<float*>(sm_tok + kRows);                    // [kRows]
    __shared__ unsigned sh_last;
    __shared__ Part sh_part[2];
    __shared__ Work sh_work;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c4 = lane & 3;
    const int G = p.G;
    us::pdl_wait();

    // ---- this CTA's tiles
    Work wk;
    Cursor<kRows, Sh::kTile> cur;
    if (!find_work<kRows, Sh::kTile>(p, wk, cur)) return;
    const int count = (int)(wk.t1 - wk.t0);
    if (threadIdx.x == 0) sh_work = wk;                    // read at a segment's end: no registers for it meanwhile

    // ---- producer: the warp's positions of tile `pc` into stage s, 16 bytes a lane
    // at a time; the page numbers are loaded one tile ahead.
    Cursor<kRows, Sh::kTile> pc = cur;
    uint8_t* wring = ring + warp * kStages * Sh::kStageBytes;
    uint32_t have = 0;                                     // kSub bits a stage: which blocks it holds
    int page[kSub];
    auto copy = [&](int s, int sub, int64_t e) {           // the 16-position block at entry e
        const uint32_t st = us::smem_addr(wring + s * Sh::kStageBytes) + lane * 16;
        const uint8_t *k = p.c.k + e * Sh::kRow + lane * 16, *v = p.c.v + e * Sh::kRow + lane * 16;
#pragma unroll
        for (int u = 0; u < kBlock * Sh::kRow / 512; ++u) {
            cp_async16(st + sub * kBlock * Sh::kRow + u * 512, k + u * 512);
            cp_async16(st + (kStep + sub * kBlock) * Sh::kRow + u * 512, v + u * 512);
        }
        if (lane < kBlock / 4)
            cp_async16(st + 2 * kStep * Sh::kRow + sub * kBlock * 4, reinterpret_cast<const uint8_t*>(p.c.scale) + e * 4 + lane * 16);
    };
    auto find_pages = [&]() {
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb) {
            const int pos = pc.tile * Sh::kTile + warp * kStep + sb * kBlock;
            page[sb] = -1;
            if (pos < pc.r.ctx + pc.r.n) page[sb] = p.c.table[(int64_t)pc.b * p.c.max_pages + (pos >> p.c.page_shift)];
        }
    };
    auto issue = [&](int s, bool more) {
        have &= ~(((1u << kSub) - 1u) << (s * kSub));
#pragma unroll
        for (int sb = 0; sb < kSub; ++sb) {
            const int pos = pc.tile * Sh::kTile + warp * kStep + sb * kBlock;
            if (page[sb] >= 0 && page[sb] < p.c.num_pages) {
                copy(s, sb, us::kv_entry(p.c, page[sb], pc.h, pos));
                have |= 1u << (s * kSub + sb);
            } else if (pos < pc.r.ctx + pc.r.n) {
                us::set_status(p.c.status, US_ERR_CORRUPT);
            }
        }
        if (more) {
            pc.next(p);
            find_pages();
        }
    };
    // The first stages: their page numbers at once, a lane a block.
    const int ahead = count < kStages ? count : kStages;
    {
        const int st = lane / kSub, sub = lane - st * kSub;
        Cursor<kRows, Sh::kTile> at = cur;
        for (int i = 0; i < st && st < ahead; ++i) at.next(p);
        const int pos = at.tile * Sh::kTile + warp * kStep + sub * kBlock;
        const bool want = st < ahead && pos < at.r.ctx + at.r.n;
        const int id = want ? p.c.table[(int64_t)at.b * p.c.max_pages + (pos >> p.c.page_shift)] : -1;
        const bool ok = id >= 0 && id < p.c.num_pages;
        if (want && !ok) us::set_status(p.c.status, US_ERR_CORRUPT);
        const int64_t e = ok ? us::kv_entry(p.c, id, at.h, pos) : -1;
#pragma unroll
        for (int i = 0; i < kStages * kSub; ++i) {
            const int64_t ei = __shfl_sync(0xffffffffu, e, i);
            if (ei >= 0) {
                copy(i / kSub, i % kSub, ei);
                have |= 1u << i;
            }
            if (i % kSub == kSub - 1) cp_async_commit();
        }
        for (int i = 0; i < ahead && i + 1 < count; ++i) pc.next(p);
        if (ahead < count) find_pages();
    }

    // ---- consumer state: references, sums and O^T of the warp's positions.  Weights are
    // 2^(s - m); a row's m is 11 less than its largest s + log2(V's scale), so that an
    // entry which a row does not see, or hardly weighs, takes no bits from its weights.
    float m[NT][2], l[NT][2], o[kMT][NT][4];
    float room = kMost;                                    // 0 from where an m is large on
    uint32_t qf[Sh::kKS][NT][2];
    const float sc = p.scale * 1.4426950408889634f;        // weights as powers of two
    int parts = 0;
    const int rt = ((g & 1) << 2) | (g >> 1);              // token of row g (k index 2c -> c, 2c + 1 -> c + 4)

    auto begin_segment = [&]() {
        const int rows = cur.r.n * G;
        room = kMost;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < kMT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][nt][e] = 0.f;
            const int r = cur.rb * kRows + 8 * nt + g;
            const int i = r / G;
            const uint16_t* q = p.Q + (int64_t)(cur.r.row0 + i) * p.ldq + (cur.h * G + r - i * G) * D;
#pragma unroll
            for (int w = 0; w < kKW; ++w) {
                if constexpr (ELEM == US_I4) {
                    uint4 u = make_uint4(0, 0, 0, 0);
                    if (r < rows) u = *reinterpret_cast<const uint4*>(q + c4 * (D / 4) + 8 * w);
                    qf[2 * w][nt][0] = __byte_perm(u.x, u.z, 0x5410), qf[2 * w][nt][1] = __byte_perm(u.y, u.w, 0x5410);
                    qf[2 * w + 1][nt][0] = __byte_perm(u.x, u.z, 0x7632), qf[2 * w + 1][nt][1] = __byte_perm(u.y, u.w, 0x7632);
                } else {
                    uint2 u = make_uint2(0, 0);
                    if (r < rows) u = *reinterpret_cast<const uint2*>(q + (w >> 2) * 64 + c4 * 16 + 4 * (w & 3));
                    qf[w][nt][0] = __byte_perm(u.x, u.y, 0x5410), qf[w][nt][1] = __byte_perm(u.x, u.y, 0x7632);
                }
            }
        }
        if (threadIdx.x < kRows) {
            const int r = cur.rb * kRows + threadIdx.x, i = r / G;
            sm_tok[threadIdx.x] = r < rows ? i : -1;
            sm_mask[threadIdx.x] = r < rows && p.mask ? p.mask[cur.r.row0 + i] : 0;
        }
        __syncthreads();
    };

    begin_segment();
    int s = 0;
    for (int it = 0; it < count; ++it) {
        cp_async_wait<kStages - 1>();
        __syncwarp();                                      // every lane's part of the stage is there
        const uint32_t blocks = (have >> (s * kSub)) & ((1u << kSub) - 1u);
        if (blocks) {
            const uint8_t* st = wring + s * Sh::kStageBytes;
            const int pos = cur.tile * Sh::kTile + warp * kStep;
            float sx[kSub][NT][4], vs[kSub][2], lv[kSub][2];
            const bool edge = pos + kStep > cur.r.ctx || blocks != (1u << kSub) - 1u;
#pragma unroll
            for (int sb = 0; sb < kSub; ++sb) {
                // ---- S^T = Ck Q^T
                float (&sa)[NT][4] = sx[sb];
                float so[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sa[nt][e] = so[nt][e] = 0.f;
                uint32_t k0[kKW], k1[kKW];
                const uint8_t* kr = st + (sb * kBlock + rt) * Sh::kRow + c4 * (kKW >= 4 ? 16 : 4 * kKW);
                lds_words(kr, k0);
                lds_words(kr + 8 * Sh::kRow, k1);
#pragma unroll
                for (int w = 0; w < kKW; ++w) {
                    if constexpr (ELEM == US_I4) {
                        uint32_t x[4], y[4];
                        decode_i4(k0[w], x);
                        decode_i4(k1[w], y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            us::mma_m16n8k16_f16(sa[nt], x[0], y[0], x[2], y[2], qf[2 * w][nt][0], qf[2 * w][nt][1]);
                            us::mma_m16n8k16_f16(so[nt], x[1], y[1], x[3], y[3], qf[2 * w + 1][nt][0], qf[2 * w + 1][nt][1]);
                        }
                    } else {
                        uint32_t x[2], y[2];
                        decode_i8(k0[w], x);
                        decode_i8(k1[w], y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            us::mma_m16n8k16_f16(w & 1 ? so[nt] : sa[nt], x[0], y[0], x[1], y[1], qf[w][nt][0], qf[w][nt][1]);
                    }
                }
                // ---- scores (elements 0, 1: token rt; 2, 3: token rt + 8), masks
                const uint32_t* ss = reinterpret_cast<const uint32_t*>(st + 2 * kStep * Sh::kRow) + sb * kBlock;
                const uint32_t s0 = ss[rt], s1 = ss[rt + 8];
                const float ks[2] = {us::half_bits_to_float((uint16_t)s0) * sc, us::half_bits_to_float((uint16_t)s1) * sc};
                vs[sb][0] = us::half_bits_to_float((uint16_t)(s0 >> 16));
                vs[sb][1] = us::half_bits_to_float((uint16_t)(s1 >> 16));
#pragma unroll
                for (int u = 0; u < 2; ++u) lv[sb][u] = fmaxf(lg2(fabsf(vs[sb][u])), -24.f);   // fp16's smallest, also for 0 and NaN
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sa[nt][e] = (sa[nt][e] + so[nt][e]) * ks[e >> 1];
                if (edge) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int j = ((blocks >> sb) & 1u) ? pos + sb * kBlock + rt + 8 * u - cur.r.ctx : cur.r.n;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int r = 8 * nt + 2 * c4 + e;
                                const bool seen = j < 0 || (j < cur.r.n && (p.mask ? (sm_mask[r] >> (j & 63)) & 1 : j <= sm_tok[r]));
                                if (!seen) sa[nt][2 * u + e] = -INFINITY;
                            }
                    }
                }
            }
            // ---- running maxima, rescaled only where one has grown by 2^4
            // (an unseen entry's scale may be anything: -inf and NaN move no maximum)
            bool grow = false;
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    mx[nt][e] = fmaxf(sx[0][nt][e] + lv[0][0], sx[0][nt][e + 2] + lv[0][1]);
                    if constexpr (kSub == 2) mx[nt][e] = max3(mx[nt][e], sx[1][nt][e] + lv[1][0], sx[1][nt][e + 2] + lv[1][1]);
                    grow |= mx[nt][e] > m[nt][e] + room;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = mx[nt][e];
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        x = fmaxf(x - (fabsf(x) < kFine ? kTop : 0.f), m[nt][e]);
                        if (x != -INFINITY && fabsf(x) >= kFine) room = 0.f;
                        const float f = x == -INFINITY ? 1.f : ex2(m[nt][e] - x);
                        m[nt][e] = x;
                        l[nt][e] *= f;
#pragma unroll
                        for (int t = 0; t < kMT; ++t) {
                            o[t][nt][e] *= f;
                            o[t][nt][e + 2] *= f;
                        }
                    }
            }
#pragma unroll
            for (int sb = 0; sb < kSub; ++sb) {
                // ---- weights; with V's scale, as fp16, they are the B operand of O^T
                uint32_t pf[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w[4], x[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float mm = m[nt][e & 1];
                        w[e] = ex2(sx[sb][nt][e] - (mm == -INFINITY ? 0.f : mm));
                        l[nt][e & 1] += w[e];
                        x[e] = w[e] * vs[sb][e >> 1];
                    }
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (sx[sb][nt][e] == -INFINITY) x[e] = 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < 2; ++u) pf[nt][u] = transpose8x8(pack_half2(x[2 * u], x[2 * u + 1]));
                }
                // ---- O^T += Cv^T P^T
                uint32_t v[4][kVW];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    lds_words(st + (kStep + sb * kBlock + c4 + 4 * i) * Sh::kRow + g * (4 * kVW), v[i]);
#pragma unroll
                for (int w = 0; w < kVW; ++w)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const uint32_t x01 = __byte_perm(v[0][w], v[1][w], hh ? 0x7632 : 0x5410);
                        const uint32_t x23 = __byte_perm(v[2][w], v[3][w], hh ? 0x7632 : 0x5410);
                        if constexpr (ELEM == US_I4) {
                            uint32_t a[4], b[4];
                            decode_i4(x01, a);
                            decode_i4(x23, b);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                us::mma_m16n8k16_f16(o[4 * w + 2 * hh][nt], a[0], a[1], b[0], b[1], pf[nt][0], pf[nt][1]);
                                us::mma_m16n8k16_f16(o[4 * w + 2 * hh + 1][nt], a[2], a[3], b[2], b[3], pf[nt][0], pf[nt][1]);
                            }
                        } else {
                            uint32_t a[2], b[2];
                            decode_i8(x01, a);
                            decode_i8(x23, b);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                us::mma_m16n8k16_f16(o[2 * w + hh][nt], a[0], a[1], b[0], b[1], pf[nt][0], pf[nt][1]);
                        }
                    }
            }
        }
        const bool ends = cur.tile + 1 == cur.tiles || it + 1 == count;
        __syncwarp();                                      // every lane has read the stage
        if (it + kStages < count) issue(s, it + kStages + 1 < count);
        cp_async_commit();
        s = s + 1 == kStages ? 0 : s + 1;

        // ---- the end of the segment, or of this CTA's part of it
        if (ends) {
            const int rows = min(kRows, cur.r.n * G - cur.rb * kRows);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float x = l[nt][e];
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                    if (g == 0) {
                        sm_m[warp * kRows + 8 * nt + 2 * c4 + e] = m[nt][e];
                        sm_l[warp * kRows + 8 * nt + 2 * c4 + e] = x;
                    }
                }
            __syncthreads();
            // segment [s0, s1) of the tile sequence, this CTA's part, who else has one
            const int64_t s0 = sh_work.t0 + it - cur.tile, s1 = s0 + cur.tiles;
            const Part part = sh_work.sharers(s0, s1, cur, rows);
            const bool whole = part.first == part.last;
            float* slot = p.ws_slots + part.slot(blockIdx.x) * Sh::kSlotFloats;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 8 * nt + 2 * c4 + e;
                    float t = sm_m[r];
#pragma unroll
                    for (int w = 1; w < kWarps; ++w) t = fmaxf(t, sm_m[w * kRows + r]);
                    const float f = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - t);
#pragma unroll
                    for (int q = 0; q < kMT; ++q) o[q][nt][e] *= f, o[q][nt][e + 2] *= f;
                }
            if (threadIdx.x < kRows) {                      // row maxima and sums over the warps
                const int r = threadIdx.x;
                float t = sm_m[r], sum = 0.f;
#pragma unroll
                for (int w = 1; w < kWarps; ++w) t = fmaxf(t, sm_m[w * kRows + r]);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float mw = sm_m[w * kRows + r];
                    sum += sm_l[w * kRows + r] * (mw == -INFINITY ? 0.f : ex2(mw - t));
                }
                sm_inv[r] = sum == 0.f ? 0.f : 1.f / sum;
                if (!whole) {
                    __stcg(slot + r, t);
                    __stcg(slot + kRows + r, sum);
                }
            }
            constexpr int kPer = 8 / NT;                    // 16-dimension blocks joined at a time
#pragma unroll
            for (int ch = 0; ch < (kMT + kPer - 1) / kPer; ++ch) {
                constexpr int kBlocks = kPer < kMT ? kPer : kMT;
                if (ch) __syncthreads();
#pragma unroll
                for (int q = 0; q < kBlocks; ++q)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            join[((warp * kBlocks + q) * NT + nt) * 128 + e * 32 + lane] = o[ch * kBlocks + q][nt][e];
                __syncthreads();
                // four neighbouring dimensions of a row at a time
#pragma unroll
                for (int x = threadIdx.x; x < kBlocks * NT * 32; x += kThreads) {
                    const int e = (x >> 5) & 1, nt = (x >> 6) % NT, q = 2 * ((x >> 6) / NT);
                    float y[4] = {};
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) {
                        const float* jw = join + ((w * kBlocks + q) * NT + nt) * 128 + e * 32 + lane;
                        y[0] += jw[0], y[1] += jw[64], y[2] += jw[128 * NT], y[3] += jw[128 * NT + 64];
                    }
                    const int r = 8 * nt + 2 * c4 + e;
                    if (whole) {
                        if (r < rows) {
                            const float inv = sm_inv[r];
                            uint16_t* out = out_row<kRows>(p, cur.r.row0, cur.h, cur.rb, r, D) + g * (D / 8) + 2 * (ch * kBlocks + q);
                            *reinterpret_cast<uint2*>(out) =
                                make_uint2(pack_out(y[0] * inv, y[1] * inv), pack_out(y[2] * inv, y[3] * inv));
                        }
                    } else {
                        __stcg(reinterpret_cast<float4*>(slot + 2 * kRows) + ch * kBlocks * NT * 32 + x,
                               make_float4(y[0], y[1], y[2], y[3]));
                    }
                }
            }
            if (!whole) {                                  // joined after the loop, which needs the registers
                if (threadIdx.x == 0) sh_part[parts] = part;
                ++parts;
            }
            if (it + 1 < count) {
                cur.next(p);
                begin_segment();                           // its barrier also frees the join buffer
            }
        } else {
            ++cur.tile;
        }
    }
    // ---- shared segments (at most two a CTA): the last CTA to arrive joins them
    for (int i = 0; i < parts; ++i) {
        __syncthreads();
        const Part a = sh_part[i];
        if (threadIdx.x == 0) {                            // one thread's fences order the whole CTA's accesses
            __threadfence();
            sh_last = atomicAdd(p.ws_count + a.first, 1u) == (unsigned)(a.last - a.first);
            __threadfence();
        }
        __syncthreads();
        if (!sh_last) continue;
        if (threadIdx.x == 0) p.ws_count[a.first] = 0;
        join_states<ELEM, D, NT, W>(p, join, sm_inv, a);
    }
    us::pdl_launch_dependents();
}

template <int ELEM, int D, int NT, int W>
struct Plan {
    using Sh = Shape<ELEM, D, NT, W>;
    static int grid() { return us::num_sms() * Sh::kMinB < 1024 ? us::num_sms() * Sh::kMinB : 1024; }
    static size_t ws() { return 4096 + (size_t)2 * grid() * Sh::kSlotFloats * 4; }
    static us_status launch(UsAttnParams p, cudaStream_t st) {
        p.ws_count = static_cast<unsigned*>(p.ws);
        p.ws_slots = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + 4096);
        auto kern = attn_mma_kernel<ELEM, D, NT, W>;
        static std::atomic<bool> ready[64];            // the attribute is set once a device, by whichever thread
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return US_ERR_CUDA;
        if (!ready[dev].load(std::memory_order_acquire)) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::kSmem) != cudaSuccess)
                return US_ERR_CUDA;
            ready[dev].store(true, std::memory_order_release);
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)grid());
        cfg.blockDim = dim3(Sh::kThreads);
        cfg.dynamicSmemBytes = Sh::kSmem;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? US_OK : US_ERR_CUDA;
    }
};

// f(Plan) for the cache's type and head width and the rows per key head.  Eight
// warps a CTA, two CTAs an SM, for up to 8 rows: on 48 requests of 4096 to 8192
// positions in int4 83 us (97 with two CTAs of four warps and twice the positions a
// step), on one token of two requests of 131000 77 (78), on one of 777 9.0 (9.1).
template <class F>
auto with_plan(const UsAttnParams& p, F f) {
    const int rows = p.a.max_n * p.G;
#define US_ATTN_PICK(E, D) (rows <= 8 ? f(Plan<E, D, 1, 8>()) : f(Plan<E, D, 2, 4>()))
    if (p.c.D == 64 && rows > 16) return p.c.elem == US_I8 ? f(Plan<US_I8, 64, 4, 4>()) : f(Plan<US_I4, 64, 4, 4>());
    if (p.c.elem == US_I8) return p.c.D == 64 ? US_ATTN_PICK(US_I8, 64) : US_ATTN_PICK(US_I8, 128);
    return p.c.D == 64 ? US_ATTN_PICK(US_I4, 64) : US_ATTN_PICK(US_I4, 128);
#undef US_ATTN_PICK
}

}  // namespace

namespace us {

size_t attn_ws(const UsAttnParams& p) {
    if (attn_tc_serves(p)) return attn_tc_ws(p);
    return with_plan(p, [](auto plan) { return decltype(plan)::ws(); });
}

us_status launch_attn(const UsAttnParams& p, cudaStream_t st) {
    if (attn_tc_serves(p)) return launch_attn_tc(p, st);
    return with_plan(p, [&](auto plan) { return decltype(plan)::launch(p, st); });
}

}  // namespace us

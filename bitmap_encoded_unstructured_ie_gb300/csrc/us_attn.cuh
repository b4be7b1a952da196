// us_attn.cuh -- what the attention kernels share: the even partition of the
// (request, key head, row block, tile) sequence over the CTAs, and the codes as
// fp16 pairs.
#pragma once

#include "us_kv.cuh"

namespace us {
namespace attn {

// Waits for phase `parity` of `bar`, at most kWaitLimitNs (then US_ERR_TIMEOUT is
// recorded).  A try, a sleep of some 20 ns, a try: try_wait alone comes back at once
// and its loop took most of the issue slots; with a time hint it woke warps late.
US_DEV bool wait_bar(uint64_t* bar, uint32_t parity, unsigned* status) {
    if (us::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = us::globaltimer_ns();
    for (;;) {
#pragma unroll 1
        for (int n = 0; n < 64; ++n) {
            __nanosleep(20);
            if (us::mbar_try_wait(bar, parity)) return true;
        }
        if (us::globaltimer_ns() - t0 > us::kWaitLimitNs) break;
    }
    us::set_status(status, US_ERR_TIMEOUT);
    return false;
}

US_DEV void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
US_DEV void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
US_DEV void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
US_DEV void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Scores from here on lie 2^-4 and more apart.  A reference that is less than the largest
// score by a few powers of two would be rounded to where a weight is beyond fp16 (2^16),
// so there the largest score itself is the reference.
constexpr float kFine = 0x1p19f;

US_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
US_DEV float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// two fp32 operations in one instruction
US_DEV uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
US_DEV void unpair(uint64_t x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x)); }
US_DEV uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
US_DEV uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
US_DEV uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
US_DEV float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
US_DEV uint32_t hsub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
US_DEV uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
US_DEV uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b), *reinterpret_cast<__half2*>(&c));
    return *reinterpret_cast<const uint32_t*>(&r);
}
US_DEV uint32_t pack_half2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Outputs, at most 65504 in magnitude (entries of the largest values stand for up to 65532).
US_DEV uint32_t pack_out(float lo, float hi) { return us::saturate_half2(pack_half2(lo, hi)); }
// Both halves of a word of codes as exact fp16 pairs: 0x6400 | u is the fp16
// number 1024 + u, and flipping a code's sign bit makes it u = code + 8 (+ 128).
// int4: nibbles (0, 4), (1, 5), (2, 6), (3, 7); int8: bytes (0, 2), (1, 3).
US_DEV void decode_i4(uint32_t x, uint32_t (&q)[4]) {
    const uint32_t y = x >> 8;
    q[0] = hsub2(us::lop3<us::kLopAndXor>(x, 0x000F000Fu, 0x64086408u), 0x64086408u);
    q[1] = hfma2(us::lop3<us::kLopAndXor>(x, 0x00F000F0u, 0x64806480u), 0x2C002C00u, 0xD480D480u);   // x/16 - 72
    q[2] = hsub2(us::lop3<us::kLopAndXor>(y, 0x000F000Fu, 0x64086408u), 0x64086408u);
    q[3] = hfma2(us::lop3<us::kLopAndXor>(y, 0x00F000F0u, 0x64806480u), 0x2C002C00u, 0xD480D480u);
}
US_DEV void decode_i8(uint32_t x, uint32_t (&q)[2]) {
    q[0] = hsub2(us::lop3<us::kLopAndXor>(x, 0x00FF00FFu, 0x64806480u), 0x64806480u);
    q[1] = hsub2(us::lop3<us::kLopAndXor>(x >> 8, 0x00FF00FFu, 0x64806480u), 0x64806480u);
}

// a / b, in 32 bits where that does
US_DEV int64_t quotient(int64_t a, int64_t b) {
    return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// A request's tokens, context and row blocks; none where its arguments are not
// usable.
struct Request {
    int row0, n, ctx, nrb;
};

// Tiles that row block rb of ROWS rows reads: a chain's rows see no position
// behind their own.
template <int ROWS, int TILE, class P>
US_DEV int tiles_of(const P& p, const Request& r, int rb) {
    unsigned end = (unsigned)r.n;
    if (!p.mask && rb + 1 < r.nrb) end = (unsigned)((rb + 1) * ROWS - 1) / (unsigned)p.G + 1u;   // n G < 2^30
    return (int)(((unsigned)r.ctx + end + TILE - 1u) / TILE);
}

// The request whose tokens are rows o0 .. o1 - 1, with `ctx` positions before them.
template <int ROWS, class P>
US_DEV Request make_request(const P& p, int o0, int o1, int ctx, unsigned* status) {
    Request r = {o0, us::kv_row_count(p.a, o0, o1, status), 0, 0};
    if (r.n > 0) {
        r.ctx = us::kv_context(p.c, ctx, r.n, status);
        if (r.ctx >= 0) r.nrb = (int)((unsigned)(r.n * p.G + ROWS - 1) / ROWS);
    } else if (P::kOffsets && ctx < 0) {
        us::set_status(status, US_ERR_INVALID_ARG);        // (positions of no token are not looked at, offsets are)
    }
    return r;
}
template <int ROWS, class P>
US_DEV Request load_request(const P& p, int b, unsigned* status) {
    const int o0 = p.a.off[b], o1 = p.a.off[b + 1];
    return make_request<ROWS>(p, o0, o1, p.context(b, o0, o1), status);
}

// Tiles of one key head of a request.  A chain's row blocks are walked without
// dividing: the tokens of (rb + 1) ROWS rows from those of rb ROWS.
template <int ROWS, int TILE, class P>
US_DEV int64_t head_tiles(const P& p, const Request& r) {
    if (r.nrb == 0) return 0;
    const unsigned last = ((unsigned)r.ctx + (unsigned)r.n + TILE - 1u) / TILE;
    if (p.mask) return (int64_t)r.nrb * last;
    int64_t sum = last;
    if (r.nrb > 1) {
        const unsigned G = (unsigned)p.G, q = ROWS / G, m = ROWS % G;
        for (unsigned rb = 1, end = 0, over = 0; rb < (unsigned)r.nrb; ++rb) {
            end += q, over += m;
            if (over >= G) over -= G, ++end;
            sum += ((unsigned)r.ctx + end + (over ? 1u : 0u) + TILE - 1u) / TILE;
        }
    }
    return sum;
}

// A place in the tile sequence.
template <int ROWS, int TILE>
struct Cursor {
    Request r;
    int b, h, rb, tile, tiles;                             // tiles: of this row block
    template <class P>
    US_DEV void next(const P& p) {
        if (++tile < tiles) return;
        tile = 0;
        if (++rb == r.nrb) {
            rb = 0;
            if (++h == p.c.Hkv) {
                h = 0;
                do {
                    ++b;
                    if (b < p.c.B) r = load_request<ROWS>(p, b, nullptr);
                } while (b < p.c.B && r.nrb == 0);
                if (b == p.c.B) return;
            }
        }
        tiles = tiles_of<ROWS, TILE>(p, r, rb);
    }
    // to the row block behind this one
    template <class P>
    US_DEV void next_segment(const P& p) {
        tile = tiles - 1;
        next(p);
    }
};

// A segment (request, key head, row block) shared by CTAs first .. last; second:
// the first of them leaves its state in its second slot, because its part is not
// the first thing it does.
struct Part {
    int first, last, row0, h, rb, rows;
    bool second;
    US_DEV int64_t slot(int cta) const { return (int64_t)2 * cta + (cta == first && second ? 1 : 0); }
};

// A CTA's share [t0, t1) of the sequence of tiles: `per` tiles a CTA, one more for
// the first `extra` of them.
struct Work {
    int64_t t0, t1, per;
    int extra;
    US_DEV int64_t begin(int cta) const { return cta * per + min(cta, extra); }
    US_DEV int owner(int64_t t) const {
        const int64_t rest = t - extra * (per + 1);
        return rest < 0 ? (int)quotient(t, per + 1) : extra + (int)quotient(rest, per);
    }
    template <class C>
    US_DEV Part sharers(int64_t s0, int64_t s1, const C& at, int rows) const {
        Part a;
        a.first = owner(s0);
        a.last = owner(s1 - 1);
        a.second = s0 > begin(a.first);
        a.row0 = at.r.row0, a.h = at.h, a.rb = at.rb, a.rows = rows;
        return a;
    }
};

// The share of this CTA and where it begins; false if there is none for it.  Each
// warp finds it for itself, without a barrier: a lane adds up the tiles of B / 32
// requests, a scan over the lanes finds the one with the share's first tile (4500
// cycles by a scan over the block with 64-bit divisions, at 16 row blocks of a chain
// 15000).
template <int ROWS, int TILE, class P>
US_DEV bool find_work(const P& p, Work& w, Cursor<ROWS, TILE>& at) {
    const int lane = threadIdx.x & 31;
    unsigned* status = blockIdx.x == 0 && threadIdx.x < 32 ? p.c.status : nullptr;
    const int each = (p.c.B + 31) / 32, b0 = lane * each, b1 = min(b0 + each, p.c.B);
    int64_t mine = 0, head = 0;
    Request r = {0, 0, 0, 0};
    for (int b = b0; b < b1; b += 4) {                     // four requests' loads at once
        int off[5], pos[4];
#pragma unroll
        for (int u = 0; u < 5; ++u) off[u] = b + u <= b1 ? p.a.off[b + u] : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) pos[u] = b + u < b1 ? p.context(b + u, off[u], off[u + 1]) : 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (b + u >= b1) break;
            r = make_request<ROWS>(p, off[u], off[u + 1], pos[u], status);
            head = head_tiles<ROWS, TILE>(p, r);
            mine += head * p.c.Hkv;
        }
    }
    int64_t incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    const int ctas = total < (int64_t)gridDim.x ? (int)total : (int)gridDim.x;
    if ((int)blockIdx.x >= ctas) return false;
    w.per = quotient(total, ctas);
    w.extra = (int)(total - w.per * ctas);
    w.t0 = w.begin(blockIdx.x), w.t1 = w.begin(blockIdx.x + 1);
    int64_t x = w.t0 - (incl - mine);
    const bool here = x >= 0 && x < mine;
    int b = b0;
    if (here && each > 1) {
        for (;; ++b) {
            r = load_request<ROWS>(p, b, nullptr);
            head = head_tiles<ROWS, TILE>(p, r);
            if (x < head * p.c.Hkv) break;
            x -= head * p.c.Hkv;
        }
    }
    const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
    at.b = __shfl_sync(0xffffffffu, b, src);
    at.r.row0 = __shfl_sync(0xffffffffu, r.row0, src);
    at.r.n = __shfl_sync(0xffffffffu, r.n, src);
    at.r.ctx = __shfl_sync(0xffffffffu, r.ctx, src);
    at.r.nrb = __shfl_sync(0xffffffffu, r.nrb, src);
    x = __shfl_sync(0xffffffffu, x, src);
    head = __shfl_sync(0xffffffffu, head, src);
    at.h = 0;
    if (x >= head) at.h = (int)quotient(x, head), x -= at.h * head;
    at.rb = 0;
    at.tiles = tiles_of<ROWS, TILE>(p, at.r, 0);
    if (p.mask) {
        if (x >= at.tiles) at.rb = (int)quotient(x, at.tiles), x -= (int64_t)at.rb * at.tiles;
    } else {
        while (x >= at.tiles) {
            x -= at.tiles;
            at.tiles = tiles_of<ROWS, TILE>(p, at.r, ++at.rb);
        }
    }
    at.tile = (int)x;
    return true;
}

// Where a row's fp16 outputs go: D values at row r of row block rb, head h.
template <int ROWS, class P>
US_DEV uint16_t* out_row(const P& p, int row0, int h, int rb, int r, int D) {
    const int rr = rb * ROWS + r, i = rr / p.G;
    return p.O + (int64_t)(row0 + i) * p.ldo + (int64_t)(h * p.G + rr - i * p.G) * D;
}

}  // namespace attn
}  // namespace us

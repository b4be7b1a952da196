// us_kv.cuh -- the paged, quantised key/value cache as the kernels see it.
//
// A cache entry is one (position, key head): D codes of K, D codes of V (int8,
// or int4 two per byte, even element in the low nibble) and a pair of fp16
// scales.  Position p of request b lies in page table[b][p / page_size], slot
// p % page_size; the entries of one page and head are contiguous.
#pragma once

#include "us_common.cuh"

struct UsKvCache {
    int elem, D, Hkv, page_shift, num_pages, B, max_pages, row_bytes;
    uint8_t* k;
    uint8_t* v;
    uint16_t* scale;                 // (K scale, V scale) per entry
    const int32_t* table;
    unsigned* status;
};

// The tokens of one call: request b owns rows off[b] .. off[b+1]-1 and, unless
// stated otherwise, positions pos[b] .. of the cache.
struct UsKvCall {
    const int32_t* off;
    const int32_t* pos;
    int T, max_n;
};

namespace us {
namespace attn {
struct Part;
}
}  // namespace us

// Attention over the cache: Q and O token-major rows of Hq heads.
struct UsAttnParams {
    UsKvCache c;
    UsKvCall a;
    const uint16_t* Q;
    uint16_t* O;
    int64_t ldq, ldo;
    int Hq, G;                       // G = Hq / Hkv
    float scale;
    const uint64_t* mask;            // per token, or nullptr: a chain
    void* ws;
    unsigned* ws_count;              // arrival counters, zero between calls
    float* ws_slots;                 // partial states
    us::attn::Part* ws_parts;        // shared segments
};

namespace us {

// Rows of request b: first row and count (0 if the offsets are not usable).
US_DEV int kv_row_count(const UsKvCall& a, int o0, int o1, unsigned* status) {
    if (o0 >= 0 && o1 >= o0 && o1 <= a.T && o1 - o0 <= a.max_n) return o1 - o0;
    set_status(status, US_ERR_INVALID_ARG);
    return 0;
}
US_DEV int kv_rows(const UsKvCall& a, int b, int& row0, unsigned* status) {
    row0 = a.off[b];
    return kv_row_count(a, row0, a.off[b + 1], status);
}

// Page of position p of request b, or -1 (recorded) if there is none.
US_DEV int kv_page(const UsKvCache& c, int b, int p) {
    const int i = p >> c.page_shift;
    if (p < 0 || i >= c.max_pages) {
        set_status(c.status, US_ERR_INVALID_ARG);
        return -1;
    }
    const int id = c.table[(int64_t)b * c.max_pages + i];
    if (id >= 0 && id < c.num_pages) return id;
    set_status(c.status, US_ERR_CORRUPT);
    return -1;
}

// Index of the entry of head h at slot p % page_size of page `id`.
US_DEV int64_t kv_entry(const UsKvCache& c, int id, int h, int p) {
    return ((((int64_t)id * c.Hkv + h) << c.page_shift)) + (p & ((1 << c.page_shift) - 1));
}

// base + i for positions: wraps negative instead of overflowing (kv_page refuses it)
US_DEV int kv_pos(int base, int i) { return (int)((unsigned)base + (unsigned)i); }

// fp16 pairs at most 65504 in magnitude; NaN stays.
US_DEV uint32_t saturate_half2(uint32_t x) {
    const uint32_t hi = 0x7BFF7BFFu, lo = 0xFBFFFBFFu;
    const __half2 r = __hmin2_nan(__hmax2_nan(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&lo)),
                                  *reinterpret_cast<const __half2*>(&hi));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// ctx if the page table's row can hold n positions behind it, else -1 (recorded).
US_DEV int kv_context(const UsKvCache& c, int ctx, int n, unsigned* status) {
    if (ctx >= 0 && ctx <= ((int64_t)c.max_pages << c.page_shift) - n) return ctx;
    set_status(status, US_ERR_INVALID_ARG);
    return -1;
}

}  // namespace us

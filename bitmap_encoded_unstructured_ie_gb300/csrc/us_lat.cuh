// us_lat.cuh -- the paged cache of latent rows as the kernels see it.
#pragma once

#include "us_kv.cuh"

struct UsLatCache {
    UsKvCache c;                     // pages and table alone
    int Dc, W;                       // W = Dc + Dr values a row
    uint16_t* rows;
};

namespace us {

constexpr int kLatDr = 64;

// First value of position p of request b, or -1 (recorded).
US_DEV int64_t lat_row(const UsLatCache& L, int b, int p) {
    const int id = kv_page(L.c, b, p);
    return id < 0 ? -1 : (((int64_t)id << L.c.page_shift) + (p & ((1 << L.c.page_shift) - 1))) * L.W;
}

}  // namespace us

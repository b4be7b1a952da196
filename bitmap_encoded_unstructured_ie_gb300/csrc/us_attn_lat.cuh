// us_attn_lat.cuh -- parameters of the attention over latent rows and over expanded
// rows, and the join of the states that several CTAs hold of one segment.
#pragma once

#include "us_attn.cuh"
#include "us_lat.cuh"

// Of the base: c has the pages and one key head, G = Hq.
struct UsAttnLatParams : UsAttnParams {
    const uint16_t* rows;
    int Dc, W;
};

struct UsAttnRowsParams {
    us_attn_kv_rows k;
    const uint16_t* Q;
    uint16_t* O;
    int64_t ldq, ldo;
    int B, T, max_n;
    const int32_t* off;
    const int32_t* kv_off;
    float scale;
    void* ws;
    unsigned* status;
};

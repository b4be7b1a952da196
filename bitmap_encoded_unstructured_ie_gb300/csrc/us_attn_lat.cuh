// us_attn_lat.cuh -- parameters of the attention over latent rows and over expanded rows.
#pragma once

#include "us_lat.cuh"

struct UsAttnLatParams {
    UsLatCache L;
    UsKvCall a;
    const uint16_t* Q;
    uint16_t* O;
    int64_t ldq, ldo;
    int Hq;
    float scale;
    const uint64_t* mask;            // per token, or nullptr: a chain
    void* ws;
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

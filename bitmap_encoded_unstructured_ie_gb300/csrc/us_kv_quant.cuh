// us_kv_quant.cuh -- quantising one row of the K/V cache: shared by us_kv_write and by
// us_kv_append, whose entries are the same bits.
#pragma once

#include "us_kv.cuh"

namespace us {

// x as eight fp32 values, infinities at the largest fp16 value, NaN as 0
US_DEV void unpack8(uint4 w, float (&x)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float f = us::half_bits_to_float((uint16_t)(u[i >> 1] >> (16 * (i & 1))));
        x[i] = f == f ? fminf(fmaxf(f, -65504.f), 65504.f) : 0.f;
    }
}

// Eight codes (as fp32 whole numbers plus 1.5 2^23, whose low bits they are) -> bytes or nibbles.
template <int ELEM>
US_DEV uint2 pack_codes(const float (&v)[8]) {
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(v[i]);
    if constexpr (ELEM == US_I8) {
        return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    } else {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) w |= (b[i] & 0xFu) << (4 * i);
        return make_uint2(w, 0u);
    }
}

// Quantises one row held N times eight values a lane by D / (8 N) neighbouring lanes (all
// 32 lanes of the warp take part); returns the scale.
//
// rint(x / s) without a division: q = x (1/s), corrected once by its exact
// remainder.  x and s have 11 bits, so x / s is either exactly a half-way point
// k + 1/2, which has few bits and is what the correction then arrives at, or at
// least 2^-20 of itself away from one, where an error of 2^-22 does not matter.
// Rows with infinities, NaN or a subnormal scale (whose codes may need the clamp)
// take the plain way.
template <int ELEM, int D, int N>
US_DEV uint16_t quantise_row(const uint4 (&in)[N], uint2 (&codes)[N]) {
    constexpr float q = ELEM == US_I8 ? 127.f : 7.f, kRound = 12582912.f;
    auto h2 = [](uint32_t x) { return *reinterpret_cast<const __half2*>(&x); };
    __half2 m2 = h2(in[0].x & 0x7FFF7FFFu);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const uint32_t u[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
#pragma unroll
        for (int i = k ? 0 : 1; i < 4; ++i) m2 = __hmax2_nan(m2, h2(u[i] & 0x7FFF7FFFu));
    }
#pragma unroll
    for (int d = D / (16 * N); d > 0; d >>= 1) m2 = __hmax2_nan(m2, __shfl_xor_sync(0xffffffffu, m2, d));
    const __half m = __hmax_nan(__low2half(m2), __high2half(m2));
    float amax = __half2float(m);
    uint16_t s16 = us::float_to_half_bits(amax / q);
    if (__any_sync(0xffffffffu, !(amax <= 65504.f) || (s16 < 0x0400u && s16 != 0u))) {
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float v[8];
            unpack8(in[k], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
        }
#pragma unroll
        for (int d = D / (16 * N); d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        s16 = us::float_to_half_bits(amax / q);
        if (s16 == 0) s16 = 0x3C00u;                          // 1.0
        const float s = us::half_bits_to_float(s16);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            float v[8];
            unpack8(in[k], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(rintf(v[i] / s), -q - 1.f), q) + kRound;
            codes[k] = pack_codes<ELEM>(v);
        }
    } else {
        if (s16 == 0) s16 = 0x3C00u;
        const float s = us::half_bits_to_float(s16), inv = 1.f / s;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const uint32_t u[4] = {in[k].x, in[k].y, in[k].z, in[k].w};
            float v[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = __half22float2(h2(u[i]));
                const float a = x.x * inv, b = x.y * inv;
                v[2 * i] = fmaf(fmaf(-a, s, x.x), inv, a) + kRound;
                v[2 * i + 1] = fmaf(fmaf(-b, s, x.y), inv, b) + kRound;
            }
            codes[k] = pack_codes<ELEM>(v);
        }
    }
    return s16;
}
template <int ELEM, int D>
US_DEV uint16_t quantise_row(uint4 in, uint2& codes) {
    const uint4 x[1] = {in};
    uint2 c[1];
    const uint16_t s = quantise_row<ELEM, D, 1>(x, c);
    codes = c[0];
    return s;
}

template <int ELEM>
US_DEV void store_codes(uint8_t* dst, uint2 w) {
    if constexpr (ELEM == US_I8) *reinterpret_cast<uint2*>(dst) = w;
    else *reinterpret_cast<uint32_t*>(dst) = w.x;
}

}  // namespace us

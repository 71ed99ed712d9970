// int8_code.h -- the scale and the multiplier of a row of int8 codes: plain
// arithmetic on the row's largest magnitude, compiled for the device by the row
// quantisers and for the host by the CPU tests.
#pragma once

#include <cmath>
#include <cstdint>
#include <cstring>

#ifdef __CUDACC__
#define MOE_CODE_HD __host__ __device__
#else
#define MOE_CODE_HD
#endif

namespace moe {

// scale: what a code of 1 stands for; inv: what a value is multiplied by.
struct Int8Scale {
    float scale, inv;
};

MOE_CODE_HD inline float float_of_bits(uint32_t u)
{
    float f;
    memcpy(&f, &u, sizeof f);
    return f;
}

MOE_CODE_HD inline uint32_t bits_of_float(float f)
{
    uint32_t u;
    memcpy(&u, &f, sizeof u);
    return u;
}

// scale = amax / 127 rounded to fp32; code = round(v * inv) to even, which has to be
// that of v * 127 / amax.  Of bf16 values the only tie of that is 63.5, at half the
// largest magnitude; every other value is further from one than the roundings of inv
// and of the product reach.  So inv is 127 / amax rounded up, not to nearest: the
// product at the tie is then 63.5 or a little above, and rounds to 64 (rounded to
// nearest, inv is too small for 14 of the 128 mantissas of amax).  The largest
// magnitude itself gives at most 127 (1 + 2^-22), code 127.
// A row whose largest magnitude is below 2^-100 counts as all zero (scale 1,
// codes 0): amax / 127 and 127 / amax are then both normal fp32 numbers.  A row
// that holds a NaN or an infinity gets the scale NaN, so that it stays visible
// in every product made of it.
MOE_CODE_HD inline Int8Scale int8_scale(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F800000u) return {float_of_bits(0x7FC00000u), 0.f};
    const float amax = float_of_bits(amax_bits);
    if (amax < 7.888609052210118e-31f) return {1.f, 0.f};   // 2^-100
    float inv = 127.f / amax;
    if (fmaf(inv, amax, -127.f) < 0.f) inv = float_of_bits(bits_of_float(inv) + 1u);   // one rounding: the sign is exact
    return {amax / 127.f, inv};
}

}  // namespace moe

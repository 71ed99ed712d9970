// Host harness for the CPU test of the int8 codes' scale: compiles
// grouped_gemm_02_b200/csrc/int8_code.h (what the row quantisers call).
#include "../grouped_gemm_02_b200/csrc/int8_code.h"

// scale, inv and the codes of n values of a row with this largest magnitude
extern "C" void int8_codes_of(float amax, const float* v, int n, float* scale, float* inv, int* codes)
{
    uint32_t bits;
    memcpy(&bits, &amax, sizeof bits);
    const moe::Int8Scale s = moe::int8_scale(bits);
    *scale = s.scale;
    *inv = s.inv;
    for (int i = 0; i < n; i++) codes[i] = (int)nearbyintf(v[i] * s.inv);
}

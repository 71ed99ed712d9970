// Host harness for the CPU test of how a dense int8 product is cut: compiles
// grouped_gemm_02_b200/csrc/int8_shape.h (what the entry point calls).
#include "../grouped_gemm_02_b200/csrc/int8_shape.h"

// out: form, chunk, units, split, tiles
extern "C" void int8_shape_of(int64_t T, int64_t K, int64_t N, int sms, int can_pair, int pairs, int64_t* out)
{
    const moe::Int8Shape s = moe::i8_shape(T, K, N, sms, can_pair != 0, pairs);
    out[0] = s.form;
    out[1] = s.chunk;
    out[2] = s.units;
    out[3] = s.split;
    out[4] = s.tiles;
}

extern "C" int int8_grouped_pair_of(int64_t P, int64_t K, int64_t N, int64_t E, int sms, int can_pair, int pairs)
{
    return moe::i8_grouped_pair(P, K, N, E, sms, can_pair != 0, pairs) ? 1 : 0;
}

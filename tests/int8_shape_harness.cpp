// Host harness for the CPU test of how a dense int8 product is cut: compiles
// grouped_gemm_02_b200/csrc/int8_shape.h (what the entry point calls).
#include "../grouped_gemm_02_b200/csrc/int8_shape.h"

static moe::Int8Device device(int sms, int can_pair, const int* clusters)
{
    moe::Int8Device d;
    d.sms = sms;
    d.pairs = can_pair ? sms / 2 : 0;
    for (int i = 2; i <= moe::kI8MaxSplit; i++) d.clusters[i] = clusters[i];
    return d;
}

// clusters: of 0 .. kI8MaxSplit CTAs that fit at once.  out: form, chunk, units, split, tiles
extern "C" void int8_shape_of(int64_t T, int64_t K, int64_t N, int sms, int can_pair, const int* clusters, int pairs,
                              int64_t* out)
{
    const moe::Int8Shape s = moe::i8_shape(T, K, N, device(sms, can_pair, clusters), pairs);
    out[0] = s.form;
    out[1] = s.chunk;
    out[2] = s.units;
    out[3] = s.split;
    out[4] = s.tiles;
}

extern "C" int int8_grouped_pair_of(int64_t P, int64_t K, int64_t N, int64_t E, int sms, int can_pair, int pairs)
{
    const int none[moe::kI8MaxSplit + 1] = {};
    return moe::i8_grouped_pair(P, K, N, E, device(sms, can_pair, none), pairs) ? 1 : 0;
}

// int8_shape.h -- how a dense int8 product is cut: the form of the kernel, the
// rows of a tile and the CTAs that share a tile's K range.  Plain arithmetic on
// the sizes, compiled for the host by the entry point and by the CPU tests.
#pragma once

#include <cstdint>

namespace moe {

constexpr int I8_SINGLE = 0, I8_PAIR = 1, I8_SPLIT = 2;
constexpr int kI8BlockK = 128;                   // codes per K block

struct Int8Shape {
    int form, chunk, units, split;
    int64_t tiles;          // of 128 channels (I8_PAIR: 256) and `chunk` rows
};

// Nanoseconds of a product cut this way, up to a constant (launch and start-up).
// A tile streams K/128 blocks; a block costs the larger of its bytes at what one
// SM draws from L2 (119 bytes/ns alone, 13400 for all SMs together) and its MMAs
// (1.5 ns a column); a tile costs 170 ns more and 15 ns a column of epilogue.
// Pairs start 2.5 us later; joining a split tile costs 2.7 us on 2 CTAs, 1.6 on 4
// and 8, and 10 ns a column.  The constants were fitted to 2,000 timings on a
// B200 (T 1..4096, K 512..16384, N 512..7168, every form and row count); the cut
// with the smallest cost is then within 1% of the fastest one measured in the
// geometric mean, and within 15% for every size.  A fixed rule (256 rows a tile)
// is up to 1.8 times slower where few tiles would leave SMs idle: T=256 K=7168
// N=2048 23.6 us against 13.8.
inline double i8_cost(int64_t T, int64_t K, int64_t N, int sms, int form, int chunk, int split)
{
    const int64_t units = (T + chunk - 1) / chunk;
    const int64_t tiles = (N + (form == I8_PAIR ? 255 : 127)) / (form == I8_PAIR ? 256 : 128) * units;
    const int64_t ctas = tiles * (form == I8_PAIR ? 2 : split);
    const int64_t slots = sms > 0 ? sms : 1;
    const double waves = (double)((ctas + slots - 1) / slots);
    const double blocks = (double)((K + kI8BlockK - 1) / kI8BlockK) / split;
    const double bytes = (128.0 + (form == I8_PAIR ? chunk / 2 : chunk)) * 128.0;
    const double all = 13400.0 / (double)(ctas < slots ? ctas : slots);
    const double load = bytes / (all < 119.0 ? all : 119.0), mma = 1.5 * chunk;
    double t = waves * (blocks * (load > mma ? load : mma) + 170.0) + 15.0 * chunk;
    if (form == I8_PAIR) t += 2500.0;
    if (form == I8_SPLIT) t += (split == 2 ? 2700.0 : 1600.0) + 10.0 * chunk;
    return t;
}

// The cheapest cut.  Rows a tile: a multiple of 16 (I8_PAIR: 32), at most 256.
// pairs: -1 the rule, 0 no CTA pairs, 1 pairs only (when the device runs them).
// Eight CTAs share a tile only while half the SMs hold all clusters: clusters of
// eight pack badly (16 of them did not fit a B200 at once: 13.0 us against 7.6
// with four CTAs a tile at T=1 K=7168 N=2048).
inline Int8Shape i8_shape(int64_t T, int64_t K, int64_t N, int sms, bool can_pair, int pairs)
{
    static const int kRows[] = {16, 32, 48, 64, 96, 128, 160, 192, 224, 256};
    const int64_t nk = (K + kI8BlockK - 1) / kI8BlockK;
    Int8Shape best{I8_SINGLE, 256, 0, 1, 0};
    double least = -1.0;
    for (int c : kRows) {
        const int64_t units = (T + c - 1) / c;
        for (int f = 0; f < 5; f++) {
            const int form = f == 0 ? I8_SINGLE : f == 1 ? I8_PAIR : I8_SPLIT, split = f < 2 ? 1 : 1 << (f - 1);
            const int64_t tiles = (N + (form == I8_PAIR ? 255 : 127)) / (form == I8_PAIR ? 256 : 128) * units;
            if (tiles >= (int64_t(1) << 30)) continue;
            if (form == I8_PAIR ? (!can_pair || pairs == 0 || c % 32 != 0) : (can_pair && pairs == 1)) continue;
            if (form == I8_SPLIT && (split > nk || tiles * split > (split == 8 ? sms / 2 : sms))) continue;
            const double t = i8_cost(T, K, N, sms, form, c, split);
            if (least < 0.0 || t < least) {
                least = t;
                best = Int8Shape{form, c, (int)units, split, tiles};
            }
        }
        if (c >= T && c >= 32) break;   // wider tiles would hold the same rows
    }
    return best;
}

// Whether a grouped product of P rows over E experts runs on CTA pairs.  The host
// knows the mean segment only; the rows of a tile are chosen on the device.  Pairs
// run where they are at least a fifth cheaper by i8_cost and the experts' weights,
// at 6500 bytes/ns, do not take longer than the single CTAs' work.  Measured on
// K = N = 2048, single CTAs against pairs: 64 experts with 4 rows each 42.5 and
// 44.2 us, 128 rows 67 and 67, 256 rows 95 and 87, 512 rows 166 and 154; 16
// experts with 512 rows at K = N = 1024 20.8 and 23.2 (the estimate: 4% cheaper).
inline bool i8_grouped_pair(int64_t P, int64_t K, int64_t N, int64_t E, int sms, bool can_pair, int pairs)
{
    if (!can_pair) return false;
    if (pairs >= 0) return pairs == 1;
    const int64_t blocks = P < E ? P : E, rows = (P + E - 1) / E;
    const int chunk = rows >= 256 ? 256 : (int)((rows + 31) / 32 * 32);
    // the mean segments end to end, as one dense product of whole tiles
    const int64_t T = blocks * ((rows + chunk - 1) / chunk) * chunk;
    const double single = i8_cost(T, K, N, sms, I8_SINGLE, chunk, 1), pair = i8_cost(T, K, N, sms, I8_PAIR, chunk, 1);
    return pair < 0.8 * single && (double)blocks * (double)N * (double)K / 6500.0 < single;
}

}  // namespace moe

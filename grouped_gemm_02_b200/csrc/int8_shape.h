// int8_shape.h -- how a dense int8 product is cut: the form of the kernel, the
// rows of a tile and the CTAs that share a tile's K range.  Plain arithmetic on
// the sizes, compiled for the host by the entry point and by the CPU tests.
#pragma once

#include <cstdint>

namespace moe {

constexpr int I8_SINGLE = 0, I8_PAIR = 1, I8_SPLIT = 2;
constexpr int kI8BlockK = 128;                   // codes per K block

// What a device can hold at once: SMs, CTA pairs (0: none), and clusters of 2 to 8
// CTAs that share a tile.  Large clusters pack badly into a GPC (a B200 holds 74 of
// 2, 33 of 4, 22 of 6 and 15 of 8), and a cluster that has to wait for another one
// doubles the time, so the counts come from the occupancy query and a cut never
// exceeds them.
constexpr int kI8MaxSplit = 8;

struct Int8Device {
    int sms = 0, pairs = 0;
    int clusters[kI8MaxSplit + 1] = {};     // by CTAs a cluster
};

struct Int8Shape {
    int form, chunk, units, split;
    int64_t tiles;          // of 128 channels (I8_PAIR: 256) and `chunk` rows
};

// Nanoseconds of a product cut this way, up to a constant (launch and start-up).
// A tile streams K/128 blocks; a block costs the larger of its bytes at what an SM
// draws from L2 (92 bytes/ns) and its MMAs (1.4 ns a column); a tile costs 215 ns
// more, and the last one's epilogue 7 ns a column.  Pairs start 2.8 us later.
// Joining a shared tile costs 2.2 us, 30 ns a CTA and 19 ns a column.  The constants
// were fitted when every box of rows was 16 or 64 high.  Checked on the present
// kernel, 2,967 timings on a B200 of every form, row count and cluster size at 121
// sizes (T 1..4096, K 512..16384, N 512..7168): the cut with the smallest cost is
// within 0.8% of the fastest one measured in the geometric mean, within 8.5% for every
// size.  Always 256 rows a tile on single CTAs (fewer where T is smaller) is up to 2.7
// times slower where few tiles leave SMs idle: T=256 K=16384 N=2048 49 us against 18.
inline double i8_cost(int64_t T, int64_t K, int64_t N, int sms, int form, int chunk, int split)
{
    const int64_t units = (T + chunk - 1) / chunk;
    const int64_t tiles = (N + (form == I8_PAIR ? 255 : 127)) / (form == I8_PAIR ? 256 : 128) * units;
    const int64_t ctas = tiles * (form == I8_PAIR ? 2 : split), slots = sms > 0 ? sms : 1;
    const double waves = (double)((ctas + slots - 1) / slots);
    const double blocks = (double)((K + kI8BlockK - 1) / kI8BlockK) / split;
    const double load = (128.0 + (form == I8_PAIR ? chunk / 2 : chunk)) * 128.0 / 92.0, mma = 1.4 * chunk;
    double t = waves * (blocks * (load > mma ? load : mma) + 215.0) + 7.0 * chunk;
    if (form == I8_PAIR) t += 2800.0;
    if (form == I8_SPLIT) t += 2200.0 + 30.0 * split + 19.0 * chunk;
    return t;
}

// The cheapest cut.  Rows a tile: a multiple of 16 (I8_PAIR: 32), at most 256.
// pairs: -1 the rule, 0 no CTA pairs, 1 pairs only (when the device runs them).
inline Int8Shape i8_shape(int64_t T, int64_t K, int64_t N, const Int8Device& dev, int pairs)
{
    static const int kRows[] = {16, 32, 48, 64, 96, 128, 160, 192, 224, 256};
    const int64_t nk = (K + kI8BlockK - 1) / kI8BlockK;
    Int8Shape best{I8_SINGLE, 256, 0, 1, 0};
    double least = -1.0;
    for (int c : kRows) {
        const int64_t units = (T + c - 1) / c;
        for (int f = 0; f <= kI8MaxSplit; f++) {
            const int form = f == 0 ? I8_SINGLE : f == 1 ? I8_PAIR : I8_SPLIT, split = f < 2 ? 1 : f;
            const int64_t tiles = (N + (form == I8_PAIR ? 255 : 127)) / (form == I8_PAIR ? 256 : 128) * units;
            if (tiles >= (int64_t(1) << 30)) continue;
            if (form == I8_PAIR ? (dev.pairs == 0 || pairs == 0 || c % 32 != 0) : (dev.pairs > 0 && pairs == 1)) continue;
            if (form == I8_SPLIT && (split > nk || tiles > dev.clusters[split])) continue;
            const double t = i8_cost(T, K, N, dev.sms, form, c, split);
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
// K = N = 2048, single CTAs against pairs: 64 experts with 4 rows each 41.3 and
// 43.7 us, 128 rows 66 and 62, 256 rows 91 and 84, 512 rows 160 and 141; 16
// experts with 512 rows at K = N = 1024 19.4 and 22.6 (by i8_cost 4% cheaper).
inline bool i8_grouped_pair(int64_t P, int64_t K, int64_t N, int64_t E, const Int8Device& dev, int pairs)
{
    if (dev.pairs == 0) return false;
    if (pairs >= 0) return pairs == 1;
    const int64_t blocks = P < E ? P : E, rows = (P + E - 1) / E;
    const int chunk = rows >= 256 ? 256 : (int)((rows + 31) / 32 * 32);
    // the mean segments end to end, as one dense product of whole tiles
    const int64_t T = blocks * ((rows + chunk - 1) / chunk) * chunk;
    const double single = i8_cost(T, K, N, dev.sms, I8_SINGLE, chunk, 1);
    const double pair = i8_cost(T, K, N, dev.sms, I8_PAIR, chunk, 1);
    return pair < 0.8 * single && (double)blocks * (double)N * (double)K / 6500.0 < single;
}

}  // namespace moe

// int8.cuh -- the matrix product in 8-bit integers with one scale a token and
// one a channel, on tcgen05 (kind::i8, int32 accumulation in TMEM):
//
//   out[r, n] = bf16( sum_k xq[r, k] Wq[e, n, k]  *  sx[r]  *  sw[e, n] )
//
// of one weight matrix for every row (dense, e = 0) or of expert e's matrix for
// the rows offsets[e] .. offsets[e + 1) (grouped).  The sum is exact: a product
// is at most 2^14, so K <= 2^16 keeps it at 2^30 at most; it is rounded to fp32
// once, scaled in fp32 (by the channel first: a row's scale may be near the end of
// the range, a weight's is not) and rounded to bf16 once.
//
// As in the bf16 expert GEMM the weights fill the M slot (128 channels) and the
// rows the N slot (16..256), so a decode batch costs a 16-wide MMA.  A K block is
// 128 codes, one 128-byte swizzle row; the last one of a K that is not a
// multiple of 128 is filled with zeros by the TMA.  Three forms:
//
//   I8_SINGLE  one CTA a tile, persistent over the tile list
//   I8_PAIR    CTA pairs (cta_group::2): 256 channels a tile, each CTA loads its
//              128 channels and half of the rows -- two thirds of the shared
//              memory traffic per MMA, which bounds wide tiles of 8-bit operands
//   I8_SPLIT   a cluster of 2 to 8 CTAs shares one tile's K range and adds
//              the int32 sums through distributed shared memory: dense products
//              with fewer tiles than SMs, bound by the weights' bytes.  The sums
//              are integers, so the split changes no bit.
//
// Warp roles: warp 0 TMA producer, warp 1 MMA issuer, warps 2-9 epilogue (two a
// TMEM lane quadrant, every other 16 columns each); two TMEM accumulators of 256
// columns; every wait is bounded.  All loads come after griddepcontrol.wait: the
// weights may be the output of the kernel before (a quantiser).
//
// Bound: at prefill the tensor cores, under the power cap (T=4096 K=7168 N=4096 on
// one B200: 77 us, 3.1 PTOP/s, tensor pipe 86% of the active cycles); at K = 2048 and below the
// epilogue's stores beside the loads (T=8192 N=7168 98 us, 2.5 PTOP/s; without its
// stores 74); at decode HBM (256 rows over 53 experts, K=N=2048: 41 us, 5.4 TB/s).
#pragma once

#include "common.cuh"
#include "grouped_gemm.cuh"
#include "int8_shape.h"
#include "ptx.cuh"

namespace moe {

constexpr int kI8MaxK = 1 << 16;
constexpr int kI8Epilogues = 8;                  // epilogue warps
constexpr int kI8Threads = 64 + 32 * kI8Epilogues;
constexpr int kI8RingBytes = 192 * 1024;
constexpr int kI8ScaleBytes = 2 * 256 * 4;       // the tile's row scales, for each half of the epilogue warps
constexpr int kI8TurnBytes = 2 * 2 * 16 * 256;   // [half][buffer][16 rows][128 channels] bf16

// The tiles of a grouped product, built by every CTA for itself from counts and
// offsets: one block for each expert with rows, heaviest first, cut into `units`
// tiles of `chunk` rows.
struct I8Plan {
    int4 blk[kMaxExperts];          // expert, first row, rows, chunk
    int n[kMaxExperts];             // rows by expert (zeros up to a multiple of 4: the ranking reads int4)
    int units[kMaxExperts];
    int tb[kMaxExperts + 1];        // prefix of units
    int nb, widest, cap;
};
constexpr int kI8SmemBytes = 1024 + kI8RingBytes + kBarBytes + (int)sizeof(I8Plan) + kI8ScaleBytes + kI8TurnBytes;
static_assert(kI8SmemBytes <= 227 * 1024, "shared memory budget");
static_assert(sizeof(I8Plan) % 16 == 0 && kBarBytes % 16 == 0, "the scales are read as float4");
static_assert(128 * 256 * 4 <= kI8RingBytes, "the int32 tile of I8_SPLIT reuses the ring");

struct Int8Args {
    const int32_t* counts;  // grouped: rows of each expert, and where they begin; dense: null
    const int32_t* offsets;
    int E;
    int T;                  // rows; dense: cut into `units` chunks of `chunk` rows
    int units, chunk;
    int N, K;
    const float* sx;        // [rows]
    const float* sw;        // [E, N]
    bf16* out;              // [rows, N]
    uint32_t* err;
};

struct I8Tile {
    int e, m, row0, rows, n_mma, ma, b_row0, b_n;
};

// Tile t of the launch.  rank: this CTA's place in its pair.
template <int FORM>
__device__ __forceinline__ I8Tile i8_tile(int t, const Int8Args& a, const I8Plan* sp, int rank)
{
    constexpr int kRows = FORM == I8_PAIR ? 256 : 128;
    I8Tile tl;
    int start, row_base, n;
    const int mt = (a.N + kRows - 1) / kRows;
    if (!a.counts) {
        const int u = t / mt;
        tl.m = t - u * mt;
        tl.e = 0;
        start = u * a.chunk;
        row_base = 0;
        n = min(a.chunk, a.T - start);
    } else {
        // tile t of block lo: channel block m of the unit's rows; the units of one channel
        // block run together and share its weights in L2
        int lo = 0, hi = sp->nb - 1;
        const int tu = t / mt;     // prefix entries count units
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (sp->tb[mid] <= tu) lo = mid;
            else hi = mid - 1;
        }
        const int units = sp->units[lo];
        const int local = t - sp->tb[lo] * mt;
        const int4 b = sp->blk[lo];
        tl.e = b.x;
        tl.m = local / units;
        start = (local - tl.m * units) * b.w;
        row_base = b.y;
        n = min(b.w, b.z - start);
    }
    tl.rows = n;
    tl.row0 = row_base + start;
    tl.n_mma = FORM == I8_PAIR ? (n + 31) & ~31 : (n + 15) & ~15;
    if (FORM == I8_PAIR) {
        tl.ma = 2 * tl.m + rank;
        tl.b_n = tl.n_mma >> 1;
        tl.b_row0 = tl.row0 + rank * tl.b_n;
    } else {
        tl.ma = tl.m;
        tl.b_n = tl.n_mma;
        tl.b_row0 = tl.row0;
    }
    return tl;
}

// Rows of B that the CTA of this rank loads for a tile: its share of the tile's
// rows, whole 64s and 16s and a last box for the rest.  The rest of a dense product
// is always T % 16 rows, a box of that height; an expert's is brought in a box of 4,
// 8 or 16 (the rows behind it are other experts', or zeros past the last row).
// Rows that no box brings stay as they are in shared memory: they only reach columns
// that are not stored.  Rows cost time even where they are few, and boxes that lie
// mostly past the last row cost more: with 16-row boxes throughout, K=2048 N=108544
// took 43 us at T=4 and 45 at T=17 against 39 at T=16; now 37, 39 and 39.
__device__ __forceinline__ int i8_rows_loaded(const Int8Args& a, const I8Tile& tl, int rank)
{
    const int rows = min(tl.b_n, max(0, tl.rows - rank * tl.b_n)), rest = rows & 15;
    if (!a.counts || rest == 0) return rows;
    return (rows & ~15) + (rest <= 4 ? 4 : rest <= 8 ? 8 : 16);
}

// Builds the plan of a grouped product (every thread of the CTA).  Returns false
// when a segment lies outside the rows, or the segments hold more rows than there
// are (they overlap, and the prefix of units might pass 32 bits).  slots: CTAs (or pairs) of the launch.
//
// The rows of a tile: at most `cap`, the one of 256, 128, 64 and 32 that costs
// the least by the terms of i8_cost (waves of tiles, each by its bytes at an
// SM's share of L2): few, wide segments take narrower tiles until the SMs are
// busy.  A block of n rows is cut into ceil(n / cap) units of equal width.
__device__ __forceinline__ bool i8_plan(const Int8Args& a, I8Plan* p, int mt, int nk, int slots, bool pair)
{
    constexpr int kMine = (kMaxExperts + kI8Threads - 1) / kI8Threads;   // experts a thread takes
    const int tid = threadIdx.x, lane = tid & 31;
    const int align = pair ? 32 : 16;
    int n[kMine], o[kMine], rank[kMine];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kMine; i++) {
        const int e = tid + i * kI8Threads;
        n[i] = e < a.E ? a.counts[e] : 0;
        o[i] = e < a.E ? a.offsets[e] : 0;
    }
#pragma unroll
    for (int i = 0; i < kMine; i++) {
        const int e = tid + i * kI8Threads;
        bad |= n[i] < 0 || n[i] > a.T || (n[i] > 0 && (o[i] < 0 || o[i] > a.T - n[i]));
        if (e < ((a.E + 3) & ~3)) p->n[e] = n[i];
    }
    if (__syncthreads_or(bad)) return false;
#pragma unroll
    for (int i = 0; i < kMine; i++) {
        const int e = tid + i * kI8Threads;
        int r = 0;      // more rows first, then the lower expert
        if (n[i] > 0) {
#pragma unroll 4
            for (int j = 0; j < a.E; j += 4) {
                const int4 m = *reinterpret_cast<const int4*>(p->n + j);
                r += m.x > n[i] || (m.x == n[i] && j < e);
                r += m.y > n[i] || (m.y == n[i] && j + 1 < e);
                r += m.z > n[i] || (m.z == n[i] && j + 2 < e);
                r += m.w > n[i] || (m.w == n[i] && j + 3 < e);
            }
        }
        rank[i] = r;
    }
    if (tid < 32) {
        // total units under each cap, and the widest segment
        int u[4] = {0, 0, 0, 0}, most = 0, nb = 0;
        int64_t all = 0;
        for (int e = lane; e < a.E; e += 32) {
            const int m = p->n[e];
#pragma unroll
            for (int i = 0; i < 4; i++) u[i] += (m + (256 >> i) - 1) / (256 >> i);
            most = max(most, m);
            nb += m > 0;
            all += m;
        }
        // a lane's sum is below 2^35: its halves add up in 32 bits
        all = (int64_t)__reduce_add_sync(0xffffffffu, (int)(all >> 16)) * 65536 +
              __reduce_add_sync(0xffffffffu, (int)(all & 0xFFFF));
        most = __reduce_max_sync(0xffffffffu, most);
        float least = 0.f;
        int cap = 256;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int units = __reduce_add_sync(0xffffffffu, u[i]);
            const int w = min(256 >> i, max(most, 1));
            const float waves = (float)(((int64_t)units * mt + slots - 1) / slots);
            const float kb = fmaxf((128.f + (pair ? 0.5f : 1.f) * (float)w) * (128.f / 92.f), 1.4f * (float)w);
            const float cost = waves * ((float)nk * kb + 215.f) + 7.f * (float)w;
            if (i == 0 || cost < least) {
                least = cost;
                cap = 256 >> i;
            }
        }
        nb = __reduce_add_sync(0xffffffffu, nb);
        if (lane == 0) {
            p->cap = all > a.T ? 0 : cap;
            p->nb = nb;
        }
    }
    __syncthreads();
    const int cap = p->cap;
    if (cap == 0) return false;
#pragma unroll
    for (int i = 0; i < kMine; i++) {
        if (n[i] == 0) continue;
        const int units = (n[i] + cap - 1) / cap;
        const int chunk = ((n[i] + units - 1) / units + align - 1) / align * align;
        p->blk[rank[i]] = make_int4(tid + i * kI8Threads, o[i], n[i], chunk);
        p->units[rank[i]] = units;
    }
    __syncthreads();
    if (tid < 32) {
        // prefix of units over the blocks, 32 at a time
        const int nb = p->nb;
        int run = 0, widest = 0;
        for (int i = 0; i < nb; i += 32) {
            const bool in = i + lane < nb;
            int v = in ? p->units[i + lane] : 0;
            if (in) widest = max(widest, p->blk[i + lane].w);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += x;
            }
            if (in) p->tb[i + lane + 1] = run + v;
            run += __shfl_sync(0xffffffffu, v, 31);
        }
        widest = __reduce_max_sync(0xffffffffu, widest);
        if (lane == 0) {
            p->tb[0] = 0;
            p->widest = max(widest, align);
        }
    }
    __syncthreads();
    return true;
}

// 16 columns of one warp's accumulator quadrant, lane = channel, as bf16 pairs of
// neighbouring columns (w[p] holds columns 2p and 2p + 1 of this lane's channel),
// turned so that each lane holds 8 consecutive channels of a column: on return
// o[r] is channels 8 (lane / 8) .. + 7 of column 8 r + lane % 8.  Three rounds of
// exchange between lanes that differ in bit 0, 1 and 2: 16 shuffles for 16
// columns, and the global store is then 16 bytes a lane instead of 2.
__device__ __forceinline__ void i8_turn16(const uint32_t (&w)[8], uint4 (&o)[2], int lane)
{
    const bool b0 = lane & 1, b1 = lane & 2, b2 = lane & 4;
    uint32_t a[8];      // column 2p + b0: channels 2 (lane / 2), + 1
#pragma unroll
    for (int p = 0; p < 8; p++) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, w[p], 1);
        a[p] = b0 ? __byte_perm(r, w[p], 0x7632) : __byte_perm(w[p], r, 0x5410);
    }
    uint32_t b[4][2];   // column 4q + 2 b1 + b0: channels 4 (lane / 4) .. + 3
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const uint32_t r = __shfl_xor_sync(0xffffffffu, b1 ? a[2 * q] : a[2 * q + 1], 2);
        b[q][0] = b1 ? r : a[2 * q];
        b[q][1] = b1 ? a[2 * q + 1] : r;
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const uint32_t r0 = __shfl_xor_sync(0xffffffffu, b2 ? b[2 * h][0] : b[2 * h + 1][0], 4);
        const uint32_t r1 = __shfl_xor_sync(0xffffffffu, b2 ? b[2 * h][1] : b[2 * h + 1][1], 4);
        o[h] = b2 ? make_uint4(r0, r1, b[2 * h + 1][0], b[2 * h + 1][1]) : make_uint4(b[2 * h][0], b[2 * h][1], r0, r1);
    }
}

template <int FORM>
__global__ void __launch_bounds__(kI8Threads, 1)
    int8_gemm_kernel(const __grid_constant__ CUtensorMap mA, const __grid_constant__ CUtensorMap mB16,
                     const __grid_constant__ CUtensorMap mB64, const __grid_constant__ CUtensorMap mB4,
                     const __grid_constant__ CUtensorMap mB8, const Int8Args a)
{
    // mA: 128 channels a box; mB64, mB16: 64 and 16 rows; the rest: grouped mB8 and mB4,
    // of 8 and 4 rows, dense mB4, of T % 16 rows
    constexpr bool PAIR = FORM == I8_PAIR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    SmemCtl* ctl = reinterpret_cast<SmemCtl*>(smem + kI8RingBytes);
    I8Plan* splan = reinterpret_cast<I8Plan*>(smem + kI8RingBytes + kBarBytes);
    const uint32_t ring = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = FORM != I8_SINGLE ? (int)ptx::cluster_ctarank() : 0;
    const bool leader = !PAIR || rank == 0;
    const int split = FORM == I8_SPLIT ? (int)(gridDim.x / ptx::nclusters_x()) : 1;   // CTAs that share a tile
    const int first = FORM == I8_SINGLE ? (int)blockIdx.x : (int)ptx::cluster_id_x();
    const int step = FORM == I8_SINGLE ? (int)gridDim.x : (int)ptx::nclusters_x();

    // Barriers, descriptors and TMEM first: this part may run while the kernel before drains.
    if (threadIdx.x == 0) {
        for (int s = 0; s < kMaxStages; s++) {
            ptx::mbar_init(ptx::smem_u32(&ctl->full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&ctl->empty[s]), 1);
        }
        for (int i = 0; i < 2; i++) {
            ptx::mbar_init(ptx::smem_u32(&ctl->tfull[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&ctl->tempty[i]), PAIR ? 2 * kI8Epilogues : kI8Epilogues);
        }
        ptx::mbar_init(ptx::smem_u32(&ctl->drain), 1);
        ctl->abort = 0;
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == 0 && lane == 0) {
        ptx::prefetch_tensormap(&mA);
        ptx::prefetch_tensormap(&mB16);
        ptx::prefetch_tensormap(&mB64);
    }
    if (warp == 1) {
        if (PAIR) {
            ptx::tmem_alloc_pair(ptx::smem_u32(&ctl->tmem_base), kTmemCols);
            ptx::tmem_relinquish_pair();
        } else {
            ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem_base), kTmemCols);
            ptx::tmem_relinquish();
        }
    }
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int kRows = PAIR ? 256 : 128;
    const int mt = (a.N + kRows - 1) / kRows;
    const int nk = (a.K + kI8BlockK - 1) / kI8BlockK;
    int total = a.units * mt, widest = min(a.chunk, a.T);
    if (a.counts) {
        const bool ok = i8_plan(a, splan, mt, nk, step, PAIR);
        if (!ok && threadIdx.x == 0) atomicOr(a.err, DEVERR_PLAN);
        // segments that do not fit the rows: every CTA sees the same counts and takes no tile
        total = ok ? splan->tb[splan->nb] * mt : 0;
        widest = ok ? splan->widest : 32;
    }
    const int n_max = PAIR ? max(32, (widest + 31) & ~31) : max(16, (widest + 15) & ~15);
    const uint32_t stage_bytes = kATileBytes + (uint32_t)(PAIR ? n_max / 2 : n_max) * kBRowBytes;
    const int stages = min(kMaxStages, (int)(kI8RingBytes / stage_bytes));
    // I8_SPLIT: this CTA's K blocks (the host launches no more CTAs a tile than K blocks)
    const int kb0 = FORM == I8_SPLIT ? (int)((int64_t)nk * rank / split) : 0;
    const int kb1 = FORM == I8_SPLIT ? (int)((int64_t)nk * (rank + 1) / split) : nk;

    ptx::tc_fence_before();
    if (PAIR) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem_base = ctl->tmem_base;
    auto leader_bar = [&](uint64_t* bar) -> uint32_t {
        return PAIR ? ptx::mapa_shared(ptx::smem_u32(bar), 0) : ptx::smem_u32(bar);
    };

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (ptx::elect_one()) {
            const uint64_t pol = ptx::policy_evict_normal();
            uint32_t armed = 0, armed_ph = 0;
            bool ok = true;
            int s = 0;
            uint32_t ph = 0;
            for (int t = first; ok && t < total; t += step) {
                const I8Tile tl = i8_tile<FORM>(t, a, splan, rank);
                const int a_row = tl.e * a.N + tl.ma * 128;
                const int rows = i8_rows_loaded(a, tl, PAIR ? rank : 0), rest = rows & 15;
                // the leader of a pair counts both CTAs' bytes
                const int all_rows = PAIR ? i8_rows_loaded(a, tl, 0) + i8_rows_loaded(a, tl, 1) : rows;
                const uint32_t tx = (PAIR ? 2u : 1u) * kATileBytes + (uint32_t)all_rows * kBRowBytes;
                const CUtensorMap* last = a.counts && rest == 8 ? &mB8 : &mB4;
                for (int kb = kb0; kb < kb1; kb++) {
                    if (!bounded_wait(ptx::smem_u32(&ctl->empty[s]), ph ^ 1u, ctl, a.err)) {
                        ok = false;
                        break;
                    }
                    const uint32_t a_dst = ring + (uint32_t)s * stage_bytes;
                    const uint32_t full = leader_bar(&ctl->full[s]);
                    if (leader) {
                        ptx::mbar_arrive_expect_tx(ptx::smem_u32(&ctl->full[s]), tx);
                        armed |= 1u << s;
                        armed_ph = (armed_ph & ~(1u << s)) | (ph << s);
                    }
                    const int kc = kb * kI8BlockK;
                    tma_load<PAIR>(a_dst, &mA, full, kc, a_row, pol);
                    const uint32_t b_dst = a_dst + kATileBytes;
                    int r = 0;
                    for (; r + 64 <= rows; r += 64)
                        tma_load<PAIR>(b_dst + r * kBRowBytes, &mB64, full, kc, tl.b_row0 + r, pol);
                    for (; r + 16 <= rows; r += 16)
                        tma_load<PAIR>(b_dst + r * kBRowBytes, &mB16, full, kc, tl.b_row0 + r, pol);
                    if (rest) tma_load<PAIR>(b_dst + r * kBRowBytes, last, full, kc, tl.b_row0 + r, pol);
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
            }
            if (!ok) {
                // drain (bounded): every stage armed here has landed before the block leaves
                const uint64_t t0 = ptx::globaltimer();
                for (int i = 0; i < stages; i++) {
                    if (!(armed >> i & 1u)) continue;
                    const uint32_t bar = ptx::smem_u32(&ctl->full[i]);
                    while (!ptx::mbar_try_wait(bar, (armed_ph >> i) & 1u) &&
                           ptx::globaltimer() - t0 < kWaitTimeoutNs) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer (the leader of a pair)
        if (leader && ptx::elect_one()) {
            int s = 0, acc = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true, issued = false;
            for (int t = first; ok && t < total; t += step) {
                const I8Tile tl = i8_tile<FORM>(t, a, splan, rank);
                if (!bounded_wait(ptx::smem_u32(&ctl->tempty[acc]), aph ^ 1u, ctl, a.err)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t d_tmem = tmem_base + (uint32_t)acc * 256u;
                const uint32_t idesc = ptx::idesc_s8_s32(PAIR ? 256 : 128, (uint32_t)tl.n_mma);
                for (int kb = kb0; kb < kb1; kb++) {
                    if (!bounded_wait(ptx::smem_u32(&ctl->full[s]), ph, ctl, a.err)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t a_addr = ring + (uint32_t)s * stage_bytes;
                    const uint32_t b_addr = a_addr + kATileBytes;
#pragma unroll
                    for (int kk = 0; kk < kI8BlockK / 32; kk++) {
                        const uint64_t ad = ptx::sw128_kmajor_desc(a_addr + kk * 32);
                        const uint64_t bd = ptx::sw128_kmajor_desc(b_addr + kk * 32);
                        const uint32_t accum = (kb > kb0 || kk > 0) ? 1u : 0u;
                        if (PAIR) ptx::mma_i8_ss_pair(d_tmem, ad, bd, idesc, accum);
                        else ptx::mma_i8_ss(d_tmem, ad, bd, idesc, accum);
                    }
                    issued = true;
                    if (PAIR) ptx::mma_commit_pair(ptx::smem_u32(&ctl->empty[s]), 3);
                    else ptx::mma_commit(ptx::smem_u32(&ctl->empty[s]));
                    if (++s == stages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (!ok) break;
                if (PAIR) ptx::mma_commit_pair(ptx::smem_u32(&ctl->tfull[acc]), 3);
                else ptx::mma_commit(ptx::smem_u32(&ctl->tfull[acc]));
                acc ^= 1;
                if (acc == 0) aph ^= 1u;
            }
            if (!ok && issued) {
                if (PAIR) ptx::mma_commit_pair(ptx::smem_u32(&ctl->drain), 1);
                else ptx::mma_commit(ptx::smem_u32(&ctl->drain));
                const uint64_t t0 = ptx::globaltimer();
                while (!ptx::mbar_try_wait(ptx::smem_u32(&ctl->drain), 0) &&
                       ptx::globaltimer() - t0 < kWaitTimeoutNs) {
                }
            }
        }
    } else {
        // ------------------------------------------------------------ epilogue (warps 2-9)
        const int quad = warp & 3, half = (warp - 2) >> 2;
        uint8_t* s_half = smem + kI8RingBytes + kBarBytes + sizeof(I8Plan);
        float* s_sx = reinterpret_cast<float*>(s_half) + half * 256;
        uint4* s_turn = reinterpret_cast<uint4*>(s_half + kI8ScaleBytes + half * (kI8TurnBytes / 2));
        uint32_t chunks = 0;    // 16-column chunks so far: the turn buffer alternates across tiles too
        int acc = 0;
        uint32_t aph = 0;
        for (int t = first; t < total; t += step) {
            const I8Tile tl = i8_tile<FORM>(t, a, splan, rank);
            // scales, fetched before the accumulator wait: a channel a lane, the tile's rows in shared memory
            const int ch = tl.ma * 128 + quad * 32 + lane;
            const float sw = (FORM != I8_SPLIT && ch < a.N) ? __ldg(a.sw + (size_t)tl.e * a.N + ch) : 0.f;
            if (FORM != I8_SPLIT) {
                // the half's four warps share the scales; the last tile's were read before
                // its last chunk's barrier
                for (int i = quad * 32 + lane; i < tl.n_mma; i += 128)
                    s_sx[i] = i < tl.rows ? __ldg(a.sx + tl.row0 + i) : 0.f;
            }
            const bool ok = bounded_wait(ptx::smem_u32(&ctl->tfull[acc]), aph, ctl, a.err);
            // the half leaves together: its warps meet at the chunks' barriers
            if (ptx::named_barrier_or(1 + half, 128, !ok)) break;
            ptx::tc_fence_after();
            const uint32_t taddr = tmem_base + (uint32_t)acc * 256u + ((uint32_t)(quad * 32) << 16);
            for (int c0 = 16 * half; c0 < tl.n_mma; c0 += 32) {
                uint32_t v[16];
                ptx::tmem_ld16(taddr + (uint32_t)c0, v);
                ptx::tmem_ld_wait();
                if (FORM == I8_SPLIT) {
                    // this CTA's int32 sums, [column][channel], over the ring: every load of
                    // it has been consumed and the cluster runs one tile
                    int* red = reinterpret_cast<int*>(smem);
#pragma unroll
                    for (int j = 0; j < 16; j++)
                        red[(c0 + j) * 128 + quad * 32 + lane] = (int)v[j];
                } else {
                    uint32_t w[8];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float4 sc = reinterpret_cast<const float4*>(s_sx + c0)[j];
                        const __nv_bfloat162 lo = __floats2bfloat162_rn((float)(int)v[4 * j] * sw * sc.x,
                                                                        (float)(int)v[4 * j + 1] * sw * sc.y);
                        const __nv_bfloat162 hi = __floats2bfloat162_rn((float)(int)v[4 * j + 2] * sw * sc.z,
                                                                        (float)(int)v[4 * j + 3] * sw * sc.w);
                        w[2 * j] = *reinterpret_cast<const uint32_t*>(&lo);
                        w[2 * j + 1] = *reinterpret_cast<const uint32_t*>(&hi);
                    }
                    uint4 o[2];
                    i8_turn16(w, o, lane);
                    // through shared memory into rows of 128 channels: a warp stores four whole
                    // 256-byte rows (64-byte pieces from each quadrant's warp cost 15 to 20% of
                    // the product at K = 2048).  16-byte units are swizzled by the row.
                    uint4* buf = s_turn + (chunks++ & 1u) * 256;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int r = 8 * h + (lane & 7);
                        buf[r * 16 + ((quad * 4 + (lane >> 3)) ^ (r & 7))] = o[h];
                    }
                    ptx::named_barrier(1 + half, 128);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const int r = 4 * quad + 2 * h + (lane >> 4), u = lane & 15;
                        const int col = c0 + r, oc = tl.ma * 128 + u * 8;
                        if (col < tl.rows && oc < a.N)   // N % 8 == 0: all 8 channels or none
                            *reinterpret_cast<uint4*>(a.out + (size_t)(tl.row0 + col) * a.N + oc) =
                                buf[r * 16 + (u ^ (r & 7))];
                    }
                }
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) ptx::mbar_arrive_cluster(leader_bar(&ctl->tempty[acc]));
                else ptx::mbar_arrive(ptx::smem_u32(&ctl->tempty[acc]));
            }
            acc ^= 1;
            if (acc == 0) aph ^= 1u;
        }
    }

    ptx::tc_fence_before();
    if (FORM != I8_SINGLE) ptx::cluster_sync();
    else __syncthreads();
    if (FORM == I8_SPLIT) {
        // every CTA of the cluster adds a share of the tile: the flattened (column,
        // 4 channels) items, dealt over the cluster's threads
        if (first < total) {
            const I8Tile tl = i8_tile<FORM>(first, a, splan, rank);
            const int items = tl.rows * 32;
            for (int i = rank * kI8Threads + (int)threadIdx.x; i < items; i += split * kI8Threads) {
                const int col = i >> 5, c4 = (i & 31) * 4;
                const int ch = tl.ma * 128 + c4;
                if (ch >= a.N) continue;       // N % 4 == 0: all four channels or none
                int sum[4] = {0, 0, 0, 0}, gave_up = 0;
                for (int p = 0; p < split; p++) {
                    int v[4];
                    ptx::ld_cluster_v4(ptx::mapa_shared(ring + (uint32_t)(col * 128 + c4) * 4u, p), v);
                    gave_up |= ptx::ld_cluster_s32(ptx::mapa_shared(ptx::smem_u32(&ctl->abort), p));
#pragma unroll
                    for (int j = 0; j < 4; j++) sum[j] += v[j];
                }
                // a CTA whose wait ran out left no sums: the tile stays as it was, as in the other forms
                if (gave_up) continue;
                const float sx = __ldg(a.sx + tl.row0 + col);
                const float4 sw = __ldg(reinterpret_cast<const float4*>(a.sw + ch));
                __nv_bfloat162 lo = __floats2bfloat162_rn((float)sum[0] * sw.x * sx, (float)sum[1] * sw.y * sx);
                __nv_bfloat162 hi = __floats2bfloat162_rn((float)sum[2] * sw.z * sx, (float)sum[3] * sw.w * sx);
                *reinterpret_cast<uint2*>(a.out + (size_t)(tl.row0 + col) * a.N + ch) =
                    make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
            }
        }
        ptx::cluster_sync();   // no CTA leaves while another may still read its sums
    }
    __syncwarp();
    if (warp == 1) {
        ptx::tc_fence_after();
        if (PAIR) ptx::tmem_dealloc_pair(tmem_base, kTmemCols);
        else ptx::tmem_dealloc(tmem_base, kTmemCols);
    }
}

}  // namespace moe

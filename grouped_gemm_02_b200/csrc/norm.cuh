// norm.cuh -- the residual's addition with a root-mean-square norm, its result
// in bf16, in e4m3 with 1 x 128 scales or in int8 with one scale a row; its
// gradient; and the int8 row quantiser.
//
//   s    = bf16(x + r)                         the residual stream (r absent: s = x)
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   y    = bf16(s * rstd * w)
//   q    = the codes of y: those of moe_quantize_fp8_rows (1 x 128 blocks) or of
//          moe_quantize_int8_rows (one scale a row), bit for bit
//
// Roundings: s once (the stream is kept in bf16 and the norm is of what is
// kept), y once, and the codes are taken from the rounded y, so that what reads
// y and what reads q see the same row.
//
// Bound: HBM.  Every input is read once and every output written once: a row
// stays in the registers of one group of warps between the reduction and the
// normalisation.  T=16384 d=7168 with a residual on one B200: bf16 137 us (6.8
// TB/s), e4m3 132 us (6.2 TB/s), int8 134 us (6.1 TB/s); the gradient at T=4099
// d=7168 42 us (5.6 TB/s).  Next to the bytes it is the instructions that count (the
// e4m3 form issues in two thirds of its slots), so the arithmetic runs on pairs of
// fp32 values.
#pragma once

#include "common.cuh"
#include "fp8.cuh"
#include "int8_code.h"
#include "ptx.cuh"

namespace moe {

constexpr int kNormMaxD = 32768;             // 1024 threads x 32 values
constexpr float kMaxFloat = 3.402823466e+38f;
constexpr int kDoubleInf = 0x7FF00000, kDoubleLow = (1023 - 50) << 20;   // high words of infinity and of 2^-50
constexpr int NORM_BF16 = 0, NORM_FP8 = 1, NORM_INT8 = 2;

// How rows are laid over a CTA: a row belongs to a group of `warps` warps whose
// threads hold `vpt` vectors each (32 bytes in the forward kernels, 16 in the
// gradient); `groups` rows share a CTA.
struct RowShape {
    int vpt, warps, groups;
};

__host__ __device__ inline int row_warps(int nvec, int vpt) { return (nvec + 32 * vpt - 1) / (32 * vpt); }

// The layout of `nvec` vectors at `vpt` a thread: short rows share a CTA, up to 8 warps.
__host__ __device__ inline RowShape row_shape(int nvec, int vpt)
{
    RowShape s{vpt, row_warps(nvec, vpt), 1};
    while (s.groups < 8 && s.warps * s.groups * 2 <= 8) s.groups *= 2;
    return s;
}

struct f8 {
    float v[8];
};

// Two fp32 values in a register pair: one instruction for both, each rounded as the
// scalar operation rounds.  With scalar operations the gradient of T=4099 d=7168 took
// 44.7 us against 42.1, the forward pass 1 to 3% longer.
using f2 = unsigned long long;

__device__ __forceinline__ f2 f2_of(float lo, float hi)
{
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ float2 f2_get(f2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
    return r;
}

__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c)
{
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ f2 f2_mul(f2 a, f2 b)
{
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ f2 f2_add(f2 a, f2 b)
{
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// The two bf16 values of a word, and back.
__device__ __forceinline__ f2 f2_bf16(uint32_t w)
{
    return f2_of(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ uint32_t f2_pack(f2 a)
{
    const float2 v = f2_get(a);
    const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&p);
}

struct w4 {
    uint32_t w[4];
};

__device__ __forceinline__ w4 words(const uint4& u) { return w4{{u.x, u.y, u.z, u.w}}; }

__device__ __forceinline__ f8 unpack8(const uint4& u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    f8 r;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        r.v[2 * i] = __uint_as_float(w[i] << 16);
        r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return r;
}

__device__ __forceinline__ uint4 pack8(const f8& f)
{
    uint4 u;
    uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f.v[2 * i], f.v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return u;
}

// bf16(a + b), the sum of the squares of a or of c a (four in each half, then the
// halves), and bf16(((p a) w)(r0 + r1)), eight values at a time.
__device__ __forceinline__ uint4 add_bf16x8(const uint4& a, const uint4& b)
{
    const w4 x = words(a), y = words(b);
    w4 o;
#pragma unroll
    for (int j = 0; j < 4; j++) o.w[j] = f2_pack(f2_add(f2_bf16(x.w[j]), f2_bf16(y.w[j])));
    return make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
}

__device__ __forceinline__ float squares8(const uint4& a)
{
    const w4 x = words(a);
    f2 q = f2_mul(f2_bf16(x.w[0]), f2_bf16(x.w[0]));
#pragma unroll
    for (int j = 1; j < 4; j++) {
        const f2 v = f2_bf16(x.w[j]);
        q = f2_fma(v, v, q);
    }
    const float2 h = f2_get(q);
    return h.x + h.y;
}

__device__ __forceinline__ float squares8(const uint4& a, float c)
{
    const w4 x = words(a);
    const f2 cc = f2_of(c, c);
    f2 q = f2_of(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const f2 v = f2_mul(f2_bf16(x.w[j]), cc);
        q = f2_fma(v, v, q);
    }
    const float2 h = f2_get(q);
    return h.x + h.y;
}

__device__ __forceinline__ uint4 scale_bf16x8(const uint4& a, const uint4& w, float p, float r0, float r1)
{
    const w4 x = words(a), y = words(w);
    const f2 pp = f2_of(p, p), p0 = f2_of(r0, r0), p1 = f2_of(r1, r1);
    w4 o;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const f2 sw = f2_mul(f2_mul(f2_bf16(x.w[j]), pp), f2_bf16(y.w[j]));
        o.w[j] = f2_pack(f2_fma(sw, p0, f2_mul(sw, p1)));
    }
    return make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
}

// 16 bf16 values: 32 bytes, one load or store where the address allows it.  With
// 16 bytes a thread (and 8 of codes) the e4m3 norm took 4 to 8% longer.
struct v16 {
    uint4 lo, hi;
};

__device__ __forceinline__ v16 load16(const bf16* p, bool al32)
{
    v16 r;
    if (al32) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.lo.x), "=r"(r.lo.y), "=r"(r.lo.z), "=r"(r.lo.w), "=r"(r.hi.x), "=r"(r.hi.y),
                       "=r"(r.hi.z), "=r"(r.hi.w)
                     : "l"(p));
    } else {
        r.lo = reinterpret_cast<const uint4*>(p)[0];
        r.hi = reinterpret_cast<const uint4*>(p)[1];
    }
    return r;
}

__device__ __forceinline__ void store16(bf16* p, const v16& v, bool al32)
{
    if (al32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v.lo.x), "r"(v.lo.y),
                     "r"(v.lo.z), "r"(v.lo.w), "r"(v.hi.x), "r"(v.hi.y), "r"(v.hi.z), "r"(v.hi.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = v.lo;
        reinterpret_cast<uint4*>(p)[1] = v.hi;
    }
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ uint32_t warp_umax(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// Barrier over one group of warps (id 1.. for group 0..); a group of one warp needs no hardware barrier.
__device__ __forceinline__ void group_barrier(int group, int warps)
{
    if (warps == 1) __syncwarp();
    else ptx::named_barrier(1 + group, warps * 32);
}

// Sum over the group's threads, the same in every thread.  `slot` is this
// group's own scratch of `warps` values, not read by an earlier reduction that a
// warp of the group may still be in.
__device__ __forceinline__ double group_sum(double v, double* slot, int group, int warps)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, w = (int)(threadIdx.x >> 5) - group * warps;
    if (lane == 0) slot[w] = v;
    group_barrier(group, warps);
    v = slot[0];
    for (int i = 1; i < warps; i++) v += slot[i];
    return v;
}

__device__ __forceinline__ uint32_t group_umax(uint32_t v, uint32_t* slot, int group, int warps)
{
    v = warp_umax(v);
    if (warps == 1) return v;
    const int lane = threadIdx.x & 31, w = (int)(threadIdx.x >> 5) - group * warps;
    if (lane == 0) slot[w] = v;
    group_barrier(group, warps);
    return warp_umax(lane < warps ? slot[lane] : 0u);
}

// The magnitude bits of the largest of 8 bf16 values (a NaN ranks above infinity), as fp32 bits.
// Integer maxima, one value at a time: with packed bf16 maxima the int8 norm took a tenth
// longer (T=16384 d=7168, 16 bytes a thread: 147 us against 132).
__device__ __forceinline__ uint32_t amax_bits8(const uint4& u)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) m = max(m, max((w[i] << 16) & 0x7FFFFFFFu, w[i] & 0x7FFF0000u));
    return m;
}

// ---------------------------------------------------------------- int8 codes
// One scale a row (int8_code.h).
__device__ __forceinline__ uint2 int8_codes8(const uint4& u, float inv)
{
    const f8 f = unpack8(u);
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; i++) {
        // |v * inv| <= 127 (1 + 2^-22): rounds to at most 127.  inv = 0 (a NaN or
        // infinite row) makes 0 or NaN, and a NaN converts to code 0.
        const int c = __float2int_rn(f.v[i] * inv);
        w[i >> 2] |= (uint32_t)(c & 0xFF) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
}

// ---------------------------------------------------------------- e4m3 codes
// 16 values of a 1 x 128 block spread over 8 consecutive lanes: the block's
// exponent (the rule of the row quantiser in fp8.cuh) and this lane's codes.
// amax = 1.f x 2^(x - 127): the smallest e with amax <= 448 2^e = 1.75 2^(8 + e) is
// x - 135, one more above 1.75, held to -127 (a subnormal amax has x = 0).  The
// quantiser's maximum passes over a NaN, and takes infinity's exponent from frexpf:
// blocks that hold either go through its own functions.
__device__ __forceinline__ int e4m3_block_exp(const v16& u)
{
    uint32_t a = max(amax_bits8(u.lo), amax_bits8(u.hi));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (a >= 0x7F800000u) {      // the same for the 8 lanes of a block
        const unsigned lanes = 0xFFu << (threadIdx.x & 24);
        const f8 f = unpack8(u.lo), g = unpack8(u.hi);
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i++) m = fmaxf(m, fmaxf(fabsf(f.v[i]), fabsf(g.v[i])));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(lanes, m, o));
        return fp8_scale_exp(m);
    }
    if (a == 0u) return 0;
    return max(-127, (int)(a >> 23) - 135 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0));
}

__device__ __forceinline__ uint2 e4m3_codes8(const uint4& u, int e)
{
    const f8 f = unpack8(u);
    const float m = pow2f(-e);   // v * 2^-e: the same single rounding as ldexpf(v, -e)
    uint32_t w[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t p = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(f.v[2 * i] * m, f.v[2 * i + 1] * m),
                                                              __NV_SATFINITE, __NV_E4M3);
        w[i >> 1] |= p << (16 * (i & 1));
    }
    return make_uint2(w[0], w[1]);
}

// ---------------------------------------------------------------- forward
struct NormArgs {
    const bf16* x;
    const bf16* residual;   // may be null
    const bf16* weight;     // null (the int8 row quantiser): y = x, no norm
    bf16* xsum;             // with residual: may be x or residual (each element is read before it is written)
    bf16* y;                // may be null when there are codes
    uint8_t* q;
    float* scale;           // int8: [T]; e4m3: [T, d / 128]
    int64_t T;
    int d;
    float eps;
    double inv_d;
    bool al32;              // every bf16 pointer is 32-byte aligned
};

// One row a group; a thread holds WPT times 16 values.  d % 64 == 0 (e4m3: d % 128 == 0).
template <int OUT, int WPT>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs a, int warps)
{
    __shared__ double s_sum[2][32];
    __shared__ uint32_t s_max[32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int gt = warps * 32;                       // threads of a group
    const int group = (int)threadIdx.x / gt, ti = (int)threadIdx.x - group * gt;
    const int64_t row = (int64_t)blockIdx.x * ((int)blockDim.x / gt) + group;
    if (row >= a.T) return;                          // the whole group leaves
    const int nw = a.d / 16;
    const int64_t base = row * a.d;
    const v16 zero{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    v16 u[WPT];
#pragma unroll
    for (int i = 0; i < WPT; i++) {
        const int v = i * gt + ti;
        u[i] = v < nw ? load16(a.x + base + 16 * v, a.al32) : zero;
    }
    if (a.residual) {
        v16 r[WPT];
#pragma unroll
        for (int i = 0; i < WPT; i++) {
            const int v = i * gt + ti;
            r[i] = v < nw ? load16(a.residual + base + 16 * v, a.al32) : zero;
        }
#pragma unroll
        for (int i = 0; i < WPT; i++) {
            const int v = i * gt + ti;
            u[i].lo = add_bf16x8(u[i].lo, r[i].lo);
            u[i].hi = add_bf16x8(u[i].hi, r[i].hi);
            if (v < nw) store16(a.xsum + base + 16 * v, u[i], a.al32);
        }
    }
    if (a.weight) {
        double ss = 0.0;
#pragma unroll
        for (int i = 0; i < WPT; i++) {
            ss += (double)squares8(u[i].lo) + (double)squares8(u[i].hi);
        }
        ss = group_sum(ss, s_sum[0] + group * warps, group, warps);
        // Squares of bf16 values are exact in fp32 between 2^-63 and 2^64; eight at a time
        // add up there, and their sums, the mean and eps in 64 bits.  Where a square was
        // beyond fp32 the sum is infinite; where all were below it and eps is so small that
        // they count, it is tiny: such a row (the same for its whole group) is summed again
        // with its values scaled by a power of two.  They are read again: kept for this in
        // registers they cost the common path spills (e4m3 at T=16384 d=7168 133 us
        // against 131).
        const int sh = __double2hiint(ss) & 0x7FFFFFFF;   // compared as its high word; a NaN may have either sign
        if (sh >= kDoubleInf || (sh < kDoubleLow && a.eps < 0x1p-110f)) {
            const bool low = sh < kDoubleLow;
            const float c = low ? 0x1p64f : 0x1p-70f;
            double s2 = 0.0;
#pragma unroll
            for (int i = 0; i < WPT; i++) {
                const int v = i * gt + ti;
                if (v < nw) {
                    u[i] = load16((a.residual ? a.xsum : a.x) + base + 16 * v, a.al32);
                    s2 += (double)squares8(u[i].lo, c) + (double)squares8(u[i].hi, c);
                }
            }
            ss = group_sum(s2, s_sum[1] + group * warps, group, warps) * (low ? 0x1p-128 : 0x1p140);
        }
        // var = 4^e m with m in [1/4, 1), and 1 / sqrt(m) is r0 + r1, in (1, 2]: r0 from rsqrtf
        // (within 2 units in the last place), r1 one Newton step from its residual 1 - m r0^2.
        // 2^-e s w is then y or down to half of it: it leaves the range only where y does (s w
        // itself may: the multiplication by 2^-e costs e4m3 and int8 2 of their 132
        // and 134 us).
        // The two products are exact, and y is rounded to fp32 once before it is to bf16: a
        // y whose last place differs from the definition's can flip a code.
        const double var = ss * a.inv_d + (double)a.eps;
        const int vx = __double2hiint(var) & 0x7FFFFFFF;
        const bool finite = vx < kDoubleInf;
        const int e = finite ? (((vx >> 20) - 1023) >> 1) + 1 : 0;
        const double m = __hiloint2double(vx - 2 * e * (1 << 20), __double2loint(var));
        const float p = __uint_as_float(e < 127 ? (uint32_t)(127 - e) << 23 : 0x00400000u >> (e - 127));   // 2^-e, e <= 128
        const float vh = (float)m, vl = (float)(m - (double)vh);
        const float r0 = rsqrtf(vh), h = vh * r0;
        const float res = fmaf(-h, r0, 1.f) - (fmaf(vh, r0, -h) + vl * r0) * r0;
        const float r1 = finite ? 0.5f * r0 * res : 0.f;   // an infinite mean keeps r0 = 0
#pragma unroll
        for (int i = 0; i < WPT; i++) {
            const int v = i * gt + ti;
            if (v < nw) {
                const v16 wv = load16(a.weight + 16 * v, a.al32);
                u[i].lo = scale_bf16x8(u[i].lo, wv.lo, p, r0, r1);
                u[i].hi = scale_bf16x8(u[i].hi, wv.hi, p, r0, r1);
                if (OUT == NORM_BF16 || a.y) store16(a.y + base + 16 * v, u[i], a.al32);
            }
        }
    }
    if (OUT == NORM_FP8) {
        uint4* qr = reinterpret_cast<uint4*>(a.q + base);
#pragma unroll
        for (int i = 0; i < WPT; i++) {
            const int v = i * gt + ti;
            const int e = e4m3_block_exp(u[i]);
            if (v < nw) {
                const uint2 p = e4m3_codes8(u[i].lo, e), q = e4m3_codes8(u[i].hi, e);
                qr[v] = make_uint4(p.x, p.y, q.x, q.y);
                if ((ti & 7) == 0) a.scale[row * (a.d / 128) + (v >> 3)] = pow2f(e);
            }
        }
    } else if (OUT == NORM_INT8) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < WPT; i++) m = max(m, max(amax_bits8(u[i].lo), amax_bits8(u[i].hi)));
        m = group_umax(m, s_max + group * warps, group, warps);
        const Int8Scale sc = int8_scale(m);
        uint4* qr = reinterpret_cast<uint4*>(a.q + base);
#pragma unroll
        for (int i = 0; i < WPT; i++) {
            const int v = i * gt + ti;
            if (v < nw) {
                const uint2 p = int8_codes8(u[i].lo, sc.inv), q = int8_codes8(u[i].hi, sc.inv);
                qr[v] = make_uint4(p.x, p.y, q.x, q.y);
            }
        }
        if (ti == 0) a.scale[row] = sc.scale;
    }
}

// ---------------------------------------------------------------- gradient
// With n = s * rstd, g = dy * w, m = mean(g * n):
//   ds = (g - n * m) * rstd (+ dxsum, the stream's own gradient)   -> dx, bf16
//   dw = sum over rows of dy * n                                   -> fp32
// rstd is formed again from s, which is read anyway.  Each group walks the rows
// group, group + groups, ... and keeps its columns' dw in registers; a CTA adds
// its groups and writes one row of partials[CTA][d], and norm_dw_kernel adds the
// CTAs, all in a fixed order: no atomics, the same bits in every run.  A single
// CTA writes its row to dweight itself.
struct NormGradArgs {
    const bf16* dy;
    const bf16* s;
    const bf16* weight;
    const bf16* dxsum;      // may be null
    bf16* dx;               // may be dy or dxsum
    float* partials;        // [CTAs, d]
    int64_t T;
    int d;
    float eps;
};

// Layout of the gradient's rows: 2 vectors a thread up to d = 4096 and 4 above,
// so that a row takes at most 512 threads up to d = 16384 and a thread may hold
// 128 registers (its columns' dw are 8 a vector).  Wider rows take 1024 threads
// of 64 registers, which then read the weight again for every row.  Measured
// (T=4099, scalar arithmetic): d=7168 44.7 us with 4 vectors, 48.7 with 2, 66.7
// with 1 -- the sums over a row cost every warp the same, so few warps with much
// of the row each are better -- and d=2048 17.4 with 2, 20.2 with 4, where a row
// is short.
__host__ __device__ inline RowShape norm_grad_shape(int d) { return row_shape(d / 8, d <= 4096 ? 2 : 4); }

// Rows in flight a group: every thread copies its own vectors of s, dy and dxsum
// into its own slots of shared memory (cp.async, no barrier), `stages` rows deep.
// Two CTAs an SM share about 200 KB, so a CTA takes as many stages as fit 100 KB,
// at most 4, and one that needs more than that for two runs alone on its SM.
// Without the copies ahead (loads straight into registers) an SM's loads stop
// while its rows are reduced: T=4099 d=7168 78 us.
__host__ __device__ inline int norm_grad_stage_bytes(const RowShape& s) { return s.groups * s.warps * 32 * s.vpt * 48; }

__host__ __device__ inline int norm_grad_stages(const RowShape& s)
{
    const int bytes = norm_grad_stage_bytes(s);
    const int n = 100 * 1024 / bytes;
    return n >= 4 ? 4 : n >= 2 ? n : 2 * bytes <= 200 * 1024 ? 2 : 1;
}

// CTAs of a launch: two a B200 SM where their rows fit (T=4099 d=7168: 44.7 us
// against 58.0 with one and twice the stages), one where they do not (T=1024
// d=16384: 28.8 us against 35.7 with two in turn).  Fixed numbers, so that the
// workspace and every bit of the result follow from the sizes alone.
constexpr int kNormGradCtas = 296;

__host__ __device__ inline int64_t norm_grad_ctas(int64_t T, int d)
{
    const RowShape s = norm_grad_shape(d);
    const int most = norm_grad_stages(s) * norm_grad_stage_bytes(s) <= 110 * 1024 ? kNormGradCtas : kNormGradCtas / 2;
    const int64_t ctas = (T + s.groups - 1) / s.groups;
    return ctas < most ? ctas : most;
}

constexpr int kNormGradSmemBytes = 200 * 1024;   // the most any shape takes (d = 16384: two stages of 512 x 4 vectors)

// A row's sums in 64 bits, for one whose sums left fp32 (the same for its whole group).
// `mine`: this thread's vectors of s, then of dy, blockDim.x apart.  Loops that are not unrolled
// leave the common path its registers; with more than 512 threads, which have 64 each,
// it is inlined (T=256 d=32768 30.4 us against 32.5 by a call), else called (T=4099
// d=2048 15.6 us against 16.6 inlined).
template <int VPT>
__device__ __forceinline__ double2 norm_grad_sums64(const uint4* mine, const bf16* weight, int d, int warps)
{
    __shared__ double slot[2][32];
    const int nt = (int)blockDim.x, nvec = d / 8, gt = warps * 32;
    const int group = (int)threadIdx.x / gt, ti = (int)threadIdx.x - group * gt;
    double ss = 0.0, dot = 0.0;
#pragma unroll 1
    for (int i = 0; i < VPT; i++) {
        if (i * gt + ti >= nvec) continue;
#pragma unroll 1
        for (int j = 0; j < 4; j++) {
            const float2 s = f2_get(f2_bf16(reinterpret_cast<const uint32_t*>(mine + i * nt)[j]));
            const float2 g = f2_get(f2_bf16(reinterpret_cast<const uint32_t*>(mine + (VPT + i) * nt)[j]));
            const float2 w = f2_get(f2_bf16(__ldg(reinterpret_cast<const uint32_t*>(weight) + 4 * (i * gt + ti) + j)));
            ss += (double)s.x * s.x + (double)s.y * s.y;
            dot += (double)g.x * w.x * s.x + (double)g.y * w.y * s.y;
        }
    }
    // the scratch was last read before the barrier of this row's fp32 sums
    ss = group_sum(ss, slot[0] + group * warps, group, warps);
    dot = group_sum(dot, slot[1] + group * warps, group, warps);
    return make_double2(ss, dot);
}

template <int VPT>
__device__ __noinline__ double2 norm_grad_sums64_call(const uint4* mine, const bf16* weight, int d, int warps)
{
    return norm_grad_sums64<VPT>(mine, weight, d, warps);
}

template <int VPT, int MAXT>
__global__ void __launch_bounds__(MAXT) rmsnorm_grad_kernel(const NormGradArgs a, int warps, int stages)
{
    extern __shared__ __align__(16) uint8_t s_rows[];
    __shared__ float s_red[2][2][32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int gt = warps * 32;
    const int per_cta = (int)blockDim.x / gt;
    const int group = (int)threadIdx.x / gt, ti = (int)threadIdx.x - group * gt;
    const int64_t stride = (int64_t)gridDim.x * per_cta, g0 = (int64_t)blockIdx.x * per_cta + group;
    const int nvec = a.d / 8;
    const int nt = blockDim.x;
    uint4* slots = reinterpret_cast<uint4*>(s_rows) + threadIdx.x;    // [stage][tensor][i] of this thread, nt apart
    constexpr bool kKeepW = MAXT <= 512;
    auto weight = [&](int i) {
        const int v = i * gt + ti;
        return v < nvec ? __ldg(reinterpret_cast<const uint4*>(a.weight) + v) : make_uint4(0u, 0u, 0u, 0u);
    };
    f2 dw[VPT][4];
    uint4 w[kKeepW ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        if (kKeepW) w[i] = weight(i);
#pragma unroll
        for (int j = 0; j < 4; j++) dw[i][j] = f2_of(0.f, 0.f);
    }
    auto fetch = [&](int64_t row, int st) {
        if (row < a.T) {
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int v = i * gt + ti;
                if (v < nvec) {
                    uint4* p = slots + (st * 3 * VPT + i) * nt;
                    ptx::cp_async16(p, reinterpret_cast<const uint4*>(a.s + row * a.d) + v);
                    ptx::cp_async16(p + VPT * nt, reinterpret_cast<const uint4*>(a.dy + row * a.d) + v);
                    if (a.dxsum) ptx::cp_async16(p + 2 * VPT * nt, reinterpret_cast<const uint4*>(a.dxsum + row * a.d) + v);
                }
            }
        }
        ptx::cp_async_commit();      // an empty group past the last row keeps the count
    };
    for (int st = 0; st < stages - 1; st++) fetch(g0 + st * stride, st);
    int par = 0, st = 0;
    for (int64_t row = g0; row < a.T; row += stride, par ^= 1) {
        // the slot of the row before last is free: this thread has used its values
        fetch(row + (stages - 1) * stride, st == 0 ? stages - 1 : st - 1);
        ptx::cp_async_wait(stages - 1);
        const uint4* mine = slots + st * 3 * VPT * nt;
        if (++st == stages) st = 0;
        f2 ss2 = f2_of(0.f, 0.f), dot2 = f2_of(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            if (i * gt + ti >= nvec) continue;
            const w4 s = words(mine[i * nt]), g = words(mine[(VPT + i) * nt]), wf = words(kKeepW ? w[i] : weight(i));
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const f2 sv = f2_bf16(s.w[j]);
                ss2 = f2_fma(sv, sv, ss2);
                dot2 = f2_fma(f2_mul(f2_bf16(g.w[j]), f2_bf16(wf.w[j])), sv, dot2);
            }
        }
        const float2 sp = f2_get(ss2), dp = f2_get(dot2);
        float ss = sp.x + sp.y, dot = dp.x + dp.y;
        // both sums through one barrier; the scratch alternates from row to row
        ss = warp_sum(ss);
        dot = warp_sum(dot);
        if (warps > 1) {
            const int lane = threadIdx.x & 31, wi = (int)(threadIdx.x >> 5);
            if (lane == 0) {
                s_red[par][0][wi] = ss;
                s_red[par][1][wi] = dot;
            }
            group_barrier(group, warps);
            ss = warp_sum(lane < warps ? s_red[par][0][group * warps + lane] : 0.f);
            dot = warp_sum(lane < warps ? s_red[par][1][group * warps + lane] : 0.f);
        }
        float rstd = rsqrtf(ss / (float)a.d + a.eps);
        float m = dot * rstd / (float)a.d;            // mean(g * n)
        // a sum beyond fp32 (a value above 1.8e19, or a product of the three), or squares
        // below it that count because eps is as small
        if (!(ss <= kMaxFloat && fabsf(m) <= kMaxFloat) || (ss < 0x1p-80f && a.eps < 0x1p-110f)) {
            const double2 q = MAXT > 512 ? norm_grad_sums64<VPT>(mine, a.weight, a.d, warps)
                                         : norm_grad_sums64_call<VPT>(mine, a.weight, a.d, warps);
            const double r = 1.0 / sqrt(q.x / (double)a.d + (double)a.eps);
            rstd = (float)r;
            m = (float)(q.y * r / (double)a.d);
        }
        const f2 rstd2 = f2_of(rstd, rstd), mneg2 = f2_of(-m, -m);
#pragma unroll
        for (int i = 0; i < VPT; i++) {
            const int v = i * gt + ti;
            if (v >= nvec) continue;
            const w4 s = words(mine[i * nt]), g = words(mine[(VPT + i) * nt]), wf = words(kKeepW ? w[i] : weight(i));
            w4 r{{0u, 0u, 0u, 0u}}, o;
            if (a.dxsum) r = words(mine[(2 * VPT + i) * nt]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const f2 gv = f2_bf16(g.w[j]), n = f2_mul(f2_bf16(s.w[j]), rstd2);
                const f2 t = f2_fma(n, mneg2, f2_mul(gv, f2_bf16(wf.w[j])));
                o.w[j] = f2_pack(f2_fma(t, rstd2, f2_bf16(r.w[j])));
                dw[i][j] = f2_fma(gv, n, dw[i][j]);
            }
            reinterpret_cast<uint4*>(a.dx + row * a.d)[v] = make_uint4(o.w[0], o.w[1], o.w[2], o.w[3]);
        }
    }
    ptx::cp_async_wait(0);
    float* part = a.partials + (int64_t)blockIdx.x * a.d;
    if (per_cta > 1) {
        // the groups one after the other, into the row buffer: nothing of it is in use any more
        float* sum = reinterpret_cast<float*>(s_rows);
        for (int g = 0; g < per_cta; g++) {
            __syncthreads();
            if (g != group) continue;
#pragma unroll
            for (int i = 0; i < VPT; i++) {
                const int v = i * gt + ti;
                if (v >= nvec) continue;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    f2* at = reinterpret_cast<f2*>(sum) + 4 * v + j;
                    if (g > 0) dw[i][j] = f2_add(dw[i][j], *at);
                    *at = dw[i][j];
                }
            }
        }
        if (group != per_cta - 1) return;      // the last group holds the total
    }
#pragma unroll
    for (int i = 0; i < VPT; i++) {
        const int v = i * gt + ti;
        if (v < nvec) {
            ulonglong2* p = reinterpret_cast<ulonglong2*>(part) + 2 * v;
            p[0] = make_ulonglong2(dw[i][0], dw[i][1]);
            p[1] = make_ulonglong2(dw[i][2], dw[i][3]);
        }
    }
}

// dweight[c] = sum over CTAs of partials[g][c], in a fixed order: a CTA of 512
// threads takes 32 columns, 16 threads a column each every 16th row (at most 19,
// loads in flight together), then those 16 sums in order.
__global__ void __launch_bounds__(512) norm_dw_kernel(const float* __restrict__ partials, int rows, int d,
                                                      float* __restrict__ dweight)
{
    __shared__ float s_part[16][33];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int cx = threadIdx.x & 31, gy = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + cx;      // d % 32 == 0
    float v[(kNormGradCtas + 15) / 16];
#pragma unroll
    for (int i = 0; i < (kNormGradCtas + 15) / 16; i++) {
        const int g = 16 * i + gy;
        v[i] = g < rows ? partials[(int64_t)g * d + c] : 0.f;
    }
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < (kNormGradCtas + 15) / 16; i++) acc += v[i];
    s_part[gy][cx] = acc;
    __syncthreads();
    if (gy == 0) {
        float t = s_part[0][cx];
#pragma unroll
        for (int i = 1; i < 16; i++) t += s_part[i][cx];
        dweight[c] = t;
    }
}

}  // namespace moe

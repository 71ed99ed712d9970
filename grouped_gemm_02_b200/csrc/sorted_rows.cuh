// sorted_rows.cuh -- rows sorted by expert and back with the gates applied, and
// the gradient of both.
//
//   sort        xpq[pos] = xq[t], sxp[pos] = sx[t]           pos = inv_perm[t k + j]
//   back        out[t]   = sum_j w[t, j] y_p[pos] (+ shared[t])
//   back'       dy_p[pos] = w[t, j] dout[t],   dw[t, j] = <dout[t], y_p[pos]>
//   sort'       dx[t]    = sum_j dxp[pos] (+ addend[t])
//
// A pair without a position (inv_perm outside [0, T k): its expert id was out
// of range) adds nothing, gets dw = 0, and no row is written for it.  Sums are
// fp32 in ascending j (a dot product in a fixed tree), no atomics; rows are
// rounded to bf16 once.
//
// Bound: HBM (2 P d bytes a pass over the sorted rows).  All kernels walk tokens
// in order, so the token's own row is read or written once for its k pairs.
#pragma once

#include "common.cuh"
#include "norm.cuh"
#include "permute.cuh"
#include "ptx.cuh"

namespace moe {

// Position of pair q, or -1 where it has none.
__device__ __forceinline__ int pair_pos(const int32_t* inv_perm, int64_t q, int64_t P)
{
    const int pos = __ldg(inv_perm + q);
    return (pos >= 0 && pos < P) ? pos : -1;
}

// ---------------------------------------------------------------- sort: positions
// Stable positions of up to kSortPairs pairs in two launches, 1024 pairs a CTA:
//   chunk_hist_kernel   hist[b][e] = pairs of expert e in chunk b
//   chunk_rank_kernel   every CTA adds up hist for itself: an expert's total (and
//                       from the totals its offset) and its pairs in earlier
//                       chunks; then pos = offset + earlier + rank in the chunk
// A chunk's CTA reads all of hist (chunks x E counts, from L2), which takes the
// place of a scan in a launch of its own; past kSortPairs that costs more than
// the scan and the general path (run_permute) runs.
constexpr int kSortChunk = 1024;
constexpr int64_t kSortPairs = int64_t(1) << 18;

__host__ __device__ inline int sort_chunks(int64_t P) { return (int)((P + kSortChunk - 1) / kSortChunk); }

__global__ void __launch_bounds__(kSortChunk) chunk_hist_kernel(const int32_t* __restrict__ idx, int P, int E,
                                                                int32_t* __restrict__ hist, uint32_t* __restrict__ err)
{
    __shared__ int32_t cnt[kMaxExperts];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int tid = threadIdx.x, q = blockIdx.x * kSortChunk + tid;
    const int e = q < P ? idx[q] : -1;
    if (tid < E) cnt[tid] = 0;
    __syncthreads();
    const bool in = e >= 0 && e < E;
    if (q < P && !in) atomicOr(err, DEVERR_EXPERT_RANGE);
    // one addition for the lanes that share an expert: a hot expert takes most of a chunk
    const unsigned peers = __match_any_sync(0xffffffffu, in ? e : -1);
    if (in && (tid & 31) == __ffs(peers) - 1) atomicAdd(&cnt[e], __popc(peers));
    __syncthreads();
    if (tid < E) hist[blockIdx.x * E + tid] = cnt[tid];
}

__global__ void __launch_bounds__(kSortChunk) chunk_rank_kernel(const int32_t* __restrict__ idx, int P, int E,
                                                                const int32_t* __restrict__ hist, int chunks,
                                                                int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ perm,
                                                                int32_t* __restrict__ inv_perm)
{
    __shared__ __align__(16) uint8_t s_wcnt[32][kMaxExperts];   // pairs of a warp (at most 32) by expert
    __shared__ int s_sum[2][kSortChunk];
    __shared__ int s_base[kMaxExperts];
    __shared__ int warp_sums[32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, chunk = blockIdx.x;
    const int q = chunk * kSortChunk + tid;
    int e = q < P ? idx[q] : -1;
    if (e < 0 || e >= E) {
        if (q < P) inv_perm[q] = -1;
        e = -1;
    }
    reinterpret_cast<uint4*>(&s_wcnt[0][0])[tid] = make_uint4(0, 0, 0, 0);   // 1024 x 16 B = the whole table
    // totals and earlier pairs by expert: `parts` threads an expert, each every parts-th chunk
    int e2 = 32;
    while (e2 < E) e2 *= 2;
    const int parts = kSortChunk / e2, pe = tid & (e2 - 1), pp = tid / e2;
    int total = 0, before = 0;
    if (pe < E) {
#pragma unroll 4
        for (int b = pp; b < chunks; b += parts) {
            const int v = __ldg(hist + b * E + pe);
            total += v;
            before += b < chunk ? v : 0;
        }
    }
    s_sum[0][tid] = total;
    s_sum[1][tid] = before;
    __syncthreads();
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (e >= 0 && lane == __ffs(peers) - 1) s_wcnt[warp][e] = (uint8_t)__popc(peers);
    total = before = 0;
    if (tid < E) {
        for (int i = 0; i < parts; i++) {
            total += s_sum[0][i * e2 + tid];
            before += s_sum[1][i * e2 + tid];
        }
    }
    const int incl = block_inclusive_scan(total, warp_sums);
    if (tid < E) {
        s_base[tid] = incl - total + before;
        if (chunk == 0) {
            counts[tid] = total;
            offsets[tid] = incl - total;
            if (tid == E - 1) offsets[E] = incl;
        }
    }
    __syncthreads();
    if (e >= 0) {
        int pos = s_base[e] + rank;
        for (int w = 0; w < warp; w++) pos += s_wcnt[w][e];
        perm[pos] = q;
        inv_perm[q] = pos;
    }
}

// ---------------------------------------------------------------- sort: int8 rows with a scale each
// Copies chunk c of token t's row (512 bytes: a 16-byte vector a lane) to its
// pairs' positions; the first chunk's warp also writes the scales.  `mine`: the
// position of pair t k + lane, or -1.
__device__ __forceinline__ void copy_row_chunk(const uint8_t* __restrict__ xq, const float* __restrict__ sx, int64_t t,
                                               int c, int mine, int k, int d, uint8_t* __restrict__ xpq,
                                               float* __restrict__ sxp)
{
    const int v = c * 32 + (int)(threadIdx.x & 31), nvec = d / 16;
    uint4 buf = make_uint4(0u, 0u, 0u, 0u);
    if (v < nvec) buf = __ldg(reinterpret_cast<const uint4*>(xq + t * d) + v);
    if (c == 0 && mine >= 0) sxp[mine] = sx[t];
    for (int j = 0; j < k; j++) {
        const int pos = __shfl_sync(0xffffffffu, mine, j);
        if (pos >= 0 && v < nvec) reinterpret_cast<uint4*>(xpq + (int64_t)pos * d)[v] = buf;
    }
}

// One warp per (token, chunk).
__global__ void __launch_bounds__(256) gather_rows_int8_kernel(const uint8_t* __restrict__ xq,
                                                               const float* __restrict__ sx,
                                                               const int32_t* __restrict__ inv_perm, int64_t T, int k,
                                                               int d, uint8_t* __restrict__ xpq,
                                                               float* __restrict__ sxp)
{
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int nch = (d / 16 + 31) / 32;
    const int lane = threadIdx.x & 31;
    const int64_t items = T * nch, P = T * k;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32; w < items;
         w += (int64_t)gridDim.x * blockDim.x / 32) {
        const int64_t t = w / nch;
        const int mine = lane < k ? pair_pos(inv_perm, t * k + lane, P) : -1;
        copy_row_chunk(xq, sx, t, (int)(w - t * nch), mine, k, d, xpq, sxp);
    }
}

// At most 1024 pairs (one a thread): the whole sort in one launch.  Every CTA
// finds all positions for itself -- a second launch would cost more than the
// repeated ranking -- and copies its share of the rows; CTA 0 also writes the
// index arrays and reports bad expert ids.
__global__ void __launch_bounds__(kSortChunk) sort_small_kernel(const int32_t* __restrict__ idx,
                                                                const uint8_t* __restrict__ xq,
                                                                const float* __restrict__ sx, int T, int k, int d,
                                                                int E, int32_t* __restrict__ counts,
                                                                int32_t* __restrict__ offsets,
                                                                int32_t* __restrict__ perm,
                                                                int32_t* __restrict__ inv_perm,
                                                                uint8_t* __restrict__ xpq, float* __restrict__ sxp,
                                                                uint32_t* __restrict__ err)
{
    __shared__ __align__(16) uint8_t s_wcnt[32][kMaxExperts];   // pairs of a warp (at most 32) by expert
    __shared__ int s_off[kMaxExperts];
    __shared__ int s_pos[kSortChunk];
    __shared__ int warp_sums[32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int P = T * k;
    const bool first = blockIdx.x == 0;
    int e = tid < P ? idx[tid] : -1;
    const bool bad = tid < P && (e < 0 || e >= E);
    if (bad) e = -1;
    if (bad && first) atomicOr(err, DEVERR_EXPERT_RANGE);
    reinterpret_cast<uint4*>(&s_wcnt[0][0])[tid] = make_uint4(0, 0, 0, 0);   // 1024 x 16 B = the whole table
    __syncthreads();
    const unsigned peers = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(peers & ((1u << lane) - 1u));
    if (e >= 0 && lane == __ffs(peers) - 1) s_wcnt[warp][e] = (uint8_t)__popc(peers);
    __syncthreads();
    const int warps = (P + 31) / 32;
    int total = 0;
    if (tid < E)
        for (int w = 0; w < warps; w++) total += s_wcnt[w][tid];
    const int incl = block_inclusive_scan(total, warp_sums);
    if (tid < E) {
        s_off[tid] = incl - total;
        if (first) {
            counts[tid] = total;
            offsets[tid] = incl - total;
            if (tid == E - 1) offsets[E] = incl;
        }
    }
    __syncthreads();
    int pos = -1;
    if (e >= 0) {
        pos = s_off[e] + rank;
        for (int w = 0; w < warp; w++) pos += s_wcnt[w][e];
        if (first) perm[pos] = tid;
    }
    s_pos[tid] = pos;
    if (first && tid < P) inv_perm[tid] = pos;
    __syncthreads();
    const int nch = (d / 16 + 31) / 32, items = T * nch;
    // dealt over the CTAs first: few rows are then written by many SMs
    for (int w = warp * gridDim.x + blockIdx.x; w < items; w += gridDim.x * 32) {
        const int t = w / nch;
        const int mine = lane < k ? s_pos[t * k + lane] : -1;
        copy_row_chunk(xq, sx, t, w - t * nch, mine, k, d, xpq, sxp);
    }
}

// ---------------------------------------------------------------- back, and the gradient of sort
// out[t] = sum_j w[t, j] rows[pos] + add[t]; w null: weights 1.  k <= KM (k rounded up
// to 1, 2, 4 or 8), and a thread takes V = 8 / KM vectors of a token's row, so that
// 5 to 8 loads of 16 bytes are in flight together (with one vector a thread k = 1
// reached 30% of the bytes that k = 8 did: T=4093 d=7168 60 us against 17).  BRIEF:
// short rows, a warp a token and four tokens a CTA; otherwise a CTA has one token, whose
// positions and gates are then the same registers for every thread (a wide row is cut
// over several CTAs, and each reads them).
// add and out may be the same buffer (no __restrict__, no read-only loads): a vector
// is read and then written by the same thread.  Reading a thread's vectors of add
// ahead takes registers from calls without it (T=4093 d=7168 k=1 18.6 us against 16.6;
// with add 27.0 against 33.3).
template <int KM, bool BRIEF>
__global__ void __launch_bounds__(BRIEF ? 128 : 64) return_rows_kernel(const bf16* __restrict__ rows,
                                                         const int32_t* __restrict__ inv_perm,
                                                         const float* __restrict__ gates, const bf16* add,
                                                         int64_t T, int k, int d, bf16* out)
{
    constexpr int V = kMaxTopK / KM;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int nvec = d / 8;
    const int64_t P = T * k;
    const int64_t t = BRIEF ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    if (BRIEF && t >= T) return;
    int pos[KM];
    float w[KM];
#pragma unroll
    for (int j = 0; j < KM; j++) {
        pos[j] = j < k ? pair_pos(inv_perm, t * k + j, P) : -1;
        w[j] = (j < k && gates) ? __ldg(gates + t * k + j) : 1.f;
    }
    const int v0 = blockIdx.y * (blockDim.x * V) + threadIdx.x;
    uint4 u[V][KM];
#pragma unroll
    for (int i = 0; i < V; i++)
#pragma unroll
        for (int j = 0; j < KM; j++)
            if (pos[j] >= 0 && v0 + i * (int)blockDim.x < nvec)
                u[i][j] = __ldg(reinterpret_cast<const uint4*>(rows + (int64_t)pos[j] * d) + v0 + i * blockDim.x);
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int v = v0 + i * blockDim.x;
        if (v >= nvec) continue;
        f8 acc;
#pragma unroll
        for (int c = 0; c < 8; c++) acc.v[c] = 0.f;
#pragma unroll
        for (int j = 0; j < KM; j++) {
            if (pos[j] >= 0) {
                const f8 r = unpack8(u[i][j]);
#pragma unroll
                for (int c = 0; c < 8; c++) acc.v[c] = fmaf(w[j], r.v[c], acc.v[c]);
            }
        }
        if (add) {
            const f8 r = unpack8(reinterpret_cast<const uint4*>(add + t * d)[v]);
#pragma unroll
            for (int c = 0; c < 8; c++) acc.v[c] += r.v[c];
        }
        reinterpret_cast<uint4*>(out + t * d)[v] = pack8(acc);
    }
}

// ---------------------------------------------------------------- gradient of back
// The threads of a token hold V = 8 / KM vectors of its gradient row at a time, write
// each pair's scaled copy and add up the k dot products.  BRIEF: as above.
// rows and drows may be the same buffer (no __restrict__, no read-only loads):
// a vector is read and then written by the same thread.
template <int KM, int MAXT, bool BRIEF = false>
__global__ void __launch_bounds__(MAXT)
    return_rows_grad_kernel(const bf16* __restrict__ dout, const bf16* rows, const int32_t* __restrict__ inv_perm,
                            const float* __restrict__ gates, int64_t T, int k, int d, bf16* drows,
                            float* __restrict__ dgates)
{
    constexpr int V = kMaxTopK / KM;
    __shared__ float s_dot[KM][MAXT / 32];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int64_t P = T * k;
    const int64_t t = BRIEF ? (int64_t)blockIdx.x * blockDim.y + threadIdx.y : blockIdx.x;
    const int warps = (int)(blockDim.x >> 5), lane = threadIdx.x & 31;     // warps of a token
    const int first = BRIEF ? threadIdx.y * warps : 0, warp = first + (int)(threadIdx.x >> 5);
    const bool live = !BRIEF || t < T;
    const int nvec = live ? d / 8 : 0;
    int pos[KM];
    float w[KM], dot[KM];
#pragma unroll
    for (int j = 0; j < KM; j++) {
        pos[j] = live && j < k ? pair_pos(inv_perm, t * k + j, P) : -1;
        w[j] = live && j < k ? __ldg(gates + t * k + j) : 0.f;
        dot[j] = 0.f;
    }
    for (int v0 = threadIdx.x; v0 < nvec; v0 += V * blockDim.x) {
        uint4 u[V][KM], ug[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int v = v0 + i * blockDim.x;
            if (V == 1 || v < nvec) {
#pragma unroll
                for (int j = 0; j < KM; j++)
                    if (pos[j] >= 0) u[i][j] = reinterpret_cast<const uint4*>(rows + (int64_t)pos[j] * d)[v];
                ug[i] = __ldg(reinterpret_cast<const uint4*>(dout + t * d) + v);
            }
        }
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int v = v0 + i * blockDim.x;
            if (V > 1 && v >= nvec) continue;
            const f8 g = unpack8(ug[i]);
#pragma unroll
            for (int j = 0; j < KM; j++) {
                if (pos[j] >= 0) {
                    const f8 r = unpack8(u[i][j]);
                    f8 o;
#pragma unroll
                    for (int c = 0; c < 8; c++) {
                        dot[j] = fmaf(g.v[c], r.v[c], dot[j]);
                        o.v[c] = w[j] * g.v[c];
                    }
                    reinterpret_cast<uint4*>(drows + (int64_t)pos[j] * d)[v] = pack8(o);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KM; j++) {
        const float s = warp_sum(dot[j]);
        if (lane == 0) s_dot[j][warp] = s;
    }
    __syncthreads();
    if (live && (int)threadIdx.x < k) {
        float s = s_dot[threadIdx.x][first];
        for (int i = 1; i < warps; i++) s += s_dot[threadIdx.x][first + i];
        dgates[t * k + threadIdx.x] = s;
    }
}

}  // namespace moe

// Shared pieces of the attention with a learned relative position bias: the
// bias table a CTA keeps in shared memory, the split of the work over CTAs, and
// the layout of the table gradient's partial sums.
//
// The bias of head h is T[h][bucket], the bucket given by the displacement
// (i_t - i_u, j_t - j_u) of query t and key u inside their window: displacement
// index (i_t - i_u + M - 1) (2M - 1) + (j_t - j_u + M - 1), sent through the
// caller's bucket map, or taken as the bucket itself without one (Swin's table).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "geometry.cuh"
#include "kernels.cuh"

namespace fswin {

namespace relb {

constexpr int kSms = 148;  // SMs of a B200: bounds the CTAs, and with them the partial sums in the workspace

// Row pitch (fp32 words) of the bias table in shared memory.  Row threads of a
// warp hold 32 consecutive slots, boxes of bw tokens a row, and read table words
// of their own (row, column) shifted by a common amount: bw consecutive words per
// box row.  A pitch of 16 (bw = 16) or 8 or 24 (bw <= 8) modulo 32 puts the box
// rows of a warp into different banks, so a warp's 32 reads take one pass.  At M =
// 64 the padded table would not fit beside the tiles.
__host__ __device__ constexpr int bias_pitch(int M, int bw) {
    int p = 2 * M - 1;
    if (bw >= 32 || M == 64) return p;
    if (bw == 16) {
        while (p % 32 != 16) ++p;
    } else {
        while (p % 32 != 8 && p % 32 != 24) ++p;
    }
    return p;
}

__host__ __device__ constexpr int displacements(int M) { return (2 * M - 1) * (2 * M - 1); }

// The head's table in the softmax's base-2 units.  A bucket outside the table
// adds no bias.  Finite entries are held within +-2^126, so that log2(e) times
// them stays finite and a row whose every entry is the type's lowest value is the
// uniform row it is in exact arithmetic; -inf stays -inf (the pair never attends).
__device__ __forceinline__ float bias_entry(const __nv_bfloat16* table_h, const int* buckets, int n_buckets, int delta) {
    const int b = buckets ? __ldg(buckets + delta) : delta;
    if (b < 0 || b >= n_buckets) return 0.f;
    float v = __bfloat162float(table_h[b]);
    if (!isinf(v)) v = v > 8.5e37f ? 8.5e37f : (v < -8.5e37f ? -8.5e37f : v);  // a NaN stays one
    return v * 1.4426950408889634f;
}

__device__ __forceinline__ void build_bias(float* tab, int pitch, const __nv_bfloat16* table_h, const int* buckets,
                                           int n_buckets, int M, int tid, int nt) {
    const int side = 2 * M - 1;
    for (int e = tid; e < side * side; e += nt) {
        const int y = e / side, x = e - y * side;
        tab[y * pitch + x] = bias_entry(table_h, buckets, n_buckets, e);
    }
}

// A row's log-sum-exp in base-2 units for the gradient's P = exp2(t - lse2).  +inf
// (no probability) for a row without a key, and for one whose every entry is so
// large that its log-sum-exp in fp32 no longer tells the row's scores apart.
__device__ __forceinline__ float grad_lse2(float lse) {
    const float v = lse * 1.4426950408889634f;
    return fabsf(v) > 1e30f ? INFINITY : v;  // a NaN stays one
}

// Every CTA serves one head (its table, and the table gradient it sums, belong to
// that head) and walks that head's tiles with the head's other CTAs.  Consecutive
// CTAs serve consecutive heads, so the heads of a tile, whose 64-byte rows are
// adjacent in memory, are read at about the same time.
__host__ inline int streams_per_head(long long tiles, int heads, int ctas) {
    long long n = ctas / heads;
    if (n < 1) n = 1;
    if (n > tiles) n = tiles;
    return static_cast<int>(n < 1 ? 1 : n);
}

// Table gradient: part[(k * heads + h)][displacement] of the CTA k of head h,
// summed over k in order, then over the displacements of each bucket in order.
cudaError_t launch_table_grad(const float* part, int streams, const Geo& g, const RelbPtrs& p, float* disp,
                              cudaStream_t stream);

cudaError_t launch_small_fwd(const Geo& g, const RelbPtrs& p, unsigned int* status, unsigned long long limit_ns,
                             int num_sms, cudaStream_t stream);
cudaError_t launch_small_bwd(const Geo& g, const RelbPtrs& p, float* part, int streams, unsigned int* status,
                             unsigned long long limit_ns, cudaStream_t stream);
// CTAs of a backward kernel for windows of fewer than 128 tokens.
__host__ inline int small_bwd_ctas(const Geo& g) { return (g.M == 8 ? 2 : 3) * kSms; }

}  // namespace relb

}  // namespace fswin

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
#include "ptx.cuh"

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
// uniform row it is in any floating-point type; -inf stays -inf (the pair never attends).
__device__ __forceinline__ float bias_entry(const __nv_bfloat16* table_h, const int* buckets, int n_buckets, int delta) {
    const int b = buckets ? __ldg(buckets + delta) : delta;
    if (b < 0 || b >= n_buckets) return 0.f;
    float v = __bfloat162float(table_h[b]);
    if (!isinf(v)) v = v > 8.5e37f ? 8.5e37f : (v < -8.5e37f ? -8.5e37f : v);  // a NaN stays one
    return v * 1.4426950408889634f;
}

// Beyond this magnitude (base 2) a log-sum-exp is a far one: the fp32 steps on the way to
// it are 2^-11 there, and the gradient's P = exp2(t - lse2) has them as a relative error.
// Up to here that is below 2^-11, a quarter of what P's rounding to bf16 may add; at 2^24
// it is a factor of two, at 2^31 zero or infinity.  An entry of half that makes a table a
// far one.
constexpr float kFar = 4096.f;
__device__ __forceinline__ bool finite_beyond(float v, float limit) { return fabsf(v) > limit && !isinf(v); }

// Returns whether this thread has met a far entry.
__device__ __forceinline__ bool build_bias(float* tab, int pitch, const __nv_bfloat16* table_h, const int* buckets,
                                           int n_buckets, int M, int tid, int nt) {
    const int side = 2 * M - 1;
    bool far = false;
    for (int e = tid; e < side * side; e += nt) {
        const int y = e / side, x = e - y * side;
        const float v = bias_entry(table_h, buckets, n_buckets, e);
        tab[y * pitch + x] = v;
        far |= finite_beyond(v, kFar / 2);
    }
    return far;
}

// A row's log-sum-exp in base-2 units for the gradient's P = exp2(t - lse2).  +inf
// (no probability) for a row without a key.
__device__ __forceinline__ float grad_lse2(float lse) {
    const float v = lse * 1.4426950408889634f;
    return fabsf(v) > 1e30f ? INFINITY : v;  // a NaN stays one
}

// s + the dot product of eight channels, in an order of its own: the same bits wherever
// the four chunks of two rows are added up.
__device__ __forceinline__ float add_chunk(float s, const uint4& a, const uint4& b) {
    const uint32_t as[4] = {a.x, a.y, a.z, a.w}, bs[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        s = fmaf(bf16lo_to_f32(as[e]), bf16lo_to_f32(bs[e]), fmaf(bf16hi_to_f32(as[e]), bf16hi_to_f32(bs[e]), s));
    return s;
}
// Rows of 64-byte-swizzled tiles in shared memory.
static __device__ __noinline__ float shared_dot(const uint8_t* tile_a, int a, const uint8_t* tile_b, int b) {
    float s = 0.f;
#pragma unroll 1
    for (int c = 0; c < 4; ++c)
        s = add_chunk(s, *reinterpret_cast<const uint4*>(tile_a + a * kRowBytes + ((c ^ ((a >> 1) & 3)) << 4)),
                      *reinterpret_cast<const uint4*>(tile_b + b * kRowBytes + ((c ^ ((b >> 1) & 3)) << 4)));
    return s;
}

// Rows whose every key has a large bias (the type's lowest value as a mask, say) have a
// log-sum-exp in which the sum of their exponentials is lost.  For them P = exp2((t - m) -
// log2 l) with the maximum m and the sum l of the row's own scores, formed again here, key
// by key on the CUDA cores: rare, so it may be slow.  The scores t that join them in P are
// formed in the same way (add_chunk), not taken from the tensor product: beside a bias of 1e9
// a score is rounded to multiples of 128, and where the two products round to different
// sides of such a step, a row's one key would weigh 2^128 or nothing.
// The result (x, y) stands for the two terms of log2 P = (t + x) + y; y < 0 marks a row that
// has them, also where l = 1.  A far log-sum-exp that the scores alone make (no far entry)
// stays what it is.  Where every row is such a one a backward takes 1.6 ms in place of 0.15
// (64 x 64 x 64 tokens, 3 heads, M = 8) or 23 in place of 0.98 (16 x 128 x 128, M = 32); with
// large entries but no such row 0.15 in place of 0.11 and 0.96 in place of 0.94.
// X, r: the row's tile and slot.  lse2: its log-sum-exp, far.
static __device__ __noinline__ float2 far_row(const Geo& g, const uint8_t* q, const uint8_t* k,
                                              const __nv_bfloat16* table_h, const int* buckets, int n_buckets,
                                              long long X, int r, int h, float lse2) {
    Win w = tile_win(g, X);
    const int widx = r >> (g.lnbw + g.lBT);
    if (widx) w = win_of(g, w.gw + widx);
    int pi, pj;
    tile_row_pos(g, X, r, &pi, &pj);
    auto row_at = [&](const uint8_t* base, int i, int j) -> const uint4* {  // null outside the grid
        int row = w.wr * g.M + i + g.s, col = w.wc * g.M + j + g.s;
        if (row >= g.Hp) row -= g.Hp;
        if (col >= g.Wp) col -= g.Wp;
        if (row >= g.H || col >= g.W) return nullptr;
        return reinterpret_cast<const uint4*>(
            base + (((static_cast<long long>(w.b) * g.H + row) * g.W + col) * g.heads + h) * kRowBytes);
    };
    const bool cut_i = g.s && (w.wr + 1) * g.M == g.Hp, cut_j = g.s && w.wc + 1 == g.nWw;
    const int edge = g.M - g.s;
    const uint4* mine = row_at(q, pi, pj);  // the row is a token
    float m = -INFINITY, l = 0.f;
    bool far = false;
    for (int u = 0; u < g.N; ++u) {
        const int i = u / g.M, j = u - i * g.M;
        if ((cut_i && (i >= edge) != (pi >= edge)) || (cut_j && (j >= edge) != (pj >= edge))) continue;
        const uint4* key = row_at(k, i, j);
        float s = 0.f;
        for (int c = 0; key && c < 4; ++c) s = add_chunk(s, __ldg(mine + c), __ldg(key + c));
        const float bias = bias_entry(table_h, buckets, n_buckets, (pi - i + g.M - 1) * (2 * g.M - 1) + pj - j + g.M - 1);
        far |= finite_beyond(bias, kFar / 2);
        const float t = fmaf(s, g.scale_log2, bias);
        if (t > m) {
            l = fmaf(l, ex2_approx(m - t), 1.f);
            m = t;
        } else if (t != -INFINITY) {
            l += ex2_approx(t - m);  // a NaN stays one
        }
    }
    if (!far) return make_float2(-grad_lse2(lse2 * 0.69314718055994530942f), 0.f);
    const float y = -lg2_approx(l);
    return fabsf(m) > kFar ? make_float2(-m, y == 0.f ? -1e-30f : y) : make_float2(y - m, 0.f);
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

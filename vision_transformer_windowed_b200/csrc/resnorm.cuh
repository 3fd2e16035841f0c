// The residual step of a layer: r = x + g_b gamma o drop(post(f)), n = pre(r),
// row by row.  Pieces shared by its forward and backward kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "geometry.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace fswin {

namespace resn {

enum : int { kNone = 0, kLayer = 1, kRms = 2 };

struct Params {
    ResnormPtrs p;
    unsigned int rows;
    int C;
    FastDiv tokens;     // rows of a sample
    int pre, post;
    float eps, inv_c, keep_scale;
    unsigned int thr;   // an element is dropped when its random word is below this
    int drop;
    float* part;        // backward: [parameter][block][C]
    float* rowdot;      // backward: per row dr . u (the gate's gradient)
    int blocks;
};

// ---------------------------------------------------------------- Philox4x32-10
// J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC11: ten rounds of two 32 x 32 -> 64 bit products.  Counter:
// (element / 4, offset), key: seed; element e takes word e mod 4.  The mask is a
// function of (seed, offset, element), so the backward draws it again and nothing
// is stored.
__device__ __forceinline__ uint4 philox(unsigned long long counter, unsigned long long offset, unsigned long long seed) {
    uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32);
    uint32_t c2 = static_cast<uint32_t>(offset), c3 = static_cast<uint32_t>(offset >> 32);
    uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
        const unsigned long long a = static_cast<unsigned long long>(c0) * 0xD2511F53u;
        const unsigned long long b = static_cast<unsigned long long>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
        c3 = static_cast<uint32_t>(a);
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
}

// ---------------------------------------------------------------- rows in registers
// A row is held by a group of L lanes, V chunks of W channels a lane: chunk
// lane + L i.  W = 8: 16-byte bf16 accesses (every tensor 16-byte aligned).  Where the
// channel count is no multiple of 8 a row starts `shift` elements behind a 16-byte
// boundary; its chunks then start at that boundary, and its first and last are
// partly another row's (read and written element by element).  A group only walks rows
// of one shift, so that its lanes always hold the same channels.  W = 1: tensors at any
// element.  Elements outside the row read as zero and are not written.  S: rows that
// may be shifted; the others' kernels are free of the element-wise accesses, which keep
// the loads of a row from being issued together (forward of 128 x 4096 rows of 96
// channels 80 -> 130 us with them).
template <int W, int L, int V, bool S>
struct Row {
    static constexpr int E = W * V;
    int col[V];
    int C;
    unsigned int full, edge;  // chunks wholly, and (S) partly, inside the row
    __device__ __forceinline__ void init(int lane, int channels, int shift) {
        C = channels;
        full = edge = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            col[i] = (lane + L * i) * W - (S ? shift : 0);
            if (col[i] >= 0 && col[i] + W <= C) full |= 1u << i;
            else if (S && col[i] + W > 0 && col[i] < C) edge |= 1u << i;
        }
    }
    __device__ __forceinline__ bool in(int e) const {  // element e of the lane's
        const int i = e / W;
        return ((full >> i) & 1u) || (S && ((edge >> i) & 1u) && col[i] + e % W >= 0 && col[i] + e % W < C);
    }

    __device__ __forceinline__ static void zero(float (&x)[E]) {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = 0.f;
    }

    // aligned: the row's chunks are 16-byte aligned in this tensor (parameters of a
    // shifted row are not)
    template <typename T>
    __device__ __forceinline__ void load(const T* row, float (&x)[E], bool aligned = true) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int e = 0; e < W; ++e) x[i * W + e] = 0.f;
            if constexpr (W == 1) {
                if ((full >> i) & 1u) x[i] = static_cast<float>(row[col[i]]);
            } else if (((full >> i) & 1u) && (!S || aligned)) {
                if constexpr (sizeof(T) == 2) {
                    const uint4 v = *reinterpret_cast<const uint4*>(row + col[i]);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[i * W + 2 * e] = bf16lo_to_f32(w[e]);
                        x[i * W + 2 * e + 1] = bf16hi_to_f32(w[e]);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float4 v = *reinterpret_cast<const float4*>(row + col[i] + 4 * q);
                        x[i * W + 4 * q] = v.x;
                        x[i * W + 4 * q + 1] = v.y;
                        x[i * W + 4 * q + 2] = v.z;
                        x[i * W + 4 * q + 3] = v.w;
                    }
                }
            } else if (S && (((full | edge) >> i) & 1u)) {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (col[i] + e >= 0 && col[i] + e < C) x[i * W + e] = static_cast<float>(row[col[i] + e]);
            }
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&x)[E], bool aligned = true) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float* y = x + i * W;
            if constexpr (W == 1) {
                if ((full >> i) & 1u) row[col[i]] = static_cast<T>(x[i]);
            } else if (((full >> i) & 1u) && (!S || aligned)) {
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<uint4*>(row + col[i]) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                                         pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
                } else {
                    *reinterpret_cast<float4*>(row + col[i]) = make_float4(y[0], y[1], y[2], y[3]);
                    *reinterpret_cast<float4*>(row + col[i] + 4) = make_float4(y[4], y[5], y[6], y[7]);
                }
            } else if (S && (((full | edge) >> i) & 1u)) {
#pragma unroll
                for (int e = 0; e < W; ++e)
                    if (col[i] + e >= 0 && col[i] + e < C) row[col[i] + e] = static_cast<T>(y[e]);
            }
        }
    }
    // v in elements of the row, 0 outside it.
    __device__ __forceinline__ float inside(int e, float v) const {
        if constexpr (S) return in(e) ? v : 0.f;
        else return ((full >> (e / W)) & 1u) ? v : 0.f;
    }

    // Bit e: element e of the lane's is kept.
    __device__ __forceinline__ uint32_t mask(const Params& prm, unsigned int row, unsigned long long seed,
                                             unsigned long long offset) const {
        static_assert(E <= 32, "a bit an element");
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // a partly foreign first chunk starts in the row before: row C + col is never negative
            const unsigned long long at = static_cast<unsigned long long>(static_cast<long long>(row) * prm.C + col[i]);
            if constexpr (W == 1) {
                const uint4 w = philox(at >> 2, offset, seed);
                const uint32_t s = static_cast<uint32_t>(at) & 3u;
                const uint32_t word = s == 0 ? w.x : (s == 1 ? w.y : (s == 2 ? w.z : w.w));
                if (word >= prm.thr) bits |= 1u << i;
            } else {  // chunks start at multiples of 8
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 w = philox((at >> 2) + q, offset, seed);
                    if (w.x >= prm.thr) bits |= 1u << (i * W + 4 * q);
                    if (w.y >= prm.thr) bits |= 2u << (i * W + 4 * q);
                    if (w.z >= prm.thr) bits |= 4u << (i * W + 4 * q);
                    if (w.w >= prm.thr) bits |= 8u << (i * W + 4 * q);
                }
            }
        }
        return bits;
    }
};
// x of the kept elements times keep_scale, 0 (whatever x holds) of the dropped ones.
template <int E>
__device__ __forceinline__ void drop(float (&x)[E], uint32_t bits, float keep_scale) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = (bits >> e) & 1u ? x[e] * keep_scale : 0.f;
}

// A bf16 row as it was loaded, until its values are wanted: half the registers.
template <int W, int L, int V, bool S>
struct Held {
    static constexpr bool kRaw = W == 8 && !S;
    uint4 raw[kRaw ? V : 1];
    float x[kRaw ? 1 : W * V];
    __device__ __forceinline__ void zero() {
        if constexpr (kRaw) {
#pragma unroll
            for (int i = 0; i < V; ++i) raw[i] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            Row<W, L, V, S>::zero(x);
        }
    }
    __device__ __forceinline__ void load(const Row<W, L, V, S>& g, const __nv_bfloat16* row) {
        if constexpr (kRaw) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                raw[i] = make_uint4(0u, 0u, 0u, 0u);
                if ((g.full >> i) & 1u) raw[i] = *reinterpret_cast<const uint4*>(row + g.col[i]);
            }
        } else {
            g.load(row, x);
        }
    }
    __device__ __forceinline__ void take(float (&y)[W * V]) const {
        if constexpr (kRaw) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    y[i * W + 2 * e] = bf16lo_to_f32(w[e]);
                    y[i * W + 2 * e + 1] = bf16hi_to_f32(w[e]);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < W * V; ++e) y[e] = x[e];
        }
    }
};

// A row of the stream, bf16 or fp32, likewise.
template <int W, int L, int V, bool S>
struct HeldF32 {
    float x[W * V];
    __device__ __forceinline__ void zero() { Row<W, L, V, S>::zero(x); }
    __device__ __forceinline__ void load(const Row<W, L, V, S>& g, const float* row) { g.load(row, x); }
    __device__ __forceinline__ void take(float (&y)[W * V]) const {
#pragma unroll
        for (int e = 0; e < W * V; ++e) y[e] = x[e];
    }
};
template <typename TX, int W, int L, int V, bool S>
using Stream = std::conditional_t<sizeof(TX) == 2, Held<W, L, V, S>, HeldF32<W, L, V, S>>;

constexpr int kThreads = 256;  // of a block, or L where a row takes more
template <int L>
__host__ __device__ constexpr int threads_of() {
    return L > kThreads ? L : kThreads;
}
template <int L>
__host__ __device__ constexpr int groups_of() {
    return threads_of<L>() / L;
}
// Shared floats of the row sums: one a warp.
constexpr int kScratch = 32;

// Sum of a value over the L lanes of a row, the same in every lane; groups of several
// warps meet at a barrier of their own.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (L > 32) {
        constexpr int kWarps = L / 32;
        const int group = threadIdx.x / L, warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) scratch[warp] = v;
        named_bar_sync(1 + group, L);
        v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += scratch[group * kWarps + w];
        named_bar_sync(1 + group, L);
    }
    return v;
}

// Normalises a row in place of `x` (chunks outside the row stay zero) and returns
// 1 / deviation: mean and centred squares in two passes over registers, so a large
// mean costs no digits.
template <int W, int L, int V, bool S>
__device__ __forceinline__ float normalise(const Row<W, L, V, S>& g, float (&x)[W * V], int kind, const Params& prm,
                                           float* scratch) {
    if (kind == kLayer) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < W * V; ++e) s += x[e];
        const float mean = row_sum<L>(s, scratch) * prm.inv_c;
#pragma unroll
        for (int e = 0; e < W * V; ++e) x[e] -= g.inside(e, mean);  // x is 0 outside
    }
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < W * V; ++e) q = fmaf(x[e], x[e], q);
    const float inv = rsqrtf(row_sum<L>(q, scratch) * prm.inv_c + prm.eps);
#pragma unroll
    for (int e = 0; e < W * V; ++e) x[e] *= inv;
    return inv;
}

// Blocks of the backward, each with a partial sum of the parameters' gradients:
// two a SM of a B200.
constexpr int kMaxBwdBlocks = 2 * 148;

// Rows of one shift follow each other at this distance: a row starts (row C) mod 8
// elements behind a 16-byte boundary.
inline unsigned int shift_period(int C) { return C % 8 == 0 ? 1u : (C % 4 == 0 ? 2u : (C % 2 == 0 ? 4u : 8u)); }

// Blocks for `rows` rows, `groups` a block: at most `most` (rounded down), a multiple of
// what keeps every group at one shift.
inline unsigned int grid_of(unsigned int rows, int groups, unsigned int most, int C) {
    const unsigned int period = shift_period(C), step = period / static_cast<unsigned>(groups) > 1 ? period / groups : 1u;
    unsigned int n = (rows + groups - 1) / groups;
    n = (n + step - 1) / step * step;
    const unsigned int cap = most / step * step;
    return n < cap ? n : cap;
}

inline void fill_params(const ResnormShape& sh, const ResnormPtrs& p, Params* out) {
    out->p = p;
    out->p.samples = sh.samples;
    out->rows = static_cast<unsigned int>(sh.samples * sh.tokens);
    out->C = sh.channels;
    out->tokens = make_fastdiv(static_cast<uint32_t>(sh.tokens > 0 ? sh.tokens : 1));
    out->pre = sh.pre;
    out->post = sh.post;
    out->eps = sh.eps;
    out->inv_c = 1.f / static_cast<float>(sh.channels);
    out->drop = sh.drop_p > 0.0;
    out->thr = static_cast<unsigned int>(sh.drop_p * 4294967296.0);
    out->keep_scale = static_cast<float>(1.0 / (1.0 - sh.drop_p));
}

}  // namespace resn

}  // namespace fswin

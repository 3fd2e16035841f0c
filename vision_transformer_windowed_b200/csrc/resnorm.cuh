// The residual step of a layer: r = x + g_b gamma o drop(post(f)), n = pre(r),
// row by row.  Pieces shared by its forward and backward kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "geometry.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace fswin {

namespace resn {

enum : int { kNone = 0, kLayer = 1, kRms = 2 };
constexpr int kMaxChannels = 8192;

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
// lane + L i.  W = 8 (16-byte bf16 accesses) where the channel count and every
// pointer allow it, else W = 1.  `has` bit i: chunk i lies inside the row; the
// others read as zero and are not written.
template <int W, int L, int V>
struct Row {
    static constexpr int E = W * V;
    int col[V];
    unsigned int has;
    __device__ __forceinline__ void init(int lane, int C) {
        has = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            col[i] = (lane + L * i) * W;
            if (col[i] < C) has |= 1u << i;
        }
    }
    __device__ __forceinline__ bool in(int i) const { return (has >> i) & 1u; }

    template <typename T>
    __device__ __forceinline__ void load(const T* row, float (&x)[E], float fill = 0.f) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int e = 0; e < W; ++e) x[i * W + e] = fill;
            if (!in(i)) continue;
            if constexpr (W == 1) {
                x[i] = static_cast<float>(row[col[i]]);
            } else if constexpr (sizeof(T) == 2) {
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
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(T* row, const float (&x)[E]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (!in(i)) continue;
            if constexpr (W == 1) {
                row[col[i]] = static_cast<T>(x[i]);
            } else if constexpr (sizeof(T) == 2) {
                const float* y = x + i * W;
                *reinterpret_cast<uint4*>(row + col[i]) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                                     pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            } else {
                const float* y = x + i * W;
                *reinterpret_cast<float4*>(row + col[i]) = make_float4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<float4*>(row + col[i] + 4) = make_float4(y[4], y[5], y[6], y[7]);
            }
        }
    }
    // Factors keep_scale or 0 of the row's elements.
    __device__ __forceinline__ void mask(const Params& prm, unsigned int row, unsigned long long seed,
                                         unsigned long long offset, float (&k)[E]) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const unsigned long long at = static_cast<unsigned long long>(row) * prm.C + col[i];
            if constexpr (W == 1) {
                const uint4 w = philox(at >> 2, offset, seed);
                const uint32_t s = static_cast<uint32_t>(at) & 3u;
                const uint32_t word = s == 0 ? w.x : (s == 1 ? w.y : (s == 2 ? w.z : w.w));
                k[i] = word >= prm.thr ? prm.keep_scale : 0.f;
            } else {  // C is a multiple of 8, so the chunk starts at a multiple of 8
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint4 w = philox((at >> 2) + q, offset, seed);
                    k[i * W + 4 * q] = w.x >= prm.thr ? prm.keep_scale : 0.f;
                    k[i * W + 4 * q + 1] = w.y >= prm.thr ? prm.keep_scale : 0.f;
                    k[i * W + 4 * q + 2] = w.z >= prm.thr ? prm.keep_scale : 0.f;
                    k[i * W + 4 * q + 3] = w.w >= prm.thr ? prm.keep_scale : 0.f;
                }
            }
        }
    }
};

// Sum of a value over the L lanes of a row, the same in every lane.  Groups of
// more than a warp are the whole block.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* scratch) {
#pragma unroll
    for (int o = (L < 32 ? L : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if constexpr (L > 32) {
        if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int w = 0; w < L / 32; ++w) v += scratch[w];
        __syncthreads();
    }
    return v;
}

// Normalises a row in place of `x` (chunks outside the row stay zero) and returns
// 1 / deviation: mean and centred squares in two passes over registers, so a large
// mean costs no digits.
template <int W, int L, int V>
__device__ __forceinline__ float normalise(const Row<W, L, V>& g, float (&x)[W * V], int kind, const Params& prm,
                                           float* scratch) {
    if (kind == kLayer) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < W * V; ++e) s += x[e];
        const float mean = row_sum<L>(s, scratch) * prm.inv_c;
#pragma unroll
        for (int e = 0; e < W * V; ++e) x[e] = g.in(e / W) ? x[e] - mean : 0.f;
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

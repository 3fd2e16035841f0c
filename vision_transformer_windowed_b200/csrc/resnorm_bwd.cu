// Backward of the residual step: dx, df and the parameters' gradients.
//
//   t = w_pre o dn, dr' = dr + (t - rh mean(t rh) [- mean(t)]) / dev(r)     (rh: the normalised r)
//   dx = dr', du = g_b dr', dg_b = sum dr' o u, dgamma = sum du o drop(y),
//   dy = drop(gamma o du), df = dy, or through the post norm likewise
// The norms' rows are formed again from r and f, and the mask is drawn again, so
// nothing but r and f is kept from the forward.  Memory-bound in the large: dr, dn,
// r, f read and dx, df written once.  The parameters' gradients add up in registers
// over the rows of a block (a lane always holds the same channels), then over the
// block's row groups, and a second launch adds the blocks' sums in order: no
// atomics, the same bits every run.
#include "resnorm.cuh"

namespace fswin {

namespace resn {

constexpr int kBwdThreads = 256;

// Parameters with a gradient of C values, in the order of `part`.
enum : int { kPreW = 0, kPreB = 1, kScaleG = 2, kPostW = 3, kPostB = 4, kGrads = 5 };

template <int W, int L, int V>
__device__ __forceinline__ void norm_grad(float (&t)[W * V], const float (&hat)[W * V], float inv, int kind,
                                          const Row<W, L, V>& g, const Params& prm, float* scratch) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int e = 0; e < W * V; ++e) {
        a = fmaf(t[e], hat[e], a);
        b += t[e];
    }
    const float c1 = row_sum<L>(a, scratch) * prm.inv_c;
    const float c2 = kind == kLayer ? row_sum<L>(b, scratch) * prm.inv_c : 0.f;
#pragma unroll
    for (int e = 0; e < W * V; ++e) t[e] = g.in(e / W) ? (t[e] - fmaf(hat[e], c1, c2)) * inv : 0.f;
}

// kPost: with a post norm (its two sums double the registers, so it has kernels of
// its own).
template <typename TX, int W, int L, int V, bool kPost>
__global__ void __launch_bounds__(L > 32 ? L : kBwdThreads) bwd_kernel(const __grid_constant__ Params prm) {
    constexpr int E = W * V;
    constexpr int kGroups = L > 32 ? 1 : kBwdThreads / L;
    constexpr int kWarps = (L > 32 ? L : kBwdThreads) / 32;
    extern __shared__ float sums[];  // [channel span] of one parameter, per warp (groups inside a warp)
    __shared__ float scratch[L > 32 ? L / 32 : 1];
    const ResnormPtrs& p = prm.p;
    const int lane = L > 32 ? threadIdx.x : threadIdx.x % L;
    Row<W, L, V> g;
    g.init(lane, prm.C);
    unsigned long long seed = 0, offset = 0;
    if (prm.drop) {
        seed = static_cast<unsigned long long>(p.rng[0]);
        offset = static_cast<unsigned long long>(p.rng[1]);
    }
    const TX* gate = static_cast<const TX*>(p.gate);
    const bool branch = p.scale || p.dgate || kPost;  // the branch's value is needed, not its gradient alone
    float acc[kPost ? kGrads : 3][E];
#pragma unroll
    for (int k = 0; k < (kPost ? kGrads : 3); ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[k][e] = 0.f;

    const unsigned int own = L > 32 ? 0 : threadIdx.x / L;
    for (unsigned int base = blockIdx.x * kGroups; base < prm.rows; base += gridDim.x * kGroups) {
        const unsigned int row = base + own;
        const bool live = row < prm.rows;
        const unsigned int at_row = live ? row : prm.rows - 1u;
        const long long at = static_cast<long long>(at_row) * prm.C;
        float d[E];  // dr', in the end dx
#pragma unroll
        for (int e = 0; e < E; ++e) d[e] = 0.f;
        if (live && p.dr) g.load(static_cast<const TX*>(p.dr) + at, d);
        float y[E];
        const float gt = gate ? static_cast<float>(gate[fdiv(prm.tokens, at_row)]) : 1.f;
        const bool take = branch && (gt != 0.f || p.dgate);
        if (take) {
            g.load(static_cast<const __nv_bfloat16*>(p.f) + at, y);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = 0.f;
        }
        if (prm.pre != kNone && p.dn) {
            float t[E], hat[E];
            g.load(static_cast<const TX*>(p.r) + at, hat);
#pragma unroll
            for (int e = 0; e < E; ++e) t[e] = 0.f;
            if (live) g.load(static_cast<const __nv_bfloat16*>(p.dn) + at, t);
            const float inv = normalise(g, hat, prm.pre, prm, scratch);
            if (p.pre_w) {
                float w[E];
                g.load(static_cast<const TX*>(p.pre_w), w);
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    acc[kPreW][e] = fmaf(t[e], hat[e], acc[kPreW][e]);
                    acc[kPreB][e] += t[e];
                    t[e] *= w[e];
                }
            } else if (p.pre_b) {
#pragma unroll
                for (int e = 0; e < E; ++e) acc[kPreB][e] += t[e];
            }
            norm_grad(t, hat, inv, prm.pre, g, prm, scratch);
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] += t[e];
        }
        if (live) g.store(static_cast<TX*>(p.dx) + at, d);
        // the branch: y becomes drop(post(f)), d becomes dy
        float hat[kPost ? E : 1];
        float inv = 0.f;
        if constexpr (kPost) {
            inv = normalise(g, y, prm.post, prm, scratch);
#pragma unroll
            for (int e = 0; e < E; ++e) hat[e] = y[e];
            float w[E];
            if (p.post_w) {
                g.load(static_cast<const TX*>(p.post_w), w);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] *= w[e];
            }
            if (p.post_b) {
                g.load(static_cast<const TX*>(p.post_b), w);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] += w[e];
            }
        }
        float k[E];
        if (prm.drop) {
            g.mask(prm, at_row, seed, offset, k);
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = k[e] != 0.f ? y[e] * k[e] : 0.f;
        }
        float sc[E];
        if (p.scale) g.load(static_cast<const TX*>(p.scale), sc);
        if (p.dgate) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(d[e], p.scale ? y[e] * sc[e] : y[e], s);
            s = row_sum<L>(s, scratch);
            if (live && lane == 0) prm.rowdot[row] = s;
        }
        if (gt == 0.f) {  // a dropped sample: no gradient reaches the branch or what scales it
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = 0.f;
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] *= gt;
        }
        if (p.scale) {
            if (gt != 0.f) {
#pragma unroll
                for (int e = 0; e < E; ++e) acc[kScaleG][e] = fmaf(d[e], y[e], acc[kScaleG][e]);
            }
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] *= sc[e];
        }
        if (prm.drop) {
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] = k[e] != 0.f ? d[e] * k[e] : 0.f;
        }
        if constexpr (kPost) {
            if (gt != 0.f) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    acc[kPostW][e] = fmaf(d[e], hat[e], acc[kPostW][e]);
                    acc[kPostB][e] += d[e];
                }
            }
            if (p.post_w) {
                float w[E];
                g.load(static_cast<const TX*>(p.post_w), w);
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] *= w[e];
            }
            norm_grad(d, hat, inv, prm.post, g, prm, scratch);
            if (gt == 0.f) {
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] = 0.f;
            }
        }
        if (live) g.store(static_cast<__nv_bfloat16*>(p.df) + at, d);
    }

    // the block's sums: over the row groups of a warp by shuffles, over the warps in
    // shared memory, in a fixed order
    auto reduce = [&](int slot, float (&a)[E], const void* wanted) {
        if (!wanted) return;
        float* out = prm.part + (static_cast<long long>(slot) * prm.blocks + blockIdx.x) * prm.C;
        if constexpr (L > 32) {
            g.store(out, a);
        } else {
#pragma unroll
            for (int o = 16; o >= L; o >>= 1)
#pragma unroll
                for (int e = 0; e < E; ++e) a[e] += __shfl_xor_sync(0xFFFFFFFFu, a[e], o);
            float* mine = sums + (threadIdx.x >> 5) * (L * E);
            if ((threadIdx.x & 31) < L) {
#pragma unroll
                for (int e = 0; e < E; ++e) mine[lane * E + e] = a[e];
            }
            __syncthreads();
            if (threadIdx.x < L) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    float s = 0.f;
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) s += sums[w * (L * E) + lane * E + e];
                    a[e] = s;
                }
                g.store(out, a);
            }
            __syncthreads();
        }
    };
    reduce(kPreW, acc[kPreW], p.dpre_w);
    reduce(kPreB, acc[kPreB], p.dpre_b);
    reduce(kScaleG, acc[kScaleG], p.dscale);
    if constexpr (kPost) {
        reduce(kPostW, acc[kPostW], p.dpost_w);
        reduce(kPostB, acc[kPostB], p.dpost_b);
    }
}

// Sums of the blocks' partials (32 channels a block, eight slices of the blocks
// added in order), and of the rows of a sample for the gate.
template <typename TX>
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ Params prm, int col_blocks) {
    __shared__ float s[256];
    const ResnormPtrs& p = prm.p;
    void* const outs[kGrads] = {p.dpre_w, p.dpre_b, p.dscale, p.dpost_w, p.dpost_b};
    const int t = threadIdx.x;
    if (blockIdx.x < static_cast<unsigned>(col_blocks * kGrads)) {
        const int slot = blockIdx.x / col_blocks, c = (blockIdx.x % col_blocks) * 32 + (t & 31), q = t >> 5;
        TX* out = static_cast<TX*>(outs[slot]);
        if (!out) return;
        float a = 0.f;
        if (c < prm.C) {
            const float* src = prm.part + static_cast<long long>(slot) * prm.blocks * prm.C + c;
            const int per = (prm.blocks + 7) / 8, b1 = min(prm.blocks, (q + 1) * per);
#pragma unroll 4
            for (int b = q * per; b < b1; ++b) a += src[static_cast<long long>(b) * prm.C];
        }
        s[t] = a;
        __syncthreads();
        if (t < 32 && c < prm.C) {
#pragma unroll
            for (int w = 1; w < 8; ++w) a += s[w * 32 + t];
            out[c] = static_cast<TX>(a);
        }
        return;
    }
    const unsigned int b = blockIdx.x - col_blocks * kGrads;
    const unsigned int n = prm.rows / static_cast<unsigned int>(p.samples);
    const float* src = prm.rowdot + static_cast<unsigned long long>(b) * n;
    float a = 0.f;
#pragma unroll 4
    for (unsigned int i = t; i < n; i += 256) a += src[i];
    s[t] = a;
    __syncthreads();
#pragma unroll
    for (int o = 128; o > 0; o >>= 1) {
        if (t < o) s[t] += s[t + o];
        __syncthreads();
    }
    if (t == 0) static_cast<TX*>(p.dgate)[b] = static_cast<TX>(s[0]);
}

// Blocks of the backward kernel, by the row shape's threads and groups.
inline int bwd_blocks(unsigned int rows, int L) {
    const int groups = L > 32 ? 1 : kBwdThreads / L;
    const long long need = (static_cast<long long>(rows) + groups - 1) / groups;
    const long long most = kMaxBwdBlocks;
    return static_cast<int>(need < most ? need : most);
}

template <typename TX>
struct LaunchBwd {
    Params& prm;
    cudaStream_t stream;
    template <int W, int L, int V, bool kPost>
    cudaError_t go() const {
        constexpr int threads = L > 32 ? L : kBwdThreads;
        prm.blocks = bwd_blocks(prm.rows, L);
        const int smem = L > 32 ? 0 : threads / 32 * L * W * V * 4;
        bwd_kernel<TX, W, L, V, kPost><<<prm.blocks, threads, smem, stream>>>(prm);
        return cudaGetLastError();
    }
    template <bool kPost>
    cudaError_t wide() const {
        const int n = prm.C / 8;
        if (n <= 8) return go<8, 4, 2, kPost>();
        if (n > 8 && n <= 12 && !kPost) return go<8, 4, 3, false>();
        if (n <= 16) return go<8, 8, 2, kPost>();
        if (n <= 24 && !kPost) return go<8, 8, 3, false>();
        if (n <= 32) return go<8, 16, 2, kPost>();
        if (n <= 48 && !kPost) return go<8, 16, 3, false>();
        if (n <= 64) return go<8, 32, 2, kPost>();
        if (n <= 96 && !kPost) return go<8, 32, 3, false>();
        if (n <= 128) return go<8, 64, 2, kPost>();
        if (n <= 256) return go<8, 128, 2, kPost>();
        if (n <= 512) return go<8, 256, 2, kPost>();
        return go<8, 512, 2, kPost>();
    }
    template <bool kPost>
    cudaError_t narrow() const {
        const int n = prm.C;
        if (n <= 32) return go<1, 8, 4, kPost>();
        if (n <= 128) return go<1, 32, 4, kPost>();
        if (n <= 512) return go<1, 128, 4, kPost>();
        if (n <= 2048) return go<1, 256, 8, kPost>();
        return go<1, 1024, 8, kPost>();
    }
    cudaError_t run(bool wide_rows) const {
        if (prm.rows > 0) {
            const cudaError_t e = wide_rows ? (prm.post != kNone ? wide<true>() : wide<false>())
                                            : (prm.post != kNone ? narrow<true>() : narrow<false>());
            if (e != cudaSuccess) return e;
        }
        const ResnormPtrs& p = prm.p;
        if (!p.dpre_w && !p.dpre_b && !p.dscale && !p.dpost_w && !p.dpost_b && !p.dgate) return cudaSuccess;
        const int col_blocks = (prm.C + 31) / 32;
        const unsigned samples = p.dgate ? static_cast<unsigned>(p.samples) : 0u;
        sum_kernel<TX><<<col_blocks * kGrads + samples, 256, 0, stream>>>(prm, col_blocks);
        return cudaGetLastError();
    }
};

}  // namespace resn

size_t resnorm_bwd_workspace_bytes(const ResnormShape& sh) {
    using namespace resn;
    auto round256 = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = static_cast<size_t>(sh.samples) * static_cast<size_t>(sh.tokens);
    const size_t blocks = rows < kMaxBwdBlocks ? rows : kMaxBwdBlocks;
    return round256(kGrads * blocks * static_cast<size_t>(sh.channels) * 4) + round256(rows * 4);
}

cudaError_t launch_resnorm_bwd(const ResnormShape& sh, const ResnormPtrs& p, cudaStream_t stream) {
    using namespace resn;
    Params prm{};
    fill_params(sh, p, &prm);
    const size_t rows = prm.rows, blocks = rows < kMaxBwdBlocks ? rows : kMaxBwdBlocks;
    prm.part = reinterpret_cast<float*>(p.ws);
    prm.rowdot = reinterpret_cast<float*>(
        p.ws + ((kGrads * blocks * static_cast<size_t>(sh.channels) * 4 + 255) & ~size_t(255)));
    const bool wide = sh.wide(p);
    if (sh.stream_f32) return LaunchBwd<float>{prm, stream}.run(wide);
    return LaunchBwd<__nv_bfloat16>{prm, stream}.run(wide);
}

}  // namespace fswin

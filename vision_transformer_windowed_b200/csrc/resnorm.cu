// Forward of the residual step: r = x + g_b gamma o drop(post(f)), n = pre(r).
//
// Memory-bound: x and f are read once, r and n written once (8 bytes a channel for
// a bf16 stream).  A row lives in the registers of a group of lanes from its load to
// its store, both norms' sums included; the dropout mask is drawn in registers.
#include "resnorm.cuh"

namespace fswin {

namespace resn {

constexpr int kThreads = 256;

template <typename TX, int W, int L, int V>
__global__ void __launch_bounds__(L > 32 ? L : kThreads) fwd_kernel(const __grid_constant__ Params prm) {
    __shared__ float scratch[L > 32 ? L / 32 : 1];
    const ResnormPtrs& p = prm.p;
    constexpr int kGroups = L > 32 ? 1 : kThreads / L;
    const int lane = L > 32 ? threadIdx.x : threadIdx.x % L;
    Row<W, L, V> g;
    g.init(lane, prm.C);
    unsigned long long seed = 0, offset = 0;
    if (prm.drop) {
        seed = static_cast<unsigned long long>(p.rng[0]);
        offset = static_cast<unsigned long long>(p.rng[1]);
    }
    const TX* gate = static_cast<const TX*>(p.gate);
    const unsigned int own = L > 32 ? 0 : threadIdx.x / L;
    // whole warps stay in the loop together: their reductions need every lane
    for (unsigned int base = blockIdx.x * kGroups; base < prm.rows; base += gridDim.x * kGroups) {
        const unsigned int row = base + own;
        const bool live = row < prm.rows;
        const unsigned int at_row = live ? row : prm.rows - 1u;
        const long long at = static_cast<long long>(at_row) * prm.C;
        float x[W * V], y[W * V];
        g.load(static_cast<const TX*>(p.x) + at, x);
        const float gt = gate ? static_cast<float>(gate[fdiv(prm.tokens, at_row)]) : 1.f;
        if (gt != 0.f) {
            g.load(static_cast<const __nv_bfloat16*>(p.f) + at, y);
        } else {  // a dropped sample takes nothing from its branch, whatever that holds
#pragma unroll
            for (int e = 0; e < W * V; ++e) y[e] = 0.f;
        }
        if (prm.post != kNone) {
            normalise(g, y, prm.post, prm, scratch);
            float w[W * V];
            if (p.post_w) {
                g.load(static_cast<const TX*>(p.post_w), w);
#pragma unroll
                for (int e = 0; e < W * V; ++e) y[e] *= w[e];
            }
            if (p.post_b) {
                g.load(static_cast<const TX*>(p.post_b), w);
#pragma unroll
                for (int e = 0; e < W * V; ++e) y[e] += w[e];
            }
        }
        if (prm.drop) {
            float k[W * V];
            g.mask(prm, at_row, seed, offset, k);
#pragma unroll
            for (int e = 0; e < W * V; ++e) y[e] = k[e] != 0.f ? y[e] * k[e] : 0.f;
        }
        if (p.scale) {
            float w[W * V];
            g.load(static_cast<const TX*>(p.scale), w);
#pragma unroll
            for (int e = 0; e < W * V; ++e) y[e] *= w[e];
        }
        if (gt != 0.f) {
#pragma unroll
            for (int e = 0; e < W * V; ++e) x[e] = fmaf(gt, y[e], x[e]);
        }
        if (live) g.store(static_cast<TX*>(p.r) + at, x);
        if (prm.pre == kNone) continue;
        // the norm takes the sum before it is rounded to the stream's type
        normalise(g, x, prm.pre, prm, scratch);
        if (p.pre_w) {
            g.load(static_cast<const TX*>(p.pre_w), y);
#pragma unroll
            for (int e = 0; e < W * V; ++e) x[e] *= y[e];
        }
        if (p.pre_b) {
            g.load(static_cast<const TX*>(p.pre_b), y);
#pragma unroll
            for (int e = 0; e < W * V; ++e) x[e] += y[e];
        }
        if (live) g.store(static_cast<__nv_bfloat16*>(p.n) + at, x);
    }
}

template <typename TX>
struct Launch {
    const Params& prm;
    int num_sms;
    cudaStream_t stream;
    template <int W, int L, int V>
    cudaError_t go() const {
        constexpr int threads = L > 32 ? L : kThreads, groups = L > 32 ? 1 : kThreads / L;
        const long long blocks = (static_cast<long long>(prm.rows) + groups - 1) / groups;
        const long long most = static_cast<long long>(num_sms) * (2048 / threads);
        fwd_kernel<TX, W, L, V><<<static_cast<unsigned>(blocks < most ? blocks : most), threads, 0, stream>>>(prm);
        return cudaGetLastError();
    }
    // Row shapes: eight-channel chunks, at most four a lane, the fewest idle lanes
    // for the channel counts of Swin stages (96 k: chunks divide by 12).
    cudaError_t wide() const {
        const int n = prm.C / 8;
        if (n <= 4) return go<8, 4, 1>();
        if (n <= 8) return go<8, 4, 2>();
        if (n <= 12) return go<8, 4, 3>();
        if (n <= 16) return go<8, 8, 2>();
        if (n <= 24) return go<8, 8, 3>();
        if (n <= 32) return go<8, 16, 2>();
        if (n <= 48) return go<8, 16, 3>();
        if (n <= 64) return go<8, 32, 2>();
        if (n <= 96) return go<8, 32, 3>();
        if (n <= 128) return go<8, 32, 4>();
        if (n <= 256) return go<8, 64, 4>();
        if (n <= 512) return go<8, 128, 4>();
        return go<8, 256, 4>();
    }
    cudaError_t narrow() const {
        const int n = prm.C;
        if (n <= 32) return go<1, 8, 4>();
        if (n <= 128) return go<1, 32, 4>();
        if (n <= 512) return go<1, 128, 4>();
        if (n <= 2048) return go<1, 256, 8>();
        return go<1, 1024, 8>();
    }
};

}  // namespace resn

cudaError_t launch_resnorm_fwd(const ResnormShape& sh, const ResnormPtrs& p, int num_sms, cudaStream_t stream) {
    using namespace resn;
    Params prm{};
    fill_params(sh, p, &prm);
    const bool wide = sh.wide(p);
    if (sh.stream_f32) {
        const Launch<float> l{prm, num_sms, stream};
        return wide ? l.wide() : l.narrow();
    }
    const Launch<__nv_bfloat16> l{prm, num_sms, stream};
    return wide ? l.wide() : l.narrow();
}

}  // namespace fswin

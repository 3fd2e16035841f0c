// Forward of the residual step: r = x + g_b gamma o drop(post(f)), n = pre(r).
//
// Memory-bound: x and f are read once, r and n written once (8 bytes a channel for
// a bf16 stream).  A row lives in the registers of a group of lanes from its load to
// its store, both norms' sums included; the dropout mask is drawn in registers.
// 128 x 4096 rows of 96 channels, bf16, gate and layer norm: 62 us, 6.5 TB/s, the rate
// of a plain copy; 64 x 256 rows of 384 channels, fp32 stream, with dropout and layer
// scale: 21 us, 3.6 TB/s (1024 blocks of 444 at a time).
#include "resnorm.cuh"

namespace fswin {

namespace resn {

// Blocks an SM that the registers have to leave room for: the loads of many rows in flight
// are what hides the memory's latency (the first case above: two blocks an SM 79 us, three
// 62 us).  Rows held as bf16 until they are wanted leave that room.
template <int W, int L, int V, bool kPost>
__host__ __device__ constexpr int resident() {
    return L > 256 ? 1 : (kPost ? (W * V <= 16 ? 3 : 2) : (W * V <= 16 ? 4 : (W * V <= 24 ? 3 : 2)));
}

// kPost: with a post norm, which takes the branch's row in fp32 beside the stream's.
template <typename TX, int W, int L, int V, bool S, bool kPost>
__global__ void __launch_bounds__(threads_of<L>(), resident<W, L, V, kPost>())
    fwd_kernel(const __grid_constant__ Params prm) {
    __shared__ float scratch[kScratch];
    const ResnormPtrs& p = prm.p;
    constexpr int kGroups = groups_of<L>();
    const unsigned int own = threadIdx.x / L;
    // the same for all rows of this group (grid_of)
    const int shift = !S ? 0 : static_cast<int>((static_cast<unsigned long long>(blockIdx.x * kGroups + own) * prm.C) & 7u);
    Row<W, L, V, S> g;
    g.init(threadIdx.x % L, prm.C, shift);
    unsigned long long seed = 0, offset = 0;
    if (prm.drop) {
        seed = static_cast<unsigned long long>(p.rng[0]);
        offset = static_cast<unsigned long long>(p.rng[1]);
    }
    const TX* gate = static_cast<const TX*>(p.gate);
    // whole warps stay in the loop together: their reductions need every lane
    for (unsigned int base = blockIdx.x * kGroups; base < prm.rows; base += gridDim.x * kGroups) {
        const unsigned int row = base + own;
        const bool live = row < prm.rows;
        // rows past the last are formed from the last one's, and not stored; a shifted
        // group must not read a row of another shift
        const unsigned int at_row = live ? row : prm.rows - 1u;
        const long long at = static_cast<long long>(at_row) * prm.C;
        Stream<TX, W, L, V, S> held;
        Held<W, L, V, S> f;
        if (!S || live) held.load(g, static_cast<const TX*>(p.x) + at);
        else held.zero();
        const float gt = gate ? static_cast<float>(gate[fdiv(prm.tokens, at_row)]) : 1.f;
        // a dropped sample takes nothing from its branch, whatever that holds
        if (gt != 0.f && (!S || live)) f.load(g, static_cast<const __nv_bfloat16*>(p.f) + at);
        else f.zero();
        float x[W * V], y[W * V];
        f.take(y);
        if constexpr (kPost) {
            normalise(g, y, prm.post, prm, scratch);
            float w[W * V];
            if (p.post_w) {
                g.load(static_cast<const TX*>(p.post_w), w, !S);
#pragma unroll
                for (int e = 0; e < W * V; ++e) y[e] *= w[e];
            }
            if (p.post_b) {
                g.load(static_cast<const TX*>(p.post_b), w, !S);
#pragma unroll
                for (int e = 0; e < W * V; ++e) y[e] += w[e];
            }
        }
        if (prm.drop) {
            drop(y, g.mask(prm, at_row, seed, offset), prm.keep_scale);
        }
        if (p.scale) {
            float w[W * V];
            g.load(static_cast<const TX*>(p.scale), w, !S);
#pragma unroll
            for (int e = 0; e < W * V; ++e) y[e] *= w[e];
        }
        held.take(x);
        if (gt != 0.f) {
#pragma unroll
            for (int e = 0; e < W * V; ++e) x[e] = fmaf(gt, y[e], x[e]);
        }
        if (live) g.store(static_cast<TX*>(p.r) + at, x);
        if (prm.pre == kNone) continue;
        // the norm takes the sum before it is rounded to the stream's type
        normalise(g, x, prm.pre, prm, scratch);
        if (p.pre_w) {
            g.load(static_cast<const TX*>(p.pre_w), y, !S);
#pragma unroll
            for (int e = 0; e < W * V; ++e) x[e] *= y[e];
        }
        if (p.pre_b) {
            g.load(static_cast<const TX*>(p.pre_b), y, !S);
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
    template <int W, int L, int V, bool S>
    cudaError_t go() const {
        const unsigned grid = grid_of(prm.rows, groups_of<L>(), static_cast<unsigned>(num_sms) * (2048 / threads_of<L>()), prm.C);
        if (prm.post != kNone) fwd_kernel<TX, W, L, V, S, true><<<grid, threads_of<L>(), 0, stream>>>(prm);
        else fwd_kernel<TX, W, L, V, S, false><<<grid, threads_of<L>(), 0, stream>>>(prm);
        return cudaGetLastError();
    }
    // Row shapes: eight-channel chunks, at most four a lane, the fewest idle lanes
    // for the channel counts of Swin stages (96 k: chunks divide by 12).
    cudaError_t wide() const {
        const int n = prm.C / 8;
        if (n <= 4) return go<8, 4, 1, false>();
        if (n <= 8) return go<8, 4, 2, false>();
        if (n <= 12) return go<8, 4, 3, false>();
        if (n <= 16) return go<8, 8, 2, false>();
        if (n <= 24) return go<8, 8, 3, false>();
        if (n <= 32) return go<8, 16, 2, false>();
        if (n <= 48) return go<8, 16, 3, false>();
        if (n <= 64) return go<8, 32, 2, false>();
        if (n <= 96) return go<8, 32, 3, false>();
        if (n <= 128) return go<8, 32, 4, false>();
        if (n <= 256) return go<8, 64, 4, false>();
        if (n <= 512) return go<8, 128, 4, false>();
        return go<8, 256, 4, false>();
    }
    cudaError_t shifted() const {  // one chunk more than the channels fill
        const int n = (prm.C + 14) / 8;
        if (n <= 8) return go<8, 8, 1, true>();
        if (n <= 32) return go<8, 32, 1, true>();
        if (n <= 128) return go<8, 128, 1, true>();
        if (n <= 512) return go<8, 256, 2, true>();
        return go<8, 256, 4, true>();
    }
    cudaError_t narrow() const {
        const int n = prm.C;
        if (n <= 32) return go<1, 8, 4, false>();
        if (n <= 128) return go<1, 32, 4, false>();
        if (n <= 512) return go<1, 128, 4, false>();
        if (n <= 2048) return go<1, 256, 8, false>();
        return go<1, 1024, 8, false>();
    }
    cudaError_t run(bool wide_rows) const {
        if (!wide_rows) return narrow();
        return prm.C % 8 ? shifted() : wide();
    }
};

}  // namespace resn

cudaError_t launch_resnorm_fwd(const ResnormShape& sh, const ResnormPtrs& p, int num_sms, cudaStream_t stream) {
    using namespace resn;
    Params prm{};
    fill_params(sh, p, &prm);
    const bool wide = sh.wide(p);
    if (sh.stream_f32) return Launch<float>{prm, num_sms, stream}.run(wide);
    return Launch<__nv_bfloat16>{prm, num_sms, stream}.run(wide);
}

}  // namespace fswin

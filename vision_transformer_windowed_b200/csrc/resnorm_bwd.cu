// Backward of the residual step: dx, df and the parameters' gradients.
//
//   t = w_pre o dn, dr' = dr + (t - rh mean(t rh) [- mean(t)]) / dev(r)     (rh: the normalised r)
//   dx = dr', du = g_b dr', dg_b = sum dr' o u, dgamma = sum du o drop(y),
//   dy = drop(gamma o du), df = dy, or through the post norm likewise
// The norms' rows are formed again from r and f, and the mask is drawn again, so
// nothing but r and f is kept from the forward.  dr, dn, r, f are read and dx, df
// written once: 64 x 256 rows of 384 channels, fp32 stream, with dropout, layer scale and
// gate take 32 us, 3.5 TB/s; 3 x 1111 rows of 1001 channels with both norms 30 us (a chunk a
// lane: 34).  No unit is full (the first: issue slots 45 %, integer pipe 41 %, DRAM 30 %): the
// 16 warps an SM wait, for memory most, then for their reductions.  The parameters' gradients add up over the rows of a block (a lane
// always holds the same channels), then over the block's row groups, and a second launch
// adds the blocks' sums in order: no atomics, the same bits every run.
#include "resnorm.cuh"

namespace fswin {

namespace resn {

// Parameters with a gradient of C values, in the order of `part`.
enum : int { kPreW = 0, kPreB = 1, kScaleG = 2, kPostW = 3, kPostB = 4, kGrads = 5 };

template <int W, int L, int V, bool S>
__device__ __forceinline__ void norm_grad(float (&t)[W * V], const float (&hat)[W * V], float inv, int kind,
                                          const Row<W, L, V, S>& g, const Params& prm, float* scratch) {
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int e = 0; e < W * V; ++e) {
        a = fmaf(t[e], hat[e], a);
        b += t[e];
    }
    const float c1 = row_sum<L>(a, scratch) * prm.inv_c;
    const float c2 = kind == kLayer ? row_sum<L>(b, scratch) * prm.inv_c : 0.f;
    // t and hat are 0 outside the row
#pragma unroll
    for (int e = 0; e < W * V; ++e) t[e] = (t[e] - fmaf(hat[e], c1, g.inside(e, c2))) * inv;
}

// A block's sums of one parameter's gradient: in shared memory, each group of lanes its
// own, in the order of its lanes' registers (a lane's next four elements L lanes x four
// further on, so that sixteen-byte accesses of neighbours adjoin).  They would take E
// registers a lane and parameter otherwise, which left one block a SM and 24 channels
// a lane, or two and 8 (backward of 64 x 256 rows of 384 channels: 38 and 48 us; from
// shared memory 32 us).
template <int W, int L, int V>
struct Sums {
    static constexpr int E = W * V, U = W == 1 ? 1 : 4;
    static constexpr int kFloats = threads_of<L>() * E;
    float* mine;  // of this lane
    __device__ __forceinline__ Sums(float* all, int slot) {
        mine = all + slot * kFloats + (threadIdx.x / L) * (L * E) + (threadIdx.x % L) * U;
    }
    __device__ __forceinline__ void clear() const {
#pragma unroll
        for (int u = 0; u < E / U; ++u)
#pragma unroll
            for (int e = 0; e < U; ++e) mine[u * U * L + e] = 0.f;
    }
    // value(e): what element e adds
    template <typename F>
    __device__ __forceinline__ void add(const F& value) const {
#pragma unroll
        for (int u = 0; u < E / U; ++u) {
            if constexpr (U == 4) {
                float4* at = reinterpret_cast<float4*>(mine + u * U * L);
                float4 v = *at;
                v.x += value(u * 4);
                v.y += value(u * 4 + 1);
                v.z += value(u * 4 + 2);
                v.w += value(u * 4 + 3);
                *at = v;
            } else {
                mine[u * L] += value(u);
            }
        }
    }
    // position of a channel in a group's sums, the group's rows starting at `shift`
    __device__ __forceinline__ static int at(int c, int shift) {
        const int pos = c + shift, chunk = pos / W;
        return ((chunk / L) * (W / U) + (pos % W) / U) * (L * U) + (chunk % L) * U + pos % U;
    }
};

template <typename TX, int W, int L, int V, bool S>
__global__ void __launch_bounds__(threads_of<L>(), L <= 256 && W * V <= 24 ? 2 : 1)
    bwd_kernel(const __grid_constant__ Params prm) {
    constexpr int E = W * V;
    constexpr int kGroups = groups_of<L>();
    extern __shared__ __align__(16) float sums[];
    __shared__ float scratch[kScratch];
    const ResnormPtrs& p = prm.p;
    const int lane = threadIdx.x % L;
    const unsigned int own = threadIdx.x / L;
    // the same for all rows of this group (grid_of)
    const int shift = !S ? 0 : static_cast<int>((static_cast<unsigned long long>(blockIdx.x * kGroups + own) * prm.C) & 7u);
    Row<W, L, V, S> g;
    g.init(lane, prm.C, shift);
    unsigned long long seed = 0, offset = 0;
    if (prm.drop) {
        seed = static_cast<unsigned long long>(p.rng[0]);
        offset = static_cast<unsigned long long>(p.rng[1]);
    }
    const TX* gate = static_cast<const TX*>(p.gate);
    const bool post = prm.post != kNone;
    const bool branch = p.scale || p.dgate || post;  // the branch's value is needed, not its gradient alone
    // the sums that are asked for, one after the other
    const void* const wanted[kGrads] = {p.dpre_w, p.dpre_b, p.dscale, p.dpost_w, p.dpost_b};
    auto slot = [&](int k) {
        int s = 0;
#pragma unroll
        for (int i = 0; i < kGrads; ++i) s += i < k && wanted[i] ? 1 : 0;
        return Sums<W, L, V>(sums, s);
    };
#pragma unroll
    for (int k = 0; k < kGrads; ++k)
        if (wanted[k]) slot(k).clear();

    for (unsigned int base = blockIdx.x * kGroups; base < prm.rows; base += gridDim.x * kGroups) {
        const unsigned int row = base + own;
        const bool live = row < prm.rows;
        // rows past the last are formed from the last one's r and f, and neither stored nor
        // added up; a shifted group must not read a row of another shift, and its row of
        // zeros has no deviation (with eps = 0 it normalises to NaN)
        const unsigned int at_row = live ? row : prm.rows - 1u;
        const bool reads = !S || live;
        const long long at = static_cast<long long>(at_row) * prm.C;
        float d[E];  // dr', in the end dx
        Held<W, L, V, S> f, dn;
        const float gt = gate ? static_cast<float>(gate[fdiv(prm.tokens, at_row)]) : 1.f;
        g.zero(d);
        if (live && p.dr) g.load(static_cast<const TX*>(p.dr) + at, d);
        if (reads && branch && (gt != 0.f || p.dgate)) f.load(g, static_cast<const __nv_bfloat16*>(p.f) + at);
        else f.zero();
        if (prm.pre != kNone && p.dn) {
            float t[E], hat[E];
            if (S) g.zero(hat);
            if (reads) g.load(static_cast<const TX*>(p.r) + at, hat);
            if (live) dn.load(g, static_cast<const __nv_bfloat16*>(p.dn) + at);
            else dn.zero();
            const float inv = normalise(g, hat, prm.pre, prm, scratch);
            dn.take(t);
            if (live && wanted[kPreW]) slot(kPreW).add([&](int e) { return t[e] * hat[e]; });
            if (live && wanted[kPreB]) slot(kPreB).add([&](int e) { return t[e]; });
            if (p.pre_w) {
                float w[E];
                g.load(static_cast<const TX*>(p.pre_w), w, !S);
#pragma unroll
                for (int e = 0; e < E; ++e) t[e] *= w[e];
            }
            norm_grad(t, hat, inv, prm.pre, g, prm, scratch);
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] += t[e];
        }
        if (live) g.store(static_cast<TX*>(p.dx) + at, d);
        // the branch: y becomes drop(post(f)), d becomes dy
        float y[E], hat[E];
        float inv = 0.f;
        f.take(y);
        if (post) {
            inv = normalise(g, y, prm.post, prm, scratch);
#pragma unroll
            for (int e = 0; e < E; ++e) hat[e] = y[e];
            float w[E];
            if (p.post_w) {
                g.load(static_cast<const TX*>(p.post_w), w, !S);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] *= w[e];
            }
            if (p.post_b) {
                g.load(static_cast<const TX*>(p.post_b), w, !S);
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] += w[e];
            }
        }
        uint32_t keep = 0;
        if (prm.drop) {
            keep = g.mask(prm, at_row, seed, offset);
            drop(y, keep, prm.keep_scale);
        }
        float sc[E];
        if (p.scale) g.load(static_cast<const TX*>(p.scale), sc, !S);
        if (p.dgate) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(d[e], p.scale ? y[e] * sc[e] : y[e], s);
            s = row_sum<L>(s, scratch);
            if (live && lane == 0) prm.rowdot[row] = s;
        }
        if (gt == 0.f) {  // a dropped sample: no gradient reaches the branch or what scales it
            g.zero(d);
            g.zero(y);
            if (post) g.zero(hat);
        } else {
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] *= gt;
        }
        if (p.scale) {
            if (live && wanted[kScaleG]) slot(kScaleG).add([&](int e) { return d[e] * y[e]; });
#pragma unroll
            for (int e = 0; e < E; ++e) d[e] *= sc[e];
        }
        if (prm.drop) drop(d, keep, prm.keep_scale);
        if (post) {
            if (live && wanted[kPostW]) slot(kPostW).add([&](int e) { return d[e] * hat[e]; });
            if (live && wanted[kPostB]) slot(kPostB).add([&](int e) { return d[e]; });
            if (p.post_w) {
                float w[E];
                g.load(static_cast<const TX*>(p.post_w), w, !S);
#pragma unroll
                for (int e = 0; e < E; ++e) d[e] *= w[e];
            }
            norm_grad(d, hat, inv, prm.post, g, prm, scratch);
            if (gt == 0.f) g.zero(d);
        }
        if (live) g.store(static_cast<__nv_bfloat16*>(p.df) + at, d);
    }

    // the block's sums: its groups' in order, channel by channel
    __syncthreads();
    for (int k = 0, s = 0; k < kGrads; ++k) {
        if (!wanted[k]) continue;
        float* out = prm.part + (static_cast<long long>(k) * prm.blocks + blockIdx.x) * prm.C;
        const float* all = sums + s * Sums<W, L, V>::kFloats;
        for (int c = threadIdx.x; c < prm.C; c += threads_of<L>()) {
            float a = 0.f;
#pragma unroll 4
            for (int w = 0; w < kGroups; ++w) {
                const int sh = !S ? 0 : static_cast<int>((static_cast<unsigned long long>(blockIdx.x * kGroups + w) * prm.C) & 7u);
                a += all[w * (L * E) + Sums<W, L, V>::at(c, sh)];
            }
            out[c] = a;
        }
        ++s;
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
    const unsigned int first = blockIdx.x - col_blocks * kGrads, step = gridDim.x - col_blocks * kGrads;
    const unsigned int n = prm.rows / static_cast<unsigned int>(p.samples);
    for (long long b = first; b < p.samples; b += step) {
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
        __syncthreads();
    }
}

template <typename TX>
struct LaunchBwd {
    Params& prm;
    cudaStream_t stream;
    template <int W, int L, int V, bool S>
    cudaError_t go() const {
        static SmemOptIn opt_in;
        const ResnormPtrs& p = prm.p;
        const void* const wanted[kGrads] = {p.dpre_w, p.dpre_b, p.dscale, p.dpost_w, p.dpost_b};
        int slots = 0;
        for (const void* w : wanted) slots += w ? 1 : 0;
        constexpr int per = Sums<W, L, V>::kFloats * 4;
        static_assert(kGrads * per <= 200 * 1024, "the sums overflow shared memory");
        const cudaError_t e = opt_in.ensure(reinterpret_cast<const void*>(bwd_kernel<TX, W, L, V, S>), kGrads * per);
        if (e != cudaSuccess) return e;
        prm.blocks = static_cast<int>(grid_of(prm.rows, groups_of<L>(), kMaxBwdBlocks, prm.C));
        bwd_kernel<TX, W, L, V, S><<<prm.blocks, threads_of<L>(), slots * per, stream>>>(prm);
        return cudaGetLastError();
    }
    // Two chunks a lane, or three where that leaves fewer lanes idle (96 k channels).
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
        if (n <= 128) return go<8, 64, 2, false>();
        if (n <= 256) return go<8, 128, 2, false>();
        if (n <= 512) return go<8, 256, 2, false>();
        return go<8, 512, 2, false>();
    }
    cudaError_t shifted() const {  // one chunk more than the channels fill
        const int n = (prm.C + 14) / 8;
        if (n <= 8) return go<8, 8, 1, true>();
        if (n <= 32) return go<8, 16, 2, true>();
        if (n <= 128) return go<8, 64, 2, true>();
        if (n <= 512) return go<8, 256, 2, true>();
        return go<8, 512, 2, true>();
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
        if (prm.rows > 0) {
            const cudaError_t e = !wide_rows ? narrow() : (prm.C % 8 ? shifted() : wide());
            if (e != cudaSuccess) return e;
        }
        const ResnormPtrs& p = prm.p;
        if (!p.dpre_w && !p.dpre_b && !p.dscale && !p.dpost_w && !p.dpost_b && !p.dgate) return cudaSuccess;
        const int col_blocks = (prm.C + 31) / 32;
        // (samples up to 2^31 - 1 would not fit a grid with the columns)
        const unsigned samples = !p.dgate ? 0u : static_cast<unsigned>(p.samples < (1 << 16) ? p.samples : 1 << 16);
        sum_kernel<TX><<<col_blocks * kGrads + samples, 256, 0, stream>>>(prm, col_blocks);
        return cudaGetLastError();
    }
};

}  // namespace resn

size_t resnorm_bwd_workspace_bytes(const ResnormShape& sh) {
    using namespace resn;
    auto round256 = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t rows = static_cast<size_t>(sh.samples) * static_cast<size_t>(sh.tokens);
    const size_t blocks = kMaxBwdBlocks;
    return round256(kGrads * blocks * static_cast<size_t>(sh.channels) * 4) + round256(rows * 4);
}

cudaError_t launch_resnorm_bwd(const ResnormShape& sh, const ResnormPtrs& p, cudaStream_t stream) {
    using namespace resn;
    Params prm{};
    fill_params(sh, p, &prm);
    const size_t blocks = kMaxBwdBlocks;
    prm.part = reinterpret_cast<float*>(p.ws);
    prm.rowdot = reinterpret_cast<float*>(
        p.ws + ((kGrads * blocks * static_cast<size_t>(sh.channels) * 4 + 255) & ~size_t(255)));
    const bool wide = sh.wide(p);
    if (sh.stream_f32) return LaunchBwd<float>{prm, stream}.run(wide);
    return LaunchBwd<__nv_bfloat16>{prm, stream}.run(wide);
}

}  // namespace fswin

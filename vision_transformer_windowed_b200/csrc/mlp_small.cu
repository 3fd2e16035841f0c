// Forward of the gated feed-forward block where all its weights fit into shared memory
// (the first stages of a Swin model): y = (act(x Wg^T + bg) o (x Wu^T + bu)) Wd^T + bd in
// one pass, h never leaves the SM.
//
// One persistent CTA an SM, 24 warps.  Warp 0 copies the weights once and then x, 128
// tokens a tile, two tiles ahead.  Warp 1 issues the products, 64 hidden channels (a
// chunk) at a time: g and u of chunk i + 2 in one product of 128 columns, then y += h Wd^T
// of chunk i with h taken from tensor memory.  Warps 4-19 compute h, eight warps the even
// chunks and eight the odd ones; it replaces their u columns as bf16.  Warps 20-23 store
// y.  Tensor memory: three chunks of g and u (128 columns each), so that a group of warps
// finds its next chunk ready (with two chunks and two tiles of y a tenth slower), and
// one tile of y, or two of up to 64 channels.
//
// 524288 x 96 x 256 with gelu take 126 us (two kernels 189: h alone is 268 MB, written and
// read).  No unit is full (issue slots 64 %, special function 54 %, multiply-add 52 %, tensor
// 29 %).  With a product in the activation's place it takes 100 us: what a chunk passes on
// its way (product, tensor memory to registers and back, product) takes most of the time,
// and the activation, which the other group's chunk hides in part, a quarter on top.
#include "mlp.cuh"

namespace fswin {

namespace mlp {

namespace small {

constexpr int kChunk = 64;                  // hidden channels of a chunk
constexpr int kBlock = 32;                  // contraction channels of x's and the first weights' tiles
constexpr int kTileM = 128;
constexpr int kMaxC = 128;
constexpr int kTileBytes = kTileM * kBlock * 2;
constexpr int kWorkers = 16, kStorers = 4;  // warps
constexpr int kThreads = 128 + 32 * (kWorkers + kStorers);
constexpr int kStoreBytes = 32 * 64;        // a warp's 32 rows x 32 bf16 columns
constexpr int kMaxSmem = 232448;
constexpr uint32_t kBufs = 3;               // chunks of g and u in tensor memory
constexpr uint32_t kColY = 128 * kBufs;     // y's accumulators, behind theirs

struct Bars {
    // gu_full: one for each buffer and group of warps, which so waits for every phase of its own
    uint64_t weights, x_full[2], x_free[2], gu_full[2 * kBufs], h_ready[kBufs], y_full[2], y_free[2], done;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 256, "barrier block overflows its slot");

struct Maps {
    CUtensorMap x, gate, up, down, y;
};
struct Params {
    int tokens, C, F;
    int chunks, blocks, n_y;  // of hidden channels, of x's channels; columns of the second product
    int off_down, off_x, off_store, off_bias, off_bars;
    unsigned int tiles;
    int act;
    const __nv_bfloat16 *b_gate, *b_up, *b_down;
    unsigned int* status;
    unsigned long long limit_ns;
};

// Waits for this warp's loads from tensor memory; the values are not used before it.
__device__ __forceinline__ void settle(uint32_t (&a)[16], uint32_t (&b)[16]) {
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(a[i]), "+r"(b[i]));
}

__global__ void __launch_bounds__(kThreads, 1) fwd_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params prm) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    Bars* bars = reinterpret_cast<Bars*>(smem + prm.off_bars);
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    float* bias = reinterpret_cast<float*>(smem + prm.off_bias);  // gate, up (a chunk's 64 each), down

    if (tid == 0) {
        mbar_init(&bars->weights, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->x_full[i], 1);
            mbar_init(&bars->x_free[i], 1);
            mbar_init(&bars->y_full[i], 1);
            mbar_init(&bars->y_free[i], kStorers);
        }
        for (uint32_t i = 0; i < 2 * kBufs; ++i) mbar_init(&bars->gu_full[i], 1);
        for (uint32_t i = 0; i < kBufs; ++i) mbar_init(&bars->h_ready[i], kWorkers / 2);
        mbar_init(&bars->done, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    const int padded = prm.chunks * kChunk;
    for (int i = tid; i < padded; i += kThreads) {
        bias[(i / kChunk) * 2 * kChunk + i % kChunk] = bias_at(prm.b_gate, i, prm.F);
        bias[(i / kChunk) * 2 * kChunk + kChunk + i % kChunk] = bias_at(prm.b_up, i, prm.F);
    }
    for (int i = tid; i < kMaxC; i += kThreads) bias[2 * padded + i] = bias_at(prm.b_down, i, prm.C);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const uint32_t sbase = smem_u32(smem);
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    const unsigned int count = (prm.tiles - blockIdx.x + gridDim.x - 1) / gridDim.x;  // tiles of this CTA
    const int chunks = prm.chunks, blocks = prm.blocks;
    const unsigned int all = count * chunks;  // chunks of this CTA
    const uint32_t y_bufs = prm.n_y <= 64 ? 2u : 1u;

    if (warp == 0) {
        const uint32_t down_bytes = prm.n_y * kChunk * 2;
        if (elect_one()) {
            mbar_arrive_expect_tx(&bars->weights, chunks * (blocks * kTileBytes + down_bytes));
            for (int c = 0; c < chunks; ++c) {
                for (int b = 0; b < blocks; ++b) {
                    const uint32_t dst = sbase + (c * blocks + b) * kTileBytes;
                    tma_load_2d(dst, &maps.gate, &bars->weights, b * kBlock, c * kChunk);
                    tma_load_2d(dst + kTileBytes / 2, &maps.up, &bars->weights, b * kBlock, c * kChunk);
                }
                tma_load_2d(sbase + prm.off_down + c * down_bytes, &maps.down, &bars->weights, c * kChunk, 0);
            }
        }
        __syncwarp();
        for (unsigned int n = 0; n < count; ++n) {
            const uint32_t s = n & 1u;
            if (!mbar_wait_warp(&bars->x_free[s], ((n >> 1) & 1u) ^ 1u, ctl, 0x8201)) break;
            const int row = static_cast<int>(blockIdx.x + n * gridDim.x) * kTileM;
            if (elect_one()) {
                mbar_arrive_expect_tx(&bars->x_full[s], blocks * kTileBytes);
                for (int b = 0; b < blocks; ++b)
                    tma_load_2d(sbase + prm.off_x + (s * blocks + b) * kTileBytes, &maps.x, &bars->x_full[s], b * kBlock, row);
            }
            __syncwarp();
        }
    } else if (warp == 1) {
        const uint32_t id_gu = make_idesc_bf16(kTileM, 2 * kChunk, false, false);
        const uint32_t id_y = make_idesc_bf16(kTileM, prm.n_y, false, false);
        const int steps = (prm.C + 15) / 16;
        // g and u of the next chunk, into its buffer
        struct {
            unsigned int n, i;
            int c;
            uint32_t buf, bar;
        } next{0, 0, 0, 0, 0};
        auto issue_gu = [&]() {
            const uint32_t s = next.n & 1u;
            if (next.c == 0 && !mbar_wait_warp(&bars->x_full[s], (next.n >> 1) & 1u, ctl, 0x8202)) return false;
            tc_fence_after();
            const bool last = next.c == chunks - 1;
            if (elect_one()) {
                const uint32_t x = sbase + prm.off_x + s * blocks * kTileBytes, w = sbase + next.c * blocks * kTileBytes;
                for (int k = 0; k < steps; ++k) {
                    const uint32_t at = (k >> 1) * kTileBytes;
                    umma_ss(tmem + 128 * next.buf, make_sdesc(x + at, 16, 512, kSw64) + 2 * (k & 1),
                            make_sdesc(w + at, 16, 512, kSw64) + 2 * (k & 1), id_gu, k > 0);
                }
                umma_commit(&bars->gu_full[next.bar]);
                if (last) umma_commit(&bars->x_free[s]);
            }
            __syncwarp();
            next.n += last ? 1u : 0u;
            next.c = last ? 0 : next.c + 1;
            next.buf = next.buf == kBufs - 1 ? 0 : next.buf + 1;
            next.bar = next.bar == 2 * kBufs - 1 ? 0 : next.bar + 1;
            ++next.i;
            return true;
        };
        bool ok = mbar_wait_warp(&bars->weights, 0, ctl, 0x8203);
        for (uint32_t i = 0; i + 1 < kBufs && next.i < all && ok; ++i) ok = issue_gu();
        uint32_t buf = 0, turn = 0, yb = 0, yturn = 0;
        for (unsigned int n = 0; n < count && ok; ++n) {
            const uint32_t y = tmem + kColY + 64 * yb;
            for (int c = 0; c < chunks; ++c) {
                // into the buffer whose h has gone into a product already issued
                if (next.i < all && !(ok = issue_gu())) break;
                if (c == 0 && !(ok = mbar_wait_warp(&bars->y_free[yb], (yturn & 1u) ^ 1u, ctl, 0x8204))) break;
                if (!(ok = mbar_wait_warp(&bars->h_ready[buf], turn & 1u, ctl, 0x8205))) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t h = tmem + 128 * buf + kChunk;
                    const uint64_t w = make_sdesc(sbase + prm.off_down + c * prm.n_y * kChunk * 2, 16, 1024, kSw128);
                    const int left = (prm.F - c * kChunk + 15) / 16;
                    for (int k = 0; k < (left < 4 ? left : 4); ++k)
                        umma_ts(y, h + 32 * (k >> 1) + 8 * (k & 1), w + 2 * k, id_y, c > 0 || k > 0);
                    if (c == chunks - 1) umma_commit(&bars->y_full[yb]);
                }
                __syncwarp();
                if (++buf == kBufs) {
                    buf = 0;
                    ++turn;
                }
            }
            if (++yb == y_bufs) {
                yb = 0;
                ++yturn;
            }
        }
        if (elect_one()) umma_commit(&bars->done);  // every product issued here has completed before the columns are freed
        mbar_wait_warp(&bars->done, 0, ctl, 0x82ff);
    } else if (warp >= 4 && warp < 4 + kWorkers) {
        const int ew = warp - 4, group = ew >> 3, half = (ew >> 2) & 1;
        const uint32_t own = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 32 * half;
        int c = group % chunks;
        uint32_t buf = group, bar = group, turn = 0;
        for (unsigned int i = group; i < all; i += 2, c = (c + 2) % chunks) {
            if (!mbar_wait_warp(&bars->gu_full[bar], turn & 1u, ctl, 0x8206)) break;
            const uint32_t base = own + 128 * buf;
            tc_fence_after();
            const float* b = bias + c * 2 * kChunk + 32 * half;
            // 16 channels at a time; the second sixteen's g arrives while the first are computed
            uint32_t gv[2][16], uv[16];
            tmem_ld16(base, gv[0]);
            tmem_ld16(base + kChunk, uv);
            settle(gv[0], uv);
            tmem_ld16(base + 16, gv[1]);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                if (sub == 1) {
                    tmem_ld16(base + kChunk + 16, uv);
                    settle(gv[1], uv);
                }
                uint32_t out[8];
#pragma unroll
                for (int q = 0; q < 2; ++q) {  // eight channels
                    unsigned long long g[4], f[4], s[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 v = *reinterpret_cast<const float4*>(b + 16 * sub + 8 * q + 4 * e);
                        const uint32_t* t = gv[sub] + 8 * q + 4 * e;
                        g[2 * e] = add_pair(pair(t[0], t[1]), pair(v.x, v.y));
                        g[2 * e + 1] = add_pair(pair(t[2], t[3]), pair(v.z, v.w));
                    }
                    activate<false>(g, prm.act, f, s);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 v = *reinterpret_cast<const float4*>(b + kChunk + 16 * sub + 8 * q + 4 * e);
                        const uint32_t* t = uv + 8 * q + 4 * e;
                        float lo, hi;
                        unpair(mul_pair(f[2 * e], add_pair(pair(t[0], t[1]), pair(v.x, v.y))), lo, hi);
                        out[4 * q + 2 * e] = pack_bf16x2(lo, hi);
                        unpair(mul_pair(f[2 * e + 1], add_pair(pair(t[2], t[3]), pair(v.z, v.w))), lo, hi);
                        out[4 * q + 2 * e + 1] = pack_bf16x2(lo, hi);
                    }
                }
                tmem_st8(base + kChunk + 8 * sub, out);  // over u's columns that this warp has read
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->h_ready[buf]);
            buf = buf + 2 >= kBufs ? buf + 2 - kBufs : buf + 2;
            bar += 2;
            if (bar >= 2 * kBufs) {
                bar -= 2 * kBufs;
                ++turn;
            }
        }
    } else if (warp >= 4 + kWorkers) {
        const int quad = warp & 3;
        const float* b = bias + 2 * padded;
        uint32_t sbuf = 0, yb = 0, yturn = 0;
        for (unsigned int n = 0; n < count; ++n) {
            if (!mbar_wait_warp(&bars->y_full[yb], yturn & 1u, ctl, 0x8207)) break;
            tc_fence_after();
            const uint32_t acc = tmem + kColY + 64 * yb + (static_cast<uint32_t>(quad * 32) << 16);
            const int row = static_cast<int>(blockIdx.x + n * gridDim.x) * kTileM + quad * 32;
            for (int c = 0; c < prm.C; c += 32, ++sbuf) {
                uint32_t v[32];
                tmem_ld32(acc + c, v);
                bulk_wait_read_but1();  // the buffer's last store has read it
                __syncwarp();
                tmem_wait_ld();
                if (c + 32 >= prm.C) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->y_free[yb]);
                }
                const int buf = prm.off_store + (quad * 2 + static_cast<int>(sbuf & 1u)) * kStoreBytes;
                uint8_t* dst = smem + buf + lane * 64;
                const int sw = (lane >> 1) & 3;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 a = *reinterpret_cast<const float4*>(b + c + 8 * q + 4 * e);
                        const uint32_t* t = v + 8 * q + 4 * e;
                        w[2 * e] = pack_bf16x2(__uint_as_float(t[0]) + a.x, __uint_as_float(t[1]) + a.y);
                        w[2 * e + 1] = pack_bf16x2(__uint_as_float(t[2]) + a.z, __uint_as_float(t[3]) + a.w);
                    }
                    *reinterpret_cast<uint4*>(dst + ((q ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d(&maps.y, sbase + buf, c, row);
                    bulk_commit();
                }
            }
            if (++yb == y_bufs) {
                yb = 0;
                ++yturn;
            }
        }
        bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Shared memory of a launch: chunks of the first weights, of the last, x twice, stores,
// biases, barriers.
int layout(const MlpShape& sh, Params* p) {
    p->C = sh.channels;
    p->F = sh.hidden;
    p->chunks = (sh.hidden + kChunk - 1) / kChunk;
    p->blocks = (sh.channels + kBlock - 1) / kBlock;
    p->n_y = (sh.channels + 15) / 16 * 16;
    p->off_down = p->chunks * p->blocks * kTileBytes;
    p->off_x = p->off_down + p->chunks * p->n_y * kChunk * 2;
    p->off_store = p->off_x + 2 * p->blocks * kTileBytes;
    p->off_bias = p->off_store + kStorers * 2 * kStoreBytes;
    p->off_bars = p->off_bias + (2 * p->chunks * kChunk + kMaxC) * 4;
    return p->off_bars + 256 + 1024;
}

}  // namespace small

}  // namespace mlp

bool mlp_fits(const MlpShape& sh) {
    mlp::small::Params p{};
    return sh.channels <= mlp::small::kMaxC && sh.hidden <= 1024 && mlp::small::layout(sh, &p) <= mlp::small::kMaxSmem;
}

cudaError_t launch_mlp_small_fwd(const MlpShape& sh, const MlpPtrs& p, unsigned int* status, unsigned long long limit_ns,
                                 int num_sms, cudaStream_t stream) {
    using namespace mlp;
    using namespace mlp::small;
    small::Params prm{};
    const int smem = layout(sh, &prm);
    const int T = static_cast<int>(sh.tokens);
    prm.tokens = T;
    prm.tiles = (static_cast<unsigned>(T) + kTileM - 1) / kTileM;
    prm.act = sh.act;
    prm.b_gate = static_cast<const __nv_bfloat16*>(p.b_gate);
    prm.b_up = static_cast<const __nv_bfloat16*>(p.b_up);
    prm.b_down = static_cast<const __nv_bfloat16*>(p.b_down);
    prm.status = status;
    prm.limit_ns = limit_ns;
    small::Maps maps{};
    if (encode_matrix(&maps.x, p.x, T, sh.channels, kTileM, kBlock, false) ||
        encode_matrix(&maps.gate, p.w_gate, sh.hidden, sh.channels, kChunk, kBlock, false) ||
        encode_matrix(&maps.up, p.w_up, sh.hidden, sh.channels, kChunk, kBlock, false) ||
        encode_matrix(&maps.down, p.w_down, sh.channels, sh.hidden, prm.n_y, kChunk, true) ||
        encode_matrix(&maps.y, p.y, T, sh.channels, 32, 32, false))
        return cudaErrorInvalidValue;
    static SmemOptIn optin;
    if (cudaError_t e = optin.ensure(reinterpret_cast<const void*>(fwd_kernel), kMaxSmem)) return e;
    const unsigned int grid = prm.tiles < static_cast<unsigned>(num_sms) ? prm.tiles : num_sms;
    fwd_kernel<<<grid, small::kThreads, smem, stream>>>(maps, prm);
    return cudaGetLastError();
}

}  // namespace fswin

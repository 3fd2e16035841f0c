// Gated feed-forward block: y = h W_down^T + b_down, h = act(x W_gate^T + b_gate) o (x W_up^T + b_up),
// and its backward, as persistent tensor-core kernels over one pipeline.
//
// Pipeline (one CTA an SM, 12 or 20 warps): warp 0 copies operand blocks of 64
// contraction channels into a ring with TMA (128-byte swizzle), warp 1 issues
// tcgen05 products into one of two 256-column TMEM accumulators, the warps from 4 on
// turn the other accumulator into the result.  Operands are taken as they lie in memory:
// contraction-major, or (weights and activations of the gradient products)
// row-major with the contraction over rows, which the matrix descriptors express.
// A contraction that does not fill its last block ends at its last 16 channels.
//
//   kGate:   h = act(x Wg^T + bg) o (x Wu^T + bu): the two weight tiles lie one after
//            the other in a stage, so one product of up to 256 columns makes both
//   kLinear: y = h Wd^T + bd
//   kGrad:   g, u again, dh = dy Wd; h, dg = dh o u o act'(g), du = dh o act(g)
//   kDx:     dx = dg Wg + du Wu, one contraction over both
//   kDw:     dWg = dg^T x, dWu = du^T x, dWd^T = h^T dy, the tokens split over CTAs with
//            fp32 partial results that a second kernel adds in order; 16-column
//            products with a tile of ones give dg's and du's bias gradients, two
//            warps add up dy's columns as they pass.  Tiles of 256 x 192, both
//            accumulators to one: a larger tile moves less through shared memory
//            (128 x 192: 98 us in place of 80)
//
// At 32768 x 384 x 1024 (silu): kGate 42 us (1230 TFLOP/s), kLinear 28 (920), kGrad 100
// (770), kDx 48 (1070), kDw 80 (970).  Shared-memory bandwidth bounds them: a tile of
// kGrad moves 336 KB in, its products read as much and its epilogue passes 96 KB, 6000
// clocks at 128 bytes, the time it takes; kDw also waits for reads that miss L2.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mlp.cuh"

namespace fswin {

namespace mlp {

enum : int { kGate, kLinear, kGrad, kDx, kDw };
// Warps of the epilogue: sixteen where it computes the activation (kGate: four a
// scheduler hide each other's latencies, 176 -> 130 us at 524288 x 96 x 256), else eight.
__host__ __device__ constexpr int epi_warps(int op) { return op == kGate ? 16 : 8; }
__host__ __device__ constexpr int threads_of(int op) { return 128 + 32 * epi_warps(op); }
constexpr int kBlockK = 64;
constexpr int kBlockM = 128;
constexpr int kABytes = kBlockM * kBlockK * 2;
constexpr int kStages = 4;                        // at most
constexpr int kTallMaxN = 192;
// A stage: A, and B of up to 256 rows; kGrad: x, three times 64 weight rows, dy; tall
// tiles: twice A's rows and up to 192 columns.
__host__ __device__ constexpr int stage_bytes(int op, bool tall) {
    return op == kGrad ? 2 * kABytes + 3 * 8192 : (tall ? 2 * kABytes + kTallMaxN * 128 : 3 * kABytes);
}
__host__ __device__ constexpr int stages_of(int op, bool tall) { return op == kGrad || tall ? 3 : kStages; }
constexpr int kStoreBytes = 32 * 64;              // a warp's 32 rows x 32 bf16 columns
constexpr int kRingBytes = 12 * kABytes;
constexpr int kOnesOff = stages_of(kDw, true) * stage_bytes(kDw, true);  // kDw: 16 rows x 64 of 1.0 behind its ring
constexpr int kOnesBytes = 2048;
constexpr int kStoreOff = kRingBytes;
constexpr int kBarOff = kStoreOff + 16 * kStoreBytes;
constexpr uint32_t kColOnes = 240;                // bias gradient columns of kDw, beside each half's

struct Bars {
    uint64_t full[kStages], free_[kStages], acc_full[2], acc_free[2], done;
    uint32_t tmem_base;
    int abort_flag;
};
constexpr int kSmemBytes = kBarOff + 256 + 1024;
static_assert(stages_of(kGate, false) * stage_bytes(kGate, false) <= kRingBytes &&
                  stages_of(kGrad, false) * stage_bytes(kGrad, false) <= kRingBytes &&
                  kOnesOff + kOnesBytes <= kRingBytes,
              "the ring overflows its place");
static_assert(stage_bytes(kGrad, false) % 1024 == 0 && stage_bytes(kDw, true) % 1024 == 0 && kOnesOff % 1024 == 0, "tile alignment");
static_assert(sizeof(Bars) <= 256, "barrier block overflows its slot");
static_assert(kSmemBytes <= 232448, "more shared memory than a CTA may have");

struct Problem {       // kDw: one of the three weight gradients
    int m, n, tiles_n, first;  // first: its first tile in the launch
    FastDiv by_n;      // tiles_n
    int turned;        // the result lies as [n][m], and the bias gradient is of the n columns
    float* part;       // [splits][m][n], or [splits][n][m]
    float* bias_part;  // [splits][m], or [splits][2][n]; or null
};

struct Maps {
    CUtensorMap a[3], b[3], out[3];
};

struct Params {
    int m, n, k;       // result rows and columns, contraction length (of one segment)
    int segments;      // kDx: 2
    int bn;            // columns of a tile
    int tiles_n;
    FastDiv by_n, by_splits;  // tiles_n, splits
    unsigned int tiles;
    int act;           // 0 silu, 1 gelu
    const __nv_bfloat16 *bias0, *bias1;
    Problem pr[3];
    int splits, blocks_per_split;  // kDw, in blocks of 64 tokens
    unsigned int* status;
    unsigned long long limit_ns;
};

// Adds 32 bias columns, one a lane, to every lane's row of 32: through the warp's
// shared memory, from which each lane reads them all.
__device__ __forceinline__ void add_bias(unsigned long long (&x)[16], float* place, float mine, int lane) {
    __syncwarp();
    place[lane] = mine;
    __syncwarp();
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float4 b = *reinterpret_cast<const float4*>(place + 4 * q);
        x[2 * q] = add_pair(x[2 * q], pair(b.x, b.y));
        x[2 * q + 1] = add_pair(x[2 * q + 1], pair(b.z, b.w));
    }
}

// 32 accumulator columns of this thread's row, in pairs; wait_cols before they are used.
struct Cols {
    uint32_t v[32];
    __device__ __forceinline__ void load(uint32_t taddr) { tmem_ld32(taddr, v); }
    __device__ __forceinline__ void get(unsigned long long (&x)[16]) const {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = pair(v[2 * e], v[2 * e + 1]);
    }
};

// kTall: tiles of 256 rows, both accumulators to one (kDw, and kLinear and kDx over long
// contractions).
template <int OP, bool kTall>
__global__ void __launch_bounds__(threads_of(OP), 1) mlp_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params prm) {
    constexpr int kEpiWarps = epi_warps(OP), kThreads = threads_of(OP);
    constexpr int stages = stages_of(OP, kTall), kStageBytes = stage_bytes(OP, kTall), kTileM = kTall ? 2 * kBlockM : kBlockM;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    Bars* bars = reinterpret_cast<Bars*>(smem + kBarOff);
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    uint8_t* ones = smem + kOnesOff;  // kDw only

    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars->full[i], 1);
            mbar_init(&bars->free_[i], OP == kDw ? 3 : 1);  // kDw: the products, and warps 2 and 3
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->acc_full[i], 1);
            mbar_init(&bars->acc_free[i], kEpiWarps);
        }
        mbar_init(&bars->done, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    if (OP == kDw) {
        for (int i = tid; i < kOnesBytes / 4; i += kThreads) reinterpret_cast<uint32_t*>(ones)[i] = 0x3F803F80u;
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const uint32_t sbase = smem_u32(smem);
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};

    // A tile of the launch: its problem (kDw), first row and column, first block and
    // number of blocks of its contraction.
    struct Tile {
        int pr, m0, n0, kb0, nkb, split;
    };
    const int kblocks = (prm.k + kBlockK - 1) / kBlockK;
    auto tile_of = [&](unsigned int t) {
        Tile x{0, 0, 0, 0, kblocks * (OP == kDx ? prm.segments : 1), 0};
        if (OP == kDw) {
            const int q = static_cast<int>(fdiv(prm.by_splits, t));
            x.split = static_cast<int>(t) - q * prm.splits;
            x.pr = q >= prm.pr[2].first ? 2 : (q >= prm.pr[1].first ? 1 : 0);
            const Problem& p = prm.pr[x.pr];
            const int i = q - p.first, mt = static_cast<int>(fdiv(p.by_n, static_cast<uint32_t>(i)));
            x.m0 = mt * kTileM;
            x.n0 = (i - mt * p.tiles_n) * prm.bn;
            x.kb0 = x.split * prm.blocks_per_split;
            x.nkb = min(prm.blocks_per_split, kblocks - x.kb0);
        } else {
            const int mt = static_cast<int>(fdiv(prm.by_n, t));
            x.m0 = mt * kTileM;
            x.n0 = (static_cast<int>(t) - mt * prm.tiles_n) * prm.bn;
        }
        return x;
    };
    // Columns that a tile's products make: the tile's width, or what is left of the
    // result, in steps of 16.
    auto width_of = [&](const Tile& x) {
        const int left = (OP == kDw ? prm.pr[x.pr].n : prm.n) - x.n0;
        const int w = left < prm.bn ? left : prm.bn;
        return (w + 15) & ~15;
    };

    // 128-row halves of a tile that hold rows of the result.
    auto halves_of = [&](const Tile& x) {
        return kTall && (OP == kDw ? prm.pr[x.pr].m : prm.m) - x.m0 > kBlockM ? 2 : 1;
    };

    if (warp == 0) {
        {
            uint32_t st = 0, ph = 0;
            bool ok = true;
            for (unsigned int t = blockIdx.x; t < prm.tiles && ok; t += gridDim.x) {
                const Tile x = tile_of(t);
                for (int i = 0; i < x.nkb; ++i) {
                    if (!(ok = mbar_wait_warp(&bars->free_[st], ph ^ 1u, ctl, 0x8101))) break;
                    uint64_t* bar = &bars->full[st];
                    const uint32_t s = sbase + st * kStageBytes, sb = s + (kTall ? 2 : 1) * kABytes;
                    const int k0 = (x.kb0 + i) * kBlockK;
                    if (!elect_one()) {
                        // the elected lane copies
                    } else if (OP == kGate) {
                        mbar_arrive_expect_tx(bar, kABytes + 2 * prm.bn * 128);
                        tma_load_2d(s, &maps.a[0], bar, k0, x.m0);
                        tma_load_2d(sb, &maps.b[0], bar, k0, x.n0);
                        tma_load_2d(sb + prm.bn * 128, &maps.b[1], bar, k0, x.n0);
                    } else if (OP == kLinear) {
                        const int halves = halves_of(x);
                        mbar_arrive_expect_tx(bar, halves * kABytes + prm.bn * 128);
                        for (int h = 0; h < halves; ++h) tma_load_2d(s + h * kABytes, &maps.a[0], bar, k0, x.m0 + h * kBlockM);
                        tma_load_2d(sb, &maps.b[0], bar, k0, x.n0);
                    } else if (OP == kGrad) {
                        mbar_arrive_expect_tx(bar, 2 * kABytes + 3 * 64 * 128);
                        tma_load_2d(s, &maps.a[0], bar, k0, x.m0);
                        tma_load_2d(sb, &maps.b[0], bar, k0, x.n0);
                        tma_load_2d(sb + 64 * 128, &maps.b[1], bar, k0, x.n0);
                        tma_load_2d(sb + 2 * 64 * 128, &maps.b[2], bar, x.n0, k0);
                        tma_load_2d(s + kABytes + 3 * 8192, &maps.a[1], bar, k0, x.m0);
                    } else if (OP == kDx) {
                        const int seg = i >= kblocks ? 1 : 0, kk = k0 - seg * kblocks * kBlockK;
                        const int halves = halves_of(x);
                        mbar_arrive_expect_tx(bar, halves * kABytes + prm.bn * 128);
                        for (int h = 0; h < halves; ++h) tma_load_2d(s + h * kABytes, &maps.a[seg], bar, kk, x.m0 + h * kBlockM);
                        for (int b = 0; b < prm.bn / 64; ++b) tma_load_2d(sb + b * 8192, &maps.b[seg], bar, x.n0 + 64 * b, kk);
                    } else {
                        const int halves = halves_of(x);
                        mbar_arrive_expect_tx(bar, halves * kABytes + prm.bn * 128);
                        for (int b = 0; b < 2 * halves; ++b) tma_load_2d(s + b * 8192, &maps.a[x.pr], bar, x.m0 + 64 * b, k0);
                        for (int b = 0; b < prm.bn / 64; ++b)
                            tma_load_2d(sb + b * 8192, &maps.b[x.pr], bar, x.n0 + 64 * b, k0);
                    }
                    __syncwarp();
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
    } else if (warp == 1) {
        {
            uint32_t st = 0, ph = 0, n = 0;
            bool ok = true;
            for (unsigned int t = blockIdx.x; t < prm.tiles && ok; t += gridDim.x, ++n) {
                const Tile x = tile_of(t);
                const uint32_t buf = kTall ? 0u : n & 1u, turn = kTall ? n : n >> 1;
                const uint32_t acc = tmem + 256 * buf;
                if (!mbar_wait_warp(&bars->acc_free[buf], (turn & 1u) ^ 1u, ctl, 0x8102)) break;
                tc_fence_after();
                const int width = width_of(x);
                const uint32_t id = OP == kGate   ? make_idesc_bf16(kBlockM, 2 * prm.bn, false, false)
                                    : OP == kGrad ? make_idesc_bf16(kBlockM, 128, false, false)
                                    : OP == kDw   ? make_idesc_bf16(kBlockM, width, true, true)
                                                  : make_idesc_bf16(kBlockM, width, false, OP == kDx);
                const uint32_t id_dh = make_idesc_bf16(kBlockM, 64, false, true);
                const uint32_t id_ones = make_idesc_bf16(kBlockM, 16, true, false);
                const bool bias = OP == kDw && x.n0 == 0 && prm.pr[x.pr].bias_part != nullptr && !prm.pr[x.pr].turned;
                const int halves = halves_of(x);
                for (int i = 0; i < x.nkb; ++i) {
                    if (!(ok = mbar_wait_warp(&bars->full[st], ph, ctl, 0x8103))) break;
                    tc_fence_after();
                    const uint32_t s = sbase + st * kStageBytes, sb = s + (kTall ? 2 : 1) * kABytes;
                    const int kb = OP == kDx && i >= kblocks ? i - kblocks : x.kb0 + i;
                    const int left = prm.k - kb * kBlockK;
                    const int steps = left >= kBlockK ? kBlockK / 16 : (left + 15) / 16;
                    const bool issue = elect_one();
                    for (int k = 0; issue && k < steps; ++k) {
                        const uint32_t more = i > 0 || k > 0;
                        if (OP == kDw) {
                            for (int h = 0; h < halves; ++h) {
                                const uint64_t da = make_sdesc(s + h * kABytes, 8192, 1024, kSw128) + 128 * k;
                                umma_ss(acc + 256 * h, da, make_sdesc(sb, 8192, 1024, kSw128) + 128 * k, id, more);
                                if (bias)
                                    umma_ss(acc + 256 * h + kColOnes, da, make_sdesc(smem_u32(ones), 16, 1024, kSw128) + 2 * k,
                                            id_ones, more);
                            }
                        } else {
                            const uint64_t db = OP == kDx ? make_sdesc(sb, 8192, 1024, kSw128) + 128 * k
                                                          : make_sdesc(sb, 16, 1024, kSw128) + 2 * k;
                            for (int h = 0; h < halves; ++h)
                                umma_ss(acc + 256 * h, make_sdesc(s + h * kABytes, 16, 1024, kSw128) + 2 * k, db, id, more);
                            if (OP == kGrad)
                                umma_ss(acc + 128, make_sdesc(s + kABytes + 3 * 8192, 16, 1024, kSw128) + 2 * k,
                                        make_sdesc(sb + 2 * 64 * 128, 8192, 1024, kSw128) + 128 * k, id_dh, more);
                        }
                    }
                    if (issue) umma_commit(&bars->free_[st]);
                    __syncwarp();
                    if (++st == stages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok && elect_one()) umma_commit(&bars->acc_full[buf]);
                __syncwarp();
            }
            if (elect_one()) umma_commit(&bars->done);  // every product issued here has completed before the columns are freed
            mbar_wait_warp(&bars->done, 0, ctl, 0x81ff);
        }
    } else if (OP == kDw && warp < 4) {
        // dy's columns: a warp adds 32 of a block's 64 tokens in the tiles of the first
        // rows, an eighth of a box's columns a lane, four tokens at a time
        uint32_t st = 0, ph = 0;
        bool ok = true;
        for (unsigned int t = blockIdx.x; t < prm.tiles && ok; t += gridDim.x) {
            const Tile x = tile_of(t);
            const Problem& p = prm.pr[x.pr];
            const bool adds = p.turned && x.m0 == 0 && p.bias_part;
            float sum[kTallMaxN / 64][8] = {};
            for (int i = 0; i < x.nkb; ++i) {
                if (!(ok = mbar_wait_warp(&bars->full[st], ph, ctl, 0x8105))) break;
                if (adds) {
                    const uint8_t* b = smem + st * kStageBytes + 2 * kABytes;
#pragma unroll
                    for (int c = 0; c < kTallMaxN / 64; ++c) {
                        if (c >= prm.bn / 64) break;
#pragma unroll
                        for (int r = 0; r < 8; ++r) {
                            const int row = (warp - 2) * 32 + r * 4 + (lane >> 3);
                            const uint4 v = *reinterpret_cast<const uint4*>(b + c * 8192 + row * 128 + (((lane ^ row) & 7) << 4));
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                sum[c][2 * e] += bf16lo_to_f32(w[e]);
                                sum[c][2 * e + 1] += bf16hi_to_f32(w[e]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->free_[st]);
                if (++st == stages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (!adds) continue;
            float* dst = p.bias_part + (static_cast<long long>(x.split) * 2 + warp - 2) * p.n + x.n0;
#pragma unroll
            for (int c = 0; c < kTallMaxN / 64; ++c) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum[c][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[c][e], 8);
                    sum[c][e] += __shfl_xor_sync(0xFFFFFFFFu, sum[c][e], 16);
                }
                const int col = c * 64 + lane * 8;  // of the tile
                if (lane < 8 && col < prm.bn && x.n0 + col < p.n) {
                    *reinterpret_cast<float4*>(dst + col) = make_float4(sum[c][0], sum[c][1], sum[c][2], sum[c][3]);
                    *reinterpret_cast<float4*>(dst + col + 4) = make_float4(sum[c][4], sum[c][5], sum[c][6], sum[c][7]);
                }
            }
        }
    } else if (warp >= 4) {
        const int ew = warp - 4, quad = ew & 3, first = 32 * (ew >> 2);  // its first columns
        constexpr int kStep = 8 * kEpiWarps, kBufs = 16 / kEpiWarps;     // columns of a round, store buffers a warp
        const int row_in = quad * 32 + lane;
        uint32_t n = 0, sbuf = 0;
        // A warp's store buffer, once its last store has read it: takes the bias columns,
        // then a 32 x 32 block of results in bf16, stored by TMA (which leaves out what
        // lies outside the result).
        auto buffer = [&]() {
            if (kBufs == 2) bulk_wait_read_but1();
            else bulk_wait_read_all();
            __syncwarp();
            return kStoreOff + (ew * kBufs + (kBufs == 2 ? static_cast<int>(sbuf & 1u) : 0)) * kStoreBytes;
        };
        auto put = [&](const CUtensorMap* m, const unsigned long long (&x)[16], int col, int row0) {
            const int buf = buffer();
            uint8_t* dst = smem + buf + lane * 64;
            const int sw = (lane >> 1) & 3;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float lo, hi;
                    unpair(x[4 * c + e], lo, hi);
                    w[e] = pack_bf16x2(lo, hi);
                }
                *reinterpret_cast<uint4*>(dst + ((c ^ sw) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_2d(m, sbase + buf, col, row0);
                bulk_commit();
            }
            ++sbuf;
        };
        for (unsigned int t = blockIdx.x; t < prm.tiles; t += gridDim.x, ++n) {
            const Tile x = tile_of(t);
            const uint32_t tbuf = kTall ? 0u : n & 1u, turn = kTall ? n : n >> 1;
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars->acc_full[tbuf], turn & 1u, ctl, 0x8104));
            if (!ok) break;
            tc_fence_after();
            const uint32_t acc = tmem + 256 * tbuf + (static_cast<uint32_t>(quad * 32) << 16);
            if (OP == kDw) {
                const Problem& p = prm.pr[x.pr];
                const int width = width_of(x);
                for (int h = 0; h < halves_of(x); ++h) {
                    const int row = x.m0 + h * kBlockM + row_in;
                    float* part = p.part + static_cast<long long>(x.split) * p.m * p.n;
                    for (int c = first; c < width; c += kStep) {
                        uint32_t v[32];
                        tmem_ld32(acc + 256 * h + c, v);
                        tmem_wait_ld();
                        const int col = x.n0 + c;
                        if (row >= p.m) {
                            // nothing to store
                        } else if (p.turned) {  // a warp's 32 rows adjoin
                            float* dst = part + static_cast<long long>(col) * p.m + row;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (col + e < p.n) dst[static_cast<long long>(e) * p.m] = __uint_as_float(v[e]);
                        } else {
                            float* dst = part + static_cast<long long>(row) * p.n + col;
#pragma unroll
                            for (int e = 0; e < 32; e += 4)
                                if (col + e < p.n)
                                    *reinterpret_cast<uint4*>(dst + e) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        }
                    }
                    if (first == 0 && x.n0 == 0 && p.bias_part && !p.turned) {
                        uint32_t v[16];
                        tmem_ld16(acc + 256 * h + kColOnes, v);
                        tmem_wait_ld();
                        if (row < p.m) p.bias_part[static_cast<long long>(x.split) * p.m + row] = __uint_as_float(v[0]);
                    }
                }
            } else {
                const int left = prm.n - x.n0, width = left < prm.bn ? left : prm.bn;
                // kTall: the halves' columns one after the other
                for (int i = first, all = halves_of(x) * ((width + 31) & ~31); i < all; i += kStep) {
                    const int h = kTall && i >= ((width + 31) & ~31) ? 1 : 0, c = i - h * ((width + 31) & ~31);
                    const int col = x.n0 + c, row0 = x.m0 + h * kBlockM + quad * 32;
                    Cols ca, cu, cd;
                    ca.load(acc + 256 * h + c);
                    if (OP == kGate || OP == kGrad) cu.load(acc + prm.bn + c);
                    if (OP == kGrad) cd.load(acc + 128 + c);
                    const float b0 = OP == kDx ? 0.f : bias_at(prm.bias0, col + lane, prm.n);
                    const float b1 = OP == kGate || OP == kGrad ? bias_at(prm.bias1, col + lane, prm.n) : 0.f;
                    float* wbias = reinterpret_cast<float*>(smem + buffer());
                    tmem_wait_ld();
                    unsigned long long a[16];
                    ca.get(a);
                    if (OP != kDx && prm.bias0) add_bias(a, wbias, b0, lane);
                    if (OP == kGate || OP == kGrad) {
                        unsigned long long u[16];
                        cu.get(u);
                        if (prm.bias1) add_bias(u, wbias, b1, lane);
                        if (OP == kGate) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                unsigned long long f[4], s[4];
                                activate<false>(a + e, prm.act, f, s);
#pragma unroll
                                for (int i = 0; i < 4; ++i) a[e + i] = mul_pair(f[i], u[e + i]);
                            }
                        } else {
                            unsigned long long dh[16];
                            cd.get(dh);
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                unsigned long long f[4], s[4];
                                activate<true>(a + e, prm.act, f, s);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    a[e + i] = mul_pair(f[i], u[e + i]);
                                    u[e + i] = mul_pair(mul_pair(dh[e + i], u[e + i]), s[i]);  // dg
                                    dh[e + i] = mul_pair(dh[e + i], f[i]);                     // du
                                }
                            }
                            put(&maps.out[1], u, col, row0);
                            put(&maps.out[2], dh, col, row0);
                        }
                    }
                    put(&maps.out[0], a, col, row0);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->acc_free[tbuf]);
        }
        bulk_wait_all();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// Weight and bias gradients: the splits' partial results added in order.
struct SumParams {
    const float* part[6];
    __nv_bfloat16* out[6];
    long long size[6];
    long long blocks[7];  // first block of each result
    int splits[6];
};
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ SumParams p) {
    int i = 0;
    while (blockIdx.x >= p.blocks[i + 1]) ++i;
    const long long e = ((blockIdx.x - p.blocks[i]) * 256 + threadIdx.x) * 4;
    if (e >= p.size[i]) return;  // sizes are multiples of 8
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < p.splits[i]; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(p.part[i] + k * p.size[i] + e);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *reinterpret_cast<uint2*>(p.out[i] + e) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

template <int OP, bool kTall = OP == kDw>
cudaError_t launch(const Maps& maps, const Params& prm, int num_sms, cudaStream_t stream) {
    static SmemOptIn optin;
    if (cudaError_t e = optin.ensure(reinterpret_cast<const void*>(mlp_kernel<OP, kTall>), kSmemBytes)) return e;
    const unsigned int grid = prm.tiles < static_cast<unsigned>(num_sms) ? prm.tiles : num_sms;
    mlp_kernel<OP, kTall><<<grid, threads_of(OP), kSmemBytes, stream>>>(maps, prm);
    return cudaGetLastError();
}

// The equal tiles of at most `most` columns (a multiple of `step`) that cover n.
inline int tile_width(int n, int most, int step) {
    const int tiles = (n + most - 1) / most;
    return ((n + tiles - 1) / tiles + step - 1) / step * step;
}

// Tiles of a kLinear or kDx launch whose m, n, k and segments are set.  Tall ones read
// less into shared memory but leave their epilogue uncovered, so they are for long
// contractions (dx at 32768 x 384 x 1024, 32 blocks: 56 -> 48 us; at 131072 x 192 x 512,
// 16 blocks: 61 -> 63 us), and for enough rows to give every SM a tile.
inline bool take_tall(Params* p, int step, int num_sms) {
    const long long blocks = static_cast<long long>((p->k + kBlockK - 1) / kBlockK) * (p->segments ? p->segments : 1);
    p->bn = tile_width(p->n, kTallMaxN, step);
    p->tiles_n = (p->n + p->bn - 1) / p->bn;
    long long rows = (static_cast<long long>(p->m) + 2 * kBlockM - 1) / (2 * kBlockM);
    const bool tall = blocks >= 24 && rows * p->tiles_n >= num_sms;
    if (!tall) {
        p->bn = tile_width(p->n, 256, step);
        p->tiles_n = (p->n + p->bn - 1) / p->bn;
        rows = (static_cast<long long>(p->m) + kBlockM - 1) / kBlockM;
    }
    p->tiles = static_cast<unsigned>(rows * p->tiles_n);
    p->by_n = make_fastdiv(p->tiles_n);
    return tall;
}

// Splits of the tokens for the weight gradients: of 1 .. 16 the one with the least
// work on the busiest SM (waves / splits), more splits costing 1 % each for their
// partial results; no split shorter than four blocks.  From the shape alone (a B200's SMs),
// so that the workspace holds the partial results of the splits that are taken, no more.
constexpr int kSms = 148;
constexpr int kMaxSplits = 16;
inline int pick_splits(int tiles, int kblocks) {
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= kMaxSplits; ++s) {
        const int per = (kblocks + s - 1) / s;
        if (s > 1 && (per < 4 || (kblocks + per - 1) / per != s)) continue;
        const double waves = static_cast<double>((static_cast<long long>(tiles) * s + kSms - 1) / kSms);
        const double c = waves * per * (1.0 + 0.01 * s);
        if (c < cost) {
            cost = c;
            best = s;
        }
    }
    return best;
}

// The weight gradients' launch: tiles of 256 hidden channels and bn channels, three times
// over, each split.
struct DwPlan {
    int bn, tiles_n, tiles, kblocks, splits;
};
inline DwPlan dw_plan(const MlpShape& sh) {
    DwPlan p;
    p.bn = tile_width(sh.channels, kTallMaxN, 64);
    p.tiles_n = (sh.channels + p.bn - 1) / p.bn;
    p.tiles = (sh.hidden + 2 * kBlockM - 1) / (2 * kBlockM) * p.tiles_n;
    p.kblocks = static_cast<int>((sh.tokens + kBlockK - 1) / kBlockK);
    p.splits = pick_splits(3 * p.tiles, p.kblocks);
    return p;
}

}  // namespace mlp

// ------------------------------------------------------------------ host
namespace {

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

struct BwdLayout {
    size_t h, dg, du, part[3], bias[3], total;
};
BwdLayout bwd_layout(const MlpShape& sh) {
    const size_t tf = round256(static_cast<size_t>(sh.tokens) * sh.hidden * 2);
    const size_t splits = static_cast<size_t>(mlp::dw_plan(sh).splits);
    const size_t cf = static_cast<size_t>(sh.channels) * sh.hidden * 4 * splits;
    BwdLayout L{};
    size_t o = 0;
    L.h = o;  o += tf;
    L.dg = o; o += tf;
    L.du = o; o += tf;
    for (int i = 0; i < 3; ++i) {
        L.part[i] = o;
        o += round256(cf);
        L.bias[i] = o;
        o += round256(static_cast<size_t>(i == 2 ? sh.channels : sh.hidden) * 8 * splits);  // two a split at most
    }
    L.total = o;
    return L;
}

}  // namespace

size_t mlp_fwd_workspace_bytes(const MlpShape& sh) {
    return mlp_fits(sh) ? 256 : round256(static_cast<size_t>(sh.tokens) * sh.hidden * 2);
}
size_t mlp_bwd_workspace_bytes(const MlpShape& sh) { return bwd_layout(sh).total; }

cudaError_t launch_mlp_fwd(const MlpShape& sh, const MlpPtrs& p, unsigned int* status, unsigned long long limit_ns,
                           int num_sms, cudaStream_t stream) {
    if (mlp_fits(sh)) return launch_mlp_small_fwd(sh, p, status, limit_ns, num_sms, stream);
    using namespace mlp;
    const int T = static_cast<int>(sh.tokens), C = sh.channels, F = sh.hidden;
    const int rows_m = (T + kBlockM - 1) / kBlockM;
    Maps maps{};
    Params prm{};
    prm.status = status;
    prm.limit_ns = limit_ns;
    prm.act = sh.act;
    prm.m = T;
    prm.n = F;
    prm.k = C;
    prm.bn = tile_width(F, 128, 32);
    prm.tiles_n = (F + prm.bn - 1) / prm.bn;
    prm.tiles = static_cast<unsigned>(rows_m) * prm.tiles_n;
    prm.by_n = make_fastdiv(prm.tiles_n);
    prm.bias0 = static_cast<const __nv_bfloat16*>(p.b_gate);
    prm.bias1 = static_cast<const __nv_bfloat16*>(p.b_up);
    if (encode_matrix(&maps.a[0], p.x, T, C, kBlockM, kBlockK, true) ||
        encode_matrix(&maps.b[0], p.w_gate, F, C, prm.bn, kBlockK, true) ||
        encode_matrix(&maps.b[1], p.w_up, F, C, prm.bn, kBlockK, true) ||
        encode_matrix(&maps.out[0], p.ws, T, F, 32, 32, false))
        return cudaErrorInvalidValue;
    cudaError_t e = launch<kGate>(maps, prm, num_sms, stream);
    if (e != cudaSuccess) return e;
    prm.n = C;
    prm.k = F;
    const bool tall = take_tall(&prm, 32, num_sms);
    prm.bias0 = static_cast<const __nv_bfloat16*>(p.b_down);
    if (encode_matrix(&maps.a[0], p.ws, T, F, kBlockM, kBlockK, true) ||
        encode_matrix(&maps.b[0], p.w_down, C, F, prm.bn, kBlockK, true) ||
        encode_matrix(&maps.out[0], p.y, T, C, 32, 32, false))
        return cudaErrorInvalidValue;
    return tall ? launch<kLinear, true>(maps, prm, num_sms, stream) : launch<kLinear>(maps, prm, num_sms, stream);
}

cudaError_t launch_mlp_bwd(const MlpShape& sh, const MlpPtrs& p, unsigned int* status, unsigned long long limit_ns,
                           int num_sms, cudaStream_t stream) {
    using namespace mlp;
    const int T = static_cast<int>(sh.tokens), C = sh.channels, F = sh.hidden;
    const int rows_m = (T + kBlockM - 1) / kBlockM;
    const BwdLayout L = bwd_layout(sh);
    uint8_t *h = p.ws + L.h, *dg = p.ws + L.dg, *du = p.ws + L.du;
    Maps maps{};
    Params prm{};
    prm.status = status;
    prm.limit_ns = limit_ns;
    prm.act = sh.act;
    // h, dg, du
    prm.m = T;
    prm.n = F;
    prm.k = C;
    prm.bn = 64;
    prm.tiles_n = (F + 63) / 64;
    prm.tiles = static_cast<unsigned>(rows_m) * prm.tiles_n;
    prm.by_n = make_fastdiv(prm.tiles_n);
    prm.bias0 = static_cast<const __nv_bfloat16*>(p.b_gate);
    prm.bias1 = static_cast<const __nv_bfloat16*>(p.b_up);
    if (encode_matrix(&maps.a[0], p.x, T, C, kBlockM, kBlockK, true) ||
        encode_matrix(&maps.a[1], p.dy, T, C, kBlockM, kBlockK, true) ||
        encode_matrix(&maps.b[0], p.w_gate, F, C, 64, kBlockK, true) ||
        encode_matrix(&maps.b[1], p.w_up, F, C, 64, kBlockK, true) ||
        encode_matrix(&maps.b[2], p.w_down, C, F, kBlockK, 64, true) ||
        encode_matrix(&maps.out[0], h, T, F, 32, 32, false) || encode_matrix(&maps.out[1], dg, T, F, 32, 32, false) ||
        encode_matrix(&maps.out[2], du, T, F, 32, 32, false))
        return cudaErrorInvalidValue;
    cudaError_t e = launch<kGrad>(maps, prm, num_sms, stream);
    if (e != cudaSuccess) return e;
    // dx
    prm.n = C;
    prm.k = F;
    prm.segments = 2;
    const bool tall = take_tall(&prm, 64, num_sms);
    if (encode_matrix(&maps.a[0], dg, T, F, kBlockM, kBlockK, true) ||
        encode_matrix(&maps.a[1], du, T, F, kBlockM, kBlockK, true) ||
        encode_matrix(&maps.b[0], p.w_gate, F, C, kBlockK, 64, true) ||
        encode_matrix(&maps.b[1], p.w_up, F, C, kBlockK, 64, true) ||
        encode_matrix(&maps.out[0], p.dx, T, C, 32, 32, false))
        return cudaErrorInvalidValue;
    e = tall ? launch<kDx, true>(maps, prm, num_sms, stream) : launch<kDx>(maps, prm, num_sms, stream);
    if (e != cudaSuccess) return e;
    // weights and biases
    prm.k = T;
    const DwPlan plan = dw_plan(sh);
    prm.bn = plan.bn;
    const void *as[3] = {dg, du, h}, *bs[3] = {p.x, p.x, p.dy};
    void* const outs[6] = {p.dw_gate, p.dw_up, p.dw_down, p.db_gate, p.db_up, p.db_down};
    for (int i = 0; i < 3; ++i) {
        Problem& q = prm.pr[i];
        q.m = F;
        q.n = C;
        q.tiles_n = plan.tiles_n;
        q.by_n = make_fastdiv(plan.tiles_n);
        q.first = i * plan.tiles;
        q.turned = i == 2;
        q.part = reinterpret_cast<float*>(p.ws + L.part[i]);
        q.bias_part = outs[3 + i] ? reinterpret_cast<float*>(p.ws + L.bias[i]) : nullptr;
        if (encode_matrix(&maps.a[i], as[i], T, F, kBlockK, 64, true) || encode_matrix(&maps.b[i], bs[i], T, C, kBlockK, 64, true))
            return cudaErrorInvalidValue;
    }
    prm.splits = plan.splits;
    prm.blocks_per_split = (plan.kblocks + prm.splits - 1) / prm.splits;
    prm.by_splits = make_fastdiv(prm.splits);
    prm.tiles = static_cast<unsigned>(3 * plan.tiles) * prm.splits;
    if ((e = launch<kDw>(maps, prm, num_sms, stream)) != cudaSuccess) return e;
    SumParams sum{};
    int count = 0;
    long long blocks = 0;
    for (int i = 0; i < 6; ++i) {
        if (!outs[i]) continue;
        const Problem& q = prm.pr[i % 3];
        sum.part[count] = i < 3 ? q.part : q.bias_part;
        sum.splits[count] = i == 5 ? 2 * prm.splits : prm.splits;
        sum.out[count] = static_cast<__nv_bfloat16*>(outs[i]);
        sum.size[count] = i < 3 ? static_cast<long long>(C) * F : (i == 5 ? C : F);
        sum.blocks[count] = blocks;
        blocks += (sum.size[count] / 4 + 255) / 256;
        ++count;
    }
    for (int i = count; i < 7; ++i) sum.blocks[i] = blocks;
    sum_kernel<<<static_cast<unsigned>(blocks), 256, 0, stream>>>(sum);
    return cudaGetLastError();
}

}  // namespace fswin

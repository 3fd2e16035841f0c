// Attention with a learned relative position bias: windows of 128 tokens or more
// (M = 16, 32, 64), the table gradient's sums, and the launches of every size.
//
//   S_tu = q_t . k_u / sqrt(32) + T[bucket(i_t - i_u, j_t - j_u)],  P = softmax(S + mask),  O = P V
//   dV = P^T dO, dP = dO V^T, dS = P o (dP - rowsum(dO o O)), dQ = dS K / sqrt(32),
//   dK = dS^T Q / sqrt(32),  dT[b] = sum of dS over the windows and the pairs of bucket b
//
// The bias never becomes an N x N matrix: a CTA serves one head, keeps that head's
// (2M-1)^2 displacement table in shared memory (fp32, in base-2 units), and a row
// thread reads the words of its row's displacements: for 16 keys of one box row
// they are consecutive, at constant offsets from one pointer.  That is one shared
// load a score beside the one exponential a score, which the special function
// unit serves at half the rate of those loads.
//
// Times on one B200 (3 heads): forward of 32 x 128 x 128 tokens, M = 32, shifted: 537 us,
// 294 TFLOP/s, the exponentials alone 274 us; of 2 x 200 x 334, M = 16: 80 us.  Backward of
// 16 x 128 x 128, M = 32: prep 34 us (6.2 TB/s), main 861 us (299 TFLOP/s), post 23 us
// (6.6 TB/s), sums 5 us, the second launch for far tables 5 us.  M = 64, 16 x 128 x 128: forward
// 1302 us, main 6250 us; shifted by 32: 895 and 2346 us.  No unit is full (8 x 128 x 128, M =
// 32, forward and main: issue slots 59 and 52 %, special function 59 and 22 %, tensor 14 and
// 14 %, DRAM 5 %): the waits between the links of a chain are what is left.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "dgeo.cuh"
#include "geometry.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "relbias.cuh"
#include "rows.cuh"
#include "schedule.cuh"

namespace fswin {

namespace relb {

constexpr float kScale = 0.17677669529663688f;  // 1 / sqrt(32)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kSmemLimit = 232448;  // shared memory a CTA can use

// A tile's 128 slots as four chunks of 32: the table offset of chunk c relative to
// the tile's first slot is (c >> 1) x + (c & 1) y, and a chunk's second 16 slots lie
// `half` further on.  kBW: the geometry's box width (boxes of a tile follow each
// other along the columns; at kBW = 4 and M = 16 four of them fill a window row).
template <int kBW>
struct ChunkOffsets {
    int x, y, half;
    __device__ __forceinline__ ChunkOffsets(const Geo& g, int pitch) {
        if (kBW == 64) { x = pitch; y = 32; half = 16; }
        else if (kBW == 32) { x = 2 * pitch; y = pitch; half = 16; }
        else if (kBW == 16) { x = 4 * pitch; y = 2 * pitch; half = pitch; }
        else if (kBW == 8) { x = 8; y = 4 * pitch; half = 2 * pitch; }
        else { x = g.M == 16 ? 4 * pitch : 16; y = 8; half = 4; }
    }
    __device__ __forceinline__ int at(int c) const { return ((c & 2) ? x : 0) + ((c & 1) ? y : 0); }
};

// The 16 table words of a 16-slot group from the word of its first slot: one box
// row of 16, two of 8 or four of 4.  kSign: the direction in which they lie.
template <int kBW, int kSign>
struct BiasRows {
    static constexpr int kRows = kBW >= 16 ? 1 : 16 / kBW;
    const float* rp[kRows];
    __device__ __forceinline__ BiasRows(const float* p, int pitch) {
#pragma unroll
        for (int x = 0; x < kRows; ++x) rp[x] = p + kSign * x * pitch;
    }
    __device__ __forceinline__ float operator[](int e) const {
        return kRows == 1 ? rp[0][kSign * e] : rp[e / kBW][kSign * (e % kBW)];
    }
};

// Table offset of the first slot of tile u of a window.
__device__ __forceinline__ int tile_offset(const Geo& g, int u, int pitch) {
    int i, j;
    tile_row_pos(g, u, 0, &i, &j);
    return i * pitch + j;
}

// The shift-region mask of a window depends on its kind alone (bit 1: in the last row
// of windows, bit 0: in the last column): its tokens from row or column M - s on form
// regions of their own.  One table a CTA: per kind and region class the 16-slot groups
// of each tile that lie in the class, and per kind and tile the tiles it attends.
struct Masks {
    uint8_t groups[4][4][32];
    uint32_t act[4][32];
};

__device__ __forceinline__ uint32_t region_class(const Geo& g, int kind, int i, int j) {
    const uint32_t e = g.M - g.s;
    return ((kind & 2) && static_cast<uint32_t>(i) >= e ? 2u : 0u) | ((kind & 1) && static_cast<uint32_t>(j) >= e ? 1u : 0u);
}

// Ends with a __syncthreads of its own after the first half; the caller's follows.
__device__ __forceinline__ void build_masks(const Geo& g, Masks* m, int tid, int nt) {
    if (!g.s) return;
    for (int x = tid; x < 4 * g.tpw; x += nt) {
        const int kind = x / g.tpw, u = x - kind * g.tpw;
        uint32_t by_class[4] = {0u, 0u, 0u, 0u};
        for (int c = 0; c < 8; ++c) {
            int i, j;
            tile_row_pos(g, u, 16 * c, &i, &j);
            const uint32_t cls = region_class(g, kind, i, j);
#pragma unroll
            for (uint32_t k = 0; k < 4; ++k) by_class[k] |= (cls == k ? 1u : 0u) << c;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) m->groups[kind][k][u] = static_cast<uint8_t>(by_class[k]);
    }
    __syncthreads();
    for (int x = tid; x < 4 * g.tpw; x += nt) {
        const int kind = x / g.tpw, u = x - kind * g.tpw;
        uint32_t act = 0;
        for (int v = 0; v < g.tpw; ++v)
            for (int k = 0; k < 4; ++k)
                if (m->groups[kind][k][u] && m->groups[kind][k][v]) act |= 1u << v;
        m->act[kind][u] = act;
    }
}

// A work item: tile u (0 .. tpw - 1) of a window.
struct Item {
    int b, wr, wc, kind, u;
    uint32_t act;   // tiles of the window that share a pair with it
    long long w0;   // the window's first tile
};

__device__ __forceinline__ Item item_of(const Geo& g, const Masks* m, long long X) {
    Item I;
    const uint32_t gw = static_cast<uint32_t>(X >> g.ltpw);
    I.u = static_cast<int>(X) & (g.tpw - 1);
    I.w0 = X - I.u;
    I.b = static_cast<int>(fdiv(g.fd_nW, gw));
    const uint32_t rem = gw - static_cast<uint32_t>(I.b) * g.nW;
    I.wr = static_cast<int>(fdiv(g.fd_nWw, rem));
    I.wc = static_cast<int>(rem) - I.wr * g.nWw;
    I.kind = g.s ? ((I.wr + 1) * g.M == g.Hp ? 2 : 0) | (I.wc + 1 == g.nWw ? 1 : 0) : 0;
    I.act = I.kind ? m->act[I.kind][I.u] : low_bits(g.tpw);
    return I;
}

// Token of slot r of the item's tile (window position i, j); false outside the grid.
__device__ __forceinline__ bool item_token(const Geo& g, const Item& I, int i, int j, int h, long long* tok) {
    int row = I.wr * g.M + i + g.s, col = I.wc * g.M + j + g.s;
    if (row >= g.Hp) row -= g.Hp;
    if (col >= g.Wp) col -= g.Wp;
    *tok = ((static_cast<long long>(I.b) * g.H + row) * g.W + col) * g.heads + h;
    return row < g.H && col < g.W;
}

// TMA loads of tile u of the item's window from two tensors into consecutive tiles.
__device__ __forceinline__ void load_tiles(const Geo& g, const CUtensorMap* m0, const CUtensorMap* m1, uint8_t* dst,
                                           uint64_t* bar, const Item& I, int u, int h) {
    for (int x = 0; x < g.bpt; ++x) {
        const int k = (u << g.lbpt) + x;
        int row = I.wr * g.M + ((k >> g.lnbc) << g.lbh) + g.s, col = I.wc * g.M + ((k & (g.nbc - 1)) << g.lbw) + g.s;
        if (row >= g.Hp) row -= g.Hp;
        if (col >= g.Wp) col -= g.Wp;
        uint8_t* p = dst + x * g.BT * kRowBytes;
        tma_load_5d(p, m0, bar, 0, h, col, row, I.b);
        if (m1) tma_load_5d(p + kTileBytes, m1, bar, 0, h, col, row, I.b);
    }
}

// ------------------------------------------------------------------ forward
namespace fwd {

// Four workers a CTA, each with 128 TMEM columns and a key tile's chain of its own:
// S = Q K^T, softmax, P V, O += P V.  A worker waits for itself at every link, so the
// SM runs four such chains beside each other: with two (S and P V of neighbouring
// tiles overlapped instead) the special function unit was a third busy.
//   warps 4 w .. 4 w + 3: worker w's softmax, thread = query row, O in registers
//   warp 16 + w:          its copies (TMA, two key/value tiles in flight) and products
// TMEM: S [0, 128); P (bf16) over columns already read [0, 64), P V [64, 96).
constexpr int kWorkers = 4;
constexpr int kThreads = kWorkers * 128 + 128;
constexpr uint32_t kColP = 0, kColO = 64;

struct WorkerBars {
    uint64_t q_full[2], q_free[2], kv_full[2], s_full, p_ready, pv_full, o_read, done;
};
struct Bars {
    WorkerBars w[kWorkers];
    uint32_t tmem_base;
    int abort_flag;
    Masks masks;
};

struct Params {
    Geo g;
    uint8_t* o;
    const __nv_bfloat16* table;
    const int* buckets;
    int n_buckets;
    float* lse;
    unsigned int* status;
    unsigned long long limit_ns;
    int streams;     // CTAs of a head
    int pitch;
    int q_tiles;     // query tiles a worker holds: the next item's comes in early where two fit
    int worker_bytes, tab_off, bar_off;
};

template <int kBW>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ Params prm) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    Bars* bars = reinterpret_cast<Bars*>(smem + prm.bar_off);
    float* tab = reinterpret_cast<float*>(smem + prm.tab_off);
    const Geo& g = prm.g;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const int h = blockIdx.x % g.heads;
    const int wk = warp < 4 * kWorkers ? warp >> 2 : warp - 4 * kWorkers;
    WorkerBars& wb = bars->w[wk];
    const long long stride = static_cast<long long>(kWorkers) * prm.streams;
    const long long X0 = static_cast<long long>(kWorkers) * (blockIdx.x / g.heads) + wk;
    const int pitch = prm.pitch, nq = prm.q_tiles;

    if (tid == 0) {
        for (int w = 0; w < kWorkers; ++w) {
            WorkerBars& b = bars->w[w];
            for (int i = 0; i < 2; ++i) {
                mbar_init(&b.q_full[i], 1);
                mbar_init(&b.q_free[i], 4);
                mbar_init(&b.kv_full[i], 1);
            }
            mbar_init(&b.s_full, 1);
            mbar_init(&b.p_ready, 4);
            mbar_init(&b.pv_full, 1);
            mbar_init(&b.o_read, 4);
            mbar_init(&b.done, 1);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 4 * kWorkers) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    build_masks(g, &bars->masks, tid, kThreads);
    build_bias(tab, pitch, prm.table + static_cast<long long>(h) * prm.n_buckets, prm.buckets, prm.n_buckets, g.M, tid,
               kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base + 128 * wk;
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    // a worker's buffers: the Q tiles (an item's O rows are staged over its Q), two K, V stages
    uint8_t* wsm = smem + wk * prm.worker_bytes;
    uint8_t* kvs = wsm + nq * kTileBytes;

    if (warp >= 4 * kWorkers) {
        if (X0 < g.tiles) {
            const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t id_pv = make_idesc_bf16(kTile, kHeadDim, false, true);
            const uint32_t wbase = smem_u32(wsm);
            const uint64_t dK0 = make_sdesc(wbase, 16, 512, kSw64);
            const uint64_t dMN0 = make_sdesc(wbase, 8192, 512, kSw64);
            const Masks* masks = &bars->masks;
            auto load_q = [&](long long X, uint32_t b) {
                const Item I = item_of(g, masks, X);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&wb.q_full[b], kTileBytes);
                    load_tiles(g, &mq, nullptr, wsm + b * kTileBytes, &wb.q_full[b], I, I.u, h);
                }
                __syncwarp();
            };
            long long LX = X0;  // the key/value tiles of all items in one sequence, two ahead
            Item L{};
            uint32_t Lst = 0;
            auto load_kv = [&]() {
                if (L.act == 0) {
                    if (LX >= g.tiles) return;
                    L = item_of(g, masks, LX);
                    LX += stride;
                }
                const int u = __ffs(L.act) - 1;
                L.act &= L.act - 1u;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&wb.kv_full[Lst], 2 * kTileBytes);
                    load_tiles(g, &mk, &mv, kvs + Lst * 2 * kTileBytes, &wb.kv_full[Lst], L, u, h);
                }
                __syncwarp();
                Lst ^= 1u;
            };
            load_q(X0, 0);
            load_kv();
            if (nq == 2 && X0 + stride < g.tiles) load_q(X0 + stride, 1);
            load_kv();
            uint32_t j = 0, it = 0;
            bool ok = true;
            for (long long X = X0; X < g.tiles && ok; X += stride, ++it) {
                const uint32_t qb = nq == 2 ? it & 1u : 0u;
                const int count = __popc(item_of(g, masks, X).act);
                if (!mbar_wait_warp(&wb.q_full[qb], nq == 2 ? (it >> 1) & 1u : it & 1u, ctl, 0x7601)) break;
                const uint64_t qo = qb * (kTileBytes >> 4);
                for (int c = 0; c < count; ++c, ++j) {
                    const uint32_t st = j & 1u, ph = j & 1u;
                    const uint64_t ko = (nq + 2 * st) * (kTileBytes >> 4), vo = ko + (kTileBytes >> 4);
                    if (!(ok = mbar_wait_warp(&wb.kv_full[st], (j >> 1) & 1u, ctl, 0x7602))) break;
                    if (j > 0 && !(ok = mbar_wait_warp(&wb.o_read, ph ^ 1u, ctl, 0x7603))) break;  // the last P V is read
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kHeadDim / 16; ++k)
                            umma_ss(tmem, dK0 + qo + 2 * k, dK0 + ko + 2 * k, id_s, k > 0);
                        umma_commit(&wb.s_full);
                    }
                    __syncwarp();
                    // the next tile's copies, into the stage whose product was waited for, while
                    // this tile's softmax runs: the copying thread's address arithmetic (thousands
                    // of cycles among sixteen busy warps) stays off the chain
                    if (j > 0) load_kv();
                    if (nq == 2 && c == 0 && it > 0 && X + stride < g.tiles) {
                        // the item before has stored its O from there
                        if (!(ok = mbar_wait_warp(&wb.q_free[qb ^ 1u], ((it - 1u) >> 1) & 1u, ctl, 0x7604))) break;
                        load_q(X + stride, qb ^ 1u);
                    }
                    if (!(ok = mbar_wait_warp(&wb.p_ready, ph, ctl, 0x7605))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            umma_ts(tmem + kColO, tmem + kColP + 8 * k, dMN0 + vo + 64 * k, id_pv, k > 0);
                        umma_commit(&wb.pv_full);
                    }
                    __syncwarp();
                    if (!(ok = mbar_wait_warp(&wb.pv_full, ph, ctl, 0x7606))) break;  // the stage is free
                }
                if (ok && nq == 1 && X + stride < g.tiles) {
                    if (!mbar_wait_warp(&wb.q_free[0], it & 1u, ctl, 0x7607)) break;
                    load_q(X + stride, 0);
                }
            }
            if (elect_one()) umma_commit(&wb.done);  // every product issued here has completed before the columns are freed
            mbar_wait_warp(&wb.done, 0, ctl, 0x76ff);
        }
    } else {
        const int r = tid & (kTile - 1), quad = warp & 3;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const float sl2 = g.scale_log2;
        auto wwait = [&](uint64_t* bar, uint32_t phase, unsigned int where) -> bool {
            return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, ctl, where));
        };
        const ChunkOffsets<kBW> co(g, pitch);
        const unsigned long long sl2_2 = pair(sl2, sl2);
        uint32_t n = 0, it = 0;  // key tiles and items seen
        bool ok = true;
        for (long long X = X0; X < g.tiles && ok; X += stride, ++it) {
            const Item I = item_of(g, &bars->masks, X);
            int pi, pj;
            long long tok;
            tile_row_pos(g, I.u, r, &pi, &pj);
            const bool valid = item_token(g, I, pi, pj, h, &tok);
            const float* brow = tab + (pi + g.M - 1) * pitch + pj + g.M - 1;
            const uint8_t* groups = bars->masks.groups[I.kind][region_class(g, I.kind, pi, pj)];
            float m = -INFINITY;
            unsigned long long l = 0, o[16];  // pairs: the row sum in two parts, O
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0;
            for (uint32_t act = I.act; act != 0u; act &= act - 1u, ++n) {
                const int kt = __ffs(act) - 1;
                const uint32_t a16 = I.kind ? groups[kt] : 0xFFu;
                if (!wwait(&wb.s_full, n & 1u, 0x7608)) { ok = false; break; }
                tc_fence_after();
                const float* btile = brow - tile_offset(g, kt, pitch);
                // one key tile's probabilities; kMasked: some of its groups are not attended
                auto softmax_tile = [&](auto masked) {
                    constexpr bool kMasked = decltype(masked)::value;
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32(trow + 32 * c, v);
                        const BiasRows<kBW, -1> b0(btile - co.at(c), pitch), b1(btile - co.at(c) - co.half, pitch);
                        unsigned long long t[16];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            t[e] = pair(b0[2 * e], b0[2 * e + 1]);
                            t[8 + e] = pair(b1[2 * e], b1[2 * e + 1]);
                        }
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) t[e] = fma_pair(pair(v[2 * e], v[2 * e + 1]), sl2_2, t[e]);
                        if (kMasked) {
                            const bool on0 = (a16 >> (2 * c)) & 1u, on1 = (a16 >> (2 * c + 1)) & 1u;
                            const unsigned long long none = pair(-INFINITY, -INFINITY);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                t[e] = on0 ? t[e] : none;
                                t[8 + e] = on1 ? t[8 + e] : none;
                            }
                        }
                        // The running maximum only moves when a chunk exceeds it by more than
                        // 2^64: probabilities up to 2^64 stay far inside bf16's and fp32's range,
                        // and the final division uses the same maximum as the sum.
                        float c2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x, y;
                            unpair(t[e], x, y);
                            c2[e & 1] = fmax3(c2[e & 1], x, y);
                        }
                        const float cm = fmaxf(c2[0], c2[1]);
                        const bool grow = cm > m + 64.f;
                        if (__any_sync(0xFFFFFFFFu, grow)) {
                            const float alpha = grow ? ex2_approx(m - cm) : 1.f;
                            const unsigned long long alpha2 = pair(alpha, alpha);
                            if (grow) m = cm;
                            l = mul_pair(l, alpha2);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = mul_pair(o[e], alpha2);
                            tmem_wait_st();
#pragma unroll 1
                            for (int k = 0; k < 2 * c; ++k) {  // this tile's chunks already written
                                uint32_t pw[8];
                                tmem_ld8(trow + kColP + 8 * k, pw);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    pw[e] = pack_bf16x2(bf16lo_to_f32(pw[e]) * alpha, bf16hi_to_f32(pw[e]) * alpha);
                                tmem_st8(trow + kColP + 8 * k, pw);
                            }
                        }
                        const float mu = m == -INFINITY ? 0.f : -m;  // no key so far: P = 0
                        const unsigned long long mu2 = pair(mu, mu);
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float p0, p1;
                                unpair(add_pair(t[8 * hh + e], mu2), p0, p1);
                                p0 = ex2_approx(p0);
                                p1 = ex2_approx(p1);
                                l = add_pair(l, pair(p0, p1));
                                w[e] = pack_bf16x2(p0, p1);  // P joins the tensor product in V's type
                            }
                            tmem_st8(trow + kColP + 16 * c + 8 * hh, w);  // over columns of S already read
                        }
                    }
                };
                if (I.kind) softmax_tile(std::true_type{});
                else softmax_tile(std::false_type{});
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wb.p_ready);
                if (!wwait(&wb.pv_full, n & 1u, 0x7609)) { ok = false; break; }
                tc_fence_after();
                uint32_t v[32];
                tmem_ld32(trow + kColO, v);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wb.o_read);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = add_pair(o[e], pair(v[2 * e], v[2 * e + 1]));
            }
            if (!ok) break;
            float la, lb, x[32];
            unpair(l, la, lb);
            la += lb;
            const float inv = 1.f / la;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                unpair(o[e], x[2 * e], x[2 * e + 1]);
                x[2 * e] = la == 0.f ? 0.f : x[2 * e] * inv;  // no key: O = 0
                x[2 * e + 1] = la == 0.f ? 0.f : x[2 * e + 1] * inv;
            }
            const uint32_t qb = nq == 2 ? it & 1u : 0u;
            uint8_t* ost = wsm + qb * kTileBytes;
            store_row_swz(ost, r, x);
            if (valid && prm.lse != nullptr) prm.lse[tok] = (m + lg2_approx(la)) * kLn2;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // eight whole 64-byte rows a store
                const int rl = (lane >> 2) + 8 * i, c = lane & 3;
                const long long tk = __shfl_sync(0xFFFFFFFFu, tok, rl);
                const bool vd = __shfl_sync(0xFFFFFFFFu, valid ? 1 : 0, rl) != 0;
                const int row = quad * 32 + rl;
                if (vd)
                    *reinterpret_cast<uint4*>(prm.o + tk * kRowBytes + 16 * c) =
                        *reinterpret_cast<const uint4*>(ost + row * kRowBytes + ((c ^ ((row >> 1) & 3)) << 4));
            }
            fence_proxy_async_smem();  // the rows are read before TMA writes the next Q over them
            __syncwarp();
            if (lane == 0) mbar_arrive(&wb.q_free[qb]);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 4 * kWorkers) tmem_dealloc(bars->tmem_base, 512);
}

}  // namespace fwd

// ------------------------------------------------------------------ backward
namespace bwd {

struct WsLayout {
    size_t acc, rowv, far, flags, part, disp, total;
    int streams;  // partial sums of the table gradient a head
};

// Workers (independent pipelines) of a CTA of the main kernel: two while their
// buffers and table sums fit shared memory, one at M = 64.
__host__ inline int workers(const Geo& g) { return g.M == 64 ? 1 : 2; }

__host__ inline WsLayout ws_layout(const Geo& g) {
    auto round256 = [](size_t x) { return (x + 255) & ~size_t(255); };
    const size_t ht = static_cast<size_t>(g.heads) * static_cast<size_t>(g.tiles);
    WsLayout L{};
    size_t o = 0;
    if (g.N >= kTile) {
        L.acc = o;  o += round256(ht * kTile * kHeadDim * 4);  // fp32 dQ [heads][tiles][128][32], 16-byte chunks permuted
        L.rowv = o; o += round256(ht * kTile * 8);             // per (head, tile): -lse log2(e) [128], -D [128]
        L.far = o;  o += round256(ht * kTile * 8);             // far_row's terms, of rows whose -lse log2(e) is -inf
        L.flags = o; o += round256(ht * 16);                   // per (head, tile), a bit a row: it has two terms
        const int W = workers(g);
        L.streams = W * streams_per_head((g.tiles + W - 1) / W, g.heads, kSms);
    } else {
        L.streams = streams_per_head(g.tiles, g.heads, small_bwd_ctas(g));
    }
    L.part = o; o += round256(static_cast<size_t>(L.streams) * g.heads * displacements(g.M) * 4);
    L.disp = o; o += round256(static_cast<size_t>(g.heads) * displacements(g.M) * 4);
    L.total = o;
    return L;
}

struct Params {
    Geo g;
    const uint8_t *q, *k, *o, *dout;
    uint8_t *dq, *dk, *dv;
    const float* lse;
    const __nv_bfloat16* table;
    const int* buckets;
    int n_buckets;
    float* acc;
    float* rowv;
    float2* far;
    uint32_t* flags;
    float* part;
    unsigned int* status;
    unsigned long long limit_ns;
    int streams;  // CTAs of a head
    int pitch, kv_stages;
    int worker_bytes, acc_off, tab_off, bar_off;
};

// prep: per (tile, head), thread = slot row: D = dO . O and the row's log-sum-exp
// in base-2 units, and the zeroed dQ accumulator row.  Memory only, but for rows whose
// log-sum-exp is a far one.
__global__ void __launch_bounds__(128, 16) prep_kernel(const __grid_constant__ Params p) {
    const Geo& g = p.g;
    const long long T = blockIdx.x / g.heads;
    const int h = static_cast<int>(blockIdx.x - T * g.heads);
    const long long ht = static_cast<long long>(h) * g.tiles + T;
    const int r = threadIdx.x;
    int pi, pj;
    long long tok;
    float D = 0.f;
    float2 l = make_float2(-INFINITY, 0.f);  // a row outside the grid: no probability
    uint4* acc = reinterpret_cast<uint4*>(p.acc + ht * kTile * kHeadDim);
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[c * 128 + r] = make_uint4(0, 0, 0, 0);
    if (slot_token(g, T, r, h, &pi, &pj, &tok)) {
        const uint4* a = reinterpret_cast<const uint4*>(p.dout + tok * kRowBytes);
        const uint4* b = reinterpret_cast<const uint4*>(p.o + tok * kRowBytes);
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 x = __ldg(a + c), y = __ldg(b + c);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                d[e] = fmaf(bf16lo_to_f32(xs[e]), bf16lo_to_f32(ys[e]),
                            fmaf(bf16hi_to_f32(xs[e]), bf16hi_to_f32(ys[e]), d[e]));
        }
        D = (d[0] + d[1]) + (d[2] + d[3]);
        const float lse = __ldg(p.lse + tok);
        l.x = -grad_lse2(lse);
        if (finite_beyond(lse * 1.4426950408889634f, kFar))
            l = far_row(g, p.q, p.k, p.table + static_cast<long long>(h) * p.n_buckets, p.buckets, p.n_buckets, T, r, h,
                        lse * 1.4426950408889634f);
    }
    // Rows with a second term have no probability for the main kernel; the one for far
    // tables looks here for every row that has none (a second term of 0: no key).
    const uint32_t two = __ballot_sync(0xFFFFFFFFu, l.y != 0.f);
    if ((r & 31) == 0) p.flags[ht * 4 + (r >> 5)] = two;
    if (l.y != 0.f || l.x == -INFINITY) {
        p.far[ht * kTile + r] = l;
        l.x = -INFINITY;
    }
    p.rowv[ht * 2 * kTile + r] = l.x;  // negated: the main kernel adds them, packed
    p.rowv[ht * 2 * kTile + kTile + r] = -D;
}

// Main kernel: a worker is eight warps with 256 TMEM columns, its own buffers and
// barriers; two warpgroups split a step's query columns, thread = key row (and query
// row of dQ).  Item = (key tile, head): the query tiles of its window in turn.  A step
//   S^T = K Q^T, dP^T = V dO^T; P^T and dS^T (bf16, the products' operand type) over
//   columns that the warpgroup has read, dS also to shared memory; dV = P^T dO,
//   dK = dS^T Q, dQ = dS K
// adds dV (first warpgroup) and dK (second) up in registers; dQ is staged over the
// step's Q and dO tiles and added into the fp32 accumulator tile with one bulk
// reduction.  While the three products run, one warpgroup (they take turns) sums dS
// over equal displacements.  Two workers a CTA fill each other's waits; a warpgroup of
// its own copies (warps 2, 3) and issues the products (warps 0, 1): issued by a
// computing thread, the copies cost its warp 2.7 thousand cycles a step and the
// products 1.7, for which the other warps then waited.
// TMEM columns: S^T [0,128), dP^T [128,256).  P^T of the first warpgroup [0,32), of the
// second [64,96); dS^T [128,160) and [192,224); dV [32,64), dQ [96,128), dK [160,192).
constexpr uint32_t kColS = 0, kColDP = 128, kColDV = 32, kColDQ = 96, kColDK = 160;
constexpr int kStageBytes = 2 * kTileBytes + 1024;  // Q, dO, and the rows' -lse2 and -D

struct WorkerBars {
    // dq_ready per stage: the copies may lag a step behind the next one's dQ
    uint64_t kv_full[2], st_full[2], s_full, p_ready, mma_done, dq_ready[2], done;
};
struct Bars {
    WorkerBars w[2];
    uint32_t tmem_base;
    int abort_flag;
    Masks masks;
};

// A worker's shared memory: dS, K and V (kv_stages), two query stages, the table sums.
constexpr int kKVOff = 4 * kTileBytes;
__host__ __device__ constexpr int stage_off(int kv_stages) { return kKVOff + kv_stages * 2 * kTileBytes; }
__host__ __device__ constexpr int sums_off(int kv_stages) { return stage_off(kv_stages) + 2 * kStageBytes; }

// Adds one step's dS (bf16 in shared memory, [key row][query], 128-byte swizzle)
// into the worker's displacement sums.  The tile's slots fall into row segments of
// w = min(bw, 32) tokens; a pair of segments (key a, query b) is a w x w block
// whose entries of equal query column minus key row share a displacement.  Warp
// `quad` takes the blocks whose row displacement is quad modulo 4, so no two warps
// touch one sum and every sum has a fixed order.  Lane (g, kp, m) walks block g's
// keys 4 kk + kp and query quads kk + m (mod w / 4): eight bytes a load, and its
// four columns e belong to displacement 4 m + e - kp, or w less once the quads wrap,
// each with a register of its own: a small sum beside a large one keeps its digits, and
// a value that is not finite stays with its own.  Blocks of equal displacement follow
// each other and add up there first.  What is added is dS as the products take it, in
// bf16: it lies in shared memory only so, and half a step of a term, 2^-8, is what the
// products' results (dQ, dK) carry too; the sums are fp32.
template <int kBW>  // 4, 8, 16, 32, 64: the geometry's box width
struct Diag {
    static constexpr int w = kBW < 32 ? kBW : 32;
    static constexpr int quads = w / 4;
    static constexpr int conc = 32 / w;         // blocks a warp walks at once
    static constexpr int nseg = kTile / w;
    unsigned long long A[2], B[2];  // columns (0, 1), (2, 3): before the quads wrap, and after

    __device__ __forceinline__ void clear() { A[0] = A[1] = B[0] = B[1] = 0; }
    // One predicate a load.  (A sum of all columns and one with a weight of 0 or 1, and the
    // second from their difference, took 858 us in place of 875 at 16 x 128 x 128 tokens, M =
    // 32, and 176 in place of 173 at 2 x 200 x 334, M = 16: the difference lost the digits of
    // a small sum beside a large one.)
    __device__ __forceinline__ void add(unsigned long long v0, unsigned long long v1, int quad) {
        asm("{\n\t.reg .pred p;\n\tsetp.lt.s32 p, %6, %7;\n\t"
            "@p add.rn.f32x2 %0, %0, %4;\n\t@p add.rn.f32x2 %1, %1, %5;\n\t"
            "@!p add.rn.f32x2 %2, %2, %4;\n\t@!p add.rn.f32x2 %3, %3, %5;\n\t}"
            : "+l"(A[0]), "+l"(A[1]), "+l"(B[0]), "+l"(B[1])
            : "l"(v0), "l"(v1), "r"(quad), "n"(quads));
    }
    // Shared address of the lane's first load of a key segment's rows: key kp, query
    // column 0; and the lane's offsets from there for every kk (the swizzle of key row
    // r: 16-byte chunk index xor r & 7).
    __device__ __forceinline__ void walk(uint32_t rows, const uint32_t (&off)[quads], uint32_t flip, int m) {
#pragma unroll
        for (int kk = 0; kk < quads; ++kk) {
            uint32_t x, y;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(rows + (off[kk] ^ flip)));
            const unsigned long long v0 = pair(x << 16, x & 0xFFFF0000u), v1 = pair(y << 16, y & 0xFFFF0000u);
            if (quads > 1) {
                add(v0, v1, kk + m);
            } else {
                A[0] = add_pair(A[0], v0);
                A[1] = add_pair(A[1], v1);
            }
        }
    }
    // dst: the sum of displacement 4 m - kp of this lane's block.  Lanes of one block
    // hold distinct displacements for one e, and so do the blocks walked at once; the
    // wrapped ones of a neighbouring block may coincide with those, so they follow in
    // a step of their own.
    __device__ __forceinline__ void flush(float* dst, int m) {
        float a[4], b[4];
        unpair(A[0], a[0], a[1]);
        unpair(A[1], a[2], a[3]);
        unpair(B[0], b[0], b[1]);
        unpair(B[1], b[2], b[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dst[e] += a[e];
            if (conc > 1) __syncwarp();
            if (quads > 1 && m > 0) dst[e - w] += b[e];
            __syncwarp();
        }
        clear();
    }

    static __device__ __forceinline__ void step(const Geo& g, uint32_t ds, float* sums, int ku, int qt,
                                                int quad, int lane, int side) {
        const int kp = lane & 3, m = (lane >> 2) & (quads - 1), gi = lane / (4 * quads);
        uint32_t off[quads];
#pragma unroll
        for (int kk = 0; kk < quads; ++kk) {
            const uint32_t r = 4 * kk + kp, p = (kk + m) & (quads - 1);
            off[kk] = ((r >> 3) << 10) + ((r & 7) << 7) + ((((p >> 1) ^ (r & 7)) << 4) | ((p & 1) << 3));
        }
        // window positions of the tiles' first slots; a segment's from there
        int ki0, kj0, qi0, qj0;
        tile_row_pos(g, ku, 0, &ki0, &kj0);
        tile_row_pos(g, qt, 0, &qi0, &qj0);
        float* origin = sums + (qi0 - ki0 + g.M - 1) * side + (qj0 - kj0 + g.M - 1) + 4 * m - kp;
        Diag d;
        d.clear();
        int last = 0;
        bool some = false;
        auto block = [&](int a, int b, int di, int dj) {  // di, dj: of the segments, relative to the tiles
            const int at = di * side + dj;
            // the blocks walked at once move on together
            if (some && __any_sync(0xFFFFFFFFu, at != last)) d.flush(origin + last, m);
            last = at;
            some = true;
            const int q0 = b * w;
            // key rows a w ..: whole eight-row groups, or (w = 4) half of one, whose rows
            // 4 .. 7 have the swizzle's bit 2 set
            const uint32_t rows = ds + ((q0 >> 6) << 14) + (((a * w) >> 3) << 10) + (w == 4 ? ((a & 1) << 9) : 0);
            const uint32_t flip = (((q0 & 63) >> 3) ^ (w == 4 ? ((a & 1) << 2) : 0)) << 4 | (w == 4 ? ((q0 & 4) << 1) : 0);
            d.walk(rows, off, flip, m);
        };
        if (kBW == 64) {  // two rows of two 32-column segments
#pragma unroll 1
            for (int ab = 0; ab < 16; ++ab) {  // key row, query row, halves: equal displacements in a row
                const int ra = ab >> 3, rb = (ab >> 2) & 1, ha = (ab >> 1) & 1, hb = ab & 1;
                if (((qi0 - ki0 + rb - ra) & 3) != quad) continue;
                block(2 * ra + ha, 2 * rb + hb, rb - ra, 32 * (hb - ha));
            }
        } else {
            // boxes of bh rows (a multiple of 4, at multiples of 4): segment = box bh + row;
            // boxes of a tile along the columns, but at kBW = 4, M = 16 two rows of four
            constexpr int bh = kBW == 32 ? 4 : (kBW == 16 ? 8 : kBW);
            constexpr int per = bh / 4;  // matching rows a box
            const int wrapped = kBW == 4 && g.M == 16;
            const int xb = gi / per;
            const int bi = wrapped ? (xb >> 2) * 4 : 0, bj = (wrapped ? xb & 3 : xb) * kBW;
#pragma unroll 1
            for (int a = 0; a < nseg; ++a) {
                const int xa = a / bh, ra = a & (bh - 1);
                const int rb = ((ra + quad) & 3) + 4 * (gi % per);
                const int ai = wrapped ? (xa >> 2) * 4 : 0, aj = (wrapped ? xa & 3 : xa) * kBW;
                block(a, xb * bh + rb, bi + rb - ai - ra, bj - aj);
            }
        }
        if (some) d.flush(origin + last, m);
    }
};

// kFarTable: a second launch for rows with two terms (prep_kernel), from which CTAs leave at
// once whose head's table has no far entry, or whose windows no such row.  It forms dK and dV
// again, with those rows among the others, and adds to dQ and the table's sums the part of
// those rows alone.  A branch of the one kernel, or a way out of it, would be simpler, but
// made it slower for every call (16 x 128 x 128, M = 32: 875 us; with either 912 to 915, and
// the second launch takes 5).
template <int kBW, int kWorkers, bool kFarTable>
__global__ void __launch_bounds__(256 * kWorkers + 128, 1)
    main_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                const __grid_constant__ Params prm) {
    constexpr int kThreads = 256 * kWorkers + 128;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    Bars* bars = reinterpret_cast<Bars*>(smem + prm.bar_off);
    float* tab = reinterpret_cast<float*>(smem + prm.tab_off);
    const Geo& g = prm.g;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const bool computes = warp < 8 * kWorkers;
    const int wk = computes ? warp >> 3 : warp & 1;  // (one worker: its second helpers have no item)
    const int h = blockIdx.x % g.heads;
    WorkerBars& wb = bars->w[wk];
    const int pitch = prm.pitch, side = 2 * g.M - 1, kvs = prm.kv_stages;
    uint8_t* wsm = smem + wk * prm.worker_bytes;
    float* sums = reinterpret_cast<float*>(wsm + prm.acc_off);
    const long long stride = static_cast<long long>(kWorkers) * prm.streams;
    const long long X0 = static_cast<long long>(kWorkers) * (blockIdx.x / g.heads) + wk;
    const long long item0 = static_cast<long long>(h) * g.tiles;
    const __nv_bfloat16* table_h = prm.table + static_cast<long long>(h) * prm.n_buckets;
    if (kFarTable &&
        !__syncthreads_or(build_bias(tab, pitch, table_h, prm.buckets, prm.n_buckets, g.M, tid, kThreads)))
        return;
    if (kFarTable) {  // the four words of every query tile of every item
        uint32_t some = 0;
        const long long first = static_cast<long long>(kWorkers) * (blockIdx.x / g.heads);
        for (int w = 0; w < kWorkers; ++w)
            for (long long X = first + w; X < g.tiles; X += stride)
                for (int e = tid; e < 4 * g.tpw; e += kThreads)
                    some |= __ldg(prm.flags + (item0 + (X & ~static_cast<long long>(g.tpw - 1))) * 4 + e);
        if (!__syncthreads_or(some != 0)) return;
    }

    if (tid == 0) {
        for (int w = 0; w < kWorkers; ++w) {
            WorkerBars& b = bars->w[w];
            for (int i = 0; i < 2; ++i) {
                mbar_init(&b.kv_full[i], 1);
                mbar_init(&b.st_full[i], 1);
                mbar_init(&b.dq_ready[i], 8);
            }
            mbar_init(&b.s_full, 1);
            mbar_init(&b.p_ready, 8);
            mbar_init(&b.mma_done, 1);
            mbar_init(&b.done, 1);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8 * kWorkers) {
        tmem_alloc(&bars->tmem_base, 256 * kWorkers);
        tmem_relinquish();
    }
    build_masks(g, &bars->masks, tid, kThreads);
    if (!kFarTable) build_bias(tab, pitch, table_h, prm.buckets, prm.n_buckets, g.M, tid, kThreads);
    if (computes)
        for (int e = tid & 255; e < side * side; e += 256) sums[e] = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base + 256 * wk;
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    const int st0 = stage_off(kvs);

    if (!computes) {
        const int role = (warp - 8 * kWorkers) >> 1;  // 0: products, 1: copies
        if (wk < kWorkers && X0 < g.tiles && role == 1) {
            // the query tiles of all items in one sequence, two steps ahead
            long long LX = X0, Tst0 = 0, Tst1 = 0;
            Item L{};
            uint32_t Lst = 0;
            auto load_kv = [&](long long X, uint32_t b) {
                const Item I = item_of(g, &bars->masks, X);
                if (elect_one()) {
                    mbar_arrive_expect_tx(&wb.kv_full[b], 2 * kTileBytes);
                    load_tiles(g, &mk, &mv, wsm + kKVOff + b * 2 * kTileBytes, &wb.kv_full[b], I, I.u, h);
                }
                __syncwarp();
            };
            auto load_step = [&]() {
                if (L.act == 0) {
                    if (LX >= g.tiles) return;
                    L = item_of(g, &bars->masks, LX);
                    LX += stride;
                }
                const int u = __ffs(L.act) - 1;
                const long long T = L.w0 + u;
                L.act &= L.act - 1u;
                uint8_t* d = wsm + st0 + Lst * kStageBytes;
                uint64_t* bar = &wb.st_full[Lst];
                if (elect_one()) {
                    mbar_arrive_expect_tx(bar, kStageBytes);
                    load_tiles(g, &mq, &mdo, d, bar, L, u, h);
                    bulk_load(d + 2 * kTileBytes, prm.rowv + (item0 + T) * 2 * kTile, 1024, bar);
                }
                __syncwarp();
                if (Lst) Tst1 = T;
                else Tst0 = T;
                Lst ^= 1u;
            };
            load_kv(X0, 0);
            load_step();
            load_step();
            if (kvs == 2 && X0 + stride < g.tiles) load_kv(X0 + stride, 1);
            uint32_t step = 0, item = 0;
            bool ok = true;
            for (long long X = X0; X < g.tiles && ok; X += stride, ++item) {
                const int count = __popc(item_of(g, &bars->masks, X).act);
                for (int c = 0; c < count; ++c, ++step) {
                    if (!(ok = mbar_wait_warp(&wb.dq_ready[step & 1u], (step >> 1) & 1u, ctl, 0x7501))) break;
                    uint8_t* d = wsm + st0 + (step & 1u) * kStageBytes;
                    if (lane == 0) {  // one lane throughout: the waits below are for its own groups
                        bulk_reduce_add_f32(prm.acc + (item0 + ((step & 1u) ? Tst1 : Tst0)) * kTile * kHeadDim, d,
                                            2 * kTileBytes);
                        bulk_commit();
                    }
                    __syncwarp();
                    // the item's products are done with its keys and values
                    if (c == count - 1 && X + kvs * stride < g.tiles) load_kv(X + kvs * stride, kvs == 2 ? item & 1u : 0u);
                    bulk_wait_read_all();
                    __syncwarp();
                    load_step();
                }
            }
            bulk_wait_all();
        } else if (wk < kWorkers && X0 < g.tiles) {
            const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t id_dv = make_idesc_bf16(kTile, kHeadDim, false, true);
            const uint32_t id_dq = make_idesc_bf16(kTile, kHeadDim, true, true);
            const uint32_t wbase = smem_u32(wsm);
            const uint64_t dK0 = make_sdesc(wbase, 16, 512, kSw64);
            const uint64_t dMN0 = make_sdesc(wbase, 8192, 512, kSw64);
            const uint64_t dDS = make_sdesc(wbase, 16384, 1024, kSw128);
            uint32_t step = 0, item = 0;
            bool ok = true;
            for (long long X = X0; X < g.tiles && ok; X += stride, ++item) {
                const int count = __popc(item_of(g, &bars->masks, X).act);
                const uint32_t kvb = kvs == 2 ? item & 1u : 0u;
                const uint64_t ko = (kKVOff + kvb * 2 * kTileBytes) >> 4, vo = ko + (kTileBytes >> 4);
                if (!mbar_wait_warp(&wb.kv_full[kvb], kvs == 2 ? (item >> 1) & 1u : item & 1u, ctl, 0x7502)) break;
                for (int c = 0; c < count; ++c, ++step) {
                    const uint32_t b = step & 1u;
                    const uint64_t qo = static_cast<uint64_t>((st0 + b * kStageBytes) >> 4), dof = qo + (kTileBytes >> 4);
                    if (!(ok = mbar_wait_warp(&wb.st_full[b], (step >> 1) & 1u, ctl, 0x7503))) break;
                    if (step > 0 && !(ok = mbar_wait_warp(&wb.dq_ready[b ^ 1u], ((step - 1u) >> 1) & 1u, ctl, 0x7504))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kHeadDim / 16; ++k) {
                            umma_ss(tmem + kColS, dK0 + ko + 2 * k, dK0 + qo + 2 * k, id_s, k > 0);
                            umma_ss(tmem + kColDP, dK0 + vo + 2 * k, dK0 + dof + 2 * k, id_s, k > 0);
                        }
                        umma_commit(&wb.s_full);
                    }
                    __syncwarp();
                    if (!(ok = mbar_wait_warp(&wb.p_ready, b, ctl, 0x7505))) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            umma_ts(tmem + kColDV, tmem + kColS + 8 * k + (k < 4 ? 0 : 32), dMN0 + dof + 64 * k, id_dv, k > 0);
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            umma_ts(tmem + kColDK, tmem + kColDP + 8 * k + (k < 4 ? 0 : 32), dMN0 + qo + 64 * k, id_dv, k > 0);
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            umma_ss(tmem + kColDQ, dDS + 128 * k, dMN0 + ko + 64 * k, id_dq, k > 0);
                        umma_commit(&wb.mma_done);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) umma_commit(&wb.done);  // every product issued here has completed before the columns are freed
            mbar_wait_warp(&wb.done, 0, ctl, 0x75ff);
        }
    } else {
        const int wg = (warp >> 2) & 1, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const float sl2 = g.scale_log2;
        const ChunkOffsets<kBW> co(g, pitch);
        const unsigned long long sl2_2 = pair(sl2, sl2);
        auto wwait = [&](uint64_t* bar, uint32_t phase, unsigned int where) -> bool {
            return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, ctl, where));
        };
        uint8_t* dsrow = wsm + wg * 16384 + (r >> 3) * 1024 + (r & 7) * 128;
        const uint32_t wbase = smem_u32(wsm);
        uint32_t step = 0, item = 0;
        bool ok = true;
        for (long long X = X0; X < g.tiles && ok; X += stride, ++item) {
            const uint32_t kvb = kvs == 2 ? item & 1u : 0u;  // where the item's keys are
            const Item I = item_of(g, &bars->masks, X);
            int ki, kj;
            long long ktok;
            tile_row_pos(g, I.u, r, &ki, &kj);
            const bool kvalid = item_token(g, I, ki, kj, h, &ktok);
            const float* brow = tab + (g.M - 1 - ki) * pitch + g.M - 1 - kj;
            const uint8_t* groups = bars->masks.groups[I.kind][region_class(g, I.kind, ki, kj)];
            unsigned long long acc[16];  // dV (first warpgroup) or dK (second) of this key row, in pairs
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[e] = 0;
            for (uint32_t act = I.act; act != 0u; act &= act - 1u, ++step) {
                const int T = __ffs(act) - 1;  // query tile of the window
                const uint32_t ph = step & 1u;
                uint8_t* stg = wsm + st0 + ph * kStageBytes;
                const uint32_t a16 = I.kind ? groups[T] : 0xFFu;
                const float* bt = brow + tile_offset(g, T, pitch);
                const float4* neg_l = reinterpret_cast<const float4*>(stg + 2 * kTileBytes);  // of four queries each
                const float4* neg_d = neg_l + kTile / 4;
                if (!wwait(&wb.st_full[ph], (step >> 1) & 1u, 0x7506) || !wwait(&wb.s_full, ph, 0x7507) ||
                    (kFarTable && !wwait(&wb.kv_full[kvb], kvs == 2 ? (item >> 1) & 1u : item & 1u, 0x750a))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // log2 P of query c from its score t: rows without one in `l` have two terms, or no key
                auto far_exponent = [&](float t, float l, int c, float bias, bool* two) -> float {
                    *two = false;
                    if (l != -INFINITY) return t + l;
                    const float2 f = __ldg(prm.far + (item0 + I.w0 + T) * kTile + c);
                    if (f.y == 0.f) return t + f.x;
                    *two = true;
                    const float d = shared_dot(stg, c, wsm + kKVOff + kvb * 2 * kTileBytes, r);
                    return (fmaf(d, sl2, bias) + f.x) + f.y;
                };
                auto gradient_half = [&](auto masked) {
                    constexpr bool kMasked = decltype(masked)::value;
#pragma unroll 1
                    for (int hc = 0; hc < 4; ++hc) {  // 16 queries: one piece of box rows, one region
                        const int c16 = 4 * wg + hc;
                        uint32_t sv[16], pv[16];
                        tmem_ld16(trow + kColS + 16 * c16, sv);
                        tmem_ld16(trow + kColDP + 16 * c16, pv);
                        const BiasRows<kBW, 1> bias(bt + co.at(c16 >> 1) + ((c16 & 1) ? co.half : 0), pitch);
                        unsigned long long t[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) t[e] = pair(bias[2 * e], bias[2 * e + 1]);
                        uint32_t wp[8], wd[8], ws[8];  // ws: what dQ and the table's sums take of wd
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; e += 2) {
                            const float4 L = neg_l[4 * c16 + e / 2], D = neg_d[4 * c16 + e / 2];
#pragma unroll
                            for (int f = 0; f < 2; ++f) {
                                const int i = e + f;
                                float p0, p1, d0, d1;
                                bool two[2] = {true, true};
                                if (kFarTable) {
                                    const int c = 16 * c16 + 2 * i;
                                    unpair(fma_pair(pair(sv[2 * i], sv[2 * i + 1]), sl2_2, t[i]), p0, p1);
                                    p0 = far_exponent(p0, f ? L.z : L.x, c, bias[2 * i], &two[0]);
                                    p1 = far_exponent(p1, f ? L.w : L.y, c + 1, bias[2 * i + 1], &two[1]);
                                } else {
                                    unpair(add_pair(fma_pair(pair(sv[2 * i], sv[2 * i + 1]), sl2_2, t[i]),
                                                    f ? pair(L.z, L.w) : pair(L.x, L.y)), p0, p1);
                                }
                                p0 = ex2_approx(p0);
                                p1 = ex2_approx(p1);
                                unpair(mul_pair(add_pair(pair(pv[2 * i], pv[2 * i + 1]),
                                                         f ? pair(D.z, D.w) : pair(D.x, D.y)), pair(p0, p1)), d0, d1);
                                wp[i] = pack_bf16x2(p0, p1);
                                wd[i] = pack_bf16x2(d0, d1);
                                if (kFarTable) ws[i] = wd[i] & ((two[0] ? 0xFFFFu : 0u) | (two[1] ? 0xFFFF0000u : 0u));
                            }
                        }
                        if (kMasked) {
                            const bool on = (a16 >> c16) & 1u;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                wp[e] = on ? wp[e] : 0u;
                                wd[e] = on ? wd[e] : 0u;
                                if (kFarTable) ws[e] = on ? ws[e] : 0u;
                            }
                        }
                        tmem_st8(trow + kColS + 64 * wg + 8 * hc, wp);
                        tmem_st8(trow + kColDP + 64 * wg + 8 * hc, wd);
#pragma unroll
                        for (int q4 = 0; q4 < 2; ++q4)
                            *reinterpret_cast<uint4*>(dsrow + (((2 * hc + q4) ^ (r & 7)) << 4)) =
                                kFarTable ? make_uint4(ws[4 * q4], ws[4 * q4 + 1], ws[4 * q4 + 2], ws[4 * q4 + 3])
                                          : make_uint4(wd[4 * q4], wd[4 * q4 + 1], wd[4 * q4 + 2], wd[4 * q4 + 3]);
                    }
                };
                if (kFarTable || I.kind) gradient_half(std::true_type{});
                else gradient_half(std::false_type{});
                tmem_wait_st();
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wb.p_ready);
                if (static_cast<int>(ph) == wg) {
                    if (!wwait(&wb.p_ready, ph, 0x7508)) { ok = false; break; }  // every row's dS is written
                    Diag<kBW>::step(g, wbase, sums, I.u, T, quad, lane, side);
                }
                if (!wwait(&wb.mma_done, ph, 0x7509)) { ok = false; break; }
                tc_fence_after();
                {
                    uint32_t v[32], q[16];
                    tmem_ld32(trow + (wg == 0 ? kColDV : kColDK), v);
                    tmem_ld16(trow + kColDQ + 16 * wg, q);
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[e] = add_pair(acc[e], pair(v[2 * e], v[2 * e + 1]));
                    // half of dQ's query row over the step's Q and dO tiles, 16-byte chunks
                    // permuted by the row so that the warp's stores spread over the banks
                    // (the accumulator tile keeps the permutation)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        *reinterpret_cast<uint4*>(stg + r * 128 + (((4 * wg + c) ^ (r & 7)) << 4)) =
                            make_uint4(q[4 * c], q[4 * c + 1], q[4 * c + 2], q[4 * c + 3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wb.dq_ready[ph]);
            }
            if (!ok) break;
            if (kvalid) {
                float x[32];
                const float f = wg == 0 ? 1.f : kScale;
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    unpair(acc[e], x[2 * e], x[2 * e + 1]);
                    x[2 * e] *= f;
                    x[2 * e + 1] *= f;
                }
                uint4* dst = reinterpret_cast<uint4*>((wg == 0 ? prm.dv : prm.dk) + ktok * kRowBytes);
#pragma unroll
                for (int c = 0; c < 4; ++c) dst[c] = pack_chunk(x, c);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8 * kWorkers) tmem_dealloc(bars->tmem_base, 256 * kWorkers);
    if (computes) {
        float* dst = prm.part + (X0 * g.heads + h) * static_cast<long long>(side * side);
        for (int e = tid & 255; e < side * side; e += 256) dst[e] = kFarTable ? dst[e] + sums[e] : sums[e];
    }
}

// post: per (tile, head): dq from the accumulator, eight lanes a row, so that a warp reads
// four whole rows and writes four whole rows at a time (32 x 32 windows of 16 x 128 x 128 x 3 heads: 41 -> 23 us against a row a lane).
__global__ void __launch_bounds__(128) post_kernel(const __grid_constant__ Params p) {
    const Geo& g = p.g;
    const long long T = blockIdx.x / g.heads;
    const int h = static_cast<int>(blockIdx.x - T * g.heads);
    const int lane = threadIdx.x & 31, row0 = threadIdx.x - lane;
    int pi, pj;
    long long tok;
    if (!slot_token(g, T, threadIdx.x, h, &pi, &pj, &tok)) tok = -1;
    const float4* acc =
        reinterpret_cast<const float4*>(p.acc + (static_cast<long long>(h) * g.tiles + T) * kTile * kHeadDim) + row0 * 8;
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __ldcs(acc + 32 * i + lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = 4 * i + (lane >> 3);
        const long long t = __shfl_sync(0xFFFFFFFFu, tok, r);
        if (t >= 0)
            *reinterpret_cast<uint2*>(p.dq + t * kRowBytes + 8 * ((lane ^ r) & 7)) =
                make_uint2(pack_bf16x2(v[i].x * kScale, v[i].y * kScale), pack_bf16x2(v[i].z * kScale, v[i].w * kScale));
    }
}

}  // namespace bwd

// ------------------------------------------------------------------ table gradient
// Sum of the partials of a (head, displacement): eight slices of the streams side by
// side, each in order, then the slices in order.  Without a bucket map the displacement
// is the bucket and the result the gradient itself.
__global__ void __launch_bounds__(256) table_sum_kernel(const float* part, int streams, int heads, int nd, float* disp,
                                                        __nv_bfloat16* dtable) {
    __shared__ float slice[8][32];
    const int lane = threadIdx.x & 31, q = threadIdx.x >> 5;
    const int e = blockIdx.x * 32 + lane, h = blockIdx.y;
    const int per = (streams + 7) / 8, k1 = min(streams, (q + 1) * per);
    float s = 0.f;
    if (e < nd) {
        const float* src = part + static_cast<long long>(h) * nd + e;
        const long long step = static_cast<long long>(heads) * nd;
#pragma unroll 8
        for (int k = q * per; k < k1; ++k) s += __ldg(src + k * step);
    }
    slice[q][lane] = s;
    __syncthreads();
    if (q == 0 && e < nd) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += slice[i][lane];
        if (disp)
            disp[static_cast<long long>(h) * nd + e] = s;
        else
            dtable[static_cast<long long>(h) * nd + e] = __float2bfloat16(s);
    }
}

// Gradient of a bucket: block (bucket, eight heads); threads scan the map and add the
// displacements that are theirs and the bucket's, the block adds the threads in a
// fixed tree.
__global__ void __launch_bounds__(128) table_bucket_kernel(const float* disp, const int* buckets, int heads, int nd,
                                                           int n_buckets, __nv_bfloat16* dtable) {
    __shared__ float part[4][8];
    const int bucket = blockIdx.x, h0 = blockIdx.y * 8, hn = min(8, heads - h0);
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int e = threadIdx.x; e < nd; e += 128) {
        if (__ldg(buckets + e) != bucket) continue;
#pragma unroll
        for (int h = 0; h < 8; ++h)
            if (h < hn) s[h] += disp[static_cast<long long>(h0 + h) * nd + e];
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s[h] += __shfl_xor_sync(0xFFFFFFFFu, s[h], o);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5][h] = s[h];
    }
    __syncthreads();
    if (threadIdx.x < static_cast<unsigned>(hn)) {
        const int h = threadIdx.x;
        dtable[static_cast<long long>(h0 + h) * n_buckets + bucket] =
            __float2bfloat16((part[0][h] + part[1][h]) + (part[2][h] + part[3][h]));
    }
}

cudaError_t launch_table_grad(const float* part, int streams, const Geo& g, const RelbPtrs& p, float* disp,
                              cudaStream_t stream) {
    const int nd = displacements(g.M);
    __nv_bfloat16* dt = static_cast<__nv_bfloat16*>(p.dtable);
    table_sum_kernel<<<dim3((nd + 31) / 32, g.heads), 256, 0, stream>>>(part, streams, g.heads, nd,
                                                                      p.buckets ? disp : nullptr, dt);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.buckets) return e;
    table_bucket_kernel<<<dim3(p.n_buckets, (g.heads + 7) / 8), 128, 0, stream>>>(disp, p.buckets, g.heads, nd,
                                                                               p.n_buckets, dt);
    return cudaGetLastError();
}

}  // namespace relb

// ------------------------------------------------------------------ launches
size_t relbias_bwd_workspace_bytes(const Geo& g) { return relb::bwd::ws_layout(g).total; }

cudaError_t launch_relbias_fwd(const Geo& g, const RelbPtrs& p, const RelbMaps& maps, unsigned int* status,
                               unsigned long long limit_ns, int num_sms, cudaStream_t stream,
                               cudaEvent_t const* events) {
    using namespace relb;
    cudaError_t e = events ? cudaEventRecord(events[0], stream) : cudaSuccess;
    if (e != cudaSuccess) return e;
    if (g.N < kTile) {
        e = launch_small_fwd(g, p, status, limit_ns, num_sms, stream);
    } else {
        static SmemOptIn optin[5];
        using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, fwd::Params);
        static const Kernel kernels[5] = {fwd::fwd_kernel<4>, fwd::fwd_kernel<8>, fwd::fwd_kernel<16>,
                                          fwd::fwd_kernel<32>, fwd::fwd_kernel<64>};
        const int kind = ilog2_exact(g.bw) - 2;
        const Kernel kern = kernels[kind];
        if ((e = optin[kind].ensure(reinterpret_cast<const void*>(kern), kSmemLimit)) != cudaSuccess) return e;
        fwd::Params prm{};
        prm.g = g;
        prm.o = static_cast<uint8_t*>(p.o_out);
        prm.table = static_cast<const __nv_bfloat16*>(p.table);
        prm.buckets = p.buckets;
        prm.n_buckets = p.n_buckets;
        prm.lse = p.lse_out;
        prm.status = status;
        prm.limit_ns = limit_ns;
        prm.pitch = bias_pitch(g.M, g.bw);
        prm.q_tiles = g.M == 64 ? 1 : 2;  // the table of M = 64 takes the second tiles' place
        prm.worker_bytes = (prm.q_tiles + 4) * kTileBytes;
        prm.tab_off = fwd::kWorkers * prm.worker_bytes;
        prm.bar_off = (prm.tab_off + (2 * g.M - 1) * prm.pitch * 4 + 127) / 128 * 128;
        const int smem = prm.bar_off + static_cast<int>(sizeof(fwd::Bars)) + 1024;
        prm.streams = streams_per_head((g.tiles + fwd::kWorkers - 1) / fwd::kWorkers, g.heads, num_sms);
        kern<<<static_cast<unsigned>(prm.streams) * g.heads, fwd::kThreads, smem, stream>>>(maps.q, maps.k, maps.v, prm);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess && events) e = cudaEventRecord(events[1], stream);
    return e;
}

cudaError_t launch_relbias_bwd(const Geo& g, const RelbPtrs& p, const RelbMaps& maps, unsigned int* status,
                               unsigned long long limit_ns, cudaStream_t stream, cudaEvent_t const* events) {
    using namespace relb;
    const bwd::WsLayout L = bwd::ws_layout(g);
    float* part = reinterpret_cast<float*>(p.ws + L.part);
    float* disp = reinterpret_cast<float*>(p.ws + L.disp);
    cudaError_t e = cudaSuccess;
    auto mark = [&](int i) {
        if (events && e == cudaSuccess) e = cudaEventRecord(events[i], stream);
    };
    mark(0);
    if (g.N < kTile) {
        mark(1);
        if (e == cudaSuccess) e = launch_small_bwd(g, p, part, L.streams, status, limit_ns, stream);
        mark(2);
        mark(3);
    } else {
        bwd::Params prm{};
        prm.g = g;
        prm.q = static_cast<const uint8_t*>(p.q);
        prm.k = static_cast<const uint8_t*>(p.k);
        prm.o = static_cast<const uint8_t*>(p.o);
        prm.dout = static_cast<const uint8_t*>(p.dout);
        prm.dq = static_cast<uint8_t*>(p.dq);
        prm.dk = static_cast<uint8_t*>(p.dk);
        prm.dv = static_cast<uint8_t*>(p.dv);
        prm.lse = p.lse;
        prm.table = static_cast<const __nv_bfloat16*>(p.table);
        prm.buckets = p.buckets;
        prm.n_buckets = p.n_buckets;
        prm.acc = reinterpret_cast<float*>(p.ws + L.acc);
        prm.rowv = reinterpret_cast<float*>(p.ws + L.rowv);
        prm.far = reinterpret_cast<float2*>(p.ws + L.far);
        prm.flags = reinterpret_cast<uint32_t*>(p.ws + L.flags);
        prm.part = part;
        prm.status = status;
        prm.limit_ns = limit_ns;
        const int W = bwd::workers(g);
        prm.streams = L.streams / W;
        prm.pitch = bias_pitch(g.M, g.bw);
        const int table = (2 * g.M - 1) * prm.pitch * 4, sums = (displacements(g.M) * 4 + 1023) / 1024 * 1024;
        auto total = [&](int kv) {
            return W * (bwd::sums_off(kv) + sums) + (table + 127) / 128 * 128 + static_cast<int>(sizeof(bwd::Bars)) + 1024;
        };
        prm.kv_stages = total(2) <= kSmemLimit ? 2 : 1;  // the next item's keys and values in flight, where they fit
        prm.acc_off = bwd::sums_off(prm.kv_stages);
        prm.worker_bytes = prm.acc_off + sums;
        prm.tab_off = W * prm.worker_bytes;
        prm.bar_off = (prm.tab_off + table + 127) / 128 * 128;
        const int smem = total(prm.kv_stages);
        const long long ht = static_cast<long long>(g.heads) * g.tiles;
        bwd::prep_kernel<<<static_cast<unsigned>(ht), 128, 0, stream>>>(prm);
        e = cudaGetLastError();
        mark(1);
        if (e == cudaSuccess) {
            static SmemOptIn optin[2][2][5];
            using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, bwd::Params);
            static const Kernel kernels[2][2][5] = {
                // the nulls: boxes of 64 tokens, M = 64 only
                {{bwd::main_kernel<4, 1, false>, bwd::main_kernel<8, 1, false>, bwd::main_kernel<16, 1, false>,
                  bwd::main_kernel<32, 1, false>, bwd::main_kernel<64, 1, false>},
                 {bwd::main_kernel<4, 2, false>, bwd::main_kernel<8, 2, false>, bwd::main_kernel<16, 2, false>,
                  bwd::main_kernel<32, 2, false>, nullptr}},
                {{bwd::main_kernel<4, 1, true>, bwd::main_kernel<8, 1, true>, bwd::main_kernel<16, 1, true>,
                  bwd::main_kernel<32, 1, true>, bwd::main_kernel<64, 1, true>},
                 {bwd::main_kernel<4, 2, true>, bwd::main_kernel<8, 2, true>, bwd::main_kernel<16, 2, true>,
                  bwd::main_kernel<32, 2, true>, nullptr}},
            };
            const int kind = ilog2_exact(g.bw) - 2;
            for (int far = 0; far < 2 && e == cudaSuccess; ++far) {
                const Kernel kern = kernels[far][W - 1][kind];
                e = optin[far][W - 1][kind].ensure(reinterpret_cast<const void*>(kern), kSmemLimit);
                if (e != cudaSuccess) break;
                kern<<<static_cast<unsigned>(prm.streams) * g.heads, 256 * W + 128, smem, stream>>>(maps.q, maps.k, maps.v,
                                                                                             maps.dout, prm);
                e = cudaGetLastError();
            }
        }
        mark(2);
        if (e == cudaSuccess) {
            bwd::post_kernel<<<static_cast<unsigned>(ht), 128, 0, stream>>>(prm);
            e = cudaGetLastError();
        }
        mark(3);
    }
    if (e == cudaSuccess) e = launch_table_grad(part, L.streams, g, p, disp, stream);
    mark(4);
    return e;
}

}  // namespace fswin

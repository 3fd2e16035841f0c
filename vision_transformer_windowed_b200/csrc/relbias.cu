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
#include <cuda.h>
#include <cuda_runtime.h>

#include "dgeo.cuh"
#include "geometry.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "relbias.cuh"
#include "rows.cuh"
#include "schedule.cuh"
#include "tile_io.cuh"

namespace fswin {

namespace relb {

constexpr float kScale = 0.17677669529663688f;  // 1 / sqrt(32)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kSmemLimit = 232448;  // shared memory a CTA can use

// The 16 table words of a 16-slot group: rp[x] points at the word of the group's
// first slot in its x-th box row (one row of 16, two of 8, four of 4).
template <int kBW, int kSign>
struct BiasRows {
    const float* rp[kBW >= 16 ? 1 : 16 / kBW];
    __device__ __forceinline__ BiasRows(const float* p, int pitch) {
#pragma unroll
        for (int x = 0; x < (kBW >= 16 ? 1 : 16 / kBW); ++x) rp[x] = p + kSign * x * pitch;
    }
    __device__ __forceinline__ float operator[](int e) const {
        return kBW >= 16 ? rp[0][kSign * e] : rp[e / kBW][kSign * (e % kBW)];
    }
};

// Table offset of the first slot of 16-slot group c of a window's tile.
__device__ __forceinline__ int group_offset(const Geo& g, long long tile, int c, int pitch) {
    int i, j;
    tile_row_pos(g, tile, 16 * c, &i, &j);
    return i * pitch + j;
}

// ------------------------------------------------------------------ forward
namespace fwd {

// Two workers a CTA, each with 256 TMEM columns: S [0, 128), P (bf16) [128, 192),
// O [192, 224).  Warps 4 w .. 4 w + 3: worker w's softmax, thread = query row;
// warp 8 + w issues its products, warp 10 + w its copies.  The next key tile's S
// starts as soon as the four warps have read the present one into registers.
constexpr int kThreads = 384;
constexpr int kMaxStages = 4;
constexpr uint32_t kColP = 128, kColO = 192;

struct WorkerBars {
    uint64_t q_full[2], q_free[2], kv_full[kMaxStages], kv_free[kMaxStages], s_full, s_free, p_ready, pv_done, done;
};
struct Bars {
    WorkerBars w[2];
    uint32_t tmem_base;
    int abort_flag;
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
    int stages;      // key/value tiles in flight a worker
    int worker_bytes, tab_off, bar_off;
};

template <int kBW>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const __grid_constant__ Params prm) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + prm.bar_off);
    float* tab = reinterpret_cast<float*>(smem + prm.tab_off);
    const Geo& g = prm.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.x % g.heads;
    const int wk = warp < 8 ? warp >> 2 : warp & 1;
    WorkerBars& wb = bars->w[wk];
    const long long stride = 2ll * prm.streams;
    const long long X0 = 2ll * (blockIdx.x / g.heads) + wk;
    const long long item0 = static_cast<long long>(h) * g.tiles;
    const int pitch = prm.pitch, stages = prm.stages;

    if (tid == 0) {
        for (int w = 0; w < 2; ++w) {
            WorkerBars& b = bars->w[w];
            for (int i = 0; i < 2; ++i) {
                mbar_init(&b.q_full[i], 1);
                mbar_init(&b.q_free[i], 1);
            }
            for (int i = 0; i < kMaxStages; ++i) {
                mbar_init(&b.kv_full[i], 1);
                mbar_init(&b.kv_free[i], 1);
            }
            mbar_init(&b.s_full, 1);
            mbar_init(&b.s_free, 4);
            mbar_init(&b.p_ready, 4);
            mbar_init(&b.pv_done, 1);
            mbar_init(&b.done, 1);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
    }
    build_bias(tab, pitch, prm.table + static_cast<long long>(h) * prm.n_buckets, prm.buckets, prm.n_buckets, g.M, tid,
               kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base + 256 * wk;
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    // a worker's buffers: two Q tiles, the O staging tile, the K, V stages
    uint8_t* wsm = smem + wk * prm.worker_bytes;
    uint8_t* ost = wsm + 2 * kTileBytes;
    uint8_t* kvs = wsm + 3 * kTileBytes;

    if (warp >= 10) {
        if (lane == 0) {
            uint32_t qi = 0, st = 0, sph = 0;
            bool ok = true;
            for (long long X = X0; X < g.tiles && ok; X += stride, ++qi) {
                const FwdItem I = d_fwd_item(g, item0 + X);
                const uint32_t b = qi & 1u;
                if (!mbar_wait(&wb.q_free[b], ((qi >> 1) & 1u) ^ 1u, ctl, 0x7601)) break;
                mbar_arrive_expect_tx(&wb.q_full[b], kTileBytes);
                tile_tma(g, &mq, wsm + b * kTileBytes, &wb.q_full[b], X, h, false);
                for (int u = 0; u < I.nkv; ++u) {
                    if (!((I.act >> u) & 1u)) continue;
                    if (!(ok = mbar_wait(&wb.kv_free[st], sph ^ 1u, ctl, 0x7602))) break;
                    mbar_arrive_expect_tx(&wb.kv_full[st], 2 * kTileBytes);
                    uint8_t* d = kvs + st * 2 * kTileBytes;
                    tile_tma(g, &mk, d, &wb.kv_full[st], I.kv0 + u, h, false);
                    tile_tma(g, &mv, d + kTileBytes, &wb.kv_full[st], I.kv0 + u, h, false);
                    if (++st == static_cast<uint32_t>(stages)) {
                        st = 0;
                        sph ^= 1u;
                    }
                }
            }
        }
    } else if (warp >= 8) {
        if (lane == 0) {
            const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
            const uint32_t id_pv = make_idesc_bf16(kTile, kHeadDim, false, true);
            const uint32_t wbase = smem_u32(wsm);
            const uint64_t dK0 = make_sdesc(wbase, 16, 512, kSw64);
            const uint64_t dMN0 = make_sdesc(wbase, 8192, 512, kSw64);
            // the worker's key tiles of all its items in one sequence; S runs one tile
            // ahead of P V, so at most one item ahead: their tile counts alternate
            long long X = X0;                        // item of the next S
            uint32_t qi = 0, left_s = 0, st_s = 0, ph_s = 0, n_s = 0;
            uint32_t vi = 0, left_v = 0, st_v = 0, n_v = 0;
            uint32_t count0 = 0, count1 = 0;         // key tiles of the even and of the odd items
            auto do_s = [&]() -> bool {
                if (left_s == 0) {
                    left_s = __popc(d_fwd_item(g, item0 + X).act);
                    if (qi & 1u) count1 = left_s;
                    else count0 = left_s;
                    if (!mbar_wait(&wb.q_full[qi & 1u], (qi >> 1) & 1u, ctl, 0x7603)) return false;
                }
                if (!mbar_wait(&wb.kv_full[st_s], ph_s, ctl, 0x7604)) return false;
                if (n_s > 0 && !mbar_wait(&wb.s_free, (n_s - 1u) & 1u, ctl, 0x7605)) return false;
                tc_fence_after();
                const uint64_t qo = (qi & 1u) * (kTileBytes >> 4);
                const uint64_t ko = (3 + 2 * st_s) * (kTileBytes >> 4);
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k) umma_ss(tmem, dK0 + qo + 2 * k, dK0 + ko + 2 * k, id_s, k > 0);
                umma_commit(&wb.s_full);
                if (++st_s == static_cast<uint32_t>(stages)) {
                    st_s = 0;
                    ph_s ^= 1u;
                }
                ++n_s;
                if (--left_s == 0) {
                    umma_commit(&wb.q_free[qi & 1u]);
                    ++qi;
                    X += stride;
                }
                return true;
            };
            bool ok = X >= g.tiles || do_s();
            while (ok && n_v < n_s) {
                // the next S, behind the softmax of the present one
                if ((left_s > 0 || X < g.tiles) && !do_s()) break;
                if (!mbar_wait(&wb.p_ready, n_v & 1u, ctl, 0x7606)) break;
                tc_fence_after();
                const bool first = left_v == 0;
                if (first) left_v = vi++ & 1u ? count1 : count0;
                const uint64_t vo = (4 + 2 * st_v) * (kTileBytes >> 4);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_ts(tmem + kColO, tmem + kColP + 8 * k, dMN0 + vo + 64 * k, id_pv, (k > 0 || !first) ? 1u : 0u);
                umma_commit(&wb.kv_free[st_v]);
                umma_commit(&wb.pv_done);
                if (++st_v == static_cast<uint32_t>(stages)) st_v = 0;
                ++n_v;
                --left_v;
            }
            umma_commit(&wb.done);  // every product issued here has completed before the columns are freed
            mbar_wait(&wb.done, 0, ctl, 0x76ff);
        }
    } else {
        const int r = tid & (kTile - 1), quad = warp & 3;
        const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
        const float sl2 = g.scale_log2;
        auto wwait = [&](uint64_t* bar, uint32_t phase, unsigned int where) -> bool {
            return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, ctl, where));
        };
        uint32_t n = 0;  // key tiles seen
        bool ok = true;
        for (long long X = X0; X < g.tiles && ok; X += stride) {
            const FwdItem I = d_fwd_item(g, item0 + X);
            int pi, pj;
            long long tok;
            const bool valid = slot_token(g, X, r, h, &pi, &pj, &tok);
            const float* brow = tab + (pi + g.M - 1) * pitch + pj + g.M - 1;
            const uint32_t myseg = I.masked ? seg_at(d_tile_segs(g, X, I.win), r >> g.lBT) : 0u;
            float m = -INFINITY, l = 0.f;
            bool first = true;
            for (int u = 0; u < I.nkv && ok; ++u) {
                if (!((I.act >> u) & 1u)) continue;
                const long long kt = I.kv0 + u;
                const uint32_t a16 = I.masked ? d_allow16(g, myseg, kt, I.win) : 0xFFu;
                if (!wwait(&wb.s_full, n & 1u, 0x7607)) { ok = false; break; }
                tc_fence_after();
                float l4[4] = {0.f, 0.f, 0.f, 0.f};
                bool waited = n == 0;
                uint32_t v[2][32];
                tmem_ld32(trow, v[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_wait_ld();
                    if (c < 3) {
                        tmem_ld32(trow + 32 * (c + 1), v[(c + 1) & 1]);
                    } else {  // S is in registers: the next one may start
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&wb.s_free);
                    }
                    float t[32];
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const BiasRows<kBW, -1> b(brow - group_offset(g, kt, 2 * c + hh, pitch), pitch);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const int a = 16 * hh + e;
                            ffma2(t[a], t[a + 1], __uint_as_float(v[c & 1][a]), __uint_as_float(v[c & 1][a + 1]), sl2, sl2,
                                  b[e], b[e + 1]);
                        }
                    }
                    if (I.masked) {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh)
                            if (!((a16 >> (2 * c + hh)) & 1u)) {
#pragma unroll
                                for (int e = 0; e < 16; ++e) t[16 * hh + e] = -INFINITY;
                            }
                    }
                    // The running maximum only moves when a chunk exceeds it by more than
                    // 2^64: probabilities up to 2^64 stay far inside bf16's and fp32's range,
                    // and the final division uses the same maximum as the sum.
                    float c4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 32; e += 2) c4[(e >> 1) & 3] = fmax3(c4[(e >> 1) & 3], t[e], t[e + 1]);
                    const float cm = fmaxf(fmaxf(c4[0], c4[1]), fmaxf(c4[2], c4[3]));
                    const bool grow = cm > m + 64.f;
                    if (!waited) {  // P and O: the previous tile's product is done with them
                        if (!wwait(&wb.pv_done, (n - 1u) & 1u, 0x7608)) { ok = false; break; }
                        tc_fence_after();
                        waited = true;
                    }
                    if (__any_sync(0xFFFFFFFFu, grow)) {
                        const float alpha = grow ? ex2_approx(m - cm) : 1.f;
                        if (grow) m = cm;
                        l *= alpha;
#pragma unroll
                        for (int e = 0; e < 4; ++e) l4[e] *= alpha;
                        if (!first) {
#pragma unroll 1
                            for (int k = 0; k < 2; ++k) {
                                uint32_t ov[16];
                                tmem_ld16(trow + kColO + 16 * k, ov);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                                tmem_st16(trow + kColO + 16 * k, ov);
                            }
                        }
                        tmem_wait_st();
#pragma unroll 1
                        for (int k = 0; k < c; ++k) {  // this tile's chunks already written
                            uint32_t pw[16];
                            tmem_ld16(trow + kColP + 16 * k, pw);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                pw[e] = pack_bf16x2(bf16lo_to_f32(pw[e]) * alpha, bf16hi_to_f32(pw[e]) * alpha);
                            tmem_st16(trow + kColP + 16 * k, pw);
                        }
                    }
                    const float mu = m == -INFINITY ? 0.f : m;  // no key so far: P = 0
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float t0, t1;
                        fadd2(t0, t1, t[2 * e], t[2 * e + 1], -mu, -mu);
                        const float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                        const int a = (e & 1) * 2;
                        fadd2(l4[a], l4[a + 1], l4[a], l4[a + 1], p0, p1);
                        w[e] = pack_bf16x2(p0, p1);  // P joins the tensor product in V's type
                    }
                    tmem_st16(trow + kColP + 16 * c, w);
                }
                if (!ok) break;
                l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&wb.p_ready);
                first = false;
                ++n;
            }
            if (!ok || first) break;
            if (!wwait(&wb.pv_done, (n - 1u) & 1u, 0x7609)) break;
            tc_fence_after();
            uint32_t ov[32];
            tmem_ld32(trow + kColO, ov);
            tmem_wait_ld();
            tc_fence_before();  // ordered before the next item's product by its p_ready
            const float inv = 1.f / l;
            float x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = l == 0.f ? 0.f : __uint_as_float(ov[e]) * inv;  // no key: O = 0
            store_row_swz(ost, r, x);
            if (valid && prm.lse != nullptr) prm.lse[tok] = (m + lg2_approx(l)) * kLn2;
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
            __syncwarp();
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(bars->tmem_base, 512);
}

}  // namespace fwd

// ------------------------------------------------------------------ backward
namespace bwd {

struct WsLayout {
    size_t acc, rowv, part, disp, total;
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
        L.rowv = o; o += round256(ht * kTile * 8);             // per slot row: lse log2(e), D
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
    const uint8_t *o, *dout;
    uint8_t *dq, *dk, *dv;
    const float* lse;
    const __nv_bfloat16* table;
    const int* buckets;
    int n_buckets;
    float* acc;
    float2* rowv;
    float* part;
    unsigned int* status;
    unsigned long long limit_ns;
    int streams;  // CTAs of a head
    int pitch, kv_stages;
    int worker_bytes, acc_off, tab_off, bar_off;
};

// prep: per (tile, head), thread = slot row: D = dO . O and the row's log-sum-exp
// in base-2 units, and the zeroed dQ accumulator row.  Memory only.
__global__ void __launch_bounds__(128) prep_kernel(const __grid_constant__ Params p) {
    const Geo& g = p.g;
    const long long T = blockIdx.x / g.heads;
    const int h = static_cast<int>(blockIdx.x - T * g.heads);
    const long long ht = static_cast<long long>(h) * g.tiles + T;
    const int r = threadIdx.x;
    int pi, pj;
    long long tok;
    float D = 0.f, lse2 = INFINITY;  // a row outside the grid: no probability
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
        lse2 = grad_lse2(__ldg(p.lse + tok));
    }
    p.rowv[ht * kTile + r] = make_float2(lse2, D);
}

// Main kernel: a worker is four warps (thread = key row, and query row of dQ)
// with 256 TMEM columns, its own buffers and barriers.  Item = (key tile, head):
// the query tiles of its window in turn.  Per step
//   S^T = K Q^T, dP^T = V dO^T; P^T and dS^T (bf16, the products' operand type) over
//   consumed columns, dS also to shared memory; dV = P^T dO, dK = dS^T Q, dQ = dS K;
// dV and dK add up in registers, dQ is staged over the step's Q and dO tiles and
// added into the fp32 accumulator tile with one bulk reduction.  While those three
// products run, the warps sum dS over equal displacements (add_diagonals).  Two
// workers a CTA fill each other's waits.  TMEM columns:
constexpr uint32_t kColS = 0, kColDP = 128, kColP = 0, kColDS = 128, kColDV = 64, kColDQ = 96, kColDK = 192;
constexpr int kStageBytes = 2 * kTileBytes + 1024;  // Q, dO, and the rows' (lse2, D)

struct WorkerBars {
    uint64_t kv_full[2], st_full[2], s_full, mma_done, grp, done;
};
struct Bars {
    WorkerBars w[2];
    uint32_t tmem_base;
    int abort_flag;
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
// four columns e belong to displacement 4 m + e - kp, or w less once the quads wrap.
template <int kBW>  // 4, 8, 16, 32, 64: the geometry's box width
struct Diag {
    static constexpr int w = kBW < 32 ? kBW : 32;
    static constexpr int quads = w / 4;
    static constexpr int conc = 32 / w;         // blocks a warp walks at once
    static constexpr int nseg = kTile / w;

    // key and query tile of the step, by their window positions of segment 0's row
    static __device__ __forceinline__ void block(const Geo& g, uint32_t ds, float* sums, long long ku, long long qt,
                                                 int a, int b, int kp, int m, int side) {
        float A[4] = {0.f, 0.f, 0.f, 0.f}, B[4] = {0.f, 0.f, 0.f, 0.f};
        const int q0 = b * w;
        const uint32_t qbase = ds + ((q0 >> 6) << 14);
#pragma unroll
        for (int kk = 0; kk < quads; ++kk) {
            const int r = a * w + 4 * kk + kp;
            const int p = kk + m;
            const int col = (q0 & 63) + 4 * (p & (quads - 1));  // first of four query columns inside the 64-column half
            const uint32_t addr = qbase + ((r >> 3) << 10) + ((r & 7) << 7) + ((((col >> 3) ^ (r & 7)) << 4) | ((col & 4) << 1));
            uint32_t x, y;
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x), "=r"(y) : "r"(addr));
            const float v[4] = {bf16lo_to_f32(x), bf16hi_to_f32(x), bf16lo_to_f32(y), bf16hi_to_f32(y)};
            const bool wrap = p >= quads;
            const float fa = wrap ? 0.f : 1.f, fb = wrap ? 1.f : 0.f;
            ffma2(A[0], A[1], v[0], v[1], fa, fa, A[0], A[1]);
            ffma2(A[2], A[3], v[2], v[3], fa, fa, A[2], A[3]);
            ffma2(B[0], B[1], v[0], v[1], fb, fb, B[0], B[1]);
            ffma2(B[2], B[3], v[2], v[3], fb, fb, B[2], B[3]);
        }
        int ia, ja, ib, jb;
        tile_row_pos(g, ku, a * w, &ia, &ja);
        tile_row_pos(g, qt, q0, &ib, &jb);
        float* dst = sums + (ib - ia + g.M - 1) * side + (jb - ja + g.M - 1) + 4 * m - kp;
        // lanes of one block hold distinct displacements for one e, and so do the
        // blocks walked at once; the wrapped ones of a neighbour may coincide, so
        // they follow in a step of their own
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            dst[e] += A[e];
            __syncwarp();
            if (m > 0) dst[e - w] += B[e];
            __syncwarp();
        }
    }

    static __device__ __forceinline__ void step(const Geo& g, uint32_t ds, float* sums, long long ku, long long qt,
                                                int quad, int lane, int side) {
        const int kp = lane & 3, m = (lane >> 2) & (quads - 1), gi = lane / (4 * quads);
        if (kBW == 64) {  // two rows of two 32-column segments
            const int ra0 = static_cast<int>(ku & (g.tpw - 1)) * 2, rb0 = static_cast<int>(qt & (g.tpw - 1)) * 2;
#pragma unroll 1
            for (int ab = 0; ab < 16; ++ab) {
                const int a = ab >> 2, b = ab & 3;
                if (((rb0 + (b >> 1) - ra0 - (a >> 1)) & 3) != quad) continue;
                block(g, ds, sums, ku, qt, a, b, kp, m, side);
            }
            return;
        }
        // Boxes of bh rows (a multiple of 4, at multiples of 4): segment = box * bh + row
        constexpr int bh = kBW == 32 ? 4 : (kBW == 16 ? 8 : kBW);
        constexpr int per = bh / 4;  // matching rows a box
#pragma unroll 1
        for (int a = 0; a < nseg; ++a) {
            const int row = ((a & (bh - 1)) + quad) & 3;
            const int b = (gi / per) * bh + row + 4 * (gi % per);
            block(g, ds, sums, ku, qt, a, b, kp, m, side);
        }
    }
};

template <int kBW, int kWorkers>
__global__ void __launch_bounds__(128 * kWorkers, 1)
    main_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mdo,
                const __grid_constant__ Params prm) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars* bars = reinterpret_cast<Bars*>(smem + prm.bar_off);
    float* tab = reinterpret_cast<float*>(smem + prm.tab_off);
    const Geo& g = prm.g;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int wk = warp >> 2, quad = warp & 3, r = tid & (kTile - 1);
    const int h = blockIdx.x % g.heads;
    WorkerBars& wb = bars->w[wk];
    const int pitch = prm.pitch, side = 2 * g.M - 1, kvs = prm.kv_stages;
    uint8_t* wsm = smem + wk * prm.worker_bytes;
    float* sums = reinterpret_cast<float*>(wsm + prm.acc_off);
    const long long stride = static_cast<long long>(kWorkers) * prm.streams;
    const long long X0 = static_cast<long long>(kWorkers) * (blockIdx.x / g.heads) + wk;
    const long long item0 = static_cast<long long>(h) * g.tiles;

    if (tid == 0) {
        for (int w = 0; w < kWorkers; ++w) {
            WorkerBars& b = bars->w[w];
            for (int i = 0; i < 2; ++i) {
                mbar_init(&b.kv_full[i], 1);
                mbar_init(&b.st_full[i], 1);
            }
            mbar_init(&b.s_full, 1);
            mbar_init(&b.mma_done, 1);
            mbar_init(&b.grp, 4);
            mbar_init(&b.done, 1);
        }
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&bars->tmem_base, 256 * kWorkers);
        tmem_relinquish();
    }
    build_bias(tab, pitch, prm.table + static_cast<long long>(h) * prm.n_buckets, prm.buckets, prm.n_buckets, g.M, tid,
               128 * kWorkers);
    for (int e = r; e < side * side; e += kTile) sums[e] = 0.f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base + 256 * wk;
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
    const uint32_t id_dv = make_idesc_bf16(kTile, kHeadDim, false, true);
    const uint32_t id_dq = make_idesc_bf16(kTile, kHeadDim, true, true);
    const uint32_t wbase = smem_u32(wsm);
    const uint64_t dK0 = make_sdesc(wbase, 16, 512, kSw64);
    const uint64_t dMN0 = make_sdesc(wbase, 8192, 512, kSw64);
    const uint64_t dDS = make_sdesc(wbase, 16384, 1024, kSw128);
    const float sl2 = g.scale_log2;
    const int st0 = stage_off(kvs);
    uint32_t gph = 0;
    auto wwait = [&](uint64_t* bar, uint32_t phase, unsigned int where) -> bool {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, ctl, where));
    };
    auto group_sync = [&](unsigned int where) -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(&wb.grp);
        const bool passed = wwait(&wb.grp, gph, where);
        gph ^= 1u;
        return passed;
    };

    // The copying thread (lane 0 of the worker's second warp) runs one step ahead.
    const bool loader = quad == 1 && lane == 0;
    long long LX = X0;      // item of the next step to load
    long long Lq0 = 0;
    uint32_t Lact = 0, Lst = 0;
    auto load_kv = [&](long long X, int b) {
        uint8_t* d = wsm + kKVOff + b * 2 * kTileBytes;
        mbar_arrive_expect_tx(&wb.kv_full[b], 2 * kTileBytes);
        tile_tma(g, &mk, d, &wb.kv_full[b], X, h, false);
        tile_tma(g, &mv, d + kTileBytes, &wb.kv_full[b], X, h, false);
    };
    auto load_step = [&]() {
        if (Lact == 0) {
            if (LX >= g.tiles) return;
            const BwdItem I = d_bwd_item(g, item0 + LX);
            Lq0 = I.q0;
            Lact = I.act;
            LX += stride;
            if (Lact == 0) return;
        }
        const int n = __ffs(Lact) - 1;
        Lact &= Lact - 1u;
        const long long T = Lq0 + n;
        uint8_t* d = wsm + st0 + Lst * kStageBytes;
        uint64_t* bar = &wb.st_full[Lst];
        mbar_arrive_expect_tx(bar, kStageBytes);
        tile_tma(g, &mq, d, bar, T, h, false);
        tile_tma(g, &mdo, d + kTileBytes, bar, T, h, false);
        bulk_load(d + 2 * kTileBytes, prm.rowv + (item0 + T) * kTile, 1024, bar);
        Lst ^= 1u;
    };
    if (loader && X0 < g.tiles) {
        load_kv(X0, 0);
        load_step();
        load_step();
    }
    __syncwarp();

    uint32_t step = 0, item = 0;
    bool ok = true;
    for (long long X = X0; X < g.tiles && ok; X += stride, ++item) {
        const BwdItem I = d_bwd_item(g, item0 + X);
        const int kvb = kvs == 2 ? static_cast<int>(item & 1u) : 0;
        const uint32_t kvph = kvs == 2 ? (item >> 1) & 1u : item & 1u;
        // the other buffer's item is finished: the next item's keys and values
        if (loader && kvs == 2 && X + stride < g.tiles) load_kv(X + stride, kvb ^ 1);
        int ki, kj;
        long long ktok;
        const bool kvalid = slot_token(g, X, r, h, &ki, &kj, &ktok);
        const float* brow = tab + (g.M - 1 - ki) * pitch + g.M - 1 - kj;
        const uint32_t keyseg = I.masked ? seg_at(d_tile_segs(g, X, I.win), r >> g.lBT) : 0u;
        float dv[32], dk[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) dv[e] = dk[e] = 0.f;
        const uint64_t ko = (kKVOff + kvb * 2 * kTileBytes) >> 4, vo = ko + (kTileBytes >> 4);
        bool first = true;
        for (int n = 0; n < I.nq && ok; ++n) {
            if (!bwd_active(g, I, n)) continue;
            const long long T = I.q0 + n;
            const uint32_t b = step & 1u, ph = step & 1u;
            uint8_t* stg = wsm + st0 + b * kStageBytes;
            const uint64_t qo = static_cast<uint64_t>((st0 + b * kStageBytes) >> 4), dof = qo + (kTileBytes >> 4);
            if (first && !wwait(&wb.kv_full[kvb], kvph, 0x7501)) { ok = false; break; }
            first = false;
            if (!wwait(&wb.st_full[b], (step >> 1) & 1u, 0x7502)) { ok = false; break; }
            if (r == 0) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k) {
                    umma_ss(tmem + kColS, dK0 + ko + 2 * k, dK0 + qo + 2 * k, id_s, k > 0);
                    umma_ss(tmem + kColDP, dK0 + vo + 2 * k, dK0 + dof + 2 * k, id_s, k > 0);
                }
                umma_commit(&wb.s_full);
            }
            if (loader && step > 0) {  // the other stage: its reduction has left it, the next step's rows come in
                bulk_wait_read_all();
                load_step();
            }
            const uint32_t a16 = I.masked ? d_allow16(g, keyseg, T, I.win) : 0xFFu;
            const float4* vec = reinterpret_cast<const float4*>(stg + 2 * kTileBytes);  // (lse2, D) of two queries
            if (!wwait(&wb.s_full, ph, 0x7503)) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint8_t* base = wsm + (c >> 1) * 16384 + (r >> 3) * 1024 + (r & 7) * 128;
                uint32_t sv[32], pv[32];
                tmem_ld32(trow + kColS + 32 * c, sv);
                tmem_ld32(trow + kColDP + 32 * c, pv);
                tmem_wait_ld();
                uint32_t wp[16], wd[16];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const BiasRows<(kBW > 16 ? 16 : kBW), 1> bias(brow + group_offset(g, T, 2 * c + hh, pitch), pitch);
                    const bool on = (a16 >> (2 * c + hh)) & 1u;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        const int a = 16 * hh + e;
                        const float4 LD = vec[16 * c + a / 2];
                        float t0, t1, d0, d1;
                        fadd2(t0, t1, bias[e], bias[e + 1], -LD.x, -LD.z);
                        ffma2(t0, t1, __uint_as_float(sv[a]), __uint_as_float(sv[a + 1]), sl2, sl2, t0, t1);
                        float p0 = ex2_approx(t0), p1 = ex2_approx(t1);
                        fadd2(d0, d1, __uint_as_float(pv[a]), __uint_as_float(pv[a + 1]), -LD.y, -LD.w);
                        fmul2(d0, d1, d0, d1, p0, p1);
                        if (!on) p0 = p1 = d0 = d1 = 0.f;
                        wp[a / 2] = pack_bf16x2(p0, p1);
                        wd[a / 2] = pack_bf16x2(d0, d1);
                    }
                }
                tmem_st16(trow + kColP + 16 * c, wp);
                tmem_st16(trow + kColDS + 16 * c, wd);
#pragma unroll
                for (int q4 = 0; q4 < 4; ++q4) {
                    const int cc = 4 * (c & 1) + q4;
                    *reinterpret_cast<uint4*>(base + ((cc ^ (r & 7)) << 4)) =
                        make_uint4(wd[4 * q4], wd[4 * q4 + 1], wd[4 * q4 + 2], wd[4 * q4 + 3]);
                }
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            if (!group_sync(0x7504)) { ok = false; break; }  // every row's P^T, dS^T and dS written
            if (r == 0) {
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_ts(tmem + kColDV, tmem + kColP + 8 * k, dMN0 + dof + 64 * k, id_dv, k > 0);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_ts(tmem + kColDK, tmem + kColDS + 8 * k, dMN0 + qo + 64 * k, id_dv, k > 0);
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    umma_ss(tmem + kColDQ, dDS + 128 * k, dMN0 + ko + 64 * k, id_dq, k > 0);
                umma_commit(&wb.mma_done);
            }
            Diag<kBW>::step(g, wbase, sums, X, T, quad, lane, side);
            if (!wwait(&wb.mma_done, ph, 0x7505)) { ok = false; break; }
            tc_fence_after();
            {
                uint32_t v[32];
                tmem_ld32(trow + kColDV, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    fadd2(dv[e], dv[e + 1], dv[e], dv[e + 1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                tmem_ld32(trow + kColDK, v);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    fadd2(dk[e], dk[e + 1], dk[e], dk[e + 1], __uint_as_float(v[e]), __uint_as_float(v[e + 1]));
                tmem_ld32(trow + kColDQ, v);
                tmem_wait_ld();
                // dQ of this query row over the step's Q and dO tiles, 16-byte chunks
                // permuted by the row so that the warp's stores spread over the banks
                // (the accumulator tile keeps the permutation)
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    *reinterpret_cast<uint4*>(stg + r * 128 + ((c ^ (r & 7)) << 4)) =
                        make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            if (!group_sync(0x7506)) { ok = false; break; }  // dQ staged; products, sums and K, V rows read
            if (loader) {
                bulk_reduce_add_f32(prm.acc + (item0 + T) * kTile * kHeadDim, stg, 2 * kTileBytes);
                bulk_commit();
            }
            ++step;
        }
        if (!ok) break;
        if (loader && kvs == 1 && X + stride < g.tiles) load_kv(X + stride, 0);
        if (kvalid) {
            uint4* dst = reinterpret_cast<uint4*>(prm.dv + ktok * kRowBytes);
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = pack_chunk(dv, c);
#pragma unroll
            for (int e = 0; e < 32; ++e) dk[e] *= kScale;
            dst = reinterpret_cast<uint4*>(prm.dk + ktok * kRowBytes);
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = pack_chunk(dk, c);
        }
    }
    if (loader) bulk_wait_all();
    if (r == 0) {
        umma_commit(&wb.done);  // every product issued here has completed before the columns are freed
        mbar_wait(&wb.done, 0, ctl, 0x75ff);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(bars->tmem_base, 256 * kWorkers);
    float* dst = prm.part + (X0 * g.heads + h) * static_cast<long long>(side * side);
    for (int e = r; e < side * side; e += kTile) dst[e] = sums[e];
}

// post: per (tile, head), thread = slot row: dq from the accumulator.
__global__ void __launch_bounds__(128) post_kernel(const __grid_constant__ Params p) {
    const Geo& g = p.g;
    const long long T = blockIdx.x / g.heads;
    const int h = static_cast<int>(blockIdx.x - T * g.heads);
    const int r = threadIdx.x;
    int pi, pj;
    long long tok;
    if (!slot_token(g, T, r, h, &pi, &pj, &tok)) return;
    const float4* acc =
        reinterpret_cast<const float4*>(p.acc + (static_cast<long long>(h) * g.tiles + T) * kTile * kHeadDim) + r * 8;
    float x[32];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const float4 v = __ldcs(acc + (c ^ (r & 7)));
        x[4 * c] = v.x * kScale;
        x[4 * c + 1] = v.y * kScale;
        x[4 * c + 2] = v.z * kScale;
        x[4 * c + 3] = v.w * kScale;
    }
    uint4* dst = reinterpret_cast<uint4*>(p.dq + tok * kRowBytes);
#pragma unroll
    for (int c = 0; c < 4; ++c) dst[c] = pack_chunk(x, c);
}

}  // namespace bwd

// ------------------------------------------------------------------ table gradient
// Sum of the partials of a (head, displacement) in stream order; without a bucket
// map the displacement is the bucket and the result the gradient itself.
__global__ void __launch_bounds__(256) table_sum_kernel(const float* part, int streams, int heads, int nd, int n_buckets,
                                                        float* disp, __nv_bfloat16* dtable) {
    const int e = blockIdx.x * 256 + threadIdx.x, h = blockIdx.y;
    if (e >= nd) return;
    const float* src = part + static_cast<long long>(h) * nd + e;
    const long long step = static_cast<long long>(heads) * nd;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    int k = 0;
    for (; k + 4 <= streams; k += 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += __ldg(src + (k + i) * step);
    }
    for (; k < streams; ++k) s[0] += __ldg(src + k * step);
    const float sum = (s[0] + s[1]) + (s[2] + s[3]);
    if (disp)
        disp[static_cast<long long>(h) * nd + e] = sum;
    else  // n_buckets == nd
        dtable[static_cast<long long>(h) * n_buckets + e] = __float2bfloat16(sum);
}

// Warp per bucket: finds the bucket's displacements in order, lanes take heads.
__global__ void __launch_bounds__(256) table_bucket_kernel(const float* disp, const int* buckets, int heads, int nd,
                                                           int n_buckets, __nv_bfloat16* dtable) {
    const int bucket = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (bucket >= n_buckets) return;
    for (int h0 = 0; h0 < heads; h0 += 32) {
        float s = 0.f;
        for (int e0 = 0; e0 < nd; e0 += 32) {
            const int e = e0 + lane;
            uint32_t hit = __ballot_sync(0xFFFFFFFFu, e < nd && __ldg(buckets + e) == bucket);
            while (hit) {
                const int d = e0 + __ffs(hit) - 1;
                hit &= hit - 1u;
                if (h0 + lane < heads) s += disp[static_cast<long long>(h0 + lane) * nd + d];
            }
        }
        if (h0 + lane < heads) dtable[static_cast<long long>(h0 + lane) * n_buckets + bucket] = __float2bfloat16(s);
    }
}

cudaError_t launch_table_grad(const float* part, int streams, const Geo& g, const RelbPtrs& p, float* disp,
                              cudaStream_t stream) {
    const int nd = displacements(g.M);
    __nv_bfloat16* dt = static_cast<__nv_bfloat16*>(p.dtable);
    table_sum_kernel<<<dim3((nd + 255) / 256, g.heads), 256, 0, stream>>>(part, streams, g.heads, nd, p.n_buckets,
                                                                        p.buckets ? disp : nullptr, dt);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (p.buckets)
        table_bucket_kernel<<<(p.n_buckets + 7) / 8, 256, 0, stream>>>(disp, p.buckets, g.heads, nd, p.n_buckets, dt);
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
        static SmemOptIn optin[3];
        const int kind = g.bw >= 16 ? 2 : (g.bw == 8 ? 1 : 0);
        auto* kern = kind == 2 ? fwd::fwd_kernel<16> : (kind == 1 ? fwd::fwd_kernel<8> : fwd::fwd_kernel<4>);
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
        prm.stages = g.M == 64 ? 3 : fwd::kMaxStages;  // the table of M = 64 takes the fourth stage's place
        prm.worker_bytes = (3 + 2 * prm.stages) * kTileBytes;
        prm.tab_off = 2 * prm.worker_bytes;
        prm.bar_off = (prm.tab_off + (2 * g.M - 1) * prm.pitch * 4 + 127) / 128 * 128;
        const int smem = prm.bar_off + static_cast<int>(sizeof(fwd::Bars)) + 1024;
        prm.streams = streams_per_head((g.tiles + 1) / 2, g.heads, num_sms);
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
        prm.rowv = reinterpret_cast<float2*>(p.ws + L.rowv);
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
            static SmemOptIn optin[2][5];
            using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, bwd::Params);
            static const Kernel kernels[2][5] = {
                {bwd::main_kernel<4, 1>, bwd::main_kernel<8, 1>, bwd::main_kernel<16, 1>, bwd::main_kernel<32, 1>,
                 bwd::main_kernel<64, 1>},
                {bwd::main_kernel<4, 2>, bwd::main_kernel<8, 2>, bwd::main_kernel<16, 2>, bwd::main_kernel<32, 2>,
                 nullptr},  // boxes of 64 tokens: M = 64 only
            };
            const int kind = ilog2_exact(g.bw) - 2;
            const Kernel kern = kernels[W - 1][kind];
            e = optin[W - 1][kind].ensure(reinterpret_cast<const void*>(kern), kSmemLimit);
            if (e == cudaSuccess) {
                kern<<<static_cast<unsigned>(prm.streams) * g.heads, 128 * W, smem, stream>>>(maps.q, maps.k, maps.v,
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

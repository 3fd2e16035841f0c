// Attention with a learned relative position bias, windows of fewer than 128
// tokens: M = 8 on the tensor cores (two windows to a 128-slot tile), M = 4 on
// the CUDA cores (a half warp is a window).  A work item is one (tile, head); all
// of its attention, and every gradient of its tokens, stays inside it.
//
// Windows that share a tile must not reach each other, not even through a
// product 0 x inf.  At M = 8 a row therefore keeps only the 64 columns of its own
// window: the probabilities are a compact [128 rows x 64] operand, multiplied once
// with each window's 64 value rows into an accumulator of its own, and a row reads
// its own window's.  That is the same tensor work as one 128-column product, half
// the TMEM traffic, and nothing has to be filled with zeros.
#include <cuda.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "dgeo.cuh"
#include "geometry.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "relbias.cuh"
#include "rows.cuh"

namespace fswin {

namespace relb {

constexpr float kScale = 0.17677669529663688f;  // 1 / sqrt(32)
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int kM8 = 8, kP8 = bias_pitch(8, 8);  // window side, table pitch (the same for boxes of 8 and of 4)
static_assert(bias_pitch(8, 4) == kP8, "one pitch for both shifts");

// Window position of local slot e of an 8 x 8 window stored in boxes of kBW x kBW.
template <int kBW>
__host__ __device__ constexpr int slot_i(int e) {
    return kBW == 8 ? e >> 3 : ((e >> 5) << 2) + ((e >> 2) & 3);
}
template <int kBW>
__host__ __device__ constexpr int slot_j(int e) {
    return kBW == 8 ? e & 7 : (((e >> 4) & 1) << 2) + (e & 3);
}
// Table offset of local slot e relative to window position (0, 0).
template <int kBW>
__host__ __device__ constexpr int slot_off(int e) {
    return slot_i<kBW>(e) * kP8 + slot_j<kBW>(e);
}

// cp.async copies of a warp's 32 rows: lane l moves 16-byte chunk l % 4 of rows
// l / 4 + 8 i, eight whole 64-byte rows an instruction.
__device__ __forceinline__ void load_rows(uint8_t* tile, const uint8_t* src, long long tok, bool valid, int warp,
                                          int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rl = (lane >> 2) + 8 * i, c = lane & 3;
        const long long tk = __shfl_sync(0xFFFFFFFFu, tok, rl);
        const bool vd = __shfl_sync(0xFFFFFFFFu, valid ? 1 : 0, rl) != 0;
        const int row = warp * 32 + rl;
        cp_async16(smem_u32(tile + row * kRowBytes + ((c ^ ((row >> 1) & 3)) << 4)),
                   vd ? src + tk * kRowBytes + 16 * c : src, vd ? 16u : 0u);
    }
}

__device__ __forceinline__ void save_rows(uint8_t* dst, const uint8_t* tile, long long tok, bool valid, int warp,
                                          int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int rl = (lane >> 2) + 8 * i, c = lane & 3;
        const long long tk = __shfl_sync(0xFFFFFFFFu, tok, rl);
        const bool vd = __shfl_sync(0xFFFFFFFFu, valid ? 1 : 0, rl) != 0;
        const int row = warp * 32 + rl;
        if (vd)
            *reinterpret_cast<uint4*>(dst + tk * kRowBytes + 16 * c) =
                *reinterpret_cast<const uint4*>(tile + row * kRowBytes + ((c ^ ((row >> 1) & 3)) << 4));
    }
}

// Row r of tile X of 8 x 8 windows: its token of head h (in `tok`; false outside the
// grid) and the 16-slot groups of its window that it attends (bit b: local slots
// [16 b, 16 b + 16)).  A shift makes regions only in the last row and column of
// windows, cut at 4, and its 4 x 4 boxes are the groups: box b lies in row b >> 1 and
// column b & 1 of the window's boxes.
template <int kBW>
__device__ __forceinline__ bool row_of(const Geo& g, long long X, int r, int h, long long* tok, uint32_t* groups) {
    const uint32_t gw = static_cast<uint32_t>(2 * X) + (r >> 6);
    const int e = r & 63;
    const int b = static_cast<int>(fdiv(g.fd_nW, gw));
    const uint32_t rem = gw - static_cast<uint32_t>(b) * g.nW;
    const int wr = static_cast<int>(fdiv(g.fd_nWw, rem)), wc = static_cast<int>(rem) - wr * g.nWw;
    int row = wr * 8 + slot_i<kBW>(e) + g.s, col = wc * 8 + slot_j<kBW>(e) + g.s;
    if (row >= g.Hp) row -= g.Hp;
    if (col >= g.Wp) col -= g.Wp;
    *tok = ((static_cast<long long>(b) * g.H + row) * g.W + col) * g.heads + h;
    uint32_t m = 0xFu;
    if (kBW == 4) {
        if ((wr + 1) * 8 == g.Hp) m &= (e >> 5) & 1 ? 0xCu : 0x3u;
        if (wc + 1 == g.nWw) m &= (e >> 4) & 1 ? 0xAu : 0x5u;
    }
    *groups = m;
    return gw < g.wins && row < g.H && col < g.W;
}

// The four rows whose 16-byte chunk lane % 4 this lane moves for its warp (rows lane / 4
// + 8 i of the warp's 32): their byte offsets in a token tensor, negative for rows
// outside the grid.
__device__ __forceinline__ void chunk_offsets(long long (&off)[4], long long tok, bool valid, int lane) {
    const long long mine = valid ? tok * kRowBytes : -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long long o = __shfl_sync(0xFFFFFFFFu, mine, (lane >> 2) + 8 * i);
        off[i] = o < 0 ? -1 : o + 16 * (lane & 3);
    }
}
__device__ __forceinline__ uint32_t chunk_place(int warp, int lane, int i) {
    const int row = warp * 32 + (lane >> 2) + 8 * i;
    return row * kRowBytes + (((lane & 3) ^ ((row >> 1) & 3)) << 4);
}
__device__ __forceinline__ void load_chunks(uint32_t tile, const uint8_t* src, const long long (&off)[4], int warp, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        cp_async16(tile + chunk_place(warp, lane, i), off[i] < 0 ? src : src + off[i], off[i] < 0 ? 0u : 16u);
}
__device__ __forceinline__ void save_chunks(uint8_t* dst, const uint8_t* tile, const long long (&off)[4], int warp, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (off[i] >= 0)
            *reinterpret_cast<uint4*>(dst + off[i]) = *reinterpret_cast<const uint4*>(tile + chunk_place(warp, lane, i));
}

// ------------------------------------------------------------------ M = 8 forward
namespace fwd8 {

constexpr int kThreads = 128;
constexpr int kSlotBytes = 3 * kTileBytes;  // q, k, v tiles of one item
constexpr int kTabOff = 2 * kSlotBytes;     // two slots
constexpr int kTabBytes = 15 * kP8 * 4;
constexpr int kBarOff = (kTabOff + kTabBytes + 15) / 16 * 16;
constexpr int kSmemBytes = kBarOff + 64 + 1024;  // + alignment of the base
constexpr uint32_t kTmemCols = 128;
// S [0, 128); compact P (bf16) [0, 32); the two windows' O [64, 96), [96, 128).
// P and O only take columns whose scores have been read.
constexpr uint32_t kColP = 0, kColO = 64;

struct Bars {
    uint64_t s_full, p_ready, o_full, grp, done;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 64, "barrier block overflows its slot");

struct Params {
    Geo g;
    const uint8_t *q, *k, *v;
    uint8_t* o;
    const __nv_bfloat16* table;
    const int* buckets;
    int n_buckets;
    float* lse;
    unsigned int* status;
    unsigned long long limit_ns;
    int streams;
};

// Four CTAs an SM, each one row a thread: the chain copy -> S -> softmax -> O of
// an item is latency-bound, so other CTAs' items fill the gaps (64 x 64 x 64 tokens, 3
// heads, shifted: 41 us, 4.9 TB/s).
template <int kBW>
__global__ void __launch_bounds__(kThreads, 4) fwd_kernel(const __grid_constant__ Params prm) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    Bars* bars = reinterpret_cast<Bars*>(smem + kBarOff);
    float* tab = reinterpret_cast<float*>(smem + kTabOff);
    const Geo& g = prm.g;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31, r = tid, wi = warp >> 1;
    const int h = blockIdx.x % g.heads, stream = blockIdx.x / g.heads;

    if (tid == 0) {
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->p_ready, 4);
        mbar_init(&bars->o_full, 1);
        mbar_init(&bars->grp, 4);
        mbar_init(&bars->done, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    const uint32_t sbase = smem_u32(smem);
    // an item's rows: this row's token and groups, and the warp's copies
    auto copy_item = [&](int slot, const long long (&off)[4]) {
        const uint32_t sl = sbase + slot * kSlotBytes;
        load_chunks(sl, prm.q, off, warp, lane);
        load_chunks(sl + kTileBytes, prm.k, off, warp, lane);
        load_chunks(sl + 2 * kTileBytes, prm.v, off, warp, lane);
    };
    long long X = stream, Xn = X + prm.streams, tok = 0, tok_n = 0, off[4], off_n[4];
    uint32_t grp4 = 0, grp4_n = 0;
    bool valid = false, valid_n = false;
    if (X < g.tiles) {
        valid = row_of<kBW>(g, X, r, h, &tok, &grp4);
        chunk_offsets(off, tok, valid, lane);
        copy_item(0, off);
    }
    cp_async_commit();
    if (Xn < g.tiles) {
        valid_n = row_of<kBW>(g, Xn, r, h, &tok_n, &grp4_n);
        chunk_offsets(off_n, tok_n, valid_n, lane);
        copy_item(1, off_n);
    }
    cp_async_commit();
    build_bias(tab, kP8, prm.table + static_cast<long long>(h) * prm.n_buckets, prm.buckets, prm.n_buckets, kM8, tid,
               kThreads);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
    const uint32_t id_pv = make_idesc_bf16(kTile, kHeadDim, false, true);  // P (TMEM) x V
    const uint64_t dK0 = make_sdesc(sbase, 16, 512, kSw64);     // K-major, 64-byte rows
    const uint64_t dMN0 = make_sdesc(sbase, 8192, 512, kSw64);  // MN-major, 64-byte rows
    const unsigned long long sl2_2 = pair(g.scale_log2, g.scale_log2);
    const int e_r = r & 63;  // local slot: its window position does not depend on the item
    const float* brow = tab + (slot_i<kBW>(e_r) + kM8 - 1) * kP8 + slot_j<kBW>(e_r) + kM8 - 1;
    uint32_t gph = 0, ph = 0;
    auto wwait = [&](uint64_t* bar, uint32_t phase, unsigned int where) -> bool {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, ctl, where));
    };
    for (int j = 0; X < g.tiles; ++j) {
        uint8_t* sl = smem + (j & 1) * kSlotBytes;
        cp_async_wait<1>();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->grp);
        if (!wwait(&bars->grp, gph, 0x7301)) break;  // every row's copies landed; the previous item's O was read
        gph ^= 1;
        const uint64_t qo = static_cast<uint64_t>(((j & 1) * kSlotBytes) >> 4);
        if (warp == 0) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kHeadDim / 16; ++k)
                    umma_ss(tmem, dK0 + qo + 2 * k, dK0 + qo + (kTileBytes >> 4) + 2 * k, id_s, k > 0);
                umma_commit(&bars->s_full);
            }
            __syncwarp();
        }
        if (!wwait(&bars->s_full, ph, 0x7302)) break;
        tc_fence_after();
        unsigned long long t[32];
        {
            uint32_t v[32];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                tmem_ld32(trow + 64 * wi + 32 * c, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int a = 32 * c + 2 * e;
                    t[16 * c + e] = pair(brow[-slot_off<kBW>(a)], brow[-slot_off<kBW>(a + 1)]);
                }
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    t[16 * c + e] = fma_pair(pair(v[2 * e], v[2 * e + 1]), sl2_2, t[16 * c + e]);
            }
        }
        if (kBW == 4 && grp4 != 0xFu) {
            const unsigned long long none = pair(-INFINITY, -INFINITY);
#pragma unroll
            for (int e = 0; e < 32; ++e) t[e] = (grp4 >> (e >> 3)) & 1u ? t[e] : none;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            float x, y;
            unpair(t[e], x, y);
            mx[e & 3] = fmax3(mx[e & 3], x, y);
        }
        const float m = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
        const float mu = m == -INFINITY ? 0.f : -m;  // a row whose every key is masked: P = 0
        const unsigned long long mu2 = pair(mu, mu);
        unsigned long long l2[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float p0, p1;
                unpair(add_pair(t[16 * c + e], mu2), p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                l2[e & 1] = add_pair(l2[e & 1], pair(p0, p1));
                w[e] = pack_bf16x2(p0, p1);  // P joins the tensor product in V's type
            }
            tmem_st16(trow + kColP + 16 * c, w);
        }
        float la, lb;
        unpair(add_pair(l2[0], l2[1]), la, lb);
        const float l = la + lb;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_ready);
        if (warp == 0 && mbar_wait_warp(&bars->p_ready, ph, ctl, 0x7203)) {
            tc_fence_after();
            const uint64_t vo = qo + (2 * kTileBytes >> 4);
            if (elect_one()) {
#pragma unroll
                for (int w = 0; w < 2; ++w)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        umma_ts(tmem + kColO + 32 * w, tmem + kColP + 8 * k, dMN0 + vo + 256 * w + 64 * k, id_pv, k > 0);
                umma_commit(&bars->o_full);
            }
            __syncwarp();
        }
        if (!wwait(&bars->o_full, ph, 0x7304)) break;
        tc_fence_after();
        {
            uint32_t v[32];
            tmem_ld32(trow + kColO + 32 * wi, v);
            tmem_wait_ld();
            tc_fence_before();  // ordered before the next item's products by its group barrier
            const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // no key: O = 0; a NaN stays one
            float x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = l == 0.f ? 0.f : __uint_as_float(v[e]) * inv;
            store_row_swz(sl, r, x);  // over q
        }
        if (valid && prm.lse != nullptr) prm.lse[tok] = (m + lg2_approx(l)) * kLn2;
        __syncwarp();
        save_chunks(prm.o, sl, off, warp, lane);
        __syncwarp();  // the staged rows are read: the slot takes the rows of the item after the next
        X = Xn;
        tok = tok_n;
        valid = valid_n;
        grp4 = grp4_n;
#pragma unroll
        for (int i = 0; i < 4; ++i) off[i] = off_n[i];
        Xn += prm.streams;
        if (Xn < g.tiles) {
            valid_n = row_of<kBW>(g, Xn, r, h, &tok_n, &grp4_n);
            chunk_offsets(off_n, tok_n, valid_n, lane);
            copy_item(j & 1, off_n);
        }
        cp_async_commit();
        ph ^= 1;
    }
    cp_async_wait<0>();
    if (warp == 0) {  // every product issued here has completed before the columns are freed
        if (elect_one()) umma_commit(&bars->done);
        mbar_wait_warp(&bars->done, 0, ctl, 0x72ff);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace fwd8

// ------------------------------------------------------------------ M = 8 backward
namespace bwd8 {

constexpr int kThreads = 160;  // four row warps, one mover warp
constexpr int kWarpMover = 4;
constexpr int kSlotBytes = 4 * kTileBytes;          // q, k, v, dO tiles of one item
constexpr int kOOff = 2 * kSlotBytes;               // o tile
constexpr int kDSOff = kOOff + kTileBytes;          // dS: per window 64 keys x 64 queries, 128-byte swizzle
constexpr int kVecOff = kDSOff + 2 * kTileBytes;    // -lse2[128], -D[128], far_row's second term[128]
constexpr int kTabOff = kVecOff + 3 * kTile * 4;
constexpr int kBarOff = (kTabOff + 15 * kP8 * 4 + 15) / 16 * 16;
constexpr int kSmemBytes = kBarOff + 128 + 1024;
static_assert(kDSOff % 1024 == 0, "128-byte swizzled operand must be 1024-byte aligned");
static_assert(64 * kTile * 4 <= 2 * kSlotBytes, "the table gradient's staging takes the slots");
constexpr uint32_t kTmemCols = 256;
// S^T [0,128), dP^T [128,256); compact P^T and dS^T (bf16, the 64 queries of the
// key's window) over columns already read, and per window dV, dK, dQ over the rest
constexpr uint32_t kColS = 0, kColDP = 128, kColP = 0, kColDS = 128;
constexpr uint32_t kColDV = 64, kColDK = 192;
__host__ __device__ constexpr uint32_t col_dq(int w) { return w ? 160u : 32u; }

struct Bars {
    uint64_t s_full, p_ready, mma2_done, grp, done;
    uint64_t slot_full[2], o_full, o_free, staged;
    uint32_t tmem_base;
    int abort_flag;
};
static_assert(sizeof(Bars) <= 128, "barrier block overflows its slot");

struct Params {
    Geo g;
    const uint8_t *q, *k, *v, *o, *dout;
    uint8_t *dq, *dk, *dv;
    const __nv_bfloat16* table;
    const int* buckets;
    int n_buckets;
    const float* lse;
    float* part;  // [streams][heads][225]
    unsigned int* status;
    unsigned long long limit_ns;
    int streams;
};

// Thread = key row: its 64 scores and dP against the queries of its window, P^T
// and dS^T back to TMEM, dS to shared memory for dQ = dS K.  dS also adds up in 64
// fp32 registers a thread over all the items of the CTA (one head): the table
// gradient costs one addition a pair, and its sum over equal displacements is
// taken once, at the end.  Two CTAs an SM (64 registers of sums a thread): 64 x 64 x 64
// tokens, 3 heads, shifted: 103 us, 3.9 TB/s, bound by the chain of an item's products.
template <int kBW>
__global__ void __launch_bounds__(kThreads, 2) bwd_kernel(const __grid_constant__ Params prm) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_smem(smem_raw);
    Bars* bars = reinterpret_cast<Bars*>(smem + kBarOff);
    float* tab = reinterpret_cast<float*>(smem + kTabOff);
    const Geo& g = prm.g;
    const int tid = threadIdx.x, warp = uniform_warp(), lane = tid & 31;
    const int h = blockIdx.x % g.heads, stream = blockIdx.x / g.heads;
    const long long n = g.tiles > stream ? (g.tiles - stream + prm.streams - 1) / prm.streams : 0;
    auto tile_at = [&](long long j) { return stream + j * prm.streams; };

    if (tid == 0) {
        mbar_init(&bars->s_full, 1);
        mbar_init(&bars->p_ready, 4);
        mbar_init(&bars->mma2_done, 1);
        mbar_init(&bars->grp, 4);
        mbar_init(&bars->done, 1);
        mbar_init(&bars->slot_full[0], 32);  // one cp.async arrival per mover lane
        mbar_init(&bars->slot_full[1], 32);
        mbar_init(&bars->o_full, 32);
        mbar_init(&bars->o_free, 4);
        mbar_init(&bars->staged, 4);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    const __nv_bfloat16* table_h = prm.table + static_cast<long long>(h) * prm.n_buckets;
    const bool met_far = build_bias(tab, kP8, table_h, prm.buckets, prm.n_buckets, kM8, tid, kThreads);
    tc_fence_before();
    const bool far_table = __syncthreads_or(met_far) != 0;
    tc_fence_after();
    const uint32_t tmem = bars->tmem_base;
    const Ctl ctl{prm.status, &bars->abort_flag, prm.limit_ns};
    auto wwait = [&](uint64_t* bar, uint32_t phase, unsigned int where) -> bool {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, phase, ctl, where));
    };
    // row warps: sum over the items of dS of (this key slot, query slots 2 e, 2 e + 1)
    unsigned long long dacc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) dacc[e] = 0;

    if (warp == kWarpMover) {
        // rows of each item one item ahead, and the stores of the staged gradients
        long long off[2][4][4];  // per slot and warp of rows: this lane's four chunks
        const uint32_t sbase = smem_u32(smem);
        auto geo = [&](long long j, int b) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                long long tok;
                uint32_t groups;
                const bool valid = row_of<kBW>(g, tile_at(j), lane + 32 * q, h, &tok, &groups);
                chunk_offsets(off[b][q], tok, valid, lane);
            }
        };
        auto load = [&](uint32_t tile, const uint8_t* src, int b) {
#pragma unroll
            for (int q = 0; q < 4; ++q) load_chunks(tile, src, off[b][q], q, lane);
        };
        auto load_slot = [&](int b) {
            const uint32_t sl = sbase + b * kSlotBytes;
            load(sl, prm.q, b);
            load(sl + kTileBytes, prm.k, b);
            load(sl + 2 * kTileBytes, prm.v, b);
            load(sl + 3 * kTileBytes, prm.dout, b);
            cp_async_mbar_arrive(&bars->slot_full[b]);
        };
        auto load_o = [&](int b) {
            load(sbase + kOOff, prm.o, b);
            cp_async_mbar_arrive(&bars->o_full);
        };
        if (n > 0) {
            geo(0, 0);
            load_slot(0);
            load_o(0);
        }
        if (n > 1) {
            geo(1, 1);
            load_slot(1);
        }
        for (long long j = 0; j < n; j += 2) {
            bool stop = false;
#pragma unroll
            for (int b = 0; b < 2; ++b) {  // item j + b lives in slot b: constant indices, registers
                const long long jj = j + b;
                if (stop || jj >= n) break;
                const uint32_t ph = static_cast<uint32_t>(b);
                if (jj + 1 < n) {
                    if (!wwait(&bars->o_free, ph, 0x7401)) { stop = true; break; }
                    load_o(b ^ 1);
                }
                if (!wwait(&bars->staged, ph, 0x7402)) { stop = true; break; }
                uint8_t* sl = smem + b * kSlotBytes;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    save_chunks(prm.dq, sl, off[b][q], q, lane);
                    save_chunks(prm.dk, sl + kTileBytes, off[b][q], q, lane);
                    save_chunks(prm.dv, sl + 2 * kTileBytes, off[b][q], q, lane);
                }
                __syncwarp();  // the staged rows are read: the slot takes item jj + 2's rows
                if (jj + 2 < n) {
                    geo(jj + 2, b);
                    load_slot(b);
                }
            }
            if (stop) break;
        }
        cp_async_wait<0>();
    } else {
        const uint32_t id_s = make_idesc_bf16(kTile, kTile, false, false);
        const uint32_t id_dv = make_idesc_bf16(kTile, kHeadDim, false, true);  // P^T or dS^T (TMEM) x dO or Q
        const uint32_t id_dq = make_idesc_bf16(kTile, kHeadDim, true, true);   // dS (smem) x K
        const uint32_t sbase = smem_u32(smem);
        const uint64_t dK0 = make_sdesc(sbase, 16, 512, kSw64);
        const uint64_t dMN0 = make_sdesc(sbase, 8192, 512, kSw64);
        const uint64_t dDS = make_sdesc(sbase + kDSOff, 8192, 1024, kSw128);  // the windows' blocks are the two halves of M
        const int r = tid, wi = warp >> 1;
        const uint32_t trow = tmem + (static_cast<uint32_t>(warp * 32) << 16);
        const unsigned long long sl2_2 = pair(g.scale_log2, g.scale_log2);
        float* neg_l = reinterpret_cast<float*>(smem + kVecOff);  // -lse2 and -D of the tile's queries
        float* neg_d = neg_l + kTile;
        float* far_y = neg_d + kTile;
        const int e_r = r & 63;
        const float* brow = tab + (kM8 - 1 - slot_i<kBW>(e_r)) * kP8 + kM8 - 1 - slot_j<kBW>(e_r);
        uint8_t* dsrow = smem + kDSOff + wi * 8192 + (e_r >> 3) * 1024 + (r & 7) * 128;
        uint32_t gph = 0;
        uint32_t groups = 0;
        auto lse_of = [&](long long j) {
            long long tok;
            const bool valid = row_of<kBW>(g, tile_at(j), r, h, &tok, &groups);
            return valid ? __ldg(prm.lse + tok) : -INFINITY;  // outside the grid: no probability
        };
        float lse = n > 0 ? lse_of(0) : 0.f;
        for (long long j = 0; j < n; ++j) {
            const uint32_t ph = static_cast<uint32_t>(j & 1);
            uint8_t* sl = smem + (j & 1) * kSlotBytes;
            if (!wwait(&bars->slot_full[j & 1], static_cast<uint32_t>((j >> 1) & 1), 0x7304) ||
                !wwait(&bars->o_full, ph, 0x7305))
                break;
            {
                float a[32], b[32];
                load_row_swz(smem + kOOff, r, a, false);
                load_row_swz(sl + 3 * kTileBytes, r, b, false);
                float d4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    ffma2(d4[0], d4[1], a[e], a[e + 1], b[e], b[e + 1], d4[0], d4[1]);
                    ffma2(d4[2], d4[3], a[e + 2], a[e + 3], b[e + 2], b[e + 3], d4[2], d4[3]);
                }
                neg_d[r] = -((d4[0] + d4[1]) + (d4[2] + d4[3]));
            }
            neg_l[r] = -grad_lse2(lse);
            if (far_table) {
                float2 f = make_float2(-grad_lse2(lse), 0.f);
                if (finite_beyond(lse * 1.4426950408889634f, kFar))
                    f = far_row(g, prm.q, prm.k, table_h, prm.buckets, prm.n_buckets, tile_at(j), r, h,
                                lse * 1.4426950408889634f);
                neg_l[r] = f.x;
                far_y[r] = f.y;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->o_free);
            fence_proxy_async_smem();
            if (lane == 0) mbar_arrive(&bars->grp);
            if (!wwait(&bars->grp, gph, 0x7306)) break;  // rows landed, D and lse2 in place, the last item's products read
            gph ^= 1;
            const uint64_t qo = static_cast<uint64_t>(((j & 1) * kSlotBytes) >> 4);
            const uint64_t ko = qo + (kTileBytes >> 4), vo = qo + (2 * kTileBytes >> 4), dof = qo + (3 * kTileBytes >> 4);
            if (warp == 0) {
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kHeadDim / 16; ++k) {
                        umma_ss(tmem + kColS, dK0 + ko + 2 * k, dK0 + qo + 2 * k, id_s, k > 0);
                        umma_ss(tmem + kColDP, dK0 + vo + 2 * k, dK0 + dof + 2 * k, id_s, k > 0);
                    }
                    umma_commit(&bars->s_full);
                }
                __syncwarp();
            }
            const uint32_t grp4 = groups;
            if (j + 1 < n) lse = lse_of(j + 1);
            if (!wwait(&bars->s_full, ph, 0x7307)) break;
            tc_fence_after();
            // log2 P of query q from its score t: rows with two terms have scores of their own
            auto far_exponent = [&](float t, float l, int q, float bias) -> float {
                if (far_y[q] == 0.f) return t + l;
                return (fmaf(shared_dot(sl, q, sl + kTileBytes, r), g.scale_log2, bias) + l) + far_y[q];
            };
            auto gradient = [&](auto far) {
                constexpr bool kFarTable = decltype(far)::value;  // rows may have a second term
#pragma unroll
                for (int c = 0; c < 4; ++c) {  // 16 queries: one region
                    uint32_t sv[16], pv[16];
                    tmem_ld16(trow + kColS + 64 * wi + 16 * c, sv);
                    tmem_ld16(trow + kColDP + 64 * wi + 16 * c, pv);
                    unsigned long long t[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        t[e] = pair(brow[slot_off<kBW>(16 * c + 2 * e)], brow[slot_off<kBW>(16 * c + 2 * e + 1)]);
                    tmem_wait_ld();
                    const bool on = kBW == 8 || ((grp4 >> c) & 1u);
                    uint32_t wp[8], wd[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float4 L = *reinterpret_cast<const float4*>(neg_l + 64 * wi + 16 * c + 2 * e);
                        const float4 D = *reinterpret_cast<const float4*>(neg_d + 64 * wi + 16 * c + 2 * e);
#pragma unroll
                        for (int f = 0; f < 2; ++f) {
                            const int i = e + f;
                            float p0, p1;
                            if (kFarTable) {
                                const int q = 64 * wi + 16 * c + 2 * i;
                                unpair(fma_pair(pair(sv[2 * i], sv[2 * i + 1]), sl2_2, t[i]), p0, p1);
                                p0 = far_exponent(p0, f ? L.z : L.x, q, brow[slot_off<kBW>(16 * c + 2 * i)]);
                                p1 = far_exponent(p1, f ? L.w : L.y, q + 1, brow[slot_off<kBW>(16 * c + 2 * i + 1)]);
                            } else {
                                unpair(add_pair(fma_pair(pair(sv[2 * i], sv[2 * i + 1]), sl2_2, t[i]),
                                                f ? pair(L.z, L.w) : pair(L.x, L.y)), p0, p1);
                            }
                            p0 = ex2_approx(p0);
                            p1 = ex2_approx(p1);
                            unsigned long long d =
                                mul_pair(add_pair(pair(pv[2 * i], pv[2 * i + 1]), f ? pair(D.z, D.w) : pair(D.x, D.y)),
                                         pair(p0, p1));
                            wp[i] = pack_bf16x2(p0, p1);  // P and dS join their products in bf16, the operands' type
                            if (kBW == 4) {
                                wp[i] = on ? wp[i] : 0u;
                                d = on ? d : 0ull;
                            }
                            dacc[8 * c + i] = add_pair(dacc[8 * c + i], d);
                            float d0, d1;
                            unpair(d, d0, d1);
                            wd[i] = pack_bf16x2(d0, d1);
                        }
                    }
                    tmem_st8(trow + kColP + 8 * c, wp);
                    tmem_st8(trow + kColDS + 8 * c, wd);
#pragma unroll
                    for (int q4 = 0; q4 < 2; ++q4)
                        *reinterpret_cast<uint4*>(dsrow + (((2 * c + q4) ^ (r & 7)) << 4)) =
                            make_uint4(wd[4 * q4], wd[4 * q4 + 1], wd[4 * q4 + 2], wd[4 * q4 + 3]);
                }
            };
            if (far_table) gradient(std::true_type{});
            else gradient(std::false_type{});
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->p_ready);
            if (warp == 0 && mbar_wait_warp(&bars->p_ready, ph, ctl, 0x7203)) {
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_ts(tmem + kColDV + 32 * w, tmem + kColP + 8 * k, dMN0 + dof + 256 * w + 64 * k, id_dv, k > 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_ts(tmem + kColDK + 32 * w, tmem + kColDS + 8 * k, dMN0 + qo + 256 * w + 64 * k, id_dv, k > 0);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma_ss(tmem + col_dq(w), dDS + 128 * k, dMN0 + ko + 256 * w + 64 * k, id_dq, k > 0);
                    }
                    umma_commit(&bars->mma2_done);
                }
                __syncwarp();
            }
            if (!wwait(&bars->mma2_done, ph, 0x7308)) break;
            tc_fence_after();
#pragma unroll 1
            for (int which = 0; which < 3; ++which) {  // dq, dk, dv staged over q, k, v
                const uint32_t col = which == 0 ? col_dq(wi) : (which == 1 ? kColDK : kColDV) + 32 * wi;
                uint32_t v[32];
                tmem_ld32(trow + col, v);
                tmem_wait_ld();
                const float sc = which < 2 ? kScale : 1.f;
                float x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]) * sc;
                store_row_swz(sl + which * kTileBytes, r, x);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->staged);
        }
        if (warp == 0) {
            if (elect_one()) umma_commit(&bars->done);
            mbar_wait_warp(&bars->done, 0, ctl, 0x72ff);
        }
    }
    tc_fence_before();
    __syncthreads();  // every copy into and out of the slots is done
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
    // table gradient of this CTA: stage [query slot][row], then sum the pairs of
    // each displacement in a fixed order
    float* st = reinterpret_cast<float*>(smem);
    if (warp < 4) {
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            float a, b;
            unpair(dacc[e], a, b);
            st[2 * e * kTile + tid] = a;
            st[(2 * e + 1) * kTile + tid] = b;
        }
    }
    __syncthreads();
    for (int d = tid; d < 225; d += kThreads) {
        const int di = d / 15 - 7, dj = d % 15 - 7;
        float sum = 0.f;
        for (int iu = di < 0 ? -di : 0; iu < (di > 0 ? 8 - di : 8); ++iu)
            for (int ju = dj < 0 ? -dj : 0; ju < (dj > 0 ? 8 - dj : 8); ++ju) {
                const int it = iu + di, jt = ju + dj;
                const int u = kBW == 8 ? iu * 8 + ju : ((iu >> 2) * 2 + (ju >> 2)) * 16 + (iu & 3) * 4 + (ju & 3);
                const int t = kBW == 8 ? it * 8 + jt : ((it >> 2) * 2 + (jt >> 2)) * 16 + (it & 3) * 4 + (jt & 3);
                sum += st[t * kTile + u] + st[t * kTile + u + 64];
            }
        prm.part[static_cast<size_t>(blockIdx.x) * 225 + d] = sum;
    }
}

}  // namespace bwd8

// ------------------------------------------------------------------ M = 4
// Windows of 16 tokens: a 128-row tensor tile would use one score in eight, so
// each thread computes its row with fp32 multiply-adds from shared memory (a half
// warp is a window, all of whose threads read the same key row: a broadcast).
// The two windows of a warp read key rows whose numbers differ in bit 1, so that
// the 64-byte swizzle puts them into different banks.  No shift fits M = 4.  64 x 64 x 64
// tokens, 3 heads: forward 78 us (2.6 TB/s), backward 196 us (2.1 TB/s).
namespace m4 {

constexpr int kThreads = 128, kP4 = bias_pitch(4, 4);

struct Params {
    Geo g;
    const uint8_t *q, *k, *v, *o, *dout;
    uint8_t *o_out, *dq, *dk, *dv;
    const __nv_bfloat16* table;
    const int* buckets;
    int n_buckets;
    const float* lse;
    float* lse_out;
    float* part;  // [streams][heads][49]
    int streams;
};

// Row of a tile through loads that stay in program order: with all sixteen key
// rows of a window hoisted to the front the registers would not hold them.
__device__ __forceinline__ void load_row_ordered(const uint8_t* tile, int row, float (&x)[32]) {
    const uint32_t base = smem_u32(tile + row * kRowBytes);
    const uint32_t sw = (row >> 1) & 3;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 v = ld_shared_v4(base + ((c ^ sw) << 4));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[8 * c + 2 * e] = bf16lo_to_f32(w[e]);
            x[8 * c + 2 * e + 1] = bf16hi_to_f32(w[e]);
        }
    }
}

__device__ __forceinline__ float dot_row(const uint8_t* tile, int row, const float (&a)[32]) {
    float b[32], s[4] = {0.f, 0.f, 0.f, 0.f};
    load_row_ordered(tile, row, b);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        ffma2(s[0], s[1], a[e], a[e + 1], b[e], b[e + 1], s[0], s[1]);
        ffma2(s[2], s[3], a[e + 2], a[e + 3], b[e + 2], b[e + 3], s[2], s[3]);
    }
    return (s[0] + s[1]) + (s[2] + s[3]);
}

__device__ __forceinline__ void axpy_row(const uint8_t* tile, int row, float f, float (&acc)[32]) {
    float b[32];
    load_row_ordered(tile, row, b);
#pragma unroll
    for (int e = 0; e < 32; e += 2) ffma2(acc[e], acc[e + 1], b[e], b[e + 1], f, f, acc[e], acc[e + 1]);
}

__global__ void __launch_bounds__(kThreads, 4) fwd_kernel(const __grid_constant__ Params prm) {
    __shared__ __align__(128) uint8_t smem[3 * kTileBytes];
    __shared__ float tab[7 * kP4];
    const Geo& g = prm.g;
    const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
    const int h = blockIdx.x % g.heads, stream = blockIdx.x / g.heads;
    build_bias(tab, kP4, prm.table + static_cast<long long>(h) * prm.n_buckets, prm.buckets, prm.n_buckets, 4, r,
               kThreads);
    __syncthreads();
    const int e_r = r & 15, flip = (lane >> 4) << 1, w0 = r & ~15;
    const float* brow = tab + ((e_r >> 2) + 3) * kP4 + (e_r & 3) + 3;
    for (long long X = stream; X < g.tiles; X += prm.streams) {
        int pi, pj;
        long long tok;
        const bool valid = slot_token(g, X, r, h, &pi, &pj, &tok);
        load_rows(smem, prm.q, tok, valid, warp, lane);
        load_rows(smem + kTileBytes, prm.k, tok, valid, warp, lane);
        load_rows(smem + 2 * kTileBytes, prm.v, tok, valid, warp, lane);
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();  // a warp reads only the rows that it copied
        float a[32], s[16];
        load_row_swz(smem, r, a, false);
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            const int uu = u ^ flip;
            s[u] = fmaf(dot_row(smem + kTileBytes, w0 + uu, a), g.scale_log2, brow[-((uu >> 2) * kP4 + (uu & 3))]);
            m = fmaxf(m, s[u]);
        }
        const float mu = m == -INFINITY ? 0.f : m;
        float l = 0.f, acc[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            const float p = ex2_approx(s[u] - mu);
            l += p;
            axpy_row(smem + 2 * kTileBytes, w0 + (u ^ flip), p, acc);
        }
        const float inv = 1.f / l;
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = l == 0.f ? 0.f : acc[e] * inv;
        if (valid && prm.lse_out != nullptr) prm.lse_out[tok] = (m + lg2_approx(l)) * kLn2;
        store_row_swz(smem, r, acc);  // over this thread's own q row
        __syncwarp();
        save_rows(prm.o_out, smem, tok, valid, warp, lane);
        __syncwarp();
    }
}

constexpr int kXPitch = 17;  // exchange of P and dS inside a window: [query][key] with a padded pitch
constexpr int kBwdSmem = 5 * kTileBytes + 2 * 8 * 16 * kXPitch * 4;

__global__ void __launch_bounds__(kThreads, 3) bwd_kernel(const __grid_constant__ Params prm) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float tab[7 * kP4];
    float* xp = reinterpret_cast<float*>(smem + 5 * kTileBytes);  // P of the tile's 8 windows
    float* xd = xp + 8 * 16 * kXPitch;                            // dS
    const Geo& g = prm.g;
    const int r = threadIdx.x, warp = r >> 5, lane = r & 31;
    const int h = blockIdx.x % g.heads, stream = blockIdx.x / g.heads;
    build_bias(tab, kP4, prm.table + static_cast<long long>(h) * prm.n_buckets, prm.buckets, prm.n_buckets, 4, r,
               kThreads);
    __syncthreads();
    const int e_r = r & 15, flip = (lane >> 4) << 1, w0 = r & ~15;
    const float* brow = tab + ((e_r >> 2) + 3) * kP4 + (e_r & 3) + 3;
    uint8_t *tq = smem, *tk = smem + kTileBytes, *tv = smem + 2 * kTileBytes, *tdo = smem + 3 * kTileBytes,
            *to = smem + 4 * kTileBytes;
    float* myp = xp + (r >> 4) * 16 * kXPitch;
    float* myd = xd + (r >> 4) * 16 * kXPitch;
    float dacc[16];  // sum over the items of dS of (this query slot, key slot u ^ flip)
#pragma unroll
    for (int u = 0; u < 16; ++u) dacc[u] = 0.f;
    for (long long X = stream; X < g.tiles; X += prm.streams) {
        int pi, pj;
        long long tok;
        const bool valid = slot_token(g, X, r, h, &pi, &pj, &tok);
        load_rows(tq, prm.q, tok, valid, warp, lane);
        load_rows(tk, prm.k, tok, valid, warp, lane);
        load_rows(tv, prm.v, tok, valid, warp, lane);
        load_rows(tdo, prm.dout, tok, valid, warp, lane);
        load_rows(to, prm.o, tok, valid, warp, lane);
        cp_async_commit();
        const float lse = valid ? __ldg(prm.lse + tok) : -INFINITY;
        const float lse2 = grad_lse2(lse);
        const bool is_far = finite_beyond(lse * 1.4426950408889634f, kFar);
        cp_async_wait<0>();
        __syncwarp();
        float p[16];
        {
            float a[32];
            load_row_swz(tq, r, a, false);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int uu = u ^ flip;
                const float s = dot_row(tk, w0 + uu, a), b = brow[-((uu >> 2) * kP4 + (uu & 3))];
                p[u] = is_far ? fmaf(s, g.scale_log2, b) : ex2_approx(fmaf(s, g.scale_log2, b - lse2));
            }
            if (is_far) {  // the maximum and the sum of the row's scores, as in the forward
                float m = p[0], l = 0.f;
#pragma unroll
                for (int u = 1; u < 16; ++u) m = fmaxf(m, p[u]);
#pragma unroll
                for (int u = 0; u < 16; ++u) l += p[u] = ex2_approx(p[u] - m);
                const float inv = 1.f / l;
#pragma unroll
                for (int u = 0; u < 16; ++u) p[u] *= inv;
            }
#pragma unroll
            for (int u = 0; u < 16; ++u) myp[e_r * kXPitch + (u ^ flip)] = p[u];
        }
        float acc[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = 0.f;
        {
            float a[32];
            load_row_swz(tdo, r, a, false);
            const float D = dot_row(to, r, a);
#pragma unroll
            for (int u = 0; u < 16; ++u) {
                const int uu = u ^ flip;
                const float d = p[u] * (dot_row(tv, w0 + uu, a) - D);
                dacc[u] += d;
                myd[e_r * kXPitch + uu] = d;
                axpy_row(tk, w0 + uu, d, acc);
            }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] *= kScale;
        store_row_swz(to, r, acc);  // dq, over this thread's own o row
        __syncwarp();               // the windows' P and dS are in place
        float acv[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] = acv[e] = 0.f;
#pragma unroll 4
        for (int t = 0; t < 16; ++t) {  // as key row: the queries of its window
            const int tt = t ^ flip;
            axpy_row(tq, w0 + tt, myd[tt * kXPitch + e_r], acc);
            axpy_row(tdo, w0 + tt, myp[tt * kXPitch + e_r], acv);
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) acc[e] *= kScale;
        __syncwarp();  // every thread of the warp has read the k and v rows
        store_row_swz(tk, r, acc);
        store_row_swz(tv, r, acv);
        __syncwarp();
        save_rows(prm.dq, to, tok, valid, warp, lane);
        save_rows(prm.dk, tk, tok, valid, warp, lane);
        save_rows(prm.dv, tv, tok, valid, warp, lane);
        __syncwarp();
    }
    __syncthreads();
    float* st = reinterpret_cast<float*>(smem);  // [key slot][row]
#pragma unroll
    for (int u = 0; u < 16; ++u) st[(u ^ flip) * kThreads + r] = dacc[u];
    __syncthreads();
    if (r < 49) {
        const int di = r / 7 - 3, dj = r % 7 - 3;
        float sum = 0.f;
        for (int iu = di < 0 ? -di : 0; iu < (di > 0 ? 4 - di : 4); ++iu)
            for (int ju = dj < 0 ? -dj : 0; ju < (dj > 0 ? 4 - dj : 4); ++ju)
                for (int w = 0; w < 8; ++w) sum += st[(iu * 4 + ju) * kThreads + w * 16 + (iu + di) * 4 + ju + dj];
        prm.part[static_cast<size_t>(blockIdx.x) * 49 + r] = sum;
    }
}

}  // namespace m4

// ------------------------------------------------------------------ launches
cudaError_t launch_small_fwd(const Geo& g, const RelbPtrs& p, unsigned int* status, unsigned long long limit_ns,
                             int num_sms, cudaStream_t stream) {
    if (g.M == 4) {
        m4::Params prm{};
        prm.g = g;
        prm.q = static_cast<const uint8_t*>(p.q);
        prm.k = static_cast<const uint8_t*>(p.k);
        prm.v = static_cast<const uint8_t*>(p.v);
        prm.o_out = static_cast<uint8_t*>(p.o_out);
        prm.lse_out = p.lse_out;
        prm.table = static_cast<const __nv_bfloat16*>(p.table);
        prm.buckets = p.buckets;
        prm.n_buckets = p.n_buckets;
        prm.streams = streams_per_head(g.tiles, g.heads, 4 * num_sms);
        m4::fwd_kernel<<<static_cast<unsigned>(prm.streams) * g.heads, m4::kThreads, 0, stream>>>(prm);
        return cudaGetLastError();
    }
    static SmemOptIn optin8, optin4;
    const bool b8 = g.bw == 8;
    auto* kern = b8 ? fwd8::fwd_kernel<8> : fwd8::fwd_kernel<4>;
    if (cudaError_t e = (b8 ? optin8 : optin4).ensure(reinterpret_cast<const void*>(kern), fwd8::kSmemBytes)) return e;
    fwd8::Params prm{};
    prm.g = g;
    prm.q = static_cast<const uint8_t*>(p.q);
    prm.k = static_cast<const uint8_t*>(p.k);
    prm.v = static_cast<const uint8_t*>(p.v);
    prm.o = static_cast<uint8_t*>(p.o_out);
    prm.lse = p.lse_out;
    prm.table = static_cast<const __nv_bfloat16*>(p.table);
    prm.buckets = p.buckets;
    prm.n_buckets = p.n_buckets;
    prm.status = status;
    prm.limit_ns = limit_ns;
    prm.streams = streams_per_head(g.tiles, g.heads, 4 * num_sms);
    kern<<<static_cast<unsigned>(prm.streams) * g.heads, fwd8::kThreads, fwd8::kSmemBytes, stream>>>(prm);
    return cudaGetLastError();
}

cudaError_t launch_small_bwd(const Geo& g, const RelbPtrs& p, float* part, int streams, unsigned int* status,
                             unsigned long long limit_ns, cudaStream_t stream) {
    const unsigned grid = static_cast<unsigned>(streams) * g.heads;
    if (g.M == 4) {
        static SmemOptIn optin;
        if (cudaError_t e = optin.ensure(reinterpret_cast<const void*>(m4::bwd_kernel), m4::kBwdSmem)) return e;
        m4::Params prm{};
        prm.g = g;
        prm.q = static_cast<const uint8_t*>(p.q);
        prm.k = static_cast<const uint8_t*>(p.k);
        prm.v = static_cast<const uint8_t*>(p.v);
        prm.o = static_cast<const uint8_t*>(p.o);
        prm.dout = static_cast<const uint8_t*>(p.dout);
        prm.dq = static_cast<uint8_t*>(p.dq);
        prm.dk = static_cast<uint8_t*>(p.dk);
        prm.dv = static_cast<uint8_t*>(p.dv);
        prm.lse = p.lse;
        prm.table = static_cast<const __nv_bfloat16*>(p.table);
        prm.buckets = p.buckets;
        prm.n_buckets = p.n_buckets;
        prm.part = part;
        prm.streams = streams;
        m4::bwd_kernel<<<grid, m4::kThreads, m4::kBwdSmem, stream>>>(prm);
        return cudaGetLastError();
    }
    static SmemOptIn optin8, optin4;
    const bool b8 = g.bw == 8;
    auto* kern = b8 ? bwd8::bwd_kernel<8> : bwd8::bwd_kernel<4>;
    if (cudaError_t e = (b8 ? optin8 : optin4).ensure(reinterpret_cast<const void*>(kern), bwd8::kSmemBytes)) return e;
    bwd8::Params prm{};
    prm.g = g;
    prm.q = static_cast<const uint8_t*>(p.q);
    prm.k = static_cast<const uint8_t*>(p.k);
    prm.v = static_cast<const uint8_t*>(p.v);
    prm.o = static_cast<const uint8_t*>(p.o);
    prm.dout = static_cast<const uint8_t*>(p.dout);
    prm.dq = static_cast<uint8_t*>(p.dq);
    prm.dk = static_cast<uint8_t*>(p.dk);
    prm.dv = static_cast<uint8_t*>(p.dv);
    prm.lse = p.lse;
    prm.table = static_cast<const __nv_bfloat16*>(p.table);
    prm.buckets = p.buckets;
    prm.n_buckets = p.n_buckets;
    prm.part = part;
    prm.status = status;
    prm.limit_ns = limit_ns;
    prm.streams = streams;
    kern<<<grid, bwd8::kThreads, bwd8::kSmemBytes, stream>>>(prm);
    return cudaGetLastError();
}

}  // namespace relb

}  // namespace fswin

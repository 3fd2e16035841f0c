// Host-side launch entry points of the kernels, shared by api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "geometry.cuh"

namespace fswin {

// Opts a kernel into more than the default 48 KB of dynamic shared memory.  The
// attribute is per device, so it is set once for every device the kernel is
// launched on (the first launch there, with that device current), under a lock
// because several host threads may launch at once.
class SmemOptIn {
   public:
    cudaError_t ensure(const void* func, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kDevices)
            return cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        std::lock_guard<std::mutex> lk(mu_);
        if (!done_[dev]) {
            e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e != cudaSuccess) return e;
            done_[dev] = true;
        }
        return cudaSuccess;
    }

   private:
    static constexpr int kDevices = 64;
    std::mutex mu_;
    bool done_[kDevices] = {};
};

// Checks that the current device can run the kernels (sm_100) and sets up the
// library's per-device state; returns an fs_status code (0 when usable).
int device_ready();

long long fwd_items(const Geo& g);
// train_ws: NULL, or the backward's workspace (windows of >= 128 tokens): the
// forward then first writes the rotated q', k' tile images there (the images
// the backward's prep would write) and reads Q', K' from them, instead of
// rotating every K tile again for each query tile of its window.
cudaError_t launch_fwd(const Geo& g, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const CUtensorMap& mo, const void* q, const void* k, const void* v, void* o,
                       const float* theta, float* lse, unsigned int* status,
                       unsigned long long limit_ns, int num_sms, cudaStream_t stream, cudaEvent_t const* events,
                       uint8_t* train_ws = nullptr);

struct BwdPtrs {
    const void *q, *k, *v, *o, *dout;
    const float *lse, *theta;
    void *dq, *dk, *dv;
    float* dtheta;
    uint8_t* ws;
};

// TMA maps (window boxes) of the backward's token tensors.
struct BwdMaps {
    CUtensorMap q, k, v, o, dout, dq, dk, dv;
};

long long bwd_items(const Geo& g);
size_t bwd_workspace_bytes(const Geo& g);
// Offsets of the rotated q', k' tile images in the backward's workspace, and
// the launch that writes them (windows of >= 128 tokens).
void bwd_image_offsets(const Geo& g, size_t* qimg, size_t* kimg);
cudaError_t launch_rope_images(const Geo& g, const void* q, const void* k, const float* theta, uint8_t* ws,
                               cudaStream_t stream);
// events: NULL, or 5 events recorded before the first and after each of the
// four launches (prep, main, post, d theta; windows of fewer than 128 tokens
// run one kernel in the place of the first three).
// images_ready: the workspace already holds the q', k' images of these inputs
// (written by a training forward, windows of >= 128 tokens): prep skips them.
cudaError_t launch_bwd(const Geo& g, const BwdPtrs& p, const BwdMaps& maps, unsigned int* status,
                       unsigned long long limit_ns, int num_sms, cudaStream_t stream, cudaEvent_t const* events,
                       bool images_ready = false);

// Windows of fewer than 128 tokens (the tile holds whole windows): the whole
// backward of a tile in one kernel (d theta partials, 4 x 16 per (head, tile),
// into `part`), and the forward.
cudaError_t launch_small_bwd(const Geo& g, const BwdPtrs& p, float* part, unsigned int* dtheta_cnt,
                             unsigned int* status, unsigned long long limit_ns, int num_sms, cudaStream_t stream);
cudaError_t launch_small_fwd(const Geo& g, const void* q, const void* k, const void* v, const float* theta, void* o,
                             float* lse, unsigned int* status, unsigned long long limit_ns, int num_sms,
                             cudaStream_t stream);

// Heads of d = 64 channels, every window size (plain one-tile pipelines).  The
// backward's workspace holds an fp32 dQ' accumulator of 256 bytes per
// token-head row and the d theta partials.
size_t wide_bwd_workspace_bytes(const Geo& g);
// events: NULL, or (forward) 2 events recorded before and after the kernel,
// (backward) 5 events recorded before the first and after each of prep, main,
// post and the d theta sum.
cudaError_t launch_wide_fwd(const Geo& g, const void* q, const void* k, const void* v, const float* theta, void* o,
                            float* lse, unsigned int* status, unsigned long long limit_ns, int num_sms,
                            cudaStream_t stream, cudaEvent_t const* events);
cudaError_t launch_wide_bwd(const Geo& g, const BwdPtrs& p, unsigned int* status, unsigned long long limit_ns,
                            int num_sms, cudaStream_t stream, cudaEvent_t const* events);

// Windowed attention with a low-rank additive bias U_h W_h^T (heads of 32
// channels, every window size; theta may be null: no rotation, no d theta).
struct LrbPtrs {
    const void *q, *k, *v, *o, *dout;  // bf16 [B, H, W, heads, 32]
    const float *lse, *theta;           // theta: [heads][2][8] or null
    const float *u, *w;                 // [heads][M*M][16]
    void *o_out, *dq, *dk, *dv;         // o_out: the forward's O
    float *lse_out, *dtheta, *du, *dw;
    uint8_t* ws;
};
size_t lrbias_bwd_workspace_bytes(const Geo& g);
// events as for the 64-channel kernels (the backward's last mark follows the
// d theta and dU / dW sums).
cudaError_t launch_lrbias_fwd(const Geo& g, const LrbPtrs& p, unsigned int* status, unsigned long long limit_ns,
                              int num_sms, cudaStream_t stream, cudaEvent_t const* events);
cudaError_t launch_lrbias_bwd(const Geo& g, const LrbPtrs& p, unsigned int* status, unsigned long long limit_ns,
                              int num_sms, cudaStream_t stream, cudaEvent_t const* events);

// Windowed attention with a learned relative position bias by buckets (heads of
// 32 channels, every window size).
struct RelbPtrs {
    const void *q, *k, *v, *o, *dout;  // bf16 [B, H, W, heads, 32]
    const void* table;                 // bf16 [heads][n_buckets]
    const int* buckets;                // [(2M-1)^2] displacement -> bucket, or null: the displacement is the bucket
    int n_buckets;
    const float* lse;
    void *o_out, *dq, *dk, *dv, *dtable;  // o_out: the forward's O; dtable: bf16 [heads][n_buckets]
    float* lse_out;
    uint8_t* ws;
};
size_t relbias_bwd_workspace_bytes(const Geo& g);
// events as for the 64-channel kernels (the backward's last mark follows the
// table gradient's sum; windows of fewer than 128 tokens run one kernel in the
// place of prep, main and post).
// TMA maps of the token tensors, read by windows of 128 tokens or more.
struct RelbMaps {
    CUtensorMap q, k, v, dout;
};
cudaError_t launch_relbias_fwd(const Geo& g, const RelbPtrs& p, const RelbMaps& maps, unsigned int* status,
                               unsigned long long limit_ns, int num_sms, cudaStream_t stream,
                               cudaEvent_t const* events);
cudaError_t launch_relbias_bwd(const Geo& g, const RelbPtrs& p, const RelbMaps& maps, unsigned int* status,
                               unsigned long long limit_ns, cudaStream_t stream, cudaEvent_t const* events);

// The residual step of a layer with its norms: r = x + g_b gamma o drop(post(f)),
// n = pre(r), and its backward.
struct ResnormPtrs {
    const void *x, *f;                                       // forward: stream type, bf16
    const void *gate, *scale, *post_w, *post_b, *pre_w, *pre_b;  // stream type, each may be null
    const long long* rng;                                    // (seed, offset), read when elements are dropped
    void *r, *n;                                             // r: the backward reads it
    const void *dr, *dn;                                     // either may be null
    void *dx, *df, *dgate, *dscale, *dpost_w, *dpost_b, *dpre_w, *dpre_b;
    uint8_t* ws;
    long long samples;
};
struct ResnormShape {
    long long samples, tokens;
    int channels;
    bool stream_f32;
    int pre, post;  // 0 none, 1 layer norm, 2 rms norm
    float eps;
    double drop_p;
    // Sixteen-byte accesses: every tensor is aligned, and a row that starts anywhere in
    // a chunk of eight channels takes at most 1024 chunks.
    bool wide(const ResnormPtrs& p) const {
        const void* all[] = {p.x,  p.f,  p.scale, p.post_w, p.post_b, p.pre_w, p.pre_b,
                             p.r,  p.n,  p.dr,    p.dn,     p.dx,     p.df};
        uintptr_t bits = 0;
        for (const void* q : all) bits |= reinterpret_cast<uintptr_t>(q);
        return (bits & 15u) == 0 && (channels % 8 == 0 || channels <= 8192 - 14);
    }
};
size_t resnorm_bwd_workspace_bytes(const ResnormShape& sh);
cudaError_t launch_resnorm_fwd(const ResnormShape& sh, const ResnormPtrs& p, int num_sms, cudaStream_t stream);
cudaError_t launch_resnorm_bwd(const ResnormShape& sh, const ResnormPtrs& p, cudaStream_t stream);

// The gated feed-forward block y = (act(x Wg^T + bg) o (x Wu^T + bu)) Wd^T + bd and
// its backward, all bf16: x, y, dy, dx [tokens, channels], w_gate, w_up [hidden,
// channels], w_down [channels, hidden].
struct MlpShape {
    long long tokens;
    int channels, hidden, act;  // act: 0 silu, 1 gelu
};
struct MlpPtrs {
    const void *x, *dy, *w_gate, *w_up, *w_down, *b_gate, *b_up, *b_down;
    void *y, *dx, *dw_gate, *dw_up, *dw_down, *db_gate, *db_up, *db_down;
    uint8_t* ws;
};
size_t mlp_fwd_workspace_bytes(const MlpShape& sh);
size_t mlp_bwd_workspace_bytes(const MlpShape& sh);
// Where all weights fit into shared memory the forward is one kernel, without workspace.
bool mlp_fits(const MlpShape& sh);
cudaError_t launch_mlp_small_fwd(const MlpShape& sh, const MlpPtrs& p, unsigned int* status, unsigned long long limit_ns,
                                 int num_sms, cudaStream_t stream);
cudaError_t launch_mlp_fwd(const MlpShape& sh, const MlpPtrs& p, unsigned int* status, unsigned long long limit_ns,
                           int num_sms, cudaStream_t stream);
cudaError_t launch_mlp_bwd(const MlpShape& sh, const MlpPtrs& p, unsigned int* status, unsigned long long limit_ns,
                           int num_sms, cudaStream_t stream);

// TMA map of a row-major bf16 matrix: box of box_rows x box_cols (box_cols 64 with
// the 128-byte swizzle, 32 with the 64-byte one).  0 on success.  Needs the
// library's per-device state (device_ready).
int encode_matrix(CUtensorMap* m, const void* base, long long rows, long long cols, int box_rows, int box_cols,
                  bool swizzle128);

// Fixed-order d theta sum: part [heads][per_head][16] -> dtheta [heads][16] (one
// launch; cnt: heads counters that are zero when it starts).
namespace bwdk {
cudaError_t launch_dtheta(const float* part, long long per_head, int heads, float* scratch, unsigned int* cnt,
                          float* dtheta, cudaStream_t stream);
}

// The attention block with its projections (inference), windows of fewer than
// 128 tokens, at most three heads: y = attention(x W_qkv^T + b_qkv) W_o^T + b_o.
struct BlockPtrs {
    const void *x, *w_qkv, *w_o;  // bf16 [B,H,W,C], [3C,C], [C,C]
    const float *b_qkv, *b_o, *theta;
    void* y;  // bf16 [B,H,W,C]
};
cudaError_t launch_block_fwd(const Geo& g, const BlockPtrs& p, unsigned int* status, unsigned long long limit_ns,
                             int num_sms, cudaStream_t stream);

}  // namespace fswin

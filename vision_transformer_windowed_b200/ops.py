"""Torch-facing wrappers of the C ABI: they allocate outputs with PyTorch, pass
raw device pointers and the current CUDA stream, and nothing else.  Every step
of the attention runs in the CUDA kernels of libfswin.so.

Method: FlashSwin ("FLASHSWIN: Unlocking Large Windows and Dense Tokens in Swin
Vision Transformers with Memory Efficient Attention", thelatestinai.com/papers/
2610.04664, Figure 1B): exact windowed softmax attention with window-local
learnable 2D RoPE, the fused FlashAttention-style kernel replacing Swin's
materialised score matrix.

Shapes: q, k, v [B, H, W, heads, d] bf16 with d = 32 or 64, H >= M and W >= M.  H or W
need not be a multiple of the window M: the grid is then worked on padded at
the bottom and right with zero tokens to the next multiple (the Swin layer's
padding), and only the H x W real tokens are read and written.

The autograd functions are differentiable once: a backward through their
gradients raises.
"""
from __future__ import annotations

from collections import namedtuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib

HEAD_DIM = 32


def _shape(q: torch.Tensor, M: int, s: int) -> _lib.Shape:
    if q.dim() != 5:
        raise ValueError("expected a [B, H, W, heads, d] tensor")
    B, H, W, heads, d = q.shape
    return _lib.make_shape(B, H, W, heads, d, M, s)


def _check_tensor(name: str, t: torch.Tensor, shape, dtype) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def winattn_fwd(q, k, v, theta, M: int, s: int, o=None, lse=None, need_lse: bool = True, workspace=None):
    """O, LSE = fused windowed-RoPE attention forward (bf16 in/out, fp32 LSE).

    need_lse=False (and no lse buffer): inference forward, O only; LSE is returned as None.
    workspace (the backward's, from alloc_workspace): the training forward, which
    also leaves the rotated q', k' tiles there for winattn_bwd(..., after_train_fwd=True)."""
    sh = _shape(q, M, s)
    B, H, W, heads, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, q.shape, torch.bfloat16)
    _check_tensor("theta", theta, (heads, 2, d // 4), torch.float32)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and need_lse:
        lse = torch.empty((B, H, W, heads), device=q.device, dtype=torch.float32)
    _check_tensor("o", o, q.shape, torch.bfloat16)
    if lse is not None:
        _check_tensor("lse", lse, (B, H, W, heads), torch.float32)
    if workspace is not None:
        if lse is None:
            raise ValueError("the training forward writes lse")
        _lib.fs_winattn_fwd_train(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), theta.data_ptr(), o.data_ptr(),
                                  lse.data_ptr(), workspace.data_ptr(), workspace.numel(), _stream(q.device))
        return o, lse
    _lib.fs_winattn_fwd(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), theta.data_ptr(), o.data_ptr(),
                        lse.data_ptr() if lse is not None else 0, _stream(q.device))
    return o, lse


def winattn_block_fwd(x, w_qkv, b_qkv, w_o, b_o, theta, M: int, s: int, heads: int, y=None):
    """y = windowed-RoPE attention of (x W_qkv^T + b_qkv) per head, then W_o, b_o
    (the attention block of a Swin layer, inference; M*M < 128, heads <= 3)."""
    B, H, W, C = x.shape
    d = C // heads
    sh = _lib.make_shape(B, H, W, heads, d, M, s)
    _check_tensor("x", x, (B, H, W, C), torch.bfloat16)
    _check_tensor("w_qkv", w_qkv, (3 * C, C), torch.bfloat16)
    _check_tensor("b_qkv", b_qkv, (3 * C,), torch.float32)
    _check_tensor("w_o", w_o, (C, C), torch.bfloat16)
    _check_tensor("b_o", b_o, (C,), torch.float32)
    _check_tensor("theta", theta, (heads, 2, d // 4), torch.float32)
    if y is None:
        y = torch.empty_like(x)
    _check_tensor("y", y, (B, H, W, C), torch.bfloat16)
    _lib.fs_winattn_block_fwd(sh, x.data_ptr(), w_qkv.data_ptr(), b_qkv.data_ptr(), w_o.data_ptr(), b_o.data_ptr(),
                              theta.data_ptr(), y.data_ptr(), _stream(x.device))
    return y


def bwd_workspace_bytes(B: int, H: int, W: int, heads: int, M: int, s: int, d: int = HEAD_DIM) -> int:
    return _lib.fs_winattn_bwd_workspace_bytes(_lib.make_shape(B, H, W, heads, d, M, s))


def alloc_workspace(q: torch.Tensor, M: int, s: int) -> torch.Tensor:
    n = _lib.fs_winattn_bwd_workspace_bytes(_shape(q, M, s))
    return torch.empty(max(n, 256), device=q.device, dtype=torch.uint8)


def winattn_bwd(q, k, v, o, dout, lse, theta, M: int, s: int, workspace=None, dq=None, dk=None, dv=None,
                dtheta=None, after_train_fwd: bool = False):
    """dQ, dK, dV, dtheta of sum(O * dout) (recompute-based backward).

    after_train_fwd: `workspace` is the one a training forward (winattn_fwd with
    that workspace) of the same q, k, theta filled, unchanged since; its rotated
    q', k' tiles are reused."""
    sh = _shape(q, M, s)
    B, H, W, heads, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_tensor(name, t, q.shape, torch.bfloat16)
    _check_tensor("lse", lse, (B, H, W, heads), torch.float32)
    _check_tensor("theta", theta, (heads, 2, d // 4), torch.float32)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    dtheta = torch.empty_like(theta) if dtheta is None else dtheta
    if workspace is None:
        if after_train_fwd:
            raise ValueError("after_train_fwd needs the training forward's workspace")
        workspace = alloc_workspace(q, M, s)
    call = _lib.fs_winattn_bwd_train if after_train_fwd else _lib.fs_winattn_bwd
    call(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(), lse.data_ptr(),
         theta.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dtheta.data_ptr(),
         workspace.data_ptr(), workspace.numel(), _stream(q.device))
    return dq, dk, dv, dtheta


class WindowAttentionRoPE(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run in libfswin.so.

    theta are the inverse frequencies; with the log parameterisation of the
    paper (theta = exp(omega), thelatestinai.com/papers/2610.04664, Figure S4)
    autograd through ``torch.exp`` gives d omega = theta * d theta.
    """

    @staticmethod
    def forward(ctx, q, k, v, theta, M: int, s: int, reuse_rotated: bool = False):
        # reuse_rotated: the training pair, whose forward leaves the rotated q', k'
        # tiles in the backward's workspace; the workspace (about 262 bytes per
        # token-head) then stays allocated until the backward, beside the saved
        # q, k, v, o (256 bytes per token-head)
        ws = alloc_workspace(q, M, s) if reuse_rotated else None
        o, lse = winattn_fwd(q, k, v, theta, M, s, workspace=ws)
        ctx.save_for_backward(q, k, v, o, lse, theta, *(() if ws is None else (ws,)))
        ctx.M, ctx.s, ctx.reuse = M, s, reuse_rotated
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, theta, *ws = ctx.saved_tensors
        dq, dk, dv, dth = winattn_bwd(q, k, v, o, dout.contiguous(), lse, theta, ctx.M, ctx.s,
                                      workspace=ws[0] if ctx.reuse else None, after_train_fwd=ctx.reuse)
        return dq, dk, dv, dth, None, None, None


def window_attention(q, k, v, theta, M: int, s: int, reuse_rotated: bool = False):
    """Autograd windowed-RoPE attention.  reuse_rotated=True runs the training
    pair (faster at windows of >= 128 tokens; keeps the backward's workspace
    from the forward to the backward)."""
    return WindowAttentionRoPE.apply(q, k, v, theta, M, s, reuse_rotated)


# ------------------------------------------------------------ low-rank bias
# The FlashBias-T variant of the same pages (thelatestinai.com/papers/2610.04664,
# Table 2 and Table S1 captions): a trainable rank-16 factorization U_h W_h^T of
# an additive bias over window-local positions, shared by every window and added
# to the scaled scores before the shift mask.  Heads of 32 channels; theta may be
# None (no rotation).
LRBIAS_RANK = 16


def _check_factors(q, u, w, M: int) -> None:
    heads = q.shape[3]
    for name, t in (("u", u), ("w", w)):
        _check_tensor(name, t, (heads, M * M, LRBIAS_RANK), torch.float32)


def winattn_lrbias_fwd(q, k, v, theta, u, w, M: int, s: int, o=None, lse=None, need_lse: bool = True):
    """O, LSE of windowed attention with the low-rank bias u_t . w_u (bf16 in/out, fp32 LSE)."""
    sh = _shape(q, M, s)
    B, H, W, heads, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, q.shape, torch.bfloat16)
    if theta is not None:
        _check_tensor("theta", theta, (heads, 2, d // 4), torch.float32)
    _check_factors(q, u, w, M)
    if o is None:
        o = torch.empty_like(q)
    if lse is None and need_lse:
        lse = torch.empty((B, H, W, heads), device=q.device, dtype=torch.float32)
    _check_tensor("o", o, q.shape, torch.bfloat16)
    if lse is not None:
        _check_tensor("lse", lse, (B, H, W, heads), torch.float32)
    _lib.fs_winattn_lrbias_fwd(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                               theta.data_ptr() if theta is not None else 0, u.data_ptr(), w.data_ptr(),
                               LRBIAS_RANK, o.data_ptr(), lse.data_ptr() if lse is not None else 0,
                               _stream(q.device))
    return o, lse


def alloc_lrbias_workspace(q: torch.Tensor, M: int, s: int) -> torch.Tensor:
    n = _lib.fs_winattn_lrbias_bwd_workspace_bytes(_shape(q, M, s))
    return torch.empty(max(n, 256), device=q.device, dtype=torch.uint8)


def winattn_lrbias_bwd(q, k, v, o, dout, lse, theta, u, w, M: int, s: int, workspace=None, dq=None, dk=None,
                       dv=None, dtheta=None, du=None, dw=None):
    """dQ, dK, dV, dtheta (None without theta), dU, dW of sum(O * dout)."""
    sh = _shape(q, M, s)
    B, H, W, heads, d = q.shape
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _check_tensor(name, t, q.shape, torch.bfloat16)
    _check_tensor("lse", lse, (B, H, W, heads), torch.float32)
    if theta is not None:
        _check_tensor("theta", theta, (heads, 2, d // 4), torch.float32)
    _check_factors(q, u, w, M)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    dtheta = (torch.empty_like(theta) if dtheta is None else dtheta) if theta is not None else None
    du = torch.empty_like(u) if du is None else du
    dw = torch.empty_like(w) if dw is None else dw
    for name, t, ref in (("dq", dq, q), ("dk", dk, q), ("dv", dv, q), ("du", du, u), ("dw", dw, w)):
        _check_tensor(name, t, ref.shape, ref.dtype)
    if dtheta is not None:
        _check_tensor("dtheta", dtheta, theta.shape, torch.float32)
    if workspace is None:
        workspace = alloc_lrbias_workspace(q, M, s)
    _lib.fs_winattn_lrbias_bwd(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                               lse.data_ptr(), theta.data_ptr() if theta is not None else 0, u.data_ptr(),
                               w.data_ptr(), LRBIAS_RANK, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                               dtheta.data_ptr() if dtheta is not None else 0, du.data_ptr(), dw.data_ptr(),
                               workspace.data_ptr(), workspace.numel(), _stream(q.device))
    return dq, dk, dv, dtheta, du, dw


class WindowAttentionLowRankBias(torch.autograd.Function):
    """Autograd wrapper of the low-rank-bias attention (forward and backward in libfswin.so)."""

    @staticmethod
    def forward(ctx, q, k, v, theta, u, w, M: int, s: int):
        o, lse = winattn_lrbias_fwd(q, k, v, theta, u, w, M, s)
        ctx.save_for_backward(q, k, v, o, lse, u, w, *(() if theta is None else (theta,)))
        ctx.M, ctx.s, ctx.has_theta = M, s, theta is not None
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, u, w, *rest = ctx.saved_tensors
        theta = rest[0] if ctx.has_theta else None
        dq, dk, dv, dth, du, dw = winattn_lrbias_bwd(q, k, v, o, dout.contiguous(), lse, theta, u, w, ctx.M, ctx.s)
        return dq, dk, dv, dth, du, dw, None, None


def window_attention_lrbias(q, k, v, theta, u, w, M: int, s: int):
    return WindowAttentionLowRankBias.apply(q, k, v, theta, u, w, M, s)


# ------------------------------------------------- learned relative position bias
# The additive bias of a Swin layer, by buckets: S_tu = q_t . k_u / sqrt(d) +
# table[h][b(i_t - i_u, j_t - j_u)].  Without a bucket map every displacement has
# an entry of its own, in the order of Swin's relative_position_index (Swin's
# [(2M-1)^2, heads] table transposed).  Heads of 32 channels, no rotation.
def log_distance_buckets(M: int, exact: int = 4, device="cuda"):
    """(buckets int32 [2M-1, 2M-1], their number): per axis, signed distances below `exact` keep a bucket each and
    longer ones share one an octave; the two axes' buckets multiply."""
    if M < 1 or exact < 1:
        raise ValueError("M and exact must be positive")

    def axis(x):
        a = abs(x)
        b = a if a < exact else exact + (a // exact).bit_length() - 1
        return b if x >= 0 else -b

    one = torch.tensor([axis(x) for x in range(-(M - 1), M)], dtype=torch.int32)
    one = one - one.min()
    n = int(one.max()) + 1
    return (one[:, None] * n + one[None, :]).contiguous().to(device), n * n


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _need(name: str, t: torch.Tensor, dtype, shape, device: int) -> None:
    """One argument's checks in one test; only a failing argument takes the slow road to its message."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    _check_tensor(name, t, shape, dtype)
    raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{device}")


def _device_of(name: str, t: torch.Tensor) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


class _on:
    """Makes the tensors' device current for the launches (a no-op when it is); gives its current stream."""

    def __init__(self, device: int):
        self.device = device
        self.prev = torch._C._cuda_getDevice()

    def __enter__(self) -> int:
        if self.prev != self.device:
            torch.cuda.set_device(self.device)
        return torch._C._cuda_getCurrentRawStream(self.device)

    def __exit__(self, *exc):
        if self.prev != self.device:
            torch.cuda.set_device(self.prev)


def _workspace(need: int, workspace, device: int) -> torch.Tensor:
    if workspace is None:
        return torch.empty(max(need, 256), device=torch.device("cuda", device), dtype=torch.uint8)
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{device}")
    return workspace


def _check_relbias(q, k, v, table, M: int, buckets) -> int:
    device, shape = _device_of("q", q), q.shape
    for name, t in (("q", q), ("k", k), ("v", v)):
        _need(name, t, torch.bfloat16, shape, device)
    if table.dim() != 2:
        raise ValueError("table must be [heads, buckets]")
    _need("table", table, torch.bfloat16, (shape[3], table.shape[1]), device)
    if buckets is not None:
        _need("buckets", buckets, torch.int32, (2 * M - 1, 2 * M - 1), device)
    elif table.shape[1] != (2 * M - 1) ** 2:
        raise ValueError(f"without a bucket map the table has {(2 * M - 1) ** 2} entries a head, got {table.shape[1]}")
    return device


def winattn_relbias_fwd(q, k, v, table, M: int, s: int, buckets=None, o=None, lse=None, need_lse: bool = True):
    """O, LSE of windowed attention with the bias table[h][bucket of the displacement] (bf16 in/out, fp32 LSE).

    table: bf16 [heads, n]; buckets: int32 [2M-1, 2M-1] (query minus key, row then column, each plus M-1), or None:
    n = (2M-1)^2.  A bucket outside [0, n) adds no bias.  need_lse=False: inference, LSE is returned as None."""
    sh = _shape(q, M, s)
    device = _check_relbias(q, k, v, table, M, buckets)
    if o is None:
        o = torch.empty_like(q)
    else:
        _need("o", o, torch.bfloat16, q.shape, device)
    if lse is not None:
        _need("lse", lse, torch.float32, q.shape[:4], device)
    elif need_lse:
        lse = torch.empty(q.shape[:4], device=q.device, dtype=torch.float32)
    with _on(device) as stream:
        _lib.fs_winattn_relbias_fwd(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), table.data_ptr(), _ptr(buckets),
                                    table.shape[1], o.data_ptr(), _ptr(lse), stream)
    return o, lse


def alloc_relbias_workspace(q: torch.Tensor, M: int, s: int) -> torch.Tensor:
    n = _lib.fs_winattn_relbias_bwd_workspace_bytes(_shape(q, M, s))
    return torch.empty(max(n, 256), device=q.device, dtype=torch.uint8)


def winattn_relbias_bwd(q, k, v, o, dout, lse, table, M: int, s: int, buckets=None, workspace=None, dq=None, dk=None,
                        dv=None, dtable=None):
    """dQ, dK, dV, dtable (bf16, like the table) of sum(O * dout)."""
    sh = _shape(q, M, s)
    device, shape = _check_relbias(q, k, v, table, M, buckets), q.shape
    for name, t in (("o", o), ("dout", dout), ("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None:
            _need(name, t, torch.bfloat16, shape, device)
    _need("lse", lse, torch.float32, shape[:4], device)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(q) if dk is None else dk
    dv = torch.empty_like(q) if dv is None else dv
    if dtable is None:
        dtable = torch.empty_like(table)
    else:
        _need("dtable", dtable, torch.bfloat16, table.shape, device)
    ws = _workspace(_lib.fs_winattn_relbias_bwd_workspace_bytes(sh) if workspace is None else 0, workspace, device)
    with _on(device) as stream:
        _lib.fs_winattn_relbias_bwd(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), dout.data_ptr(),
                                    lse.data_ptr(), table.data_ptr(), _ptr(buckets), table.shape[1], dq.data_ptr(),
                                    dk.data_ptr(), dv.data_ptr(), dtable.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    return dq, dk, dv, dtable


class WindowAttentionRelativeBias(torch.autograd.Function):
    """Autograd wrapper of the relative-position-bias attention (forward and backward in libfswin.so)."""

    @staticmethod
    def forward(ctx, q, k, v, table, M: int, s: int, buckets=None):
        o, lse = winattn_relbias_fwd(q, k, v, table, M, s, buckets=buckets)
        ctx.save_for_backward(q, k, v, o, lse, table, *(() if buckets is None else (buckets,)))
        ctx.M, ctx.s = M, s
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, table, *rest = ctx.saved_tensors
        dq, dk, dv, dtable = winattn_relbias_bwd(q, k, v, o, dout.contiguous(), lse, table, ctx.M, ctx.s,
                                                 buckets=rest[0] if rest else None)
        return dq, dk, dv, dtable, None, None, None


def window_attention_relbias(q, k, v, table, M: int, s: int, buckets=None):
    """Autograd windowed attention with a learned relative position bias by buckets."""
    return WindowAttentionRelativeBias.apply(q, k, v, table, M, s, buckets)


# --------------------------------------------------------- residual step and norms
# What stands between the blocks of a Swin layer: the branch's post norm, dropout,
# layer scale and gate, the residual sum, and the next block's pre norm, in one pass
# over the rows.
_NORMS = {None: 0, "layer": 1, "rms": 2}
_STEP_PARAMS = ("gate", "scale", "post_weight", "post_bias", "pre_weight", "pre_bias")
ResidualNormGrads = namedtuple("ResidualNormGrads", ("dx", "df") + tuple("d" + n for n in _STEP_PARAMS))


def _resnorm_shape(stream, f, params, pre, post, eps: float, p: float, rng):
    """(shape, device) of a residual step whose arguments pass the checks; `stream`: x, or r in the backward; params in
    the order of _STEP_PARAMS."""
    if pre not in _NORMS or post not in _NORMS:
        raise ValueError("pre and post must be None, 'layer' or 'rms'")
    shape, dtype = stream.shape, stream.dtype
    if len(shape) < 2:
        raise ValueError("expected a [samples, ..., channels] tensor")
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError(f"the residual stream must be bfloat16 or float32, got {dtype}")
    B, C = shape[0], shape[-1]
    device = _device_of("x", stream)
    _need("x", stream, dtype, shape, device)
    _need("f", f, torch.bfloat16, shape, device)
    for name, t in zip(_STEP_PARAMS, params):
        if t is not None:
            _need(name, t, dtype, (B,) if name == "gate" else (C,), device)
    for kind, which, w, b in ((post, "post", params[2], params[3]), (pre, "pre", params[4], params[5])):
        if kind is None and (w is not None or b is not None):
            raise ValueError(f"{which}_weight and {which}_bias need {which}='layer' or 'rms'")
    if not 0.0 <= p < 1.0:
        raise ValueError("p must lie in [0, 1)")
    if p > 0.0:
        if rng is None:
            raise ValueError("dropout needs rng, an int64 tensor (seed, offset)")
        _need("rng", rng, torch.int64, (2,), device)
    tokens = stream.numel() // (B * C) if B and C else 0
    return _lib.ResnormShape(B, tokens, C, dtype is torch.float32, _NORMS[pre], _NORMS[post], eps, p), device


def residual_norm_fwd(x, f, gate=None, scale=None, post=None, post_weight=None, post_bias=None, pre="layer",
                      pre_weight=None, pre_bias=None, eps: float = 1e-5, p: float = 0.0, rng=None, r=None, n=None):
    """r = x + gate[b] * scale * dropout(post(f)), n = pre(r) (None without pre).

    x: the residual stream [B, ..., C], bf16 or fp32; f: a block's output, bf16.  gate: one value a sample (stochastic
    depth or learned; a zero gate takes nothing from f); scale: one a channel (layer scale); post, pre: None, "layer"
    or "rms", with weight and bias or without.  Parameters are of x's type, n is bf16.  p: dropout probability, drawn
    from rng, an int64 CUDA tensor (seed, offset) that the kernel reads when it runs; advance the offset between
    steps.  r may be x and n may be f, to work in place."""
    params = (gate, scale, post_weight, post_bias, pre_weight, pre_bias)
    sh, device = _resnorm_shape(x, f, params, pre, post, eps, p, rng)
    if r is None:
        r = torch.empty_like(x)
    else:
        _need("r", r, x.dtype, x.shape, device)
    if pre is None:
        n = None
    elif n is None:
        n = torch.empty_like(f)
    else:
        _need("n", n, torch.bfloat16, x.shape, device)
    with _on(device) as stream:
        _lib.fs_resnorm_fwd(sh, x.data_ptr(), f.data_ptr(), *map(_ptr, params), _ptr(rng) if p > 0.0 else 0,
                            r.data_ptr(), _ptr(n), stream)
    return r, n


def residual_norm_bwd(dr, dn, r, f, gate=None, scale=None, post=None, post_weight=None, post_bias=None, pre="layer",
                      pre_weight=None, pre_bias=None, eps: float = 1e-5, p: float = 0.0, rng=None, workspace=None,
                      skip=()):
    """Gradients of sum(r * dr) + sum(n * dn) as ResidualNormGrads; None for an absent parameter and for the names in
    `skip` ("gate", "scale", ...).  dr or dn may be None (zero); r is the forward's, rng as the forward read it."""
    params = (gate, scale, post_weight, post_bias, pre_weight, pre_bias)
    sh, device = _resnorm_shape(r, f, params, pre, post, eps, p, rng)
    if dr is not None:
        _need("dr", dr, r.dtype, r.shape, device)
    if dn is not None:
        if pre is None:
            raise ValueError("dn without a pre norm")
        _need("dn", dn, torch.bfloat16, r.shape, device)
    ws = _workspace(_lib.fs_resnorm_bwd_workspace_bytes(sh) if workspace is None else 0, workspace, device)
    out = [None if t is None or name in skip else torch.empty_like(t) for name, t in zip(_STEP_PARAMS, params)]
    dx, df = torch.empty_like(r), torch.empty_like(f)
    with _on(device) as stream:
        _lib.fs_resnorm_bwd(sh, _ptr(dr), _ptr(dn), r.data_ptr(), f.data_ptr(), *map(_ptr, params),
                            _ptr(rng) if p > 0.0 else 0, dx.data_ptr(), df.data_ptr(), *map(_ptr, out), ws.data_ptr(),
                            ws.numel(), stream)
    return ResidualNormGrads(dx, df, *out)


class ResidualNorm(torch.autograd.Function):
    """Autograd wrapper of the residual step (forward and backward in libfswin.so)."""

    @staticmethod
    def forward(ctx, x, f, gate, scale, post_weight, post_bias, pre_weight, pre_bias, rng, pre, post, eps, p):
        params = (gate, scale, post_weight, post_bias, pre_weight, pre_bias)
        if p > 0.0:
            rng = rng.clone()  # the caller may advance its own before the backward
        kw = dict(zip(_STEP_PARAMS, params), pre=pre, post=post, eps=eps, p=p, rng=rng)
        r, n = residual_norm_fwd(x, f, **kw)
        ctx.set_materialize_grads(False)
        tensors = params + (rng if p > 0.0 else None,)
        ctx.present = [t is not None for t in tensors]
        ctx.save_for_backward(r, f, *(t for t in tensors if t is not None))
        ctx.options = dict(pre=pre, post=post, eps=eps, p=p)
        return r, n

    @staticmethod
    @once_differentiable
    def backward(ctx, dr, dn):
        if dr is None and dn is None:
            return (None,) * 13
        r, f, *rest = ctx.saved_tensors
        tensors = [rest.pop(0) if there else None for there in ctx.present]
        needs = dict(zip(_STEP_PARAMS, ctx.needs_input_grad[2:8]))
        g = residual_norm_bwd(None if dr is None else dr.contiguous(), None if dn is None else dn.contiguous(), r, f,
                              **dict(zip(_STEP_PARAMS, tensors)), rng=tensors[-1], **ctx.options,
                              skip=[name for name, wanted in needs.items() if not wanted])
        return (*g, None, None, None, None, None)


def residual_norm(x, f, gate=None, scale=None, post=None, post_weight=None, post_bias=None, pre="layer",
                  pre_weight=None, pre_bias=None, eps: float = 1e-5, p: float = 0.0, rng=None):
    """Autograd residual step; arguments and results as residual_norm_fwd."""
    return ResidualNorm.apply(x, f, gate, scale, post_weight, post_bias, pre_weight, pre_bias, rng, pre, post, eps, p)


# ------------------------------------------------------------- gated feed-forward
_ACTS = {"silu": 0, "gelu": 1}
_MLP_PARAMS = ("w_gate", "w_up", "w_down", "b_gate", "b_up", "b_down")
GatedMlpGrads = namedtuple("GatedMlpGrads", ("dx",) + tuple("d" + n for n in _MLP_PARAMS))


def _mlp_shape(x, w_gate, w_up, w_down, b_gate, b_up, b_down, act: str):
    """(shape, device) of a gated feed-forward block whose arguments pass the checks."""
    if act not in _ACTS:
        raise ValueError("act must be 'silu' or 'gelu'")
    if x.dim() < 1 or w_gate.dim() != 2:
        raise ValueError("expected x [..., channels] and w_gate [hidden, channels]")
    C, F = x.shape[-1], w_gate.shape[0]
    device = _device_of("x", x)
    for name, t, shape in (("x", x, x.shape), ("w_gate", w_gate, (F, C)), ("w_up", w_up, (F, C)),
                           ("w_down", w_down, (C, F)), ("b_gate", b_gate, (F,)), ("b_up", b_up, (F,)),
                           ("b_down", b_down, (C,))):
        if t is not None:
            _need(name, t, torch.bfloat16, shape, device)
    return _lib.MlpShape(x.numel() // C if C else 0, C, F, _ACTS[act]), device


def gated_mlp_fwd(x, w_gate, w_up, w_down, b_gate=None, b_up=None, b_down=None, act: str = "silu", y=None,
                  workspace=None):
    """y = (act(x w_gate^T + b_gate) * (x w_up^T + b_up)) w_down^T + b_down, all bf16.

    x [..., C]; w_gate, w_up [F, C]; w_down [C, F]; C and F multiples of 8; act "silu" or "gelu"."""
    sh, device = _mlp_shape(x, w_gate, w_up, w_down, b_gate, b_up, b_down, act)
    if y is None:
        y = torch.empty_like(x)
    else:
        _need("y", y, torch.bfloat16, x.shape, device)
    ws = _workspace(_lib.fs_gated_mlp_fwd_workspace_bytes(sh) if workspace is None else 0, workspace, device)
    with _on(device) as stream:
        _lib.fs_gated_mlp_fwd(sh, x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), _ptr(b_gate),
                              _ptr(b_up), _ptr(b_down), y.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    return y


def gated_mlp_bwd(dy, x, w_gate, w_up, w_down, b_gate=None, b_up=None, b_down=None, act: str = "silu", workspace=None):
    """Gradients of sum(y * dy) as GatedMlpGrads, None for absent biases."""
    sh, device = _mlp_shape(x, w_gate, w_up, w_down, b_gate, b_up, b_down, act)
    _need("dy", dy, torch.bfloat16, x.shape, device)
    out = [None if t is None else torch.empty_like(t) for t in (x, w_gate, w_up, w_down, b_gate, b_up, b_down)]
    ws = _workspace(_lib.fs_gated_mlp_bwd_workspace_bytes(sh) if workspace is None else 0, workspace, device)
    with _on(device) as stream:
        _lib.fs_gated_mlp_bwd(sh, dy.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
                              _ptr(b_gate), _ptr(b_up), *map(_ptr, out), ws.data_ptr(), ws.numel(), stream)
    return GatedMlpGrads(*out)


class GatedMlp(torch.autograd.Function):
    """Autograd wrapper of the gated feed-forward block (forward and backward in libfswin.so)."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, b_gate, b_up, b_down, act):
        params = (w_gate, w_up, w_down, b_gate, b_up, b_down)
        ctx.present = [t is not None for t in params]
        ctx.save_for_backward(x, *(t for t in params if t is not None))
        ctx.act = act
        return gated_mlp_fwd(x, *params, act=act)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, *rest = ctx.saved_tensors
        params = [rest.pop(0) if there else None for there in ctx.present]
        return (*gated_mlp_bwd(dy.contiguous(), x, *params, act=ctx.act), None)


def gated_mlp(x, w_gate, w_up, w_down, b_gate=None, b_up=None, b_down=None, act: str = "silu"):
    """Autograd gated feed-forward block; arguments as gated_mlp_fwd."""
    return GatedMlp.apply(x, w_gate, w_up, w_down, b_gate, b_up, b_down, act)

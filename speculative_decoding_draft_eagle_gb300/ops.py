"""Python binding of the C ABI, with the same names: argument marshalling only.

Every computation runs in the CUDA library; torch supplies device memory,
streams and output allocation.  Functions take torch CUDA tensors and enqueue
on the current torch stream (or ``stream=``).
"""

from __future__ import annotations

import ctypes
import math
from typing import List, Optional, Sequence, Tuple

import torch

from ._lib import Logits, Pages, Rope, check, lib

__all__ = [
    "stt_attn_fwd",
    "stt_attn_bwd",
    "stt_attn_bwd_workspace_size",
    "stt_attn_bwd_ex",
    "stt_attn_bwd_ex_workspace_size",
    "soft_ce_fwd_bwd_inplace",
    "soft_ce_fwd_bwd_inplace_ex",
    "soft_ce_fwd_bwd_inplace_noalloc",
    "soft_ce_workspace_size",
    "stt_verify",
    "stt_lm_head_ce",
    "rope_frequencies",
    "stt_qkv_rope_fwd",
    "stt_qkv_rope_bwd",
    "stt_qkv_rope_bwd_workspace_size",
    "stt_kv_append",
    "stt_paged_attn",
    "stt_paged_attn_workspace_size",
    "stt_logits_process",
    "stt_device_error",
    "stt_debug_set_wait_budget",
    "stt_debug_inject",
    "stt_version",
]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr_array(ts: Sequence[torch.Tensor]):
    arr = (ctypes.c_void_p * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = t.data_ptr()
    return arr


def _attn_dims(q, k_blocks, v_blocks, T):
    if q.dim() != 4:
        raise ValueError("q must be [B, H, Q_LEN, D]")
    B, H, Q_LEN, D = q.shape
    if len(k_blocks) == 0 or len(k_blocks) != len(v_blocks):
        raise ValueError("k_blocks and v_blocks must both hold k+1 tensors")
    H_kv = k_blocks[0].shape[1]
    _need(q, "q", torch.bfloat16)
    for j, (kb, vb) in enumerate(zip(k_blocks, v_blocks)):
        _need(kb, f"k_blocks[{j}]", torch.bfloat16, (B, H_kv, Q_LEN, D))
        _need(vb, f"v_blocks[{j}]", torch.bfloat16, (B, H_kv, Q_LEN, D))
    Tl = [int(x) for x in (T.tolist() if isinstance(T, torch.Tensor) else T)]
    if len(Tl) != B:
        raise ValueError("T must hold B values")
    T_arr = (ctypes.c_int32 * B)(*Tl)
    return B, H, H_kv, D, Q_LEN, len(k_blocks) - 1, T_arr


def stt_attn_fwd(q: torch.Tensor, k_blocks: Sequence[torch.Tensor],
                 v_blocks: Sequence[torch.Tensor], T, scale: Optional[float] = None,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sparse-tree TTT attention forward at step k = len(k_blocks) - 1.

    Returns (out bf16 [B,H,Q_LEN,D], lse fp32 [B,H,Q_LEN])."""
    B, H, H_kv, D, Q_LEN, k, T_arr = _attn_dims(q, k_blocks, v_blocks, T)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Q_LEN), device=q.device, dtype=torch.float32)
    _need(out, "out", torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, Q_LEN))
    ka, va = _ptr_array(k_blocks), _ptr_array(v_blocks)
    st = lib().stt_attn_fwd(_ptr(q), ka, va, T_arr, B, H, H_kv, D, Q_LEN, k, scale, _ptr(out),
                            _ptr(lse), _stream(stream))
    check("stt_attn_fwd", st)
    return out, lse


def stt_attn_bwd_workspace_size(B, H, H_kv, D, Q_LEN, k) -> int:
    return int(lib().stt_attn_bwd_workspace_size(B, H, H_kv, D, Q_LEN, k))


def stt_attn_bwd(q: torch.Tensor, k_blocks: Sequence[torch.Tensor],
                 v_blocks: Sequence[torch.Tensor], T, out: torch.Tensor, dout: torch.Tensor,
                 lse: torch.Tensor, scale: Optional[float] = None,
                 dq: Optional[torch.Tensor] = None, dk_blocks: Optional[List[torch.Tensor]] = None,
                 dv_blocks: Optional[List[torch.Tensor]] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Backward of stt_attn_fwd.  Returns (dq, dk_blocks, dv_blocks), all fp32."""
    B, H, H_kv, D, Q_LEN, k, T_arr = _attn_dims(q, k_blocks, v_blocks, T)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _need(out, "out", torch.bfloat16, q.shape)
    _need(dout, "dout", torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, Q_LEN))
    dev = q.device
    if dq is None:
        dq = torch.empty(q.shape, device=dev, dtype=torch.float32)
    kv_shape = (B, H_kv, Q_LEN, D)
    if dk_blocks is None:
        dk_blocks = [torch.empty(kv_shape, device=dev, dtype=torch.float32) for _ in range(k + 1)]
    if dv_blocks is None:
        dv_blocks = [torch.empty(kv_shape, device=dev, dtype=torch.float32) for _ in range(k + 1)]
    _need(dq, "dq", torch.float32, q.shape)
    for j in range(k + 1):
        _need(dk_blocks[j], f"dk_blocks[{j}]", torch.float32, kv_shape)
        _need(dv_blocks[j], f"dv_blocks[{j}]", torch.float32, kv_shape)
    need = stt_attn_bwd_workspace_size(B, H, H_kv, D, Q_LEN, k)
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    st = lib().stt_attn_bwd(_ptr(q), _ptr_array(k_blocks), _ptr_array(v_blocks), T_arr, B, H,
                            H_kv, D, Q_LEN, k, scale, _ptr(out), _ptr(dout), _ptr(lse), _ptr(dq),
                            _ptr_array(dk_blocks), _ptr_array(dv_blocks), _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream(stream))
    check("stt_attn_bwd", st)
    return dq, dk_blocks, dv_blocks


STT_BWD_ACCUMULATE_KV = 0x1
STT_BWD_BF16_GRADS = 0x2


def stt_attn_bwd_ex_workspace_size(B, H, H_kv, D, Q_LEN, k, flags) -> int:
    return int(lib().stt_attn_bwd_ex_workspace_size(B, H, H_kv, D, Q_LEN, k, flags))


def stt_attn_bwd_ex(q: torch.Tensor, k_blocks: Sequence[torch.Tensor],
                    v_blocks: Sequence[torch.Tensor], T, out: torch.Tensor, dout: torch.Tensor,
                    lse: torch.Tensor, dq: torch.Tensor, dk_blocks: Sequence[torch.Tensor],
                    dv_blocks: Sequence[torch.Tensor], scale: Optional[float] = None,
                    accumulate: bool = False, workspace: Optional[torch.Tensor] = None,
                    stream=None):
    """Backward of stt_attn_fwd into caller-given gradient buffers, all fp32 or all
    bf16 (the dtype of ``dq`` selects STT_BWD_BF16_GRADS).  With ``accumulate``
    the block gradients are added to dk_blocks / dv_blocks (STT_BWD_ACCUMULATE_KV);
    dq is always overwritten."""
    B, H, H_kv, D, Q_LEN, k, T_arr = _attn_dims(q, k_blocks, v_blocks, T)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _need(out, "out", torch.bfloat16, q.shape)
    _need(dout, "dout", torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (B, H, Q_LEN))
    gd = dq.dtype
    if gd not in (torch.float32, torch.bfloat16):
        raise ValueError("gradients must be float32 or bfloat16")
    _need(dq, "dq", gd, q.shape)
    if len(dk_blocks) != k + 1 or len(dv_blocks) != k + 1:
        raise ValueError("dk_blocks and dv_blocks must hold k+1 tensors")
    kv_shape = (B, H_kv, Q_LEN, D)
    for j in range(k + 1):
        _need(dk_blocks[j], f"dk_blocks[{j}]", gd, kv_shape)
        _need(dv_blocks[j], f"dv_blocks[{j}]", gd, kv_shape)
    flags = (STT_BWD_ACCUMULATE_KV if accumulate else 0) | (
        STT_BWD_BF16_GRADS if gd == torch.bfloat16 else 0)
    need = stt_attn_bwd_ex_workspace_size(B, H, H_kv, D, Q_LEN, k, flags)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, device=q.device, dtype=torch.uint8)
    st = lib().stt_attn_bwd_ex(_ptr(q), _ptr_array(k_blocks), _ptr_array(v_blocks), T_arr, B, H,
                               H_kv, D, Q_LEN, k, scale, _ptr(out), _ptr(dout), _ptr(lse),
                               _ptr(dq), _ptr_array(dk_blocks), _ptr_array(dv_blocks), flags,
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream(stream))
    check("stt_attn_bwd_ex", st)
    return dq, dk_blocks, dv_blocks


def soft_ce_workspace_size(N: int, V: int) -> int:
    return int(lib().soft_ce_workspace_size(N, V))


def soft_ce_fwd_bwd_inplace(z: torch.Tensor, p: torch.Tensor, g: torch.Tensor,
                            row_loss: Optional[torch.Tensor] = None,
                            loss: Optional[torch.Tensor] = None,
                            workspace: Optional[torch.Tensor] = None, want_row_loss: bool = True,
                            stream=None):
    """In-place soft-CE: z is overwritten with dL/dz.  Returns (loss [1], row_loss [N] or None)."""
    if z.dim() != 2:
        raise ValueError("z must be [N, V]")
    N, V = z.shape
    _need(z, "z", torch.float32)
    _need(p, "p", torch.float32, (N, V))
    _need(g, "g", torch.float32, (N,))
    dev = z.device
    if loss is None:
        loss = torch.empty(1, device=dev, dtype=torch.float32)
    _need(loss, "loss", torch.float32)
    if row_loss is None and want_row_loss:
        row_loss = torch.empty(N, device=dev, dtype=torch.float32)
    if row_loss is not None:
        _need(row_loss, "row_loss", torch.float32, (N,))
    need = soft_ce_workspace_size(N, V)
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    st = lib().soft_ce_fwd_bwd_inplace(_ptr(z), _ptr(p), _ptr(g), N, V, _ptr(row_loss),
                                       _ptr(loss), _ptr(workspace),
                                       workspace.numel() * workspace.element_size(),
                                       _stream(stream))
    check("soft_ce_fwd_bwd_inplace", st)
    return loss, row_loss


STT_CE_BF16 = 0x1
STT_CE_G_PER_ELEMENT = 0x2


def soft_ce_fwd_bwd_inplace_ex(z: torch.Tensor, p: torch.Tensor, g: torch.Tensor,
                               row_loss: Optional[torch.Tensor] = None,
                               loss: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None, stream=None):
    """In-place soft-CE in any of the admitted forms: z and p both fp32 or both
    bf16 (STT_CE_BF16), g fp32 of shape [N] (per row) or [N, V] (per element,
    STT_CE_G_PER_ELEMENT).  z is overwritten with dL/dz in its own dtype.
    Returns (loss [1], row_loss [N])."""
    if z.dim() != 2:
        raise ValueError("z must be [N, V]")
    N, V = z.shape
    if z.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("z must be float32 or bfloat16")
    _need(z, "z", z.dtype)
    _need(p, "p", z.dtype, (N, V))
    if g.dim() == 2:
        _need(g, "g", torch.float32, (N, V))
    else:
        _need(g, "g", torch.float32, (N,))
    flags = (STT_CE_BF16 if z.dtype == torch.bfloat16 else 0) | (
        STT_CE_G_PER_ELEMENT if g.dim() == 2 else 0)
    dev = z.device
    if loss is None:
        loss = torch.empty(1, device=dev, dtype=torch.float32)
    if row_loss is None:
        row_loss = torch.empty(N, device=dev, dtype=torch.float32)
    _need(loss, "loss", torch.float32)
    _need(row_loss, "row_loss", torch.float32, (N,))
    need = soft_ce_workspace_size(N, V)
    if workspace is None:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    st = lib().soft_ce_fwd_bwd_inplace_ex(_ptr(z), _ptr(p), _ptr(g), N, V, flags, _ptr(row_loss),
                                          _ptr(loss), _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(stream))
    check("soft_ce_fwd_bwd_inplace_ex", st)
    return loss, row_loss


def soft_ce_fwd_bwd_inplace_noalloc(z: torch.Tensor, p: torch.Tensor, g: torch.Tensor,
                                    row_loss: Optional[torch.Tensor] = None,
                                    loss: Optional[torch.Tensor] = None, stream=None):
    """Same as soft_ce_fwd_bwd_inplace but without a workspace: the library's own
    fixed scratch is used (at most 65536 rows), for callers that cannot allocate
    device memory.  Calls must not overlap on the GPU."""
    if z.dim() != 2:
        raise ValueError("z must be [N, V]")
    N, V = z.shape
    _need(z, "z", torch.float32)
    _need(p, "p", torch.float32, (N, V))
    _need(g, "g", torch.float32, (N,))
    if loss is None:
        loss = torch.empty(1, device=z.device, dtype=torch.float32)
    _need(loss, "loss", torch.float32)
    if row_loss is not None:
        _need(row_loss, "row_loss", torch.float32, (N,))
    st = lib().soft_ce_fwd_bwd_inplace_noalloc(_ptr(z), _ptr(p), _ptr(g), N, V, _ptr(row_loss),
                                               _ptr(loss), _stream(stream))
    check("soft_ce_fwd_bwd_inplace_noalloc", st)
    return loss, row_loss


STT_ERR_TIMEOUT = -5


def stt_lm_head_ce(h: torch.Tensor, W: torch.Tensor, p: torch.Tensor, g: torch.Tensor,
                   dh: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                   row_loss: Optional[torch.Tensor] = None, loss: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """Draft LM head z = h W^T fused with the soft-CE: loss and the fp32 gradients
    of h [N, Hd] and W [V, Hd] (both bf16), z never materialised.
    Returns (loss [1], row_loss [N], dh [N, Hd], dW [V, Hd])."""
    if h.dim() != 2 or W.dim() != 2:
        raise ValueError("h must be [N, Hd] and W [V, Hd]")
    N, Hd = h.shape
    V = W.shape[0]
    _need(h, "h", torch.bfloat16)
    _need(W, "W", torch.bfloat16, (V, Hd))
    _need(p, "p", torch.float32, (N, V))
    _need(g, "g", torch.float32, (N,))
    dev = h.device
    if dh is None:
        dh = torch.empty((N, Hd), device=dev, dtype=torch.float32)
    if dW is None:
        dW = torch.empty((V, Hd), device=dev, dtype=torch.float32)
    if row_loss is None:
        row_loss = torch.empty(N, device=dev, dtype=torch.float32)
    if loss is None:
        loss = torch.empty(1, device=dev, dtype=torch.float32)
    _need(dh, "dh", torch.float32, (N, Hd))
    _need(dW, "dW", torch.float32, (V, Hd))
    _need(row_loss, "row_loss", torch.float32, (N,))
    _need(loss, "loss", torch.float32)
    need = int(lib().stt_lm_head_ce_workspace_size(N, Hd, V))
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    st = lib().stt_lm_head_ce(_ptr(h), _ptr(W), _ptr(p), _ptr(g), N, Hd, V, _ptr(dh), _ptr(dW),
                              _ptr(row_loss), _ptr(loss), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    check("stt_lm_head_ce", st)
    return loss, row_loss, dh, dW


def stt_verify(p_target: torch.Tensor, p_draft: torch.Tensor, draft_tokens: torch.Tensor,
               u_accept: torch.Tensor, u_sample: torch.Tensor,
               n_accepted: Optional[torch.Tensor] = None,
               out_tokens: Optional[torch.Tensor] = None, stream=None):
    """Rejection-sampling verification of draft tokens.  p_target, p_draft fp32
    [B, gamma, V]; draft_tokens int32 [B, gamma]; u_accept fp32 [B, gamma];
    u_sample fp32 [B].  Returns (n_accepted int32 [B], out_tokens int32 [B, gamma])."""
    if p_target.dim() != 3:
        raise ValueError("p_target must be [B, gamma, V]")
    B, gamma, V = p_target.shape
    _need(p_target, "p_target", torch.float32)
    _need(p_draft, "p_draft", torch.float32, (B, gamma, V))
    _need(draft_tokens, "draft_tokens", torch.int32, (B, gamma))
    _need(u_accept, "u_accept", torch.float32, (B, gamma))
    _need(u_sample, "u_sample", torch.float32, (B,))
    dev = p_target.device
    if n_accepted is None:
        n_accepted = torch.empty(B, device=dev, dtype=torch.int32)
    if out_tokens is None:
        out_tokens = torch.empty((B, gamma), device=dev, dtype=torch.int32)
    _need(n_accepted, "n_accepted", torch.int32, (B,))
    _need(out_tokens, "out_tokens", torch.int32, (B, gamma))
    st = lib().stt_verify(_ptr(p_target), _ptr(p_draft), _ptr(draft_tokens), _ptr(u_accept),
                          _ptr(u_sample), B, gamma, V, _ptr(n_accepted), _ptr(out_tokens),
                          _stream(stream))
    check("stt_verify", st)
    return n_accepted, out_tokens


def _check_devices(*ts: Optional[torch.Tensor]):
    """The library launches on the current device: every tensor must live there."""
    dev = torch.cuda.current_device()
    for t in ts:
        if t is not None and t.device.index != dev:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{dev}")


def _own(stream, *ts: Optional[torch.Tensor]):
    """Tensors allocated here (on the current stream) and used on `stream`: their
    memory is not handed out again before that stream is done with them."""
    if stream is None:
        return
    if not isinstance(stream, torch.cuda.Stream):
        if int(stream) == 0:
            stream = torch.cuda.default_stream()
        else:
            stream = torch.cuda.ExternalStream(int(stream))
    for t in ts:
        if t is not None:
            t.record_stream(stream)


def _need_rows(t: torch.Tensor, name: str, width: int, dims: int):
    """bf16 rows `width` wide, dense but for the distance between rows; returns it."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != dims or t.shape[-1] != width:
        raise ValueError(f"{name} must have {dims} dimensions, the last of size {width}, "
                         f"got {tuple(t.shape)}")
    ld = width
    if t.shape[-2] > 1:
        ld = t.stride(-2)
    elif dims == 3 and t.shape[0] > 1:
        ld = t.stride(0)
    if t.numel() and ((width > 1 and t.stride(-1) != 1) or ld < width or
                      (dims == 3 and t.shape[0] > 1 and t.stride(0) != t.shape[1] * ld)):
        raise ValueError(f"{name} must be dense apart from the distance between its rows")
    return ld


def rope_frequencies(R: int, base: float = 10000.0, factor: float = 1.0,
                     original_positions: Optional[int] = None, slow_turns: float = 1.0,
                     fast_turns: float = 32.0, device="cuda") -> torch.Tensor:
    """Rotation frequencies base^(-2i/R), i = 0..R/2-1, in radians per position (fp64).

    With `factor` > 1 the positions are stretched for contexts longer than the
    `original_positions` trained on: a pair that makes at most `slow_turns` turns
    over them is slowed by `factor`, one that makes at least `fast_turns` keeps its
    frequency, and those between are blended linearly in their number of turns.
    Without `original_positions` every pair is slowed (position interpolation)."""
    if R < 2 or R % 2:
        raise ValueError("R must be even and positive")
    if not base > 0 or not factor > 0:
        raise ValueError("base and factor must be positive")
    f = float(base) ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    keep = torch.zeros_like(f)
    if original_positions is not None:
        if not fast_turns > slow_turns:
            raise ValueError("fast_turns must be greater than slow_turns")
        turns = original_positions * f / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
    return (f * keep + f / factor * (1 - keep)).to(device)


def _rope(freq, w_q, w_k, D, eps, interleaved, amplitude) -> Rope:
    R = 0
    if freq is not None:
        if freq.dim() != 1:
            raise ValueError("freq must be [R/2]")
        _need(freq, "freq", torch.float64)
        R = 2 * freq.numel()
    for name, w in (("w_q", w_q), ("w_k", w_k)):
        if w is not None:
            _need(w, name, torch.bfloat16, (D,))
    return Rope(freq=_ptr(freq) if R else None, w_q=_ptr(w_q), w_k=_ptr(w_k), R=R,
                flags=STT_ROPE_INTERLEAVED if interleaved else 0, amplitude=float(amplitude),
                eps=float(eps))


STT_ROPE_INTERLEAVED = 0x1
STT_ROPE_BF16_GRADS = 0x2


def stt_qkv_rope_fwd(qkv: torch.Tensor, H: int, H_kv: int, D: int,
                     positions: Optional[torch.Tensor] = None,
                     freq: Optional[torch.Tensor] = None, w_q: Optional[torch.Tensor] = None,
                     w_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     interleaved: bool = False, amplitude: float = 1.0,
                     q: Optional[torch.Tensor] = None, k: Optional[torch.Tensor] = None,
                     v: Optional[torch.Tensor] = None, stream=None):
    """Projection rows qkv bf16 [B, S, (H + 2 H_kv) D] (rows may be a slice of wider
    ones) to the attention's q [B, H, S, D], k and v [B, H_kv, S, D]: RMS norm of
    every query and key head with the weights w_q, w_k bf16 [D] (None: no norm), and
    rotation of each head's first 2 len(freq) elements by positions int32 [B, S]
    (None: 0..S-1) times freq (fp64 radians per position, see rope_frequencies)."""
    ld = _need_rows(qkv, "qkv", (H + 2 * H_kv) * D, 3)
    B, S = qkv.shape[:2]
    rope = _rope(freq, w_q, w_k, D, eps, interleaved, amplitude)
    if positions is not None:
        _need(positions, "positions", torch.int32, (B, S))
    fresh = []
    outs = []
    for name, t, h in (("q", q, H), ("k", k, H_kv), ("v", v, H_kv)):
        if t is None:
            t = torch.empty((B, h, S, D), device=qkv.device, dtype=torch.bfloat16)
            fresh.append(t)
        _need(t, name, torch.bfloat16, (B, h, S, D))
        outs.append(t)
    _check_devices(qkv, positions, freq, w_q, w_k, *outs)
    st = lib().stt_qkv_rope_fwd(_ptr(qkv), ld, _ptr(positions), B, S, H, H_kv, D,
                                ctypes.byref(rope), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]),
                                _stream(stream))
    check("stt_qkv_rope_fwd", st)
    _own(stream, *fresh)
    return tuple(outs)


def stt_qkv_rope_bwd_workspace_size(D: int) -> int:
    return int(lib().stt_qkv_rope_bwd_workspace_size(D))


def stt_qkv_rope_bwd(dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor,
                     qkv: Optional[torch.Tensor] = None,
                     positions: Optional[torch.Tensor] = None,
                     freq: Optional[torch.Tensor] = None, w_q: Optional[torch.Tensor] = None,
                     w_k: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     interleaved: bool = False, amplitude: float = 1.0,
                     dqkv: Optional[torch.Tensor] = None, dw_q: Optional[torch.Tensor] = None,
                     dw_k: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradient of stt_qkv_rope_fwd from dq, dk, dv (all fp32 or all bf16, in the
    layout of q, k, v).  qkv is needed where a weight is given.  Returns (dqkv bf16
    [B, S, (H + 2 H_kv) D], dw_q, dw_k fp32 [D] or None)."""
    if dq.dim() != 4 or dk.dim() != 4:
        raise ValueError("dq must be [B, H, S, D] and dk, dv [B, H_kv, S, D]")
    B, H, S, D = dq.shape
    H_kv = dk.shape[1]
    if dq.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("dq must be float32 or bfloat16")
    _need(dq, "dq", dq.dtype)
    _need(dk, "dk", dq.dtype, (B, H_kv, S, D))
    _need(dv, "dv", dq.dtype, (B, H_kv, S, D))
    C = (H + 2 * H_kv) * D
    rope = _rope(freq, w_q, w_k, D, eps, interleaved, amplitude)
    norm = w_q is not None or w_k is not None
    ld = C
    if qkv is not None:
        ld = _need_rows(qkv, "qkv", C, 3)
        if tuple(qkv.shape[:2]) != (B, S):
            raise ValueError(f"qkv must have shape {(B, S, C)}, got {tuple(qkv.shape)}")
    elif norm:
        raise ValueError("qkv is needed for the gradient of the norm")
    if positions is not None:
        _need(positions, "positions", torch.int32, (B, S))
    fresh = []

    def out(t, name, shape, dtype):
        if t is None:
            t = torch.empty(shape, device=dq.device, dtype=dtype)
            fresh.append(t)
        return t

    dqkv = out(dqkv, "dqkv", (B, S, C), torch.bfloat16)
    ld_d = _need_rows(dqkv, "dqkv", C, 3)
    if tuple(dqkv.shape[:2]) != (B, S):
        raise ValueError(f"dqkv must have shape {(B, S, C)}, got {tuple(dqkv.shape)}")
    if (dw_q is not None and w_q is None) or (dw_k is not None and w_k is None):
        raise ValueError("a weight's gradient is asked for without the weight")
    if w_q is not None:
        dw_q = out(dw_q, "dw_q", (D,), torch.float32)
        _need(dw_q, "dw_q", torch.float32, (D,))
    if w_k is not None:
        dw_k = out(dw_k, "dw_k", (D,), torch.float32)
        _need(dw_k, "dw_k", torch.float32, (D,))
    if norm and workspace is None:
        workspace = out(None, "workspace", (stt_qkv_rope_bwd_workspace_size(D),), torch.uint8)
    _check_devices(dq, dk, dv, qkv, positions, freq, w_q, w_k, dqkv, dw_q, dw_k, workspace)
    st = lib().stt_qkv_rope_bwd(
        _ptr(dq), _ptr(dk), _ptr(dv), _ptr(qkv) if norm else None, ld, _ptr(positions), B, S, H,
        H_kv, D, ctypes.byref(rope), STT_ROPE_BF16_GRADS if dq.dtype == torch.bfloat16 else 0,
        _ptr(dqkv), ld_d, _ptr(dw_q), _ptr(dw_k), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream))
    check("stt_qkv_rope_bwd", st)
    _own(stream, *fresh)
    return dqkv, dw_q, dw_k


def _pages(k_cache, v_cache, cu_q, seq_lens, page_table) -> Pages:
    for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
        if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16 or t.dim() != 4:
            raise ValueError(f"{name} must be bfloat16 [num_pages, H_kv, page_size, D]")
        if t.numel() and t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError(f"{name}: the elements of a head must be contiguous")
    if v_cache.shape != k_cache.shape or v_cache.stride() != k_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, max_pages]")
    B, max_pages = page_table.shape
    _need(page_table, "page_table", torch.int32)
    _need(cu_q, "cu_q", torch.int32, (B + 1,))
    _need(seq_lens, "seq_lens", torch.int32, (B,))
    n, H_kv, page, D = k_cache.shape
    # A dimension of one element has no stride of its own.
    stride = [s if size > 1 else max(8, (D + 7) // 8 * 8)
              for s, size in zip(k_cache.stride(), k_cache.shape)]
    return Pages(k=_ptr(k_cache), v=_ptr(v_cache), table=_ptr(page_table), cu_q=_ptr(cu_q),
                 seq_lens=_ptr(seq_lens), stride_page=stride[0], stride_head=stride[1],
                 stride_tok=stride[2], B=B, H_kv=H_kv, D=D, page_size=page, num_pages=n,
                 max_pages=max_pages)


def stt_kv_append(qkv: torch.Tensor, H: int, k_cache: torch.Tensor, v_cache: torch.Tensor,
                  cu_q: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                  positions: Optional[torch.Tensor] = None, freq: Optional[torch.Tensor] = None,
                  w_q: Optional[torch.Tensor] = None, w_k: Optional[torch.Tensor] = None,
                  eps: float = 1e-6, interleaved: bool = False, amplitude: float = 1.0,
                  q: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """New tokens into a paged cache.  qkv bf16 [N, (H + 2 H_kv) D]: the projection's
    rows, sequence b's being cu_q[b]..cu_q[b+1]-1 (int32 [B + 1]); its n rows become
    keys seq_lens[b] - n.. of it (int32 [B], new keys among them) in the pages
    page_table[b] (int32 [B, max_pages]).  Caches bf16 [num_pages, H_kv, page_size, D],
    any strides with contiguous heads (a [pages, page_size, H_kv, D] cache passes as
    its transpose).  Norm and rotation as stt_qkv_rope_fwd, at positions int32 [N]
    (None: the key's index).  Returns the queries bf16 [N, H, D]; rows behind the
    last sequence are left as they are."""
    pages = _pages(k_cache, v_cache, cu_q, seq_lens, page_table)
    D = pages.D
    ld = _need_rows(qkv, "qkv", (H + 2 * pages.H_kv) * D, 2)
    N = qkv.shape[0]
    rope = _rope(freq, w_q, w_k, D, eps, interleaved, amplitude)
    if positions is not None:
        _need(positions, "positions", torch.int32, (N,))
    fresh = None
    if q is None:
        q = fresh = torch.empty((N, H, D), device=qkv.device, dtype=torch.bfloat16)
    _need(q, "q", torch.bfloat16, (N, H, D))
    _check_devices(qkv, k_cache, v_cache, cu_q, seq_lens, page_table, positions, freq, w_q, w_k, q)
    st = lib().stt_kv_append(_ptr(qkv), ld, _ptr(positions), N, H, ctypes.byref(pages),
                             ctypes.byref(rope), _ptr(q), _stream(stream))
    check("stt_kv_append", st)
    _own(stream, fresh)
    return q


def stt_paged_attn_workspace_size(N: int, B: int, H: int, H_kv: int, D: int) -> int:
    return int(lib().stt_paged_attn_workspace_size(N, B, H, H_kv, D))


def stt_paged_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   cu_q: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor,
                   scale: Optional[float] = None, tree_mask: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None
                   ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Attention of a ragged batch of new tokens over their sequences' pages (batch
    and caches as stt_kv_append, whose keys are already in the cache).  q bf16
    [N, H, D], rows possibly a slice of wider ones.  New token i of n sees the keys
    up to its own, or with tree_mask (int32 [N, words]) every key before the new ones
    and new token j iff bit j % 32 of word j / 32 of its row is set.
    Returns (out bf16 [N, H, D], lse fp32 [N, H]); rows behind the last sequence are
    left as they are."""
    pages = _pages(k_cache, v_cache, cu_q, seq_lens, page_table)
    if q.dim() != 3 or q.shape[2] != pages.D:
        raise ValueError(f"q must be [N, H, {pages.D}]")
    N, H, D = q.shape
    if q.numel() and H > 1 and q.stride(1) != D:
        raise ValueError("q must be dense apart from the distance between its rows")
    ld = _need_rows(q.flatten(1) if q.is_contiguous() else
                    q.as_strided((N, H * D), (q.stride(0), q.stride(2))), "q", H * D, 2)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    words = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2:
            raise ValueError("tree_mask must be [N, words]")
        words = tree_mask.shape[1]
        _need(tree_mask, "tree_mask", torch.int32, (N, words))
    fresh = []

    def new(shape, dtype):
        fresh.append(torch.empty(shape, device=q.device, dtype=dtype))
        return fresh[-1]

    if out is None:
        out = new((N, H, D), torch.bfloat16)
    if lse is None:
        lse = new((N, H), torch.float32)
    _need(out, "out", torch.bfloat16, (N, H, D))
    _need(lse, "lse", torch.float32, (N, H))
    if workspace is None:
        workspace = new((stt_paged_attn_workspace_size(N, pages.B, H, pages.H_kv, D),),
                        torch.uint8)
    _check_devices(q, k_cache, v_cache, cu_q, seq_lens, page_table, tree_mask, out, lse, workspace)
    st = lib().stt_paged_attn(_ptr(q), ld, N, H, ctypes.byref(pages), scale, _ptr(tree_mask),
                              words, _ptr(out), _ptr(lse), _ptr(workspace),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    check("stt_paged_attn", st)
    _own(stream, *fresh)
    return out, lse


STT_LOGITS_BF16 = 0x1
STT_LOGITS_RAW = 0x2


def stt_logits_process(z: torch.Tensor, rows: int = 1,
                       temperature: Optional[torch.Tensor] = None,
                       repetition: Optional[torch.Tensor] = None,
                       frequency: Optional[torch.Tensor] = None,
                       presence: Optional[torch.Tensor] = None,
                       tokens: Optional[torch.Tensor] = None,
                       cu_tokens: Optional[torch.Tensor] = None,
                       n_prompt: Optional[torch.Tensor] = None,
                       draft_tokens: Optional[torch.Tensor] = None,
                       bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                       raw: bool = False, out: Optional[torch.Tensor] = None, stream=None
                       ) -> torch.Tensor:
    """Logits z [N, V] (fp32 or bf16; `rows` consecutive draft positions for each of
    the B = N / rows sequences) to the distributions stt_verify tests against, fp32
    [N, V]: penalties over each row's history, bias, grammar mask, temperature (0:
    greedy), softmax; with `raw` the logits before the softmax.

    temperature, repetition, frequency, presence: fp32 [B].  tokens int32 [total],
    sequence b's being cu_tokens[b]..cu_tokens[b+1]-1 (int32 [B + 1]) with a prompt of
    n_prompt[b] (int32 [B]); position i's history also holds the first i of
    draft_tokens int32 [B, >= rows - 1].  bias fp32 [V], [1, V] or [B, V]; mask int32
    [N, ceil(V / 32)], bit v % 32 of word v / 32 set where v is allowed.  out may be z
    itself where that is fp32."""
    if z.dim() != 2:
        raise ValueError("z must be [N, V]")
    N, V = z.shape
    if z.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("z must be float32 or bfloat16")
    _need(z, "z", z.dtype)
    if rows < 1 or N % rows:
        raise ValueError("rows must be positive and divide N")
    B = N // rows
    for name, t in (("temperature", temperature), ("repetition", repetition),
                    ("frequency", frequency), ("presence", presence)):
        if t is not None:
            _need(t, name, torch.float32, (B,))
    if (tokens is None) != (cu_tokens is None):
        raise ValueError("tokens and cu_tokens go together")
    if tokens is not None:
        if tokens.dim() != 1:
            raise ValueError("tokens must be [total]")
        _need(tokens, "tokens", torch.int32)
        _need(cu_tokens, "cu_tokens", torch.int32, (B + 1,))
    if n_prompt is not None:
        if tokens is None:
            raise ValueError("n_prompt is given without tokens")
        _need(n_prompt, "n_prompt", torch.int32, (B,))
    draft_ld = 0
    if draft_tokens is not None:
        if draft_tokens.dim() != 2 or draft_tokens.shape[1] < rows - 1:
            raise ValueError(f"draft_tokens must be [B, at least {rows - 1}]")
        draft_ld = draft_tokens.shape[1]
        _need(draft_tokens, "draft_tokens", torch.int32, (B, draft_ld))
    bias_rows = 0
    if bias is not None:
        bias_rows = 1 if bias.dim() == 1 else bias.shape[0]
        if bias_rows not in (1, B):
            raise ValueError("bias must be [V], [1, V] or [B, V]")
        _need(bias, "bias", torch.float32, (V,) if bias.dim() == 1 else (bias_rows, V))
    if mask is not None:
        _need(mask, "mask", torch.int32, (N, (V + 31) // 32))
    fresh = None
    if out is None:
        out = fresh = torch.empty((N, V), device=z.device, dtype=torch.float32)
    _need(out, "out", torch.float32, (N, V))
    _check_devices(z, temperature, repetition, frequency, presence, tokens, cu_tokens, n_prompt,
                   draft_tokens, bias, mask, out)
    # An empty history has no address.
    has = tokens is not None and tokens.numel() > 0
    p = Logits(temperature=_ptr(temperature), repetition=_ptr(repetition),
               frequency=_ptr(frequency), presence=_ptr(presence),
               tokens=_ptr(tokens) if has else None, cu_tokens=_ptr(cu_tokens) if has else None,
               n_prompt=_ptr(n_prompt) if has else None,
               draft=_ptr(draft_tokens) if draft_ld else None, bias=_ptr(bias), mask=_ptr(mask),
               draft_ld=draft_ld, bias_rows=bias_rows)
    flags = (STT_LOGITS_BF16 if z.dtype == torch.bfloat16 else 0) | (STT_LOGITS_RAW if raw else 0)
    st = lib().stt_logits_process(_ptr(z), N, V, rows, ctypes.byref(p), flags, _ptr(out),
                                  _stream(stream))
    check("stt_logits_process", st)
    _own(stream, fresh)
    return out


def stt_device_error(stream=None) -> int:
    """Synchronises the stream, then reads and clears the device error word
    (0 when no bounded wait ran out).  STT_ERR_TIMEOUT is reported through
    the returned word's STT_DEVERR_*_WAIT bits, not raised."""
    w = ctypes.c_uint32(0)
    st = lib().stt_device_error(_stream(stream), ctypes.byref(w))
    if st != STT_ERR_TIMEOUT:
        check("stt_device_error", st)
    return int(w.value)


def stt_debug_set_wait_budget(ns: int) -> None:
    """Bounded-wait budget of every kernel on the current device (0: default)."""
    check("stt_debug_set_wait_budget", lib().stt_debug_set_wait_budget(int(ns)))


def stt_debug_inject(what: int) -> None:
    """Test hook: STT_INJECT_* bits (0 switches injection off)."""
    check("stt_debug_inject", lib().stt_debug_inject(int(what)))


def stt_version() -> int:
    return int(lib().stt_version())
